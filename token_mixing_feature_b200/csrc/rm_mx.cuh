// Block-scaled 8-bit values: e4m3 codes with one power-of-two scale (E8M0, a
// byte holding the exponent + 127; 255 = NaN) for each block of 128, and the
// sm_100a tensor-core instructions that read both (kind::mxf8f6f4).
#pragma once

#include <cuda_fp8.h>

#include "rm_device.cuh"

namespace rm {

constexpr int kBlk = 128;   // elements that share a scale along a row

// ------------------------------------------------------------------- scales
// |x| as an integer: ordered like the magnitudes, infinity and NaN on top, so
// one unsigned maximum finds both the largest magnitude and any NaN.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Scale byte of a block whose largest magnitude is `amax` (abs_bits): the
// smallest e in [-127, 127] with amax <= 448 * 2^e = 1.75 * 2^(e + 8), read off
// the exponent and mantissa fields; 127 (scale 1) for a zero block, 255 (NaN)
// for one with an infinity or a NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    // exponent field, plus one where the mantissa exceeds 1.75's, less 8
    const int b = max((int)((amax + 0x1fffffu) >> 23) - 8, 0);
    return amax >= 0x7f800000u ? 255u : amax == 0u ? 127u : (uint32_t)b;
}
// 2^-e of a scale byte as a float: a normal number for every finite block
// (byte <= 247), and NaN for byte 255, which makes the block's codes NaN.
__device__ __forceinline__ float scale_inverse(uint32_t byte) {
    return __uint_as_float(byte == 255u ? 0x7fffffffu : (254u - byte) << 23);
}

// Largest of magnitudes, NaN if any is.
__device__ __forceinline__ float max_abs(float m, float2 v) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(v.x)), "f"(fabsf(v.y)));
    return r;
}

// Four e4m3 codes, nearest even; |x * inv| <= 448 by the choice of the scale.
__device__ __forceinline__ uint32_t e4m3x4(float2 a, float2 b) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3) |
           ((uint32_t)__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3) << 16);
}

// The largest of each of NC values over LANES neighbouring lanes (16 or 32),
// all NC at once: as long as a lane holds several values it gives half of them
// away for the other lane's share of the rest.  Value i ends in the lanes whose
// number among the LANES, without its low SHIFT bits, is i.
template <int NC, int LANES>
struct BlockMax {
    static constexpr int LOGV = NC <= 1 ? 0 : NC <= 2 ? 1 : NC <= 4 ? 2 : 3, V = 1 << LOGV;
    static constexpr int SHIFT = (LANES == 32 ? 5 : 4) - LOGV;
    static __device__ __forceinline__ uint32_t reduce(const uint32_t (&in)[NC], int lane) {
        uint32_t m[V];
#pragma unroll
        for (int i = 0; i < V; ++i) m[i] = i < NC ? in[i] : 0u;
        int n = V;
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) {
            if (n > 1) {
                n >>= 1;
                const bool up = lane & o;
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    if (j < n) {
                        const uint32_t keep = up ? m[j + n] : m[j], give = up ? m[j] : m[j + n];
                        m[j] = max(keep, __shfl_xor_sync(0xffffffffu, give, o));
                    }
                }
            } else {
                m[0] = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
            }
        }
        return m[0];
    }
};

// ------------------------------------------------------------- tensor cores
// Instruction descriptor of kind::mxf8f6f4: e4m3 A and B (format code 0), both
// K-major, E8M0 scales; the two scale ids name the byte of each row's 32-bit
// scale word that the instruction applies.
__host__ __device__ constexpr uint32_t idesc_mx_e4m3(int M, int N, int a_id, int b_id) {
    return ((uint32_t)b_id << 4)            // B scale id
           | ((uint32_t)(N >> 3) << 17)     // N / 8
           | (1u << 23)                     // scale type: E8M0
           | ((uint32_t)(M >> 4) << 24)     // M / 16
           | ((uint32_t)a_id << 29);        // A scale id
}

// Unswizzled K-major descriptor of a scale atom: 32 rows of 16 bytes.
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1u << 16) | ((uint64_t)(128u >> 4) << 32) |
           ((uint64_t)1u << 46);
}

// One scale atom (128 rows x one 32-bit word of four K blocks' scales; row r's
// word at byte (r % 32) * 16 + (r / 32) * 4 of shared memory) into four tensor
// memory columns, repeated in every 32-lane quarter.
template <int CG>
__device__ __forceinline__ void tc_copy_scales(uint32_t taddr, uint64_t desc) {
    if constexpr (CG == 2)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// D[tmem] (+)= (A scaled) (B scaled)^T, K = 32, one scale per row and 32 K.
template <int CG>
__device__ __forceinline__ void tc_mma_mx(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t a_scale, uint32_t b_scale, uint32_t accumulate) {
    if constexpr (CG == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate)
            : "memory");
}

// The 32-bit word of scales of K blocks [4 chunk, 4 chunk + 4) of one row
// (scale 1 past the last block), from the one or two aligned words that hold
// them: no word without one of the row's bytes is read.  No branches, so that a
// loader's words are on their way together (byte by byte under conditions, a
// row length that is no multiple of four doubled a product's time).
__device__ __forceinline__ uint32_t scale_word(const uint8_t* row, int chunk, int blocks) {
    const uint8_t* p = row + 4 * (long long)chunk;
    const int n = min(4, blocks - 4 * chunk);
    const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(p) & 3u;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p - off);
    const uint32_t lo = __ldcg(q), hi = off + n > 4 ? __ldcg(q + 1) : 0u;
    const uint32_t keep = 0xffffffffu >> (32 - 8 * n);
    return (__funnelshift_r(lo, hi, 8 * off) & keep) | (0x7f7f7f7fu & ~keep);
}

// One lane of a converged warp, the same one every time.  Work issued by one
// thread inside a loop that the whole warp runs keeps its operands (tensor
// core descriptors, addresses, predicates) in the warp's uniform registers,
// where tcgen05 and bulk copies take them; in a branch that a single lane
// entered they are moved there one by one for every instruction (an MMA then
// took 140-170 cycles to issue, more than it takes to run).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// mbar_wait that keeps to short budgets too: it polls for those.  (A thread that
// parks on the barrier comes back when the hardware likes, whatever its hint, so no
// wait for less than some 10 us could run out.)  The pair's MMA issuer parks all the
// same: with the poll in its loop 1024 x 4096 x 4096 took 18.6 instead of 16.9 us, and
// it ends soon after the loaders and epilogues around it have given up.
__device__ __forceinline__ bool mx_wait(uint32_t bar, uint32_t parity, const WaitCtx& w, int site, bool honour_abort = true) {
    if (w.budget_ns >= 20000u) return mbar_wait(bar, parity, w, site, honour_abort);
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if (honour_abort && *w.abort) return false;
        if (globaltimer_ns() - t0 > w.budget_ns) {
            record_error(w.err, RM_ERR_DEVICE_TIMEOUT, site);
            *w.abort = 1;
            return false;
        }
    }
}

// mbar_wait for a phase that the other CTA of the pair has arrived on with
// release at cluster scope (its scale atoms in its own shared memory).
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, const WaitCtx& w, int site) {
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(20000u)
            : "memory");
        if (ok) return true;
        if (*w.abort) return false;
        if (globaltimer_ns() - t0 > w.budget_ns) {
            record_error(w.err, RM_ERR_DEVICE_TIMEOUT, site);
            *w.abort = 1;
            return false;
        }
    }
}

__device__ __forceinline__ void st_cluster_u32(uint32_t a, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ float2 lds_f32x2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts16(uint32_t a, uint16_t v) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(v) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t a, uint2 v) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(v.x), "r"(v.y) : "memory");
}

// Wait until all but the last N bulk groups have read their shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// The opt-in to more than 48 KB of shared memory, once per kernel and device.
struct SmemGrant {
    bool done[64] = {};
    template <typename F>
    cudaError_t ask(F* kernel, int bytes) {
        int d = 0;
        cudaError_t e = cudaGetDevice(&d);
        if (e != cudaSuccess || (d < 64 && __atomic_load_n(&done[d], __ATOMIC_ACQUIRE))) return e;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess && d < 64) __atomic_store_n(&done[d], true, __ATOMIC_RELEASE);
        return e;
    }
};


}  // namespace rm
