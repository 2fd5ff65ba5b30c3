// Matrix product of block-scaled 8-bit operands on the 5th-generation tensor
// cores:
//     out[g, m, n] = act( sum_k A[g,m,k] 2^ea[g,m,k/128] W[g,n,k] 2^ew[g,n/bw,k/128]
//                         + bias[g,n] ) + resid[g,m,n]
// with e4m3 codes, E8M0 scales, and out in bf16, fp32, or e4m3 with a scale
// for each 128 columns (the next product's operand).
//
// tcgen05.mma kind::mxf8f6f4 multiplies each row's 32 K elements by that
// row's power-of-two scale inside the tensor core, so a block of 128 costs no
// rescaling of the accumulator: its four K = 32 instructions name the same
// scale byte.  A row's scales of four consecutive K blocks are the bytes of
// one 32-bit word of tensor memory; the words of 128 rows ("an atom", 512
// bytes) are copied there by tcgen05.cp once for every 512 of K.
//
// Roles of a CTA:
//   warp 0      TMA producer: 128-byte K slices of A and W into the ring
//   warp 1      MMA issuer (one thread): scale copies, MMAs, commits
//   warps 2, 3  scale loaders: global bytes -> atoms in shared memory, taking
//               turns chunk by chunk (a chunk is 512 of K)
//   warps 4-11  epilogue, two groups of four warps (32 accumulator rows a
//               warp, a row a thread, 128 columns each)
// All waits are bounded (rm_device.cuh).
#include <cuda.h>
#include <cuda_bf16.h>

#include <cstring>

#include "rm_mx.cuh"
#include "rm_tmap.h"

namespace rm {
namespace {

constexpr int BM = 128;
constexpr int BK = 128;            // K elements (bytes) of a ring stage
constexpr int kSlots = 4;          // scale atoms in flight (chunks of 512 K)
constexpr int kEpiWarps = 8;
constexpr int kThreads = (4 + kEpiWarps) * 32;

struct MxParams {
    int G, M, N, K;
    int a_g_inner, w_g_inner;   // map coordinate order (k, g, row) if 1, else (k, row, g)
    int a_gmul, w_gmul;         // 0: the operand is shared by all groups
    const uint8_t* a_scale;
    long long as_gs, as_ld;
    const uint8_t* w_scale;
    long long ws_gs, ws_ld;
    int w_shift;                // row n's scales are row n >> w_shift of w_scale
    int a_vec, w_vec;           // the scale rows start on 4-byte boundaries
    const float* bias;
    const void* resid;
    long long r_gs, r_ld;
    void* out;
    long long o_gs, o_ld;
    int o_wide;                 // the output rows start on 32-byte boundaries
    uint8_t* out_scale;
    long long os_gs, os_ld;
    int act;
    DeviceErr err;
    unsigned long long budget_ns;
};

// Tile of 128 * CG x BN (CG = 2: a CTA pair).
template <int BN, int CG>
struct Cfg {
    static constexpr int TM = BM * CG;
    static constexpr int B_ROWS = BN / CG;                 // W rows a CTA loads
    static constexpr int A_BYTES = BM * BK, B_BYTES = B_ROWS * BK;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int B_ATOMS = (BN + 127) / 128;       // every CTA holds all BN columns' scales
    static constexpr int SLOT_BYTES = 512 * (1 + B_ATOMS);
    static constexpr int SLOT_COLS = 4 * (1 + B_ATOMS);
    static constexpr int STAGES_RAW = (227 * 1024 - 1024 - 512 - kSlots * SLOT_BYTES) / STAGE_BYTES;
    static constexpr int STAGES = STAGES_RAW > 8 ? 8 : STAGES_RAW;
    static constexpr int NBARS = 2 * STAGES + 2 * kSlots + 5;
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + kSlots * SLOT_BYTES + 8 * NBARS + 16;
    // Accumulators: two of BN columns for BN = 128.  Two of 256 do not fit
    // beside the scales, so they overlap by 48 columns, which the epilogue
    // empties first (the next tile's MMAs wait for those alone).
    static constexpr int ACC1 = BN == 256 ? 208 : BN;
    static constexpr int SCALE_COL = ACC1 + BN;
    static constexpr int TMEM_COLS = SCALE_COL + kSlots * SLOT_COLS <= 512 ? 512 : 0;
    static_assert(BN == 128 || BN == 256, "a group of epilogue warps takes 128 columns");
    static_assert(TMEM_COLS == 512 && SMEM_BYTES <= 227 * 1024, "on-chip memory");
};

struct Tile {
    int g, m0, n0;
};
__device__ __forceinline__ Tile decode(long long idx, int mblk, int nblk, int tm, int bn) {
    // the M tiles of one W tile run next to each other, so that W is read from L2
    Tile t;
    const long long per_g = (long long)mblk * nblk;
    t.g = (int)(idx / per_g);
    const int r = (int)(idx - (long long)t.g * per_g);
    const int nb = r / mblk;
    t.n0 = nb * bn;
    t.m0 = (r - nb * mblk) * tm;
    return t;
}

// out = act(v): GELU through tanh.approx (relative error 2^-11) where the
// result is stored in 16 or 8 bits, through exp for fp32 results.
template <bool PRECISE>
__device__ __forceinline__ float2 activation(float2 v, int act) {
    if (act == RM_ACT_GELU_TANH) {
        if constexpr (!PRECISE) return gelu_tanh_pair(v);
        const float c = 2.0f * 0.7978845608028654f;   // v * sigmoid(2u), u = sqrt(2/pi) (v + 0.044715 v^3)
        v.x = v.x / (1.0f + expf(-c * fmaf(0.044715f * v.x * v.x, v.x, v.x)));
        v.y = v.y / (1.0f + expf(-c * fmaf(0.044715f * v.y * v.y, v.y, v.y)));
    } else if (act == RM_ACT_GELU_ERF) {
        v.x = 0.5f * v.x * erfcf(-0.7071067811865476f * v.x);
        v.y = 0.5f * v.y * erfcf(-0.7071067811865476f * v.y);
    } else if (act == RM_ACT_RELU) {
        v.x = v.x < 0.f ? 0.f : v.x;   // (keeps NaN)
        v.y = v.y < 0.f ? 0.f : v.y;
    }
    return v;
}

// 32 (or 2 x 16) bytes to global memory.
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8], bool wide) {
    if (wide) {
        stg256(p, w);
    } else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// bias, activation and residual of NV columns from n of row m, in place.
// Columns from N on are left as they are.
template <int OUT, int NV>
__device__ __forceinline__ void finish(float (&v)[NV], const MxParams& p, int g, int m, int n) {
    if (p.bias) {
        const float* b = p.bias + (long long)g * p.N + n;
#pragma unroll
        for (int q = 0; q < NV / 4; ++q) {
            if (n + 4 * q < p.N) {
                const float4 x = reinterpret_cast<const float4*>(b)[q];
                v[4 * q] += x.x, v[4 * q + 1] += x.y, v[4 * q + 2] += x.z, v[4 * q + 3] += x.w;
            }
        }
    }
    if (p.act != RM_ACT_NONE) {
#pragma unroll
        for (int e = 0; e < NV; e += 2) {
            const float2 y = activation<OUT == RM_F32>(make_float2(v[e], v[e + 1]), p.act);
            v[e] = y.x, v[e + 1] = y.y;
        }
    }
    if (OUT != RM_E4M3 && p.resid) {
        if constexpr (OUT == RM_BF16) {
            const __nv_bfloat16* r = static_cast<const __nv_bfloat16*>(p.resid) + g * p.r_gs + m * p.r_ld + n;
#pragma unroll
            for (int q = 0; q < NV / 8; ++q) {
                if (n + 8 * q < p.N) {
                    float2 f[4];
                    unpack_pairs(reinterpret_cast<const uint4*>(r)[q], f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[8 * q + 2 * e] += f[e].x, v[8 * q + 2 * e + 1] += f[e].y;
                }
            }
        } else {
            const float* r = static_cast<const float*>(p.resid) + g * p.r_gs + m * p.r_ld + n;
#pragma unroll
            for (int q = 0; q < NV / 4; ++q) {
                if (n + 4 * q < p.N) {
                    const float4 x = reinterpret_cast<const float4*>(r)[q];
                    v[4 * q] += x.x, v[4 * q + 1] += x.y, v[4 * q + 2] += x.z, v[4 * q + 3] += x.w;
                }
            }
        }
    }
}

// Store NV columns from n of row m (N is a multiple of 16).
template <int OUT, int NV>
__device__ __forceinline__ void store_row(const float (&v)[NV], const MxParams& p, int g, int m, int n) {
    if constexpr (OUT == RM_BF16) {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + g * p.o_gs + m * p.o_ld + n;
#pragma unroll
        for (int q = 0; q < NV / 16; ++q) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(v[16 * q + 2 * i], v[16 * q + 2 * i + 1]);
            if (n + 16 * q < p.N) store32(o + 16 * q, w, p.o_wide);
        }
    } else if constexpr (OUT == RM_F32) {
        float* o = static_cast<float*>(p.out) + g * p.o_gs + m * p.o_ld + n;
#pragma unroll
        for (int q = 0; q < NV / 8; ++q) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[8 * q + i]);
            if (n + 8 * q < p.N) store32(o + 8 * q, w, p.o_wide);
        }
    } else {   // NV = 128: one block, quantised from fp32
        uint32_t mx = 0;
#pragma unroll
        for (int e = 0; e < NV; ++e) mx = max(mx, n + (e & ~15) < p.N ? abs_bits(v[e]) : 0u);
        const uint32_t b = scale_byte(mx);
        const float inv = scale_inverse(min(b, 254u));
        uint8_t* o = static_cast<uint8_t*>(p.out) + g * p.o_gs + m * p.o_ld + n;
        p.out_scale[g * p.os_gs + m * p.os_ld + (n >> 7)] = (uint8_t)b;
#pragma unroll
        for (int q = 0; q < NV / 32; ++q) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float* x = v + 32 * q + 4 * i;
                w[i] = b == 255u ? kNanCodes : e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
            }
            if (n + 32 * q + 32 <= p.N) store32(o + 32 * q, w, p.o_wide);
            else if (n + 32 * q < p.N) *reinterpret_cast<uint4*>(o + 32 * q) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

template <int NV>
__device__ __forceinline__ void load_acc(uint32_t taddr, float (&v)[NV]) {
#pragma unroll
    for (int q = 0; q < NV / 16; ++q) {
        float w[16];
        tmem_ld16(taddr + 16 * q, w);
#pragma unroll
        for (int e = 0; e < 16; ++e) v[16 * q + e] = w[e];
    }
    tmem_ld_wait();
}

template <int BN, int CG, int OUT>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_mx_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW, const MxParams p) {
    using C = Cfg<BN, CG>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    unsigned char* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    const uint32_t slot0 = sbase + C::STAGES * C::STAGE_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::STAGES * C::STAGE_BYTES + kSlots * C::SLOT_BYTES);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * C::STAGES;
    const uint32_t sfull0 = empty0 + 8 * C::STAGES, sempty0 = sfull0 + 8 * kSlots;
    const uint32_t tfull0 = sempty0 + 8 * kSlots, tempty0 = tfull0 + 16, drain_bar = tempty0 + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NBARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(sfull0 + 8 * s, CG);
            mbar_init(sempty0 + 8 * s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull0 + 8 * a, 1);
            mbar_init(tempty0 + 8 * a, CG * 32 * (BN == 128 ? kEpiWarps / 2 : kEpiWarps));
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmW);
    }
    if (warp == 0) {
        if constexpr (CG == 2) {
            tmem_alloc_pair(smem_u32(tmem_slot), C::TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_enter();   // operands, scales and bias may all come from the previous kernel

    const WaitCtx wc{abort_flag, p.budget_ns, p.err};
    const int mblk = (p.M + C::TM - 1) / C::TM, nblk = (p.N + BN - 1) / BN;
    const int num_kb = (p.K + BK - 1) / BK;
    const long long total = (long long)p.G * mblk * nblk;
    const long long unit = blockIdx.x / CG, nunits = gridDim.x / CG;

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, issued = 0, issued_phase = 0;
            bool ok = true;
            for (long long idx = unit; idx < total && ok; idx += nunits) {
                const Tile t = decode(idx, mblk, nblk, C::TM, BN);
                const int ar = t.m0 + (int)rank * BM, wr = t.n0 + (int)rank * C::B_ROWS;
                const int ag = t.g * p.a_gmul, wg = t.g * p.w_gmul;
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait(empty0 + 8 * stage, phase ^ 1u, wc, SITE_MX_PRODUCER)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = full0 + 8 * stage, sa = sbase + stage * C::STAGE_BYTES;
                    if (leader) mbar_arrive_expect_tx(fb, CG * C::STAGE_BYTES);
                    if constexpr (CG == 2) {   // the pair counts bytes on the even CTA's barrier
                        const uint32_t fbl = mapa_shared(fb, 0);
                        tma_load_3d_pair(sa, &tmA, fbl, kb * BK, p.a_g_inner ? ag : ar, p.a_g_inner ? ar : ag);
                        tma_load_3d_pair(sa + C::A_BYTES, &tmW, fbl, kb * BK, p.w_g_inner ? wg : wr,
                                         p.w_g_inner ? wr : wg);
                    } else {
                        tma_load_3d(sa, &tmA, fb, kb * BK, p.a_g_inner ? ag : ar, p.a_g_inner ? ar : ag);
                        tma_load_3d(sa + C::A_BYTES, &tmW, fb, kb * BK, p.w_g_inner ? wg : wr, p.w_g_inner ? wr : wg);
                    }
                    issued |= 1u << stage;
                    issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
                    if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            if (leader)   // every issued copy lands before shared memory goes away
                for (int s = 0; s < C::STAGES; ++s)
                    if (issued & (1u << s))
                        mbar_wait(full0 + 8 * s, (issued_phase >> s) & 1u, wc, SITE_MX_DRAIN, false);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            constexpr uint32_t idesc0 = idesc_mx_e4m3(C::TM, BN, 0, 0);
            int stage = 0, slot = 0;
            uint32_t phase = 0, sphase = 0;
            bool ok = true, any = false;
            int it = 0;
            for (long long idx = unit; idx < total && ok; idx += nunits, ++it) {
                const int acc = it & 1;
                // BN = 128: the tile before the last one has left this accumulator.
                // BN = 256: the last tile's epilogue has begun on every warp (so the
                // tile before it is done) and emptied the overlapping columns.
                if (BN == 128 ? !mbar_wait(tempty0 + 8 * acc, ((uint32_t)(it >> 1) & 1u) ^ 1u, wc, SITE_MX_MMA)
                              : it > 0 && !mbar_wait(tempty0, (uint32_t)(it - 1) & 1u, wc, SITE_MX_MMA))
                    break;
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(acc * C::ACC1);
                for (int kb = 0; kb < num_kb; ++kb) {
                    const uint32_t sa_col = tmem + C::SCALE_COL + slot * C::SLOT_COLS, sb_col = sa_col + 4;
                    if ((kb & 3) == 0) {
                        if (!mbar_wait(sfull0 + 8 * slot, sphase, wc, SITE_MX_SCALES)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t ss = slot0 + slot * C::SLOT_BYTES;
                        tc_copy_scales<CG>(sa_col, smem_desc_scales(ss));
#pragma unroll
                        for (int a = 0; a < C::B_ATOMS; ++a)
                            tc_copy_scales<CG>(sb_col + 4 * a, smem_desc_scales(ss + 512 * (1 + a)));
                        any = true;
                    }
                    if (!mbar_wait(full0 + 8 * stage, phase, wc, SITE_MX_MMA)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = sbase + stage * C::STAGE_BYTES;
                    const uint64_t ad = smem_desc_k_sw128(sa), bd = smem_desc_k_sw128(sa + C::A_BYTES);
                    const uint32_t id = idesc0 | ((uint32_t)(kb & 3) << 4) | ((uint32_t)(kb & 3) << 29);
#pragma unroll
                    for (int k = 0; k < BK / 32; ++k)
                        tc_mma_mx<CG>(d, ad + 2 * k, bd + 2 * k, id, sa_col, sb_col, (kb | k) != 0 ? 1u : 0u);
                    any = true;
                    const bool chunk_end = (kb & 3) == 3 || kb == num_kb - 1;
                    if constexpr (CG == 2) {
                        tc_commit_pair_mc(empty0 + 8 * stage, 0x3);
                        if (chunk_end) tc_commit_pair_mc(sempty0 + 8 * slot, 0x3);
                    } else {
                        tc_commit(empty0 + 8 * stage);
                        if (chunk_end) tc_commit(sempty0 + 8 * slot);
                    }
                    if (chunk_end && ++slot == kSlots) { slot = 0; sphase ^= 1u; }
                    if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                if constexpr (CG == 2) tc_commit_pair_mc(tfull0 + 8 * acc, 0x3);
                else tc_commit(tfull0 + 8 * acc);
            }
            if (any) {   // everything issued completes before tensor memory is released
                if constexpr (CG == 2) tc_commit_pair(drain_bar);
                else tc_commit(drain_bar);
                mbar_wait(drain_bar, 0, wc, SITE_MX_DRAIN, false);
            }
        }
        __syncwarp();
    } else if (warp < 4) {
        // Scale loaders: chunk c of the CTA's stream of chunks by warp 2 + c % 2.
        const int chunks = (num_kb + 3) / 4;
        long long c = 0;
        bool ok = true;
        for (long long idx = unit; idx < total && ok; idx += nunits) {
            const Tile t = decode(idx, mblk, nblk, C::TM, BN);
            const uint8_t* as = p.a_scale + t.g * p.as_gs;
            const uint8_t* ws = p.w_scale + t.g * p.ws_gs;
            for (int ch = 0; ch < chunks; ++ch, ++c) {
                if ((int)(c & 1) != warp - 2) continue;
                const int slot = (int)(c % kSlots);
                uint32_t w[1 + C::B_ATOMS][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = t.m0 + (int)rank * BM + 32 * j + lane;
                    w[0][j] = r < p.M ? scale_word(as + r * p.as_ld, ch, num_kb, p.a_vec) : 0x7f7f7f7fu;
                }
#pragma unroll
                for (int a = 0; a < C::B_ATOMS; ++a)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = t.n0 + 128 * a + 32 * j + lane;
                        w[1 + a][j] =
                            r < p.N ? scale_word(ws + (r >> p.w_shift) * p.ws_ld, ch, num_kb, p.w_vec) : 0x7f7f7f7fu;
                    }
                // the slot is free once the MMAs that read its last content (and
                // the tensor memory copy of it) have completed
                if (!mbar_wait(sempty0 + 8 * slot, (uint32_t)(c / kSlots & 1) ^ 1u, wc, SITE_MX_SCALES)) {
                    ok = false;
                    break;
                }
                const uint32_t dst = slot0 + slot * C::SLOT_BYTES + lane * 16;
#pragma unroll
                for (int a = 0; a < 1 + C::B_ATOMS; ++a)
                    sts128(dst + 512 * a, make_uint4(w[a][0], w[a][1], w[a][2], w[a][3]));
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    if (CG == 2 && !leader) mbar_arrive_cluster(mapa_shared(sfull0 + 8 * slot, 0));
                    else mbar_arrive(sfull0 + 8 * slot);
                }
            }
        }
        __syncwarp();
    } else {
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const uint32_t tempty_l = CG == 2 ? mapa_shared(tempty0, 0) : tempty0;
        int it = 0;
        for (long long idx = unit; idx < total; idx += nunits, ++it) {
            const int acc = it & 1;
            if (BN == 128 && acc != half) continue;   // the groups take tiles in turn
            if (!mbar_wait(tfull0 + 8 * acc, (uint32_t)(it >> 1) & 1u, wc, SITE_MX_EPILOGUE)) break;
            tc_fence_after();
            const Tile t = decode(idx, mblk, nblk, C::TM, BN);
            const int col0 = BN == 128 ? 0 : 128 * half;   // this group's 128 columns
            const uint32_t ta = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * C::ACC1 + col0);
            const int m = t.m0 + (int)rank * BM + quarter * 32 + lane, n = t.n0 + col0;
            const bool live = m < p.M;
            const uint32_t tb = tempty_l + (BN == 128 ? 8u * (uint32_t)acc : 0u);
            auto release = [&] {
                tc_fence_before();
                if (CG == 2 && !leader) mbar_arrive_cluster_relaxed(tb);
                else mbar_arrive(tb);
            };
            if constexpr (OUT == RM_E4M3) {
                float v[128];
                load_acc(ta, v);
                release();
                if (live && n < p.N) {
                    finish<OUT>(v, p, t.g, m, n);
                    store_row<OUT>(v, p, t.g, m, n);
                }
            } else {
                // the accumulators' overlap (columns 208-255 of the first) goes first
                const int first = BN == 256 && acc == 0 && half == 1 ? 1 : 0;
#pragma unroll 1
                for (int k = 0; k < 2; ++k) {
                    const int c = 64 * (k ^ first);
                    float v[64];
                    load_acc(ta + c, v);
                    if (k == (BN == 256 ? 0 : 1)) release();
                    if (live && n + c < p.N) {
                        finish<OUT>(v, p, t.g, m, n + c);
                        store_row<OUT>(v, p, t.g, m, n + c);
                    }
                }
            }
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync_all();   // the peer may still signal this CTA's barriers
    if (warp == 0) {
        tc_fence_after();
        if constexpr (CG == 2) tmem_dealloc_pair(tmem, C::TMEM_COLS);
        else tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// Operand map: dims (K, rows, groups) with the smaller of the two strides
// first.  A single row or group takes any legal stride.
bool operand_map(CUtensorMap* m, const void* base, int K, int rows, int G, long long ld, long long gs, uint32_t box,
                 int* g_inner, int* gmul) {
    *gmul = gs == 0 ? 0 : 1;
    if (gs == 0) G = 1;
    if (rows == 1) ld = ((long long)K + 15) / 16 * 16;
    if (G == 1) gs = rows * ld;
    *g_inner = gs < ld ? 1 : 0;
    return *g_inner ? make_map_e(m, base, K, G, rows, gs, ld, 1, box, 1) : make_map_e(m, base, K, rows, G, ld, gs, box, 1, 1);
}

template <int BN, int CG, int OUT>
cudaError_t launch_tile(const rm_matmul_fp8_args& a, MxParams& p, int num_sms, cudaStream_t s) {
    using C = Cfg<BN, CG>;
    static const cudaError_t attr =
        cudaFuncSetAttribute(gemm_mx_kernel<BN, CG, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (attr != cudaSuccess) return attr;
    CUtensorMap ma, mw;
    if (!operand_map(&ma, a.A, a.K, a.M, a.G, a.a_ld, a.a_gstride, BM, &p.a_g_inner, &p.a_gmul) ||
        !operand_map(&mw, a.W, a.K, a.N, a.G, a.w_ld, a.w_gstride, C::B_ROWS, &p.w_g_inner, &p.w_gmul))
        return cudaErrorInvalidValue;
    const long long tiles =
        (long long)a.G * ((a.M + C::TM - 1) / C::TM) * ((a.N + BN - 1) / BN);
    const int units = (int)(tiles < num_sms / CG ? tiles : num_sms / CG);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(units * CG);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = CG;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, gemm_mx_kernel<BN, CG, OUT>, ma, mw, p);
}

template <int OUT>
cudaError_t launch_out(const rm_matmul_fp8_args& a, MxParams& p, int num_sms, cudaStream_t s) {
    return launch_tile<128, 1, OUT>(a, p, num_sms, s);
}

}  // namespace

cudaError_t launch_gemm_mx(const rm_matmul_fp8_args& a, int num_sms, cudaStream_t s) {
    MxParams p{};
    p.G = a.G, p.M = a.M, p.N = a.N, p.K = a.K;
    p.a_scale = a.a_scale, p.as_gs = a.as_gstride, p.as_ld = a.as_ld;
    p.w_scale = a.w_scale, p.ws_gs = a.ws_gstride, p.ws_ld = a.ws_ld;
    p.w_shift = a.w_block_rows == 128 ? 7 : 0;
    const auto quads = [](const void* b, long long x, long long y) {
        return (reinterpret_cast<uintptr_t>(b) & 3) == 0 && x % 4 == 0 && y % 4 == 0;
    };
    p.a_vec = quads(a.a_scale, a.as_gstride, a.as_ld);
    p.w_vec = quads(a.w_scale, a.ws_gstride, a.ws_ld);
    p.bias = a.bias;
    p.resid = a.resid, p.r_gs = a.r_gstride, p.r_ld = a.r_ld;
    p.out = a.out, p.o_gs = a.o_gstride, p.o_ld = a.o_ld;
    const int osz = a.out_dtype == RM_F32 ? 4 : a.out_dtype == RM_BF16 ? 2 : 1;
    p.o_wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0 && a.o_gstride * osz % 32 == 0 && a.o_ld * osz % 32 == 0;
    p.out_scale = a.out_scale, p.os_gs = a.os_gstride, p.os_ld = a.os_ld;
    p.act = a.act;
    p.err = DeviceErr{a.device_status, nullptr};
    p.budget_ns = a.wait_budget_ns ? a.wait_budget_ns : 1000000000ull;
    switch (a.out_dtype) {
        case RM_F32: return launch_out<RM_F32>(a, p, num_sms, s);
        case RM_BF16: return launch_out<RM_BF16>(a, p, num_sms, s);
        default: return launch_out<RM_E4M3>(a, p, num_sms, s);
    }
}

}  // namespace rm
