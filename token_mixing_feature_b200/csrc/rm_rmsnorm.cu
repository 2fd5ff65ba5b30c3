// Root-mean-square norm with the residual's addition, an output in the
// stream's type and / or in e4m3 with a scale for each block of 128, and its
// gradient.
//
//     s = round(x + r)                 rstd = 1 / sqrt(mean(s^2) + eps)
//     y = s * rstd * gamma             yq, ys = e4m3 blocks of y (from fp32)
//     a = gamma * dy
//     dx = rstd * (a - s * rstd^2 * mean(a * s)) + dsum
//     dgamma = sum over rows of dy * s * rstd
//
// Both directions are bound by HBM: a row is read once and everything leaves
// from the registers.  A row belongs to a group of threads (whole warps), each
// with NC chunks of 8 consecutive elements, so a block of 128 is 16
// neighbouring lanes and its largest magnitude costs four shuffles.  One CTA of
// up to 512 threads an SM; its groups walk over the rows, the next rows on
// their way into a ring in shared memory by cp.async: every thread copies the
// chunks that it will read, so the ring needs no barrier, and what is in flight
// (up to 200 KB an SM) depends neither on registers nor on where a group is in
// its row.  With the rows loaded straight into registers, 16384 x 1536 ran at
// 4.2-4.6 TB/s whatever the launch shape.
#include <cuda_bf16.h>

#include <algorithm>

#include "rm_mx.cuh"

namespace rm {
namespace {

constexpr int kCta = 512;               // threads a CTA has at most
constexpr int kRing = 200 * 1024;       // bytes of its ring
constexpr int kSms = 148;

// Eight consecutive elements as they lie in memory.
template <typename E>
struct Chunk {
    static constexpr int N = sizeof(E) / 2;   // 16-byte pieces
    uint4 u[N];
    __device__ __forceinline__ void read(uint32_t shared) {
#pragma unroll
        for (int i = 0; i < N; ++i) u[i] = lds128(shared + 16 * i);
    }
    __device__ __forceinline__ void store(void* base, long long at) const {
        uint4* p = reinterpret_cast<uint4*>(static_cast<E*>(base) + at);
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = u[i];
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < N; ++i) u[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void set(const float2 (&v)[4]) {   // rounded to the type
        if constexpr (N == 1) {
            u[0] = pack_pairs(v);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) u[i] = pack_pairs({v[2 * i], v[2 * i + 1]});
        }
    }
    __device__ __forceinline__ void pairs(float2 (&v)[4]) const {
        if constexpr (N == 1) {
            unpack_pairs(u[0], v);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float2 h[2];
                unpack_pairs(u[i], h);
                v[2 * i] = h[0], v[2 * i + 1] = h[1];
            }
        }
    }
};
__device__ __forceinline__ void load_params(const float* p, float2 (&g)[4]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    g[0] = make_float2(a.x, a.y), g[1] = make_float2(a.z, a.w), g[2] = make_float2(b.x, b.y), g[3] = make_float2(b.z, b.w);
}
// 1 / sqrt(x): the approximation (2^-22.9) and a Newton step.
__device__ __forceinline__ float inv_sqrt(float x) {
    const float r = rsqrtf(x);
    const float c = fmaf(-0.5f * x * r, r, 0.5f);
    return isinf(r) || r == 0.f ? r : fmaf(r, c, r);
}

// One chunk (8 elements) of a global row into shared memory, asynchronously.
template <typename E>
__device__ __forceinline__ void copy_chunk(uint32_t dst, const void* base, long long at) {
    const char* src = reinterpret_cast<const char*>(static_cast<const E*>(base) + at);
#pragma unroll
    for (int i = 0; i < Chunk<E>::N; ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 16 * i), "l"(src + 16 * i) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait for all but this thread's last n groups of copies.
__device__ __forceinline__ void copies_wait(int n) {
    switch (n) {
        case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
        case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    }
}

// A thread's place: its group (row) of the CTA and its rank there.
struct Place {
    int tpr, group, groups, t, first_warp, warps;
    __device__ __forceinline__ explicit Place(int tpr_) : tpr(tpr_) {
        groups = blockDim.x / tpr;
        group = threadIdx.x / tpr;
        t = threadIdx.x - group * tpr;
        warps = tpr >> 5;
        first_warp = group * warps;
    }
    // Sum over the group's threads (every thread gets it), in a fixed order.
    // red: a float per warp of the CTA, not the last call's; all threads of the
    // group call this together.
    __device__ __forceinline__ float sum(float v, float* red) const {
        v = warp_sum(v);
        if (warps > 1) {
            if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
            asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(tpr) : "memory");
            v = 0.f;
            for (int w = 0; w < warps; ++w) v += red[first_warp + w];
        }
        return v;
    }
};

template <typename E, int NC, bool RESID>
__global__ void __launch_bounds__(kCta, 1) rmsnorm_kernel(const RmsNorm p, int tpr, int stages) {
    __shared__ float red[2][kCta / 32];
    extern __shared__ __align__(16) unsigned char ring[];
    pdl_enter();
    const Place at(tpr);
    const int nch = p.D / 8;
    const float inv_d = 1.0f / (float)p.D;
    const uint32_t bytes = (uint32_t)(p.D * sizeof(E)), slot = bytes * (RESID ? 2 : 1);
    const uint32_t mine = smem_u32(ring) + (uint32_t)(at.group * stages) * slot + (uint32_t)at.t * 8 * sizeof(E);
    const uint32_t hop = (uint32_t)tpr * 8 * sizeof(E);   // from a thread's chunk to its next
    const long long step = (long long)gridDim.x * at.groups;
    long long row = (long long)blockIdx.x * at.groups + at.group;
    auto fetch = [&](long long r, int s) {
        if (r < p.rows) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = at.t + i * tpr;
                if (c < nch) {
                    copy_chunk<E>(mine + s * slot + i * hop, p.X, r * p.ld_x + 8 * c);
                    if constexpr (RESID) copy_chunk<E>(mine + s * slot + bytes + i * hop, p.R, r * p.ld_r + 8 * c);
                }
            }
        }
        copies_commit();
    };
    for (int s = 0; s < stages - 1; ++s) fetch(row + s * step, s);
    int s = 0, last = stages - 1;   // the ring's place of this row and of the row stages - 1 on
    for (int par = 0; row < p.rows; row += step, par ^= 1) {   // (one value of row per group)
        fetch(row + (stages - 1) * step, last);
        copies_wait(stages - 1);
        Chunk<E> x[NC];
        float2 sq = f2(0.f);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = at.t + i * tpr;
            if (c < nch) {
                float2 v[4];
                x[i].read(mine + s * slot + i * hop);
                x[i].pairs(v);
                if constexpr (RESID) {
                    // the stream is rounded to its type here: the statistics, the
                    // output and the gradient all see the values that are stored
                    Chunk<E> r;
                    float2 q[4];
                    r.read(mine + s * slot + bytes + i * hop);
                    r.pairs(q);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = f2_add(v[e], q[e]);
                    x[i].set(v);
                    x[i].pairs(v);
                }
                if (p.Sum) x[i].store(p.Sum, row * p.ld_sum + 8 * c);
#pragma unroll
                for (int e = 0; e < 4; ++e) sq = f2_fma(v[e], v[e], sq);
            } else {
                x[i].clear();
            }
        }
        last = s;
        s = s + 1 == stages ? 0 : s + 1;
        const float rstd = inv_sqrt(fmaf(at.sum(sq.x + sq.y, red[par]), inv_d, p.eps));
        if (p.rstd && at.t == 0) p.rstd[row] = rstd;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = at.t + i * tpr;
            const bool in = c < nch;
            float2 y[4];
            x[i].pairs(y);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = f2_mul(y[e], f2(rstd));
            if (in && p.gamma) {
                float2 g[4];
                load_params(p.gamma + 8 * c, g);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = f2_mul(y[e], g[e]);
            }
            if (in && p.Y) {
                Chunk<E> o;
                o.set(y);
                o.store(p.Y, row * p.ld_y + 8 * c);
            }
            if (p.Yq) {   // (whole warps: tpr is a multiple of 32)
                float mf = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) mf = max_abs(mf, y[e]);
                uint32_t m = in ? abs_bits(mf) : 0u;
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                const uint32_t b = scale_byte(m);
                const float2 inv = f2(scale_inverse(b));
                if (in) {
                    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.Yq) + row * p.ld_yq + 8 * c) =
                        make_uint2(e4m3x4(f2_mul(y[0], inv), f2_mul(y[1], inv)), e4m3x4(f2_mul(y[2], inv), f2_mul(y[3], inv)));
                    if ((threadIdx.x & 15) == 0) p.Ys[row * p.ld_ys + c / 16] = (uint8_t)b;
                }
            }
        }
    }
}

// Gradient: the groups keep their columns' sums of dy * s * rstd in registers;
// a CTA's groups add theirs in order and leave one partial row.
template <typename E, int NC>
__global__ void __launch_bounds__(kCta, 1) rmsnorm_bwd_kernel(const RmsNormGrad p, int tpr, int stages) {
    __shared__ float red[2][kCta / 32];
    extern __shared__ __align__(16) unsigned char ring[];
    pdl_enter();
    const Place at(tpr);
    const int nch = p.D / 8;
    const uint32_t bytes = (uint32_t)(p.D * sizeof(E)), slot = bytes * (p.dSum ? 3 : 2);
    const uint32_t mine = smem_u32(ring) + (uint32_t)(at.group * stages) * slot + (uint32_t)at.t * 8 * sizeof(E);
    const uint32_t hop = (uint32_t)tpr * 8 * sizeof(E);
    const float inv_d = 1.0f / (float)p.D;
    float2 acc[NC][4];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = f2(0.f);
    const long long step = (long long)gridDim.x * at.groups;
    long long row = (long long)blockIdx.x * at.groups + at.group;
    auto fetch = [&](long long r, int s) {
        if (r < p.rows) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = at.t + i * tpr;
                if (c < nch) {
                    const uint32_t d = mine + s * slot + i * hop;
                    copy_chunk<E>(d, p.S, r * p.ld_s + 8 * c);
                    copy_chunk<E>(d + bytes, p.dY, r * p.ld_dy + 8 * c);
                    if (p.dSum) copy_chunk<E>(d + 2 * bytes, p.dSum, r * p.ld_dsum + 8 * c);
                }
            }
        }
        copies_commit();
    };
    for (int s = 0; s < stages - 1; ++s) fetch(row + s * step, s);
    int s = 0, last = stages - 1;
    float rstd = row < p.rows ? __ldcg(p.rstd + row) : 0.f;
    for (int par = 0; row < p.rows; row += step, par ^= 1) {
        fetch(row + (stages - 1) * step, last);
        const float next_rstd = row + step < p.rows ? __ldcg(p.rstd + row + step) : 0.f;
        copies_wait(stages - 1);
        float2 dots = f2(0.f);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = at.t + i * tpr;
            if (c < nch) {
                Chunk<E> cs, cy;
                float2 sv[4], dy[4];
                cs.read(mine + s * slot + i * hop);
                cy.read(mine + s * slot + i * hop + bytes);
                cs.pairs(sv);
                cy.pairs(dy);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][e] = f2_fma(f2_mul(dy[e], f2(rstd)), sv[e], acc[i][e]);
                if (p.gamma) {
                    float2 g[4];
                    load_params(p.gamma + 8 * c, g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) dy[e] = f2_mul(dy[e], g[e]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) dots = f2_fma(dy[e], sv[e], dots);
            }
        }
        const float dot = at.sum(dots.x + dots.y, red[par]);
        const float2 k = f2(-rstd * rstd * (dot * inv_d));
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = at.t + i * tpr;
            if (c < nch) {
                Chunk<E> cs, cy;
                float2 sv[4], dy[4];
                cs.read(mine + s * slot + i * hop);
                cy.read(mine + s * slot + i * hop + bytes);
                cs.pairs(sv);
                cy.pairs(dy);
                if (p.gamma) {
                    float2 g[4];
                    load_params(p.gamma + 8 * c, g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) dy[e] = f2_mul(dy[e], g[e]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) dy[e] = f2_mul(f2_fma(sv[e], k, dy[e]), f2(rstd));
                if (p.dSum) {
                    cs.read(mine + s * slot + i * hop + 2 * bytes);
                    cs.pairs(sv);
#pragma unroll
                    for (int e = 0; e < 4; ++e) dy[e] = f2_add(dy[e], sv[e]);
                }
                cs.set(dy);
                cs.store(p.dX, row * p.ld_dx + 8 * c);
            }
        }
        last = s;
        s = s + 1 == stages ? 0 : s + 1;
        rstd = next_rstd;
    }
    if (!p.part) return;
    // (every group has finished its rows: the ring now carries the sums from
    // group to group)
    float* acc_s = reinterpret_cast<float*>(ring);
    for (int k = 0; k < at.groups; ++k) {
        __syncthreads();
        if (at.group == k) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = at.t + i * tpr;
                if (c < nch) {
                    float2* a = reinterpret_cast<float2*>(acc_s + 8 * c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (k) acc[i][e] = f2_add(acc[i][e], a[e]);
                        if (k < at.groups - 1) a[e] = acc[i][e];
                    }
                    if (k == at.groups - 1) {
                        Chunk<float> o;
                        o.set(acc[i]);
                        o.store(p.part, (long long)blockIdx.x * p.D + 8 * c);
                    }
                }
            }
        }
    }
}

// dgamma[d] = sum over the partial rows, in a fixed order: 32 columns a CTA,
// 32 warps taking every 32nd row (eight loads in flight), then the warps' sums.
__global__ void __launch_bounds__(1024) colsum_parts_kernel(const float* part, float* out, int parts, int D) {
    __shared__ float s[32][33];
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int d = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (d < D) {
        for (int r0 = warp; r0 < parts; r0 += 32 * 8) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = r0 + 32 * j < parts ? __ldcg(part + (long long)(r0 + 32 * j) * D + d) : 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) v += x[j];
        }
    }
    s[warp][lane] = v;
    __syncthreads();
    v = warp_sum(s[lane][warp]);
    if (lane == 0 && blockIdx.x * 32 + warp < D) out[blockIdx.x * 32 + warp] = v;
}

// Launch shape for rows of D whose `row_bytes` (all inputs) go through the ring.
struct Shape {
    int nc, tpr, groups, threads, stages, grid;
    size_t smem;
    Shape(long long rows, int D, size_t row_bytes) {
        const int nch = D / 8;
        // Warps a row: as few as hold it in six chunks a thread (what a row costs
        // besides, its sum and its waits, is then shared by 48 elements a thread),
        // but all of them where the SMs have a row each.
        const int most = (nch + 31) / 32;
        int w = rows <= kSms ? most : (most + 5) / 6;
        w = std::min(w, kCta / 32);
        tpr = 32 * w;
        nc = (nch + tpr - 1) / tpr;
        groups = kCta / tpr;
        if (tpr > 32) groups = std::min(groups, 15);   // (named barriers)
        groups = (int)std::min<long long>(groups, (rows + kSms - 1) / kSms);
        groups = (int)std::min<size_t>(groups, kRing / row_bytes);
        stages = (int)std::min<size_t>(4, kRing / (row_bytes * groups));
        threads = groups * tpr;
        smem = row_bytes * groups * stages;
        grid = (int)std::min<long long>((rows + groups - 1) / groups, kSms);
    }
};

template <typename E, int NC, bool RESID>
cudaError_t fwd(const RmsNorm& p, const Shape& sh, cudaStream_t s) {
    static SmemGrant grant;
    if (cudaError_t e = grant.ask(rmsnorm_kernel<E, NC, RESID>, kRing)) return e;
    return launch_pdl(rmsnorm_kernel<E, NC, RESID>, dim3(sh.grid), dim3(sh.threads), sh.smem, s, p, sh.tpr, sh.stages);
}
template <typename E, bool RESID>
cudaError_t fwd_e(const RmsNorm& p, cudaStream_t s) {
    const Shape sh(p.rows, p.D, sizeof(E) * p.D * (RESID ? 2 : 1));
    switch (sh.nc) {
        case 1: return fwd<E, 1, RESID>(p, sh, s);
        case 2: return fwd<E, 2, RESID>(p, sh, s);
        case 3: return fwd<E, 3, RESID>(p, sh, s);
        case 4: return fwd<E, 4, RESID>(p, sh, s);
        case 5: return fwd<E, 5, RESID>(p, sh, s);
        default: return fwd<E, 6, RESID>(p, sh, s);
    }
}

template <typename E, int NC>
cudaError_t bwd(const RmsNormGrad& p, const Shape& sh, cudaStream_t s) {
    static SmemGrant grant;
    if (cudaError_t e = grant.ask(rmsnorm_bwd_kernel<E, NC>, kRing)) return e;
    return launch_pdl(rmsnorm_bwd_kernel<E, NC>, dim3(sh.grid), dim3(sh.threads), sh.smem, s, p, sh.tpr, sh.stages);
}

template <typename E>
cudaError_t bwd_e(const RmsNormGrad& p, const Shape& sh, cudaStream_t s) {
    switch (sh.nc) {
        case 1: return bwd<E, 1>(p, sh, s);
        case 2: return bwd<E, 2>(p, sh, s);
        case 3: return bwd<E, 3>(p, sh, s);
        case 4: return bwd<E, 4>(p, sh, s);
        case 5: return bwd<E, 5>(p, sh, s);
        default: return bwd<E, 6>(p, sh, s);
    }
}

}  // namespace

cudaError_t launch_rmsnorm(int dtype, const RmsNorm& p, cudaStream_t s) {
    if (dtype == RM_BF16) return p.R ? fwd_e<__nv_bfloat16, true>(p, s) : fwd_e<__nv_bfloat16, false>(p, s);
    return p.R ? fwd_e<float, true>(p, s) : fwd_e<float, false>(p, s);
}

// Partial rows of the column sums: one a CTA, one CTA an SM.
int rmsnorm_bwd_parts(long long rows) { return (int)std::min<long long>(rows, kSms); }

cudaError_t launch_rmsnorm_bwd(int dtype, const RmsNormGrad& p, float* dgamma, cudaStream_t s) {
    const Shape sh(p.rows, p.D, (dtype == RM_BF16 ? 2 : 4) * (size_t)p.D * (p.dSum ? 3 : 2));
    const cudaError_t e = dtype == RM_BF16 ? bwd_e<__nv_bfloat16>(p, sh, s) : bwd_e<float>(p, sh, s);
    if (e != cudaSuccess || !dgamma) return e;
    return launch_pdl(colsum_parts_kernel, dim3((p.D + 31) / 32), dim3(1024), 0, s, (const float*)p.part, dgamma, sh.grid,
                      p.D);
}

}  // namespace rm
