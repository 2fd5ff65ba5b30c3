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
// Both directions are bound by HBM: a row is read once into registers, the
// statistics are fp32 sums, and everything leaves from the registers.  A row
// belongs to TPR consecutive threads of a CTA, each holding NC chunks of 8
// consecutive elements (one or two 16-byte loads), so a block of 128 is 16
// neighbouring lanes and its largest magnitude costs four shuffles.
#include <cuda_bf16.h>

#include <algorithm>

#include "rm_mx.cuh"

namespace rm {
namespace {

constexpr int kMinCta = 256;   // threads a CTA has at least (several rows for narrow ones)

// Eight consecutive elements as floats, and back (bf16 rounded to nearest even).
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 u = __ldcg(reinterpret_cast<const uint4*>(p));
    float2 f[4];
    unpack_pairs(u, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = f[i].x, v[2 * i + 1] = f[i].y;
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = __ldcg(reinterpret_cast<const float4*>(p)), b = __ldcg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                              pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Sum over the TPR threads of a row (every thread gets it).  red: one float
// per warp of the CTA; all threads of the CTA call this together.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = warp_sum(v);
    if constexpr (TPR > 32) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) red[warp] = v;
        __syncthreads();
        const float* r = red + warp / (TPR / 32) * (TPR / 32);
        v = 0.f;
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) v += r[w];
    }
    return v;
}

template <typename E, int TPR, int NC>
__global__ void __launch_bounds__(TPR > kMinCta ? TPR : kMinCta) rmsnorm_kernel(const RmsNorm p) {
    constexpr int CTA = TPR > kMinCta ? TPR : kMinCta;
    __shared__ float red[CTA / 32];
    pdl_enter();
    const int t = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * (CTA / TPR) + threadIdx.x / TPR;
    const bool live = row < p.rows;
    const int nch = p.D / 8;
    float v[NC][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = t + i * TPR;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
        if (live && c < nch) load8(static_cast<const E*>(p.X) + row * p.ld_x + 8 * c, v[i]);
    }
    if (p.R) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = t + i * TPR;
            if (live && c < nch) {
                float r[8];
                load8(static_cast<const E*>(p.R) + row * p.ld_r + 8 * c, r);
                // the stream is rounded to its type here: the statistics, the
                // output and the gradient all see the values that are stored
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] = to_f(from_f<E>(v[i][e] + r[e]));
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = t + i * TPR;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e], v[i][e], ss);
        if (p.Sum && live && c < nch) store8(static_cast<E*>(p.Sum) + row * p.ld_sum + 8 * c, v[i]);
    }
    ss = row_sum<TPR>(ss, red);
    const float rstd = 1.0f / sqrtf(ss / (float)p.D + p.eps);
    if (!live) return;
    if (p.rstd && t == 0) p.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = t + i * TPR;
        const bool in = c < nch;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = v[i][e] * rstd;
        if (in && p.gamma) {
            const float4 a = reinterpret_cast<const float4*>(p.gamma + 8 * c)[0];
            const float4 b = reinterpret_cast<const float4*>(p.gamma + 8 * c)[1];
            y[0] *= a.x, y[1] *= a.y, y[2] *= a.z, y[3] *= a.w, y[4] *= b.x, y[5] *= b.y, y[6] *= b.z, y[7] *= b.w;
        }
        if (in && p.Y) store8(static_cast<E*>(p.Y) + row * p.ld_y + 8 * c, y);
        if (p.Yq) {
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = max(m, abs_bits(y[e]));   // (zero past the row's end)
            // TPR is a multiple of 32 and `live` is one value per row: whole
            // half-warps take part
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            const uint32_t b = scale_byte(m);
            const float inv = scale_inverse(min(b, 254u));
            if (in) {
                uint2 q = make_uint2(e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                                     e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
                if (b == 255u) q = make_uint2(kNanCodes, kNanCodes);
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.Yq) + row * p.ld_yq + 8 * c) = q;
                if ((threadIdx.x & 15) == 0) p.Ys[row * p.ld_ys + c / 16] = (uint8_t)b;
            }
        }
    }
}

// Gradient: a CTA walks rows (grid-stride) and keeps its columns' sums of
// dy * s * rstd in registers; they leave as one partial row per CTA.
template <typename E, int TPR, int NC>
__global__ void __launch_bounds__(TPR > kMinCta ? TPR : kMinCta) rmsnorm_bwd_kernel(const RmsNormGrad p) {
    constexpr int CTA = TPR > kMinCta ? TPR : kMinCta;
    constexpr int RPC = CTA / TPR;
    __shared__ float red[2][CTA / 32];
    extern __shared__ float acc_s[];   // [D]: the CTA's column sums (RPC > 1)
    pdl_enter();
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int nch = p.D / 8;
    float g[NC][8], acc[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = t + i * TPR;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            acc[i][e] = 0.f;
            g[i][e] = 1.f;
        }
        if (p.gamma && c < nch) {
            const float* q = p.gamma + 8 * c;
#pragma unroll
            for (int e = 0; e < 8; ++e) g[i][e] = q[e];
        }
    }
    int par = 0;
    for (long long r0 = (long long)blockIdx.x * RPC; r0 < p.rows; r0 += (long long)gridDim.x * RPC, par ^= 1) {
        const long long row = r0 + grp;
        const bool live = row < p.rows;
        float s[NC][8], a[NC][8];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = t + i * TPR;
#pragma unroll
            for (int e = 0; e < 8; ++e) s[i][e] = a[i][e] = 0.f;
            if (live && c < nch) {
                load8(static_cast<const E*>(p.S) + row * p.ld_s + 8 * c, s[i]);
                load8(static_cast<const E*>(p.dY) + row * p.ld_dy + 8 * c, a[i]);
            }
        }
        const float rstd = live ? __ldcg(p.rstd + row) : 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                acc[i][e] = fmaf(a[i][e] * rstd, s[i][e], acc[i][e]);
                a[i][e] *= g[i][e];
                dot = fmaf(a[i][e], s[i][e], dot);
            }
        }
        dot = row_sum<TPR>(dot, red[par]);
        const float k = -rstd * rstd * (dot / (float)p.D);
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = t + i * TPR;
            if (c < nch) {
                float d[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] = rstd * fmaf(s[i][e], k, a[i][e]);
                if (p.dSum) {
                    float u[8];
                    load8(static_cast<const E*>(p.dSum) + row * p.ld_dsum + 8 * c, u);
#pragma unroll
                    for (int e = 0; e < 8; ++e) d[e] += u[e];
                }
                store8(static_cast<E*>(p.dX) + row * p.ld_dx + 8 * c, d);
            }
        }
    }
    if (!p.part) return;
    if constexpr (RPC > 1) {   // the CTA's rows in a fixed order
        for (int k = 0; k < RPC; ++k) {
            __syncthreads();
            if (grp == k) {
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    const int c = t + i * TPR;
                    if (c < nch)
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            if (k) acc[i][e] += acc_s[8 * c + e];
                            if (k < RPC - 1) acc_s[8 * c + e] = acc[i][e];
                        }
                }
            }
        }
    }
    if (grp == RPC - 1) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = t + i * TPR;
            if (c < nch) store8(p.part + (long long)blockIdx.x * p.D + 8 * c, acc[i]);
        }
    }
}

// dgamma[d] = sum over the partial rows, in a fixed order: 32 columns a CTA,
// 32 warps taking every 32nd row, then the warps' sums.
__global__ void __launch_bounds__(1024) colsum_parts_kernel(const float* part, float* out, int parts, int D) {
    __shared__ float s[32][33];
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int d = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (d < D)
        for (int r = warp; r < parts; r += 32) v += __ldcg(part + (long long)r * D + d);
    s[warp][lane] = v;
    __syncthreads();
    v = warp_sum(s[lane][warp]);
    if (lane == 0 && blockIdx.x * 32 + warp < D) out[blockIdx.x * 32 + warp] = v;
}

// Threads per row: the fewest (of 32 .. 512) that hold the row in at most
// `most` chunks each.
int pick_tpr(int D, int most) {
    int tpr = 32;
    while (tpr < 512 && (D / 8 + tpr - 1) / tpr > most) tpr *= 2;
    return tpr;
}

template <typename E, int TPR, int NC>
cudaError_t fwd(const RmsNorm& p, cudaStream_t s) {
    const int rpc = TPR > kMinCta ? 1 : kMinCta / TPR;
    return launch_pdl(rmsnorm_kernel<E, TPR, NC>, dim3((unsigned)((p.rows + rpc - 1) / rpc)), dim3(rpc * TPR), 0, s, p);
}
template <typename E, int TPR>
cudaError_t fwd_nc(const RmsNorm& p, cudaStream_t s) {
    switch ((p.D / 8 + TPR - 1) / TPR) {
        case 1: return fwd<E, TPR, 1>(p, s);
        case 2: return fwd<E, TPR, 2>(p, s);
        case 3: return fwd<E, TPR, 3>(p, s);
        case 4: return fwd<E, TPR, 4>(p, s);
        default: return cudaErrorInvalidValue;
    }
}
template <typename E>
cudaError_t fwd_e(const RmsNorm& p, cudaStream_t s) {
    switch (pick_tpr(p.D, 4)) {
        case 32: return fwd_nc<E, 32>(p, s);
        case 64: return fwd_nc<E, 64>(p, s);
        case 128: return fwd_nc<E, 128>(p, s);
        case 256: return fwd_nc<E, 256>(p, s);
        default: return fwd_nc<E, 512>(p, s);
    }
}

template <typename E, int TPR, int NC>
cudaError_t bwd(const RmsNormGrad& p, int grid, cudaStream_t s) {
    constexpr int rpc = TPR > kMinCta ? 1 : kMinCta / TPR;
    const size_t smem = rpc > 1 && p.part ? sizeof(float) * p.D : 0;   // (TPR < 256: D <= 4096, 16 KB)
    return launch_pdl(rmsnorm_bwd_kernel<E, TPR, NC>, dim3(grid), dim3(rpc * TPR), smem, s, p);
}
template <typename E, int TPR>
cudaError_t bwd_nc(const RmsNormGrad& p, int grid, cudaStream_t s) {
    switch ((p.D / 8 + TPR - 1) / TPR) {
        case 1: return bwd<E, TPR, 1>(p, grid, s);
        case 2: return bwd<E, TPR, 2>(p, grid, s);
        case 3: return bwd<E, TPR, 3>(p, grid, s);
        case 4: return bwd<E, TPR, 4>(p, grid, s);
        default: return cudaErrorInvalidValue;
    }
}
template <typename E>
cudaError_t bwd_e(const RmsNormGrad& p, int tpr, int grid, cudaStream_t s) {
    switch (tpr) {
        case 32: return bwd_nc<E, 32>(p, grid, s);
        case 64: return bwd_nc<E, 64>(p, grid, s);
        case 128: return bwd_nc<E, 128>(p, grid, s);
        case 256: return bwd_nc<E, 256>(p, grid, s);
        default: return bwd_nc<E, 512>(p, grid, s);
    }
}

}  // namespace

cudaError_t launch_rmsnorm(int dtype, const RmsNorm& p, cudaStream_t s) {
    return dtype == RM_BF16 ? fwd_e<__nv_bfloat16>(p, s) : fwd_e<float>(p, s);
}

int rmsnorm_bwd_parts(long long rows, int D) {
    const int tpr = pick_tpr(D, 4), rpc = tpr > kMinCta ? 1 : kMinCta / tpr;
    return (int)std::min<long long>((rows + rpc - 1) / rpc, 592);
}

cudaError_t launch_rmsnorm_bwd(int dtype, const RmsNormGrad& p, float* dgamma, cudaStream_t s) {
    const int tpr = pick_tpr(p.D, 4), grid = rmsnorm_bwd_parts(p.rows, p.D);
    cudaError_t e = dtype == RM_BF16 ? bwd_e<__nv_bfloat16>(p, tpr, grid, s) : bwd_e<float>(p, tpr, grid, s);
    if (e != cudaSuccess || !dgamma) return e;
    return launch_pdl(colsum_parts_kernel, dim3((p.D + 31) / 32), dim3(1024), 0, s, (const float*)p.part, dgamma, grid,
                      p.D);
}

}  // namespace rm
