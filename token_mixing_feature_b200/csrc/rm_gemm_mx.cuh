// Shared by the two kernels of the block-scaled 8-bit product: arguments,
// activations, waits and launch helpers.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "rm_mx.cuh"
#include "rm_tmap.h"

namespace rm {

struct MxParams {
    int G, M, N, K;
    int a_g_inner, w_g_inner;   // map coordinate order (k, g, row) if 1, else (k, row, g)
    int a_gmul, w_gmul;         // 0: the operand is shared by all groups
    const uint8_t* a_scale;
    long long as_gs, as_ld;
    const uint8_t* w_scale;
    long long ws_gs, ws_ld;
    int w_shift;                // row n's scales are row n >> w_shift of w_scale
    const float* bias;
    const void* resid;
    long long r_gs, r_ld;       // (few-row kernel)
    int o_g_inner, r_g_inner;   // map coordinate orders of out and resid (pair kernel)
    int r_gmul;
    long long o_gs, o_ld;       // (few-row kernel)
    uint8_t* out_scale;
    long long os_gs, os_ld;
    int act;
    DeviceErr err;
    unsigned long long budget_ns;
};

__device__ __forceinline__ float exp2_approx(float x) {   // within 2^-22 of the value
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 exp2_pair(float2 x) { return make_float2(exp2_approx(x.x), exp2_approx(x.y)); }
__device__ __forceinline__ float2 rcp_pair(float2 x) {
    float2 y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(x.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(x.y));
    return y;
}

// act(v) of a pair, without branches.  GELU's tanh form is v * sigmoid(2u), u =
// sqrt(2/pi) (v + 0.044715 v^3), which loses nothing where GELU is small, for every
// type of result: v/2 + v/2 tanh(u) cancels there, and with tanh.approx (2^-11) bf16
// results were 4.5 % off at v = -4.5 and zero from -5 on.  The erf form
// is v Phi(v), Phi(-a) = erfc(a / sqrt(2)) / 2 = t Q(t) exp(-a^2 / 2) with t = 1 / (1 +
// a / (2 sqrt(2))) and Q of degree 8, fitted here to erfcx(a / sqrt(2)) / (2 t) with a
// minimax relative error of 4e-8 (iteratively reweighted least squares over 0 <= a <=
// 14.8); the exponent is carried in two floats.  All of it is good to 5e-7 of the value
// down to v = -6, 1.5e-6 to where fp32 ends (v = -13).  (Abramowitz and Stegun's 7.1.26
// has 1.5e-7 of 1: 5e-5 of the value at v = -3, 2e-3 at -5.)
template <int ACT>
__device__ __forceinline__ float2 activation(float2 v) {
    if constexpr (ACT == RM_ACT_GELU_TANH) {
        const float c = -2.0f * 0.7978845608028654f * 1.4426950408889634f;   // -2 sqrt(2/pi) log2(e)
        const float2 e = exp2_pair(f2_mul(v, f2_fma(f2_mul(v, v), f2(c * 0.044715f), f2(c))));
        return f2_mul(v, rcp_pair(f2_add(e, f2(1.0f))));
    } else if constexpr (ACT == RM_ACT_GELU_ERF) {
        // (behind 16 Phi(-a) is below fp32: nothing overflows)
        const float2 a = make_float2(fminf(fabsf(v.x), 16.f), fminf(fabsf(v.y), 16.f));
        const float2 t = rcp_pair(f2_fma(a, f2(0.35355339059327379f), f2(1.0f)));
        float2 q = f2(-0.029596666f);
        q = f2_fma(t, q, f2(0.14259142f));
        q = f2_fma(t, q, f2(-0.24423045f));
        q = f2_fma(t, q, f2(0.1397563f));
        q = f2_fma(t, q, f2(-0.013811729f));
        q = f2_fma(t, q, f2(0.10155497f));
        q = f2_fma(t, q, f2(0.12149831f));
        q = f2_fma(t, q, f2(0.14119503f));
        q = f2_fma(t, q, f2(0.14104278f));
        // exp(-a^2 / 2) = exp2(n + r): n the product as it is rounded, r what that
        // and the constant's own rounding left
        const float c = -0.5f * 1.4426950408889634f, c_low = -9.629815e-09f;
        const float2 y = f2_mul(a, a), n = f2_mul(y, f2(c));
        const float2 minus_y = make_float2(-y.x, -y.y), minus_n = make_float2(-n.x, -n.y);
        const float2 r = f2_fma(f2_fma(a, a, minus_y), f2(c), f2_fma(y, f2(c_low), f2_fma(y, f2(c), minus_n)));
        const float2 e = exp2_pair(n);
        const float2 hc = f2_mul(f2_mul(q, t), f2_fma(f2_mul(r, f2(0.6931471805599453f)), e, e));   // Phi(-a)
        return f2_mul(v, make_float2(v.x < 0.f ? hc.x : 1.0f - hc.x, v.y < 0.f ? hc.y : 1.0f - hc.y));
    } else {
        return make_float2(v.x < 0.f ? 0.f : v.x, v.y < 0.f ? 0.f : v.y);   // (keeps NaN)
    }
}
template <int ACT, int NV>
__device__ __forceinline__ void activate(float (&v)[NV]) {
#pragma unroll
    for (int e = 0; e < NV; e += 2) {
        const float2 y = activation<ACT>(make_float2(v[e], v[e + 1]));
        v[e] = y.x, v[e + 1] = y.y;
    }
}

// For waits on this CTA's own copies and MMAs in flight, which no short budget
// may cut off: a second at the least.
__device__ __forceinline__ WaitCtx drain_ctx(const WaitCtx& w) {
    return WaitCtx{w.abort, w.budget_ns > 1000000000ull ? w.budget_ns : 1000000000ull, w.err};
}

// A wait of a whole warp: all lanes go on, or none.  warp_wait parks (CLUSTER: for
// what the pair's other CTA released), warp_mx_wait polls where the budget is short.
template <bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtx& w, int site) {
    return __all_sync(0xffffffffu, CLUSTER ? mbar_wait_cluster(bar, parity, w, site) : mbar_wait(bar, parity, w, site));
}
__device__ __forceinline__ bool warp_mx_wait(uint32_t bar, uint32_t parity, const WaitCtx& w, int site) {
    return __all_sync(0xffffffffu, mx_wait(bar, parity, w, site));
}

// Map of [G][rows][cols] elements of esz bytes with a box of `box` rows x 128
// bytes: dims (cols, rows, groups) with the smaller of the two strides first.
// A single row or group takes any legal stride; a group stride of 0 is an
// input that all groups share.
inline bool matrix_map(CUtensorMap* m, const void* base, int cols, int rows, int G, long long ld, long long gs, int esz,
                uint32_t box, int* g_inner, int* gmul) {
    if (gmul) *gmul = gs == 0 ? 0 : 1;
    if (gs == 0) G = 1;
    if (rows == 1) ld = ((long long)cols + 15) / 16 * 16;
    if (G == 1) gs = ld;
    *g_inner = gs < ld ? 1 : 0;
    return *g_inner ? make_map_e(m, base, cols, G, rows, gs * esz, ld * esz, 1, box, esz)
                    : make_map_e(m, base, cols, rows, G, ld * esz, gs * esz, box, 1, esz);
}

// Programmatic launch with clusters of `cluster` CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t s,
                           Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Few rows (rm_gemm_mx_few.cu).
cudaError_t launch_gemm_mx_few(const rm_matmul_fp8_args& a, MxParams& p, int num_sms, cudaStream_t s);

}  // namespace rm
