// C ABI of the block-scaled 8-bit linear layer (include/rankmixer.h): argument
// checks and launches.  No handle: the sizes come with each call, and the only
// scratch is the caller's.
#include <cuda_runtime.h>

#include <cstdint>

#include "rm_internal.h"

namespace {

inline bool al(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool al16(const void* p) { return p && al(p, 16); }
inline bool al16_or_null(const void* p) { return al(p, 16); }
inline rm_status cuda_status(cudaError_t e) { return e == cudaSuccess ? RM_OK : RM_ERR_CUDA; }
inline long long blocks(long long n) { return (n + 127) / 128; }

// Strides of n rows of `cols` elements of esz bytes (16-byte rows that do not
// overlap), of n groups of them (16-byte starts; 0: the groups share one, for
// inputs), and of n rows of scale bytes.  One row or group has no stride.
inline bool row_stride(long long ld, long long n, long long cols, int esz) {
    return n == 1 || (ld >= cols && (ld * esz) % 16 == 0 && ld < (1LL << 36));
}
inline bool group_stride(long long gs, long long n, int esz, bool input = false) {
    return n == 1 || ((gs > 0 || (input && gs == 0)) && (gs * esz) % 16 == 0 && gs < (1LL << 36));
}
inline bool scale_stride(long long gs, long long ng, long long ld, long long n, long long cols, bool input = false) {
    return (n == 1 || (ld >= blocks(cols) && ld < (1LL << 36))) &&
           (ng == 1 || ((gs > 0 || (input && gs == 0)) && gs < (1LL << 36)));
}

// Tensor-core kernels need the SM count of the current device; asked once per device.
int sm_count() {
    static int count[64];   // 0: not asked yet (every thread would write the same value)
    int d = 0, n = 0;
    if (cudaGetDevice(&d) != cudaSuccess) return 0;
    if (d < 64 && __atomic_load_n(&count[d], __ATOMIC_RELAXED)) return __atomic_load_n(&count[d], __ATOMIC_RELAXED);
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d) != cudaSuccess) return 0;
    if (d < 64) __atomic_store_n(&count[d], n, __ATOMIC_RELAXED);
    return n;
}

}  // namespace

extern "C" {

rm_status rm_rmsnorm_forward(const rm_rmsnorm_args* a, rm_stream_t stream) {
    if (!a || (a->dtype != RM_BF16 && a->dtype != RM_F32) || a->rows < 0 || a->D < 1 || !(a->eps >= 0.f))
        return RM_ERR_INVALID_ARG;
    if (a->D % 16 || a->D > 16384 || a->rows > 0x7fffffffLL) return RM_ERR_UNSUPPORTED;
    const int esz = a->dtype == RM_BF16 ? 2 : 4;
    if (a->rows == 0) return RM_OK;   // (before the pointers: an empty array's may be null)
    if ((a->Yq == nullptr) != (a->Ys == nullptr)) return RM_ERR_INVALID_ARG;
    if (!a->Sum && !a->Y && !a->Yq && !a->rstd) return RM_ERR_INVALID_ARG;
    if (!al16(a->X) || !row_stride(a->ld_x, a->rows, a->D, esz) || !al16_or_null(a->gamma) || !al(a->rstd, 4))
        return RM_ERR_INVALID_ARG;
    if (a->R && (!al16(a->R) || !row_stride(a->ld_r, a->rows, a->D, esz))) return RM_ERR_INVALID_ARG;
    if (a->Sum && (!al16(a->Sum) || !row_stride(a->ld_sum, a->rows, a->D, esz))) return RM_ERR_INVALID_ARG;
    if (a->Y && (!al16(a->Y) || !row_stride(a->ld_y, a->rows, a->D, esz))) return RM_ERR_INVALID_ARG;
    if (a->Yq && (!al16(a->Yq) || !row_stride(a->ld_yq, a->rows, a->D, 1) || !scale_stride(0, 1, a->ld_ys, a->rows, a->D)))
        return RM_ERR_INVALID_ARG;
    rm::RmsNorm p{};
    p.X = a->X, p.R = a->R, p.gamma = a->gamma, p.Sum = a->Sum, p.Y = a->Y, p.Yq = a->Yq, p.Ys = a->Ys;
    p.rstd = a->rstd;
    p.ld_x = a->ld_x, p.ld_r = a->ld_r, p.ld_sum = a->ld_sum, p.ld_y = a->ld_y, p.ld_yq = a->ld_yq, p.ld_ys = a->ld_ys;
    p.rows = a->rows, p.D = a->D, p.eps = a->eps;
    return cuda_status(rm::launch_rmsnorm(a->dtype, p, stream));
}

size_t rm_rmsnorm_backward_workspace_bytes(long long rows, int D) {
    if (rows < 1 || D < 1 || D % 16 || D > 16384) return 0;
    return sizeof(float) * (size_t)rm::rmsnorm_bwd_parts(rows) * D;
}

rm_status rm_rmsnorm_backward(const rm_rmsnorm_grad_args* a, rm_stream_t stream) {
    if (!a || (a->dtype != RM_BF16 && a->dtype != RM_F32) || a->rows < 0 || a->D < 1) return RM_ERR_INVALID_ARG;
    if (a->D % 16 || a->D > 16384 || a->rows > 0x7fffffffLL) return RM_ERR_UNSUPPORTED;
    const int esz = a->dtype == RM_BF16 ? 2 : 4;
    if (a->dgamma && !al16(a->dgamma)) return RM_ERR_INVALID_ARG;
    if (a->rows == 0)   // no rows: the sum over them is zero
        return a->dgamma ? cuda_status(cudaMemsetAsync(a->dgamma, 0, sizeof(float) * a->D, stream)) : RM_OK;
    if (!al16(a->dY) || !al16(a->S) || !al16(a->dX) || !a->rstd || !al(a->rstd, 4) || !al16_or_null(a->gamma))
        return RM_ERR_INVALID_ARG;
    if (!row_stride(a->ld_dy, a->rows, a->D, esz) || !row_stride(a->ld_s, a->rows, a->D, esz) || !row_stride(a->ld_dx, a->rows, a->D, esz))
        return RM_ERR_INVALID_ARG;
    if (a->dSum && (!al16(a->dSum) || !row_stride(a->ld_dsum, a->rows, a->D, esz))) return RM_ERR_INVALID_ARG;
    if (a->dgamma && (!al16(a->workspace) || a->workspace_bytes < rm_rmsnorm_backward_workspace_bytes(a->rows, a->D)))
        return RM_ERR_INVALID_ARG;
    rm::RmsNormGrad p{};
    p.dY = a->dY, p.S = a->S, p.dSum = a->dSum, p.gamma = a->gamma, p.rstd = a->rstd, p.dX = a->dX;
    p.part = a->dgamma ? static_cast<float*>(a->workspace) : nullptr;
    p.ld_dy = a->ld_dy, p.ld_s = a->ld_s, p.ld_dsum = a->ld_dsum, p.ld_dx = a->ld_dx;
    p.rows = a->rows, p.D = a->D;
    return cuda_status(rm::launch_rmsnorm_bwd(a->dtype, p, a->dgamma, stream));
}

rm_status rm_quantize_fp8_block(const rm_quant_block_args* a, rm_stream_t stream) {
    if (!a || (a->dtype != RM_BF16 && a->dtype != RM_F32) || a->G < 0 || a->rows < 0 || a->cols < 1)
        return RM_ERR_INVALID_ARG;
    if (a->block_rows != 1 && a->block_rows != 128) return RM_ERR_INVALID_ARG;
    if (a->cols % 16) return RM_ERR_UNSUPPORTED;
    if (a->rows > 0x7fffff00 || a->cols > 0x7fffff00 || (double)a->G * blocks(a->rows) * blocks(a->cols) > 2147483647.0)
        return RM_ERR_UNSUPPORTED;
    if (a->G == 0 || a->rows == 0) return RM_OK;
    if ((!a->dst && !a->dst_t) || (a->dst == nullptr) != (a->scale == nullptr) ||
        (a->dst_t == nullptr) != (a->scale_t == nullptr))
        return RM_ERR_INVALID_ARG;
    const int esz = a->dtype == RM_BF16 ? 2 : 4, br = a->block_rows;
    if (!al16(a->src) || !row_stride(a->src_ld, a->rows, a->cols, esz) ||
        !group_stride(a->src_gstride, a->G, esz, true))
        return RM_ERR_INVALID_ARG;
    if (a->dst && (!al16(a->dst) || !row_stride(a->dst_ld, a->rows, a->cols, 1) ||
                   !group_stride(a->dst_gstride, a->G, 1) ||
                   !scale_stride(a->scale_gstride, a->G, a->scale_ld, (a->rows + br - 1) / br, a->cols)))
        return RM_ERR_INVALID_ARG;
    if (a->dst_t && (!al16(a->dst_t) || !row_stride(a->dst_t_ld, a->cols, a->rows, 1) ||
                     !group_stride(a->dst_t_gstride, a->G, 1) ||
                     !scale_stride(a->scale_t_gstride, a->G, a->scale_t_ld, (a->cols + br - 1) / br, a->rows)))
        return RM_ERR_INVALID_ARG;
    rm::QuantBlock p{};
    p.src = a->src, p.src_gs = a->src_gstride, p.src_ld = a->src_ld;
    p.G = a->G, p.rows = a->rows, p.cols = a->cols;
    p.dst = a->dst, p.dst_gs = a->dst_gstride, p.dst_ld = a->dst_ld;
    p.scale = a->scale, p.s_gs = a->scale_gstride, p.s_ld = a->scale_ld;
    p.dst_t = a->dst_t, p.dt_gs = a->dst_t_gstride, p.dt_ld = a->dst_t_ld;
    p.scale_t = a->scale_t, p.st_gs = a->scale_t_gstride, p.st_ld = a->scale_t_ld;
    return cuda_status(rm::launch_quant_block(a->dtype, p, br, stream));
}

rm_status rm_matmul_fp8_block(const rm_matmul_fp8_args* a, rm_stream_t stream) {
    if (!a || a->G < 0 || a->M < 0 || a->N < 1 || a->K < 1) return RM_ERR_INVALID_ARG;
    if (a->out_dtype != RM_BF16 && a->out_dtype != RM_F32 && a->out_dtype != RM_E4M3) return RM_ERR_INVALID_ARG;
    if (a->act < RM_ACT_GELU_TANH || a->act > RM_ACT_NONE) return RM_ERR_INVALID_ARG;
    if (a->w_block_rows != 1 && a->w_block_rows != 128) return RM_ERR_INVALID_ARG;
    if (a->N % 16 || a->M > 0x7fffff00 || a->N > 0x7fffff00 || a->K > 0x7fffff00) return RM_ERR_UNSUPPORTED;
    if ((double)a->G * blocks(a->M) * blocks(a->N) > 2147483647.0) return RM_ERR_UNSUPPORTED;
    if (a->G == 0 || a->M == 0) return RM_OK;
    const int osz = a->out_dtype == RM_F32 ? 4 : a->out_dtype == RM_BF16 ? 2 : 1;
    if (!al16(a->A) || !al16(a->W) || !al16(a->out) || !a->a_scale || !a->w_scale) return RM_ERR_INVALID_ARG;
    const long long w_rows = ((long long)a->N + a->w_block_rows - 1) / a->w_block_rows;
    if (!row_stride(a->a_ld, a->M, a->K, 1) || !group_stride(a->a_gstride, a->G, 1, true) ||
        !scale_stride(a->as_gstride, a->G, a->as_ld, a->M, a->K, true))
        return RM_ERR_INVALID_ARG;
    if (!row_stride(a->w_ld, a->N, a->K, 1) || !group_stride(a->w_gstride, a->G, 1, true) ||
        !scale_stride(a->ws_gstride, a->G, a->ws_ld, w_rows, a->K, true))
        return RM_ERR_INVALID_ARG;
    if (!row_stride(a->o_ld, a->M, a->N, osz) || !group_stride(a->o_gstride, a->G, osz)) return RM_ERR_INVALID_ARG;
    if (a->out_dtype == RM_E4M3) {
        if (!a->out_scale || a->resid || !scale_stride(a->os_gstride, a->G, a->os_ld, a->M, a->N))
            return RM_ERR_INVALID_ARG;
    } else if (a->resid) {
        if (!al16(a->resid) || !row_stride(a->r_ld, a->M, a->N, osz) || !group_stride(a->r_gstride, a->G, osz, true))
            return RM_ERR_INVALID_ARG;
    }
    if (!al16_or_null(a->bias) || !al(a->device_status, 4)) return RM_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms < 2) return RM_ERR_CUDA;
    return cuda_status(rm::launch_gemm_mx(*a, sms, stream));
}

int rm_internal_matmul_fp8_few_rows(const rm_matmul_fp8_args* a, int num_sms) {
    return rm::gemm_mx_few_rows(*a, num_sms) ? 1 : 0;
}

}  // extern "C"
