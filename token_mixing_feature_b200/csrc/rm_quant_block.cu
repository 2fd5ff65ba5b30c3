// Block quantiser: e4m3 codes with one power-of-two scale for each block of
// 1 x 128 (or 128 x 128) of a matrix, and / or the same for its transpose, in
// one read of the matrix.
//
// A linear layer's three products want K-major operands quantised along K:
// X by rows (forward) and by columns (weight gradient), W in 128 x 128 blocks
// both ways (a square block is its own transpose's block, so W^T has the codes
// and scales of W moved, and the input gradient multiplies exactly the weights
// that the forward pass did).  HBM-bound: 2 (or 4) bytes in, 1 or 2 out.
//
// One CTA per 128 x 128 tile, 256 threads, each holding an 8 x 8 patch in
// registers: rows 8 (t / 16) .. + 8, columns 8 (t % 16) .. + 8.  A row's 128
// columns are 16 neighbouring lanes (256-byte loads of bf16); a patch column
// is 8 consecutive bytes of the transposed output, which is turned through
// shared memory so that it leaves in 16-byte pieces.
#include <cuda_bf16.h>

#include "rm_mx.cuh"

namespace rm {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t max16(uint32_t m) {   // over the 16 lanes of a row
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

template <typename E>
struct Patch;   // 8 x 8 elements as they were loaded
template <>
struct Patch<__nv_bfloat16> {
    uint4 u[8];
    __device__ __forceinline__ void load(int r, const __nv_bfloat16* p) { u[r] = __ldcg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void zero(int r) { u[r] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ float at(int r, int c) const {
        const uint32_t w = c < 2 ? u[r].x : c < 4 ? u[r].y : c < 6 ? u[r].z : u[r].w;
        return __uint_as_float(c & 1 ? w & 0xffff0000u : w << 16);
    }
};
template <>
struct Patch<float> {
    float4 u[8][2];
    __device__ __forceinline__ void load(int r, const float* p) {
        u[r][0] = __ldcg(reinterpret_cast<const float4*>(p));
        u[r][1] = __ldcg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void zero(int r) { u[r][0] = u[r][1] = make_float4(0, 0, 0, 0); }
    __device__ __forceinline__ float at(int r, int c) const {
        const float4 v = u[r][c >> 2];
        return (c & 3) == 0 ? v.x : (c & 3) == 1 ? v.y : (c & 3) == 2 ? v.z : v.w;
    }
};

template <typename E, bool TILE>
__global__ void __launch_bounds__(kThreads) quant_block_kernel(const QuantBlock p) {
    __shared__ uint32_t wmax[kThreads / 32];
    __shared__ uint32_t cmax[kThreads / 32][kBlk];
    __shared__ __align__(16) unsigned char turn[kBlk * kBlk];
    pdl_enter();
    const int tcol = (p.cols + kBlk - 1) / kBlk, trow = (p.rows + kBlk - 1) / kBlk;
    long long tile = blockIdx.x;
    const int cb = (int)(tile % tcol);
    tile /= tcol;
    const int rb = (int)(tile % trow);
    const long long g = tile / trow;
    const int lane16 = threadIdx.x & 15, pr = threadIdx.x >> 4, warp = threadIdx.x >> 5;
    const int r0 = rb * kBlk + 8 * pr, c0 = cb * kBlk + 8 * lane16;
    const bool cin = c0 < p.cols;   // (cols is a multiple of 16: whole chunks)
    Patch<E> x;
    const E* src = static_cast<const E*>(p.src) + g * p.src_gs + (long long)r0 * p.src_ld + c0;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        if (cin && r0 + r < p.rows) x.load(r, src + (long long)r * p.src_ld);
        else x.zero(r);
    }

    uint32_t tb = 0;   // the tile's scale byte (TILE)
    if constexpr (TILE) {
        uint32_t m = 0;
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
            for (int c = 0; c < 8; ++c) m = max(m, abs_bits(x.at(r, c)));
        m = __reduce_max_sync(0xffffffffu, m);
        if ((threadIdx.x & 31) == 0) wmax[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) m = max(m, wmax[w]);
        tb = scale_byte(m);
        if (threadIdx.x == 0) {
            if (p.dst) p.scale[g * p.s_gs + rb * p.s_ld + cb] = (uint8_t)tb;
            if (p.dst_t) p.scale_t[g * p.st_gs + cb * p.st_ld + rb] = (uint8_t)tb;
        }
    }

    if (p.dst) {
        uint8_t* dst = static_cast<uint8_t*>(p.dst) + g * p.dst_gs + (long long)r0 * p.dst_ld + c0;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            uint32_t b = tb;
            if constexpr (!TILE) {
                uint32_t m = 0;
#pragma unroll
                for (int c = 0; c < 8; ++c) m = max(m, abs_bits(x.at(r, c)));
                b = scale_byte(max16(m));
            }
            if (r0 + r >= p.rows) continue;   // (one row per half-warp; all shuffles of it are done)
            const float inv = scale_inverse(min(b, 254u));
            uint2 q = make_uint2(e4m3x4(x.at(r, 0) * inv, x.at(r, 1) * inv, x.at(r, 2) * inv, x.at(r, 3) * inv),
                                 e4m3x4(x.at(r, 4) * inv, x.at(r, 5) * inv, x.at(r, 6) * inv, x.at(r, 7) * inv));
            if (b == 255u) q = make_uint2(kNanCodes, kNanCodes);
            if (cin) *reinterpret_cast<uint2*>(dst + (long long)r * p.dst_ld) = q;
            if (!TILE && lane16 == 0) p.scale[g * p.s_gs + (r0 + r) * p.s_ld + cb] = (uint8_t)b;
        }
    }

    if (p.dst_t) {
        uint32_t b[8];
        if constexpr (TILE) {
#pragma unroll
            for (int c = 0; c < 8; ++c) b[c] = tb;
        } else {   // each column's largest magnitude over the tile's 128 rows
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                uint32_t m = 0;
#pragma unroll
                for (int r = 0; r < 8; ++r) m = max(m, abs_bits(x.at(r, c)));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 16));
                if ((threadIdx.x & 31) < 16) cmax[warp][8 * lane16 + c] = m;
            }
            __syncthreads();
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                uint32_t m = 0;
#pragma unroll
                for (int w = 0; w < kThreads / 32; ++w) m = max(m, cmax[w][8 * lane16 + c]);
                b[c] = scale_byte(m);
                if (pr == 0 && cin) p.scale_t[g * p.st_gs + (c0 + c) * p.st_ld + rb] = (uint8_t)b[c];
            }
        }
        // Column c of the patch: 8 bytes at slot pr of the column's 16 slots,
        // the slots permuted by the patch's column so that the 16 lanes of a
        // store meet 16 different bank pairs.
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float inv = scale_inverse(min(b[c], 254u));
            uint2 q = make_uint2(e4m3x4(x.at(0, c) * inv, x.at(1, c) * inv, x.at(2, c) * inv, x.at(3, c) * inv),
                                 e4m3x4(x.at(4, c) * inv, x.at(5, c) * inv, x.at(6, c) * inv, x.at(7, c) * inv));
            if (b[c] == 255u) q = make_uint2(kNanCodes, kNanCodes);
            *reinterpret_cast<uint2*>(turn + (8 * lane16 + c) * kBlk + ((pr ^ lane16) << 3)) = q;
        }
        __syncthreads();
        uint8_t* dst = static_cast<uint8_t*>(p.dst_t) + g * p.dt_gs;
#pragma unroll
        for (int i = 0; i < kBlk * 8 / kThreads; ++i) {   // 16-byte pieces: 8 per column
            const int k = threadIdx.x + i * kThreads, c = k >> 3, q = k & 7, sw = (c >> 3) & 15;
            const int col = cb * kBlk + c, row = rb * kBlk + 16 * q;
            if (col >= p.cols || row >= p.rows) continue;
            uint4 v = *reinterpret_cast<const uint4*>(turn + c * kBlk + (((2 * q) ^ (sw & 14)) << 3));
            if (sw & 1) v = make_uint4(v.z, v.w, v.x, v.y);
            uint8_t* out = dst + (long long)col * p.dt_ld + row;
            if (row + 16 <= p.rows) {
                *reinterpret_cast<uint4*>(out) = v;
            } else {   // the row's last bytes: what lies behind them stays as it was
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (row + j < p.rows) out[j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
            }
        }
    }
}

}  // namespace

cudaError_t launch_quant_block(int dtype, const QuantBlock& p, int block_rows, cudaStream_t s) {
    const long long tiles = (long long)p.G * ((p.rows + kBlk - 1) / kBlk) * ((p.cols + kBlk - 1) / kBlk);
    if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)tiles), block(kThreads);
    if (dtype == RM_BF16)
        return block_rows == 1 ? launch_pdl(quant_block_kernel<__nv_bfloat16, false>, grid, block, 0, s, p)
                               : launch_pdl(quant_block_kernel<__nv_bfloat16, true>, grid, block, 0, s, p);
    return block_rows == 1 ? launch_pdl(quant_block_kernel<float, false>, grid, block, 0, s, p)
                           : launch_pdl(quant_block_kernel<float, true>, grid, block, 0, s, p);
}

}  // namespace rm
