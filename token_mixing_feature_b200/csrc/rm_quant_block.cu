// Block quantiser: e4m3 codes with one power-of-two scale for each block of
// 1 x 128 (or 128 x 128) of a matrix, and / or the same for its transpose, in
// one read of the matrix.
//
// A linear layer's three products want K-major operands quantised along K:
// X by rows (forward) and by columns (weight gradient), W in 128 x 128 blocks
// both ways (a square block is its own transpose's block, so W^T has the codes
// and scales of W moved, and the input gradient multiplies exactly the weights
// that the forward pass did).  HBM-bound: 2 (or 4) bytes in, 1 or 2 out (squares
// of 32 x 6144 x 1536 bf16 both ways: 182 us, 6.6 TB/s, the copy's rate).
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

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 8 x 8 elements as they were loaded, and the largest magnitude bits of a row,
// of columns, of all (ordered like the magnitudes, NaN on top).
template <typename E>
struct Patch;
template <>
struct Patch<__nv_bfloat16> {
    uint4 u[8];
    __device__ __forceinline__ void load(int r, const __nv_bfloat16* p) { u[r] = __ldcg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void zero(int r) { u[r] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ uint32_t word(int r, int i) const { return i == 0 ? u[r].x : i == 1 ? u[r].y : i == 2 ? u[r].z : u[r].w; }
    __device__ __forceinline__ float at(int r, int c) const {
        const uint32_t w = word(r, c >> 1);
        return __uint_as_float(c & 1 ? w & 0xffff0000u : w << 16);
    }
    // two 16-bit magnitudes an instruction; as fp32 bits they are the high halves
    __device__ __forceinline__ uint32_t row_max(int r) const {
        const uint32_t m = max_u16x2(max_u16x2(u[r].x & 0x7fff7fffu, u[r].y & 0x7fff7fffu),
                                    max_u16x2(u[r].z & 0x7fff7fffu, u[r].w & 0x7fff7fffu));
        return max(m << 16, m & 0xffff0000u);
    }
    __device__ __forceinline__ void col_max(uint32_t (&m)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t v = 0;
#pragma unroll
            for (int r = 0; r < 8; ++r) v = max_u16x2(v, word(r, i) & 0x7fff7fffu);
            m[2 * i] = v << 16, m[2 * i + 1] = v & 0xffff0000u;
        }
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
    __device__ __forceinline__ uint32_t row_max(int r) const {
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c) m = max(m, abs_bits(at(r, c)));
        return m;
    }
    __device__ __forceinline__ void col_max(uint32_t (&m)[8]) const {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            m[c] = 0;
#pragma unroll
            for (int r = 0; r < 8; ++r) m[c] = max(m[c], abs_bits(at(r, c)));
        }
    }
};

// Codes of four elements of a block with 1 / scale = inv.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inv) {
    return e4m3x4(f2_mul(make_float2(a, b), f2(inv)), f2_mul(make_float2(c, d), f2(inv)));
}

// 4 x 4 bytes turned: w[j] holds byte j of the four words.
__device__ __forceinline__ void turn4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t (&w)[4]) {
    const uint32_t ab0 = __byte_perm(a, b, 0x5140), ab1 = __byte_perm(a, b, 0x7362);
    const uint32_t cd0 = __byte_perm(c, d, 0x5140), cd1 = __byte_perm(c, d, 0x7362);
    w[0] = __byte_perm(ab0, cd0, 0x5410), w[1] = __byte_perm(ab0, cd0, 0x7632);
    w[2] = __byte_perm(ab1, cd1, 0x5410), w[3] = __byte_perm(ab1, cd1, 0x7632);
}

template <typename E, bool TILE>
__global__ void __launch_bounds__(kThreads, sizeof(E) == 2 ? 4 : 2) quant_block_kernel(const QuantBlock p) {
    __shared__ uint32_t wmax[kThreads / 32];
    __shared__ __align__(16) uint32_t cmax[kThreads / 32][kBlk];
    __shared__ __align__(8) uint8_t cbyte[kBlk];
    __shared__ __align__(16) unsigned char turn[kBlk * kBlk];
    pdl_enter();
    const uint32_t tcol = (uint32_t)(p.cols + kBlk - 1) / kBlk, trow = (uint32_t)(p.rows + kBlk - 1) / kBlk;
    const uint32_t tr = blockIdx.x / tcol;
    const int cb = (int)(blockIdx.x - tr * tcol), rb = (int)(tr % trow);
    const long long g = tr / trow;
    const int lane16 = threadIdx.x & 15, pr = threadIdx.x >> 4, warp = threadIdx.x >> 5;
    const int r0 = rb * kBlk + 8 * pr, c0 = cb * kBlk + 8 * lane16;
    const bool cin = c0 < p.cols;   // (cols is a multiple of 16: whole chunks)
    Patch<E> x;
    const E* src = static_cast<const E*>(p.src) + g * p.src_gs + (long long)r0 * p.src_ld + c0;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        if (cin && r0 + r < p.rows) x.load(r, src);
        else x.zero(r);
        src += p.src_ld;
    }

    uint32_t tb = 0;   // the tile's scale byte (TILE)
    if constexpr (TILE) {
        uint32_t m = 0;
#pragma unroll
        for (int r = 0; r < 8; ++r) m = max(m, x.row_max(r));
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

    uint2 q[8];   // codes of the patch's rows
    if (TILE || p.dst) {
        float inv = scale_inverse(tb);
        using Max = BlockMax<8, 16>;
        if constexpr (!TILE) {   // the eight rows' scales, row `held` in this lane
            uint32_t m[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) m[r] = x.row_max(r);
            const uint32_t b = scale_byte(Max::reduce(m, threadIdx.x & 31));
            const int held = lane16 >> Max::SHIFT;
            inv = scale_inverse(b);
            if ((lane16 & ((1 << Max::SHIFT) - 1)) == 0 && r0 + held < p.rows)
                p.scale[g * p.s_gs + (r0 + held) * p.s_ld + cb] = (uint8_t)b;
        }
        uint8_t* dst = static_cast<uint8_t*>(p.dst) + g * p.dst_gs + (long long)r0 * p.dst_ld + c0;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const float k = TILE ? inv : __shfl_sync(0xffffffffu, inv, (threadIdx.x & 16) | (r << Max::SHIFT));
            q[r] = make_uint2(codes4(x.at(r, 0), x.at(r, 1), x.at(r, 2), x.at(r, 3), k),
                              codes4(x.at(r, 4), x.at(r, 5), x.at(r, 6), x.at(r, 7), k));
            if (p.dst && cin && r0 + r < p.rows) *reinterpret_cast<uint2*>(dst) = q[r];
            dst += p.dst_ld;
        }
    }

    if (p.dst_t) {
        // Column c of the patch: 8 bytes at slot pr of the column's 16 slots of
        // shared memory, the slots permuted by the patch's column so that the 16
        // lanes of a store meet 16 different bank pairs.
        unsigned char* put = turn + 8 * lane16 * kBlk + ((pr ^ lane16) << 3);
        if constexpr (TILE) {   // the same codes, turned
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t lo[4], hi[4];
                if (h == 0) {
                    turn4(q[0].x, q[1].x, q[2].x, q[3].x, lo);
                    turn4(q[4].x, q[5].x, q[6].x, q[7].x, hi);
                } else {
                    turn4(q[0].y, q[1].y, q[2].y, q[3].y, lo);
                    turn4(q[4].y, q[5].y, q[6].y, q[7].y, hi);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) *reinterpret_cast<uint2*>(put + (4 * h + c) * kBlk) = make_uint2(lo[c], hi[c]);
            }
        } else {   // each column's largest magnitude over the tile's 128 rows
            uint32_t m[8];
            x.col_max(m);
#pragma unroll
            for (int c = 0; c < 8; ++c) m[c] = max(m[c], __shfl_xor_sync(0xffffffffu, m[c], 16));
            if ((threadIdx.x & 31) < 16) {
                *reinterpret_cast<uint4*>(&cmax[warp][8 * lane16]) = make_uint4(m[0], m[1], m[2], m[3]);
                *reinterpret_cast<uint4*>(&cmax[warp][8 * lane16 + 4]) = make_uint4(m[4], m[5], m[6], m[7]);
            }
            __syncthreads();
            if (threadIdx.x < kBlk) {   // one column a thread: its scale byte, for all
                uint32_t v = 0;
#pragma unroll
                for (int w = 0; w < kThreads / 32; ++w) v = max(v, cmax[w][threadIdx.x]);
                const uint32_t b = scale_byte(v);
                cbyte[threadIdx.x] = (uint8_t)b;
                const int col = cb * kBlk + threadIdx.x;
                if (col < p.cols) p.scale_t[g * p.st_gs + col * p.st_ld + rb] = (uint8_t)b;
            }
            __syncthreads();
            const uint2 b8 = *reinterpret_cast<const uint2*>(cbyte + 8 * lane16);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const uint32_t b = ((c < 4 ? b8.x : b8.y) >> (8 * (c & 3))) & 255u;
                const float inv = scale_inverse(b);
                uint2 w = make_uint2(codes4(x.at(0, c), x.at(1, c), x.at(2, c), x.at(3, c), inv),
                                     codes4(x.at(4, c), x.at(5, c), x.at(6, c), x.at(7, c), inv));
                *reinterpret_cast<uint2*>(put + c * kBlk) = w;
            }
        }
        __syncthreads();
        uint8_t* dst = static_cast<uint8_t*>(p.dst_t) + g * p.dt_gs;
#pragma unroll
        for (int i = 0; i < kBlk * 8 / kThreads; ++i) {   // 16-byte pieces: 8 per column
            const int k = threadIdx.x + i * kThreads, c = k >> 3, piece = k & 7, sw = (c >> 3) & 15;
            const int col = cb * kBlk + c, row = rb * kBlk + 16 * piece;
            if (col >= p.cols || row >= p.rows) continue;
            uint4 v = *reinterpret_cast<const uint4*>(turn + c * kBlk + (((2 * piece) ^ (sw & 14)) << 3));
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
