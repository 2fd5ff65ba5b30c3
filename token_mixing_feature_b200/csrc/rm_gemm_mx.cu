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
// A pair of CTAs computes a 256 x 256 tile with 2-SM MMAs (each CTA loads 128
// rows of A and 128 of W a K slice: 64 bytes a cycle at the tensor cores' full
// rate, just what an SM can take from L2, where a single CTA's 128 x 256 tile
// would want 96).  Persistent; roles of a CTA:
//   warp 0      TMA producer: 128-byte K slices of A and W into the ring
//   warp 1      MMA issuer (the even CTA's): scale copies, MMAs, commits
//   warps 2, 3  scale loaders: global bytes -> atoms in shared memory, taking
//               turns chunk by chunk (a chunk is 512 of K)
//   warps 4-11  epilogue, two groups of four warps (32 accumulator rows a
//               warp, 128 columns a group), while the next tile's MMAs run
// All waits are bounded (rm_device.cuh).
//
// What bounds it: long K, the operands' way from L2 (8192 x 8192 x 8192: 3040-3120
// TFLOP/s in a burst, 11.5 TB/s into the SMs); short K with fp32 results, writing
// them (32 x 6144 x 1536 x 512: 1.33 GB in 228-245 us in a burst); in a long run, the
// power cap, which takes the SMs from 1965 to 1350 MHz (281 us).
#include "rm_gemm_mx.cuh"

namespace rm {
namespace {

constexpr int BM = 128;            // rows of a CTA
constexpr int TM = 2 * BM, BN = 256;   // the pair's tile
constexpr int BK = 128;            // K elements (bytes) of a ring stage
constexpr int kSlots = 4;          // chunks (512 of K) of scale atoms in shared memory ...
constexpr int kTSlots = 2;         // ... and in tensor memory
constexpr int kEpiWarps = 8;
constexpr int kThreads = (4 + kEpiWarps) * 32;

// What the epilogue does: nothing but store, bias and activation, these and the
// residual.  (Each branch of them moves a thread's 64 values between registers,
// taken or not.)
enum : int { MX_PLAIN, MX_ACT, MX_RESID };

template <int OUT, int EPI>
struct Cfg {
    static constexpr int B_ROWS = BN / 2;                  // W rows a CTA loads
    static constexpr int A_BYTES = BM * BK, B_BYTES = B_ROWS * BK;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int B_ATOMS = BN / 128;               // every CTA holds all BN columns' scales
    static constexpr int SLOT_BYTES = 512 * (1 + B_ATOMS);
    static constexpr int SLOT_COLS = 4 * (1 + B_ATOMS);
    // Staging of an epilogue warp's output: a half of fp32, a chunk of bf16 (both
    // of them where the residual arrives there), both halves of e4m3.  With 4 KB a
    // fifth ring stage fits (8192 x 8192 x 8192: 2930 -> 3120 TFLOP/s).
    static constexpr int OUT_BYTES = OUT == RM_F32 || EPI == MX_RESID ? 8192 : 4096;
    static constexpr int EPI_BYTES = kEpiWarps * (OUT_BYTES + 512);   // staging and bias of the epilogue warps
    static constexpr int STAGES = (227 * 1024 - 1024 - 512 - kSlots * SLOT_BYTES - EPI_BYTES) / STAGE_BYTES;
    static constexpr int NBARS = 2 * STAGES + 2 * kSlots + 6 + (EPI == MX_RESID ? 2 * kEpiWarps : 0);
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + EPI_BYTES + kSlots * SLOT_BYTES + 8 * NBARS + 16;
    // Accumulators: two of BN columns.  Two of 256 do not fit beside the
    // scales: they overlap by 24 columns, which the epilogue reads before the
    // rest (of the present tile's, the next tile's MMAs wait for those alone).
    static constexpr int ACC1 = 232;
    static constexpr int SCALE_COL = ACC1 + BN;
    static constexpr int TMEM_COLS = SCALE_COL + kTSlots * SLOT_COLS <= 512 ? 512 : 0;
    static_assert(TMEM_COLS == 512 && SMEM_BYTES <= 227 * 1024, "on-chip memory");
};

struct Tile {
    int g, m0, n0;
};
template <int OUT>
__device__ __forceinline__ Tile decode(uint32_t idx, uint32_t mblk, uint32_t nblk) {
    // Bands of kBand tile rows, down each column of a band in turn: a W tile is
    // read from L2 by the band's tiles, and the A tiles of a band stay there
    // (8192 x 8192 x 8192: 2740 TFLOP/s down whole columns, 2920 in bands of 8).
    // fp32 results are bound by writing them: bands of 2 keep the tiles in flight
    // to fewer, whole rows (32 x 6144 x 1536 x 512: 266 -> 254 us).
    constexpr uint32_t kBand = OUT == RM_F32 ? 2 : 8;
    const uint32_t per_g = mblk * nblk, g = idx / per_g, r = idx - g * per_g;
    const uint32_t band = r / (kBand * nblk), m0 = band * kBand, rows = min(kBand, mblk - m0);
    const uint32_t q = r - m0 * nblk, nb = q / rows;
    return Tile{(int)g, (int)(m0 + q - nb * rows) * TM, (int)nb * BN};
}

template <int NV>
__device__ __forceinline__ void activate_all(float (&v)[NV], int act) {
    switch (act) {
        case RM_ACT_GELU_TANH: activate<RM_ACT_GELU_TANH>(v); break;
        case RM_ACT_GELU_ERF: activate<RM_ACT_GELU_ERF>(v); break;
        case RM_ACT_RELU: activate<RM_ACT_RELU>(v); break;
        default: break;
    }
}

// ---- bf16 results: an epilogue warp takes its 32 rows x 128 columns in chunks
// of 64 columns, a row a thread.
constexpr int kChunk = 64;

// Columns C0 .. C1 - 1 of the chunk.
template <int C0, int C1>
__device__ __forceinline__ void load_cols(uint32_t taddr, float (&v)[kChunk]) {
#pragma unroll
    for (int q = C0 / 16; q < C1 / 16; ++q) {
        float w[16];
        tmem_ld16(taddr + 16 * q, w);
#pragma unroll
        for (int e = 0; e < 16; ++e) v[16 * q + e] = w[e];
    }
}

// bias (from shared memory) and activation, in place.
__device__ __forceinline__ void finish_row(float (&v)[kChunk], const MxParams& p, uint32_t bias) {
    if (p.bias) {
#pragma unroll
        for (int q = 0; q < kChunk / 4; ++q) {
            const float4 x = lds_f32x4(bias + 16 * q);
            const float2 lo = f2_add(make_float2(v[4 * q], v[4 * q + 1]), make_float2(x.x, x.y));
            const float2 hi = f2_add(make_float2(v[4 * q + 2], v[4 * q + 3]), make_float2(x.z, x.w));
            v[4 * q] = lo.x, v[4 * q + 1] = lo.y, v[4 * q + 2] = hi.x, v[4 * q + 3] = hi.y;
        }
    }
    activate_all(v, p.act);
}

// The residual's box in the staging buffer (32 rows x 128 bytes, in the
// 128-byte swizzle of the bulk copies), added to the chunk; and the chunk there.
__device__ __forceinline__ void add_rows(float (&v)[kChunk], uint32_t buf, int lane) {
    const uint32_t row = buf + 128u * (uint32_t)lane, sw = (uint32_t)(lane & 7);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float2 f[4];
        unpack_pairs(lds128(row + (((uint32_t)j ^ sw) << 4)), f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 y = f2_add(make_float2(v[8 * j + 2 * e], v[8 * j + 2 * e + 1]), f[e]);
            v[8 * j + 2 * e] = y.x, v[8 * j + 2 * e + 1] = y.y;
        }
    }
}
__device__ __forceinline__ void stage_rows(const float (&v)[kChunk], uint32_t buf, int lane) {
    const uint32_t row = buf + 128u * (uint32_t)lane, sw = (uint32_t)(lane & 7);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        sts128(row + (((uint32_t)j ^ sw) << 4),
               make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                          pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7])));
}

// ---- e4m3 and fp32 results: two halves of 16 rows x 128 columns, 64 values a
// thread, so that a row's 128 columns (one quantisation block; 512 bytes of
// fp32, which leave together) lie in the four lanes of a quad.  Fragment of a
// half: v[4 i + 2 h + j] is row lane / 4 + 8 h, column 8 i + 2 (lane % 4) + j.
constexpr int kFrag = 64;

// A 32-column piece of 16 accumulator rows.
__device__ __forceinline__ void load_piece(uint32_t taddr, float* v) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// bias (128 floats in shared memory) and activation, in place.
__device__ __forceinline__ void finish_quads(float (&v)[kFrag], const MxParams& p, uint32_t bias, int lane) {
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 b = lds_f32x2(bias + 32 * i + 8 * (lane & 3));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 y = f2_add(make_float2(v[4 * i + 2 * h], v[4 * i + 2 * h + 1]), b);
                v[4 * i + 2 * h] = y.x, v[4 * i + 2 * h + 1] = y.y;
            }
        }
    }
    activate_all(v, p.act);
}

// The scale of each of the thread's two rows (its quad's largest magnitude over
// the columns below N), the byte to memory; inv: its inverse.
__device__ __forceinline__ void row_scales(const float (&v)[kFrag], float (&inv)[2], const MxParams& p, int g, int row0,
                                           int n, int lane) {
    float mf[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (n + 8 * i < p.N) {
            mf[0] = max_abs(mf[0], make_float2(v[4 * i], v[4 * i + 1]));
            mf[1] = max_abs(mf[1], make_float2(v[4 * i + 2], v[4 * i + 3]));
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t mx = abs_bits(mf[h]);
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const uint32_t b = scale_byte(mx);
        const int m = row0 + (lane >> 2) + 8 * h;
        if ((lane & 3) == 0 && m < p.M) p.out_scale[g * p.os_gs + m * p.os_ld + (n >> 7)] = (uint8_t)b;
        inv[h] = scale_inverse(b);
    }
}

// The half's codes into a box of 16 rows x 128 bytes, swizzled.
__device__ __forceinline__ void stage_quads(const float (&v)[kFrag], uint32_t buf, const float (&inv)[2], int lane) {
    const int q = lane & 3, r7 = lane >> 2;   // row lane / 4 + 8 h: the swizzle's row is r7 for both h
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t row = buf + 128u * (uint32_t)(r7 + 8 * h);
        const float2 k = f2(inv[h]);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 y = f2_mul(make_float2(v[4 * i + 2 * h], v[4 * i + 2 * h + 1]), k);
            sts16(row + (((i / 2) ^ r7) << 4) + 8 * (i & 1) + 2 * q, __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3));
        }
    }
}

// fp32: the half in four boxes of 16 rows x 128 bytes, swizzled; the residual
// there added, and the half put there.
__device__ __forceinline__ uint32_t quad_at(uint32_t buf, int i, int h, int lane) {
    const int q = lane & 3, r7 = lane >> 2;
    return buf + 2048u * (uint32_t)(i / 4) + 128u * (uint32_t)(r7 + 8 * h) + (((2 * (i % 4) + q / 2) ^ r7) << 4) + 8 * (q & 1);
}
__device__ __forceinline__ void add_quads(float (&v)[kFrag], uint32_t buf, int lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 y = f2_add(make_float2(v[4 * i + 2 * h], v[4 * i + 2 * h + 1]), lds_f32x2(quad_at(buf, i, h, lane)));
            v[4 * i + 2 * h] = y.x, v[4 * i + 2 * h + 1] = y.y;
        }
}
__device__ __forceinline__ void stage_quads_f32(const float (&v)[kFrag], uint32_t buf, int lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            sts64(quad_at(buf, i, h, lane), make_uint2(__float_as_uint(v[4 * i + 2 * h]), __float_as_uint(v[4 * i + 2 * h + 1])));
}

// What a CTA's producer has issued: the stage and phase that come next, and the
// number of stages so far (its last four bits, and whether it is 8 or more; the
// producer counts on from 16 behind 31).
__device__ __forceinline__ uint32_t producer_state(int stage, uint32_t phase, uint32_t count) {
    return (uint32_t)stage | phase << 3 | (count & 15u) << 4 | (count > 7u ? 1u : 0u) << 8;
}
constexpr uint32_t kGaveUp = 1u << 9;   // beside it: a wait of the CTA ran out

// After a wait ran out, on the even CTA (one thread): every copy that either
// producer has issued lands before the pair's shared memory goes away.  Both count
// their bytes on this CTA's full barriers, 2 * BYTES a stage, which it arms.  The
// producers may have stopped a few stages apart: what only the odd one issued is armed
// here, what only this one issued gets the odd one's bytes taken off.
template <int STAGES, uint32_t BYTES>
__device__ __forceinline__ void drain_pair(uint32_t full0, uint32_t own, uint32_t odd, const WaitCtx& drain) {
    int stage = (int)(own & 7u);
    uint32_t phase = own >> 3 & 1u;
    const int issued = (own >> 8 & 1u) ? STAGES : min((int)(own >> 4 & 15u), STAGES);   // stages that may be in flight
    int ahead = (int)(((odd >> 4) - (own >> 4)) & 15u);   // the odd one's lead: STAGES at most either way
    if (ahead > 7) ahead -= 16;
    for (int i = 0; i < issued; ++i) {   // from the last one back
        if (--stage < 0) stage = STAGES - 1, phase ^= 1u;
        if (i < -ahead)
            asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(full0 + 8 * stage), "r"(BYTES) : "memory");
        mbar_wait(full0 + 8 * stage, phase, drain, SITE_MX_DRAIN, false);
    }
    stage = (int)(own & 7u), phase = own >> 3 & 1u;
    for (int i = 0; i < ahead; ++i) {
        mbar_arrive_expect_tx(full0 + 8 * stage, BYTES);
        mbar_wait(full0 + 8 * stage, phase, drain, SITE_MX_DRAIN, false);
        if (++stage == STAGES) stage = 0, phase ^= 1u;
    }
}

template <int OUT, int EPI>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_mx_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                   const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmR, const MxParams p) {
    using C = Cfg<OUT, EPI>;
    constexpr bool PLAIN = EPI == MX_PLAIN;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    unsigned char* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    const uint32_t out0 = sbase + C::STAGES * C::STAGE_BYTES;   // 1024-byte aligned
    const uint32_t slot0 = out0 + C::EPI_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::STAGES * C::STAGE_BYTES + C::EPI_BYTES + kSlots * C::SLOT_BYTES);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * C::STAGES;
    const uint32_t sfull0 = empty0 + 8 * C::STAGES, sempty0 = sfull0 + 8 * kSlots;
    const uint32_t tfull0 = sempty0 + 8 * kSlots, tdone0 = tfull0 + 16, tover_bar = tdone0 + 16, drain_bar = tover_bar + 8, rbar0 = drain_bar + 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NBARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile uint32_t* state = tmem_slot + 2;   // at the end: each CTA's producer_state

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(sfull0 + 8 * s, 2);
            mbar_init(sempty0 + 8 * s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull0 + 8 * a, 1);
            mbar_init(tdone0 + 8 * a, 2 * kEpiWarps);
        }
        mbar_init(tover_bar, 2 * kEpiWarps / 2);
        mbar_init(drain_bar, 1);
        if (EPI == MX_RESID)
            for (int i = 0; i < 2 * kEpiWarps; ++i) mbar_init(rbar0 + 8 * i, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmO);
        if (EPI == MX_RESID) prefetch_tmap(&tmR);
    }
    if (warp == 0) {
        tmem_alloc_pair(smem_u32(tmem_slot), C::TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();   // the peer's barriers exist before anyone signals them
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_enter();   // operands, scales and bias may all come from the previous kernel

    const WaitCtx wc{abort_flag, p.budget_ns, p.err}, drain = drain_ctx(wc);
    const uint32_t mblk = (p.M + TM - 1) / TM, nblk = (p.N + BN - 1) / BN;
    const int num_kb = (p.K + BK - 1) / BK;
    const uint32_t total = (uint32_t)p.G * mblk * nblk;   // below 2^31
    const uint32_t unit = blockIdx.x >> 1, nunits = gridDim.x >> 1;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        int stage = 0;
        uint32_t phase = 0, count = 0;
        bool ok = true;
        for (uint32_t idx = unit; idx < total && ok; idx += nunits) {
            const Tile t = decode<OUT>(idx, mblk, nblk);
            const int ar = t.m0 + (int)rank * BM, wr = t.n0 + (int)rank * C::B_ROWS;
            const int ag = t.g * p.a_gmul, wg = t.g * p.w_gmul;
            for (int kb = 0; kb < num_kb; ++kb) {
                if (!warp_mx_wait(empty0 + 8 * stage, phase ^ 1u, wc, SITE_MX_PRODUCER)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    const uint32_t fb = full0 + 8 * stage, sa = sbase + stage * C::STAGE_BYTES;
                    if (leader) mbar_arrive_expect_tx(fb, 2 * C::STAGE_BYTES);
                    const uint32_t fbl = mapa_shared(fb, 0);   // the pair counts bytes on the even CTA's barrier
                    tma_load_3d_pair(sa, &tmA, fbl, kb * BK, p.a_g_inner ? ag : ar, p.a_g_inner ? ar : ag);
                    tma_load_3d_pair(sa + C::A_BYTES, &tmW, fbl, kb * BK, p.w_g_inner ? wg : wr, p.w_g_inner ? wr : wg);
                }
                count = count == 31u ? 16u : count + 1u;
                if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
            }
        }
        if (lane == 0) state[rank] = producer_state(stage, phase, count);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        if (leader) {
            constexpr uint32_t idesc0 = idesc_mx_e4m3(TM, BN, 0, 0);
            int stage = 0, slot = 0;
            uint32_t phase = 0, sphase = 0, chunk = 0;
            bool ok = true, any = false;
            int it = 0;
            for (uint32_t idx = unit; idx < total && ok; idx += nunits, ++it) {
                const int acc = it & 1;
                // the epilogues have read the accumulator's last tile, and of the tile
                // before this one what the accumulators share
                if ((it > 1 && !warp_wait(tdone0 + 8 * acc, (uint32_t)((it >> 1) - 1) & 1u, wc, SITE_MX_MMA)) ||
                    (it > 0 && !warp_wait(tover_bar, (uint32_t)(it - 1) & 1u, wc, SITE_MX_MMA)))
                    break;
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(acc * C::ACC1);
                for (int kb = 0; kb < num_kb; ++kb) {
                    const bool chunk_begin = (kb & 3) == 0, chunk_end = (kb & 3) == 3 || kb == num_kb - 1;
                    // a chunk's scales: there, and their place in tensor memory no longer
                    // read (the MMAs of the chunk kTSlots before have completed)
                    const uint32_t old = chunk - kTSlots;
                    if ((chunk_begin &&
                         (!warp_wait<true>(sfull0 + 8 * slot, sphase, wc, SITE_MX_SCALES) ||
                          (chunk >= kTSlots &&
                           !warp_wait(sempty0 + 8 * (old % kSlots), (old / kSlots) & 1u, wc, SITE_MX_SCALES)))) ||
                        !warp_wait(full0 + 8 * stage, phase, wc, SITE_MX_MMA)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t sa_col = tmem + C::SCALE_COL + chunk % kTSlots * C::SLOT_COLS, sb_col = sa_col + 4;
                        if (chunk_begin) {
                            const uint32_t ss = slot0 + slot * C::SLOT_BYTES;
                            tc_copy_scales<2>(sa_col, smem_desc_scales(ss));
#pragma unroll
                            for (int a = 0; a < C::B_ATOMS; ++a)
                                tc_copy_scales<2>(sb_col + 4 * a, smem_desc_scales(ss + 512 * (1 + a)));
                        }
                        const uint32_t sa = sbase + stage * C::STAGE_BYTES;
                        const uint64_t ad = smem_desc_k_sw128(sa), bd = smem_desc_k_sw128(sa + C::A_BYTES);
                        const uint32_t id = idesc0 | ((uint32_t)(kb & 3) << 4) | ((uint32_t)(kb & 3) << 29);
#pragma unroll
                        for (int k = 0; k < BK / 32; ++k)
                            tc_mma_mx<2>(d, ad + 2 * k, bd + 2 * k, id, sa_col, sb_col, (kb | k) != 0 ? 1u : 0u);
                        tc_commit_pair_mc(empty0 + 8 * stage, 0x3);
                        if (chunk_end) tc_commit_pair_mc(sempty0 + 8 * slot, 0x3);
                        if (kb == num_kb - 1) tc_commit_pair_mc(tfull0 + 8 * acc, 0x3);
                    }
                    __syncwarp();
                    any = true;
                    if (chunk_end) {
                        ++chunk;
                        if (++slot == kSlots) { slot = 0; sphase ^= 1u; }
                    }
                    if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            if (any) {   // everything issued completes before tensor memory is released
                if (elect_one()) tc_commit_pair(drain_bar);
                __syncwarp();
                mbar_wait(drain_bar, 0, drain, SITE_MX_DRAIN, false);
            }
        }
        __syncwarp();
    } else if (warp < 4) {
        // Scale loaders: chunk c of the CTA's stream of chunks by warp 2 + c % 2.
        const int chunks = (num_kb + 3) / 4;
        long long c = 0;
        bool ok = true;
        for (uint32_t idx = unit; idx < total && ok; idx += nunits) {
            const Tile t = decode<OUT>(idx, mblk, nblk);
            const uint8_t* as = p.a_scale + t.g * p.as_gs;
            const uint8_t* ws = p.w_scale + t.g * p.ws_gs;
            for (int ch = 0; ch < chunks; ++ch, ++c) {
                if ((int)(c & 1) != warp - 2) continue;
                const int slot = (int)(c % kSlots);
                uint32_t w[1 + C::B_ATOMS][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = t.m0 + (int)rank * BM + 32 * j + lane;
                    w[0][j] = scale_word(as + min(r, p.M - 1) * p.as_ld, ch, num_kb);   // (rows behind the last: any)
                }
#pragma unroll
                for (int a = 0; a < C::B_ATOMS; ++a)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = t.n0 + 128 * a + 32 * j + lane;
                        w[1 + a][j] = scale_word(ws + (min(r, p.N - 1) >> p.w_shift) * p.ws_ld, ch, num_kb);
                    }
                // the slot is free once the MMAs that read its last content (and
                // the tensor memory copy of it) have completed
                if (!warp_mx_wait(sempty0 + 8 * slot, (uint32_t)(c / kSlots & 1) ^ 1u, wc, SITE_MX_SCALES)) {
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
                    if (leader) mbar_arrive(sfull0 + 8 * slot);
                    else mbar_arrive_cluster(mapa_shared(sfull0 + 8 * slot, 0));
                }
            }
        }
        __syncwarp();
    } else {
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        // one arrival a warp, on the even CTA's barrier, when its tcgen05.ld have completed
        const auto have_read = [&](uint32_t bar) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (leader) mbar_arrive(bar);
                else mbar_arrive_cluster_relaxed(mapa_shared(bar, 0));
            }
        };
        const uint32_t stage = out0 + (uint32_t)(warp - 4) * C::OUT_BYTES;
        const uint32_t bias_s = out0 + kEpiWarps * C::OUT_BYTES + (uint32_t)(warp - 4) * 512u;
        // The residual comes to the staging buffer that its results leave from:
        // fetch(b, ..) loads bf16's box at column c into buffer b, or fp32's four boxes
        // from there on into the one buffer, as far as they exist (all earlier stores
        // have read theirs); `due` has a bit for each buffer's copy on its way.
        const uint32_t rbar = rbar0 + 16u * (uint32_t)(warp - 4);
        uint32_t due = 0, rphase = 0;
        const auto fetch = [&](int b, int c, int row0, int g) {
            if (row0 >= p.M || c >= p.N) return;
            if (lane == 0) {
                const int boxes = OUT == RM_F32 ? min(4, (p.N - c + 31) / 32) : 1;
                bulk_wait_read<0>();
                mbar_arrive_expect_tx(rbar + 8 * b, OUT == RM_F32 ? 2048u * (uint32_t)boxes : 4096u);
                for (int i = 0; i < boxes; ++i)
                    tma_load_3d(stage + (OUT == RM_F32 ? 2048u * (uint32_t)i : 4096u * (uint32_t)b), &tmR, rbar + 8 * b, c + 32 * i,
                                p.r_g_inner ? g * p.r_gmul : row0, p.r_g_inner ? row0 : g * p.r_gmul);
            }
            due |= 1u << b;
        };
        const auto arrived = [&](int b, const WaitCtx& w, bool honour_abort) {
            const bool ok = __all_sync(0xffffffffu, mx_wait(rbar + 8 * b, rphase >> b & 1u, w, SITE_MX_EPILOGUE, honour_abort));
            if (ok) {
                rphase ^= 1u << b;
                due &= ~(1u << b);
            }
            return ok;
        };
        // e4m3: the two staging buffers by turns, one a store that is made (a half
        // behind the last row makes none, so its number does not tell the buffer)
        uint32_t codes = 0;
        int it = 0;
        for (uint32_t idx = unit; idx < total; idx += nunits, ++it) {
            const int acc = it & 1;
            const Tile t = decode<OUT>(idx, mblk, nblk);
            const int col0 = 128 * half;   // this group's 128 columns
            const int row0 = t.m0 + (int)rank * BM + quarter * 32, n = t.n0 + col0;
            if (!PLAIN && p.bias) {   // fetched while the tile's products run
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (n + 4 * lane < p.N) x = *reinterpret_cast<const float4*>(p.bias + (long long)t.g * p.N + n + 4 * lane);
                __syncwarp();
                sts128(bias_s + 16 * lane, make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(x.z),
                                                      __float_as_uint(x.w)));
                __syncwarp();
            }
            if constexpr (EPI == MX_RESID) {   // the tile's two chunks of it, or its first half
                fetch(0, OUT == RM_F32 ? n : n + kChunk * half, row0, t.g);
                if (OUT != RM_F32) fetch(1, n + (kChunk ^ kChunk * half), row0, t.g);
            }
            if (!warp_mx_wait(tfull0 + 8 * acc, (uint32_t)(it >> 1) & 1u, wc, SITE_MX_EPILOGUE)) break;
            tc_fence_after();
            const uint32_t ta = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * C::ACC1 + col0);
            // the half of the columns that holds the accumulators' overlap: the last 24
            // of the first accumulator, the first 24 of the second
            const bool owner = acc == 0 ? half == 1 : half == 0;
            const auto store = [&](uint32_t src, int c, int r) {
                tma_store_3d(&tmO, src, c, p.o_g_inner ? t.g : r, p.o_g_inner ? r : t.g);
            };
            bool ok = true;
            if constexpr (OUT == RM_BF16) {
                const int first = half;   // the overlap's chunk, if this half has it
#pragma unroll 1
                for (int k = 0; k < 2; ++k) {
                    const int c = kChunk * (k ^ first);
                    float v[kChunk];
                    if (k == 0 && owner) {   // the overlap's 32 columns, then the chunk's others
                        if (half == 1) load_cols<32, 64>(ta + c, v);
                        else load_cols<0, 32>(ta + c, v);
                        tmem_ld_wait();
                        have_read(tover_bar);
                        if (half == 1) load_cols<0, 32>(ta + c, v);
                        else load_cols<32, 64>(ta + c, v);
                    } else {
                        load_cols<0, 64>(ta + c, v);
                    }
                    tmem_ld_wait();
                    if (k == 1) have_read(tdone0 + 8 * acc);
                    if (row0 >= p.M || n + c >= p.N) continue;   // (one value per warp)
                    if constexpr (!PLAIN) finish_row(v, p, bias_s + 4 * c);
                    const uint32_t to = stage + (EPI == MX_RESID ? 4096u * (uint32_t)k : 0u);
                    if constexpr (EPI == MX_RESID) {
                        ok = arrived(k, wc, true);
                        if (!ok) break;
                        add_rows(v, to, lane);
                    } else {
                        if (lane == 0) bulk_wait_read<0>();   // the last store has read the staging
                        __syncwarp();
                    }
                    stage_rows(v, to, lane);
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        store(to, n + c, row0);
                        bulk_commit_group();
                    }
                }
            } else {
                const bool low = owner && half == 0, high = owner && half == 1;   // where the overlap's 32 columns are
                float keep[16];   // those of the second half
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const uint32_t th = ta + ((uint32_t)(16 * h) << 16);
                    float v[kFrag];
                    if (h == 0) {
                        if (owner) {
                            if (low) load_piece(th, v);
                            else load_piece(th + 96, v + 48);
                            load_piece(th + (16u << 16) + (low ? 0u : 96u), keep);
                            tmem_ld_wait();
                            have_read(tover_bar);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            if (low) v[j] = keep[j];
                            if (high) v[48 + j] = keep[j];
                        }
                    }
                    if (!low) load_piece(th, v);
                    load_piece(th + 32, v + 16);
                    load_piece(th + 64, v + 32);
                    if (!high) load_piece(th + 96, v + 48);
                    tmem_ld_wait();
                    if (h == 1) have_read(tdone0 + 8 * acc);
                    const int r0 = row0 + 16 * h;
                    if (r0 >= p.M || n >= p.N) continue;   // (one value per warp)
                    if constexpr (!PLAIN) finish_quads(v, p, bias_s, lane);
                    if constexpr (OUT == RM_F32) {
                        if constexpr (EPI == MX_RESID) {
                            ok = arrived(0, wc, true);
                            if (!ok) break;
                            add_quads(v, stage, lane);
                        } else {
                            if (lane == 0) bulk_wait_read<0>();   // the last stores have read the staging
                            __syncwarp();
                        }
                        stage_quads_f32(v, stage, lane);
                    } else {
                        float inv[2];
                        row_scales(v, inv, p, t.g, r0, n, lane);
                        if (lane == 0) bulk_wait_read<1>();   // the store before the last has read its buffer
                        __syncwarp();
                        stage_quads(v, stage + codes, inv, lane);
                    }
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (OUT == RM_F32) {
#pragma unroll
                            for (int b = 0; b < 4; ++b)
                                if (n + 32 * b < p.N) store(stage + 2048u * b, n + 32 * b, r0);
                        } else {
                            store(stage + codes, n, r0);
                        }
                        bulk_commit_group();
                    }
                    codes ^= 2048u;
                    if (EPI == MX_RESID && h == 0) fetch(0, n, row0 + 16, t.g);   // the second half's
                }
            }
            if (!ok) break;
        }
        for (int b = 0; b < 2; ++b)   // (a wait ran out: copies land before shared memory goes away)
            if (due >> b & 1u) arrived(b, drain, false);
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t mine = state[rank] | (*abort_flag ? kGaveUp : 0u);
        state[rank] = mine;
        st_cluster_u32(mapa_shared(smem_u32(tmem_slot + 2 + rank), rank ^ 1u), mine);
    }
    __syncwarp();
    cluster_sync_all();   // the peer may still signal this CTA's barriers
    if ((state[0] | state[1]) & kGaveUp) {   // (else the MMAs have waited for every copy)
        if (leader && threadIdx.x == 0) drain_pair<C::STAGES, C::STAGE_BYTES>(full0, state[0], state[1], drain);
        __syncwarp();
        cluster_sync_all();
    }
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, C::TMEM_COLS);
    }
}

template <int OUT, int EPI>
cudaError_t launch_tile(const rm_matmul_fp8_args& a, MxParams& p, int num_sms, cudaStream_t s) {
    using C = Cfg<OUT, EPI>;
    static SmemGrant grant;
    if (cudaError_t e = grant.ask(gemm_mx_kernel<OUT, EPI>, C::SMEM_BYTES)) return e;
    CUtensorMap ma, mw, mo, mr = {};
    const int osz = OUT == RM_F32 ? 4 : OUT == RM_BF16 ? 2 : 1, orows = OUT == RM_BF16 ? 32 : 16;
    if (!matrix_map(&ma, a.A, a.K, a.M, a.G, a.a_ld, a.a_gstride, 1, BM, &p.a_g_inner, &p.a_gmul) ||
        !matrix_map(&mw, a.W, a.K, a.N, a.G, a.w_ld, a.w_gstride, 1, C::B_ROWS, &p.w_g_inner, &p.w_gmul) ||
        !matrix_map(&mo, a.out, a.N, a.M, a.G, a.o_ld, a.o_gstride, osz, orows, &p.o_g_inner, nullptr))
        return cudaErrorInvalidValue;
    if (EPI == MX_RESID &&
        !matrix_map(&mr, a.resid, a.N, a.M, a.G, a.r_ld, a.r_gstride, osz, orows, &p.r_g_inner, &p.r_gmul))
        return cudaErrorInvalidValue;
    const long long tiles = (long long)a.G * ((a.M + TM - 1) / TM) * ((a.N + BN - 1) / BN);
    const int units = (int)(tiles < num_sms / 2 ? tiles : num_sms / 2);
    return launch_cluster(gemm_mx_kernel<OUT, EPI>, dim3(units * 2), kThreads, C::SMEM_BYTES, 2, s, ma, mw, mo, mr, p);
}
template <int OUT>
cudaError_t launch_out(const rm_matmul_fp8_args& a, MxParams& p, int num_sms, cudaStream_t s) {
    if constexpr (OUT != RM_E4M3)
        if (a.resid) return launch_tile<OUT, MX_RESID>(a, p, num_sms, s);
    if (a.bias || a.act != RM_ACT_NONE) return launch_tile<OUT, MX_ACT>(a, p, num_sms, s);
    return launch_tile<OUT, MX_PLAIN>(a, p, num_sms, s);
}

}  // namespace

bool gemm_mx_few_rows(const rm_matmul_fp8_args& a, int num_sms) {
    // Few rows, or at most one 64 x 128 tile an SM: the few-row kernel, which
    // starts more CTAs and splits K.  Measured, pair / few in us: M 64, N = K = 4096
    // 13.8 / 8.4; M 64, N 1024, K 16384 40.2 / 10.1; 8 groups, M 128, N 1024 (128
    // tiles), K 1024 8.1 / 7.5, K 4096 15.0 / 12.4.  Past that K is not split and the
    // pair's 256 x 256 tiles win: 5 groups, M 256, N 1104 (180 tiles), K 1024 8.1 /
    // 8.3, K 4096 15.0 / 16.8; M 1024, N = K = 4096 16.3 / 33.3.  With 32 rows at the
    // most the few-row kernel wins at any size (32 groups, N 6144, K 1536: 63.2 /
    // 59.2; at 64 rows 65.6 / 74.3).
    //
    // Where the epilogue is long and K is not, it wins as long as its tiles are one
    // wave, two on an SM.  Measured at 160 to 288 tiles, K 256 to 2048; of 8 groups, M
    // 256, N 1024 (256 tiles), K 256 / 1024 / 2048: fp32 7.8 / 6.3, 9.8 / 8.7, 12.3 / 11.7
    // (with residual 10.5 / 8.6, 12.5 / 10.8, 15.0 / 14.0); bf16 with GELU 8.4 / 7.2, 10.4 /
    // 9.5, 12.8 / 12.6; e4m3 with GELU 9.5 / 7.6, 11.6 / 9.9, 14.0 / 13.0, with ReLU 7.9 /
    // 7.0, 9.8 / 9.5, 12.4 / 12.4.  Not so for e4m3 without activation (6.8 / 7.0, 8.8 /
    // 9.3, 11.3 / 12.3), bf16 (5.9 / 6.4, 7.9 / 8.8, 10.4 / 11.8), with ReLU (6.8 / 6.5, 8.8 /
    // 9.0, 11.2 / 12.0) or residual (7.0 / 8.4, 8.9 / 10.9, 11.4 / 14.0), nor at K 4096
    // (fp32 17.2 / 17.5, e4m3 with ReLU 17.2 / 18.3).  A second wave loses everywhere (325
    // tiles, K 256, fp32 8.2 / 11.4).
    const long long tiles = (long long)a.G * ((a.M + 63) / 64) * ((a.N + 127) / 128);
    const bool gelu = a.act == RM_ACT_GELU_TANH || a.act == RM_ACT_GELU_ERF;
    const bool finish = gelu || a.out_dtype == RM_F32 || (a.out_dtype == RM_E4M3 && a.act != RM_ACT_NONE);
    const bool one_wave = tiles <= (finish && a.K <= 2048 ? 2 : 1) * num_sms;
    return a.M <= 32 || one_wave;
}

cudaError_t launch_gemm_mx(const rm_matmul_fp8_args& a, int num_sms, cudaStream_t s) {
    MxParams p{};
    p.G = a.G, p.M = a.M, p.N = a.N, p.K = a.K;
    p.a_scale = a.a_scale, p.as_gs = a.as_gstride, p.as_ld = a.as_ld;
    p.w_scale = a.w_scale, p.ws_gs = a.ws_gstride, p.ws_ld = a.ws_ld;
    p.w_shift = a.w_block_rows == 128 ? 7 : 0;
    p.bias = a.bias;
    p.resid = a.resid, p.r_gs = a.r_gstride, p.r_ld = a.r_ld;
    p.o_gs = a.o_gstride, p.o_ld = a.o_ld;
    p.out_scale = a.out_scale, p.os_gs = a.os_gstride, p.os_ld = a.os_ld;
    p.act = a.act;
    p.err = DeviceErr{a.device_status, nullptr};
    p.budget_ns = a.wait_budget_ns ? a.wait_budget_ns : 1000000000ull;
    if (gemm_mx_few_rows(a, num_sms)) return launch_gemm_mx_few(a, p, num_sms, s);
    switch (a.out_dtype) {
        case RM_F32: return launch_out<RM_F32>(a, p, num_sms, s);
        case RM_BF16: return launch_out<RM_BF16>(a, p, num_sms, s);
        default: return launch_out<RM_E4M3>(a, p, num_sms, s);
    }
}

}  // namespace rm
