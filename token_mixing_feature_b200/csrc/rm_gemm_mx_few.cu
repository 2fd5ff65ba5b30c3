// Block-scaled 8-bit product for few rows of A: serving's form, bound by
// reading the weights once.
//
// The operands change places: 128 rows of W are the tensor core's M side and
// up to NB rows of A its N side (16 at the least), so the smallest tile holds
// 128 x 16 results instead of 128 x 256 of which one row counts.  A CTA
// computes one such tile over one slice of K; a cluster of up to 8 CTAs shares
// the tile: each sends the rows of its partial result to the rows' owners
// through distributed shared memory, and an owner adds them in slice order.  So
// a projection of a few hundred columns still asks for its weights from every
// SM, without a workspace and with the same bits every time.
//
// What bounds it: one row through 1536 x 1536 takes 4.7 us, a launch and three
// trips through memory; four rows through 32 x 6144 x 1536 52.5 us in a burst, 5.8 TB/s
// of weights (88 % of the measured copy), 53.6 in a long run.
//
// Four warps: 0 loads W and A (bulk copies), 1 issues the MMAs, 2 and 3 load
// the scales; then all four carry the epilogue, a warp per row of A.
#include "rm_gemm_mx.cuh"

namespace rm {
namespace {

constexpr int BM = 128;
constexpr int BK = 128;
constexpr int kThreads = 128;
constexpr int kSlots = 4;
constexpr int kTSlots = 2;
constexpr int kRowF = BM + 4;      // floats of a result row in shared memory

template <int NB>
struct Cfg {
    static constexpr int W_BYTES = BM * BK, A_BYTES = NB * BK;
    static constexpr int STAGE_BYTES = W_BYTES + A_BYTES;
    // Two CTAs share an SM, so that one starts up while the other streams.
    static constexpr int STAGES = NB == 64 ? 3 : NB == 32 ? 4 : 5;
    static constexpr int PART_BYTES = NB * kRowF * 4;       // partial results, own and others'
    static constexpr int SLOT_BYTES = 1024, SLOT_COLS = 8;
    static constexpr int NBARS = 2 * STAGES + 2 * kSlots + 1;
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + PART_BYTES + kSlots * SLOT_BYTES + 8 * NBARS + 16;
    static constexpr int SCALE_COL = NB;
    static constexpr int TMEM_COLS = NB + kTSlots * SLOT_COLS <= 64 ? 64 : 128;
    static_assert(PART_BYTES % 16 == 0 && SMEM_BYTES <= 227 * 1024, "shared memory");
    // Tensor memory of as many CTAs as share an SM is always there: no CTA of
    // a cluster waits for another cluster's.
    static_assert(228 * 1024 / (SMEM_BYTES + 1024) * TMEM_COLS <= 512, "tensor memory");
};

__device__ __forceinline__ void st_cluster_f32(uint32_t a, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Activation, residual and output of four columns from n of row m, the 32
// lanes holding 128 columns.  n may lie behind N (all lanes call this).
template <int OUT>
__device__ __forceinline__ void put_row(float4 x, const MxParams& p, void* out, int g, int m, int n, int lane) {
    const bool in = n < p.N;
    float v[4] = {x.x, x.y, x.z, x.w};
    switch (p.act) {
        case RM_ACT_GELU_TANH: activate<RM_ACT_GELU_TANH>(v); break;
        case RM_ACT_GELU_ERF: activate<RM_ACT_GELU_ERF>(v); break;
        case RM_ACT_RELU: activate<RM_ACT_RELU>(v); break;
        default: break;
    }
    if constexpr (OUT == RM_E4M3) {
        uint32_t mx = 0;
        if (in) mx = max(max(abs_bits(v[0]), abs_bits(v[1])), max(abs_bits(v[2]), abs_bits(v[3])));
        mx = __reduce_max_sync(0xffffffffu, mx);
        const uint32_t b = scale_byte(mx);
        const float2 inv = f2(scale_inverse(b));
        if (lane == 0 && in) p.out_scale[g * p.os_gs + m * p.os_ld + (n >> 7)] = (uint8_t)b;
        if (in)
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(out) + g * p.o_gs + m * p.o_ld + n) =
                e4m3x4(f2_mul(make_float2(v[0], v[1]), inv), f2_mul(make_float2(v[2], v[3]), inv));
    } else if (in) {
        const long long r = g * p.r_gs + m * p.r_ld + n, o = g * p.o_gs + m * p.o_ld + n;
        if constexpr (OUT == RM_F32) {
            if (p.resid) {
                const float4 y = *reinterpret_cast<const float4*>(static_cast<const float*>(p.resid) + r);
                v[0] += y.x, v[1] += y.y, v[2] += y.z, v[3] += y.w;
            }
            *reinterpret_cast<float4*>(static_cast<float*>(out) + o) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
            if (p.resid) {
                const uint2 y = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.resid) + r);
                v[0] += __uint_as_float(y.x << 16), v[1] += __uint_as_float(y.x & 0xffff0000u);
                v[2] += __uint_as_float(y.y << 16), v[3] += __uint_as_float(y.y & 0xffff0000u);
            }
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + o) =
                make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        }
    }
}

// One lane's four rows of a scale atom of `rows` rows from r0 on.
__device__ __forceinline__ uint4 atom_words(const uint8_t* s, long long ld, int shift, int r0, int rows, int lane, int chunk,
                                            int blocks) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = r0 + 32 * j + lane;
        w[j] = scale_word(s + (min(r, rows - 1) >> shift) * ld, chunk, blocks);   // (rows behind the last: any)
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int NB, int OUT>
__global__ void __launch_bounds__(kThreads)
    gemm_mx_few_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW, const MxParams p,
                       void* out, int log_slices) {
    using C = Cfg<NB>;
    const int slices = 1 << log_slices;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    unsigned char* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    const uint32_t slot0 = sbase + C::STAGES * C::STAGE_BYTES, part0 = slot0 + kSlots * C::SLOT_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::STAGES * C::STAGE_BYTES + kSlots * C::SLOT_BYTES + C::PART_BYTES);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * C::STAGES;
    const uint32_t sfull0 = empty0 + 8 * C::STAGES, sempty0 = sfull0 + 8 * kSlots;
    const uint32_t done_bar = sempty0 + 8 * kSlots;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NBARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* failed = abort_flag + 1;   // a slice of this tile gave up

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slice = (int)(blockIdx.x & (slices - 1));   // = the CTA's rank in its cluster
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(sfull0 + 8 * s, 2);
            mbar_init(sempty0 + 8 * s, 1);
        }
        mbar_init(done_bar, 1);
        *abort_flag = *failed = 0;
        fence_mbar_init();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmW);
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (slices > 1) cluster_arrive();   // this CTA's shared memory may be written (awaited before the partial sums)
    pdl_enter();

    const WaitCtx wc{abort_flag, p.budget_ns, p.err}, drain = drain_ctx(wc);
    const int mblk = (p.M + NB - 1) / NB, nblk = (p.N + BM - 1) / BM;
    const uint32_t tile = blockIdx.x >> log_slices, col = tile / (uint32_t)mblk;
    const int m0 = (int)(tile - col * (uint32_t)mblk) * NB;
    const int g = (int)(col / (uint32_t)nblk);
    const int n0 = (int)(col - (uint32_t)g * (uint32_t)nblk) * BM;
    const int num_kb = (p.K + BK - 1) / BK;
    const int kb0 = (int)((long long)slice * num_kb >> log_slices);
    const int nkb = (int)((long long)(slice + 1) * num_kb >> log_slices) - kb0;
    // the slice's chunks of four K blocks are counted from its own first block
    const int chunks = (nkb + 3) / 4;

    if (warp == 0) {
        int stage = 0;
        uint32_t phase = 0, issued = 0, issued_phase = 0;
        for (int kb = 0; kb < nkb; ++kb) {
            if (!warp_mx_wait(empty0 + 8 * stage, phase ^ 1u, wc, SITE_MX_PRODUCER)) break;
            if (elect_one()) {
                const uint32_t fb = full0 + 8 * stage, sa = sbase + stage * C::STAGE_BYTES;
                mbar_arrive_expect_tx(fb, C::STAGE_BYTES);
                const int k = (kb0 + kb) * BK, wg = g * p.w_gmul, ag = g * p.a_gmul;
                tma_load_3d(sa, &tmW, fb, k, p.w_g_inner ? wg : n0, p.w_g_inner ? n0 : wg);
                tma_load_3d(sa + C::W_BYTES, &tmA, fb, k, p.a_g_inner ? ag : m0, p.a_g_inner ? m0 : ag);
            }
            __syncwarp();
            issued |= 1u << stage;
            issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
            if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
        }
        // every issued copy lands before its place is used again (the MMAs have
        // waited for all of them, unless a wait ran out)
        for (int i = 0; i < C::STAGES; ++i)
            if (issued & (1u << i)) mbar_wait(full0 + 8 * i, (issued_phase >> i) & 1u, drain, SITE_MX_DRAIN, false);
    } else if (warp == 1) {
        constexpr uint32_t idesc0 = idesc_mx_e4m3(BM, NB, 0, 0);
        int stage = 0;
        uint32_t phase = 0;
        for (int kb = 0; kb < nkb; ++kb) {
            const int c = kb >> 2;
            const bool begin = (kb & 3) == 0, end = (kb & 3) == 3 || kb == nkb - 1;
            const int old = c - kTSlots;   // its MMAs read the tensor memory that chunk c's scales go to
            if ((begin && (!warp_mx_wait(sfull0 + 8 * (c % kSlots), (uint32_t)(c / kSlots) & 1u, wc, SITE_MX_SCALES) ||
                           (old >= 0 &&
                            !warp_mx_wait(sempty0 + 8 * (old % kSlots), (uint32_t)(old / kSlots) & 1u, wc, SITE_MX_SCALES)))) ||
                !warp_mx_wait(full0 + 8 * stage, phase, wc, SITE_MX_MMA))
                break;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t sw = tmem + C::SCALE_COL + c % kTSlots * C::SLOT_COLS, sa = sw + 4;
                if (begin) {
                    const uint32_t ss = slot0 + c % kSlots * C::SLOT_BYTES;
                    tc_copy_scales<1>(sw, smem_desc_scales(ss));
                    tc_copy_scales<1>(sa, smem_desc_scales(ss + 512));
                }
                const uint32_t st = sbase + stage * C::STAGE_BYTES;
                const uint64_t wd = smem_desc_k_sw128(st), ad = smem_desc_k_sw128(st + C::W_BYTES);
                const uint32_t id = idesc0 | ((uint32_t)(kb & 3) << 4) | ((uint32_t)(kb & 3) << 29);
#pragma unroll
                for (int k = 0; k < BK / 32; ++k)
                    tc_mma_mx<1>(tmem, wd + 2 * k, ad + 2 * k, id, sw, sa, (kb | k) != 0 ? 1u : 0u);
                tc_commit(empty0 + 8 * stage);
                if (end) tc_commit(sempty0 + 8 * (c % kSlots));
            }
            __syncwarp();
            if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
        }
        if (elect_one()) tc_commit(done_bar);   // what was issued has completed
    } else {
        // warp 2: the scales of W's 128 rows, warp 3: of A's NB
        const uint8_t* s = warp == 2 ? p.w_scale + g * p.ws_gs : p.a_scale + g * p.as_gs;
        const long long ld = warp == 2 ? p.ws_ld : p.as_ld;
        const int shift = warp == 2 ? p.w_shift : 0, r0 = warp == 2 ? n0 : m0;
        const int rows = warp == 2 ? p.N : min(p.M, m0 + NB);
        for (int c = 0; c < chunks; ++c) {
            const uint4 w = atom_words(s + kb0, ld, shift, r0, rows, lane, c, nkb);
            if (!warp_mx_wait(sempty0 + 8 * (c % kSlots), ((uint32_t)(c / kSlots) & 1u) ^ 1u, wc, SITE_MX_SCALES)) break;
            sts128(slot0 + c % kSlots * C::SLOT_BYTES + (warp == 2 ? 0 : 512) + 16 * lane, w);
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(sfull0 + 8 * (c % kSlots));
        }
    }
    __syncwarp();

    float4 bias = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.bias && n0 + 4 * lane < p.N)
        bias = *reinterpret_cast<const float4*>(p.bias + (long long)g * p.N + n0 + 4 * lane);
    // The slice's sums: TMEM lane = column n0 + 32 warp + lane, TMEM column = row
    // of A.  Row r belongs to slice r % slices, which keeps what slice s sends of
    // its i-th row as row s * own + i of its partial results.
    const bool drained = mbar_wait(done_bar, 0, drain, SITE_MX_EPILOGUE, false);
    const bool ok = __all_sync(0xffffffffu, drained && *abort_flag == 0);   // this slice's sums are complete
    tc_fence_after();
    const int rows = min(NB, p.M - m0);
    const int own = NB >> log_slices;
    if (slices > 1) cluster_wait();
    if (!ok) {   // (a wait ran out) no CTA of the cluster may store rows that lack this slice
        if (lane < slices) st_cluster_u32(mapa_shared(smem_u32(tmem_slot + 2), lane), 1u);
    } else {
        const uint32_t at0 = part0 + 4 * (slice * own * kRowF + warp * 32 + lane);
#pragma unroll 1
        for (int c = 0; c < rows; c += 16) {
            float v[16];
            tmem_ld16(tmem + ((uint32_t)(warp * 32) << 16) + c, v);
            tmem_ld_wait();
            if (slices > 1) {
#pragma unroll
                for (int e = 0; e < 16; ++e)   // (rows from M on carry zeros)
                    st_cluster_f32(mapa_shared(at0 + 4 * kRowF * ((c + e) >> log_slices), (c + e) & (slices - 1)), v[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) sts32(at0 + 4 * kRowF * (c + e), __float_as_uint(v[e]));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (slices > 1) {
        cluster_arrive();
        cluster_wait();
    }
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
    if (*failed == 0) {
        const float4* part = reinterpret_cast<const float4*>(smem + (part0 - sbase)) + lane;
        const int last = (rows - 1 - slice) >> log_slices;   // this slice's last row
        for (int i = warp; i <= last; i += 16) {             // four rows of each warp's at a time
            float4 x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = part[min(i + 4 * j, last) * (kRowF / 4)];
            for (int s = 1; s < slices; ++s) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 y = part[(s * own + min(i + 4 * j, last)) * (kRowF / 4)];
                    x[j].x += y.x, x[j].y += y.y, x[j].z += y.z, x[j].w += y.w;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (i + 4 * j > last) break;
                x[j].x += bias.x, x[j].y += bias.y, x[j].z += bias.z, x[j].w += bias.w;
                put_row<OUT>(x[j], p, out, g, m0 + slice + ((i + 4 * j) << log_slices), n0 + 4 * lane, lane);
            }
        }
    }
}

template <int NB, int OUT>
cudaError_t launch_nb(const rm_matmul_fp8_args& a, MxParams& p, int num_sms, cudaStream_t s) {
    using C = Cfg<NB>;
    static SmemGrant grant;
    if (cudaError_t e = grant.ask(gemm_mx_few_kernel<NB, OUT>, C::SMEM_BYTES)) return e;
    CUtensorMap ma, mw;
    if (!matrix_map(&ma, a.A, a.K, a.M, a.G, a.a_ld, a.a_gstride, 1, NB, &p.a_g_inner, &p.a_gmul) ||
        !matrix_map(&mw, a.W, a.K, a.N, a.G, a.w_ld, a.w_gstride, 1, BM, &p.w_g_inner, &p.w_gmul))
        return cudaErrorInvalidValue;
    const long long tiles = (long long)a.G * ((a.M + NB - 1) / NB) * ((a.N + BM - 1) / BM);
    const int num_kb = (a.K + BK - 1) / BK;
    // K slices until the CTAs of a wave (two on an SM) are there, one K block a
    // slice at the least
    int log_slices = 0;
    while (log_slices < 3 && tiles << log_slices <= num_sms && 2 << log_slices <= num_kb) ++log_slices;
    if (tiles << log_slices > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_cluster(gemm_mx_few_kernel<NB, OUT>, dim3((unsigned)(tiles << log_slices)), kThreads, C::SMEM_BYTES,
                          1 << log_slices, s, ma, mw, p, a.out, log_slices);
}

template <int OUT>
cudaError_t launch_few(const rm_matmul_fp8_args& a, MxParams& p, int num_sms, cudaStream_t s) {
    if (a.M <= 16) return launch_nb<16, OUT>(a, p, num_sms, s);
    if (a.M <= 32) return launch_nb<32, OUT>(a, p, num_sms, s);
    return launch_nb<64, OUT>(a, p, num_sms, s);
}

}  // namespace

cudaError_t launch_gemm_mx_few(const rm_matmul_fp8_args& a, MxParams& p, int num_sms, cudaStream_t s) {
    switch (a.out_dtype) {
        case RM_F32: return launch_few<RM_F32>(a, p, num_sms, s);
        case RM_BF16: return launch_few<RM_BF16>(a, p, num_sms, s);
        default: return launch_few<RM_E4M3>(a, p, num_sms, s);
    }
}

}  // namespace rm
