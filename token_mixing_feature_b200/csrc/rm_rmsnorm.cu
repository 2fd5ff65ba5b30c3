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
// Both directions are bound by HBM and, next, by the instructions an element
// takes.  A row belongs to a group of whole warps, warp w holding the NC * 32
// chunks of 16 bytes from w * NC * 32 on, chunk 32 i + lane in lane `lane`: the
// i-th chunks' addresses differ by constants, and a block of 128 is 16 (bf16) or
// 32 (fp32) neighbouring lanes.  One CTA of up to 512 threads an SM (two where
// rows are short); its groups walk over the rows, the next ones on their way into
// a ring in shared memory by cp.async:
// every thread copies the chunks that it will read, so the ring needs no
// barrier, and what is in flight (up to 220 KB an SM) depends neither on
// registers nor on where a group is in its row.  With the rows loaded straight
// into registers, 16384 x 1536 ran at 4.2-4.6 TB/s whatever the launch shape; now
// 5.4 TB/s (33 us with residual, sum and 8-bit output), 16384 x 7680 6.5 TB/s, the
// gradient of 16384 x 1536 4.75 TB/s (42 us, 4.5 of them the column sums).
#include <cuda_bf16.h>

#include <algorithm>

#include "rm_mx.cuh"

namespace rm {
namespace {

constexpr int kCta = 512;               // threads a CTA has at most
constexpr int kRing = 222 * 1024;       // bytes of its ring, gamma included
constexpr int kSms = 148;
// CTAs an SM of the forward kernel whose rows are one chunk a thread: 64 registers
// a thread are enough there, and twice the rows hide more of a row's latency
// (30000 x 256 bf16 12.3 -> 9.8 us, with residual 15.7 -> 14.4).
constexpr int kShortCtas = 2;

// 16 bytes of a row as they lie in memory: CE elements, as P pairs of floats.
// A block of 128 is LANES neighbouring lanes' chunks.
template <typename E>
struct Chunk {
    static constexpr int CE = 16 / sizeof(E), P = CE / 2, LANES = 128 / CE;
    uint4 u;
    __device__ __forceinline__ void read(uint32_t shared) { u = lds128(shared); }
    __device__ __forceinline__ void store(char* p) const { *reinterpret_cast<uint4*>(p) = u; }
    __device__ __forceinline__ void clear() { u = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void set(const float2 (&v)[P]) { u = pack_pairs(v); }   // rounded to the type
    __device__ __forceinline__ void pairs(float2 (&v)[P]) const { unpack_pairs(u, v); }
};
template <int P>
__device__ __forceinline__ void load_params(const float* p, float2 (&g)[P]) {
#pragma unroll
    for (int i = 0; i < P; i += 2) {
        const float4 a = reinterpret_cast<const float4*>(p)[i / 2];
        g[i] = make_float2(a.x, a.y), g[i + 1] = make_float2(a.z, a.w);
    }
}
// Codes of a chunk with 1 / scale = k, stored.
__device__ __forceinline__ void store_codes(char* o, const float2 (&y)[4], float2 k) {
    *reinterpret_cast<uint2*>(o) = make_uint2(e4m3x4(f2_mul(y[0], k), f2_mul(y[1], k)), e4m3x4(f2_mul(y[2], k), f2_mul(y[3], k)));
}
__device__ __forceinline__ void store_codes(char* o, const float2 (&y)[2], float2 k) {
    *reinterpret_cast<uint32_t*>(o) = e4m3x4(f2_mul(y[0], k), f2_mul(y[1], k));
}
// One chunk of a global row into shared memory, asynchronously.
__device__ __forceinline__ void copy_chunk(uint32_t dst, const char* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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

// A thread's place: its group (row) of the CTA and its warp there.
struct Place {
    int group, groups, warps, warp, lane;
    __device__ __forceinline__ explicit Place(int warps_) : warps(warps_) {
        const int w = threadIdx.x >> 5;
        groups = (blockDim.x >> 5) / warps;
        group = w / warps;
        warp = w - group * warps;
        lane = threadIdx.x & 31;
    }
    // Sum over the group's threads (every thread gets it), in a fixed order.
    // red: a float per warp of the CTA, not the last call's; all threads of the
    // group call this together.
    __device__ __forceinline__ float sum(float v, float* red) const {
        v = warp_sum(v);
        if (warps > 1) {
            float* r = red + group * warps;
            if (lane == 0) r[warp] = v;
            asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * warps) : "memory");
            v = 0.f;
            for (int w = 0; w < warps; ++w) v += r[w];
        }
        return v;
    }
};

// gamma from shared memory where the launch gave it a place there (at the
// ring's start): with the ring beside it, L1 holds no row's worth of it, and
// reading it from L2 for every row doubled the traffic of wide rows.
__device__ __forceinline__ const float* stage_gamma(const float* gamma, unsigned char* ring, int D, int gamma_bytes) {
    if (!gamma || !gamma_bytes) return gamma;
    for (int i = threadIdx.x; i < D / 4; i += blockDim.x)
        reinterpret_cast<float4*>(ring)[i] = reinterpret_cast<const float4*>(gamma)[i];
    __syncthreads();
    return reinterpret_cast<const float*>(ring);
}

template <typename E, int NC, bool RESID>
__global__ void __launch_bounds__(kCta, NC == 1 ? kShortCtas : 1) rmsnorm_kernel(const RmsNorm p, int warps, int stages, int gamma_bytes) {
    __shared__ float red[2][kCta / 32];
    extern __shared__ __align__(16) unsigned char ring[];
    pdl_enter();
    const Place at(warps);
    using C = Chunk<E>;
    const int nch = p.D / C::CE, c0 = at.warp * (NC * 32) + at.lane;
    const float inv_d = 1.0f / (float)p.D;
    constexpr uint32_t HOP = 32 * 16;   // bytes from a thread's chunk to its next
    const uint32_t bytes = (uint32_t)p.D * sizeof(E), slot = bytes * (RESID ? 2 : 1);
    const uint32_t mine = smem_u32(ring) + (uint32_t)gamma_bytes + (uint32_t)(at.group * stages) * slot + (uint32_t)c0 * 16;
    const long long step = (long long)gridDim.x * at.groups;
    long long row = (long long)blockIdx.x * at.groups + at.group;
    const char* nx = static_cast<const char*>(p.X) + row * p.ld_x * (long long)sizeof(E) + 16 * c0;
    const char* nr = RESID ? static_cast<const char*>(p.R) + row * p.ld_r * (long long)sizeof(E) + 16 * c0 : nullptr;
    long long ahead = row;   // the row that nx, nr point at
    auto fetch = [&](uint32_t place) {
        if (ahead < p.rows) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                if (c0 + 32 * i < nch) {
                    copy_chunk(place + i * HOP, nx + i * HOP);
                    if constexpr (RESID) copy_chunk(place + bytes + i * HOP, nr + i * HOP);
                }
            }
        }
        copies_commit();
        ahead += step;
        nx += step * p.ld_x * (long long)sizeof(E);
        if constexpr (RESID) nr += step * p.ld_r * (long long)sizeof(E);
    };
    for (int s = 0; s < stages; ++s) fetch(mine + s * slot);
    const float* gamma = stage_gamma(p.gamma, ring, p.D, gamma_bytes);
    uint32_t now = mine;   // place of this row, and of the row `stages` on as soon as this one is read
    const uint32_t end = mine + stages * slot;
    for (int par = 0; row < p.rows; row += step, par ^= 1) {   // (one value of row per group)
        copies_wait(stages - 1);
        C x[NC];
        float2 sq = f2(0.f);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            if (c0 + 32 * i < nch) {
                float2 v[C::P];
                x[i].read(now + i * HOP);
                x[i].pairs(v);
                if constexpr (RESID) {
                    // the stream is rounded to its type here: the statistics, the
                    // output and the gradient all see the values that are stored
                    C r;
                    float2 q[C::P];
                    r.read(now + bytes + i * HOP);
                    r.pairs(q);
#pragma unroll
                    for (int e = 0; e < C::P; ++e) v[e] = f2_add(v[e], q[e]);
                    x[i].set(v);
                    x[i].pairs(v);
                }
#pragma unroll
                for (int e = 0; e < C::P; ++e) sq = f2_fma(v[e], v[e], sq);
            } else {
                x[i].clear();
            }
        }
        fetch(now);
        now = now + slot == end ? mine : now + slot;
        if (p.Sum) {
            char* o = static_cast<char*>(p.Sum) + row * p.ld_sum * (long long)sizeof(E) + 16 * c0;
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (c0 + 32 * i < nch) x[i].store(o + i * HOP);
        }
        const float rstd = __frsqrt_rn(fmaf(at.sum(sq.x + sq.y, red[par]), inv_d, p.eps));
        if (p.rstd && at.warp == 0 && at.lane == 0) p.rstd[row] = rstd;
        if (!p.Y && !p.Yq) continue;
        float2 y[NC][C::P];
        uint32_t m[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = c0 + 32 * i;
            x[i].pairs(y[i]);
#pragma unroll
            for (int e = 0; e < C::P; ++e) y[i][e] = f2_mul(y[i][e], f2(rstd));
            if (gamma && c < nch) {
                float2 g[C::P];
                load_params(gamma + C::CE * c0 + 32 * C::CE * i, g);
#pragma unroll
                for (int e = 0; e < C::P; ++e) y[i][e] = f2_mul(y[i][e], g[e]);
            }
            float mf = 0.f;
#pragma unroll
            for (int e = 0; e < C::P; ++e) mf = max_abs(mf, y[i][e]);
            m[i] = c < nch ? abs_bits(mf) : 0u;
        }
        if (p.Y) {
            char* o = static_cast<char*>(p.Y) + row * p.ld_y * (long long)sizeof(E) + 16 * c0;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                C k;
                k.set(y[i]);
                if (c0 + 32 * i < nch) k.store(o + i * HOP);
            }
        }
        if (p.Yq) {
            using Max = BlockMax<NC, C::LANES>;
            const uint32_t b = scale_byte(Max::reduce(m, at.lane));   // of the lanes' block `held` of NC
            const float inv = scale_inverse(b);
            const int held = (at.lane & (C::LANES - 1)) >> Max::SHIFT, half = at.lane & (32 - C::LANES);
            const int block = (at.warp * (NC * 32) + 32 * held + half) / C::LANES;
            if ((at.lane & ((1 << Max::SHIFT) - 1)) == 0 && held < NC && C::LANES * block < nch)
                p.Ys[row * p.ld_ys + block] = (uint8_t)b;
            char* o = static_cast<char*>(p.Yq) + row * p.ld_yq + C::CE * c0;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const float2 k = f2(__shfl_sync(0xffffffffu, inv, half | (i << Max::SHIFT)));
                if (c0 + 32 * i < nch) store_codes(o + 32 * C::CE * i, y[i], k);
            }
        }
    }
}

// Gradient: the groups keep their columns' sums of dy * s * rstd in registers;
// a CTA's groups add theirs in order and leave one partial row.
template <typename E, int NC>
__global__ void __launch_bounds__(kCta, 1) rmsnorm_bwd_kernel(const RmsNormGrad p, int warps, int stages, int gamma_bytes) {
    __shared__ float red[2][kCta / 32];
    extern __shared__ __align__(16) unsigned char ring[];
    pdl_enter();
    const Place at(warps);
    using C = Chunk<E>;
    const int nch = p.D / C::CE, c0 = at.warp * (NC * 32) + at.lane;
    const float inv_d = 1.0f / (float)p.D;
    constexpr uint32_t HOP = 32 * 16;
    const uint32_t bytes = (uint32_t)p.D * sizeof(E), slot = bytes * (p.dSum ? 3 : 2);
    const uint32_t mine = smem_u32(ring) + (uint32_t)gamma_bytes + (uint32_t)(at.group * stages) * slot + (uint32_t)c0 * 16;
    const long long step = (long long)gridDim.x * at.groups;
    long long row = (long long)blockIdx.x * at.groups + at.group;
    auto place = [&](const void* base, long long ld) {
        return static_cast<const char*>(base) + row * ld * (long long)sizeof(E) + 16 * c0;
    };
    const char* ns = place(p.S, p.ld_s);
    const char* ny = place(p.dY, p.ld_dy);
    const char* nd = p.dSum ? place(p.dSum, p.ld_dsum) : nullptr;
    long long ahead = row;
    auto fetch = [&](uint32_t to) {
        if (ahead < p.rows) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                if (c0 + 32 * i < nch) {
                    copy_chunk(to + i * HOP, ns + i * HOP);
                    copy_chunk(to + bytes + i * HOP, ny + i * HOP);
                    if (nd) copy_chunk(to + 2 * bytes + i * HOP, nd + i * HOP);
                }
            }
        }
        copies_commit();
        ahead += step;
        ns += step * p.ld_s * (long long)sizeof(E);
        ny += step * p.ld_dy * (long long)sizeof(E);
        if (nd) nd += step * p.ld_dsum * (long long)sizeof(E);
    };
    float2 acc[NC][C::P];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < C::P; ++e) acc[i][e] = f2(0.f);
    for (int s = 0; s < stages - 1; ++s) fetch(mine + s * slot);
    const float* gamma = stage_gamma(p.gamma, ring, p.D, gamma_bytes);
    uint32_t now = mine, last = mine + (stages - 1) * slot;   // places of this row and of the row stages - 1 on
    const uint32_t end = mine + stages * slot;
    float rstd = row < p.rows ? __ldcg(p.rstd + row) : 0.f;
    for (int par = 0; row < p.rows; row += step, par ^= 1) {
        fetch(last);
        const float next_rstd = row + step < p.rows ? __ldcg(p.rstd + row + step) : 0.f;
        copies_wait(stages - 1);
        C cs[NC];
        float2 a[NC][C::P], dots = f2(0.f);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            if (c0 + 32 * i < nch) {
                C cy;
                float2 sv[C::P];
                cs[i].read(now + i * HOP);
                cy.read(now + i * HOP + bytes);
                cs[i].pairs(sv);
                cy.pairs(a[i]);
#pragma unroll
                for (int e = 0; e < C::P; ++e) acc[i][e] = f2_fma(f2_mul(a[i][e], f2(rstd)), sv[e], acc[i][e]);
                if (gamma) {
                    float2 g[C::P];
                    load_params(gamma + C::CE * c0 + 32 * C::CE * i, g);
#pragma unroll
                    for (int e = 0; e < C::P; ++e) a[i][e] = f2_mul(a[i][e], g[e]);
                }
#pragma unroll
                for (int e = 0; e < C::P; ++e) dots = f2_fma(a[i][e], sv[e], dots);
            }
        }
        const float dot = at.sum(dots.x + dots.y, red[par]);
        const float2 k = f2(-rstd * rstd * (dot * inv_d));
        char* o = static_cast<char*>(p.dX) + row * p.ld_dx * (long long)sizeof(E) + 16 * c0;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            if (c0 + 32 * i < nch) {
                float2 sv[C::P];
                cs[i].pairs(sv);
#pragma unroll
                for (int e = 0; e < C::P; ++e) a[i][e] = f2_mul(f2_fma(sv[e], k, a[i][e]), f2(rstd));
                if (nd) {
                    cs[i].read(now + i * HOP + 2 * bytes);
                    cs[i].pairs(sv);
#pragma unroll
                    for (int e = 0; e < C::P; ++e) a[i][e] = f2_add(a[i][e], sv[e]);
                }
                cs[i].set(a[i]);
                cs[i].store(o + i * HOP);
            }
        }
        last = now;
        now = now + slot == end ? mine : now + slot;
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
                const int c = c0 + 32 * i;
                if (c < nch) {
                    float2* s = reinterpret_cast<float2*>(acc_s + C::CE * c);
#pragma unroll
                    for (int e = 0; e < C::P; ++e) {
                        if (k) acc[i][e] = f2_add(acc[i][e], s[e]);
                        if (k < at.groups - 1) s[e] = acc[i][e];
                    }
                    if (k == at.groups - 1) {
                        float2* out = reinterpret_cast<float2*>(p.part + (long long)blockIdx.x * p.D + C::CE * c);
#pragma unroll
                        for (int e = 0; e < C::P; ++e) out[e] = acc[i][e];
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

// Launch shape for rows of D elements of esz bytes, `inputs` of them through
// the ring.
struct Shape {
    int nc, warps, groups, threads, stages, grid, gamma_bytes;
    size_t smem;
    Shape(long long rows, int D, int esz, int inputs, bool gamma, bool gradient, int aim, int short_ctas) {
        const int most = (D * esz / 16 + 31) / 32;
        const size_t row_bytes = (size_t)D * esz * inputs;
        // Groups: as many as there are warps for with `aim` chunks a thread (what
        // a row costs besides, its sum and its waits, is shared by those), as rows an
        // SM, and as the ring has room for.
        warps = std::min((most + aim - 1) / aim, kCta / 32);
        groups = kCta / 32 / warps;
        if (warps > 1) groups = std::min(groups, 15);   // (named barriers)
        groups = (int)std::min<long long>(groups, (rows + kSms - 1) / kSms);
        // two rows a group in the ring, one at least
        const auto fit = [&](size_t room) { return (int)std::max<size_t>(1, std::min<size_t>(groups, room / (2 * row_bytes))); };
        const int with = 4 * D + row_bytes <= kRing ? fit(kRing - 4 * D) : 0, without = fit(kRing);
        // gamma in shared memory where several rows use it, no group gives way and, in
        // the forward kernel, the groups keep a second row in the ring if they had one
        // (3000 x 12288 fp32 with residual: 74.6 us, with gamma in its place 86.0).  The
        // gradient, which reads gamma between its copies and its sum, wants it near even
        // so (4096 x 8192 fp32 with dSum 93.6 us, from L2 106; 3000 x 12288 without 110 / 164).
        const auto two = [&](int g, size_t room) { return room / (row_bytes * g) >= 2; };
        const bool fits = with == without && (gradient || two(with, kRing - 4 * D) || !two(without, kRing));
        gamma_bytes = gamma && rows > 2 * kSms && fits ? 4 * D : 0;
        groups = without;
        // the warps that this leaves go to the rows (gradient of 4099 x 7184 fp32, one
        // group: 8 warps 132 us, 15 85 us; of 160 x 1536 bf16 6.1 / 5.1)
        warps = std::min(most, kCta / 32 / groups);
        nc = (most + warps - 1) / warps;
        warps = (most + nc - 1) / nc;
        stages = (int)std::min<size_t>(4, (kRing - gamma_bytes) / (row_bytes * groups));
        threads = groups * warps * 32;
        smem = gamma_bytes + row_bytes * groups * stages;
        const int ctas = nc == 1 && groups == kCta / 32 ? short_ctas : 1;   // (their rings: 64 KB at most)
        grid = (int)std::min<long long>((rows + groups - 1) / groups, kSms * ctas);
    }
};

// Chunks a thread at most (what the registers hold without spilling).  fp32
// gradients want half of that where a row has warps for it (8192 x 4096: 8 chunks
// 114 us, 4 75 us); the other way round, forward fp32 rows 33 with 8, 42 with 4
// (4099 x 7184).
template <typename E>
constexpr int kFwdChunks = sizeof(E) == 2 ? 6 : 8;
template <typename E>
constexpr int kBwdChunks = sizeof(E) == 2 ? 4 : 8;
constexpr int kBwdAim = 4;

template <typename E, int NC, bool RESID>
cudaError_t fwd(const RmsNorm& p, const Shape& sh, cudaStream_t s) {
    static SmemGrant grant;
    if (cudaError_t e = grant.ask(rmsnorm_kernel<E, NC, RESID>, kRing)) return e;
    return launch_pdl(rmsnorm_kernel<E, NC, RESID>, dim3(sh.grid), dim3(sh.threads), sh.smem, s, p, sh.warps, sh.stages,
                      sh.gamma_bytes);
}
template <typename E, bool RESID>
cudaError_t fwd_e(const RmsNorm& p, cudaStream_t s) {
    const Shape sh(p.rows, p.D, sizeof(E), RESID ? 2 : 1, p.gamma != nullptr, false, kFwdChunks<E>, kShortCtas);
    switch (sh.nc) {
        case 1: return fwd<E, 1, RESID>(p, sh, s);
        case 2: return fwd<E, 2, RESID>(p, sh, s);
        case 3: return fwd<E, 3, RESID>(p, sh, s);
        case 4: return fwd<E, 4, RESID>(p, sh, s);
        case 5:
        case 6: return fwd<E, 6, RESID>(p, sh, s);
        default: return fwd<E, kFwdChunks<E>, RESID>(p, sh, s);
    }
}

template <typename E, int NC>
cudaError_t bwd(const RmsNormGrad& p, const Shape& sh, cudaStream_t s) {
    static SmemGrant grant;
    if (cudaError_t e = grant.ask(rmsnorm_bwd_kernel<E, NC>, kRing)) return e;
    return launch_pdl(rmsnorm_bwd_kernel<E, NC>, dim3(sh.grid), dim3(sh.threads), sh.smem, s, p, sh.warps, sh.stages,
                      sh.gamma_bytes);
}

template <typename E>
cudaError_t bwd_e(const RmsNormGrad& p, int* parts, cudaStream_t s) {
    const Shape sh(p.rows, p.D, sizeof(E), p.dSum ? 3 : 2, p.gamma != nullptr, true, kBwdAim, 1);
    *parts = sh.grid;
    switch (sh.nc) {
        case 1: return bwd<E, 1>(p, sh, s);
        case 2: return bwd<E, 2>(p, sh, s);
        case 3: return bwd<E, 3>(p, sh, s);
        case 4: return bwd<E, 4>(p, sh, s);
        default: return bwd<E, kBwdChunks<E>>(p, sh, s);
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
    int parts;
    const cudaError_t e = dtype == RM_BF16 ? bwd_e<__nv_bfloat16>(p, &parts, s) : bwd_e<float>(p, &parts, s);
    if (e != cudaSuccess || !dgamma) return e;
    return launch_pdl(colsum_parts_kernel, dim3((p.D + 31) / 32), dim3(1024), 0, s, (const float*)p.part, dgamma, parts,
                      p.D);
}

}  // namespace rm
