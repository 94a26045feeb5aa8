// norm_fwd.cu -- h = residual + dropout(x), y = norm(h) and the row statistics
// (mean, 1/sqrt(var + eps)) that the backward pass needs.
//
// Four forms, chosen by the row's width:
//   fwd_warp   one warp holds a row's h in registers
//   fwd_ring   a CTA, or a cluster, holds it; the next rows' x and residual
//              arrive in a ring of shared-memory stages meanwhile
//   fwd_team   a team of CTAs across the GPU holds it (team.cuh)
//   fwd_sweep  wider rows: partial statistics per chunk, then a second read,
//              from L2 (sweep.cuh)
// Each reads x and residual from HBM once and writes h and y once.
//
// Measured (GB300, in a replayed graph, share of the 6782 GB/s copy rate; bf16,
// fp32 parameters):
//   16384 x 4096, LayerNorm, residual, dropout    89 us  0.89   (ring)
//   8192 x 8192, LayerNorm                        50 us  0.80   (ring)
//   16384 x 2048, LayerNorm                       24 us  0.81   (ring)
//   2048 x 10001, LayerNorm, residual, dropout    52 us  0.46   (ring, odd rows)
//   4096 x 8192 fp32, LayerNorm                   45 us  0.88   (ring)
//   the same with residual and dropout           113 us  0.70
//   1024 x 262144, LayerNorm                     358 us  0.44   (ring, clusters of 16)
//   1024 x 262144, RMSNorm                       239 us  0.66
//   300 x 850000, LayerNorm                      247 us  0.61   (team)
//   64 x 1000000, LayerNorm                      122 us  0.32   (sweep)
//   524288 x 128, LayerNorm                       78 us  0.51   (warp)
//   262144 x 64, LayerNorm                        38 us  0.26   (warp)
//   65536 x 512, LayerNorm                        30 us  0.66   (warp)
//   one row of 4096, RMSNorm, residual           2.2 us
// What bounds them: HBM up to some 8192 columns.  Odd rows: 44 instructions an
// element with residual and dropout (read, written and masked one at a time)
// fill 47 % of the issue slots; 15 warps an SM do not hide their loads from
// global and local memory (the two-row LayerNorm form spills 40 to 44 bytes).
// The widest LayerNorm rows read their parameters from L2 for every row and wait
// a row's exchange out, and clusters of 16 leave 40 SMs empty (teams use them all,
// but took 355 us for LayerNorm and 302 for RMSNorm on 1024 x 262144).  Short
// rows: a warp has one row's few hundred bytes in flight.  Teams at odd widths
// spill 48 to 112 bytes, sweeps of odd bf16 rows 116 to 168.
//
// Statistics: sum and M2 about the piece's own mean (of a warp, a CTA or a
// chunk), merged with the parallel-axis form of Chan et al.'s update.
#include <algorithm>

#include "planner.h"
#include "ring.cuh"
#include "sweep.cuh"
#include "team.cuh"

namespace credit {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// (h - mean) rstd gamma + beta; rstd is CUDA's rsqrtf (2 ulp).  The mean is
// subtracted first, so that a mean far above the deviation costs nothing.
template <int OP>
__device__ __forceinline__ F2 normed(F2 h, float mu, float rstd, F2 g, F2 b) {
    const F2 z = mul2(OP == kLayerNorm ? add2(h, f2(-mu)) : h, f2(rstd));
    return fma2(z, g, b);
}

// A warp's part of a row from its V tiles' h (zeros past the end): the sum,
// the mean sum inv_n, and M2 about it.
template <int OP, typename IO, int V, bool FULL>
__device__ __forceinline__ void warp_part(const F2 (&h)[V][IO::NP], int left, float inv_n, float& s,
                                          float& mu, float& m2) {
    F2 m = f2(0.f);
    if constexpr (OP == kLayerNorm) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < IO::NP; ++k) m = add2(m, h[i][k]);
        s = warp_allreduce(m.x + m.y, SumOp());
        mu = s * inv_n;
        m = f2(0.f);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < IO::NP; ++k) {
                F2 e = add2(h[i][k], f2(-mu));
                if constexpr (!FULL) e = inside<FULL, IO>(e, i * IO::kTile, k, left);
                m = fma2(e, e, m);
            }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < IO::NP; ++k) m = fma2(h[i][k], h[i][k], m);
    }
    m2 = warp_allreduce(m.x + m.y, SumOp());
}

// y of a warp's tiles; g, b, y point at the lane's first column.
template <int OP, typename T, typename IO, int V, bool FULL, typename PT>
__device__ __forceinline__ void write_tiles(F2 (&h)[V][IO::NP], const PT* gp, const PT* bp, T* y,
                                            int left, float mu, float rstd) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        F2 g[IO::NP], b[IO::NP];
        IO::template params<FULL>(gp, i * IO::kTile, left, g, 1.f);
        IO::template params<FULL>(bp, i * IO::kTile, left, b, 0.f);
#pragma unroll
        for (int k = 0; k < IO::NP; ++k) h[i][k] = normed<OP>(h[i][k], mu, rstd, g[k], b[k]);
        IO::template store<FULL>(y, i * IO::kTile, left, h[i]);
    }
}

__device__ __forceinline__ float finish(const NormFwdArgs& a, int64_t row, bool stats, float mu,
                                        float m2) {
    const float rstd = rsqrtf(fmaf(m2, a.inv_cols, a.eps));
    if (stats) {
        if (a.mean) a.mean[row] = mu;
        if (a.rstd) a.rstd[row] = rstd;
    }
    return rstd;
}

// ------------------------------------------------------------- one warp a row
template <int OP, typename T, typename IO, typename PT, int V>
__global__ void __launch_bounds__(kThreads) fwd_warp(NormFwdArgs a) {
    const int lane = threadIdx.x & 31, l0 = IO::first(lane), left = a.cols - l0;
    const DropStream d(a.drop);
    const T* const x = static_cast<const T*>(a.x) + l0;
    const T* const r = moved(static_cast<const T*>(a.residual), l0);
    const PT* const gp = moved(static_cast<const PT*>(a.gamma), l0);
    const PT* const bp = moved(static_cast<const PT*>(a.beta), l0);
    const int64_t step = (int64_t)gridDim.x * kWarps;
    int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= a.rows) return;
    typename IO::R xv[V], rv[V];
    auto fetch = [&](int64_t at) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            xv[i] = IO::template load<false>(x + at * a.cols, i * IO::kTile, left);
        if (r) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                rv[i] = IO::template load<false>(r + at * a.cols, i * IO::kTile, left);
        }
    };
    fetch(row);
    while (row < a.rows) {
        F2 h[V][IO::NP];
#pragma unroll
        for (int i = 0; i < V; ++i)
            tile_h<T, IO>(xv[i], rv[i], r != nullptr, a.drop.on && i * IO::kTile < a.cols, d,
                          i * IO::kTile, lane, (uint32_t)row, h[i]);
        const int64_t now = row;
        row += step;
        if (row < a.rows) fetch(row);  // in flight while this row is reduced and written
        if (a.h) {
            T* const ho = static_cast<T*>(a.h) + now * a.cols + l0;
#pragma unroll
            for (int i = 0; i < V; ++i) IO::template store<false>(ho, i * IO::kTile, left, h[i]);
        }
        float s, mu = 0.f, m2;
        warp_part<OP, IO, V, false>(h, left, a.inv_cols, s, mu, m2);
        const float rstd = finish(a, now, lane == 0, mu, m2);
        write_tiles<OP, T, IO, V, false>(h, gp, bp, static_cast<T*>(a.y) + now * a.cols + l0, left,
                                         mu, rstd);
    }
}

// ------------------------------------------------- a CTA or a cluster per row
// Warp w of a CTA holds the V tiles from column c0 + 128 V w on, of R rows at
// a time: every address of a turn is one register plus a constant.
template <int OP, typename T, typename IO, typename PT, int V, int R>
__global__ void __launch_bounds__(kRingThreads) fwd_ring(NormFwdArgs a, RingShape q) {
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ __align__(8) uint64_t full[kRingStages];
    __shared__ float2 wred[2][R][kRingWarps];
    __shared__ RingExchange ex;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
    const uint32_t P = cluster_nctarank(), rank = cluster_ctarank();
    const int64_t first = (int64_t)(blockIdx.x / P) * R, stride = (int64_t)q.clusters * R;
    const int slice = q.tiles * IO::kTile;
    const int c0 = (int)rank * slice, c1 = min(a.cols, c0 + slice);  // the slice's columns
    const int bytes = (c1 - c0) * (int)sizeof(T);
    const void* const src[2] = {a.x, a.residual};
    const int ns = a.residual ? 2 : 1, stage_bytes = ns * R * q.room;

    layout_fits((uint64_t)q.stages * stage_bytes, q.stages, kRingStages, q.err);
    if (threadIdx.x == 0) {
        for (int s = 0; s < q.stages; ++s) mbar_init(smem_u32(&full[s]), 1);
        if (P > 1) ex.init(P);
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    __syncthreads();
    if (P > 1) {  // every CTA's slots and mbarriers exist before any deposit
        cluster_arrive_release();
        cluster_wait_acquire();
    }
    const int feeder = W > 1;  // not the warp whose deposit a cluster waits for
    if (warp == feeder)
        for (int s = 0; s < q.stages; ++s)
            if (first + s * stride < a.rows)
                ring_issue<2, R, T, IO>(src, ns, first + s * stride, a.rows, a.cols, c0, bytes,
                                        ring + s * stage_bytes, q.room, smem_u32(&full[s]));

    const DropStream d(a.drop);
    const int base0 = c0 + warp * V * IO::kTile, j0 = base0 + IO::first(lane), left = c1 - j0;
    const bool whole = base0 + V * IO::kTile <= c1;
    const PT* const gp = moved(static_cast<const PT*>(a.gamma), j0);
    const PT* const bp = moved(static_cast<const PT*>(a.beta), j0);
    constexpr bool kHeld = V == 4;  // the parameters stay in registers
    const bool affine = whole && (kHeld || (gp && (OP != kLayerNorm || bp)));
    F2 hg[kHeld ? V : 1][IO::NP], hb[kHeld ? V : 1][IO::NP];
    if constexpr (kHeld) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            IO::template params<false>(gp, i * IO::kTile, left, hg[i], 1.f);
            if (OP == kLayerNorm) IO::template params<false>(bp, i * IO::kTile, left, hb[i], 0.f);
            else for (int e = 0; e < IO::NP; ++e) hb[i][e] = f2(0.f);
        }
    }
    // columns of this warp, of the warp and of the CTA that this lane merges
    const int part = lane & 15;
    const float inv_warp = 1.f / (float)max(1, min(c1 - base0, V * IO::kTile));
    const float wn = (float)max(0, min(c1 - (c0 + part * V * IO::kTile), V * IO::kTile));
    const float cn = (float)max(0, min(a.cols - part * slice, slice));
    const float inv_wn = 1.f / fmaxf(wn, 1.f), inv_cn = 1.f / fmaxf(cn, 1.f);
    const float inv_cta = P > 1 ? 1.f / (float)(c1 - c0) : a.inv_cols;
    T* ho = moved(static_cast<T*>(a.h), first * a.cols + j0);
    T* yo = static_cast<T*>(a.y) + first * a.cols + j0;
    int s = 0;
    uint32_t phase = 0, k = 0;
    for (int64_t row = first; row < a.rows; row += stride, ++k) {
        F2 h[R][V][IO::NP];
        float v[R];
        const bool both = R > 1 && row + 1 < a.rows;
        unsigned char* const stage = ring + s * stage_bytes;
        mbar_wait_bounded(smem_u32(&full[s]), phase, q.err);
        float mean[R], m2;
        auto take = [&](auto f, auto res, auto on) {
            constexpr bool FULL = decltype(f)::value;
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const int64_t off = ((row + j) * a.cols + c0) * (int64_t)sizeof(T);
                const T* xs = reinterpret_cast<const T*>(stage + j * q.room +
                                                         ring_shift<IO>(a.x, off)) + (j0 - c0);
                const T* rs = reinterpret_cast<const T*>(stage + (R + j) * q.room +
                                                         ring_shift<IO>(a.residual, off)) + (j0 - c0);
                F2 t = f2(0.f);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    typename IO::S rv = {};
                    if (res) rv = IO::template staged<FULL>(rs, i * IO::kTile, left);
                    tile_h<T, IO>(IO::template staged<FULL>(xs, i * IO::kTile, left), rv, res,
                                  on && (FULL || base0 + i * IO::kTile < c1), d,
                                  base0 + i * IO::kTile, lane, (uint32_t)(row + j), h[j][i]);
#pragma unroll
                    for (int e = 0; e < IO::NP; ++e)
                        t = OP == kLayerNorm ? add2(t, h[j][i][e]) : fma2(h[j][i][e], h[j][i][e], t);
                }
                if ((res || on) && ho && (j == 0 || both)) {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        IO::template store<FULL>(ho + j * a.cols, i * IO::kTile, left, h[j][i]);
                }
                v[j] = t.x + t.y;
            }
            m2 = row_sum<R>(v, lane);  // LayerNorm: the sum; RMSNorm: the sum of squares
            if constexpr (OP == kLayerNorm) {
                spread<R>(m2 * inv_warp, lane, mean);
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    F2 t = f2(0.f);
#pragma unroll
                    for (int i = 0; i < V; ++i)
#pragma unroll
                        for (int e = 0; e < IO::NP; ++e) {
                            F2 z = add2(h[j][i][e], f2(-mean[j]));
                            if constexpr (!FULL) z = inside<FULL, IO>(z, i * IO::kTile, e, left);
                            t = fma2(z, z, t);
                        }
                    v[j] = t.x + t.y;
                }
            }
        };
        const std::true_type yes;
        const std::false_type no;
        if (!whole) take(no, ns > 1, a.drop.on != 0);
        else if (ns > 1) a.drop.on ? take(yes, yes, yes) : take(yes, yes, no);
        else a.drop.on ? take(yes, no, yes) : take(yes, no, no);
        {   // the warp's (sum, M2 about its mean) of each row
            const float sum = m2;
            if constexpr (OP == kLayerNorm) m2 = row_sum<R>(v, lane);
            if ((lane & 15) == 0 && (R > 1 || lane == 0))
                wred[k & 1][R > 1 ? lane >> 4 : 0][warp] = make_float2(sum, m2);
        }
        __syncthreads();
        // every thread has read the stage: bring the turn that comes next in it
        if (warp == feeder) {
            const int64_t next = row + q.stages * stride;
            if (next < a.rows)
                ring_issue<2, R, T, IO>(src, ns, next, a.rows, a.cols, c0, bytes, stage, q.room,
                                        smem_u32(&full[s]));
        }
        const int mine = R > 1 ? lane >> 4 : 0;  // the row this half warp merges
        float2 w = part < W ? wred[k & 1][mine][part] : make_float2(0.f, 0.f);
        float sum = 0.f, mu = 0.f;
        if constexpr (OP == kLayerNorm) {
            sum = half_sum(w.x);
            mu = sum * inv_cta;
            const float e = fmaf(w.x, inv_wn, -mu);
            w.y = fmaf(wn * e, e, w.y);
        }
        m2 = half_sum(w.y);
        if (P > 1) {
            float t0[R], t1[R];
            spread<R>(sum, lane, t0);
            spread<R>(m2, lane, t1);
            if (warp == 0)
                ex.deposit(k, make_float4(t0[0], t1[0], t0[R - 1], t1[R - 1]), P, rank);
            const float4* parts = ex.wait(k, P, rank, q.err);
            const float4 c = part < (int)P ? parts[part] : make_float4(0.f, 0.f, 0.f, 0.f);
            w = mine ? make_float2(c.z, c.w) : make_float2(c.x, c.y);
            if constexpr (OP == kLayerNorm) {
                mu = half_sum(w.x) * a.inv_cols;
                const float e = fmaf(w.x, inv_cn, -mu);
                w.y = fmaf(cn * e, e, w.y);
            }
            m2 = half_sum(w.y);
        }
        const float own = rsqrtf(fmaf(m2, a.inv_cols, a.eps));
        if (rank == 0 && warp == 0 && (lane & 15) == 0 && (lane == 0 || both)) {
            if (a.mean) a.mean[row + (lane >> 4)] = mu;
            if (a.rstd) a.rstd[row + (lane >> 4)] = own;
        }
        float rstd[R];
        spread<R>(own, lane, rstd);
        if constexpr (OP == kLayerNorm) spread<R>(mu, lane, mean);
        auto give = [&](auto f) {  // FULL: gamma, and LayerNorm's beta, are there too
            constexpr bool FULL = decltype(f)::value;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                F2 g[IO::NP], b[IO::NP];
                if constexpr (kHeld) {
                    for (int e = 0; e < IO::NP; ++e) g[e] = hg[i][e], b[e] = hb[i][e];
                } else {
                    IO::template params<FULL>(gp, i * IO::kTile, left, g, 1.f, FULL);
                    if (OP == kLayerNorm) IO::template params<FULL>(bp, i * IO::kTile, left, b, 0.f, FULL);
                    else for (int e = 0; e < IO::NP; ++e) b[e] = f2(0.f);
                }
#pragma unroll
                for (int j = 0; j < R; ++j) {
#pragma unroll
                    for (int e = 0; e < IO::NP; ++e)
                        h[j][i][e] = normed<OP>(h[j][i][e], mean[j], rstd[j], g[e], b[e]);
                    if (j == 0 || both)
                        IO::template store<FULL>(yo + j * a.cols, i * IO::kTile, left, h[j][i]);
                }
            }
        };
        if (affine) give(yes); else give(no);
        yo += stride * a.cols;
        if (ho) ho += stride * a.cols;
        if (++s == q.stages) {
            s = 0;
            phase ^= 1u;
        }
    }
    if (P > 1) {  // no CTA leaves while a peer's deposit to it may be in flight
        cluster_arrive_release();
        cluster_wait_acquire();
    }
}

// ------------------------------------------------------------- a team per row
// team.cuh's pipeline: a summing and a writing warp own four tiles of the
// slice each; h is formed from the stage by both.
template <int OP, typename T, typename IO, typename PT>
__global__ void __launch_bounds__(kTeamThreads) fwd_team(NormFwdArgs a, TeamShape q) {
    constexpr int V = 4;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ __align__(8) TeamBars bars;
    __shared__ float2 wred[kTeamStages][kTeamWarps];
    __shared__ float2 tot[kTeamStages];  // mean, rstd
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = (blockDim.x >> 6) - 1;
    const int team = (int)blockIdx.x / q.size, rank = (int)blockIdx.x - team * q.size;
    const int slice = q.tiles * IO::kTile;
    const int c0 = rank * slice, c1 = min(a.cols, c0 + slice);
    const int bytes = (c1 - c0) * (int)sizeof(T);
    const void* const src[2] = {a.x, a.residual};
    const int ns = a.residual ? 2 : 1, stage_bytes = ns * q.room;
    const int turns = (int)((a.rows - team + q.teams - 1) / q.teams);
    auto row_of = [&](int k) { return team + (int64_t)k * q.teams; };

    layout_fits((uint64_t)q.stages * stage_bytes, q.stages, kTeamStages, q.err);
    bars.init(q.stages, W);

    if (warp == 2 * W) {  // collects: sums, M2 about each CTA's mean
        float n[kTeamParts], inv_n[kTeamParts];  // columns of the CTAs this lane merges
#pragma unroll
        for (int i = 0; i < kTeamParts; ++i) {
            n[i] = (float)max(0, min(a.cols - (lane + 32 * i) * slice, slice));
            inv_n[i] = 1.f / fmaxf(n[i], 1.f);
        }
        TeamExchange(q, team, rank, lane).collect(
            turns, q.stages, bars,
            [&](const float* x, const float* y) {
                float mu = 0.f, m2 = 0.f;
                if constexpr (OP == kLayerNorm) {
#pragma unroll
                    for (int i = 0; i < kTeamParts; ++i) mu += x[i];
                    mu = warp_allreduce(mu, SumOp()) * a.inv_cols;
                }
#pragma unroll
                for (int i = 0; i < kTeamParts; ++i) {
                    m2 += y[i];
                    if constexpr (OP == kLayerNorm) {
                        const float e = fmaf(x[i], inv_n[i], -mu);
                        m2 = fmaf(n[i] * e, e, m2);
                    }
                }
                m2 = warp_allreduce(m2, SumOp());
                return make_float2(mu, rsqrtf(fmaf(m2, a.inv_cols, a.eps)));
            },
            [&](int k, int st, float2 m) {
                if (lane == 0) {
                    tot[st] = m;
                    if (rank == 0) {
                        if (a.mean) a.mean[row_of(k)] = m.x;
                        if (a.rstd) a.rstd[row_of(k)] = m.y;
                    }
                }
            });
        return;
    }
    if (warp == 2 * W + 1) {  // serves
        const TeamExchange ex(q, team, rank, lane);
        const int part = lane & 15;
        const float wn = (float)max(0, min(c1 - (c0 + part * V * IO::kTile), V * IO::kTile));
        const float inv_wn = 1.f / fmaxf(wn, 1.f), inv_cta = 1.f / (float)(c1 - c0);
        bars.serve(
            turns, q.stages, q.err,
            [&](int k, int st) {
                ring_issue<2, 1, T, IO>(src, ns, row_of(k), a.rows, a.cols, c0, bytes,
                                        ring + st * stage_bytes, q.room, smem_u32(&bars.fed[st]));
                __syncwarp();
            },
            [&](int k, int st) {
                const float2 w = part < W ? wred[st][part] : make_float2(0.f, 0.f);
                float sum = 0.f, m2 = w.y;
                if constexpr (OP == kLayerNorm) {
                    sum = half_sum(w.x);
                    const float e = fmaf(w.x, inv_wn, -sum * inv_cta);
                    m2 = fmaf(wn * e, e, m2);
                }
                m2 = half_sum(m2);
                ex.deposit(k, sum, m2);
            });
        return;
    }

    TeamTurn t;
    const DropStream d(a.drop);
    const bool summing = warp < W;
    const int base0 = c0 + (summing ? warp : warp - W) * V * IO::kTile;
    const int j0 = base0 + IO::first(lane), left = c1 - j0;
    const bool whole = base0 + V * IO::kTile <= c1;
    const std::true_type yes;
    const std::false_type no;
    // h of a tile of the row in the stage
    auto tile = [&](auto f, auto res, auto on, int64_t row, int i, F2 (&h)[IO::NP]) {
        constexpr bool FULL = decltype(f)::value;
        const int64_t off = (row * a.cols + c0) * (int64_t)sizeof(T);
        const unsigned char* const p = ring + t.s * stage_bytes;
        const T* xs = reinterpret_cast<const T*>(p + ring_shift<IO>(a.x, off)) + (j0 - c0);
        const T* rs = reinterpret_cast<const T*>(p + q.room + ring_shift<IO>(a.residual, off)) +
                      (j0 - c0);
        typename IO::S rv = {};
        if (res) rv = IO::template staged<FULL>(rs, i * IO::kTile, left);
        tile_h<T, IO>(IO::template staged<FULL>(xs, i * IO::kTile, left), rv, res,
                      on && (FULL || base0 + i * IO::kTile < c1), d, base0 + i * IO::kTile, lane,
                      (uint32_t)row, h);
    };
    // f(whole, residual, dropout) with what holds for the whole call as constants
    // (a copy of x as h, without residual and dropout, takes the general code)
    const bool plain = whole && (summing || ns > 1 || a.drop.on || !a.h);
    auto pick = [&](auto f) {
        if (!plain) f(no, ns > 1, a.drop.on != 0);
        else if (ns > 1) a.drop.on ? f(yes, yes, yes) : f(yes, yes, no);
        else a.drop.on ? f(yes, no, yes) : f(yes, no, no);
    };
    if (summing) {
        const float inv_warp = 1.f / (float)max(1, min(c1 - base0, V * IO::kTile));
        for (int k = 0; k < turns; ++k, t.next(q.stages)) {
            bars.wait(bars.fed[t.s], t, q.err);
            pick([&](auto f, auto res, auto on) {
                constexpr bool FULL = decltype(f)::value;
                F2 h[V][IO::NP], v = f2(0.f);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    tile(f, res, on, row_of(k), i, h[i]);
#pragma unroll
                    for (int e = 0; e < IO::NP; ++e)
                        v = OP == kLayerNorm ? add2(v, h[i][e]) : fma2(h[i][e], h[i][e], v);
                }
                const float sum = warp_allreduce(v.x + v.y, SumOp());
                float m2 = sum;
                if constexpr (OP == kLayerNorm) {
                    const float mu = sum * inv_warp;
                    v = f2(0.f);
#pragma unroll
                    for (int i = 0; i < V; ++i)
#pragma unroll
                        for (int e = 0; e < IO::NP; ++e) {
                            F2 z = add2(h[i][e], f2(-mu));
                            if constexpr (!FULL)
                                z = inside<FULL, IO>(z, i * IO::kTile, e, left);
                            v = fma2(z, z, v);
                        }
                    m2 = warp_allreduce(v.x + v.y, SumOp());
                }
                if (lane == 0) wred[t.s][warp] = make_float2(sum, m2);
            });
            TeamBars::done(bars.summed[t.s]);
        }
        return;
    }
    const PT* const gp = moved(static_cast<const PT*>(a.gamma), j0);
    const PT* const bp = moved(static_cast<const PT*>(a.beta), j0);
    F2 g[V][IO::NP], b[V][IO::NP];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        IO::template params<false>(gp, i * IO::kTile, left, g[i], 1.f);
        IO::template params<false>(bp, i * IO::kTile, left, b[i], 0.f);
    }
    for (int k = 0; k < turns; ++k, t.next(q.stages)) {
        const int64_t at = row_of(k);
        bars.wait(bars.fed[t.s], t, q.err);
        bars.wait(bars.known[t.s], t, q.err);
        const float2 m = tot[t.s];
        T* const y = static_cast<T*>(a.y) + at * a.cols + j0;
        T* const ho = moved(static_cast<T*>(a.h), at * a.cols + j0);
        pick([&](auto f, auto res, auto on) {
            constexpr bool FULL = decltype(f)::value;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                F2 h[IO::NP];
                tile(f, res, on, at, i, h);
                if ((res || on || !FULL) && ho) IO::template store<FULL>(ho, i * IO::kTile, left, h);
#pragma unroll
                for (int e = 0; e < IO::NP; ++e)
                    h[e] = normed<OP>(h[e], m.x, m.y, g[i][e], b[i][e]);
                IO::template store<FULL>(y, i * IO::kTile, left, h);
            }
        });
        TeamBars::done(bars.written[t.s]);
    }
}

// ------------------------------------------------------------- wider rows
// One launch of sweep.cuh: row sums of one batch, outputs of the batch before.
// The sums of a row and chunk are (sum, M2 about the chunk's mean).
template <int OP, typename T, typename IO, typename PT>
__global__ void __launch_bounds__(kSweepThreads, kSweepCtas) fwd_sweep(NormFwdArgs a, Sweep q) {
    constexpr int kChunk = sweep_chunk(IO::N), kStrip = sweep_strip(IO::N);
    __shared__ float2 part[2][kSweepRows][kSweepWarps];
    __shared__ float2 rowc[kSweepGroup];  // mean, rstd
    wait_for_previous_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const DropStream d(a.drop);
    float2* const ws = reinterpret_cast<float2*>(a.ws);
    uint32_t index;
    if (sweep_sums(q, blockIdx.x, &index)) {
        const int chunk = (int)(index % (uint32_t)a.nch);
        const int64_t r0 = q.s0 + (int64_t)(index / (uint32_t)a.nch) * kSweepGroup;
        const int64_t r1 = min(q.s1, r0 + kSweepGroup);
        const int base0 = chunk * kChunk + warp * kSweepTiles * IO::kTile;
        const int j0 = base0 + IO::first(lane), left = a.cols - j0;
        const T* const x = static_cast<const T*>(a.x) + j0;
        const T* const res = moved(static_cast<const T*>(a.residual), j0);
        const float n = (float)max(0, min(a.cols - base0, kSweepTiles * IO::kTile));
        const float inv_n = 1.f / fmaxf(n, 1.f);
        int turn = 0;
        for (int64_t r = r0; r < r1; r += kSweepRows, turn ^= 1) {
            typename IO::R xv[kSweepRows][kSweepTiles], rv[kSweepRows][kSweepTiles];
            F2 h[kSweepRows][kSweepTiles][IO::NP];
            float v[kSweepRows];
#pragma unroll
            for (int j = 0; j < kSweepRows; ++j) {
                const int64_t at = min(r + j, r1 - 1) * a.cols;  // past the group: its last row
#pragma unroll
                for (int i = 0; i < kSweepTiles; ++i) {
                    xv[j][i] = IO::template load<false>(x + at, i * IO::kTile, left);
                    if (res) rv[j][i] = IO::template load<false>(res + at, i * IO::kTile, left);
                }
            }
#pragma unroll
            for (int j = 0; j < kSweepRows; ++j) {
                F2 t = f2(0.f);
#pragma unroll
                for (int i = 0; i < kSweepTiles; ++i) {
                    const int base = base0 + i * IO::kTile;
                    tile_h<T, IO>(xv[j][i], rv[j][i], res != nullptr, a.drop.on && base < a.cols, d,
                                  base, lane, (uint32_t)min(r + j, r1 - 1), h[j][i]);
#pragma unroll
                    for (int e = 0; e < IO::NP; ++e)
                        t = OP == kLayerNorm ? add2(t, h[j][i][e]) : fma2(h[j][i][e], h[j][i][e], t);
                }
                v[j] = t.x + t.y;
            }
            constexpr int G = 32 / kSweepRows;
            const float sum = sums_over_warp<kSweepRows>(v, lane);
            float m2 = sum;
            if constexpr (OP == kLayerNorm) {
#pragma unroll
                for (int j = 0; j < kSweepRows; ++j) {
                    const float mu = __shfl_sync(0xffffffffu, sum, j * G) * inv_n;
                    F2 t = f2(0.f);
#pragma unroll
                    for (int i = 0; i < kSweepTiles; ++i)
#pragma unroll
                        for (int e = 0; e < IO::NP; ++e) {
                            const F2 z = inside<false, IO>(add2(h[j][i][e], f2(-mu)), i * IO::kTile,
                                                           e, left);
                            t = fma2(z, z, t);
                        }
                    v[j] = t.x + t.y;
                }
                m2 = sums_over_warp<kSweepRows>(v, lane);
            }
            if (lane % G == 0) part[turn][lane / G][warp] = make_float2(sum, m2);
            __syncthreads();
            if (threadIdx.x < kSweepRows && r + threadIdx.x < r1) {
                // the warps' parts of the chunk, merged about the chunk's mean
                const float2* w = part[turn][threadIdx.x];
                float total = 0.f, dev = 0.f;
                for (int k = 0; k < kSweepWarps; ++k) total += w[k].x;
                const int c0 = chunk * kChunk;
                const float mu = total / (float)min(a.cols - c0, kChunk);
                for (int k = 0; k < kSweepWarps; ++k) {
                    dev += w[k].y;
                    if constexpr (OP == kLayerNorm) {
                        const float wn = (float)max(0, min(a.cols - c0 - k * kSweepTiles * IO::kTile,
                                                           kSweepTiles * IO::kTile));
                        const float e = wn > 0.f ? w[k].x / wn - mu : 0.f;
                        dev = fmaf(wn * e, e, dev);
                    }
                }
                ws[(r + threadIdx.x) * a.nch + chunk] = make_float2(total, dev);
            }
        }
        return;
    }
    const int strips = (a.cols + kStrip - 1) / kStrip, strip = (int)(index % (uint32_t)strips);
    const int64_t r0 = q.b0 + (int64_t)(index / (uint32_t)strips) * kSweepGroup;
    const int nr = (int)(min(q.b1, r0 + kSweepGroup) - r0);
    for (int i = warp; i < nr; i += kSweepWarps) {
        const float2* w = ws + (r0 + i) * a.nch;
        float sum = 0.f, m2 = 0.f, mu = 0.f;
        if constexpr (OP == kLayerNorm) {
            for (int c = lane; c < a.nch; c += 32) sum += __ldcg(w + c).x;
            mu = warp_allreduce(sum, SumOp()) * a.inv_cols;
        }
        for (int c = lane; c < a.nch; c += 32) {
            const float2 p = __ldcg(w + c);
            m2 += p.y;
            if constexpr (OP == kLayerNorm) {
                const float n = (float)min(a.cols - c * kChunk, kChunk);
                const float e = p.x / n - mu;
                m2 = fmaf(n * e, e, m2);
            }
        }
        m2 = warp_allreduce(m2, SumOp());
        const float rstd = rsqrtf(fmaf(m2, a.inv_cols, a.eps));
        if (lane == 0) {
            rowc[i] = make_float2(mu, rstd);
            if (strip == 0) {
                if (a.mean) a.mean[r0 + i] = mu;
                if (a.rstd) a.rstd[r0 + i] = rstd;
            }
        }
    }
    __syncthreads();
    const int base = strip * kStrip + warp * IO::kTile;
    if (base >= a.cols) return;
    const int j0 = base + IO::first(lane), left = a.cols - j0;
    F2 g[IO::NP], b[IO::NP];
    IO::template params<false>(moved(static_cast<const PT*>(a.gamma), j0), 0, left, g, 1.f);
    IO::template params<false>(moved(static_cast<const PT*>(a.beta), j0), 0, left, b, 0.f);
    for (int i = 0; i < nr; i += kSweepRows) {
        typename IO::R xv[kSweepRows], rv[kSweepRows];
#pragma unroll
        for (int j = 0; j < kSweepRows; ++j) {
            const int64_t at = (r0 + min(i + j, nr - 1)) * a.cols + j0;
            xv[j] = IO::template load<false>(static_cast<const T*>(a.x) + at, 0, left);
            if (a.residual)
                rv[j] = IO::template load<false>(static_cast<const T*>(a.residual) + at, 0, left);
        }
#pragma unroll
        for (int j = 0; j < kSweepRows; ++j) {
            if (i + j >= nr) break;
            const int64_t at = (r0 + i + j) * a.cols + j0;
            const float2 c = rowc[i + j];
            F2 h[IO::NP];
            tile_h<T, IO>(xv[j], rv[j], a.residual != nullptr, a.drop.on, d, base, lane,
                          (uint32_t)(r0 + i + j), h);
            if (a.h) IO::template store<false>(static_cast<T*>(a.h) + at, 0, left, h);
#pragma unroll
            for (int e = 0; e < IO::NP; ++e) h[e] = normed<OP>(h[e], c.x, c.y, g[e], b[e]);
            IO::template store<false>(static_cast<T*>(a.y) + at, 0, left, h);
        }
    }
}

template <int OP, typename T, typename IO, typename PT, int V>
cudaError_t run_warp(const NormFwdArgs& a, int sms, cudaStream_t s) {
    const int64_t want = (a.rows + kWarps - 1) / kWarps;
    fwd_warp<OP, T, IO, PT, V>
        <<<(unsigned)(want < sms * 8 ? want : sms * 8), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

// IO and WIO: the access forms of the ring and warp kernels and of the sweep.
template <int OP, typename T, typename IO, typename WIO, typename PT>
cudaError_t run_fwd(NormFwdArgs& a, int sms, cudaStream_t s) {
    const int tiles = (a.cols + IO::kTile - 1) / IO::kTile;
    if (tiles <= 1) return run_warp<OP, T, IO, PT, 1>(a, sms, s);
    if (tiles <= 2) return run_warp<OP, T, IO, PT, 2>(a, sms, s);
    if (tiles <= 4) return run_warp<OP, T, IO, PT, 4>(a, sms, s);
    const int streams = a.residual ? 2 : 1;
    if (!ring_fits(tiles, sizeof(T), streams, 2, a.rows, sms)) {
        TeamPlan team;
        if (plan_team(tiles, sizeof(T), streams, a.rows, sms, &team))
            return launch_team((const void*)fwd_team<OP, T, IO, PT>, a, team, a.ws, s);
        return run_sweep((const void*)fwd_sweep<OP, T, WIO, PT>, a,
                         sweep_batch(a.rows, (int64_t)a.cols * streams * sizeof(T), a.l2_bytes),
                         WIO::N, s);
    }
    // The ring kernel stores h where it forms it from x and something else.  A copy
    // of x is formed by a mask that keeps all (any word is at least 0, and x 1 is
    // x): a store in its code without residual and dropout, written in three
    // ways, cost the calls that want none up to 6 % (1024 x 262144 bf16 LayerNorm
    // 358 -> 379 us, 4096 x 8192 fp32 with residual and dropout 114 -> 121).
    if (a.h && !a.residual && !a.drop.on) {
        a.drop.on = 1;
        a.drop.threshold = 0;
        a.drop.scale = 1.f;
    }
    const RingKernels fn{(const void*)fwd_ring<OP, T, IO, PT, 4, 1>,
                         (const void*)fwd_ring<OP, T, IO, PT, 4, 2>,
                         (const void*)fwd_ring<OP, T, IO, PT, 8, 1>};
    RingPlan p;
    int resident;
    unsigned* err;
    if (!plan_ring(tiles, sizeof(T), streams, 2, a.rows, sms, fn, &p, &resident, &err))
        return cudaErrorInvalidConfiguration;
    return launch_ring(fn.of(p), a, p, ring_grid(p, resident, a.rows), err, s);
}

template <int OP, typename T, typename IO, typename WIO>
cudaError_t pick_param(NormFwdArgs& a, int sms, cudaStream_t s) {
    return a.half ? run_fwd<OP, T, IO, WIO, bf16>(a, sms, s)
                  : run_fwd<OP, T, IO, WIO, float>(a, sms, s);
}

template <int OP, typename T>
cudaError_t pick_fwd(TrainKey k, NormFwdArgs& a, int sms, cudaStream_t s) {
    constexpr int N = 16 / (int)sizeof(T);
    return k.vec ? pick_param<OP, T, VecIO<T, 4>, VecIO<T, N>>(a, sms, s)
                 : pick_param<OP, T, ElemIO<T, 4>, ElemIO<T, N>>(a, sms, s);
}

}  // namespace

int train_chunks(int dtype, int64_t cols) {
    const int chunk = sweep_chunk(dtype == 0 ? 4 : 8);
    return (int)((cols + chunk - 1) / chunk);
}

int64_t norm_fwd_partials(int dtype, int64_t rows, int64_t cols, int sms) {
    const int es = dtype == 0 ? 4 : 2;
    const int tiles = (int)((cols + VecIO<float, 4>::kTile - 1) / VecIO<float, 4>::kTile);
    if (tiles <= 4 || rows == 0) return 0;
    int64_t most = 0;
    for (int streams = 1; streams <= 2; ++streams) {  // without and with a residual
        if (ring_fits(tiles, es, streams, 2, rows, sms)) continue;
        TeamPlan team;
        if (plan_team(tiles, es, streams, rows, sms, &team))
            most = std::max(most, team.exchange_bytes);
        else
            most = std::max(most, rows * train_chunks(dtype, cols) * 8);
    }
    return most;
}

cudaError_t launch_norm_fwd(TrainKey k, NormFwdArgs a, int sms, cudaStream_t s) {
    if (k.op == kLayerNorm)
        return k.dtype == 0 ? pick_fwd<kLayerNorm, float>(k, a, sms, s)
                            : pick_fwd<kLayerNorm, bf16>(k, a, sms, s);
    return k.dtype == 0 ? pick_fwd<kRMSNorm, float>(k, a, sms, s)
                        : pick_fwd<kRMSNorm, bf16>(k, a, sms, s);
}

cudaError_t run_team_alone(int dev) {
    // 40 turns of 8 tiles through 4 stages, for a rank that the grid does not hold
    constexpr int kTiles = 8, kStages = 4, kRows = 40, kSize = 2, kWarps = 2;
    constexpr int kCols = kSize * kTiles * VecIO<float, 4>::kTile;
    constexpr int kRoom = (kCols / kSize * 4 + 16 + 127) / 128 * 128;
    constexpr size_t kMatrix = (size_t)kRows * kCols * 4;
    constexpr size_t kWords = (size_t)kTeamSlots * (kSize + 1) * 16;
    const void* fn = (const void*)fwd_team<kLayerNorm, float, VecIO<float, 4>, float>;
    unsigned* err = device_error_word();
    if (!err || !kernel_info(dev, fn, false)) return cudaErrorInvalidConfiguration;
    char* buf = nullptr;
    cudaError_t e = cudaMalloc(&buf, 2 * kMatrix + kWords);
    if (e != cudaSuccess) return e;
    e = cudaMemset(buf, 0, 2 * kMatrix + kWords);
    NormFwdArgs a{};
    a.x = buf;
    a.y = buf + kMatrix;
    a.rows = kRows;
    a.cols = kCols;
    a.inv_cols = 1.f / kCols;
    a.eps = 1.f;
    a.drop.scale = 1.f;
    TeamShape q{kTiles, kStages, kRoom, kSize, 1,
                reinterpret_cast<ulonglong2*>(buf + 2 * kMatrix), err};
    void* args[] = {&a, &q};
    if (e == cudaSuccess)
        e = cudaLaunchKernel(fn, dim3(1), dim3(32 * (2 * kWarps + 2)), args, kStages * kRoom, nullptr);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    const cudaError_t f = cudaFree(buf);
    return e != cudaSuccess ? e : f;
}

}  // namespace credit
