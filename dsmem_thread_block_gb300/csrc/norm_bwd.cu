// norm_bwd.cu -- the gradient of y = norm(h), h = residual + dropout(x):
// with xh = (h - mean) rstd and w = dy gamma (RMSNorm: mean = 0),
//   dtot   = rstd (w - mean_j(w) - xh mean_j(w xh)) + dh   (RMSNorm: no mean_j(w))
//   dres   = dtot,   dx = keep ? dtot / (1 - p) : 0
//   dgamma = sum_rows dy xh,   dbeta = sum_rows dy
//
// Four forms, chosen by the call's shape (form_of):
//   bwd_warp   one warp per row
//   bwd_ring   a CTA, or a cluster, per row; the next rows' dy, h and dh
//              arrive in a ring of shared-memory stages
//   bwd_team   a team of CTAs across the GPU per row (team.cuh)
//   bwd_sweep  wider rows: the two row sums per chunk, then a second read, from
//              L2 (sweep.cuh)
// In each a thread keeps the same columns for all its rows and sums their
// dgamma and dbeta in registers; the row groups' sums go to the workspace and
// bwd_params adds them.  Every sum has a fixed order: results repeat bit for
// bit.
//
// Measured (GB300, both launches in a replayed graph, share of the 6782 GB/s copy
// rate; fp32 parameters unless said otherwise):
//   16384 x 4096 bf16, LayerNorm, dh, dropout    142 us  0.70   (ring)
//   8192 x 8192 bf16, RMSNorm, dh, bf16 weight    89 us  0.89   (ring)
//   2048 x 10001 fp32, LayerNorm                  47 us  0.77   (ring, clusters of 5)
//   2048 x 10001 bf16, LayerNorm                  46 us  0.40   (ring)
//   4096 x 8192 fp32, LayerNorm                   69 us  0.86   (ring)
//   the same with dh and dropout                 136 us  0.73
//   16384 x 2048 bf16, LayerNorm                  55 us  0.54   (ring)
//   8192 x 1024 fp32, LayerNorm                   32 us  0.46   (ring)
//   512 x 70001 bf16, LayerNorm                   77 us  0.41   (team)
//   1024 x 262144 bf16, LayerNorm                328 us  0.72   (team)
//   256 x 786432 bf16, RMSNorm, bf16 weight      226 us  0.79   (team)
//   64 x 1000000 bf16, LayerNorm                 161 us  0.36   (sweep)
//   524288 x 128 bf16, LayerNorm                 158 us  0.38   (warp)
//   262144 x 64 bf16, LayerNorm                   75 us  0.20   (warp)
//   65536 x 512 bf16, LayerNorm                   56 us  0.53   (warp)
//   32 x 1024 fp32, LayerNorm                    5.5 us (two launches, one behind
//                                                 the other)
// What bounds them.  Training block: 45 instructions an element fill 57 % of the
// issue slots; the rest is their latency, which the 15 warps an SM that the
// parameter sums' registers leave do not hide (the mask is drawn between a row's
// sums and its stores).  Up to 2048 columns: CTAs of few warps leave some 900
// groups' sums, which bwd_params adds on a CTA for each 128 columns.  Odd bf16
// rows: staged and stored two bytes at a time.  Short rows: 8 to 16 warps an SM
// (153 to 221 registers above 256 columns), one row each in flight.  Spills:
// odd bf16 LayerNorm rings 60 to 76 bytes, sweeps of bf16 rows 32 to 120, odd ones
// 212 to 364.
#include <algorithm>

#include "planner.h"
#include "ring.cuh"
#include "sweep.cuh"
#include "team.cuh"

namespace credit {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

constexpr int kTileCols = VecIO<float, 4>::kTile;

// The form of a call, by its shape.  A team hides the exchange that a cluster
// waits for, and is not bound to a GPC, but clears its exchange and launches
// cooperatively, some microseconds on the host: it takes large calls of rows
// that clusters would share.  Measured, cluster and team (copy rate = 1): 4096
// rows of 16384 bf16 columns, RMSNorm 0.81 and 0.72; 3355 of 20000, 0.61 and
// 0.68; 1024 of 65536, LayerNorm, 0.49 and 0.60; 64 rows of 20000 columns 9.3
// and 10.8 us, of 65536 columns 16.0 and 15.2 us.
enum class Form { kWarp, kRing, kTeam, kSweep };

Form form_of(int tiles, int es, int streams, int64_t rows, int64_t cols, int sms, TeamPlan* team) {
    if (tiles <= 4) return Form::kWarp;
    const bool ring = ring_fits(tiles, es, streams, 1, rows, sms);
    if (ring && (cols <= 16384 || rows * cols < (1 << 22))) return Form::kRing;
    if (plan_team(tiles, es, streams, rows, sms, team)) return Form::kTeam;
    return ring ? Form::kRing : Form::kSweep;
}

struct RowStats { float mean, rstd; };

template <int OP>
__device__ __forceinline__ RowStats row_stats(const NormBwdArgs& a, int64_t row) {
    RowStats r{0.f, 0.f};
    if (row < a.rows) {
        if constexpr (OP == kLayerNorm) r.mean = a.mean[row];
        r.rstd = a.rstd[row];
    }
    return r;
}

// xh of a pair.  The mean is subtracted before the product: where a row's
// deviation is far below its mean, h rstd - mean rstd would keep the product's
// rounding.
template <int OP> __device__ __forceinline__ F2 normalised(F2 h, RowStats r) {
    return mul2(OP == kLayerNorm ? add2(h, f2(-r.mean)) : h, f2(r.rstd));
}

// Sums of a tile: s1 += w xh, s2 += w; and the columns' gradients.
template <int OP, int NP>
__device__ __forceinline__ void tile_sums(const F2* dy, const F2* h, const F2* g, RowStats r,
                                          F2& s1, F2& s2, F2* ag, F2* ab) {
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const F2 t = mul2(dy[k], normalised<OP>(h[k], r));
        ag[k] = add2(ag[k], t);
        s1 = fma2(t, g[k], s1);
        if constexpr (OP == kLayerNorm) {
            s2 = fma2(dy[k], g[k], s2);
            ab[k] = add2(ab[k], dy[k]);
        }
    }
}

// A row's dtot = w rstd + (c - xh b): what the two means make of it.
struct RowBack {
    float rstd, b, c;  // b = rstd mean_j(w xh), c = -rstd mean_j(w)
    __device__ RowBack(RowStats r, float m1, float m2) : rstd(r.rstd), b(r.rstd * m1), c(-r.rstd * m2) {}
};

// dtot of a tile from its row's two means, then the outputs; dx and dres point
// at the lane's first column, the tile lies `off` further, at column `base`.
// `on`: draw the mask (all 32 lanes call).
template <int OP, typename T, typename IO, bool FULL>
__device__ __forceinline__ void tile_out(const DropStream& d, const F2* dy, const F2* h,
                                         const F2* g, bool has_dh, const F2* dh, RowStats r,
                                         RowBack q, int64_t row, int base, int off, int left,
                                         int lane, bool on, T* dx, T* dres) {
    F2 v[IO::NP];
#pragma unroll
    for (int k = 0; k < IO::NP; ++k) {
        const F2 xh = normalised<OP>(h[k], r);
        F2 t = OP == kLayerNorm ? fma2(xh, f2(-q.b), f2(q.c)) : mul2(xh, f2(-q.b));
        if (has_dh) t = add2(t, dh[k]);
        v[k] = fma2(mul2(dy[k], g[k]), f2(q.rstd), t);
    }
    if (dres) IO::template store<FULL>(dres, off, left, v);
    if (on) {
        IO::drop(d, base, lane, (uint32_t)row, v);
#pragma unroll
        for (int k = 0; k < IO::NP; ++k) v[k] = mul2(v[k], f2(d.a.scale));
    }
    IO::template store<FULL>(dx, off, left, v);
}

// The group's sums of a thread's columns, to its workspace row; j0 is the
// lane's first column.
template <int OP, typename IO>
__device__ __forceinline__ void tile_params(const NormBwdArgs& a, int64_t group, int j0, int off,
                                            int left, const F2* ag, const F2* ab) {
    float* p = a.pws + group * 2 * a.pitch + j0;
    if (a.dgamma) IO::template store_sums<false>(p, off, left, ag);
    if (OP == kLayerNorm && a.dbeta) IO::template store_sums<false>(p + a.pitch, off, left, ab);
}

// ------------------------------------------------------------- one warp a row
template <int OP, typename T, typename IO, typename PT, int V>
__global__ void __launch_bounds__(kThreads) bwd_warp(NormBwdArgs a) {
    constexpr int kCols = V * IO::kTile;
    __shared__ float sums[2][kCols];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l0 = IO::first(lane), left = a.cols - l0;
    const DropStream d(a.drop);
    const T* const dyp = static_cast<const T*>(a.dy) + l0;
    const T* const hp = static_cast<const T*>(a.h) + l0;
    const T* const dhp = moved(static_cast<const T*>(a.dh), l0);
    const PT* const gp = moved(static_cast<const PT*>(a.gamma), l0);
    const int64_t step = (int64_t)gridDim.x * kWarps;
    int64_t row = (int64_t)blockIdx.x * kWarps + warp;
    F2 g[V][IO::NP], ag[V][IO::NP], ab[V][IO::NP];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        IO::template params<false>(gp, i * IO::kTile, left, g[i], 1.f);
#pragma unroll
        for (int k = 0; k < IO::NP; ++k) ag[i][k] = ab[i][k] = f2(0.f);
    }
    typename IO::R yv[V], hv[V], rv[V];
    auto fetch = [&](int64_t at) {
        if (at >= a.rows) return;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            yv[i] = IO::template load<false>(dyp + at * a.cols, i * IO::kTile, left);
            hv[i] = IO::template load<false>(hp + at * a.cols, i * IO::kTile, left);
            if (dhp) rv[i] = IO::template load<false>(dhp + at * a.cols, i * IO::kTile, left);
        }
    };
    fetch(row);
    RowStats next = row_stats<OP>(a, row);
    while (row < a.rows) {
        const RowStats r = next;
        F2 u[V][IO::NP], h[V][IO::NP], dh[V][IO::NP], s1 = f2(0.f), s2 = f2(0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            unpack<T, IO::NP>(yv[i], u[i]);
            unpack<T, IO::NP>(hv[i], h[i]);
            if (dhp) unpack<T, IO::NP>(rv[i], dh[i]);
        }
        const int64_t now = row;
        row += step;
        fetch(row);  // in flight while this row is reduced and written
        next = row_stats<OP>(a, row);
#pragma unroll
        for (int i = 0; i < V; ++i)
            tile_sums<OP, IO::NP>(u[i], h[i], g[i], r, s1, s2, ag[i], ab[i]);
        const float c1 = warp_allreduce(s1.x + s1.y, SumOp()) * a.inv_cols;
        const float c2 =
            OP == kLayerNorm ? warp_allreduce(s2.x + s2.y, SumOp()) * a.inv_cols : 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            tile_out<OP, T, IO, false>(d, u[i], h[i], g[i], dhp != nullptr, dh[i], r, RowBack(r, c1, c2), now,
                                       i * IO::kTile, i * IO::kTile, left, lane,
                                       a.drop.on && i * IO::kTile < a.cols,
                                       static_cast<T*>(a.dx) + now * a.cols + l0,
                                       moved(static_cast<T*>(a.dres), now * a.cols + l0));
    }
    // the CTA's warps add their sums in warp order
    for (int j = threadIdx.x; j < kCols; j += kThreads) sums[0][j] = sums[1][j] = 0.f;
    for (int w = 0; w < kWarps; ++w) {
        __syncthreads();
        if (w != warp) continue;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < IO::N; ++k) {
                const int j = i * IO::kTile + l0 + IO::at(k);
                sums[0][j] += k & 1 ? ag[i][k / 2].y : ag[i][k / 2].x;
                if constexpr (OP == kLayerNorm) sums[1][j] += k & 1 ? ab[i][k / 2].y : ab[i][k / 2].x;
            }
    }
    __syncthreads();
    float* p = a.pws + (int64_t)blockIdx.x * 2 * a.pitch;
    for (int j = threadIdx.x; j < a.cols; j += kThreads) {
        if (a.dgamma) p[j] = sums[0][j];
        if (OP == kLayerNorm && a.dbeta) p[a.pitch + j] = sums[1][j];
    }
}

// Two sums over the warp: lanes 0-15 return the first, lanes 16-31 the second.
__device__ __forceinline__ float two_sums(float a, float b, int lane) {
    const float t[2] = {a, b};
    return row_sum<2>(t, lane);
}

// ------------------------------------------------- a CTA or a cluster per row
// Warp w of a CTA owns the V tiles from column c0 + 128 V w on.  The rows are
// pipelined: an iteration sums row k and writes row k - 1, whose sums were
// merged (and exchanged with the cluster) meanwhile, with one barrier between
// iterations; so a stage is read in two iterations and its row's sums are
// never waited for at once.
template <int OP, typename T, typename IO, typename PT, int V>
__global__ void __launch_bounds__(kRingThreads) bwd_ring(NormBwdArgs a, RingShape q) {
    constexpr bool kHeld = V == 4;  // gamma stays in registers
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ __align__(8) uint64_t full[kRingStages];
    __shared__ float wred[2][2][kRingWarps];
    __shared__ RingExchange ex;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
    const int part = lane & 15, which = lane >> 4;
    const uint32_t P = cluster_nctarank(), rank = cluster_ctarank();
    const int64_t first = blockIdx.x / P;
    const int c0 = (int)rank * q.tiles * IO::kTile;
    const int c1 = min(a.cols, c0 + q.tiles * IO::kTile);
    const int bytes = (c1 - c0) * (int)sizeof(T);
    const void* const src[3] = {a.dy, a.h, a.dh};
    const int ns = a.dh ? 3 : 2, stage_bytes = ns * q.room;

    layout_fits((uint64_t)q.stages * stage_bytes, q.stages, kRingStages, q.err);
    if (threadIdx.x == 0) {
        for (int s = 0; s < q.stages; ++s) mbar_init(smem_u32(&full[s]), 1);
        if (P > 1) ex.init(P);
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    __syncthreads();
    if (P > 1) {
        cluster_arrive_release();
        cluster_wait_acquire();
    }
    auto issue = [&](int64_t row, int s) {
        if (row < a.rows)
            ring_issue<3, 1, T, IO>(src, ns, row, a.rows, a.cols, c0, bytes, ring + s * stage_bytes,
                                    q.room, smem_u32(&full[s]));
    };
    const int feeder = W > 1;  // not the warp whose deposit a cluster waits for
    if (warp == feeder)
        for (int s = 0; s < q.stages; ++s) issue(first + (int64_t)s * q.clusters, s);

    const DropStream d(a.drop);
    const int base0 = c0 + warp * V * IO::kTile, j0 = base0 + IO::first(lane), left = c1 - j0;
    const bool whole = base0 + V * IO::kTile <= c1;
    const bool simple = !a.drop.on && !a.dres;  // dx is the only matrix written
    const PT* const gp = moved(static_cast<const PT*>(a.gamma), j0);
    T* dx = static_cast<T*>(a.dx) + first * a.cols + j0;
    T* dres = moved(static_cast<T*>(a.dres), first * a.cols + j0);
    F2 held[kHeld ? V : 1][IO::NP], ag[V][IO::NP], ab[V][IO::NP];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (kHeld) IO::template params<false>(gp, i * IO::kTile, left, held[kHeld ? i : 0], 1.f);
#pragma unroll
        for (int e = 0; e < IO::NP; ++e) ag[i][e] = ab[i][e] = f2(0.f);
    }
    // gamma of tile i
    auto weight = [&](auto f, int i, F2 (&g)[IO::NP]) {
        if constexpr (kHeld) {
#pragma unroll
            for (int e = 0; e < IO::NP; ++e) g[e] = held[i][e];
        } else {
            IO::template params<decltype(f)::value>(gp, i * IO::kTile, left, g, 1.f);
        }
    };
    // stream i's slice of a row in a stage, at the lane's first column
    auto slice = [&](const unsigned char* stage, int i, const void* p, int64_t row) {
        const int64_t off = (row * a.cols + c0) * (int64_t)sizeof(T);
        return reinterpret_cast<const T*>(stage + i * q.room + ring_shift<IO>(p, off)) + (j0 - c0);
    };
    const uint32_t turns = (uint32_t)((a.rows - first + q.clusters - 1) / q.clusters);
    const int64_t stride = (int64_t)q.clusters * a.cols;
    RowStats next = row_stats<OP>(a, first), prev{0.f, 0.f};
    const float* mp = OP == kLayerNorm ? a.mean + first : nullptr;
    const float* rp = a.rstd + first;
    int64_t row = first;  // of turn k
    int s = 0, sp = 0;
    uint32_t phase = 0;
    const std::true_type yes;
    const std::false_type no;
    for (uint32_t k = 0;; ++k) {
        const RowStats r = next;
        if (k < turns) {
            if (k + 1 < turns) {
                rp += q.clusters;
                next.rstd = *rp;
                if constexpr (OP == kLayerNorm) {
                    mp += q.clusters;
                    next.mean = *mp;
                }
            }
            const unsigned char* const stage = ring + s * stage_bytes;
            mbar_wait_bounded(smem_u32(&full[s]), phase, q.err);
            const T* const ys = slice(stage, 0, a.dy, row);
            const T* const hs = slice(stage, 1, a.h, row);
            F2 s1 = f2(0.f), s2 = f2(0.f);
            auto take = [&](auto f) {
                constexpr bool FULL = decltype(f)::value;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    F2 u[IO::NP], h[IO::NP], g[IO::NP];
                    unpack<T, IO::NP>(IO::template staged<FULL>(ys, i * IO::kTile, left), u);
                    unpack<T, IO::NP>(IO::template staged<FULL>(hs, i * IO::kTile, left), h);
                    weight(f, i, g);
                    tile_sums<OP, IO::NP>(u, h, g, r, s1, s2, ag[i], ab[i]);
                }
            };
            if (whole) take(yes); else take(no);
            const float v = two_sums(s1.x + s1.y, s2.x + s2.y, lane);
            if (part == 0) wred[k & 1][which][warp] = v;
        }
        if (k > 0) {  // the row before
            float v;
            if (P > 1) {
                const float4* parts = ex.wait(k - 1, P, rank, q.err);
                v = part < (int)P ? (which ? parts[part].y : parts[part].x) : 0.f;
            } else {
                v = part < W ? wred[(k - 1) & 1][which][part] : 0.f;
            }
            float t[2];
            spread<2>(half_sum(v) * a.inv_cols, lane, t);
            const RowBack back(prev, t[0], t[1]);
            const int64_t at = row - q.clusters;
            const unsigned char* const stage = ring + sp * stage_bytes;
            const T* const ys = slice(stage, 0, a.dy, at);
            const T* const hs = slice(stage, 1, a.h, at);
            const T* const ds = slice(stage, 2, a.dh, at);
            // (the conditions that hold for the whole call are constants of the
            // tiles' code: as predicates they cost as much as the work)
            auto give = [&](auto f, auto has_dh, auto plain) {
                constexpr bool FULL = decltype(f)::value;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    F2 u[IO::NP], h[IO::NP], g[IO::NP], dh[IO::NP];
                    unpack<T, IO::NP>(IO::template staged<FULL>(ys, i * IO::kTile, left), u);
                    unpack<T, IO::NP>(IO::template staged<FULL>(hs, i * IO::kTile, left), h);
                    if (has_dh)
                        unpack<T, IO::NP>(IO::template staged<FULL>(ds, i * IO::kTile, left), dh);
                    weight(f, i, g);
                    tile_out<OP, T, IO, FULL>(
                        d, u, h, g, has_dh, dh, prev, back, at, base0 + i * IO::kTile, i * IO::kTile,
                        left, lane, !plain && a.drop.on && (FULL || base0 + i * IO::kTile < c1), dx,
                        plain ? nullptr : dres);
                }
            };
            if (!whole) give(no, ns > 2, no);
            else if (ns > 2) simple ? give(yes, yes, yes) : give(yes, yes, no);
            else simple ? give(yes, no, yes) : give(yes, no, no);
            dx += stride;
            if (dres) dres += stride;
        }
        if (k == turns) break;
        __syncthreads();
        // every thread has left row k - 1: refill its stage
        if (warp == feeder && k > 0) issue(row + (int64_t)(q.stages - 1) * q.clusters, sp);
        if (P > 1 && warp == 0) {
            float t[2];
            spread<2>(half_sum(part < W ? wred[k & 1][which][part] : 0.f), lane, t);
            ex.deposit(k, make_float4(t[0], t[1], 0.f, 0.f), P, rank);
        }
        prev = r;
        row += q.clusters;
        sp = s;
        if (++s == q.stages) {
            s = 0;
            phase ^= 1u;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        tile_params<OP, IO>(a, first, j0, i * IO::kTile, left, ag[i], ab[i]);
    if (P > 1) {  // no CTA leaves while a peer's deposit to it may be in flight
        cluster_arrive_release();
        cluster_wait_acquire();
    }
}

// ------------------------------------------------------------- a team per row
// team.cuh's pipeline: a summing and a writing warp own four tiles of the
// slice each, gamma (and the columns' sums) in registers.
template <int OP, typename T, typename IO, typename PT>
__global__ void __launch_bounds__(kTeamThreads) bwd_team(NormBwdArgs a, TeamShape q) {
    constexpr int V = 4;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ __align__(8) TeamBars bars;
    __shared__ float wred[kTeamStages][2][kTeamWarps];
    __shared__ float2 tot[kTeamStages];  // mean_j(w xh), mean_j(w)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = (blockDim.x >> 6) - 1;
    const int team = (int)blockIdx.x / q.size, rank = (int)blockIdx.x - team * q.size;
    const int c0 = rank * q.tiles * IO::kTile, c1 = min(a.cols, c0 + q.tiles * IO::kTile);
    const int bytes = (c1 - c0) * (int)sizeof(T);
    const void* const src[3] = {a.dy, a.h, a.dh};
    const int ns = a.dh ? 3 : 2, stage_bytes = ns * q.room;
    const int turns = (int)((a.rows - team + q.teams - 1) / q.teams);
    auto row_of = [&](int k) { return team + (int64_t)k * q.teams; };

    layout_fits((uint64_t)q.stages * stage_bytes, q.stages, kTeamStages, q.err);
    bars.init(q.stages, W);

    if (warp == 2 * W) {  // collects
        TeamExchange(q, team, rank, lane).collect(
            turns, q.stages, bars,
            [&](const float* x, const float* y) {
                float t1 = 0.f, t2 = 0.f;
#pragma unroll
                for (int i = 0; i < kTeamParts; ++i) {
                    t1 += x[i];
                    t2 += y[i];
                }
                t1 = warp_allreduce(t1, SumOp()) * a.inv_cols;
                return make_float2(t1, warp_allreduce(t2, SumOp()) * a.inv_cols);
            },
            [&](int, int st, float2 m) {
                if (lane == 0) tot[st] = m;
            });
        return;
    }
    if (warp == 2 * W + 1) {  // serves
        const TeamExchange ex(q, team, rank, lane);
        const int part = lane & 15, which = lane >> 4;
        bars.serve(
            turns, q.stages, q.err,
            [&](int k, int st) {
                ring_issue<3, 1, T, IO>(src, ns, row_of(k), a.rows, a.cols, c0, bytes,
                                        ring + st * stage_bytes, q.room, smem_u32(&bars.fed[st]));
                __syncwarp();
            },
            [&](int k, int st) {
                float v[2];
                spread<2>(half_sum(part < W ? wred[st][which][part] : 0.f), lane, v);
                ex.deposit(k, v[0], v[1]);
            });
        return;
    }

    TeamTurn t;
    const bool summing = warp < W;
    const int base0 = c0 + (summing ? warp : warp - W) * V * IO::kTile;
    const int j0 = base0 + IO::first(lane), left = c1 - j0;
    const bool whole = base0 + V * IO::kTile <= c1;
    const PT* const gp = moved(static_cast<const PT*>(a.gamma), j0);
    F2 g[V][IO::NP];
#pragma unroll
    for (int i = 0; i < V; ++i) IO::template params<false>(gp, i * IO::kTile, left, g[i], 1.f);
    auto slice = [&](int s, int i, const void* p, int64_t row) {
        const int64_t off = (row * a.cols + c0) * (int64_t)sizeof(T);
        return reinterpret_cast<const T*>(ring + s * stage_bytes + i * q.room +
                                          ring_shift<IO>(p, off)) + (j0 - c0);
    };
    RowStats next = row_stats<OP>(a, row_of(0));
    const std::true_type yes;
    const std::false_type no;
    // row k's stage is here; the next row's statistics are on their way
    auto enter = [&](int k) {
        const RowStats r = next;
        if (k + 1 < turns) next = row_stats<OP>(a, row_of(k + 1));
        bars.wait(bars.fed[t.s], t, q.err);
        return r;
    };
    if (summing) {
        F2 ag[V][IO::NP], ab[V][IO::NP];
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < IO::NP; ++e) ag[i][e] = ab[i][e] = f2(0.f);
        for (int k = 0; k < turns; ++k, t.next(q.stages)) {
            const RowStats r = enter(k);
            const T* const ys = slice(t.s, 0, a.dy, row_of(k));
            const T* const hs = slice(t.s, 1, a.h, row_of(k));
            F2 s1 = f2(0.f), s2 = f2(0.f);
            auto take = [&](auto f) {
                constexpr bool FULL = decltype(f)::value;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    F2 u[IO::NP], h[IO::NP];
                    unpack<T, IO::NP>(IO::template staged<FULL>(ys, i * IO::kTile, left), u);
                    unpack<T, IO::NP>(IO::template staged<FULL>(hs, i * IO::kTile, left), h);
                    tile_sums<OP, IO::NP>(u, h, g[i], r, s1, s2, ag[i], ab[i]);
                }
            };
            if (whole) take(yes); else take(no);
            const float v[2] = {s1.x + s1.y, s2.x + s2.y};
            const float sum = row_sum<2>(v, lane);
            if ((lane & 15) == 0) wred[t.s][lane >> 4][warp] = sum;
            TeamBars::done(bars.summed[t.s]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            tile_params<OP, IO>(a, team, j0, i * IO::kTile, left, ag[i], ab[i]);
        return;
    }
    const DropStream d(a.drop);
    const bool simple = !a.drop.on && !a.dres;  // dx is the only matrix written
    for (int k = 0; k < turns; ++k, t.next(q.stages)) {
        const int64_t at = row_of(k);
        const RowStats r = enter(k);
        bars.wait(bars.known[t.s], t, q.err);
        const float2 m = tot[t.s];
        const RowBack back(r, m.x, m.y);
        const T* const ys = slice(t.s, 0, a.dy, at);
        const T* const hs = slice(t.s, 1, a.h, at);
        const T* const ds = slice(t.s, 2, a.dh, at);
        T* const dx = static_cast<T*>(a.dx) + at * a.cols + j0;
        T* const dres = moved(static_cast<T*>(a.dres), at * a.cols + j0);
        auto give = [&](auto f, auto has_dh, auto plain) {
            constexpr bool FULL = decltype(f)::value;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                F2 u[IO::NP], h[IO::NP], dh[IO::NP];
                unpack<T, IO::NP>(IO::template staged<FULL>(ys, i * IO::kTile, left), u);
                unpack<T, IO::NP>(IO::template staged<FULL>(hs, i * IO::kTile, left), h);
                if (has_dh)
                    unpack<T, IO::NP>(IO::template staged<FULL>(ds, i * IO::kTile, left), dh);
                tile_out<OP, T, IO, FULL>(
                    d, u, h, g[i], has_dh, dh, r, back, at, base0 + i * IO::kTile, i * IO::kTile,
                    left, lane, !plain && a.drop.on && (FULL || base0 + i * IO::kTile < c1), dx,
                    plain ? nullptr : dres);
            }
        };
        if (!whole) give(no, ns > 2, no);
        else if (ns > 2) simple ? give(yes, yes, yes) : give(yes, yes, no);
        else simple ? give(yes, no, yes) : give(yes, no, no);
        TeamBars::done(bars.written[t.s]);
    }
}

// ------------------------------------------------------------- wider rows
// One launch of sweep.cuh: the two row sums of one batch, outputs of the batch
// before and its rows' part of the parameters' gradients, which the blocks of
// one (strip, group) add up from batch to batch.
template <int OP, typename T, typename IO, typename PT>
__global__ void __launch_bounds__(kSweepThreads, kSweepCtas) bwd_sweep(NormBwdArgs a, Sweep q) {
    constexpr int kChunk = sweep_chunk(IO::N), kStrip = sweep_strip(IO::N);
    __shared__ float part[2][2 * kSweepRows][kSweepWarps];
    __shared__ float4 rowc[kSweepGroup];  // mean, rstd, mean_j(w xh), mean_j(w)
    wait_for_previous_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float2* const ws = reinterpret_cast<float2*>(a.ws);
    uint32_t index;
    if (sweep_sums(q, blockIdx.x, &index)) {
        const int chunk = (int)(index % (uint32_t)a.nch);
        const int64_t r0 = q.s0 + (int64_t)(index / (uint32_t)a.nch) * kSweepGroup;
        const int64_t r1 = min(q.s1, r0 + kSweepGroup);
        const int j0 = chunk * kChunk + warp * kSweepTiles * IO::kTile + IO::first(lane);
        const int left = a.cols - j0;
        const T* const dyp = static_cast<const T*>(a.dy) + j0;
        const T* const hp = static_cast<const T*>(a.h) + j0;
        F2 g[kSweepTiles][IO::NP];
#pragma unroll
        for (int i = 0; i < kSweepTiles; ++i)
            IO::template params<false>(moved(static_cast<const PT*>(a.gamma), j0), i * IO::kTile,
                                       left, g[i], 1.f);
        int turn = 0;
        for (int64_t r = r0; r < r1; r += kSweepRows, turn ^= 1) {
            typename IO::R yv[kSweepRows][kSweepTiles], hv[kSweepRows][kSweepTiles];
            RowStats st[kSweepRows];
            float v[2 * kSweepRows];
#pragma unroll
            for (int j = 0; j < kSweepRows; ++j) {
                const int64_t row = min(r + j, r1 - 1);  // past the group: its last row
                st[j] = row_stats<OP>(a, row);
#pragma unroll
                for (int i = 0; i < kSweepTiles; ++i) {
                    yv[j][i] = IO::template load<false>(dyp + row * a.cols, i * IO::kTile, left);
                    hv[j][i] = IO::template load<false>(hp + row * a.cols, i * IO::kTile, left);
                }
            }
#pragma unroll
            for (int j = 0; j < kSweepRows; ++j) {
                F2 s1 = f2(0.f), s2 = f2(0.f);
#pragma unroll
                for (int i = 0; i < kSweepTiles; ++i) {
                    F2 u[IO::NP], h[IO::NP];
                    unpack<T, IO::NP>(yv[j][i], u);
                    unpack<T, IO::NP>(hv[j][i], h);
#pragma unroll
                    for (int e = 0; e < IO::NP; ++e) {
                        const F2 w = mul2(u[e], g[i][e]);  // 0 past the row
                        s1 = fma2(w, normalised<OP>(h[e], st[j]), s1);
                        s2 = add2(s2, w);
                    }
                }
                v[2 * j] = s1.x + s1.y;
                v[2 * j + 1] = s2.x + s2.y;
            }
            constexpr int G = 32 / (2 * kSweepRows);
            const float sum = sums_over_warp<2 * kSweepRows>(v, lane);
            if (lane % G == 0) part[turn][lane / G][warp] = sum;
            __syncthreads();
            if (threadIdx.x < kSweepRows && r + threadIdx.x < r1) {
                float2 t = make_float2(0.f, 0.f);
                for (int k = 0; k < kSweepWarps; ++k) {
                    t.x += part[turn][2 * threadIdx.x][k];
                    t.y += part[turn][2 * threadIdx.x + 1][k];
                }
                ws[(r + threadIdx.x) * a.nch + chunk] = t;
            }
        }
        return;
    }
    const DropStream d(a.drop);
    const int strips = (a.cols + kStrip - 1) / kStrip, strip = (int)(index % (uint32_t)strips);
    const int group = (int)(index / (uint32_t)strips);
    const int64_t r0 = q.b0 + (int64_t)group * kSweepGroup;
    const int nr = (int)(min(q.b1, r0 + kSweepGroup) - r0);
    for (int i = warp; i < nr; i += kSweepWarps) {
        const float2* w = ws + (r0 + i) * a.nch;
        float s1 = 0.f, s2 = 0.f;
        for (int c = lane; c < a.nch; c += 32) {
            const float2 t = __ldcg(w + c);
            s1 += t.x;
            s2 += t.y;
        }
        s1 = warp_allreduce(s1, SumOp());
        s2 = warp_allreduce(s2, SumOp());
        const RowStats st = row_stats<OP>(a, r0 + i);
        if (lane == 0) rowc[i] = make_float4(st.mean, st.rstd, s1 * a.inv_cols, s2 * a.inv_cols);
    }
    __syncthreads();
    const int base = strip * kStrip + warp * IO::kTile;
    if (base >= a.cols) return;
    const int j0 = base + IO::first(lane), left = a.cols - j0;
    F2 g[IO::NP], ag[IO::NP], ab[IO::NP];
    IO::template params<false>(moved(static_cast<const PT*>(a.gamma), j0), 0, left, g, 1.f);
#pragma unroll
    for (int e = 0; e < IO::NP; ++e) ag[e] = ab[e] = f2(0.f);
    for (int i = 0; i < nr; i += kSweepRows) {
        typename IO::R yv[kSweepRows], hv[kSweepRows], dv[kSweepRows];
#pragma unroll
        for (int j = 0; j < kSweepRows; ++j) {
            const int64_t at = (r0 + min(i + j, nr - 1)) * a.cols + j0;
            yv[j] = IO::template load<false>(static_cast<const T*>(a.dy) + at, 0, left);
            hv[j] = IO::template load<false>(static_cast<const T*>(a.h) + at, 0, left);
            if (a.dh) dv[j] = IO::template load<false>(static_cast<const T*>(a.dh) + at, 0, left);
        }
#pragma unroll
        for (int j = 0; j < kSweepRows; ++j) {
            if (i + j >= nr) break;
            const int64_t at = (r0 + i + j) * a.cols + j0;
            const float4 c = rowc[i + j];
            const RowStats st{c.x, c.y};
            F2 u[IO::NP], h[IO::NP], dh[IO::NP], s1 = f2(0.f), s2 = f2(0.f);
            unpack<T, IO::NP>(yv[j], u);
            unpack<T, IO::NP>(hv[j], h);
            if (a.dh) unpack<T, IO::NP>(dv[j], dh);
            tile_sums<OP, IO::NP>(u, h, g, st, s1, s2, ag, ab);
            tile_out<OP, T, IO, false>(d, u, h, g, a.dh != nullptr, dh, st, RowBack(st, c.z, c.w),
                                       r0 + i + j, base, 0, left, lane, a.drop.on,
                                       static_cast<T*>(a.dx) + at,
                                       moved(static_cast<T*>(a.dres), at));
        }
    }
    // the earlier batches' sums of these columns, then this one's
    float* const p = a.pws + (int64_t)group * 2 * a.pitch + j0;
    if (!q.first) {
        if (a.dgamma) IO::add_sums(p, left, ag);
        if (OP == kLayerNorm && a.dbeta) IO::add_sums(p + a.pitch, left, ab);
    }
    tile_params<OP, IO>(a, group, j0, 0, left, ag, ab);
}

__device__ __forceinline__ void store_param(void* p, bool half, int64_t j, float v) {
    if (half) static_cast<bf16*>(p)[j] = Elem<bf16>::from_f(v);
    else static_cast<float*>(p)[j] = v;
}

// dgamma (blockIdx.y 0) and dbeta (1): the groups' sums.  A warp adds groups
// w, w + kWarps, ... of 128 columns, the CTA's warps are added in order.
__global__ void __launch_bounds__(kThreads) bwd_params(NormBwdArgs a) {
    __shared__ float4 part[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    void* const out = blockIdx.y ? a.dbeta : a.dgamma;
    if (!out) return;
    const int j = (int)blockIdx.x * 128 + 4 * lane;  // below the pitch, a multiple of 128
    const float* p = a.pws + (blockIdx.y ? a.pitch : 0) + j;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int q = warp; q < a.groups; q += kWarps) {
        const float4 v = *reinterpret_cast<const float4*>(p + (int64_t)q * 2 * a.pitch);
        t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
    }
    part[warp][lane] = t;
    __syncthreads();
    if (threadIdx.x < 128) {
        const int c = (int)blockIdx.x * 128 + threadIdx.x;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            v += reinterpret_cast<const float*>(part[w])[threadIdx.x];
        if (c < a.cols) store_param(out, a.half, c, v);
    }
}

template <int OP, typename T, typename IO, typename PT, int V>
cudaError_t run_warp(const NormBwdArgs& a, cudaStream_t s) {
    bwd_warp<OP, T, IO, PT, V><<<(unsigned)a.groups, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

// WarpIO, IO and WIO: the access forms of the warp kernels, of the ring and team
// kernels and of the sweep.
template <int OP, typename T, typename WarpIO, typename IO, typename WIO, typename PT>
cudaError_t run_bwd(NormBwdArgs& a, int sms, cudaStream_t s) {
    const int tiles = (a.cols + IO::kTile - 1) / IO::kTile;
    if (tiles <= 1) return run_warp<OP, T, WarpIO, PT, 1>(a, s);
    if (tiles <= 2) return run_warp<OP, T, WarpIO, PT, 2>(a, s);
    if (tiles <= 4) return run_warp<OP, T, WarpIO, PT, 4>(a, s);
    const int streams = a.dh ? 3 : 2;
    TeamPlan team;
    switch (form_of(tiles, sizeof(T), streams, a.rows, a.cols, sms, &team)) {
        case Form::kTeam:
            a.groups = team.teams;  // at most the layout's
            return launch_team((const void*)bwd_team<OP, T, IO, PT>, a, team, a.ws, s);
        case Form::kSweep:
            return run_sweep((const void*)bwd_sweep<OP, T, WIO, PT>, a, a.batch, WIO::N, s);
        default: break;
    }
    const RingKernels fn{(const void*)bwd_ring<OP, T, IO, PT, 4>, nullptr,
                         (const void*)bwd_ring<OP, T, IO, PT, 8>};
    RingPlan p;
    int resident;
    unsigned* err;
    if (!plan_ring(tiles, sizeof(T), streams, 1, a.rows, sms, fn, &p, &resident, &err))
        return cudaErrorInvalidConfiguration;
    a.groups = ring_grid(p, resident, a.rows);  // at most the layout's
    return launch_ring(fn.of(p), a, p, a.groups, err, s);
}

template <int OP, typename T, typename WarpIO, typename IO, typename WIO>
cudaError_t pick_param(NormBwdArgs& a, int sms, cudaStream_t s) {
    return a.half ? run_bwd<OP, T, WarpIO, IO, WIO, bf16>(a, sms, s)
                  : run_bwd<OP, T, WarpIO, IO, WIO, float>(a, sms, s);
}

template <int OP, typename T>
cudaError_t pick_bwd(TrainKey k, NormBwdArgs& a, int sms, cudaStream_t s) {
    constexpr int N = 16 / (int)sizeof(T);
    // fp32 slices in shared memory are read an element a lane even where the rows
    // are whole lines: 2048 x 10000 LayerNorm 60 us with four columns a lane, 47
    // with one; 4096 x 8192 92 and 69, 1024 x 32768 89 and 79, 512 x 262144 335
    // and 289 (bf16 rows the other way round: 2048 x 10000 39 and 45)
    using RingIO = std::conditional_t<sizeof(T) == 4, ElemIO<T, 4>, VecIO<T, 4>>;
    return k.vec ? pick_param<OP, T, VecIO<T, 4>, RingIO, VecIO<T, N>>(a, sms, s)
                 : pick_param<OP, T, ElemIO<T, 4>, ElemIO<T, 4>, ElemIO<T, N>>(a, sms, s);
}


}  // namespace

namespace {

TrainLayout bwd_layout(int dtype, int64_t rows, int64_t cols, int sms, int l2_bytes) {
    TrainLayout l{};
    const int es = dtype == 0 ? 4 : 2;
    l.pitch = (int)((cols + kTileCols - 1) / kTileCols * kTileCols);
    l.nch = train_chunks(dtype, cols);
    if (rows == 0) return l;
    const int tiles = l.pitch / kTileCols;
    if (tiles <= 4) {  // one warp per row
        const int64_t want = (rows + kWarps - 1) / kWarps;
        l.groups = l.room_groups = (int)(want < sms * 2 ? want : sms * 2);
        return l;
    }
    // which form runs depends on the call's streams too: room for either
    l.batch = sweep_batch(rows, cols * 2 * es, l2_bytes);
    l.groups = (int)((std::min(rows, l.batch) + kSweepGroup - 1) / kSweepGroup);
    for (int streams = 2; streams <= 3; ++streams) {
        TeamPlan team;
        switch (form_of(tiles, es, streams, rows, cols, sms, &team)) {
            case Form::kTeam:
                l.room_groups = std::max(l.room_groups, team.teams);
                l.partials = std::max(l.partials, team.exchange_bytes);
                break;
            case Form::kSweep:
                l.room_groups = std::max(l.room_groups, l.groups);
                l.partials = std::max(l.partials, rows * l.nch * 8);
                break;
            default:
                l.room_groups = (int)std::max<int64_t>(
                    l.room_groups, ring_groups_bound(tiles, es, streams, rows, sms));
        }
    }
    return l;
}

}  // namespace

TrainLayout norm_bwd_layout(int dtype, int64_t rows, int64_t cols, int sms, int l2_bytes) {
    // the last shape's answer, as a training step asks for few shapes in turn
    struct Known { int dtype, sms, l2; int64_t rows, cols; TrainLayout l; };
    static thread_local Known known[8] = {};
    Known& k = known[(uint64_t)(rows * 31 + cols * 7 + dtype) % 8];
    if (k.sms == sms && k.l2 == l2_bytes && k.dtype == dtype && k.rows == rows && k.cols == cols) return k.l;
    k = Known{dtype, sms, l2_bytes, rows, cols, bwd_layout(dtype, rows, cols, sms, l2_bytes)};
    return k.l;
}

cudaError_t launch_norm_bwd(TrainKey k, NormBwdArgs a, int sms, cudaStream_t s) {
    if (a.rows > 0) {
        cudaError_t e;
        if (k.op == kLayerNorm)
            e = k.dtype == 0 ? pick_bwd<kLayerNorm, float>(k, a, sms, s)
                             : pick_bwd<kLayerNorm, bf16>(k, a, sms, s);
        else
            e = k.dtype == 0 ? pick_bwd<kRMSNorm, float>(k, a, sms, s)
                             : pick_bwd<kRMSNorm, bf16>(k, a, sms, s);
        if (e != cudaSuccess) return e;
    }
    if (a.dgamma || a.dbeta) {
        bwd_params<<<dim3((unsigned)(a.pitch / kTileCols), a.dbeta ? 2u : 1u), kThreads, 0, s>>>(a);
        return cudaGetLastError();
    }
    return cudaSuccess;
}

}  // namespace credit
