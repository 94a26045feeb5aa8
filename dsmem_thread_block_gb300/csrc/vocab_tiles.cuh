// vocab_tiles.cuh -- the tiled matrix products of the linear head's cross entropy:
// a persistent kernel whose CTAs, or pairs of CTAs, walk output tiles; a warp
// fills a ring of stages by tensor-map copies, a thread issues tcgen05 products
// into one of two accumulators in tensor memory, and eight warps (of a tile 256
// columns wide sixteen) read the other one out.
//
// Shapes.  A product of sixteen k takes 128 cycles whatever the tile's rows (64, 128)
// and columns (64 to 256) of a CTA alone, and 128 for 256 x 256 of a pair: narrow
// tiles pay only where there are too few wide ones for the SMs.  A pair stages half of
// B each, 32 KB a stage instead of 48, which is what keeps a large call at the tensor
// cores' rate.
//
// Measured (GB300, device time; the tensor pipe's share of cycles from ncu):
//   statistics 4096 x 4096 x 131072 bf16    2.23 to 2.42 ms  1970 to 1820 TFLOP/s (cuBLAS
//                                            burst 1901, sustained 1695)
//   gradient and products 4096 x 4096 x 65536  3.35 to 3.86 ms
//   the same called back to back            2.37 to 2.50 and 3.71 to 3.89 ms: power
//   the gradient in two terms               6.2 to 6.7 ms
//   32 x 1024 x 4096                        9.8 us forward, 64 tokens backward 20.9
//   512 x 2048 x 16384 fp32                 171 us, 55 of them packing; pipe 75 %
// What bounds the others: up to some 256 tokens the weight's read (64 x 4096 x 131072
// 180 us, 0.88 of the copy rate); short k the epilogue (2048 x 256 x 32768 43 to 51 us,
// some 2 us a tile of 256 columns); small calls one tile's latency (k / 16 products of 128
// cycles, then its epilogue).
//
// Precision.  The tensor cores add into an fp32 accumulator without rounding to
// nearest: a sum over k drifts towards zero by some 2^-25 of itself an addition of
// sixteen products, 7e-6 over 4096.  A product rounded to bf16 does not see that up to a
// k of 131072 (2^-12 of the terms' magnitude), and longer ones are summed in parts of that
// (kLongPart).  The logits do (one of 30 is off by 2e-4, and so is the gradient p - 1 of a token
// whose target is almost certain), and so do products of fp32 operands: there the
// accumulator holds kPromote stages at a time, and the epilogue warps add these
// parts in registers, which rounds to nearest; they do it while the next part is
// multiplied.
//
// The gradient of the logits is rounded to bf16 for the products of bf16 operands,
// divided by the significand of the largest dloss (vocab_unit).
// Each token's error is dominated by its target's, so of few tokens' some are large:
// up to 64 tokens, and where the caller asks for it, it takes two terms.  For dhidden
// they are rows of one product, whose sums are added behind (of 64 tokens the rows of
// one tile); for dweight a stage holds both terms of A beside one B.
//
// fp32 operands come as three bf16 terms, x = x0 + x1 + x2 to 24 bits.  Of their
// nine products six are formed; the others are below 2^-24 of x y.  A stage holds
// one term of both operands, so three stages in a row (terms 2, 1, 0) make a step of
// k and each term is loaded once.  The products take the order
//   x1 y1,  x2 y0, x0 y2 (term 2 is done),  x1 y0, x0 y1 (term 1),  x0 y0
// which lets the next step's terms in early: with four stages only, term 2 of the
// next step waits in the fourth, term 1 takes term 2's place half-way through, and
// term 0 is needed again a sixth into the next step.
#pragma once

#include <algorithm>
#include <type_traits>

#include "planner.h"
#include "rowops.cuh"
#include "tensor.cuh"
#include "vocab.h"

namespace credit {

// Warps of the epilogue: a quarter of them for each 32 of a tile's 128 rows, 64
// columns a warp.  (Eight for 256 columns left two of three issue slots empty.)
constexpr int vocab_warps(int columns) { return columns / kPartCols * 4; }
// whole warpgroups; one of the other four warps only waits
constexpr int vocab_threads(int columns) { return 32 * (vocab_warps(columns) + 4); }
// The sums of an epilogue thread (where they are kept in registers) take registers that
// the other four warps do not need: a thread of the epilogue's, one of the others', and
// what a thread has to have at launch for both to be there (a block that has fewer would
// wait for them forever): 96 of 640 threads, 166 of 384.
constexpr int vocab_regs(int columns) { return vocab_warps(columns) == 8 ? 208 : 104; }
constexpr int vocab_other_regs(int columns) { return vocab_warps(columns) == 8 ? 80 : 64; }
constexpr int vocab_launch_regs(int columns) {
    return (vocab_warps(columns) * vocab_regs(columns) + 4 * vocab_other_regs(columns) + vocab_warps(columns) + 3) /
           (vocab_warps(columns) + 4);
}
constexpr int kBoxBytes = 64 * kTileK * 2;      // one box of an operand with M or N innermost
constexpr int kBytesA = kTileM * kTileK * 2;
constexpr int kVocabRing = 6 * 32768;           // bytes of all stages
constexpr int kVocabStages = 16;                // most of them
constexpr int kTurnBytes = 32 * 64;             // a warp's room to turn its output around
constexpr int kVocabSmem = kVocabRing + 16 * kTurnBytes + 1024;  // aligned to 1024 by hand
// Stages of a part that is summed in registers.  Of 8, 4 and 2 a loss is off by 2.3e-7,
// 1.1e-7 and 0.7e-7 (plain fp32 products: 0.7e-7 to 2.4e-7), one of 4096 x 4096 x 131072
// takes 2155, 2230 and 2325 us, the gradient of 1000 x 1024 x 50000 192, 205 and 212.
constexpr int kPromote = 4;

// A tile is 128 rows a CTA by N columns (CG = 2: a pair shares the columns'
// operand, half of it each).
template <int N, int CG> struct TileShape {
    static constexpr int kRowsB = N / CG;       // of B a CTA stages
    static constexpr int kBytesB = kRowsB * kTileK * 2;
    static constexpr uint32_t kTmem = 2 * N;    // two accumulators
};

struct VocabBars {
    uint64_t full[kVocabStages], empty[kVocabStages], acc_full[2], acc_empty[2], drained;
};

// Wait for a phase; false once a wait of this CTA (or of its pair's, at the end) has
// given up.
__device__ __forceinline__ bool hold(uint32_t bar, uint32_t parity, unsigned* err,
                                     volatile int* dead) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
        if (*dead) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            atomicOr(err, kErrTimeout);
            *dead = 1;
            return false;
        }
    }
    return true;
}

// A tile of a launch: its product, corner and range of k.
struct Tile {
    int job, m0, n0, split, k0, kn;
};
__device__ __forceinline__ int tiles_of(const TileWork& w) { return w.mt * w.nt * w.splits; }

// Tile i of unit u (a CTA or a pair) of `units`.  The first product's tiles go
// round by round; units that get one less of them start `lead` rounds of the
// second product's before the others join.
template <int N, int CG>
__device__ __forceinline__ bool tile_at(const VocabArgs& a, int u, int units, int rank, int i, Tile* r) {
    const int n0 = tiles_of(a.work[0]), mine = n0 > u ? (n0 - u - 1) / units + 1 : 0;
    int t;
    r->job = i >= mine;
    if (!r->job) {
        t = u + i * units;
    } else {
        if (a.jobs < 2) return false;
        const int rest = n0 % units, j = i - mine, ahead = a.lead * (units - rest);
        t = u < rest ? ahead + j * units + u
                     : j < a.lead ? j * (units - rest) + u - rest : ahead + (j - a.lead) * units + u;
        if (t >= tiles_of(a.work[1])) return false;
    }
    const TileWork& w = a.work[r->job];
    const int per = w.mt * w.nt;
    r->split = t / per;
    t -= r->split * per;
    const int g = t / (w.group * w.nt);         // whole groups of tile rows
    t -= g * w.group * w.nt;
    const int rows = min(w.group, w.mt - g * w.group);
    const int n = t / rows;
    r->m0 = ((g * w.group + t - n * rows) * CG + rank) * kTileM;
    r->n0 = n * N;
    r->k0 = r->split * w.per;
    r->kn = min(w.per, w.kb - r->k0);
    return true;
}

// Where an operand's boxes of a stage lie: one box with K innermost, `boxes` of 64
// with M or N innermost.
template <int CG, int BOXES> struct Boxes {
    const CUtensorMap* map;
    int x, y, dx, dy;
    bool mn;
    __device__ Boxes(const CUtensorMap* m, bool mn_, int at, int y0, int k) : map(m), mn(mn_) {
        x = mn ? at : k * kTileK;
        y = mn ? k * kTileK + y0 : at + y0;
        dx = mn ? 0 : kTileK;
        dy = mn ? kTileK : 0;
    }
    __device__ __forceinline__ void load(int step, int term, uint32_t dst, uint32_t bar) const {
        const int u = x + step * dx, v = y + step * dy;
        tma_load_3d<CG>(dst, map, u, v, term, bar);
        if (BOXES > 1 && mn) {
#pragma unroll
            for (int j = 1; j < BOXES; ++j) tma_load_3d<CG>(dst + j * kBoxBytes, map, u + 64 * j, v, term, bar);
        }
    }
};

// The bf16 terms of a value x0 + x1 + x2: each is what is left of it rounded to
// bf16 (towards zero where that would be infinite); of a value that is not finite
// nothing is left.
__device__ __forceinline__ float first_term(float x) {
    const float hi = __bfloat162float(__float2bfloat16_rn(x));
    return isinf(hi) ? __uint_as_float(__float_as_uint(x) & 0xFFFF0000u) : hi;
}
__device__ __forceinline__ float rest_of(float x, float term) {
    return fabsf(x) <= 3.402823466e38f ? x - term : 0.f;
}

// ------------------------------------------------------------ the epilogues
// Each takes 32 columns of a warp's 32 rows at a time, from column c of the tile
// on: lane i holds those of row row0 + i.  What goes to memory is turned around in
// shared memory, so that consecutive lanes write consecutive columns.

// 32 rows of 64 bytes (32 bf16 or 16 fp32 elements); 16-byte vectors are permuted
// within a row so that both ways are free of bank conflicts.
struct Turn {
    unsigned char* room;
    int lane;
    __device__ __forceinline__ uint4* at(int row, int vec) const {
        return reinterpret_cast<uint4*>(room + row * 64) + (vec ^ ((row >> 1) & 3));
    }
    __device__ __forceinline__ void put(const uint32_t (&w)[16]) const {
        __syncwarp();   // the last block has been read
#pragma unroll
        for (int k = 0; k < 4; ++k) *at(lane, k) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        __syncwarp();
    }
    // f(row, vector of the row, its value): a lane's four vectors
    template <typename F> __device__ __forceinline__ void vectors(F f) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int row = lane / 4 + 8 * k, vec = lane % 4;
            f(row, vec, *at(row, vec));
        }
    }
    // f(row, element of the row, its value): a lane's elements, of type W
    template <typename W, typename F> __device__ __forceinline__ void elements(F f) const {
        constexpr int kRow = 64 / sizeof(W), kRows = 32 / kRow;  // of a row; rows at a time
#pragma unroll 4
        for (int r = 0; r < 32; r += kRows) {
            const int row = r + lane / kRow, e = lane % kRow;
            f(row, e, *(reinterpret_cast<const W*>(at(row, e * sizeof(W) / 16)) + e % (16 / sizeof(W))));
        }
    }
};
__device__ __forceinline__ void halves(const float (&g)[32], uint32_t (&w)[16]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = Pairs<bf16>::two(F2{g[2 * j], g[2 * j + 1]});
}

// A token's maximum and sum of exponentials over a warp's columns.
struct StatsOut {
    const VocabArgs& a;
    int64_t to;          // the target's column in the tile, if it lies there
    int left, row;
    bool live, any;      // the row, a row of the warp's
    float m = -INFINITY, s = 0.f;
    __device__ StatsOut(const VocabArgs& args, const Tile& t, int row0, unsigned char*) : a(args) {
        row = row0 + (threadIdx.x & 31);
        live = row < a.rows;
        any = row0 < a.rows;
        to = (live ? a.target[row] : -1) - a.v0 - t.n0;
        left = a.cols - t.n0;
    }
    __device__ __forceinline__ void take(int c, uint32_t (&v)[32]) {
        if (c >= left || !any) return;
        if (c + 32 > left) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (c + j >= left) v[j] = __float_as_uint(-INFINITY);
        }
        float t[4] = {m, m, m, m};
#pragma unroll
        for (int j = 0; j < 32; j += 2)
            t[j / 2 % 4] = fmaxf(t[j / 2 % 4], fmaxf(__uint_as_float(v[j]), __uint_as_float(v[j + 1])));
        const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
        // nothing is above an infinite maximum: exponents are then taken from zero
        const float base = isinf(top) ? 0.f : top;
        if (top != m) {
            s = s == 0.f ? 0.f : s * fast_ex2((m - base) * kLog2e);
            m = top;
        }
        // (base goes first: base log2(e), rounded, would be off by more than the maximum's
        // own term where logits are large, and leave that term below 1 where they are not)
        F2 sums[2] = {f2(0.f), f2(0.f)};
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            const F2 x = mul2(add2(F2{__uint_as_float(v[j]), __uint_as_float(v[j + 1])}, f2(-base)), f2(kLog2e));
            sums[j / 2 % 2] = add2(sums[j / 2 % 2], F2{fast_ex2(x.x), fast_ex2(x.y)});
        }
        const F2 both = add2(sums[0], sums[1]);
        s += both.x + both.y;
        if (to >= c && to < c + 32) {
            float z = 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (to == c + j) z = __uint_as_float(v[j]);
            if (in_bounds(live, a.err)) a.picked[row] = z;
        }
    }
    __device__ __forceinline__ void done(int part) {
        float2* const p = a.parts + (int64_t)part * a.rows + row;
        if (live && inside(p, sizeof(*p), a.parts, a.parts_room, a.err)) *p = make_float2(m, s);
    }
};

// The gradient of a token's logits, as bf16 terms.
template <VocabTerms TERMS> struct GradOut {
    const VocabArgs& a;
    int64_t to = -1;
    float scale = 0.f, both = 0.f, lse = 0.f;
    int rows;            // of the warp's that there are
    bool none;
    bf16* out;           // the warp's first row
    const Turn turn;
    __device__ GradOut(const VocabArgs& args, const Tile& t, int row0, unsigned char* room)
        : a(args), turn{room, (int)threadIdx.x & 31} {
        const int row = row0 + turn.lane;
        rows = a.rows - row0;
        if (row < a.rows) {
            const int64_t target = a.target[row];
            const bool ignored = target == a.ignore;
            scale = ignored ? 0.f : target < 0 || target >= a.vocab ? NAN : a.dloss[row];
            both = scale + (a.dlse ? a.dlse[row] : 0.f);
            lse = a.lse[row];
            if (TERMS == kTerms1) {
                const float unit = *a.unit;
                scale /= unit;
                both /= unit;
            }
            to = ignored ? -1 : target - a.v0 - t.n0;
        }
        none = both == 0.f;  // (its exponentials may be infinite)
        out = static_cast<bf16*>(a.grad) + (int64_t)row0 * a.grad_pitch + t.n0;
    }
    __device__ __forceinline__ void write(bf16* p, const float (&g)[32]) {
        uint32_t w[16];
        halves(g, w);
        turn.put(w);
        turn.vectors([&](int row, int vec, uint4 v) {
            bf16* const q = p + (int64_t)row * a.grad_pitch + 8 * vec;
            if (row < rows && inside(q, 16, a.grad, a.grad_room, a.err)) *reinterpret_cast<uint4*>(q) = v;
        });
    }
    __device__ __forceinline__ void take(int c, const uint32_t (&v)[32]) {
        if (rows <= 0) return;
        float g[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const float x = __uint_as_float(v[j]) - lse;
            const float e = TERMS != kTerms3 ? fast_ex2(x * kLog2e) : expf(x);
            g[j] = none ? 0.f : both * e;
        }
        if (to >= c && to < c + 32) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (to == c + j) g[j] -= scale;
        }
        if constexpr (TERMS == kTerms1) {
            write(out + c, g);
        } else {
#pragma unroll 1
            for (int k = 0; k < TERMS; ++k) {  // what is left of g, a term at a time
                float x[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    x[j] = first_term(g[j]);
                    g[j] = rest_of(g[j], x[j]);
                }
                write(out + k * a.grad_plane + c, x);
            }
        }
    }
    __device__ __forceinline__ void done(int) {}
};

// A product's rows, of the call's type or as fp32 sums.
template <typename T> struct ProductRow {
    const ProductOut& o;
    unsigned* const err;
    int left, rows;
    float* sums;
    T* out;
    float unit;
    const Turn turn;
    __device__ ProductRow(const VocabArgs& a, const Tile& t, int row0, unsigned char* room)
        : o(a.out[t.job]), err(a.err), turn{room, (int)threadIdx.x & 31} {
        rows = o.rows - row0;
        left = o.cols - t.n0;
        sums = o.sums ? o.sums + ((int64_t)t.split * o.rows + row0) * o.pitch + t.n0 : nullptr;
        out = static_cast<T*>(o.out) + (int64_t)row0 * o.pitch + t.n0;
        unit = o.unit ? *o.unit : 1.f;
    }
    // 64 bytes of each row, E a vector's elements, to memory from column c on
    template <int E> __device__ __forceinline__ void write(int c) const {
        if (o.vec) {  // (a row's columns are whole vectors)
            turn.vectors([&](int row, int vec, uint4 w) {
                T* const q = out + row * o.pitch + c + E * vec;
                if (row < rows && c + E * vec < left && inside(q, 16, o.out, o.room, err))
                    __stcs(reinterpret_cast<uint4*>(q), w);
            });
        } else {
            using Word = std::conditional_t<E == 4, uint32_t, uint16_t>;
            turn.template elements<Word>([&](int row, int e, Word w) {
                T* const q = out + row * o.pitch + c + e;
                if (row < rows && c + e < left && inside(q, sizeof(T), o.out, o.room, err))
                    *reinterpret_cast<Word*>(q) = w;
            });
        }
    }
    __device__ __forceinline__ void take(int c, const uint32_t (&v)[32]) {
        if (c >= left || rows <= 0) return;
        uint32_t w[16];
        if (sums || sizeof(T) == 4) {
#pragma unroll
            for (int half = 0; half < 32; half += 16) {
#pragma unroll
                for (int j = 0; j < 16; ++j) w[j] = v[half + j];
                turn.put(w);
                if (sums) {  // (rows of sums are whole vectors)
                    turn.vectors([&](int row, int vec, uint4 x) {
                        const int col = c + half + 4 * vec;
                        if (row >= rows || col >= left) return;
                        float4 f = make_float4(__uint_as_float(x.x), __uint_as_float(x.y),
                                               __uint_as_float(x.z), __uint_as_float(x.w));
                        float4* const p = reinterpret_cast<float4*>(sums + row * o.pitch + col);
                        if (!inside(p, 16, o.sums, o.room, err)) return;
                        if (o.add) {
                            const float4 b = __ldcg(p);
                            f = make_float4(b.x + f.x, b.y + f.y, b.z + f.z, b.w + f.w);
                        }
                        __stcg(p, f);
                    });
                } else {
                    write<4>(c + half);
                }
            }
        } else {
            float f[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) f[j] = unit * __uint_as_float(v[j]);
            halves(f, w);
            turn.put(w);
            write<8>(c);
        }
    }
    __device__ __forceinline__ void done(int) {}
};

// ---------------------------------------------------------------- the kernel
template <typename OUT, VocabOut KIND, VocabTerms TERMS, int N, int CG>
__global__ void __launch_bounds__(vocab_threads(N), 1)
vocab_tiles(const __grid_constant__ CUtensorMap a0, const __grid_constant__ CUtensorMap b0,
            const __grid_constant__ CUtensorMap a1, const __grid_constant__ CUtensorMap b1,
            const __grid_constant__ VocabArgs a) {
    using S = TileShape<N, CG>;
    constexpr bool PROMOTE = vocab_promotes(KIND, TERMS);
    constexpr int kWarps = vocab_warps(N), kCols = kPartCols;  // a warp's
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) VocabBars bars;
    __shared__ uint32_t tmem_base;
    __shared__ int dead_flag;
    __shared__ uint32_t fills[2];  // of A and B in all
    volatile int* const dead = &dead_flag;
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
    const int rank = CG == 1 ? 0 : (int)cluster_ctarank();
    const int unit = (int)blockIdx.x / CG, units = (int)gridDim.x / CG;
    const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
    const int stage = a.a_room + S::kBytesB, stages = min(kVocabRing / stage, kVocabStages);
    if (threadIdx.x == 0) {
        dead_flag = 0;
        fills[0] = fills[1] = 0;
        for (int s = 0; s < stages; ++s) {
            mbar_init(smem_u32(&bars.full[s]), 2);  // A and B
            mbar_init(smem_u32(&bars.empty[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&bars.acc_full[s]), 1);
            mbar_init(smem_u32(&bars.acc_empty[s]), CG * kWarps);
        }
        mbar_init(smem_u32(&bars.drained), 1);
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    if (warp == kWarps + 1) tmem_alloc<CG>(smem_u32(&tmem_base), S::kTmem);
    tmem_fence_before();
    __syncthreads();
    if constexpr (CG > 1) {  // the other CTA's barriers are there
        cluster_arrive_release();
        cluster_wait_acquire();
    }
    tmem_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
    // steps of k that the accumulators hold at a time
    auto parts_of = [](int kn) { return !PROMOTE ? kn : TERMS == kTerms1 ? kPromote : 1; };
    dependents_may_launch();
    wait_for_launches();
    fence_proxy_async();  // an operand may be an earlier launch's
    Tile t;
    if (warp >= kWarps) {
        if constexpr (PROMOTE) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(vocab_other_regs(N)));
        const uint32_t full0 = smem_u32(&bars.full[0]), empty0 = smem_u32(&bars.empty[0]);
        const uint32_t end = ring + (uint32_t)(stages * stage);
        uint32_t at = ring, bar = 0, phase = 0;  // of the present stage; bar: 8 bytes each
        auto advance = [&]() {
            at += stage;
            bar += 8;
            if (at == end) {
                at = ring;
                bar = 0;
                phase ^= 1u;
            }
        };
        // Warps 0 and 2 of this group fill the stages with A and B, warp 1 multiplies.  A
        // whole warp walks the stages and one elected lane issues: what the copies and
        // products take from uniform registers then stays there.  The warps that fill set
        // the pace of large calls: one thread for both operands in a loop over terms took
        // 3.9 ms where this takes 3.35 (backward 4096 x 4096 x 65536 bf16).
        auto arrived = [&](uint32_t b, uint32_t parity) {
            return (bool)__all_sync(0xffffffffu, hold(b, parity, a.err, dead));
        };
        auto fill = [&](auto which) {
            constexpr bool B = decltype(which)::value;
            constexpr int kBoxes = B ? S::kRowsB / 64 : kTileM / 64;
            const bool leader = elect_one();
            // both CTAs' bytes count on the first one's barriers
            const uint32_t signal0 = CG > 1 ? mapa_shared(full0, 0) : full0;
            const uint32_t offset = B ? a.a_room : 0;
            uint32_t filled = 0;  // fills in all
            bool ok = true;
            for (int i = 0; ok && tile_at<N, CG>(a, unit, units, rank, i, &t); ++i) {
                const TileWork& w = a.work[t.job];
                const CUtensorMap* const map = B ? (t.job ? &b1 : &b0) : (t.job ? &a1 : &a0);
                const Boxes<CG, kBoxes> boxes(map, B ? w.b_mn : w.a_mn, B ? t.n0 + rank * S::kRowsB : t.m0,
                                              B ? w.b_y0 : 0, t.k0);
                const uint32_t bytes = CG * (B ? S::kBytesB : w.a_bytes);
                auto one = [&](int k, int term) {
                    ok = arrived(empty0 + bar, phase ^ 1u);
                    if (!ok) return false;
                    if (leader) {
                        if (rank == 0) mbar_arrive_expect_tx(full0 + bar, bytes);
                        boxes.load(k, term, at + offset, signal0 + bar);
                        if (TERMS == kTerms2 && !B && w.both) boxes.load(k, 1, at + kBytesA, signal0 + bar);
                    }
                    ++filled;
                    advance();
                    return true;
                };
                for (int k = 0; k < t.kn; ++k)
                    if (!(TERMS != kTerms3 ? one(k, 0) : one(k, 2) && one(k, 1) && one(k, 0))) break;
            }
            // The products signal the last stages too: no CTA leaves before it has seen that
            // (of a pair the signals come from the first CTA).
            if (!B)
                for (uint32_t f = filled > (uint32_t)stages ? filled - stages : 0; ok && f < filled; ++f)
                    ok = arrived(empty0 + 8 * (f % stages), (f / stages) & 1u);
            if (leader) fills[B] = filled;
        };
        if (warp == kWarps) {
            fill(std::false_type());
        } else if (warp == kWarps + 2 && !a.alone) {
            fill(std::true_type());
        } else if (warp == kWarps + 1 && rank == 0) {
            const bool leader = elect_one();
            int n = 0;  // parts so far
            bool ok = true;
            auto there = [&](uint32_t b, uint32_t parity) {
                ok = arrived(b, parity);
                tmem_fence_after();
                return ok;
            };
            for (int i = 0; ok && tile_at<N, CG>(a, unit, units, rank, i, &t); ++i) {
                const TileWork& w = a.work[t.job];
                const uint32_t desc = mma_desc(CG * kTileM, N, w.a_mn, w.b_mn);
                // from one sixteen k to the next, in descriptors' units of 16 bytes
                const uint32_t step_a = w.a_mn ? 16 * 8 : 2, step_b = w.b_mn ? 16 * 8 : 2;
                const int steps = parts_of(t.kn);
                for (int k0 = 0; ok && k0 < t.kn; ++n) {
                    const int k1 = PROMOTE ? min(t.kn, k0 + steps) : t.kn;
                    const uint32_t acc = tmem + (n & 1) * N;
                    if (!there(smem_u32(&bars.acc_empty[n & 1]), ((n >> 1) & 1) ^ 1u)) break;
                    // the products of A in stage `sa` with B in stage `sb`
                    auto multiply = [&](uint32_t sa, uint32_t sb, bool add) {
                        const uint64_t da = smem_desc(sa, kBoxBytes, 1024);
                        const uint64_t db = smem_desc(sb + a.a_room, kBoxBytes, 1024);
                        if (leader)
#pragma unroll
                            for (int q = 0; q < kTileK / 16; ++q)
                                mma_bf16<CG>(acc, da + q * step_a, db + q * step_b, desc, add || q > 0);
                    };
                    for (int k = k0; k < k1; ++k) {
                        if constexpr (TERMS != kTerms3) {
                            if (!there(full0 + bar, phase)) break;
                            const bool both = TERMS == kTerms2 && w.both;
                            if (both) multiply(at + kBytesA, at, k > k0);
                            multiply(at, at, k > k0 || both);
                            if (leader) mma_commit<CG>(empty0 + bar);
                            advance();
                        } else {
                            const uint32_t at2 = at, bar2 = bar;
                            if (!there(full0 + bar, phase)) break;
                            advance();
                            const uint32_t at1 = at, bar1 = bar;
                            if (!there(full0 + bar, phase)) break;
                            multiply(at1, at1, k > k0);
                            advance();
                            if (!there(full0 + bar, phase)) break;
                            multiply(at2, at, true);
                            multiply(at, at2, true);
                            if (leader) mma_commit<CG>(empty0 + bar2);
                            multiply(at1, at, true);
                            multiply(at, at1, true);
                            if (leader) mma_commit<CG>(empty0 + bar1);
                            multiply(at, at, true);
                            if (leader) mma_commit<CG>(empty0 + bar);
                            advance();
                        }
                    }
                    if (ok && leader) mma_commit<CG>(smem_u32(&bars.acc_full[n & 1]));
                    k0 = k1;
                }
            }
        }
    } else {
        if constexpr (PROMOTE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(vocab_regs(N)));
        const int quarter = warp & 3, block = warp >> 2;  // of rows, of columns
        unsigned char* const room = raw + (ring - smem_u32(raw)) + kVocabRing + warp * kTurnBytes;
        int n = 0;
        bool ok = true;
        // the accumulators of part n, once they are there
        auto ready = [&]() {
            ok = __all_sync(0xffffffffu, hold(smem_u32(&bars.acc_full[n & 1]), (n >> 1) & 1, a.err, dead));
            tmem_fence_after();
            return tmem + (n & 1) * N + block * kCols + ((uint32_t)(32 * quarter) << 16);
        };
        auto release = [&]() {
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) {
                const uint32_t bar = smem_u32(&bars.acc_empty[n & 1]);
                if constexpr (CG > 1) mbar_arrive_cluster(mapa_shared(bar, 0));
                else mbar_arrive(bar);
            }
            ++n;
        };
        for (int i = 0; ok && tile_at<N, CG>(a, unit, units, rank, i, &t); ++i) {
            OUT out(a, t, t.m0 + 32 * quarter, room);
            if constexpr (PROMOTE) {
                constexpr int kLoad = kWarps == 8 ? 32 : 16;  // as registers allow
                F2 sum[kCols / 2];
#pragma unroll
                for (int j = 0; j < kCols / 2; ++j) sum[j] = f2(0.f);
                const int steps = parts_of(t.kn);
                for (int k0 = 0; k0 < t.kn; k0 += steps) {
                    const uint32_t acc = ready();
                    if (!ok) break;
#pragma unroll
                    for (int c = 0; c < kCols; c += kLoad) {
                        uint32_t v[kLoad];
                        tmem_load(acc + c, v);
                        tmem_load_wait();
#pragma unroll
                        for (int j = 0; j < kLoad; j += 2) {
                            const F2 x{__uint_as_float(v[j]), __uint_as_float(v[j + 1])};
                            sum[(c + j) / 2] = add2(sum[(c + j) / 2], x);
                        }
                    }
                    release();
                }
                if (!ok) break;
#pragma unroll
                for (int c = 0; c < kCols; c += 32) {
                    uint32_t v[32];
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        v[j] = __float_as_uint(sum[(c + j) / 2].x);
                        v[j + 1] = __float_as_uint(sum[(c + j) / 2].y);
                    }
                    out.take(block * kCols + c, v);
                }
            } else {
                const uint32_t acc = ready();
                if (!ok) break;
                for (int c = 0; c < kCols; c += 32) {
                    uint32_t v[32];
                    tmem_load(acc + c, v);
                    tmem_load_wait();
                    out.take(block * kCols + c, v);
                }
                release();
            }
            out.done(t.n0 / kCols + block);
        }
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    if constexpr (CG > 1) {  // no CTA leaves while the other may signal it
        if (threadIdx.x == 0 && *dead) st_cluster_u32(mapa_shared(smem_u32(&dead_flag), rank ^ 1), 1u);
        cluster_arrive_release();
        cluster_wait_acquire();
    }
    tmem_fence_after();
    if (*dead) {  // A wait has given up: nothing is issued any more, and nothing is left in flight.
        const bool leader = elect_one();     // (the same lane as before)
        if (warp == kWarps + 1 && leader) {  // products
            if (rank == 0) mma_commit<CG>(smem_u32(&bars.drained));
            mbar_wait_bounded(smem_u32(&bars.drained), 0, a.err);
        }
        if (warp == kWarps && leader && rank == 0) {  // copies: both CTAs' count on the first one's stages
            const uint32_t full0 = smem_u32(&bars.full[0]), most = max(fills[0], fills[1]);
            const uint32_t least = most > (uint32_t)stages ? most - stages : 0;
            bool ok = true;
            for (uint32_t f = least; f < most; ++f)  // (the other operand of a stage does not come)
                if (f >= min(fills[0], fills[1])) mbar_arrive(full0 + 8 * (f % stages));
            for (uint32_t f = least; ok && f < most; ++f)
                ok = mbar_wait_bounded(full0 + 8 * (f % stages), (f / stages) & 1u, a.err);
            if constexpr (CG > 1) {
                // A CTA that filled other stages than the first: their bytes complete no
                // phase, and one time limit is what its copies are given.
                const uint32_t there = mapa_shared(smem_u32(&fills[0]), 1);
                if (ld_cluster_u32(there) != fills[0] || ld_cluster_u32(there + 4) != fills[1]) {
                    const uint64_t t0 = globaltimer_ns();
                    while (globaltimer_ns() - t0 < kWaitLimitNs) __nanosleep(1000);
                }
            }
        }
        __syncthreads();
        if constexpr (CG > 1) {
            cluster_arrive_release();
            cluster_wait_acquire();
        }
    }
    if (warp == kWarps + 1) tmem_free<CG>(tmem, S::kTmem);
}

template <typename OUT, VocabOut KIND, VocabTerms TERMS> const void* vocab_kernel_of(VocabTile t) {
    switch (t) {
        case kPair256: return (const void*)vocab_tiles<OUT, KIND, TERMS, 256, 2>;
        case kOne256: return (const void*)vocab_tiles<OUT, KIND, TERMS, 256, 1>;
        default: return (const void*)vocab_tiles<OUT, KIND, TERMS, 128, 1>;
    }
}

}  // namespace credit
