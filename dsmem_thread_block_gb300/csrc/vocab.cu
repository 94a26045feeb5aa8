// vocab.cu -- softmax cross entropy of a linear head, the logits never stored:
//   z = h w^T,  lse_t = log sum_v exp(z_tv),  loss_t = lse_t - z_t,target
//   g_tv = (dloss_t + dlse_t) exp(z_tv - lse_t) - dloss_t [v = target_t]
//   dh = g w,  dw = g^T h
#include <algorithm>
#include <type_traits>

#include "planner.h"
#include "rowops.cuh"
#include "tensor.cuh"
#include "vocab.h"

namespace credit {

namespace {

constexpr int kStages = 4;
constexpr int kBytesA = kTileM * kTileK * 2, kBytesB = kTileN * kTileK * 2;
constexpr int kStageBytes = kBytesA + kBytesB;
constexpr int kBoxBytes = 64 * kTileK * 2;      // one box of an operand with M or N innermost
constexpr int kEpilogueWarps = 4;
constexpr int kThreads = 32 * (kEpilogueWarps + 2);
constexpr int kSmem = kStages * kStageBytes + 1024;  // aligned to 1024 by hand
constexpr uint32_t kTmemColumns = 2 * kTileN;   // two accumulators
constexpr float kLog2e = 1.4426950408889634f;

struct Bars {
    uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drained;
};

// Wait for a phase; false once a wait of this CTA has given up.
__device__ __forceinline__ bool hold(uint64_t& bar, uint32_t parity, unsigned* err,
                                     volatile int* dead) {
    const uint32_t b = smem_u32(&bar);
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(b, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(b, parity)) {
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
__device__ __forceinline__ Tile tile_at(const VocabArgs& a, int t) {
    Tile r;
    r.job = 0;
    if (a.jobs > 1 && t >= tiles_of(a.work[0])) {
        t -= tiles_of(a.work[0]);
        r.job = 1;
    }
    const TileWork& w = a.work[r.job];
    const int per = w.mt * w.nt;
    r.split = t / per;
    t -= r.split * per;
    const int g = t / (w.group * w.nt);         // whole groups of tile rows
    t -= g * w.group * w.nt;
    const int rows = min(w.group, w.mt - g * w.group);
    const int n = t / rows;
    r.m0 = (g * w.group + t - n * rows) * kTileM;
    r.n0 = n * kTileN;
    r.k0 = r.split * w.per;
    r.kn = min(w.per, w.kb - r.k0);
    return r;
}

// Terms of A and B in the order of their products, the smallest first: with
// x = x0 + x1 + x2 to 24 bits, x0 y0 + (x0 y1 + x1 y0) + (x1 y1 + x0 y2 + x2 y0)
// leaves out what is below 2^-24 of x y.
__device__ __forceinline__ int term_a(int pairs, int p) { return pairs == 1 ? 0 : (0x001102 >> (4 * p)) & 3; }
__device__ __forceinline__ int term_b(int pairs, int p) { return pairs == 1 ? 0 : (0x010120 >> (4 * p)) & 3; }

__device__ __forceinline__ void load_operand(const CUtensorMap* map, bool mn, int boxes, int at,
                                             int y0, int k, int term, uint32_t dst, uint32_t bar) {
    if (!mn) {
        tma_load_3d(dst, map, k * kTileK, at + y0, term, bar);
        return;
    }
    for (int j = 0; j < boxes; ++j)
        tma_load_3d(dst + j * kBoxBytes, map, at + 64 * j, k * kTileK + y0, term, bar);
}

// The bf16 terms of a value.
__device__ __forceinline__ void split_terms(float x, float (&t)[3]) {
    float hi = __bfloat162float(__float2bfloat16_rn(x));
    const bool finite = fabsf(x) <= 3.402823466e38f;
    if (finite && isinf(hi)) hi = __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
    const float r = finite ? x - hi : 0.f;
    const float mid = __bfloat162float(__float2bfloat16_rn(r));
    t[0] = hi;
    t[1] = mid;
    t[2] = r - mid;
}

__device__ __forceinline__ uint32_t pair_of(float lo, float hi) {
    return Pairs<bf16>::two(F2{lo, hi});
}

// ------------------------------------------------------------ the epilogues
// One token's maximum and sum of exponentials over a tile.
__device__ __forceinline__ void stats_tile(const VocabArgs& a, const Tile& t, uint32_t acc, int row) {
    const bool live = row < a.rows;
    const int64_t target = live ? a.target[row] : -1;
    const int64_t to = target - a.v0 - t.n0;       // column of the target in this tile
    const int left = a.cols - t.n0;
    float m = -INFINITY, s = 0.f;
    for (int c = 0; c < kTileN; c += 32) {
        if (c >= left) break;
        uint32_t v[32];
        tmem_load(acc + c, v);
        tmem_load_wait();
        if (c + 32 > left) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (c + j >= left) v[j] = __float_as_uint(-INFINITY);
        }
        float top = __uint_as_float(v[0]);
#pragma unroll
        for (int j = 1; j < 32; ++j) top = fmaxf(top, __uint_as_float(v[j]));
        top = fmaxf(top, m);
        // nothing is above an infinite maximum: exponents are then taken from zero
        const float base = isinf(top) ? 0.f : top;
        if (top != m) {
            s = s == 0.f ? 0.f : s * fast_ex2((m - base) * kLog2e);
            m = top;
        }
        const float off = -base * kLog2e;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            s0 += fast_ex2(fmaf(__uint_as_float(v[j]), kLog2e, off));
            s1 += fast_ex2(fmaf(__uint_as_float(v[j + 1]), kLog2e, off));
        }
        s += s0 + s1;
        if (to >= c && to < c + 32) {
            float z = 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (to == c + j) z = __uint_as_float(v[j]);
            if (live) a.picked[row] = z;
        }
    }
    if (live) a.parts[(int64_t)(t.n0 / kTileN) * a.rows + row] = make_float2(m, s);
}

// The gradient of a token's logits over a tile, as bf16 terms.
template <typename T>
__device__ __forceinline__ void grad_tile(const VocabArgs& a, const Tile& t, uint32_t acc, int row) {
    const bool live = row < a.rows;
    float scale = 0.f, both = 0.f, lse = 0.f;
    int64_t to = -1;
    if (live) {
        const int64_t target = a.target[row];
        scale = target == a.ignore ? 0.f : target < 0 || target >= a.vocab ? NAN : a.dloss[row];
        both = scale + (a.dlse ? a.dlse[row] : 0.f);
        lse = a.lse[row];
        to = target - a.v0 - t.n0;
        if (target == a.ignore) to = -1;
    }
    const bool none = both == 0.f;  // (its exponentials may be infinite)
    bf16* const out = static_cast<bf16*>(a.grad) + (int64_t)row * a.grad_pitch + t.n0;
    for (int c = 0; c < kTileN; c += 32) {
        uint32_t v[32];
        tmem_load(acc + c, v);
        tmem_load_wait();
        float g[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const float x = __uint_as_float(v[j]) - lse;
            const float e = sizeof(T) == 2 ? fast_ex2(x * kLog2e) : expf(x);
            g[j] = none ? 0.f : both * e;
        }
        if (to >= c && to < c + 32) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (to == c + j) g[j] -= scale;
        }
        if (!live) continue;
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int j = 0; j < 32; j += 8)
                *reinterpret_cast<uint4*>(out + c + j) =
                    make_uint4(pair_of(g[j], g[j + 1]), pair_of(g[j + 2], g[j + 3]),
                               pair_of(g[j + 4], g[j + 5]), pair_of(g[j + 6], g[j + 7]));
        } else {
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
                float p[8][3];
#pragma unroll
                for (int i = 0; i < 8; ++i) split_terms(g[j + i], p[i]);
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    *reinterpret_cast<uint4*>(out + k * a.grad_plane + c + j) =
                        make_uint4(pair_of(p[0][k], p[1][k]), pair_of(p[2][k], p[3][k]),
                                   pair_of(p[4][k], p[5][k]), pair_of(p[6][k], p[7][k]));
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ void product_tile(const ProductOut& o, const Tile& t, uint32_t acc,
                                             int row) {
    const bool live = row < o.rows;
    float* const sums = o.sums ? o.sums + ((int64_t)t.split * o.rows + row) * o.pitch + t.n0 : nullptr;
    T* const out = static_cast<T*>(o.out) + (int64_t)row * o.pitch + t.n0;
    const int left = o.cols - t.n0;
    for (int c = 0; c < kTileN; c += 32) {
        if (c >= left) break;
        uint32_t v[32];
        tmem_load(acc + c, v);
        tmem_load_wait();
        if (!live) continue;
        if (sums) {  // (rows of sums are whole vectors)
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                if (c + j >= left) break;
                float4 f = make_float4(__uint_as_float(v[j]), __uint_as_float(v[j + 1]),
                                       __uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
                float4* const p = reinterpret_cast<float4*>(sums + c + j);
                if (o.add) {
                    const float4 b = __ldcg(p);
                    f = make_float4(b.x + f.x, b.y + f.y, b.z + f.z, b.w + f.w);
                }
                __stcg(p, f);
            }
            continue;
        }
        constexpr int kVec = 16 / sizeof(T);
#pragma unroll
        for (int j = 0; j < 32; j += kVec) {
            if (o.vec && c + j + kVec <= left) {
                uint4 w;
                if constexpr (sizeof(T) == 4) {
                    w = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                } else {
                    auto two = [&](int k) {
                        return pair_of(__uint_as_float(v[j + k]), __uint_as_float(v[j + k + 1]));
                    };
                    w = make_uint4(two(0), two(2), two(4), two(6));
                }
                *reinterpret_cast<uint4*>(out + c + j) = w;
            } else {
#pragma unroll
                for (int k = 0; k < kVec; ++k)
                    if (c + j + k < left) {
                        if constexpr (sizeof(T) == 4) out[c + j + k] = __uint_as_float(v[j + k]);
                        else out[c + j + k] = __float2bfloat16_rn(__uint_as_float(v[j + k]));
                    }
            }
        }
    }
}

// ---------------------------------------------------------------- the kernel
// One CTA per SM walks tiles of 128 x 256: a warp fills a ring of stages by
// tensor-map copies, a thread issues the products into one of two
// accumulators, and four warps read the other one out.
template <int OUT, typename T>
__global__ void __launch_bounds__(kThreads, 1)
vocab_tiles(const __grid_constant__ CUtensorMap a0, const __grid_constant__ CUtensorMap b0,
            const __grid_constant__ CUtensorMap a1, const __grid_constant__ CUtensorMap b1,
            const __grid_constant__ VocabArgs a) {
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) Bars bars;
    __shared__ uint32_t tmem_base;
    __shared__ int dead_flag;
    volatile int* const dead = &dead_flag;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
    if (threadIdx.x == 0) {
        dead_flag = 0;
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&bars.full[s]), 1);
            mbar_init(smem_u32(&bars.empty[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&bars.acc_full[s]), 1);
            mbar_init(smem_u32(&bars.acc_empty[s]), 32 * kEpilogueWarps);
        }
        mbar_init(smem_u32(&bars.drained), 1);
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    if (warp == kEpilogueWarps + 1) tmem_alloc(smem_u32(&tmem_base), kTmemColumns);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_base;
    const int total = tiles_of(a.work[0]) + (a.jobs > 1 ? tiles_of(a.work[1]) : 0);

    if (warp == kEpilogueWarps) {
        if (lane == 0) {
            int s = 0;
            uint32_t phase = 0, filled = 0;  // fills in all
            bool ok = true;
            for (int i = blockIdx.x; ok && i < total; i += gridDim.x) {
                const Tile t = tile_at(a, i);
                const TileWork& w = a.work[t.job];
                const CUtensorMap* const ma = t.job ? &a1 : &a0;
                const CUtensorMap* const mb = t.job ? &b1 : &b0;
                for (int p = 0; ok && p < a.pairs; ++p)
                    for (int k = 0; k < t.kn; ++k) {
                        ok = hold(bars.empty[s], phase ^ 1u, a.err, dead);
                        if (!ok) break;
                        const uint32_t bar = smem_u32(&bars.full[s]), at = ring + s * kStageBytes;
                        mbar_arrive_expect_tx(bar, kStageBytes);
                        load_operand(ma, w.a_mn, kTileM / 64, t.m0, 0, t.k0 + k, term_a(a.pairs, p), at,
                                     bar);
                        load_operand(mb, w.b_mn, kTileN / 64, t.n0, w.b_y0, t.k0 + k,
                                     term_b(a.pairs, p), at + kBytesA, bar);
                        ++filled;
                        if (++s == kStages) {
                            s = 0;
                            phase ^= 1u;
                        }
                    }
            }
            // a CTA that has given up leaves no copy in flight
            if (!ok)
                for (uint32_t f = filled > kStages ? filled - kStages : 0; f < filled; ++f)
                    mbar_wait_bounded(smem_u32(&bars.full[f % kStages]), (f / kStages) & 1u, a.err);
        }
    } else if (warp == kEpilogueWarps + 1) {
        if (lane == 0) {
            int s = 0, n = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int i = blockIdx.x; ok && i < total; i += gridDim.x, ++n) {
                const Tile t = tile_at(a, i);
                const TileWork& w = a.work[t.job];
                const uint32_t desc = mma_desc(kTileM, kTileN, w.a_mn, w.b_mn);
                // bytes from one sixteen k to the next
                const uint32_t step_a = w.a_mn ? 16 * 128 : 32, step_b = w.b_mn ? 16 * 128 : 32;
                const uint32_t acc = tmem + (n & 1) * kTileN;
                ok = hold(bars.acc_empty[n & 1], ((n >> 1) & 1) ^ 1u, a.err, dead);
                if (!ok) break;
                tmem_fence_after();
                const int steps = t.kn * a.pairs;
                for (int k = 0; k < steps; ++k) {
                    ok = hold(bars.full[s], phase, a.err, dead);
                    if (!ok) break;
                    tmem_fence_after();
                    const uint32_t at = ring + s * kStageBytes;
                    const uint64_t da = smem_desc(at, kBoxBytes, 1024);
                    const uint64_t db = smem_desc(at + kBytesA, kBoxBytes, 1024);
#pragma unroll
                    for (int q = 0; q < kTileK / 16; ++q)
                        mma_bf16(acc, da + (q * step_a >> 4), db + (q * step_b >> 4), desc, k > 0 || q > 0);
                    mma_commit(smem_u32(&bars.empty[s]));
                    if (++s == kStages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
                if (ok) mma_commit(smem_u32(&bars.acc_full[n & 1]));
            }
            if (!ok) {  // nor a product
                mma_commit(smem_u32(&bars.drained));
                mbar_wait_bounded(smem_u32(&bars.drained), 0, a.err);
            }
        }
    } else {
        int n = 0;
        for (int i = blockIdx.x; i < total; i += gridDim.x, ++n) {
            const Tile t = tile_at(a, i);
            if (!__all_sync(0xffffffffu, hold(bars.acc_full[n & 1], (n >> 1) & 1, a.err, dead))) break;
            tmem_fence_after();
            const uint32_t acc = tmem + (n & 1) * kTileN + ((uint32_t)(32 * warp) << 16);
            const int row = t.m0 + 32 * warp + lane;
            if constexpr (OUT == kVocabStats) stats_tile(a, t, acc, row);
            else if constexpr (OUT == kVocabGrad) grad_tile<T>(a, t, acc, row);
            else product_tile<T>(a.out[t.job], t, acc, row);
            tmem_fence_before();
            mbar_arrive(smem_u32(&bars.acc_empty[n & 1]));
        }
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == kEpilogueWarps + 1) tmem_free(tmem, kTmemColumns);
}

// --------------------------------------------------------- the small kernels
constexpr int kMergeWarps = 32;

// Warp w merges the parts of every 32nd tile from w on for 32 tokens, a token a
// lane; the first warp merges the warps'.
__device__ __forceinline__ void merge(float& m, float& s, float mo, float so) {
    const float top = fmaxf(m, mo), base = isinf(top) ? 0.f : top;
    s = (s == 0.f ? 0.f : s * expf(m - base)) + (so == 0.f ? 0.f : so * expf(mo - base));
    m = top;
}
__global__ void __launch_bounds__(32 * kMergeWarps)
vocab_merge(VocabArgs a, int tiles, float* loss, float* lse) {
    __shared__ float2 parts[kMergeWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)blockIdx.x * 32 + lane;
    float m = -INFINITY, s = 0.f;
    if (row < a.rows)
        for (int t = warp; t < tiles; t += kMergeWarps) {
            const float2 p = a.parts[(int64_t)t * a.rows + row];
            merge(m, s, p.x, p.y);
        }
    parts[warp][lane] = make_float2(m, s);
    __syncthreads();
    if (warp || row >= a.rows) return;
    for (int w = 1; w < kMergeWarps; ++w) merge(m, s, parts[w][lane].x, parts[w][lane].y);
    const float l = (isinf(m) ? 0.f : m) + logf(s);
    const int64_t target = a.target[row];
    lse[row] = l;
    loss[row] = target == a.ignore ? 0.f
                : target < 0 || target >= a.vocab ? NAN : l - a.picked[row];
}

// Rows as bf16 terms, two columns a thread (rows of dst are whole 16-byte lines).
template <typename T>
__global__ void __launch_bounds__(256)
vocab_pack(const T* src, int64_t rows, int64_t cols, bf16* dst, int64_t pitch, int64_t plane) {
    const int64_t half = (cols + 1) / 2, n = rows * half;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / half, c = 2 * (i - r * half);
        const T* const p = src + r * cols + c;
        bf16* const q = dst + r * pitch + c;
        const bool two = c + 1 < cols;
        if constexpr (sizeof(T) == 2) {
            const uint16_t* w = reinterpret_cast<const uint16_t*>(p);
            *reinterpret_cast<uint32_t*>(q) = (uint32_t)w[0] | (two ? (uint32_t)w[1] << 16 : 0u);
        } else {
            float x[3], y[3] = {0.f, 0.f, 0.f};
            split_terms(p[0], x);
            if (two) split_terms(p[1], y);
#pragma unroll
            for (int k = 0; k < 3; ++k)
                *reinterpret_cast<uint32_t*>(q + k * plane) = pair_of(x[k], y[k]);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256)
vocab_sum(const float* sums, int splits, int64_t rows, int64_t cols, int64_t pitch, T* out) {
    const int64_t n = rows * cols;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / cols, c = i - r * cols;
        float v = 0.f;
        for (int s = 0; s < splits; ++s) v += sums[((int64_t)s * rows + r) * pitch + c];
        if constexpr (sizeof(T) == 4) out[i] = v;
        else out[i] = __float2bfloat16_rn(v);
    }
}

template <typename T> int blocks_for(int64_t n, int sms) {
    return (int)std::max<int64_t>(1, std::min<int64_t>((n + 255) / 256, (int64_t)sms * 8));
}

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                            const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                            CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                            CUtensorMapFloatOOBfill);

// The driver's encoder, found once through the runtime.
Encode encoder() {
    static const Encode fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<Encode>(p);
    }();
    return fn;
}

}  // namespace

bool term_map(const TermMatrix& m, int box_rows, CUtensorMap* map) {
    const Encode encode = encoder();
    if (!encode) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)m.cols, (cuuint64_t)m.rows, (cuuint64_t)m.terms};
    const cuuint64_t strides[2] = {(cuuint64_t)m.pitch, (cuuint64_t)m.plane};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1}, ones[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(m.p), dims, strides, box,
                  ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {
const void* kernel_of(VocabOut out, int dtype) {
    if (out == kVocabStats) return (const void*)vocab_tiles<kVocabStats, bf16>;
    if (out == kVocabGrad)
        return dtype ? (const void*)vocab_tiles<kVocabGrad, bf16> : (const void*)vocab_tiles<kVocabGrad, float>;
    return dtype ? (const void*)vocab_tiles<kVocabProduct, bf16>
                 : (const void*)vocab_tiles<kVocabProduct, float>;
}
}  // namespace

cudaError_t launch_vocab(VocabOut out, int dtype, const CUtensorMap (&maps)[4], const VocabArgs& a,
                         int sms, cudaStream_t s) {
    const void* fn = kernel_of(out, dtype);
    int dev;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!kernel_info(dev, fn, false)) return cudaErrorInvalidDeviceFunction;  // its shared memory is opted in
    int64_t total = 0;
    for (int j = 0; j < a.jobs; ++j)
        total += (int64_t)a.work[j].mt * a.work[j].nt * a.work[j].splits;
    if (total > INT32_MAX - sms) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(total, sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    void* args[] = {const_cast<CUtensorMap*>(&maps[0]), const_cast<CUtensorMap*>(&maps[1]),
                    const_cast<CUtensorMap*>(&maps[2]), const_cast<CUtensorMap*>(&maps[3]),
                    const_cast<VocabArgs*>(&a)};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

cudaError_t launch_vocab_merge(const VocabArgs& a, int tiles, float* loss, float* lse,
                               cudaStream_t s) {
    vocab_merge<<<(unsigned)((a.rows + 31) / 32), 32 * kMergeWarps, 0, s>>>(a, tiles, loss, lse);
    return cudaGetLastError();
}

cudaError_t launch_vocab_pack(int dtype, const void* src, int64_t rows, int64_t cols, void* dst,
                              int64_t pitch, int64_t plane, int sms, cudaStream_t s) {
    const int blocks = blocks_for<float>(rows * ((cols + 1) / 2), sms);
    if (dtype == 0)
        vocab_pack<float><<<blocks, 256, 0, s>>>(static_cast<const float*>(src), rows, cols,
                                                 static_cast<bf16*>(dst), pitch, plane);
    else
        vocab_pack<bf16><<<blocks, 256, 0, s>>>(static_cast<const bf16*>(src), rows, cols,
                                                static_cast<bf16*>(dst), pitch, plane);
    return cudaGetLastError();
}

cudaError_t launch_vocab_sum(int dtype, const float* sums, int splits, int64_t rows, int64_t cols,
                             int64_t pitch, void* out, int sms, cudaStream_t s) {
    const int blocks = blocks_for<float>(rows * cols, sms);
    if (dtype == 0)
        vocab_sum<float><<<blocks, 256, 0, s>>>(sums, splits, rows, cols, pitch, static_cast<float*>(out));
    else
        vocab_sum<bf16><<<blocks, 256, 0, s>>>(sums, splits, rows, cols, pitch, static_cast<bf16*>(out));
    return cudaGetLastError();
}

}  // namespace credit
