// vocab.cu -- softmax cross entropy of a linear head, the logits never stored:
//   z = h w^T,  lse_t = log sum_v exp(z_tv),  loss_t = lse_t - z_t,target
//   g_tv = (dloss_t + dlse_t) exp(z_tv - lse_t) - dloss_t [v = target_t]
//   dh = g w,  dw = g^T h
//
// The products are vocab_tiles.cuh's, those of a few tokens vocab_few.cu's; here are
// what comes before and after them, and the launches.
//   vocab_pack   operands that tensor maps cannot take (rows that are no whole 16-byte
//                lines, fp32) as bf16 terms; bound by HBM: 16384 x 2048 fp32 54 us
//   vocab_merge  the tiles' statistics of a token: alone, 4096 tokens of 256 parts 11 us, of
//                2048 34
//   vocab_rows   from logits that were summed in parts of k, where they have few tiles,
//                the statistics or the gradient
//   vocab_sum    parts of dhidden, or of dweight, in order: 4096 x 4096 20 us
//   vocab_unit   what a logits' gradient of one bf16 term is divided by: some 2 us of a call,
//                4096 tokens alone 3.6 to 4.9
// All kernels of a call are launched early (early_launch.h), which saves some 3 us of
// a small call (32 x 1024 x 4096 forward 13.4 us called without, 9.6 with).
#include "early_launch.h"
#include "vocab_tiles.cuh"

namespace credit {

namespace {

// --------------------------------------------------------- the small kernels
constexpr int kMergeRows = 4;   // of a CTA: a sector of each part

// (m, s) and another pair: the larger maximum, the sums scaled to it.
__device__ __forceinline__ void merge_pair(float& m, float& s, float mo, float so) {
    const float top = fmaxf(m, mo), base = isinf(top) ? 0.f : top;
    s = (s == 0.f ? 0.f : s * expf(m - base)) + (so == 0.f ? 0.f : so * expf(mo - base));
    m = top;
}

// The parts of four tokens: THREADS / 4 threads a token, each every THREADS / 4th
// part, 1024 threads from 512 parts on.  (A token a lane, 16 warps over the parts,
// took 17 us for 64 tokens of 1024 parts.)
template <int THREADS>
__global__ void __launch_bounds__(THREADS) vocab_merge(VocabArgs a, int nparts, float* loss, float* lse) {
    constexpr int kGroups = THREADS / kMergeRows;
    __shared__ float2 sums[THREADS / 32][kMergeRows];
    dependents_may_launch();
    wait_for_launches();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int mine = threadIdx.x % kMergeRows, group = threadIdx.x / kMergeRows;
    const int64_t row = (int64_t)blockIdx.x * kMergeRows + mine;
    const bool live = row < a.rows;
    float m = -INFINITY, s = 0.f;
    if (live)
        for (int t0 = group; t0 < nparts; t0 += 4 * kGroups) {
            float2 p[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int t = t0 + u * kGroups;
                const float2* const q = &a.parts[(int64_t)t * a.rows + row];
                p[u] = t < nparts && inside(q, sizeof(*q), a.parts, a.parts_room, a.err)
                           ? __ldcg(q) : make_float2(-INFINITY, 0.f);
            }
            float top = m;
#pragma unroll
            for (int u = 0; u < 4; ++u) top = fmaxf(top, p[u].x);
            const float base = isinf(top) ? 0.f : top;
            s = s == 0.f ? 0.f : s * expf(m - base);
#pragma unroll
            for (int u = 0; u < 4; ++u) s += p[u].y == 0.f ? 0.f : p[u].y * expf(p[u].x - base);
            m = top;
        }
#pragma unroll
    for (int o = kMergeRows; o < 32; o <<= 1) {
        const float mo = __shfl_xor_sync(0xffffffffu, m, o), so = __shfl_xor_sync(0xffffffffu, s, o);
        merge_pair(m, s, mo, so);
    }
    if (lane < kMergeRows) sums[warp][lane] = make_float2(m, s);
    __syncthreads();
    if (threadIdx.x >= kMergeRows || !live) return;
    for (int w = 1; w < THREADS / 32; ++w) merge_pair(m, s, sums[w][mine].x, sums[w][mine].y);
    const float l = (isinf(m) ? 0.f : m) + logf(s);
    const int64_t target = a.target[row];
    lse[row] = l;
    loss[row] = target == a.ignore ? 0.f
                : target < 0 || target >= a.vocab ? NAN : l - a.picked[row];
}

// A CTA a token, four columns a thread at a time.
constexpr int kRowThreads = 256;
template <int TERMS>   // 0: the statistics
__global__ void __launch_bounds__(kRowThreads)
vocab_rows(VocabArgs a, const float* sums, int splits, int64_t pitch, float* loss, float* lse) {
    __shared__ float2 parts[kRowThreads / 32];
    __shared__ float picked;
    dependents_may_launch();
    wait_for_launches();
    const int64_t row = blockIdx.x, plane = a.rows * pitch;
    const float* const first = sums + row * pitch;
    const int64_t target = a.target[row];
    const bool ignored = target == a.ignore, outside = target < 0 || target >= a.vocab;
    float scale = 0.f, both = 0.f, known = 0.f;
    if (TERMS > 0) {
        scale = ignored ? 0.f : outside ? NAN : a.dloss[row];
        both = scale + (a.dlse ? a.dlse[row] : 0.f);
        known = a.lse[row];
        if (TERMS == 1) {
            const float unit = *a.unit;
            scale /= unit;
            both /= unit;
        }
    }
    float m = -INFINITY, s = 0.f;
    for (int c = 4 * (int)threadIdx.x; c < a.cols; c += 4 * kRowThreads) {
        const float* p = first + c;
        if (!inside(p + (splits - 1) * plane, 16, sums, a.out[0].room, a.err)) continue;
        float4 f = __ldcg(reinterpret_cast<const float4*>(p));
#pragma unroll 8
        for (int k = 1; k < splits; ++k) {
            p += plane;
            const float4 g = __ldcg(reinterpret_cast<const float4*>(p));
            f = make_float4(f.x + g.x, f.y + g.y, f.z + g.z, f.w + g.w);
        }
        const float z[4] = {f.x, f.y, f.z, f.w};
        if constexpr (TERMS == 0) {
            float top = m;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < a.cols) top = fmaxf(top, z[j]);
            const float base = isinf(top) ? 0.f : top;
            s = s == 0.f ? 0.f : s * expf(m - base);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < a.cols) {
                    s += expf(z[j] - base);
                    if (target == c + j) picked = z[j];
                }
            m = top;
        } else {
            float g[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                g[j] = both == 0.f ? 0.f : both * expf(z[j] - known);
                if (target == a.v0 + c + j && !ignored) g[j] -= scale;
            }
            bf16* const out = static_cast<bf16*>(a.grad) + row * a.grad_pitch + c;
#pragma unroll
            for (int k = 0; k < TERMS; ++k) {
                float t[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    t[j] = first_term(g[j]);
                    g[j] = rest_of(g[j], t[j]);
                }
                if (inside(out + k * a.grad_plane, 8, a.grad, a.grad_room, a.err))
                    *reinterpret_cast<uint2*>(out + k * a.grad_plane) =
                        make_uint2(Elem<bf16>::pack2(t[0], t[1]), Elem<bf16>::pack2(t[2], t[3]));
            }
        }
    }
    if constexpr (TERMS == 0) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float mo = __shfl_xor_sync(0xffffffffu, m, o), so = __shfl_xor_sync(0xffffffffu, s, o);
            merge_pair(m, s, mo, so);
        }
        if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = make_float2(m, s);
        __syncthreads();
        if (threadIdx.x) return;
        for (int w = 1; w < kRowThreads / 32; ++w) merge_pair(m, s, parts[w].x, parts[w].y);
        const float l = (isinf(m) ? 0.f : m) + logf(s);
        lse[row] = l;
        loss[row] = ignored ? 0.f : outside ? NAN : l - picked;
    }
}

// The logits' gradient is divided by this number before it is rounded to one bf16 term,
// and what its products give is multiplied by it: the significand, 1 to 2, of the
// largest dloss.  That one becomes a power of two: the dloss of a mean, the same for
// every token, is not rounded at all (g = -dloss of an unlikely target: before, one
// relative error for all tokens, up to 2^-8 and 1.8e-3 of the gradient for 777 tokens),
// and others that are a little smaller lie where a rounding is least of a number.
__global__ void __launch_bounds__(1024)
vocab_unit(const float* dloss, const int64_t* target, int64_t ignore, int64_t tokens, float* unit) {
    __shared__ float tops[32];
    dependents_may_launch();
    wait_for_launches();
    float top = 0.f;
#pragma unroll 4
    for (int64_t t = threadIdx.x; t < tokens; t += 1024) {
        const float d = fabsf(dloss[t]);
        // (an infinite or subnormal one has no significand; a NaN is never larger)
        if (target[t] != ignore && d <= 3.402823466e38f && d >= 1.175494351e-38f) top = fmaxf(top, d);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x) return;
    for (int w = 1; w < 32; ++w) top = fmaxf(top, tops[w]);
    *unit = top == 0.f ? 1.f : __uint_as_float((__float_as_uint(top) & 0x007FFFFFu) | 0x3F800000u);
}

// The 16 bytes at `p`, at any even address, from the two lines that hold them.
__device__ __forceinline__ uint4 unaligned_line(const char* p) {
    const int at = (int)((uintptr_t)p & 15);
    const uint4* const line = reinterpret_cast<const uint4*>(p - at);
    const uint4 lo = __ldg(line), hi = at ? __ldg(line + 1) : lo;
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if (at & 8)
#pragma unroll
        for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
    if (at & 4)
#pragma unroll
        for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
    if (at & 2)
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows as bf16 terms, eight columns a thread (rows of dst are whole 16-byte lines,
// their last one padded with zeros); grid row y packs matrix y.
struct PackArgs {
    const void* src[2];
    bf16* dst[2];
    int64_t rows[2];
    int64_t pitch, plane[2];
    int cols;
    int64_t room[2];        // bytes at dst, and the error word (looked at by the checked build)
    unsigned* err;
};
template <typename T>
__global__ void __launch_bounds__(256) vocab_pack(PackArgs a) {
    dependents_may_launch();
    wait_for_launches();
    const bool second = blockIdx.y;
    const T* const src = static_cast<const T*>(second ? a.src[1] : a.src[0]);
    bf16* const dst = second ? a.dst[1] : a.dst[0];
    const int64_t rows = second ? a.rows[1] : a.rows[0], plane = second ? a.plane[1] : a.plane[0];
    const int64_t pitch = a.pitch;
    const int cols = a.cols, vecs = (cols + 7) / 8;
    const bool vec = (uintptr_t)src % 16 == 0 && cols % 4 == 0;
    const int64_t step = (int64_t)gridDim.x * 256, drow = step / vecs;
    const int dvec = (int)(step - drow * vecs);
    const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x;
    int64_t r = first / vecs;
    int v = (int)(first - r * vecs);
    while (r < rows) {
        const int c = 8 * v;
        const T* const p = src + r * cols + c;
        bf16* const q = dst + r * pitch + c;
        if (!inside(q + (sizeof(T) == 4 ? 2 : 0) * plane, 16, dst, second ? a.room[1] : a.room[0], a.err)) return;
        bool done = false;
        if constexpr (sizeof(T) == 2) {
            // (both lines lie inside the matrix; element by element 10778 rows of 1001
            // took 8.9 us, this way 7.4)
            const char* const b = reinterpret_cast<const char*>(p);
            const int at = (int)((uintptr_t)b & 15);
            done = c + 8 <= cols && b - at >= reinterpret_cast<const char*>(src) &&
                   b - at + 32 <= reinterpret_cast<const char*>(src + rows * cols);
            if (done) *reinterpret_cast<uint4*>(q) = unaligned_line(b);
        }
        if (!done) {
            float x[8];
            if (sizeof(T) == 4 && vec && c + 8 <= cols) {
                const float4 lo = *reinterpret_cast<const float4*>(p);
                const float4 hi = *reinterpret_cast<const float4*>(p + 4);
                x[0] = lo.x; x[1] = lo.y; x[2] = lo.z; x[3] = lo.w;
                x[4] = hi.x; x[5] = hi.y; x[6] = hi.z; x[7] = hi.w;
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = c + k < cols ? Elem<T>::to_f(p[k]) : 0.f;
            }
#pragma unroll
            for (int term = 0; term < (sizeof(T) == 4 ? 3 : 1); ++term) {
                float t[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    t[k] = sizeof(T) == 4 ? first_term(x[k]) : x[k];
                    if (sizeof(T) == 4) x[k] = rest_of(x[k], t[k]);
                }
                *reinterpret_cast<uint4*>(q + term * plane) = Elem<bf16>::pack(t);
            }
        }
        r += drow;
        v += dvec;
        if (v >= vecs) {
            v -= vecs;
            ++r;
        }
    }
}

// The splits' sums, four columns a thread.  Where there are many splits of few
// sums, G threads share a column's, each every Gth split, and the first adds theirs
// in order.
template <typename T, int G>
__global__ void __launch_bounds__(256)
vocab_sum(const float* sums, int splits, int64_t rows, int cols, int64_t pitch, const float* unit, T* out,
          bool vec, int64_t room, unsigned* err) {
    constexpr int kColumns = 256 / G;
    __shared__ float4 parts[G > 1 ? G : 1][G > 1 ? kColumns : 1];
    dependents_may_launch();
    wait_for_launches();
    const int vecs = (cols + 3) / 4, lane = (int)threadIdx.x % kColumns, group = (int)threadIdx.x / kColumns;
    const int64_t plane = rows * pitch, n = rows * vecs;
    const float by = unit ? *unit : 1.f;
    for (int64_t i0 = (int64_t)blockIdx.x * kColumns; i0 < n; i0 += (int64_t)gridDim.x * kColumns) {
        const int64_t i = i0 + lane, r = i / vecs;
        const int v = (int)(i - r * vecs);
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < n) {
            const float* p = sums + r * pitch + 4 * v + group * plane;
#pragma unroll 4
            for (int s = group; s < splits; s += G, p += G * plane) {
                if (!inside(p, 16, sums, room, err)) break;
                const float4 g = __ldcs(reinterpret_cast<const float4*>(p));
                f = make_float4(f.x + g.x, f.y + g.y, f.z + g.z, f.w + g.w);
            }
        }
        if constexpr (G > 1) {
            __syncthreads();
            parts[group][lane] = f;
            __syncthreads();
            if (group) continue;
            for (int k = 1; k < G; ++k) {
                const float4 g = parts[k][lane];
                f = make_float4(f.x + g.x, f.y + g.y, f.z + g.z, f.w + g.w);
            }
        }
        if (i >= n) continue;
        T* const q = out + r * cols + 4 * v;
        const float x[4] = {by * f.x, by * f.y, by * f.z, by * f.w};
        if (vec) {
            if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(q) = make_float4(x[0], x[1], x[2], x[3]);
            else *reinterpret_cast<uint2*>(q) = make_uint2(Elem<bf16>::pack2(x[0], x[1]),
                                                           Elem<bf16>::pack2(x[2], x[3]));
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (4 * v + k < cols) q[k] = Elem<T>::from_f(x[k]);
        }
    }
}

int blocks_for(int64_t n, int sms) {
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

cudaError_t launch_vocab(VocabOut out, VocabTerms terms, VocabTile tile, const CUtensorMap (&maps)[4],
                         const VocabArgs& args, int sms, cudaStream_t s) {
    const void* fn = out == kVocabStats ? vocab_stats_kernel(terms, tile)
                     : out == kVocabGrad ? vocab_grad_kernel(terms, tile)
                     : out == kVocabSums ? vocab_sums_kernel(terms)
                                         : vocab_product_kernel(terms, tile);
    int dev;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const KernelInfo* const info = kernel_info(dev, fn, false);  // its shared memory is opted in
    if (!info) return cudaErrorInvalidDeviceFunction;
    // (another compiler, or its flags)
    if (vocab_promotes(out, terms) && info->regs < vocab_launch_regs(vocab_tile_cols(tile)))
        return cudaErrorLaunchOutOfResources;
    const int ctas = vocab_tile_ctas(tile), most = sms / ctas;
    int64_t total = 0;
    for (int j = 0; j < args.jobs; ++j)
        total += (int64_t)args.work[j].mt * args.work[j].nt * args.work[j].splits;
    if (total > INT32_MAX / 2) return cudaErrorInvalidValue;
    const int units = (int)std::min<int64_t>(total, most);
    VocabArgs a = args;
    a.a_room = a.work[0].a_bytes;
    if (a.jobs > 1) a.a_room = std::max(a.a_room, a.work[1].a_bytes);
    a.lead = 0;
    if (a.jobs > 1) {
        // a tile of the first product is worth so many of the second
        const TileWork &x = a.work[0], &y = a.work[1];
        const int rest = (int)((int64_t)x.mt * x.nt * x.splits % units);
        if (rest) a.lead = std::min((x.per + y.per / 2) / y.per, y.mt * y.nt * y.splits / (units - rest));
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(units * ctas));
    cfg.blockDim = dim3((unsigned)vocab_threads(vocab_tile_cols(tile)));
    cfg.dynamicSmemBytes = kVocabSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0] = early_launch();
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    void* p[] = {const_cast<CUtensorMap*>(&maps[0]), const_cast<CUtensorMap*>(&maps[1]),
                 const_cast<CUtensorMap*>(&maps[2]), const_cast<CUtensorMap*>(&maps[3]), &a};
    return cudaLaunchKernelExC(&cfg, fn, p);
}

cudaError_t run_tiles_alone(int dev, int sms, VocabTile tile) {
    // one tile, more steps of k than a ring has stages
    constexpr int kDepth = 2 * kVocabStages * kTileK;
    const int rows = vocab_tile_rows(tile), cols = vocab_tile_cols(tile), pitch = 2 * kDepth;
    const size_t need = (size_t)(rows + cols) * pitch + (size_t)rows * (8 + 4 + 8 * vocab_tile_parts(tile));
    char* buf = nullptr;
    cudaError_t e = cudaMalloc(&buf, need);
    if (e != cudaSuccess) return e;
    e = cudaMemset(buf, 0, need);
    const TermMatrix h{buf, rows, kDepth, pitch, (int64_t)pitch * rows, 1};
    const TermMatrix w{buf + h.plane, cols, kDepth, pitch, (int64_t)pitch * cols, 1};
    VocabArgs a{};
    a.jobs = 1;
    a.work[0] = {1, 1, 1, kDepth / kTileK, kDepth / kTileK, 1, 0, 0, 0, kBytesA, 0};
    a.rows = rows;
    a.cols = cols;
    a.vocab = cols;
    char* const rest = buf + h.plane + w.plane;
    a.parts_room = (int64_t)rows * 8 * vocab_tile_parts(tile);
    a.target = reinterpret_cast<int64_t*>(rest);
    a.picked = reinterpret_cast<float*>(rest + (size_t)rows * 8);
    a.parts = reinterpret_cast<float2*>(rest + (size_t)rows * 12);
    a.err = device_error_word();
    a.alone = 1;
    CUtensorMap maps[4] = {};
    if (e == cudaSuccess && (!a.err || !term_map(h, kTileM, &maps[0]) ||
                             !term_map(w, cols / vocab_tile_ctas(tile), &maps[1])))
        e = cudaErrorInvalidValue;
    if (e == cudaSuccess) e = launch_vocab(kVocabStats, kTerms1, tile, maps, a, sms, nullptr);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    const cudaError_t f = cudaFree(buf);
    return e != cudaSuccess ? e : f;
}

cudaError_t launch_vocab_merge(const VocabArgs& a, int nparts, float* loss, float* lse,
                               cudaStream_t s) {
    const dim3 grid((unsigned)((a.rows + kMergeRows - 1) / kMergeRows));
    return nparts < 512 ? launch_early(vocab_merge<256>, grid, 256, s, a, nparts, loss, lse)
                        : launch_early(vocab_merge<1024>, grid, 1024, s, a, nparts, loss, lse);
}

cudaError_t launch_vocab_rows(const VocabArgs& a, const float* sums, int splits, int64_t pitch,
                              VocabTerms terms, float* loss, float* lse, cudaStream_t s) {
    auto* fn = !a.grad ? vocab_rows<0>
               : terms == kTerms1 ? vocab_rows<1> : terms == kTerms2 ? vocab_rows<2> : vocab_rows<3>;
    return launch_early(fn, dim3((unsigned)a.rows), kRowThreads, s, a, sums, splits, pitch, loss, lse);
}

cudaError_t launch_vocab_unit(const float* dloss, const int64_t* target, int64_t ignore, int64_t tokens,
                              float* unit, cudaStream_t s) {
    return launch_early(vocab_unit, dim3(1), 1024, s, dloss, target, ignore, tokens, unit);
}

cudaError_t launch_vocab_pack(int dtype, const void* const (&src)[2], const TermMatrix (&dst)[2], int n,
                              unsigned* err, int sms, cudaStream_t s) {
    PackArgs a{};
    a.err = err;
    int64_t rows = 0;
    for (int i = 0; i < n; ++i) {
        a.src[i] = src[i];
        a.dst[i] = static_cast<bf16*>(const_cast<void*>(dst[i].p));
        a.rows[i] = dst[i].rows;
        a.plane[i] = dst[i].plane / 2;
        a.room[i] = dst[i].plane * dst[i].terms;
        rows = std::max(rows, dst[i].rows);
    }
    a.pitch = dst[0].pitch / 2;
    a.cols = (int)dst[0].cols;
    const dim3 grid((unsigned)blocks_for(rows * ((a.cols + 7) / 8), sms), (unsigned)n);
    return dtype == 0 ? launch_early(vocab_pack<float>, grid, 256, s, a)
                      : launch_early(vocab_pack<bf16>, grid, 256, s, a);
}

cudaError_t launch_vocab_sum(int dtype, const float* sums, int splits, int64_t rows, int64_t cols,
                             int64_t pitch, const float* unit, void* out, int64_t room, unsigned* err, int sms,
                             cudaStream_t s) {
    const int64_t n = rows * ((cols + 3) / 4);
    const bool vec = (uintptr_t)out % 16 == 0 && cols % 4 == 0, shared = splits >= 16;
    const dim3 grid((unsigned)blocks_for(shared ? 16 * n : n, sms));
    auto run = [&](auto* fn, auto* o) {
        return launch_early(fn, grid, 256, s, sums, splits, rows, (int)cols, pitch, unit, o, vec, room,
                            err);
    };
    if (dtype == 0)
        return run(shared ? vocab_sum<float, 16> : vocab_sum<float, 1>, static_cast<float*>(out));
    return run(shared ? vocab_sum<bf16, 16> : vocab_sum<bf16, 1>, static_cast<bf16*>(out));
}

}  // namespace credit
