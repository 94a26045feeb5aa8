// vocab_few.cu -- the linear head's cross entropy of a few tokens (a step of
// generation, a score): the weight is read once in its own type and at any
// alignment, without tensor cores, whose products of 128 rows would stand idle and
// whose operands would have to be whole 16-byte lines of bf16.
//
//   few_logits    a warp holds four vocabulary rows' dot products with every token;
//                 the tokens lie in shared memory as fp32
//   few_products  a thread holds columns of every token's dhidden, and of the tokens,
//                 and walks a slice of the vocabulary: w is read and dweight written
//                 on the way
//
// Measured (device time): one token of 131072 x 4096 forward 163 us bf16 (0.97 of the
// copy rate), 301 fp32; backward 519 bf16 (0.91 of it for the three passes over the
// weight's size).  Bound by HBM for one token; by the shared-memory reads of the tokens
// for eight (131072 x 2048 fp32 212 us, x 2047 bf16 216), so aligned bf16 takes tiles
// from two tokens on.  A lane has 16 vectors in flight for one token (four took 220 us);
// of eight tokens the next step's loads are issued before a step is used, by sixteen
// warps that share one copy of the tokens (263 and 260 us without, in CTAs of eight
// warps); four tokens lose by the same (97 to 115 us at 32768 x 4096 fp32).
#include <algorithm>

#include "early_launch.h"
#include "planner.h"
#include "rowops.cuh"
#include "sweep.cuh"
#include "vocab.h"

namespace credit {

namespace {

constexpr int kThreads = 256;
// few_logits: sixteen warps an SM, in one CTA where eight tokens fill its shared memory
constexpr int few_threads(int tokens) { return tokens == 8 ? 512 : 256; }
constexpr int kRows = 4;         // vocabulary rows of a warp
constexpr int kGrads = 1024;     // gradients of logits that few_products stages at a time

// A lane's elements of a step of a row: VEC, consecutive ones in a 16-byte vector;
// else one of each 32.
template <typename T, bool VEC> struct FewIO {
    static constexpr int N = VEC ? 16 / (int)sizeof(T) : 4;
    static constexpr int kStep = 32 * N;
    using Word = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
    struct Raw { uint4 v; };
    __device__ static __forceinline__ int first(int lane) { return VEC ? lane * N : lane; }
    // the elements from column c of a row of `cols` on, zeros past its end
    __device__ static __forceinline__ Raw load(const T* row, int c, int cols) {
        Raw r{make_uint4(0, 0, 0, 0)};
        if constexpr (VEC) {
            if (c < cols) r.v = ld_global_nc_l1na_v4(row + c);
        } else {
            const Word* const w = reinterpret_cast<const Word*>(row) + c;
            if (c < cols) r.v.x = w[0];
            if (c + 32 < cols) r.v.y = w[32];
            if (c + 64 < cols) r.v.z = w[64];
            if (c + 96 < cols) r.v.w = w[96];
        }
        return r;
    }
    __device__ static __forceinline__ void unpack(const Raw& r, float (&f)[N]) {
        if constexpr (VEC) {
            Elem<T>::unpack(r.v, f);
        } else {
            const int shift = 32 - 8 * (int)sizeof(T);
            f[0] = __uint_as_float(r.v.x << shift);
            f[1] = __uint_as_float(r.v.y << shift);
            f[2] = __uint_as_float(r.v.z << shift);
            f[3] = __uint_as_float(r.v.w << shift);
        }
    }
};

template <typename T, bool VEC, int TOKENS>
__global__ void __launch_bounds__(few_threads(TOKENS)) few_logits(FewArgs a) {
    using IO = FewIO<T, VEC>;
    constexpr int N = IO::N, kSums = kRows * TOKENS, kThreads = few_threads(TOKENS), kWarps = kThreads / 32;
    extern __shared__ __align__(16) float hidden[];     // TOKENS x pitch
    __shared__ float2 parts[kWarps][TOKENS];
    dependents_may_launch();
    wait_for_launches();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, pitch = a.pitch;
    // (the tokens' room, which every step of a row stays in: zeros up to the pitch)
    if (!layout_fits((uint64_t)TOKENS * pitch * 4, 0, 0, a.err) ||
        !in_bounds((a.cols + IO::kStep - 1) / IO::kStep * IO::kStep <= pitch, a.err))
        return;
    for (int i = threadIdx.x; i < TOKENS * pitch; i += kThreads) {
        const int t = i / pitch, c = i - t * pitch;
        hidden[i] = t < a.tokens && c < a.cols ? Elem<T>::to_f(static_cast<const T*>(a.h)[(int64_t)t * a.cols + c])
                                               : 0.f;
    }
    // a lane's dot product, of row `r` of the warp's with token `t`
    const int mine = lane / (32 / kSums), t = mine % TOKENS, r = mine / TOKENS;
    const bool live = t < a.tokens, writes = live && lane % (32 / kSums) == 0;
    const int64_t target = live ? a.target[t] : -1;
    float scale = 0.f, both = 0.f, lse = 0.f;
    if (a.grad && live) {
        scale = target == a.ignore ? 0.f : target < 0 || target >= a.vocab ? NAN : a.dloss[t];
        both = scale + (a.dlse ? a.dlse[t] : 0.f);
        lse = a.lse[t];
    }
    __syncthreads();
    float m = -INFINITY, s = 0.f;
    const int64_t groups = (a.vocab + kRows - 1) / kRows;
    for (int64_t g = (int64_t)blockIdx.x * kWarps + warp; g < groups; g += (int64_t)gridDim.x * kWarps) {
        const int64_t v0 = g * kRows;
        const T* row[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k)  // (past the last row: the last again)
            row[k] = static_cast<const T*>(a.w) + min(v0 + k, a.vocab - 1) * a.cols;
        F2 sum[kRows][TOKENS];
#pragma unroll
        for (int k = 0; k < kRows; ++k)
#pragma unroll
            for (int j = 0; j < TOKENS; ++j) sum[k][j] = f2(0.f);
        // kUnroll steps' loads at once, of eight tokens the next step's before these
        // are used
        constexpr int kUnroll = TOKENS == 1 ? 4 : TOKENS == 4 ? 2 : 1;
        constexpr bool kAhead = TOKENS == 8;
        typename IO::Raw raw[kUnroll][kRows];
        auto fetch = [&](int c0) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
#pragma unroll
                for (int k = 0; k < kRows; ++k) raw[u][k] = IO::load(row[k], c0 + u * IO::kStep, a.cols);
        };
        if (kAhead) fetch(IO::first(lane));
        for (int c0 = IO::first(lane); c0 < a.cols; c0 += kUnroll * IO::kStep) {
            if (!kAhead) fetch(c0);
            typename IO::Raw now[kUnroll][kRows];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
#pragma unroll
                for (int k = 0; k < kRows; ++k) now[u][k] = raw[u][k];
            if (kAhead) fetch(c0 + kUnroll * IO::kStep);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int c = c0 + u * IO::kStep;
                if (u > 0 && c >= a.cols) break;
                float x[kRows][N];
#pragma unroll
                for (int k = 0; k < kRows; ++k) IO::unpack(now[u][k], x[k]);
#pragma unroll
                for (int j = 0; j < TOKENS; ++j) {
                    const float* const h = hidden + j * pitch + c;
#pragma unroll
                    for (int e = 0; e < N; e += 4) {
                        F2 y[2];
                        if constexpr (VEC) {
                            const float4 q = *reinterpret_cast<const float4*>(h + e);
                            y[0] = {q.x, q.y};
                            y[1] = {q.z, q.w};
                        } else {
                            y[0] = {h[32 * e], h[32 * e + 32]};
                            y[1] = {h[32 * e + 64], h[32 * e + 96]};
                        }
#pragma unroll
                        for (int k = 0; k < kRows; ++k) {
                            sum[k][j] = fma2(F2{x[k][e], x[k][e + 1]}, y[0], sum[k][j]);
                            sum[k][j] = fma2(F2{x[k][e + 2], x[k][e + 3]}, y[1], sum[k][j]);
                        }
                    }
                }
            }
        }
        __syncwarp();
        float z[kSums];
#pragma unroll
        for (int k = 0; k < kRows; ++k)
#pragma unroll
            for (int j = 0; j < TOKENS; ++j) z[k * TOKENS + j] = sum[k][j].x + sum[k][j].y;
        const float logit = sums_over_warp<kSums>(z, lane);
        const int64_t v = v0 + r;
        if (v >= a.vocab) continue;
        if (a.grad) {
            const float e = both == 0.f ? 0.f : both * expf(logit - lse);
            float* const p = a.grad + v * TOKENS + t;
            if (lane % (32 / kSums) == 0 && inside(p, 4, a.grad, a.grad_room, a.err))
                *p = live ? (v == target && target != a.ignore ? e - scale : e) : 0.f;
            continue;
        }
        const float top = fmaxf(m, logit), base = isinf(top) ? 0.f : top;
        s = (s == 0.f ? 0.f : s * expf(m - base)) + expf(logit - base);
        m = top;
        if (writes && v == target && in_bounds(t < a.tokens, a.err)) a.picked[t] = logit;
    }
    if (a.grad) return;
    // the rows of a token, then the warps
    auto merge = [&](float mo, float so) {
        const float top = fmaxf(m, mo), base = isinf(top) ? 0.f : top;
        s = (s == 0.f ? 0.f : s * expf(m - base)) + (so == 0.f ? 0.f : so * expf(mo - base));
        m = top;
    };
    __syncwarp();
#pragma unroll
    for (int o = 16; o >= 32 / kRows; o >>= 1) {
        const float mo = __shfl_xor_sync(0xffffffffu, m, o), so = __shfl_xor_sync(0xffffffffu, s, o);
        merge(mo, so);
    }
    if (writes && r == 0) parts[warp][t] = make_float2(m, s);
    __syncthreads();
    if (warp || !writes || r) return;
    for (int w = 1; w < kWarps; ++w) merge(parts[w][t].x, parts[w][t].y);
    float2* const p = a.parts + (int64_t)blockIdx.x * a.parts_pitch + t;
    if (inside(p, sizeof(*p), a.parts, a.parts_room, a.err)) *p = make_float2(m, s);
}

// Grid: x the column blocks, y the slices of the vocabulary.
template <typename T, bool VEC, int TOKENS>
__global__ void __launch_bounds__(kThreads) few_products(FewArgs a) {
    constexpr int N = FewIO<T, VEC>::N, kUnroll = TOKENS > 4 ? 2 : 4;
    __shared__ __align__(16) float grads[kGrads];
    dependents_may_launch();
    wait_for_launches();
    const int c0 = (int)blockIdx.x * kThreads * N + (VEC ? (int)threadIdx.x * N : (int)threadIdx.x);
    auto col = [&](int k) { return c0 + (VEC ? k : kThreads * k); };
    const int64_t lo = a.vocab * blockIdx.y / gridDim.y, hi = a.vocab * (blockIdx.y + 1) / gridDim.y;
    const T* const w = static_cast<const T*>(a.w);
    T* const dw = static_cast<T*>(a.dw);
    float h[TOKENS][N], sum[TOKENS][N];
#pragma unroll
    for (int t = 0; t < TOKENS; ++t)
#pragma unroll
        for (int k = 0; k < N; ++k) {
            sum[t][k] = 0.f;
            h[t][k] = dw && t < a.tokens && col(k) < a.cols
                          ? Elem<T>::to_f(static_cast<const T*>(a.h)[(int64_t)t * a.cols + col(k)]) : 0.f;
        }
    const bool there = c0 < a.cols;  // (VEC: the whole vector)
    for (int64_t v0 = lo; v0 < hi; v0 += kGrads / TOKENS) {
        const int n = (int)min(hi - v0, (int64_t)(kGrads / TOKENS));
        __syncthreads();
        for (int i = threadIdx.x; i < n * TOKENS; i += kThreads)
            grads[i] = in_bounds(i < kGrads, a.err) &&
                               inside(a.grad + v0 * TOKENS + i, 4, a.grad, a.grad_room, a.err)
                           ? a.grad[v0 * TOKENS + i] : 0.f;
        __syncthreads();
        if (!there) continue;
        for (int i0 = 0; i0 < n; i0 += kUnroll) {
            float x[kUnroll][N];
            if (a.sums)
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const T* const row = w + (v0 + min(i0 + u, n - 1)) * a.cols;
                    if constexpr (VEC) {
                        Elem<T>::unpack(ld_global_nc_l1na_v4(row + c0), x[u]);
                    } else {
#pragma unroll
                        for (int k = 0; k < N; ++k) x[u][k] = col(k) < a.cols ? Elem<T>::to_f(row[col(k)]) : 0.f;
                    }
                }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (i0 + u >= n) break;
                float g[TOKENS], y[N];
#pragma unroll
                for (int t = 0; t < TOKENS; ++t) g[t] = grads[(i0 + u) * TOKENS + t];
                if (a.sums)
#pragma unroll
                    for (int t = 0; t < TOKENS; ++t)
#pragma unroll
                        for (int k = 0; k < N; ++k) sum[t][k] = fmaf(g[t], x[u][k], sum[t][k]);
                if (!dw) continue;
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    y[k] = g[0] * h[0][k];
#pragma unroll
                    for (int t = 1; t < TOKENS; ++t) y[k] = fmaf(g[t], h[t][k], y[k]);
                }
                T* const row = dw + (v0 + i0 + u) * a.cols;
                const size_t room = (size_t)(a.vocab * a.cols) * sizeof(T);
                if constexpr (VEC) {
                    if (inside(row + c0, 16, dw, room, a.err)) st_global_cs_v4(row + c0, Elem<T>::pack(y));
                } else {
#pragma unroll
                    for (int k = 0; k < N; ++k)
                        if (col(k) < a.cols && inside(row + col(k), sizeof(T), dw, room, a.err))
                            row[col(k)] = Elem<T>::from_f(y[k]);
                }
            }
        }
    }
    if (!a.sums || !there) return;
#pragma unroll
    for (int t = 0; t < TOKENS; ++t) {
        if (t >= a.tokens) break;
        float* const p = a.sums + ((int64_t)blockIdx.y * a.tokens + t) * a.sums_pitch;
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (col(k) < a.cols && inside(p + col(k), 4, a.sums, a.sums_room, a.err)) p[col(k)] = sum[t][k];
    }
}

// f(type, vector access, tokens) with the call's constants.
template <typename F> cudaError_t with_constants(int dtype, bool vec, int tokens, F f) {
    auto typed = [&](auto type, auto v) {
        switch (few_tokens(tokens)) {
            case 1: return f(type, v, std::integral_constant<int, 1>());
            case 4: return f(type, v, std::integral_constant<int, 4>());
            default: return f(type, v, std::integral_constant<int, 8>());
        }
    };
    if (dtype == 0) return vec ? typed(0.f, std::true_type()) : typed(0.f, std::false_type());
    return vec ? typed(bf16(), std::true_type()) : typed(bf16(), std::false_type());
}

int room_of(const FewArgs& a) { return few_tokens(a.shaped) * a.pitch * 4; }

}  // namespace

int few_blocks(int tokens, int pitch, int64_t vocab, int sms) {
    const int room = few_tokens(tokens) * pitch * 4;
    const int warps = few_threads(few_tokens(tokens)) / 32;
    const int64_t groups = (vocab + kRows - 1) / kRows;
    // CTAs of an SM, as shared memory and registers allow
    const int most = std::max(1, std::min(32 / warps, 220000 / (room + 5120)));
    return (int)std::min<int64_t>((groups + warps - 1) / warps, (int64_t)sms * most);
}

int few_slices(int64_t cols, int dtype, bool vec, int64_t vocab, int sms) {
    const int n = vec ? dtype ? 8 : 4 : 4;
    const int64_t blocks = (cols + kThreads * n - 1) / (kThreads * n);
    return (int)std::max<int64_t>(1, std::min<int64_t>((4 * sms + blocks - 1) / blocks, (vocab + 31) / 32));
}

cudaError_t launch_few_logits(int dtype, bool vec, const FewArgs& a, int blocks, cudaStream_t s) {
    return with_constants(dtype, vec, a.shaped, [&](auto type, auto v, auto tokens) -> cudaError_t {
        auto* fn = &few_logits<decltype(type), decltype(v)::value, decltype(tokens)::value>;
        int dev;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (!kernel_info(dev, (const void*)fn, false)) return cudaErrorInvalidDeviceFunction;
        cudaLaunchAttribute attr = early_launch();
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)blocks);
        cfg.blockDim = dim3((unsigned)few_threads(few_tokens(a.shaped)));
        cfg.dynamicSmemBytes = (size_t)room_of(a);
        cfg.stream = s;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, fn, a);
    });
}

cudaError_t launch_few_products(int dtype, bool vec, const FewArgs& a, int slices, cudaStream_t s) {
    return with_constants(dtype, vec, a.shaped, [&](auto type, auto v, auto tokens) -> cudaError_t {
        using IO = FewIO<decltype(type), decltype(v)::value>;
        const dim3 grid((unsigned)((a.cols + kThreads * IO::N - 1) / (kThreads * IO::N)), (unsigned)slices);
        return launch_early(few_products<decltype(type), decltype(v)::value, decltype(tokens)::value>, grid,
                            kThreads, s, a);
    });
}

}  // namespace credit
