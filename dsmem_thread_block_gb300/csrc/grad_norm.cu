// grad_norm.cu -- the 2-norm of many tensors together, and their clipping:
//   norm = sqrt(sum_i sum_e g_ie^2),  out_ie = g_ie min(1, max_norm / (norm + eps))
//
// Two kernels: every CTA sums the squares of a run of 32 KB chunks, whatever tensors
// they lie in; then every CTA adds the CTAs' sums in one order and scales the same run.
// Sums are fp32 over a thread's 32 or 64 elements of a chunk and 64 bits from there on.
//
// Bound by HBM: elements are read, read again once the norm is known, and written.
// Measured (device time, share of the 6787 GB/s copy rate over those three passes):
//   805 MB of bf16, clipped      379 us  0.94
//   1.2 GB of fp32, clipped      552 us  0.97
//   360 MB of 456 tensors, norm   60 us  0.88 (one pass; a run in flight a CTA, and the
//                                 second launch)
//   2.7 MB of 12 tensors         10 us   the call's host side
// Runs are walked backwards the second time, and their ends are read with an L2 policy
// that keeps them (71 MB of 805 are not read again): 391 us without.
#include <algorithm>
#include <climits>
#include <vector>

#include "credit.h"
#include "early_launch.h"
#include "internal.h"
#include "planner.h"
#include "rowops.cuh"

using namespace credit;

namespace {

constexpr int kThreads = 256;
constexpr int kLoads = 8;                           // 16-byte vectors of a thread and chunk
constexpr int kChunkBytes = kThreads * kLoads * 16;
constexpr int kCtasPerSm = 4;
// Of L2, what the sums leave there for the scaling: the last chunks of every CTA
// (805 MB: none 391 us, a quarter 390, half 383, three quarters 382).
constexpr int kKeepNum = 1, kKeepDen = 2;

// The tensors of a launch, in its parameters: captured with it, nothing to copy
// or keep.  Chunks are counted through all tensors; a tensor's start at its
// first byte's 16-byte line.
template <int N> struct Table {
    const void* p[N];
    void* out[N];
    int64_t count[N];
    int32_t first[N + 1];   // chunk
    uint8_t half[N];        // bf16
    int32_t n;
    unsigned* err;          // (looked at by the checked build)
};
constexpr int kSmall = 64, kLarge = 960;
static_assert(sizeof(Table<kLarge>) + 64 <= 32764, "kernel parameters");

// Sums of squares of a thread and chunk.  A square overflows from 2^64 on and
// loses digits below 2^-63, so the same sum is kept of values scaled down and up,
// and the one that holds its digits is taken.
struct Squares {
    F2 mid, low, high;
    __device__ Squares() : mid(f2(0.f)), low(f2(0.f)), high(f2(0.f)) {}
    __device__ __forceinline__ void add(F2 x) {
        const F2 d = mul2(x, f2(0x1p-80f)), u = mul2(x, f2(0x1p90f));
        mid = fma2(x, x, mid);
        low = fma2(d, d, low);
        high = fma2(u, u, high);
    }
    __device__ __forceinline__ double sum() const {
        const float m = mid.x + mid.y;
        if (m <= 3.402823466e38f && m >= 0x1p-80f) return (double)m;
        // (a NaN, or an overflow)
        if (!(m < 0x1p-80f)) return (double)(low.x + low.y) * 0x1p160;
        return (double)(high.x + high.y) * 0x1p-180;
    }
};

__device__ __forceinline__ double cta_sum(double v) {
    __shared__ double parts[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) t += parts[w];
    return t;
}

// Is this chunk one of tensor i's?
template <int N>
__device__ __forceinline__ bool chunk_of(const Table<N>& t, int i, int c) {
    return in_bounds(i >= 0 && i < t.n && c >= t.first[i] && c < t.first[i + 1], t.err);
}

// The chunks of a CTA: a run of the launch's.
__device__ __forceinline__ void run_of(int chunks, int& lo, int& hi) {
    lo = (int)((int64_t)chunks * blockIdx.x / gridDim.x);
    hi = (int)((int64_t)chunks * (blockIdx.x + 1) / gridDim.x);
}

// The tensor that holds chunk c.
template <int N> __device__ __forceinline__ int tensor_of(const Table<N>& t, int c) {
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (t.first[m] <= c) lo = m; else hi = m - 1;
    }
    return lo;
}

// A thread's vectors of a chunk: f(vector's first element, elements, whole) for
// each, all loads first.
template <typename T> struct Vectors {
    static constexpr int kVec = 16 / sizeof(T);
    uint4 v[kLoads];
    int64_t e0;      // first element of the thread's first vector (below 0: before the tensor)
    __device__ __forceinline__ int64_t at(int k) const { return e0 + (int64_t)k * kThreads * kVec; }
    __device__ __forceinline__ bool whole(int k, int64_t count) const {
        return at(k) >= 0 && at(k) + kVec <= count;
    }
    __device__ __forceinline__ void load(const T* p, int64_t count, int64_t chunk, uint64_t policy) {
        const int shift = (int)(((uintptr_t)p & 15) / sizeof(T));
        e0 = chunk * (kChunkBytes / (int)sizeof(T)) + threadIdx.x * kVec - shift;
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
            v[k] = make_uint4(0, 0, 0, 0);
            if (whole(k, count)) {
                v[k] = ld_global_l2hint_v4(p + at(k), policy);
            } else if (at(k) < count) {
                T x[kVec];
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    x[e] = at(k) + e >= 0 && at(k) + e < count ? p[at(k) + e] : Elem<T>::from_f(0.f);
                v[k] = *reinterpret_cast<const uint4*>(x);
            }
        }
    }
};

template <typename T>
__device__ __forceinline__ double chunk_squares(const void* p, int64_t count, int64_t chunk,
                                                uint64_t policy) {
    Vectors<T> x;
    x.load(static_cast<const T*>(p), count, chunk, policy);
    Squares s;
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
        float f[Vectors<T>::kVec];
        Elem<T>::unpack(x.v[k], f);
#pragma unroll
        for (int e = 0; e < Vectors<T>::kVec; e += 2) s.add(F2{f[e], f[e + 1]});
    }
    return s.sum();
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const void* p, void* out, int64_t count, int64_t chunk,
                                            float factor) {
    Vectors<T> x;
    x.load(static_cast<const T*>(p), count, chunk, l2_policy_evict_first());
    T* const y = static_cast<T*>(out);
    const bool lines = (((uintptr_t)p ^ (uintptr_t)out) & 15) == 0;
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
        if (x.at(k) >= count) break;
        float f[Vectors<T>::kVec];
        Elem<T>::unpack(x.v[k], f);
#pragma unroll
        for (int e = 0; e < Vectors<T>::kVec; ++e) f[e] *= factor;
        if (lines && x.whole(k, count)) {
            __stcs(reinterpret_cast<uint4*>(y + x.at(k)), Elem<T>::pack(f));
        } else {
#pragma unroll
            for (int e = 0; e < Vectors<T>::kVec; ++e)
                if (x.at(k) + e >= 0 && x.at(k) + e < count) y[x.at(k) + e] = Elem<T>::from_f(f[e]);
        }
    }
}

template <int N>
__global__ void __launch_bounds__(kThreads)
grad_squares(const __grid_constant__ Table<N> t, double* parts, int keep) {
    dependents_may_launch();
    wait_for_launches();
    int lo, hi;
    run_of(t.first[t.n], lo, hi);
    double sum = 0.0;
    int i = tensor_of(t, lo);
    for (int c = lo; c < hi; ++c) {
        while (c >= t.first[i + 1]) ++i;
        if (!chunk_of(t, i, c)) break;
        const int64_t chunk = c - t.first[i];
        const uint64_t policy = c < hi - keep ? l2_policy_evict_first() : l2_policy_evict_last();
        sum += t.half[i] ? chunk_squares<bf16>(t.p[i], t.count[i], chunk, policy)
                         : chunk_squares<float>(t.p[i], t.count[i], chunk, policy);
    }
    sum = cta_sum(sum);
    if (threadIdx.x == 0) parts[blockIdx.x] = sum;
}

// The norm from every CTA's sum, added in one order by whoever asks.
__device__ __forceinline__ float norm_of(const double* parts, int n) {
    double v = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) v += parts[i];
    return (float)sqrt(cta_sum(v));
}

__global__ void __launch_bounds__(kThreads) grad_norm(const double* parts, int n, float* norm) {
    dependents_may_launch();
    wait_for_launches();
    const float v = norm_of(parts, n);
    if (threadIdx.x == 0) *norm = v;
}

// The same runs as grad_squares, walked backwards: their ends are still in L2.
template <int N>
__global__ void __launch_bounds__(kThreads)
grad_scale(const __grid_constant__ Table<N> t, const double* parts, int nparts, float max_norm,
           float eps, float* norm, bool in_place) {
    dependents_may_launch();
    wait_for_launches();
    const float v = norm_of(parts, nparts);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
    float factor = max_norm / (v + eps);
    if (factor > 1.f) factor = 1.f;   // (a NaN stays)
    if (in_place && factor == 1.f) return;
    int lo, hi;
    run_of(t.first[t.n], lo, hi);
    if (lo == hi) return;
    int i = tensor_of(t, hi - 1);
    for (int c = hi - 1; c >= lo; --c) {
        while (c < t.first[i]) --i;
        if (!chunk_of(t, i, c)) break;
        const int64_t chunk = c - t.first[i];
        if (t.half[i]) chunk_scale<bf16>(t.p[i], t.out[i], t.count[i], chunk, factor);
        else chunk_scale<float>(t.p[i], t.out[i], t.count[i], chunk, factor);
    }
}

// A call's tensors, those without elements left out, in launches of kLarge.
int64_t chunks_of(const credit_tensor_t& t) {
    const int64_t bytes = t.count * (t.dtype == CREDIT_F32 ? 4 : 2) + ((uintptr_t)t.data & 15);
    return (bytes + kChunkBytes - 1) / kChunkBytes;
}

struct Batch {
    int64_t begin, end;   // of the call's tensors
    int32_t n, chunks, grid;
};

// False where a launch's chunks pass 32 bits.
bool batches_of(const credit_tensor_t* t, int64_t n, int sms, std::vector<Batch>* out) {
    Batch b{0, 0, 0, 0, 0};
    int64_t chunks = 0;
    auto close = [&](int64_t end) {
        b.end = end;
        b.chunks = (int32_t)chunks;
        b.grid = (int32_t)std::min<int64_t>(chunks, (int64_t)sms * kCtasPerSm);
        if (b.n) out->push_back(b);
        b = Batch{end, end, 0, 0, 0};
        chunks = 0;
    };
    for (int64_t i = 0; i < n; ++i) {
        if (t[i].count == 0) continue;
        const int64_t c = chunks_of(t[i]);
        if (c > INT_MAX / 2) return false;
        if (b.n == kLarge || chunks + c > INT_MAX / 2) close(i);
        ++b.n;
        chunks += c;
    }
    close(n);
    return true;
}

template <int N> void fill(const credit_tensor_t* t, const Batch& b, Table<N>* table) {
    int k = 0, c = 0;
    for (int64_t i = b.begin; i < b.end; ++i) {
        if (t[i].count == 0) continue;
        table->p[k] = t[i].data;
        table->out[k] = t[i].out;
        table->count[k] = t[i].count;
        table->half[k] = t[i].dtype == CREDIT_BF16;
        table->first[k] = c;
        c += (int)chunks_of(t[i]);
        ++k;
    }
    table->first[k] = c;
    table->n = k;
    table->err = checked_error_word();
}

struct Range {
    uintptr_t lo, hi;
    bool out;
};

credit_status_t check(const credit_tensor_t* t, int64_t n, bool outs, const Range* more, int nmore) {
    std::vector<Range> r(more, more + nmore);
    for (int64_t i = 0; i < n; ++i) {
        if (t[i].dtype != CREDIT_F32 && t[i].dtype != CREDIT_BF16) return CREDIT_ERR_UNSUPPORTED;
        const int64_t es = t[i].dtype == CREDIT_F32 ? 4 : 2;
        if (t[i].count < 0 || t[i].count > INT64_MAX / 64) return CREDIT_ERR_INVALID_ARG;
        if (t[i].count == 0) continue;
        if (!t[i].data || (uintptr_t)t[i].data % es) return CREDIT_ERR_INVALID_ARG;
        const uintptr_t bytes = (uintptr_t)(t[i].count * es);
        const uintptr_t p = (uintptr_t)t[i].data, q = (uintptr_t)t[i].out;
        if (outs && (!q || q % es)) return CREDIT_ERR_INVALID_ARG;
        if (!outs || p != q) r.push_back({p, p + bytes, false});
        if (outs) r.push_back({q, q + bytes, true});
    }
    // no output meets another buffer: sorted, each range against the furthest end before it
    std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
    uintptr_t end_in = 0, end_out = 0;
    for (const Range& a : r) {
        if (a.lo == a.hi) continue;
        if (a.lo < end_out || (a.out && a.lo < end_in)) return CREDIT_ERR_INVALID_ARG;
        uintptr_t& e = a.out ? end_out : end_in;
        e = std::max(e, a.hi);
    }
    return CREDIT_OK;
}

credit_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? CREDIT_OK : CREDIT_ERR_CUDA; }

template <int N>
cudaError_t launch_batch(const credit_tensor_t* t, const Batch& b, double* parts, int nparts,
                         bool scale, float max_norm, float eps, float* norm, bool in_place, int keep,
                         cudaStream_t s) {
    Table<N> table;
    fill<N>(t, b, &table);
    cudaLaunchAttribute attr = early_launch();
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)b.grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    void* sum_args[] = {&table, &parts, &keep};
    void* scale_args[] = {&table, &parts, &nparts, &max_norm, &eps, &norm, &in_place};
    return scale ? cudaLaunchKernelExC(&cfg, (const void*)grad_scale<N>, scale_args)
                 : cudaLaunchKernelExC(&cfg, (const void*)grad_squares<N>, sum_args);
}

cudaError_t launch_any(const credit_tensor_t* t, const Batch& b, double* parts, int nparts, bool scale,
                       float max_norm, float eps, float* norm, bool in_place, int keep, cudaStream_t s) {
    return b.n <= kSmall
               ? launch_batch<kSmall>(t, b, parts, nparts, scale, max_norm, eps, norm, in_place, keep, s)
               : launch_batch<kLarge>(t, b, parts, nparts, scale, max_norm, eps, norm, in_place, keep, s);
}

credit_status_t run(const credit_tensor_t* t, int64_t n, bool clip, float max_norm, float eps,
                    float* norm, void* workspace, size_t workspace_bytes, void* stream) try {
    if (n < 0 || (n && !t) || !norm || (uintptr_t)norm % 4) return CREDIT_ERR_INVALID_ARG;
    const uintptr_t w = (uintptr_t)workspace, o = (uintptr_t)norm;
    const Range more[] = {{o, o + 4, true}, {w, w + (workspace ? workspace_bytes : 0), true}};
    credit_status_t st = check(t, n, clip, more, 2);
    if (st != CREDIT_OK) return st;
    int dev;
    if (cudaGetDevice(&dev) != cudaSuccess) { cudaGetLastError(); return CREDIT_ERR_CUDA; }
    const DevInfo* d = device_info(dev);
    if (!d) return CREDIT_ERR_CUDA;
    std::vector<Batch> batches;
    if (!batches_of(t, n, d->sms, &batches)) return CREDIT_ERR_INVALID_ARG;
    int64_t nparts = 0;
    bool in_place = true;
    for (const Batch& b : batches) nparts += b.grid;
    for (int64_t i = 0; clip && i < n; ++i)
        if (t[i].count && t[i].data != t[i].out) in_place = false;
    if (nparts > INT_MAX) return CREDIT_ERR_INVALID_ARG;
    if (nparts && (!workspace || workspace_bytes < (uint64_t)nparts * 8 || w % 16))
        return CREDIT_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    double* const parts = static_cast<double*>(workspace);
    // chunks of a CTA that stay in L2 until they are scaled
    const int keep = clip ? (int)((int64_t)d->l2_bytes / kKeepDen * kKeepNum /
                                  ((int64_t)kChunkBytes * d->sms * kCtasPerSm))
                          : 0;
    int64_t at = 0;
    for (const Batch& b : batches) {
        if ((st = from_cuda(launch_any(t, b, parts + at, 0, false, 0, 0, nullptr, false, keep, s))) !=
            CREDIT_OK)
            return st;
        at += b.grid;
    }
    if (!clip || batches.empty()) {
        return from_cuda(launch_early(grad_norm, dim3(1), kThreads, s, (const double*)parts, (int)nparts,
                                      norm));
    }
    for (size_t i = batches.size(); i-- > 0;) {
        st = from_cuda(launch_any(t, batches[i], parts, (int)nparts, true, max_norm, eps,
                                  i ? nullptr : norm, in_place, 0, s));
        if (st != CREDIT_OK) return st;
    }
    return CREDIT_OK;
} catch (...) {  // (out of host memory)
    return CREDIT_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

credit_status_t credit_grad_workspace(const credit_tensor_t* tensors, int64_t n, int device,
                                      size_t* bytes) try {
    if (!bytes || n < 0 || (n && !tensors)) return CREDIT_ERR_INVALID_ARG;
    const credit_status_t st = check(tensors, n, false, nullptr, 0);
    if (st != CREDIT_OK) return st;
    const DevInfo* d = device_info(device);
    if (!d) return CREDIT_ERR_CUDA;
    std::vector<Batch> batches;
    if (!batches_of(tensors, n, d->sms, &batches)) return CREDIT_ERR_INVALID_ARG;
    size_t parts = 0;
    for (const Batch& b : batches) parts += (size_t)b.grid;
    *bytes = parts * 8;
    return CREDIT_OK;
} catch (...) {
    return CREDIT_ERR_INVALID_ARG;
}

credit_status_t credit_grad_norm(const credit_tensor_t* tensors, int64_t n, float* norm,
                                 void* workspace, size_t workspace_bytes, void* stream) {
    return run(tensors, n, false, 0.f, 0.f, norm, workspace, workspace_bytes, stream);
}

credit_status_t credit_grad_clip(const credit_tensor_t* tensors, int64_t n, float max_norm, float eps,
                                 float* norm, void* workspace, size_t workspace_bytes, void* stream) {
    if (!(max_norm >= 0.f) || !(eps >= 0.f)) return CREDIT_ERR_INVALID_ARG;
    return run(tensors, n, true, max_norm, eps, norm, workspace, workspace_bytes, stream);
}

}  // extern "C"
