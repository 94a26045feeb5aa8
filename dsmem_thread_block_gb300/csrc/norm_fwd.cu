// norm_fwd.cu -- h = residual + dropout(x), y = norm(h) and the row statistics
// (mean, 1/sqrt(var + eps)) that the backward pass needs.
//
// General form, rows of any width: one kernel writes a partial (count, mean,
// M2 about that mean) per row and chunk of 32 warp tiles, the next merges a
// row's partials (the parallel-axis form of Chan et al.'s merge) and writes.
// Two reads of x and residual, the second from L2 where they fit it.
#include "train.cuh"

namespace credit {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTilesPerWarp = 4;
constexpr int kChunkTiles = kWarps * kTilesPerWarp;

// Merge a row's nch partials; every lane of the calling warp returns the same.
template <int OP>
__device__ __forceinline__ NormPart merge_row(const float* ws, int nch, int lane) {
    NormPart r{0.f, 0.f, 0.f};
    if constexpr (OP == kLayerNorm) {
        float n = 0.f, nm = 0.f;
        for (int c = lane; c < nch; c += 32) {
            n += ws[4 * c];
            nm = fmaf(ws[4 * c], ws[4 * c + 1], nm);
        }
        n = warp_allreduce(n, SumOp());
        nm = warp_allreduce(nm, SumOp());
        r.n = n;
        r.mu = nm / n;
        for (int c = lane; c < nch; c += 32) {
            const float d = ws[4 * c + 1] - r.mu;
            r.m2 += fmaf(ws[4 * c] * d, d, ws[4 * c + 2]);
        }
    } else {
        for (int c = lane; c < nch; c += 32) r.m2 += ws[4 * c + 2];
    }
    r.m2 = warp_allreduce(r.m2, SumOp());
    return r;
}

template <int OP, typename T, typename IO>
__global__ void __launch_bounds__(kThreads) fwd_stats(NormFwdArgs a) {
    __shared__ float red[2][kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const DropStream d(a.drop);
    const int64_t items = a.rows * a.nch;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t row = it / a.nch;
        const int64_t c0 = (it - row * a.nch) * (int64_t)(kChunkTiles * IO::kTile);
        const T* x = static_cast<const T*>(a.x) + row * a.cols;
        const T* r = a.residual ? static_cast<const T*>(a.residual) + row * a.cols : nullptr;
        float h[kTilesPerWarp][IO::N];
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kTilesPerWarp; ++i) {
            const int64_t base = c0 + (int64_t)(warp + kWarps * i) * IO::kTile;
            if (base < a.cols) {
                tile_h<T, IO>(x, r, a.drop.on, d, base, lane, (uint32_t)row, a.cols, h[i]);
            } else {
#pragma unroll
                for (int k = 0; k < IO::N; ++k) h[i][k] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < IO::N; ++k) s += OP == kLayerNorm ? h[i][k] : h[i][k] * h[i][k];
        }
        s = block_allreduce(s, red[0], SumOp(), 0.f);
        const float n = (float)min(a.cols - c0, (int64_t)(kChunkTiles * IO::kTile));
        float mu = 0.f, m2 = s;
        if constexpr (OP == kLayerNorm) {
            mu = s / n;
            m2 = 0.f;
#pragma unroll
            for (int i = 0; i < kTilesPerWarp; ++i) {
                const int64_t base = c0 + (int64_t)(warp + kWarps * i) * IO::kTile;
#pragma unroll
                for (int k = 0; k < IO::N; ++k) {
                    const float e = IO::valid(base, lane, k, a.cols) ? h[i][k] - mu : 0.f;
                    m2 = fmaf(e, e, m2);
                }
            }
            m2 = block_allreduce(m2, red[1], SumOp(), 0.f);
        } else {
            __syncthreads();  // red[0] is rewritten by the next item
        }
        if (threadIdx.x == 0) {
            float* w = a.ws + it * 4;
            w[0] = n;
            w[1] = mu;
            w[2] = m2;
        }
    }
}

template <int OP, typename T, typename IO, typename PT>
__global__ void __launch_bounds__(kThreads) fwd_apply(NormFwdArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const DropStream d(a.drop);
    const PT* gp = static_cast<const PT*>(a.gamma);
    const PT* bp = static_cast<const PT*>(a.beta);
    const int64_t items = a.rows * a.nch;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t row = it / a.nch;
        const int64_t c0 = (it - row * a.nch) * (int64_t)(kChunkTiles * IO::kTile);
        const NormPart st = merge_row<OP>(a.ws + row * a.nch * 4, a.nch, lane);
        const float rstd = 1.f / sqrtf(st.m2 / (float)a.cols + a.eps);
        if (c0 == 0 && threadIdx.x == 0) {
            if (a.mean) a.mean[row] = st.mu;
            if (a.rstd) a.rstd[row] = rstd;
        }
        const T* x = static_cast<const T*>(a.x) + row * a.cols;
        const T* r = a.residual ? static_cast<const T*>(a.residual) + row * a.cols : nullptr;
        T* y = static_cast<T*>(a.y) + row * a.cols;
        T* ho = a.h ? static_cast<T*>(a.h) + row * a.cols : nullptr;
#pragma unroll
        for (int i = 0; i < kTilesPerWarp; ++i) {
            const int64_t base = c0 + (int64_t)(warp + kWarps * i) * IO::kTile;
            if (base >= a.cols) break;
            float h[IO::N], g[IO::N], b[IO::N];
            tile_h<T, IO>(x, r, a.drop.on, d, base, lane, (uint32_t)row, a.cols, h);
            if (ho) IO::store(ho, base, lane, a.cols, Elem<T>::pack(h));
            IO::template params<PT>(gp, base, lane, a.cols, g, 1.f);
            IO::template params<PT>(bp, base, lane, a.cols, b, 0.f);
#pragma unroll
            for (int k = 0; k < IO::N; ++k) {
                const float z = OP == kLayerNorm ? (h[k] - st.mu) * rstd : h[k] * rstd;
                h[k] = fmaf(z, g[k], b[k]);
            }
            IO::store(y, base, lane, a.cols, Elem<T>::pack(h));
        }
    }
}

template <int OP, typename T, typename IO>
cudaError_t run_fwd(TrainKey k, const NormFwdArgs& a, int sms, cudaStream_t s) {
    const int64_t items = a.rows * a.nch;
    const unsigned grid = (unsigned)(items < (int64_t)sms * 32 ? items : (int64_t)sms * 32);
    fwd_stats<OP, T, IO><<<grid, kThreads, 0, s>>>(a);
    if (k.pdtype == 0) fwd_apply<OP, T, IO, float><<<grid, kThreads, 0, s>>>(a);
    else fwd_apply<OP, T, IO, bf16><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <int OP, typename T>
cudaError_t pick_fwd(TrainKey k, const NormFwdArgs& a, int sms, cudaStream_t s) {
    return k.vec ? run_fwd<OP, T, VecIO<T>>(k, a, sms, s) : run_fwd<OP, T, ElemIO<T>>(k, a, sms, s);
}

}  // namespace

int train_chunks(int dtype, int64_t cols) {
    const int64_t chunk = (int64_t)kChunkTiles * (dtype == 0 ? VecIO<float>::kTile : VecIO<bf16>::kTile);
    return (int)((cols + chunk - 1) / chunk);
}

cudaError_t launch_norm_fwd(TrainKey k, const NormFwdArgs& a, int sms, cudaStream_t s) {
    if (k.op == kLayerNorm)
        return k.dtype == 0 ? pick_fwd<kLayerNorm, float>(k, a, sms, s)
                            : pick_fwd<kLayerNorm, bf16>(k, a, sms, s);
    return k.dtype == 0 ? pick_fwd<kRMSNorm, float>(k, a, sms, s)
                        : pick_fwd<kRMSNorm, bf16>(k, a, sms, s);
}

}  // namespace credit
