// norm_bwd.cu -- the gradient of y = norm(h), h = residual + dropout(x):
// with xh = (h - mean) rstd and w = dy gamma (RMSNorm: mean = 0),
//   dtot   = rstd (w - mean_j(w) - xh mean_j(w xh)) + dh   (RMSNorm: no mean_j(w))
//   dres   = dtot,   dx = keep ? dtot / (1 - p) : 0
//   dgamma = sum_rows dy xh,   dbeta = sum_rows dy
//
// General form, rows of any width: one kernel writes the two row sums per
// row and chunk, the next owns a strip of columns of a group of rows, writes
// dx and sums the parameters' gradients over the group in registers, the last
// adds the groups.  Every sum has a fixed order: results repeat bit for bit.
#include "train.cuh"

namespace credit {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTilesPerWarp = 4;
constexpr int kChunkTiles = kWarps * kTilesPerWarp;
constexpr int kRowBlock = 32;  // rows whose sums a CTA merges at a time

template <int OP, typename T, typename IO, typename PT>
__global__ void __launch_bounds__(kThreads) bwd_stats(NormBwdArgs a) {
    __shared__ float red[2][2 * kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const PT* gp = static_cast<const PT*>(a.gamma);
    const int64_t items = a.rows * a.nch;
    int turn = 0;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x, turn ^= 1) {
        const int64_t row = it / a.nch;
        const int64_t c0 = (it - row * a.nch) * (int64_t)(kChunkTiles * IO::kTile);
        const T* dy = static_cast<const T*>(a.dy) + row * a.cols;
        const T* h = static_cast<const T*>(a.h) + row * a.cols;
        const float rstd = a.rstd[row], mean = OP == kLayerNorm ? a.mean[row] : 0.f;
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < kTilesPerWarp; ++i) {
            const int64_t base = c0 + (int64_t)(warp + kWarps * i) * IO::kTile;
            if (base < a.cols) {
                float u[IO::N], v[IO::N], g[IO::N];
                Elem<T>::unpack(IO::load(dy, base, lane, a.cols), u);
                Elem<T>::unpack(IO::load(h, base, lane, a.cols), v);
                IO::template params<PT>(gp, base, lane, a.cols, g, 1.f);
#pragma unroll
                for (int k = 0; k < IO::N; ++k) {
                    const float w = u[k] * g[k];  // 0 past the row
                    s1 = fmaf(w, (v[k] - mean) * rstd, s1);
                    s2 += w;
                }
            }
        }
        block_sum2(s1, s2, red[turn], kWarps, kThreads);
        if (threadIdx.x == 0) {
            a.ws[2 * it] = s1;
            a.ws[2 * it + 1] = s2;
        }
    }
}

template <int OP, typename T, typename IO, typename PT>
__global__ void __launch_bounds__(kThreads) bwd_apply(NormBwdArgs a) {
    __shared__ float4 rowc[kRowBlock];  // mean, rstd, mean_j(w xh), mean_j(w)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const DropStream d(a.drop);
    const int64_t base = ((int64_t)blockIdx.x * kWarps + warp) * IO::kTile;
    const bool mine = base < a.cols;
    float g[IO::N], ag[IO::N], ab[IO::N];
#pragma unroll
    for (int k = 0; k < IO::N; ++k) ag[k] = ab[k] = 0.f;
    if (mine) IO::template params<PT>(static_cast<const PT*>(a.gamma), base, lane, a.cols, g, 1.f);
    const int64_t r1 = min(a.rows, (int64_t)(blockIdx.y + 1) * a.group_rows);
    for (int64_t r0 = (int64_t)blockIdx.y * a.group_rows; r0 < r1; r0 += kRowBlock) {
        const int nr = (int)min((int64_t)kRowBlock, r1 - r0);
        __syncthreads();
        for (int i = warp; i < nr; i += kWarps) {
            const float* w = a.ws + (r0 + i) * a.nch * 2;
            float s1 = 0.f, s2 = 0.f;
            for (int c = lane; c < a.nch; c += 32) {
                s1 += w[2 * c];
                s2 += w[2 * c + 1];
            }
            s1 = warp_allreduce(s1, SumOp());
            s2 = warp_allreduce(s2, SumOp());
            if (lane == 0)
                rowc[i] = make_float4(OP == kLayerNorm ? a.mean[r0 + i] : 0.f, a.rstd[r0 + i],
                                      s1 / (float)a.cols,
                                      OP == kLayerNorm ? s2 / (float)a.cols : 0.f);
        }
        __syncthreads();
        if (!mine) continue;
#pragma unroll 2
        for (int i = 0; i < nr; ++i) {
            const int64_t o = (r0 + i) * a.cols;
            const float4 c = rowc[i];
            float u[IO::N], v[IO::N];
            Elem<T>::unpack(IO::load(static_cast<const T*>(a.dy) + o, base, lane, a.cols), u);
            Elem<T>::unpack(IO::load(static_cast<const T*>(a.h) + o, base, lane, a.cols), v);
#pragma unroll
            for (int k = 0; k < IO::N; ++k) {
                const float xh = (v[k] - c.x) * c.y;
                ag[k] = fmaf(u[k], xh, ag[k]);
                ab[k] += u[k];
                v[k] = (fmaf(-xh, c.z, u[k] * g[k]) - c.w) * c.y;
            }
            if (a.dh) {
                Elem<T>::unpack(IO::load(static_cast<const T*>(a.dh) + o, base, lane, a.cols), u);
#pragma unroll
                for (int k = 0; k < IO::N; ++k) v[k] += u[k];
            }
            if (a.dres) IO::store(static_cast<T*>(a.dres) + o, base, lane, a.cols, Elem<T>::pack(v));
            if (a.drop.on) {
                const uint32_t m = IO::keep(d, base, lane, (uint32_t)(r0 + i));
#pragma unroll
                for (int k = 0; k < IO::N; ++k) v[k] = (m >> k) & 1u ? v[k] * d.scale : 0.f;
            }
            IO::store(static_cast<T*>(a.dx) + o, base, lane, a.cols, Elem<T>::pack(v));
        }
    }
    if (mine) {
        float* p = a.pws + (int64_t)blockIdx.y * 2 * a.cols;
        if (a.dgamma) {
#pragma unroll
            for (int k = 0; k < IO::N; ++k)
                if (IO::valid(base, lane, k, a.cols)) p[IO::col(base, lane, k)] = ag[k];
        }
        if (a.dbeta) {
#pragma unroll
            for (int k = 0; k < IO::N; ++k)
                if (IO::valid(base, lane, k, a.cols)) p[a.cols + IO::col(base, lane, k)] = ab[k];
        }
    }
}

// dgamma and dbeta: the groups' sums added in group order.
template <typename PT>
__global__ void __launch_bounds__(kThreads) bwd_params(NormBwdArgs a) {
    for (int64_t j = (int64_t)blockIdx.x * kThreads + threadIdx.x; j < a.cols;
         j += (int64_t)gridDim.x * kThreads) {
        float sg = 0.f, sb = 0.f;
        for (int q = 0; q < a.groups; ++q) {
            const float* p = a.pws + (int64_t)q * 2 * a.cols;
            if (a.dgamma) sg += p[j];
            if (a.dbeta) sb += p[a.cols + j];
        }
        if (a.dgamma) static_cast<PT*>(a.dgamma)[j] = Elem<PT>::from_f(sg);
        if (a.dbeta) static_cast<PT*>(a.dbeta)[j] = Elem<PT>::from_f(sb);
    }
}

template <int OP, typename T, typename IO, typename PT>
cudaError_t run_bwd(const NormBwdArgs& a, int sms, cudaStream_t s) {
    if (a.rows > 0) {
        const int64_t items = a.rows * a.nch;
        const unsigned grid = (unsigned)(items < (int64_t)sms * 32 ? items : (int64_t)sms * 32);
        bwd_stats<OP, T, IO, PT><<<grid, kThreads, 0, s>>>(a);
        const int64_t strip = (int64_t)kWarps * IO::kTile;
        bwd_apply<OP, T, IO, PT><<<dim3((unsigned)((a.cols + strip - 1) / strip), (unsigned)a.groups),
                                   kThreads, 0, s>>>(a);
    }
    if (a.dgamma || a.dbeta) {
        const int64_t blocks = (a.cols + kThreads - 1) / kThreads;
        bwd_params<PT><<<(unsigned)(blocks < sms * 8 ? blocks : sms * 8), kThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

template <int OP, typename T>
cudaError_t pick_bwd(TrainKey k, const NormBwdArgs& a, int sms, cudaStream_t s) {
    if (k.vec)
        return k.pdtype == 0 ? run_bwd<OP, T, VecIO<T>, float>(a, sms, s)
                             : run_bwd<OP, T, VecIO<T>, bf16>(a, sms, s);
    return k.pdtype == 0 ? run_bwd<OP, T, ElemIO<T>, float>(a, sms, s)
                         : run_bwd<OP, T, ElemIO<T>, bf16>(a, sms, s);
}

}  // namespace

int train_groups(int dtype, int64_t rows, int64_t cols, int sms, int64_t* group_rows) {
    const int64_t strip = (int64_t)kWarps * (dtype == 0 ? VecIO<float>::kTile : VecIO<bf16>::kTile);
    const int64_t strips = (cols + strip - 1) / strip;
    int64_t g = (4 * (int64_t)sms + strips - 1) / strips;
    g = g < (rows + 7) / 8 ? g : (rows + 7) / 8;
    if (g < 1) g = 1;
    *group_rows = (rows + g - 1) / g;
    if (*group_rows < 1) *group_rows = 1;
    return (int)((rows + *group_rows - 1) / *group_rows);
}

cudaError_t launch_norm_bwd(TrainKey k, const NormBwdArgs& a, int sms, cudaStream_t s) {
    if (k.op == kLayerNorm)
        return k.dtype == 0 ? pick_bwd<kLayerNorm, float>(k, a, sms, s)
                            : pick_bwd<kLayerNorm, bf16>(k, a, sms, s);
    return k.dtype == 0 ? pick_bwd<kRMSNorm, float>(k, a, sms, s)
                        : pick_bwd<kRMSNorm, bf16>(k, a, sms, s);
}

}  // namespace credit
