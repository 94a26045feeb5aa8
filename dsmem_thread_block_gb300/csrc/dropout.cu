// dropout.cu -- y = residual + keep ? x / (1 - p) : 0, the mask drawn on the
// way (train.cuh) and never stored.  The same call on the incoming gradient
// is the backward pass.
//
// Measured: 16384 x 8192 bf16 with residual 135 us, 0.88 of the copy rate;
// 64 x 4096 1.9 us.  Bound by HBM: a mask costs nine instructions an element
// (36 for a block of four) of the 22 that the SMs issue in an element's time.
// Two tiles of 16 bytes a lane in flight; one measured 147 us.
#include "train.cuh"

namespace credit {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;  // tiles a warp has in flight

// Warp tiles of all rows in order, U at a time: a warp steps by the number
// of warps in the grid, its (row, tile) kept by addition, and has the loads of
// U tiles in flight before it draws their masks.
template <typename T, typename IO, int U>
__global__ void __launch_bounds__(kThreads) dropout_tiles(DropoutArgs a) {
    const int lane = threadIdx.x & 31;
    const DropStream d(a.drop);
    const int cols = (int)a.cols, tpr = (cols + IO::kTile - 1) / IO::kTile;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t drow = warps / tpr;
    const int dtile = (int)(warps - drow * tpr);
    const T* x = static_cast<const T*>(a.x);
    const T* r = static_cast<const T*>(a.residual);
    int64_t row = w / tpr;
    int tile = (int)(w - row * tpr);
    while (row < a.rows) {
        int64_t rows[U];
        int tiles[U];
        typename IO::R xv[U], rv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            rows[u] = row;
            tiles[u] = tile;
            if (row < a.rows) {
                const int j = tile * IO::kTile + IO::first(lane);
                const int64_t o = row * a.cols + j;
                xv[u] = IO::template load<false>(x + o, 0, cols - j);
                if (r) rv[u] = IO::template load<false>(r + o, 0, cols - j);
            }
            row += drow;
            tile += dtile;
            if (tile >= tpr) {
                tile -= tpr;
                ++row;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (rows[u] >= a.rows) break;
            F2 h[IO::NP];
            tile_h<T, IO>(xv[u], rv[u], r != nullptr, a.drop.on, d, tiles[u] * IO::kTile, lane,
                          (uint32_t)rows[u], h);
            const int j = tiles[u] * IO::kTile + IO::first(lane);
            IO::template store<false>(static_cast<T*>(a.y) + rows[u] * a.cols + j, 0, cols - j, h);
        }
    }
}

template <typename T, typename IO>
cudaError_t run(const DropoutArgs& a, int sms, cudaStream_t s) {
    const int64_t tiles = a.rows * ((a.cols + IO::kTile - 1) / IO::kTile);
    const int64_t want = (tiles + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t most = (int64_t)sms * 8;
    dropout_tiles<T, IO, kUnroll><<<(unsigned)(want < most ? want : most), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dropout(int dtype, bool vec, const DropoutArgs& a, int sms, cudaStream_t s) {
    if (dtype == 0)
        return vec ? run<float, VecIO<float, 4>>(a, sms, s)
                   : run<float, ElemIO<float, 4>>(a, sms, s);
    return vec ? run<bf16, VecIO<bf16, 8>>(a, sms, s) : run<bf16, ElemIO<bf16, 8>>(a, sms, s);
}

}  // namespace credit
