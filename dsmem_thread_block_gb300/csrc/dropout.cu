// dropout.cu -- y = residual + keep ? x / (1 - p) : 0, the mask drawn on the
// way (train.cuh) and never stored.  The same call on the incoming gradient
// is the backward pass.
#include "train.cuh"

namespace credit {

namespace {

constexpr int kThreads = 256;

// Warp tiles of all rows in order: a warp steps from tile to tile by the
// number of warps in the grid, its (row, tile) kept by addition.
template <typename T, typename IO>
__global__ void __launch_bounds__(kThreads) dropout_tiles(DropoutArgs a) {
    const int lane = threadIdx.x & 31;
    const DropStream d(a.drop);
    const int64_t tpr = (a.cols + IO::kTile - 1) / IO::kTile;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t drow = warps / tpr, dtile = warps - drow * tpr;
    int64_t row = w / tpr, tile = w - row * tpr;
    while (row < a.rows) {
        const int64_t o = row * a.cols;
        float h[IO::N];
        tile_h<T, IO>(static_cast<const T*>(a.x) + o,
                      a.residual ? static_cast<const T*>(a.residual) + o : nullptr, a.drop.on, d,
                      tile * IO::kTile, lane, (uint32_t)row, a.cols, h);
        IO::store(static_cast<T*>(a.y) + o, tile * IO::kTile, lane, a.cols, Elem<T>::pack(h));
        row += drow;
        tile += dtile;
        if (tile >= tpr) {
            tile -= tpr;
            ++row;
        }
    }
}

template <typename T, typename IO>
cudaError_t run(const DropoutArgs& a, int sms, cudaStream_t s) {
    const int64_t tiles = a.rows * ((a.cols + IO::kTile - 1) / IO::kTile);
    const int64_t want = (tiles + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t most = (int64_t)sms * 8;
    dropout_tiles<T, IO><<<(unsigned)(want < most ? want : most), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dropout(int dtype, bool vec, const DropoutArgs& a, int sms, cudaStream_t s) {
    if (dtype == 0)
        return vec ? run<float, VecIO<float>>(a, sms, s) : run<float, ElemIO<float>>(a, sms, s);
    return vec ? run<bf16, VecIO<bf16>>(a, sms, s) : run<bf16, ElemIO<bf16>>(a, sms, s);
}

}  // namespace credit
