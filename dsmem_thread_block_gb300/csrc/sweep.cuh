// sweep.cuh -- rows too wide for the ring kernels (ring.cuh): two passes over
// batches of rows that stay in L2.  Launch i reads batch i from HBM for its
// row sums and, at the same time, reads batch i - 1 a second time, from L2,
// and writes its outputs; so each element is read from HBM once and no launch
// waits on one kind of traffic.  A block of either pass owns a strip of
// columns, whose parameters stay in registers, of a group of rows.
//
// Measured on rows that the team kernels (team.cuh) take: 256 x 786432 bf16,
// RMSNorm backward, 376 us against a team's 226 us; so only rows that no team
// holds come here (above 856064 columns, 44 tiles for each of 152 CTAs).
// Bound by the latency of a block's first loads: two rows in flight, eight a
// block and four blocks an SM measured best of nine settings (349 to 581 us).
#pragma once

#include "train.cuh"

namespace credit {

constexpr int kSweepThreads = 256;
constexpr int kSweepWarps = kSweepThreads / 32;
constexpr int kSweepTiles = 2;   // warp tiles a warp sums of a row
constexpr int kSweepRows = 2;    // rows it has in flight
constexpr int kSweepGroup = 8;   // rows of one block
constexpr int kSweepCtas = 4;    // blocks an SM holds

struct Sweep {
    int64_t s0, s1;     // rows whose sums this launch forms
    int64_t b0, b1;     // rows whose outputs it writes
    uint32_t sums;      // blocks of the first kind
    uint32_t outs;      // and of the second
    int32_t first;      // the first batch writes the parameters' sums, later ones add
};

// Columns of a summing block and of a writing block, for N elements a lane.
__host__ __device__ constexpr int sweep_chunk(int n) { return kSweepWarps * kSweepTiles * 32 * n; }
__host__ __device__ constexpr int sweep_strip(int n) { return kSweepWarps * 32 * n; }

// The kinds alternate while both last: which one is block b, and its index.
__device__ __forceinline__ bool sweep_sums(const Sweep& q, uint32_t b, uint32_t* index) {
    const uint32_t both = 2 * min(q.sums, q.outs);
    if (b < both) {
        *index = b >> 1;
        return !(b & 1);
    }
    *index = both / 2 + (b - both);
    return q.sums > q.outs;
}

// Programmatic dependent launch: the next launch's blocks may be scheduled as
// this one's finish, and wait here until all of its writes are visible.
__device__ __forceinline__ void wait_for_previous_launch() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Sums over the warp of K values (a power of two up to 32): value v ends in
// the lanes of group v (32 / K lanes each).  Lanes halve the values they carry
// while more than one is left, then add over their group.
template <int K> __device__ __forceinline__ float sums_over_warp(float (&v)[K], int lane) {
    int o = 16;
#pragma unroll
    for (int n = K; n > 1; n >>= 1, o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float keep = up ? v[i + n / 2] : v[i], give = up ? v[i] : v[i + n / 2];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    for (; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    return v[0];
}

// Rows of a batch: its inputs take half of the L2; a whole number of row groups.
inline int64_t sweep_batch(int64_t rows, int64_t row_bytes, int l2_bytes) {
    const int64_t r = (int64_t)l2_bytes / 2 / row_bytes / kSweepGroup * kSweepGroup;
    return r < kSweepGroup ? kSweepGroup : r;
}

// Launch `fn` of (args, sweep); `after`: it may be scheduled early behind the
// launch before it.
template <typename Args>
cudaError_t launch_sweep(const void* fn, Args a, Sweep q, uint32_t blocks, bool after,
                         cudaStream_t s) {
    void* args[] = {&a, &q};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kSweepThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = after ? 1 : 0;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

// All launches of a call: batch i's sums with batch i - 1's outputs.
template <typename Args>
cudaError_t run_sweep(const void* fn, const Args& a, int64_t batch, int n, cudaStream_t s) {
    const int64_t chunks = (a.cols + sweep_chunk(n) - 1) / sweep_chunk(n);
    const int64_t strips = (a.cols + sweep_strip(n) - 1) / sweep_strip(n);
    for (int64_t r = 0; r < a.rows + batch; r += batch) {
        Sweep q{};
        q.s0 = r < a.rows ? r : a.rows;
        q.s1 = r + batch < a.rows ? r + batch : a.rows;
        q.b0 = r - batch > 0 ? r - batch : 0;
        q.b1 = r < a.rows ? r : a.rows;
        if (r == 0) q.b1 = 0;
        q.first = r == batch;
        q.sums = (uint32_t)((q.s1 - q.s0 + kSweepGroup - 1) / kSweepGroup * chunks);
        q.outs = (uint32_t)((q.b1 - q.b0 + kSweepGroup - 1) / kSweepGroup * strips);
        const cudaError_t e = launch_sweep(fn, a, q, q.sums + q.outs, r > 0, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace credit
