// ring_plan.h -- launch shapes of the ring kernels (ring.cuh).
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace credit {

constexpr int kRingStages = 12;   // most stages
constexpr int kRingWarps = 16;    // most warps of a CTA
constexpr int kRingThreads = 32 * kRingWarps;

struct RingShape {
    int32_t tiles;      // warp tiles of a CTA's slice
    int32_t stages;
    int32_t room;       // bytes of one stream's slice in a stage
    int32_t clusters;   // of the grid
    unsigned* err;
};

struct RingPlan {
    int V, W, P, R;     // tiles per warp, warps per CTA, CTAs per row, rows per turn
    int most;           // most clusters of the grid
    size_t smem;
    RingShape shape;    // `clusters` and `err` are set by the launch
};

// The instantiations a plan may choose: one and two rows of four tiles a warp,
// one row of eight.
struct RingKernels {
    const void* v4;
    const void* v4r2;
    const void* v8;
    const void* of(const RingPlan& p) const { return p.V == 8 ? v8 : p.R == 2 ? v4r2 : v4; }
};

// The shape for rows of `tiles` warp tiles in `streams` streams of `es`-byte
// elements; `turn`: most rows per turn (2: the forward kernel; 1: the backward
// kernel, which holds two turns' stages at once).  False where the rows are
// too wide (ring_fits, which needs no device) or on a CUDA error.  Also the
// clusters the device holds at once and its error word.
bool plan_ring(int tiles, int es, int streams, int turn, int64_t rows, int sms,
               const RingKernels& fn, RingPlan* out, int* resident, unsigned** err);
bool ring_fits(int tiles, int es, int streams, int turn, int64_t rows, int sms);

// Most clusters of a grid in this shape; and over every shape the backward
// kernel may be given (the row groups a workspace has room for).
int ring_most(const RingPlan& p, int sms);
int64_t ring_groups_bound(int tiles, int es, int streams, int64_t rows, int sms);

// The clusters of a launch: as many as are resident, no more than rows or
// plan.most, evened out so that none has a row more than it must.
int ring_grid(const RingPlan& p, int resident, int64_t rows);

cudaError_t launch_ring_args(const void* fn, void** args, const RingPlan& p, int clusters,
                             cudaStream_t s);

// `clusters` CTA clusters of a ring kernel with arguments (Args, RingShape).
template <typename Args>
cudaError_t launch_ring(const void* fn, Args a, const RingPlan& p, int clusters, unsigned* err,
                        cudaStream_t s) {
    RingShape q = p.shape;
    q.clusters = clusters;
    q.err = err;
    void* args[] = {&a, &q};
    return launch_ring_args(fn, args, p, clusters, s);
}

constexpr int kTeamWarps = 11;    // most summing (and as many writing) warps of a team's CTA

// A team launch (team.cuh).
struct TeamPlan {
    int tiles, stages, room, size, teams, W;
    size_t smem;
    int64_t exchange_bytes;  // of the words, which the launch clears
};

// The team shape for rows of `tiles` tiles in `streams` streams; false where a
// slice does not fit.  Host only: one CTA per SM.
bool plan_team(int tiles, int es, int streams, int64_t rows, int sms, TeamPlan* out);

// Clears the words and launches `fn` of (Args, TeamShape).
cudaError_t launch_team_args(const void* fn, void** args, const TeamPlan& p, void* words,
                             cudaStream_t s);

}  // namespace credit
