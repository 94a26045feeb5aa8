// ring_plan.cu -- launch shapes of the ring kernels (ring.cuh).
#include "ring_plan.h"

#include <algorithm>
#include <cstdlib>
#include <mutex>
#include <vector>

#include "common.cuh"
#include "planner.h"

namespace credit {

namespace {

constexpr int kTileCols = 128;          // 32 lanes of four columns
constexpr int kMostStage = 220 * 1024;  // shared memory a CTA may spend on its ring

}  // namespace

bool plan_ring(int tiles, int es, int streams, int turn, int64_t rows, int sms, RingPlan* out) {
    const int fewest = turn == 1 ? 2 : 1, want = turn == 1 ? 4 : 2;  // stages
    for (int least : {turn == 1 ? 3 : 1, fewest}) {
        for (int V : {4, 8}) {
            if (getenv("PV8") && V == 4) continue;
            for (int P = (tiles + V * kRingWarps - 1) / (V * kRingWarps); P <= kMaxCluster; ++P) {
                RingPlan p{};
                p.V = V;
                p.shape.tiles = (tiles + P - 1) / P;
                p.P = (tiles + p.shape.tiles - 1) / p.shape.tiles;  // no CTA without columns
                p.W = (p.shape.tiles + V - 1) / V;
                // a slice that starts inside a 16-byte line takes one line more
                p.shape.room = (p.shape.tiles * kTileCols * es + 16 + 127) / 128 * 128;
                const int ctas_most = std::max(1, std::min(8, 1024 / (32 * p.W)));  // per SM
                p.most = std::max(1, sms * ctas_most / p.P);
                p.R = turn == 2 && V == 4 && rows >= 2 * (int64_t)p.most ? 2 : 1;
                const int stage = p.shape.room * streams * p.R;
                const int budget = (getenv("BUD") ? atoi(getenv("BUD")) : turn == 1 ? 200 : 144) * 1024;
                int ctas = ctas_most;
                while (ctas > 1 && budget / ctas < want * stage) --ctas;
                int stages = budget / ctas / stage;
                if (stages < want) stages = std::min(want, kMostStage / stage);
                if (stages < least) continue;
                if (rows * p.P * 2 <= sms) stages = fewest;  // every cluster has one row
                p.shape.stages = std::min(stages, kRingStages);
                p.smem = (size_t)p.shape.stages * stage;
                *out = p;
                return true;
            }
        }
    }
    return false;
}

namespace {

// What a launch of (kernel, shape) needs from the device, looked up once.
struct Resident {
    const void* fn;
    int dev, W, P, clusters;
    size_t smem;
    unsigned* err;
};

}  // namespace

bool ring_resident(const void* fn, const RingPlan& p, int* clusters, unsigned** err) {
    static std::mutex mu;
    static std::vector<Resident> known;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    {
        std::lock_guard<std::mutex> lk(mu);
        for (const Resident& r : known)
            if (r.fn == fn && r.dev == dev && r.W == p.W && r.P == p.P && r.smem == p.smem) {
                *clusters = r.clusters;
                *err = r.err;
                return true;
            }
    }
    if (!kernel_info(dev, fn, true)) return false;
    Resident r{fn, dev, p.W, p.P, occupancy_clusters(dev, fn, p.P, 32 * p.W, p.smem, 1 << 20),
               p.smem, device_error_word()};
    if (r.clusters < 1 || !r.err) return false;
    std::lock_guard<std::mutex> lk(mu);
    if (known.size() >= 256) known.clear();  // shapes come and go
    known.push_back(r);
    *clusters = r.clusters;
    *err = r.err;
    return true;
}

int ring_grid(const RingPlan& p, int resident, int64_t rows) {
    const int64_t units = (rows + p.R - 1) / p.R;  // turns of all clusters
    const int64_t c = std::min<int64_t>(std::min(resident, p.most), units);
    const int64_t turns = (units + c - 1) / c;
    return (int)((units + turns - 1) / turns);
}

cudaError_t launch_ring_args(const void* fn, void** args, const RingPlan& p, int clusters,
                             cudaStream_t s) {
    const dim3 grid((unsigned)(clusters * p.P)), block((unsigned)(32 * p.W));
    if (p.P == 1) return cudaLaunchKernel(fn, grid, block, args, p.smem, s);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.P;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace credit
