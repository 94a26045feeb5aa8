// ring_plan.cu -- launch shapes of the ring kernels (ring.cuh).
#include "ring_plan.h"

#include <algorithm>
#include <map>
#include <mutex>
#include <tuple>

#include "common.cuh"
#include "planner.h"

namespace credit {

namespace {

constexpr int kTileCols = 128;          // 32 lanes of four columns
constexpr int kMostStage = 220 * 1024;  // shared memory a CTA may spend on its ring

}  // namespace

bool plan_ring(int tiles, int es, int streams, int64_t rows, int sms, RingPlan* out) {
    RingPlan p{};
    if (tiles <= 4 * kRingWarps) {
        p.V = 4;
        p.P = 1;
    } else {
        p.V = 8;
        p.P = (tiles + 8 * kRingWarps - 1) / (8 * kRingWarps);
    }
    if (p.P > kMaxCluster) return false;
    p.shape.tiles = (tiles + p.P - 1) / p.P;
    p.P = (tiles + p.shape.tiles - 1) / p.shape.tiles;  // no CTA without columns
    p.W = (p.shape.tiles + p.V - 1) / p.V;
    // a slice that starts inside a 16-byte line takes one line more
    p.shape.room = (p.shape.tiles * kTileCols * es + 16 + 127) / 128 * 128;
    const int stage = p.shape.room * streams;
    int ctas = std::max(1, std::min(8, 1024 / (32 * p.W)));  // per SM
    const int budget = (p.P == 1 ? 144 : 200) * 1024;
    while (ctas > 1 && budget / ctas < 2 * stage) --ctas;
    int stages = budget / ctas / stage;
    if (stages < 2) stages = kMostStage / stage;
    if (stages < 1) return false;
    p.most = (int)std::max<int64_t>(1, (int64_t)sms * std::max(1, std::min(8, 1024 / (32 * p.W))) / p.P);
    if (rows * p.P * 2 <= sms) stages = 1;  // every cluster has one row
    p.shape.stages = std::min(stages, kRingStages);
    p.smem = (size_t)p.shape.stages * stage;
    *out = p;
    return true;
}

int ring_clusters(int dev, const void* fn, const RingPlan& p, int64_t rows) {
    static std::mutex mu;
    static std::map<std::tuple<int, const void*, int, int, size_t>, int> resident;
    const auto key = std::make_tuple(dev, fn, p.W, p.P, p.smem);
    int most = 0;
    {
        std::lock_guard<std::mutex> lk(mu);
        const auto it = resident.find(key);
        if (it != resident.end()) most = it->second;
    }
    if (most == 0) {
        if (!kernel_info(dev, fn, true)) return 0;
        most = occupancy_clusters(dev, fn, p.P, 32 * p.W, p.smem, 1 << 20);
        if (most < 1) return 0;
        std::lock_guard<std::mutex> lk(mu);
        if (resident.size() >= 4096) resident.clear();
        resident[key] = most;
    }
    const int64_t c = std::min<int64_t>(std::min(most, p.most), rows);
    const int64_t turns = (rows + c - 1) / c;
    return (int)((rows + turns - 1) / turns);
}

cudaError_t launch_ring_args(const void* fn, void** args, const RingPlan& p, int clusters,
                             cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * p.P));
    cfg.blockDim = dim3((unsigned)(32 * p.W));
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
