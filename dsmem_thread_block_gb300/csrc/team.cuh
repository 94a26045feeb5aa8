// team.cuh -- rows wider than a cluster holds well: a team of T CTAs (one per
// SM, the whole grid resident in a cooperative launch) owns a row, each CTA a
// slice of its columns.  As in ring.cuh bulk copies bring the next rows' slices
// into a ring of stages, but the team exchanges through L2, so a row's outputs
// are written `lag` rows after its sums were formed: the exchange has that
// long, the slices stay in shared memory meanwhile, and every element is read
// from HBM once.  Teams are not bound to a GPC, so 19, 38, 76 or 152 CTAs use
// all 152 SMs where clusters of 16 leave 40 of them empty.
//
// A CTA's first W warps sum rows and the next W write them; one warp collects
// the team's parts and one feeds: it deposits the CTA's part of a row and
// issues the copies.  One barrier a row orders all of it, iteration j:
//     sum row j  |  write row j - lag  |  collect row j + 1 - lag  |
//     ------------------------------ barrier ------------------------------
//                                                | deposit row j, refill the
//                                                | stage of row j - lag
// Measured on 256 rows of 786432 bf16 columns, RMSNorm backward: warps that do
// both kinds of work and one service warp 366 us, the kinds apart 314 us.
#pragma once

#include "planner.h"
#include "ring.cuh"

namespace credit {

constexpr int kTeamSlots = 16;   // rows whose parts are held: at least twice the lag
constexpr int kTeamLag = 5;      // most rows between a row's sums and its outputs
constexpr int kTeamMost = 160;   // most CTAs of a team
constexpr int kTeamParts = kTeamMost / 32;
constexpr int kTeamThreads = 32 * (2 * kTeamWarps + 2);

struct TeamShape {
    int32_t tiles;      // warp tiles of a CTA's slice
    int32_t stages;     // at least lag + 1
    int32_t room;       // bytes of one stream's slice in a stage
    int32_t size;       // CTAs of a team
    int32_t teams;
    int32_t lag;        // 2 .. kTeamLag
    unsigned long long* words;  // [team][slot][CTA][2], zero before the launch
    unsigned* err;
};

// A part is two words of (value, turn + 1): each word arrives whole, so a word
// that carries the turn carries its value, and no fence orders two words.  A
// slot is used again kTeamSlots turns later: a CTA that deposits turn k has
// collected turn k - lag, so every CTA has deposited that one and has written
// turn k - 2 lag; with 2 lag <= kTeamSlots nobody still reads the slot.
struct TeamExchange {
    unsigned long long* words;
    int size, rank, lane;
    unsigned* err;
    bool dead = false;  // a wait gave up: the next ones do not wait again

    __device__ TeamExchange(const TeamShape& q, int team, int r, int l)
        : words(q.words + (size_t)team * kTeamSlots * q.size * 2), size(q.size), rank(r), lane(l),
          err(q.err) {}
    __device__ unsigned long long* slot(uint32_t turn) const {
        return words + (size_t)(turn % kTeamSlots) * size * 2;
    }
    // lanes 0 and 1: the CTA's two values
    __device__ void deposit(uint32_t turn, float v) const {
        if (lane < 2) {
            const unsigned long long w =
                (unsigned long long)__float_as_uint(v) | ((unsigned long long)(turn + 1) << 32);
            asm volatile("st.relaxed.gpu.global.u64 [%0], %1;"
                         :: "l"(slot(turn) + 2 * rank + lane), "l"(w) : "memory");
        }
    }
    // Lane l holds the words of CTAs l, l + 32, ... of a turn.  `fetch` only
    // issues the loads, so that they travel while the warp works on another
    // turn; `collect` loads again until every word carries the turn.
    struct Words { unsigned long long w[kTeamParts][2]; };
    __device__ void fetch(uint32_t turn, Words& f) const {
        const unsigned long long* const p = slot(turn);
#pragma unroll
        for (int i = 0; i < kTeamParts; ++i) {
            const int c = lane + 32 * i;
            if (c < size) {
                asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(f.w[i][0]) : "l"(p + 2 * c));
                asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];"
                             : "=l"(f.w[i][1]) : "l"(p + 2 * c + 1));
            }
        }
    }
    __device__ bool arrived(uint32_t turn, const Words& f) const {
        bool all = true;
#pragma unroll
        for (int i = 0; i < kTeamParts; ++i)
            if (lane + 32 * i < size)
                all = all && (uint32_t)(f.w[i][0] >> 32) == turn + 1 &&
                      (uint32_t)(f.w[i][1] >> 32) == turn + 1;
        return __all_sync(0xffffffffu, all);
    }
    // After a fetch of this turn: the parts, zeros past the team.
    __device__ void collect(uint32_t turn, Words& f, float (&a)[kTeamParts],
                            float (&b)[kTeamParts]) {
        uint64_t t0 = 0;
        for (uint32_t tries = 0; !arrived(turn, f) && !dead; ++tries) {
            fetch(turn, f);
            const uint64_t now = globaltimer_ns();
            if (tries == 0) t0 = now;
            if (__any_sync(0xffffffffu, now - t0 > kWaitLimitNs)) {
                if (lane == 0) atomicOr(err, kErrTimeout);
                dead = true;
            }
        }
#pragma unroll
        for (int i = 0; i < kTeamParts; ++i) {
            const bool in = lane + 32 * i < size;
            a[i] = in ? __uint_as_float((uint32_t)f.w[i][0]) : 0.f;
            b[i] = in ? __uint_as_float((uint32_t)f.w[i][1]) : 0.f;
        }
    }
    // The collecting warp's loop: done(j, turn, parts...) for each turn, in the
    // iteration before its row is written, then the barrier of every iteration.
    template <typename F> __device__ void collect_all(int turns, int lag, F done) {
        Words now = {}, then = {};
        for (int j = 0; j < turns + lag; ++j) {
            // at most turn j - 1, deposited before this iteration; the one after
            // it is fetched now where it has been on its way for an iteration
            const int due = j + 1 - lag;
            if (due + 1 >= 0 && due + 1 < turns && lag > 3) fetch((uint32_t)(due + 1), then);
            if (due >= 0 && due < turns) {
                float x[kTeamParts], y[kTeamParts];
                collect((uint32_t)due, now, x, y);
                done(j, due, x, y);
            }
            now = then;
            __syncthreads();
        }
    }
};

// Clears the exchange's words (the start of the call's workspace) and launches.
template <typename Args>
cudaError_t launch_team(const void* fn, Args a, const TeamPlan& p, void* words, cudaStream_t s) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    unsigned* err = device_error_word();
    if (!err || !kernel_info(dev, fn, false)) return cudaErrorInvalidConfiguration;
    TeamShape q{p.tiles, p.stages, p.room, p.size, p.teams, p.lag,
                static_cast<unsigned long long*>(words), err};
    void* args[] = {&a, &q};
    return launch_team_args(fn, args, p, words, s);
}

}  // namespace credit
