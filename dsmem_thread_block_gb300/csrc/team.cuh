// team.cuh -- rows wider than a cluster holds well: a team of T CTAs (one per
// SM, the whole grid resident in a cooperative launch) owns a row, each CTA a
// slice of its columns.  As in ring.cuh bulk copies bring the next rows' slices
// into a ring of stages, but the team exchanges through L2, so a row's outputs
// are written some rows after its sums were formed: its slice stays in shared
// memory meanwhile, and every element is read from HBM once.  Teams are not
// bound to a GPC, so 19, 38, 76 or 152 CTAs use all 152 SMs where clusters of
// 16 leave 40 of them empty.
//
// A CTA's warps pass each row (turn) on through mbarriers, one of each kind a
// stage:
//     fed      the serving warp issues the copies of a turn into a free stage
//     summed   W warps sum it, a part each; the serving warp merges the parts
//              and deposits the CTA's in L2
//     known    the collecting warp merges the team's parts: the row's statistics
//     written  W warps write the row's outputs; the stage is free
// No barrier joins them, so each kind runs as far ahead as the stages allow and
// the exchange's latency falls on no one: with one barrier a row for all of
// them the GPU took @ us for 256 rows of 786432 bf16 columns (RMSNorm
// backward), now @.
#pragma once

#include "planner.h"
#include "ring.cuh"

namespace credit {

constexpr int kTeamStages = 16;  // most stages
constexpr int kTeamSlots = 32;   // turns whose parts are held
constexpr int kTeamMost = 160;   // most CTAs of a team
constexpr int kTeamParts = kTeamMost / 32;
constexpr int kTeamThreads = 32 * (2 * kTeamWarps + 2);
static_assert(kTeamSlots >= 2 * kTeamStages, "a slot is read until two rings of turns later");

struct TeamShape {
    int32_t tiles;      // warp tiles of a CTA's slice
    int32_t stages;     // at most kTeamStages
    int32_t room;       // bytes of one stream's slice in a stage
    int32_t size;       // CTAs of a team
    int32_t teams;
    unsigned long long* words;  // [team][slot][CTA][2], zero before the launch
    unsigned* err;
};

// Where a warp stands in the ring: turns 0, 1, ... take the stages in order.
struct TeamTurn {
    int s = 0;
    uint32_t phase = 0;
    __device__ void next(int stages) {
        if (++s == stages) {
            s = 0;
            phase ^= 1u;
        }
    }
};

// The mbarriers of a CTA's stages.  None can be lapped: turn k + stages is fed
// after turn k was written by every writing warp, that after it was known, that
// after it was deposited (every CTA of the team deposits first), and that after
// it was summed; so values a stage's warps pass in shared memory (their parts,
// the row's statistics) stand until they have been read.
struct TeamBars {
    uint64_t fed[kTeamStages], summed[kTeamStages], known[kTeamStages], written[kTeamStages];
    // All threads call.
    __device__ void init(int stages, int W) {
        if (threadIdx.x == 0) {
            for (int s = 0; s < stages; ++s) {
                mbar_init(smem_u32(&fed[s]), 1);
                mbar_init(smem_u32(&summed[s]), (uint32_t)W);
                mbar_init(smem_u32(&known[s]), 1);
                mbar_init(smem_u32(&written[s]), (uint32_t)W);
            }
            fence_mbar_init();
            fence_proxy_async_smem();
        }
        __syncthreads();
    }
    __device__ static void wait(uint64_t& bar, const TeamTurn& t, unsigned* err) {
        mbar_wait_bounded(smem_u32(&bar), t.phase, err);
    }
    // Whether the turn of a stage is complete, for every lane of the warp.
    __device__ static bool ready(uint64_t& bar, const TeamTurn& t) {
        return __all_sync(0xffffffffu, mbar_test_wait(smem_u32(&bar), t.phase));
    }
    // The serving warp: feed(turn, stage) whenever a stage is free, deposit(turn,
    // stage) whenever one is summed.  (One warp for both: a 25th would leave the
    // others 72 registers instead of 80.)
    template <typename F, typename D>
    __device__ void serve(int turns, int stages, unsigned* err, F feed, D deposit) {
        int fed = 0, given = 0;
        for (; fed < min(turns, stages); ++fed) feed(fed, fed);
        TeamTurn sum, out;
        bool dead = false;  // a wait gave up: carry on without, so that all warps end
        uint64_t t0 = 0;
        while (given < turns || fed < turns) {
            bool moved = false;
            if (given < turns && (dead || ready(summed[sum.s], sum))) {
                deposit(given++, sum.s);
                sum.next(stages);
                moved = true;
            }
            if (fed < turns && fed < given + stages && (dead || ready(written[out.s], out))) {
                feed(fed++, out.s);
                out.next(stages);
                moved = true;
            }
            if (moved) {
                t0 = 0;
                continue;
            }
            const uint64_t now = globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (__any_sync(0xffffffffu, now - t0 > kWaitLimitNs)) {
                if ((threadIdx.x & 31) == 0) atomicOr(err, kErrTimeout);
                dead = true;
            }
        }
    }
    // The warp has done its part of a stage's turn.
    __device__ static void done(uint64_t& bar) {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&bar));
    }
};

// A part is two words of (value, turn + 1): each word arrives whole, so a word
// that carries the turn carries its value, and no fence orders two words.  A
// slot is used again kTeamSlots turns later: a CTA that deposits turn k has
// collected turn k - stages (its stage was free again), so every CTA has
// deposited that one and has collected turn k - 2 stages; with 2 stages <=
// kTeamSlots nobody still reads the slot.
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
    // The collecting warp: done(turn, stage, parts...) writes a turn's statistics.
    // The next turn's words are fetched while this one's are merged.
    template <typename F> __device__ void collect_all(int turns, int stages, TeamBars& bars, F done) {
        Words now = {}, then = {};
        TeamTurn t;
        for (int k = 0; k < turns; ++k) {
            if (k + 1 < turns) fetch((uint32_t)(k + 1), then);
            float x[kTeamParts], y[kTeamParts];
            collect((uint32_t)k, now, x, y);
            done(k, t.s, x, y);
            TeamBars::done(bars.known[t.s]);
            t.next(stages);
            now = then;
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
    TeamShape q{p.tiles, p.stages, p.room, p.size, p.teams,
                static_cast<unsigned long long*>(words), err};
    void* args[] = {&a, &q};
    return launch_team_args(fn, args, p, words, s);
}

}  // namespace credit
