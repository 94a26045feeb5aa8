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
//     known    the collecting warp has the row's statistics from the exchange
//     written  W warps write the row's outputs; the stage is free
// No barrier joins them, so each kind runs as far ahead as the stages allow.
//
// Measured on 256 rows of 786432 bf16 columns, RMSNorm backward: warps that sum
// and write, 366 us; the kinds apart with a barrier a row, 314 and later 272;
// mbarriers 269; statistics from one CTA a turn instead of every CTA merging
// all parts, 226 (0.79 of the copy rate).  What bounds it now is a turn's
// passage through the slowest CTA, 0.7 to 1.0 us however few columns it has:
// 1024 rows of 262144 columns take 328 us with 50 CTAs a row, 740 with 140.
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
    ulonglong2* words;  // a team: [slot][CTA] parts, [slot] statistics; zero before the launch
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
//
// A wait that gives up ends the waiting of the whole CTA: its other warps go
// through their turns without any (the call has failed, as the error word
// says), no copy is issued any more, and the serving warp leaves when those in
// flight have arrived.  A CTA ends one time limit after its team fell silent.
struct TeamBars {
    uint64_t fed[kTeamStages], summed[kTeamStages], known[kTeamStages], written[kTeamStages];
    int gave_up;
    // All threads call.
    __device__ void init(int stages, int W) {
        if (threadIdx.x == 0) {
            gave_up = 0;
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
    __device__ bool over() const { return *static_cast<const volatile int*>(&gave_up) != 0; }
    __device__ void give_up(unsigned* err) {
        atomicOr(err, kErrTimeout);
        *static_cast<volatile int*>(&gave_up) = 1;
    }
    __device__ void wait(uint64_t& bar, const TeamTurn& t, unsigned* err) {
        const uint32_t b = smem_u32(&bar);
        for (int i = 0; i < 256; ++i)
            if (mbar_try_wait(b, t.phase)) return;
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(b, t.phase)) {
            if (over()) return;
            if (globaltimer_ns() - t0 > kWaitLimitNs) return give_up(err);
        }
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
        uint64_t t0 = 0;
        while (given < turns || fed < turns) {
            bool moved = false;
            if (given < turns && ready(summed[sum.s], sum)) {
                deposit(given++, sum.s);
                sum.next(stages);
                moved = true;
            }
            // (a warp that no longer waits may have passed the stage on too early)
            if (fed < turns && fed < given + stages && ready(written[out.s], out) &&
                !__any_sync(0xffffffffu, over())) {
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
            if (__any_sync(0xffffffffu, over() || now - t0 > kWaitLimitNs)) {
                if ((threadIdx.x & 31) == 0) give_up(err);
                // the copies in flight: each stage's last
                for (int f = max(0, fed - stages); f < fed; ++f)
                    mbar_wait_bounded(smem_u32(&this->fed[f % stages]), (f / stages) & 1, err);
                return;
            }
        }
    }
    // The warp has done its part of a stage's turn.
    __device__ static void done(uint64_t& bar) {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&bar));
    }
};

// The exchange: every CTA deposits its part of a turn, turn k's leader (the CTA
// of rank k % T) merges the T parts and publishes the row's statistics, which
// every CTA reads.  So a CTA merges one turn in T, and one load (a lane a turn)
// brings it all the turns that have been published since the last.
//
// Parts and statistics are two words of (value, turn + 1): each word arrives
// whole, so a word that carries the turn carries its value, and no fence orders
// two words.  A slot is used again kTeamSlots turns later: a CTA that deposits
// turn k has the statistics of the turns up to k - stages (its stage was free
// again), so those turns' leaders have read all parts, and every CTA had the
// statistics of the turns up to k - 2 stages when it deposited that part; with
// 2 stages <= kTeamSlots nobody still reads the slot.
struct TeamExchange {
    using Pair = ulonglong2;
    Pair* parts;  // [slot][CTA]
    Pair* stats;  // [slot]
    int size, rank, lane;
    unsigned* err;

    __device__ TeamExchange(const TeamShape& q, int team, int r, int l)
        : parts(q.words + (size_t)team * kTeamSlots * (q.size + 1)),
          stats(parts + (size_t)kTeamSlots * q.size), size(q.size), rank(r), lane(l), err(q.err) {}
    __device__ static void put(Pair* p, int turn, float a, float b) {
        const unsigned long long tag = (unsigned long long)(uint32_t)(turn + 1) << 32;
        asm volatile("st.relaxed.gpu.global.v2.u64 [%0], {%1, %2};"
                     :: "l"(p), "l"(tag | __float_as_uint(a)), "l"(tag | __float_as_uint(b))
                     : "memory");
    }
    __device__ static Pair get(const Pair* p) {
        Pair v;
        asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];"
                     : "=l"(v.x), "=l"(v.y) : "l"(p) : "memory");
        return v;
    }
    __device__ static bool of(const Pair& v, int turn) {
        return (uint32_t)(v.x >> 32) == (uint32_t)(turn + 1) &&
               (uint32_t)(v.y >> 32) == (uint32_t)(turn + 1);
    }
    __device__ void deposit(int turn, float a, float b) const {
        if (lane == 0) put(parts + (size_t)(turn % kTeamSlots) * size + rank, turn, a, b);
    }
    // The collecting warp: merge(parts of CTAs lane, lane + 32, ...; zeros past
    // the team) gives a turn's statistics, done(turn, stage, statistics) hands
    // them to the writing warps.
    template <typename M, typename F>
    __device__ void collect(int turns, int stages, TeamBars& bars, M merge, F done) const {
        TeamTurn t;
        int k = 0, lead = rank;  // the turn to be known next, the turn to be merged next
        uint64_t t0 = 0;
        while (k < turns || lead < turns) {
            const bool leads = lead < turns && lead < k + stages;  // (no part of later turns)
            Pair f[kTeamParts], r = {};
            if (leads) {
#pragma unroll
                for (int i = 0; i < kTeamParts; ++i)
                    if (lane + 32 * i < size)
                        f[i] = get(parts + (size_t)(lead % kTeamSlots) * size + lane + 32 * i);
            }
            if (lane < stages && k + lane < turns) r = get(stats + (k + lane) % kTeamSlots);
            bool moved = false;
            if (leads) {
                bool all = true;
#pragma unroll
                for (int i = 0; i < kTeamParts; ++i)
                    if (lane + 32 * i < size) all = all && of(f[i], lead);
                if (__all_sync(0xffffffffu, all)) {
                    float x[kTeamParts], y[kTeamParts];
#pragma unroll
                    for (int i = 0; i < kTeamParts; ++i) {
                        const bool in = lane + 32 * i < size;
                        x[i] = in ? __uint_as_float((uint32_t)f[i].x) : 0.f;
                        y[i] = in ? __uint_as_float((uint32_t)f[i].y) : 0.f;
                    }
                    const float2 m = merge(x, y);
                    if (lane == 0) put(stats + lead % kTeamSlots, lead, m.x, m.y);
                    lead += size;
                    moved = true;
                }
            }
            const unsigned here = __ballot_sync(0xffffffffu, of(r, k + lane));
            const int n = min(__ffs((int)~here) - 1, turns - k);  // published without a gap
            for (int i = 0; i < n; ++i) {
                const float a = __shfl_sync(0xffffffffu, __uint_as_float((uint32_t)r.x), i);
                const float b = __shfl_sync(0xffffffffu, __uint_as_float((uint32_t)r.y), i);
                done(k++, t.s, make_float2(a, b));
                TeamBars::done(bars.known[t.s]);
                t.next(stages);
                moved = true;
            }
            if (moved) {
                t0 = 0;
                continue;
            }
            const uint64_t now = globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (__any_sync(0xffffffffu, bars.over() || now - t0 > kWaitLimitNs)) {
                if (lane == 0) bars.give_up(err);
                return;
            }
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
                static_cast<ulonglong2*>(words), err};
    void* args[] = {&a, &q};
    return launch_team_args(fn, args, p, words, s);
}

}  // namespace credit
