// ring.cuh -- a stream of rows through shared memory: one CTA, or a cluster
// of P CTAs each owning a slice of every row's columns, walks turns of R rows
// c, c + clusters, ... ; bulk copies bring the slices of the next turns into a
// ring of stages while the present one is reduced and written.  Two rows a
// turn share the parameters' loads, a barrier and the shuffles of a reduction
// (each half warp finishes one row's sums): 8192 x 8192 bf16 LayerNorm forward
// 62 us with one row a turn, 52 with two (49 since the parameters stay in
// registers).
#pragma once

#include "ring_plan.h"
#include "train.cuh"

namespace credit {

// The bytes [off, off + bytes) of matrix `src` as bulk copies can bring them:
// whole 16-byte lines, widened over the slice's ends where the line lies
// inside the matrix (the neighbours' bytes are not used), cut back where it
// does not (the matrix's own first and last line; `cut` bytes are then copied
// by this thread).  Byte A of the matrix lands at A - (off's line).
struct Lines {
    const char* first;    // the line of the slice's first byte
    const char* lo;
    const char* hi;
    const char* begin;
    const char* end;
    __device__ Lines(const char* src, int64_t off, int bytes, int64_t total) {
        begin = src + off;
        end = begin + bytes;
        first = (const char*)((uintptr_t)begin & ~(uintptr_t)15);
        lo = first < src ? first + 16 : first;
        hi = (const char*)(((uintptr_t)end + 15) & ~(uintptr_t)15);
        if (hi > src + total) hi -= 16;
        if (hi < lo) hi = lo;
    }
    __device__ uint32_t bulk() const { return (uint32_t)(hi - lo); }
    __device__ bool cut() const { return begin < lo || hi < end; }
};

// One warp brings the slices of R rows (those below `rows`) of NS streams into
// a stage, all lanes calling; waiters see them when the stage's mbarrier
// completes its phase.  Slice (stream i, row j) has room i R + j.  Rows that
// are not whole lines take a lane a slice: their addresses, worked out by one
// thread, were what a turn of 10001 bf16 columns waited for.
template <int NS, int R, typename T, typename IO>
__device__ __forceinline__ void ring_issue(const void* const (&src)[NS], int ns, int64_t row,
                                           int64_t rows, int cols, int c0, int bytes,
                                           unsigned char* stage, int room, uint32_t bar) {
    const uint64_t pol = l2_policy_evict_first();
    const int lane = threadIdx.x & 31;
    const int64_t pitch = (int64_t)cols * (int)sizeof(T);
    const int64_t off = row * pitch + c0 * (int)sizeof(T);
    const bool two = R > 1 && row + 1 < rows;
    if constexpr (IO::kAligned) {
        if (lane == 0) {
            mbar_arrive_expect_tx(bar, (uint32_t)((two ? 2 * ns : ns) * bytes));
#pragma unroll
            for (int i = 0; i < NS; ++i)
                if (i < ns) {
                    const char* p = static_cast<const char*>(src[i]) + off;
                    const uint32_t d = smem_u32(stage) + i * R * room;
                    bulk_g2s(d, p, (uint32_t)bytes, bar, pol);
                    if (two) bulk_g2s(d + room, p + pitch, (uint32_t)bytes, bar, pol);
                }
        }
    } else {
        const int i = lane / R, j = lane % R;
        const char* p = static_cast<const char*>(src[0]);
#pragma unroll
        for (int t = 1; t < NS; ++t) p = i == t ? static_cast<const char*>(src[t]) : p;
        const bool mine = i < ns && (j == 0 || two);
        const Lines l(p, off + j * pitch, bytes, rows * pitch);
        unsigned char* const d = stage + lane * room;
        if (mine && l.cut()) {
            const char* const head = l.lo < l.end ? l.lo : l.end;
            for (const char* c = l.begin; c < head; c += sizeof(T))
                *reinterpret_cast<T*>(d + (c - l.first)) = *reinterpret_cast<const T*>(c);
            for (const char* c = l.hi > l.begin ? l.hi : l.begin; c < l.end; c += sizeof(T))
                *reinterpret_cast<T*>(d + (c - l.first)) = *reinterpret_cast<const T*>(c);
            // a later turn's bulk copy overwrites these bytes: order it behind them
            fence_proxy_async_smem();
        }
        const uint32_t tx = __reduce_add_sync(0xffffffffu, mine ? l.bulk() : 0u);
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(bar, tx);  // releases the plain stores too
        __syncwarp();
        if (mine && l.bulk())
            bulk_g2s(smem_u32(d) + (uint32_t)(l.lo - l.first), l.lo, l.bulk(), bar, pol);
    }
}

// Where a stream's slice starts inside its room.
template <typename IO>
__device__ __forceinline__ int ring_shift(const void* src, int64_t off) {
    if constexpr (IO::kAligned) return 0;
    return (int)(((uintptr_t)src + (uintptr_t)off) & 15);
}

// The clusters' exchange of one 16-byte part per turn: each CTA deposits its
// part in every peer's slot with st.async and waits on its own mbarrier for
// the P - 1 deposits and its own arrival.  Slots and mbarriers alternate by
// turn parity: a peer's deposit for turn k + 2 comes after its wait for turn
// k + 1, which needs this CTA's deposit for turn k + 1, made after a barrier
// that follows every thread's reads of the slots of turn k.
struct RingExchange {
    float4 slots[2][kMaxCluster];
    uint64_t bar[2];

    __device__ void init(uint32_t P) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&bar[b]), 2);
            mbar_arrive_expect_tx(smem_u32(&bar[b]), (P - 1) * 16u);
        }
    }
    // Warp 0 calls, every lane with the CTA's part of turn k.
    __device__ void deposit(uint32_t k, float4 v, uint32_t P, uint32_t rank) {
        const int b = k & 1;
        const uint32_t bb = smem_u32(&bar[b]);
        if (threadIdx.x == rank) {
            slots[b][rank] = v;
            mbar_arrive(bb);
        } else if (threadIdx.x < P) {
            st_async_v4f32(mapa_shared(smem_u32(&slots[b][rank]), threadIdx.x), v.x, v.y, v.z, v.w,
                           mapa_shared(bb, threadIdx.x));
        }
    }
    // All threads call: the P parts of turn k, once they are here.
    __device__ const float4* wait(uint32_t k, uint32_t P, uint32_t rank, unsigned* err) {
        const uint32_t bb = smem_u32(&bar[k & 1]);
        mbar_wait_bounded(bb, (k >> 1) & 1u, err);
        if (threadIdx.x == rank) mbar_arrive_expect_tx(bb, (P - 1) * 16u);
        return slots[k & 1];
    }
};

// Sums over the warp of one value (R = 1) or of two rows' values (R = 2, lanes
// 0-15 return row 0's, lanes 16-31 row 1's).
template <int R> __device__ __forceinline__ float row_sum(const float (&v)[R], int lane) {
    float s;
    if constexpr (R == 1) {
        s = v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
    } else {
        const bool up = lane & 16;
        s = (up ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 16);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}
__device__ __forceinline__ float half_sum(float s) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}
// Every lane's copy of the value that the lanes of row j's half hold.
template <int R> __device__ __forceinline__ void spread(float s, int lane, float (&v)[R]) {
    if constexpr (R == 1) {
        v[0] = s;
    } else {
        const float o = __shfl_xor_sync(0xffffffffu, s, 16);
        v[0] = lane & 16 ? o : s;
        v[1] = lane & 16 ? s : o;
    }
}

}  // namespace credit
