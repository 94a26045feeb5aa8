// ring.cuh -- a stream of rows through shared memory: one CTA, or a cluster
// of P CTAs each owning a slice of every row's columns, walks the rows
// c, c + clusters, ... ; bulk copies bring the slices of the next rows into a
// ring of stages while the present one is reduced and written.
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

// One thread brings the row's slices of NS streams into a stage; waiters see
// them when the stage's mbarrier completes its phase.
template <int NS, typename T, typename IO>
__device__ __forceinline__ void ring_issue(const void* const (&src)[NS], int ns, int64_t off,
                                           int bytes, int64_t total, unsigned char* stage, int room,
                                           uint32_t bar) {
    const uint64_t pol = l2_policy_evict_first();
    if constexpr (IO::kAligned) {
        mbar_arrive_expect_tx(bar, (uint32_t)(ns * bytes));
#pragma unroll
        for (int s = 0; s < NS; ++s)
            if (s < ns)
                bulk_g2s(smem_u32(stage) + s * room, static_cast<const char*>(src[s]) + off,
                         (uint32_t)bytes, bar, pol);
    } else {
        uint32_t tx = 0;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            if (s >= ns) continue;
            const Lines l(static_cast<const char*>(src[s]), off, bytes, total);
            tx += l.bulk();
            if (l.cut()) {
                unsigned char* d = stage + s * room;
                const char* const head = l.lo < l.end ? l.lo : l.end;
                for (const char* p = l.begin; p < head; p += sizeof(T))
                    *reinterpret_cast<T*>(d + (p - l.first)) = *reinterpret_cast<const T*>(p);
                for (const char* p = l.hi > l.begin ? l.hi : l.begin; p < l.end; p += sizeof(T))
                    *reinterpret_cast<T*>(d + (p - l.first)) = *reinterpret_cast<const T*>(p);
            }
        }
        mbar_arrive_expect_tx(bar, tx);  // releases the plain stores too
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            if (s >= ns) continue;
            const Lines l(static_cast<const char*>(src[s]), off, bytes, total);
            if (l.bulk())
                bulk_g2s(smem_u32(stage) + s * room + (uint32_t)(l.lo - l.first), l.lo, l.bulk(),
                         bar, pol);
        }
    }
}

// Where a stream's slice starts inside its room.
template <typename IO>
__device__ __forceinline__ int ring_shift(const void* src, int64_t off) {
    if constexpr (IO::kAligned) return 0;
    return (int)(((uintptr_t)src + (uintptr_t)off) & 15);
}

// The clusters' exchange of one 16-byte part per row: each CTA deposits its
// part in every peer's slot with st.async and waits on its own mbarrier for
// the P - 1 deposits and its own arrival.  Slots and mbarriers alternate by
// row parity: a peer's deposit for row k + 2 comes after its wait for row
// k + 1, which needs this CTA's deposit for row k + 1, made after it read the
// slots of row k.
struct RingExchange {
    float4 slots[2][kMaxCluster];
    uint64_t bar[2];

    __device__ void init(uint32_t P) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&bar[b]), 2);
            mbar_arrive_expect_tx(smem_u32(&bar[b]), (P - 1) * 16u);
        }
    }
    // All threads of the CTA call, after the barrier that made `v` the same in
    // all of them.  Returns the P parts of row k.
    __device__ const float4* all(int64_t k, float4 v, uint32_t P, uint32_t rank, unsigned* err) {
        const int b = (int)(k & 1);
        const uint32_t bb = smem_u32(&bar[b]);
        if (threadIdx.x == rank) {
            slots[b][rank] = v;
            mbar_arrive(bb);
        } else if (threadIdx.x < P) {
            st_async_v4f32(mapa_shared(smem_u32(&slots[b][rank]), threadIdx.x), v.x, v.y, v.z, v.w,
                           mapa_shared(bb, threadIdx.x));
        }
        mbar_wait_bounded(bb, (uint32_t)(k >> 1) & 1u, err);
        if (threadIdx.x == rank) mbar_arrive_expect_tx(bb, (P - 1) * 16u);
        return slots[b];
    }
};

}  // namespace credit
