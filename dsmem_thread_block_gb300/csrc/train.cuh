// train.cuh -- what the training operators' kernels share: the counter-based
// dropout mask, access to a row's tiles and the launch arguments.
//
//   h = residual + keep ? x / (1 - p) : 0          (fp32, rounded when stored)
//   y = (h - mean) rstd gamma + beta               (RMSNorm: mean = 0, no beta)
//
// A row is read in warp tiles of 32 N columns, N elements per lane.  Two
// access forms own the columns of a tile differently: `VecIO` gives a lane N
// consecutive columns (one 8- or 16-byte access; pointers and rows 16-byte
// aligned), `ElemIO` gives element k of a lane column 32 k + lane, so that
// rows of any width and alignment are read and written 32 consecutive
// elements at a time.  The norms take N = 4 for both types: four fp32
// parameters are then one 16-byte load whose lanes are contiguous (with N = 8
// they lie 32 bytes apart and take twice the L1 passes).  Columns are counted in 32
// bits (cols <= 2^30), rows and offsets in 64.
#pragma once

#include <type_traits>

#include "internal.h"
#include "rowops.cuh"

namespace credit {

// ------------------------------------------------------------- dropout mask
// Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011): counter (column / 4, row, offset),
// key = seed; column c reads word c % 4.  The mask is a function of (row,
// column, seed, offset) alone, so the backward pass draws the same one and
// nothing is stored, whatever kernel or launch shape computes it.
//
// The twenty round keys come from the host (DropArgs, constant memory), so a
// round is two wide products and two three-way xors.
struct DropStream {
    uint32_t o0, o1;
    const DropArgs& a;
    __device__ explicit DropStream(const DropArgs& args) : a(args) {
        uint64_t o = a.offset;
        if (a.on && a.device_offset) o += *a.device_offset;
        o0 = (uint32_t)o;
        o1 = (uint32_t)(o >> 32);
    }
    // The words of the block of columns [4 group, 4 group + 4) of a row.
    __device__ __forceinline__ uint4 words(uint32_t group, uint32_t row) const {
        uint32_t c0 = group, c1 = row, c2 = o0, c3 = o1;
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
            c0 = (uint32_t)(p1 >> 32) ^ c1 ^ a.key[2 * i];
            c1 = (uint32_t)p1;
            c2 = (uint32_t)(p0 >> 32) ^ c3 ^ a.key[2 * i + 1];
            c3 = (uint32_t)p0;
        }
        return make_uint4(c0, c1, c2, c3);
    }
};

// ------------------------------------------------------------- tile access
// A lane's elements of a tile as they lie in memory.
template <int BYTES> struct Raw { uint32_t w[BYTES / 4]; };

// 8 or 16 bytes of a matrix that this pass reads once: not kept in L1, which
// is left to the parameters (read again for every row).  A plain coherent
// load: an output may be the same buffer.
__device__ __forceinline__ Raw<16> ld_once(const void* p, Raw<16>) {
    Raw<16> v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]) : "l"(p));
    return v;
}
__device__ __forceinline__ Raw<8> ld_once(const void* p, Raw<8>) {
    Raw<8> v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                 : "=r"(v.w[0]), "=r"(v.w[1]) : "l"(p));
    return v;
}
__device__ __forceinline__ void st_raw(void* p, Raw<16> v) {
    __stcs(static_cast<uint4*>(p), make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]));
}
__device__ __forceinline__ void st_raw(void* p, Raw<8> v) {
    __stcs(static_cast<uint2*>(p), make_uint2(v.w[0], v.w[1]));
}

// Raw elements <-> pairs.
template <typename T, int NP>
__device__ __forceinline__ void unpack(const Raw<NP * 2 * (int)sizeof(T)>& v, F2* f) {
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        if constexpr (sizeof(T) == 4)
            f[k] = {__uint_as_float(v.w[2 * k]), __uint_as_float(v.w[2 * k + 1])};
        else
            f[k] = Pairs<bf16>::one(v.w[k]);
    }
}
// (bf16 elements already in the upper halves of words)
template <typename T, int NP, typename = std::enable_if_t<sizeof(T) == 2>>
__device__ __forceinline__ void unpack(const Raw<NP * 8>& v, F2* f) {
#pragma unroll
    for (int k = 0; k < NP; ++k)
        f[k] = {__uint_as_float(v.w[2 * k]), __uint_as_float(v.w[2 * k + 1])};
}
template <typename T, int NP>
__device__ __forceinline__ Raw<NP * 2 * (int)sizeof(T)> pack(const F2* f) {
    Raw<NP * 2 * (int)sizeof(T)> v;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        if constexpr (sizeof(T) == 4) {
            v.w[2 * k] = __float_as_uint(f[k].x);
            v.w[2 * k + 1] = __float_as_uint(f[k].y);
        } else {
            v.w[k] = Pairs<bf16>::two(f[k]);
        }
    }
    return v;
}

// Access is by a pointer to the lane's first element of the first tile, a tile
// offset `off` (a compile-time constant wherever a warp's tiles are
// contiguous) and `left`, the columns from the lane's first element to the
// end of the row or slice.  FULL: the warp's tiles all lie inside, nothing is
// tested.
template <typename T, int ELEMS> struct VecIO {
    static constexpr bool kAligned = true;
    static constexpr int N = ELEMS;
    static constexpr int NP = N / 2;  // a lane's elements as pairs (element k: pair k / 2)
    static constexpr int kTile = 32 * N;
    using R = Raw<N * (int)sizeof(T)>;
    using S = R;
    __device__ static __forceinline__ int first(int lane) { return lane * N; }
    __device__ static __forceinline__ int at(int k) { return k; }  // element k, from the first
    // a lane's vector lies whole inside the row or whole outside
    template <bool FULL> __device__ static __forceinline__ bool in(int off, int, int left) {
        return FULL || off < left;
    }
    template <bool FULL>
    __device__ static __forceinline__ R load(const T* p, int off, int left) {
        return in<FULL>(off, 0, left) ? ld_once(p + off, R{}) : R{};
    }
    template <bool FULL>  // the same from a slice staged in shared memory
    __device__ static __forceinline__ R staged(const T* p, int off, int left) {
        R v = {};
        if (in<FULL>(off, 0, left)) v = *reinterpret_cast<const R*>(p + off);
        return v;
    }
    template <bool FULL>
    __device__ static __forceinline__ void store(T* p, int off, int left, const F2* f) {
        if (in<FULL>(off, 0, left)) st_raw(p + off, pack<T, NP>(f));
    }
    template <bool FULL>
    __device__ static __forceinline__ void store_sums(float* p, int off, int left, const F2* f) {
        if (in<FULL>(off, 0, left)) {
#pragma unroll
            for (int k = 0; k < NP; k += 2)
                *reinterpret_cast<float4*>(p + off + 2 * k) =
                    make_float4(f[k].x, f[k].y, f[k + 1].x, f[k + 1].y);
        }
    }
    // f += the sums at p, which an earlier launch of the call's chain wrote: read
    // from L2, where L1 could hold a line from before
    __device__ static __forceinline__ void add_sums(const float* p, int left, F2* f) {
        if (!in<false>(0, 0, left)) return;
#pragma unroll
        for (int k = 0; k < NP; k += 2) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(p + 2 * k));
            f[k] = add2(F2{v.x, v.y}, f[k]);
            f[k + 1] = add2(F2{v.z, v.w}, f[k + 1]);
        }
    }
    // `there`: the caller knows that p is not null
    template <bool FULL, typename PT>
    __device__ static __forceinline__ void params(const PT* p, int off, int left, F2* f,
                                                  float absent, bool there = false) {
        if (FULL && there) {
            float v[N];
            load_params<PT, N>(p, off, v);
#pragma unroll
            for (int k = 0; k < NP; ++k) f[k] = {v[2 * k], v[2 * k + 1]};
            return;
        }
#pragma unroll
        for (int k = 0; k < NP; ++k) f[k] = f2(absent);
        if (p && in<FULL>(off, 0, left)) load_param_pairs<PT, NP>(p, off, f, absent);
    }
    // Zero the lane's dropped elements (scaling is the caller's).
    __device__ static __forceinline__ void drop(const DropStream& d, int base, int lane,
                                                uint32_t row, F2* f) {
        const uint32_t g = (uint32_t)(base + lane * N) >> 2;
#pragma unroll
        for (int s = 0; s < N / 4; ++s) {
            const uint4 r = d.words(g + s, row);
            const uint32_t t = d.a.threshold;
            f[2 * s].x = r.x >= t ? f[2 * s].x : 0.f;
            f[2 * s].y = r.y >= t ? f[2 * s].y : 0.f;
            f[2 * s + 1].x = r.z >= t ? f[2 * s + 1].x : 0.f;
            f[2 * s + 1].y = r.w >= t ? f[2 * s + 1].y : 0.f;
        }
    }
};

template <typename T, int ELEMS> struct ElemIO {
    static constexpr bool kAligned = false;
    static constexpr int N = ELEMS;
    static constexpr int NP = N / 2;
    static constexpr int kTile = 32 * N;
    using R = Raw<N * (int)sizeof(T)>;
    using S = Raw<N * 4>;  // staged elements: bf16 ones in the upper halves of words
    using Word = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
    __device__ static __forceinline__ int first(int lane) { return lane; }
    __device__ static __forceinline__ int at(int k) { return 32 * k; }
    template <bool FULL> __device__ static __forceinline__ bool in(int off, int k, int left) {
        return FULL || off + 32 * k < left;
    }
    template <bool FULL>
    __device__ static __forceinline__ R load(const T* p, int off, int left) {
        const Word* r = reinterpret_cast<const Word*>(p) + off;
        R v;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint32_t e = in<FULL>(off, k, left) ? r[32 * k] : 0u;
            if constexpr (sizeof(T) == 4) v.w[k] = e;
            else if (k & 1) v.w[k / 2] |= e << 16;
            else v.w[k / 2] = e;
        }
        return v;
    }
    template <bool FULL>
    __device__ static __forceinline__ S staged(const T* p, int off, int left) {
        const Word* r = reinterpret_cast<const Word*>(p) + off;
        S v;
#pragma unroll
        for (int k = 0; k < N; ++k)
            v.w[k] = in<FULL>(off, k, left) ? (uint32_t)r[32 * k] << (32 - 8 * sizeof(T)) : 0u;
        return v;
    }
    template <bool FULL>
    __device__ static __forceinline__ void store(T* p, int off, int left, const F2* f) {
        const R v = pack<T, NP>(f);
        Word* r = reinterpret_cast<Word*>(p) + off;
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (in<FULL>(off, k, left))
                r[32 * k] = sizeof(T) == 4 ? (Word)v.w[k] : (Word)(v.w[k / 2] >> (k & 1 ? 16 : 0));
    }
    template <bool FULL>
    __device__ static __forceinline__ void store_sums(float* p, int off, int left, const F2* f) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (in<FULL>(off, k, left)) p[off + 32 * k] = k & 1 ? f[k / 2].y : f[k / 2].x;
    }
    __device__ static __forceinline__ void add_sums(const float* p, int left, F2* f) {
#pragma unroll
        for (int k = 0; k < NP; ++k)
            f[k] = add2(F2{in<false>(0, 2 * k, left) ? __ldcg(p + 64 * k) : 0.f,
                           in<false>(0, 2 * k + 1, left) ? __ldcg(p + 64 * k + 32) : 0.f}, f[k]);
    }
    template <bool FULL, typename PT>
    __device__ static __forceinline__ float param1(const PT* p, int off, int k, int left,
                                                   float absent, bool there) {
        return (there || p) && in<FULL>(off, k, left) ? load_param1<PT>(p, off + 32 * k) : absent;
    }
    template <bool FULL, typename PT>
    __device__ static __forceinline__ void params(const PT* p, int off, int left, F2* f,
                                                  float absent, bool there = false) {
#pragma unroll
        for (int k = 0; k < NP; ++k)
            f[k] = {param1<FULL>(p, off, 2 * k, left, absent, there),
                    param1<FULL>(p, off, 2 * k + 1, left, absent, there)};
    }
    // Every lane draws the block of columns 4 lane .. 4 lane + 3 of each 128
    // columns; a ballot per word hands each lane the bits of its own columns
    // 32 k + lane (block 8 k + lane / 4, word lane % 4).  All 32 lanes call.
    __device__ static __forceinline__ void drop(const DropStream& d, int base, int lane,
                                                uint32_t row, F2* f) {
#pragma unroll
        for (int s = 0; s < N / 4; ++s) {
            const uint4 r = d.words(((uint32_t)base >> 2) + 32u * s + (uint32_t)lane, row);
            const uint32_t t = d.a.threshold;
            const uint32_t b0 = __ballot_sync(0xffffffffu, r.x >= t);
            const uint32_t b1 = __ballot_sync(0xffffffffu, r.y >= t);
            const uint32_t b2 = __ballot_sync(0xffffffffu, r.z >= t);
            const uint32_t b3 = __ballot_sync(0xffffffffu, r.w >= t);
            const uint32_t lo = (lane & 1) ? b1 : b0, hi = (lane & 1) ? b3 : b2;
            const uint32_t mine = ((lane & 2) ? hi : lo) >> (lane >> 2);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                F2& p = f[2 * s + k];
                p.x = mine & (1u << (16 * k)) ? p.x : 0.f;
                p.y = mine & (1u << (16 * k + 8)) ? p.y : 0.f;
            }
        }
    }
};

// h of one tile from its raw values: residual + dropout(x), in fp32 (one
// fused multiply-add; `has_r` false: no residual).  All 32 lanes call.
template <typename T, typename IO, typename V>
__device__ __forceinline__ void tile_h(const V& xv, const V& rv, bool has_r, bool on,
                                       const DropStream& d, int base, int lane, uint32_t row,
                                       F2* h) {
    unpack<T, IO::NP>(xv, h);
    if (on) IO::drop(d, base, lane, row, h);
    if (has_r) {
        F2 r[IO::NP];
        unpack<T, IO::NP>(rv, r);
#pragma unroll
        for (int k = 0; k < IO::NP; ++k) h[k] = fma2(h[k], f2(d.a.scale), r[k]);
    } else if (on) {
#pragma unroll
        for (int k = 0; k < IO::NP; ++k) h[k] = mul2(h[k], f2(d.a.scale));
    }
}

// Pair k of a tile with the elements past the end replaced by zero.
template <bool FULL, typename IO>
__device__ __forceinline__ F2 inside(F2 v, int off, int k, int left) {
    return {IO::template in<FULL>(off, 2 * k, left) ? v.x : 0.f,
            IO::template in<FULL>(off, 2 * k + 1, left) ? v.y : 0.f};
}

// p moved by n elements, a null pointer left null.
template <typename P> __device__ __forceinline__ P* moved(P* p, int64_t n) {
    return p ? p + n : nullptr;
}

}  // namespace credit
