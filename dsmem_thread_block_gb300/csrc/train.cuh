// train.cuh -- what the training operators' kernels share: the counter-based
// dropout mask, access to a row's tiles and the launch arguments.
//
//   h = residual + keep ? x / (1 - p) : 0          (fp32, rounded when stored)
//   y = (h - mean) rstd gamma + beta               (RMSNorm: mean = 0, no beta)
//
// A row is read in warp tiles of 32 N columns, N elements per lane (N = 8 for
// bf16, 4 for fp32: one 16-byte vector).  Two access forms own the columns of
// a tile differently: `VecIO` gives a lane N consecutive columns (one 16-byte
// access; pointers and rows 16-byte aligned), `ElemIO` gives element k of a
// lane column 32 k + lane, so that rows of any width and alignment are read
// and written 32 consecutive elements at a time.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace credit {

// ------------------------------------------------------------- dropout mask
// Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011): counter (column / 4, row, offset),
// key = seed; column c reads word c % 4.  The mask is a function of (row,
// column, seed, offset) alone, so the backward pass draws the same one and
// nothing is stored, whatever kernel or launch shape computes it.
__device__ __forceinline__ uint4 philox10(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                          uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)p1;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)p0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// A call's dropout stream as the kernels use it: the offset's device part is
// read when the kernel runs, so a replayed graph can draw new masks.
struct DropStream {
    uint32_t threshold, k0, k1, o0, o1;
    float scale;
    __device__ explicit DropStream(const DropArgs& a)
        : threshold(a.threshold), k0(a.k0), k1(a.k1), scale(a.scale) {
        uint64_t o = a.offset;
        if (a.on && a.device_offset) o += *a.device_offset;
        o0 = (uint32_t)o;
        o1 = (uint32_t)(o >> 32);
    }
    // bit w: word w of the block of columns [4 group, 4 group + 4) is kept
    __device__ __forceinline__ uint32_t keep4(uint32_t group, uint32_t row) const {
        const uint4 r = philox10(group, row, o0, o1, k0, k1);
        return (r.x >= threshold ? 1u : 0u) | (r.y >= threshold ? 2u : 0u) |
               (r.z >= threshold ? 4u : 0u) | (r.w >= threshold ? 8u : 0u);
    }
};

// ------------------------------------------------------------- tile access
template <typename T> struct VecIO {
    static constexpr int N = 16 / (int)sizeof(T);
    static constexpr int kTile = 32 * N;
    __device__ static __forceinline__ int64_t col(int64_t base, int lane, int k) {
        return base + lane * N + k;
    }
    // a lane's vector lies whole inside the row or whole outside
    __device__ static __forceinline__ bool valid(int64_t base, int lane, int, int64_t cols) {
        return base + lane * N < cols;
    }
    __device__ static __forceinline__ uint4 load(const void* row, int64_t base, int lane,
                                                 int64_t cols) {
        const int64_t j = base + lane * N;
        return j < cols ? *reinterpret_cast<const uint4*>(static_cast<const T*>(row) + j)
                        : make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ static __forceinline__ void store(void* row, int64_t base, int lane, int64_t cols,
                                                 uint4 v) {
        const int64_t j = base + lane * N;
        if (j < cols) __stcs(reinterpret_cast<uint4*>(static_cast<T*>(row) + j), v);
    }
    template <typename PT>
    __device__ static __forceinline__ void params(const PT* p, int64_t base, int lane,
                                                  int64_t cols, float* f, float absent) {
        const int64_t j = base + lane * N;
        if (p && j < cols) {
            load_params<PT, N>(p, j, f);
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) f[k] = absent;
        }
    }
    __device__ static __forceinline__ void store_f32(float* p, int64_t base, int lane,
                                                     int64_t cols, const float* f) {
        const int64_t j = base + lane * N;
        if (j < cols) {
#pragma unroll
            for (int k = 0; k < N; k += 4)
                *reinterpret_cast<float4*>(p + j + k) =
                    make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
        }
    }
    // bit k: the lane's element k is kept
    __device__ static __forceinline__ uint32_t keep(const DropStream& d, int64_t base, int lane,
                                                    uint32_t row) {
        const uint32_t g = (uint32_t)((base + lane * N) >> 2);
        uint32_t m = 0;
#pragma unroll
        for (int s = 0; s < N / 4; ++s) m |= d.keep4(g + s, row) << (4 * s);
        return m;
    }
};

template <typename T> struct ElemIO {
    static constexpr int N = 16 / (int)sizeof(T);
    static constexpr int kTile = 32 * N;
    __device__ static __forceinline__ int64_t col(int64_t base, int lane, int k) {
        return base + 32 * k + lane;
    }
    __device__ static __forceinline__ bool valid(int64_t base, int lane, int k, int64_t cols) {
        return base + 32 * k + lane < cols;
    }
    __device__ static __forceinline__ uint4 load(const void* row, int64_t base, int lane,
                                                 int64_t cols) {
        uint32_t w[4];
        if constexpr (sizeof(T) == 4) {
            const uint32_t* r = static_cast<const uint32_t*>(row) + base + lane;
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = valid(base, lane, k, cols) ? r[32 * k] : 0u;
        } else {
            const uint16_t* r = static_cast<const uint16_t*>(row) + base + lane;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t lo = valid(base, lane, 2 * k, cols) ? r[64 * k] : 0u;
                const uint32_t hi = valid(base, lane, 2 * k + 1, cols) ? r[64 * k + 32] : 0u;
                w[k] = lo | (hi << 16);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ static __forceinline__ void store(void* row, int64_t base, int lane, int64_t cols,
                                                 uint4 v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if constexpr (sizeof(T) == 4) {
            uint32_t* r = static_cast<uint32_t*>(row) + base + lane;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (valid(base, lane, k, cols)) r[32 * k] = w[k];
        } else {
            uint16_t* r = static_cast<uint16_t*>(row) + base + lane;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (valid(base, lane, 2 * k, cols)) r[64 * k] = (uint16_t)w[k];
                if (valid(base, lane, 2 * k + 1, cols)) r[64 * k + 32] = (uint16_t)(w[k] >> 16);
            }
        }
    }
    template <typename PT>
    __device__ static __forceinline__ void params(const PT* p, int64_t base, int lane,
                                                  int64_t cols, float* f, float absent) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            f[k] = p && valid(base, lane, k, cols) ? load_param1<PT>(p, base + 32 * k + lane)
                                                   : absent;
    }
    __device__ static __forceinline__ void store_f32(float* p, int64_t base, int lane,
                                                     int64_t cols, const float* f) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (valid(base, lane, k, cols)) p[base + 32 * k + lane] = f[k];
    }
    // Every lane draws the block of columns 4 lane .. 4 lane + 3 of each 128
    // columns; a ballot per word hands each lane the bits of its own columns
    // 32 k + lane (block 8 k + lane / 4, word lane % 4).  All 32 lanes call.
    __device__ static __forceinline__ uint32_t keep(const DropStream& d, int64_t base, int lane,
                                                    uint32_t row) {
        uint32_t m = 0;
#pragma unroll
        for (int s = 0; s < N / 4; ++s) {
            const uint32_t b = d.keep4((uint32_t)(base >> 2) + 32u * s + (uint32_t)lane, row);
            const uint32_t b0 = __ballot_sync(0xffffffffu, b & 1u);
            const uint32_t b1 = __ballot_sync(0xffffffffu, b & 2u);
            const uint32_t b2 = __ballot_sync(0xffffffffu, b & 4u);
            const uint32_t b3 = __ballot_sync(0xffffffffu, b & 8u);
            const uint32_t lo = (lane & 1) ? b1 : b0, hi = (lane & 1) ? b3 : b2;
            const uint32_t mine = ((lane & 2) ? hi : lo) >> (lane >> 2);
#pragma unroll
            for (int k = 0; k < 4; ++k) m |= ((mine >> (8 * k)) & 1u) << (4 * s + k);
        }
        return m;
    }
};

// h of one tile: residual + dropout(x), in fp32.  `xrow` / `rrow` are the
// row's first elements (rrow null: no residual).  Columns past the row read
// as zero.  All 32 lanes call.
template <typename T, typename IO>
__device__ __forceinline__ void tile_h(const T* xrow, const T* rrow, bool on, const DropStream& d,
                                       int64_t base, int lane, uint32_t row, int64_t cols,
                                       float* h) {
    Elem<T>::unpack(IO::load(xrow, base, lane, cols), h);
    if (on) {
        const uint32_t m = IO::keep(d, base, lane, row);
#pragma unroll
        for (int k = 0; k < IO::N; ++k) h[k] = (m >> k) & 1u ? h[k] * d.scale : 0.f;
    }
    if (rrow) {
        float r[IO::N];
        Elem<T>::unpack(IO::load(rrow, base, lane, cols), r);
#pragma unroll
        for (int k = 0; k < IO::N; ++k) h[k] += r[k];
    }
}

}  // namespace credit
