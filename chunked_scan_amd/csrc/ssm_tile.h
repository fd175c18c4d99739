// ssm_tile.h -- token tiles of the selective scan: 8 tokens by 64 channels of one activation, moved by
// one wave.  In memory order a lane holds 8 adjacent channels of one token (one 16-byte access per
// activation in bf16, two in f32); in the arithmetic a lane owns one channel.  LDS turns one into the
// other.  The LDS region belongs to one wave, whose LDS accesses execute in order: no barrier, only a
// fence for the compiler.
#pragma once
#include <utility>

#include "la_mixer.h"

namespace la {

constexpr int TT = 8;  // tokens per tile

__device__ __forceinline__ void wave_lds_fence() { asm volatile("" ::: "memory"); }

template <typename E> struct Raw8;
template <> struct Raw8<__bf16> {
    u32x4 a;
};
template <> struct Raw8<float> {
    f32x4 a, b;
};

// 8 elements at p of which the first n (1..8) exist; VEC: all exist and p is 16-byte aligned.  Elements
// that do not exist repeat the last one.
template <bool VEC>
__device__ __forceinline__ Raw8<__bf16> load8(const __bf16* p, int n) {
    Raw8<__bf16> r;
    if (VEC) {
        r.a = *(const u32x4*)p;
    } else {
        const uint16_t* q = (const uint16_t*)p;
#pragma unroll
        for (int i = 0; i < 4; i++) r.a[i] = q[min(2 * i, n - 1)] | ((uint32_t)q[min(2 * i + 1, n - 1)] << 16);
    }
    return r;
}
template <bool VEC>
__device__ __forceinline__ Raw8<float> load8(const float* p, int n) {
    Raw8<float> r;
    if (VEC) {
        r.a = *(const f32x4*)p;
        r.b = *((const f32x4*)p + 1);
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            r.a[i] = p[min(i, n - 1)];
            r.b[i] = p[min(i + 4, n - 1)];
        }
    }
    return r;
}
template <bool VEC>
__device__ __forceinline__ void store8(__bf16* p, int n, const Raw8<__bf16>& r) {
    if (VEC) {
        *(u32x4*)p = r.a;
    } else {
        uint16_t* q = (uint16_t*)p;
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < n) q[i] = (uint16_t)(r.a[i >> 1] >> (16 * (i & 1)));
    }
}
template <bool VEC>
__device__ __forceinline__ void store8(float* p, int n, const Raw8<float>& r) {
    if (VEC) {
        *(f32x4*)p = r.a;
        *((f32x4*)p + 1) = r.b;
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < n) p[i] = i < 4 ? r.a[i & 3] : r.b[i & 3];
    }
}

// A wave's place in the tiles of one 64-channel block starting at d0: lane = token * 8 + chunk of 8 channels.
struct TilePlace {
    int token, col, n;  // its token; its first channel in the block and how many of its 8 exist
    bool in;            // whether any does (if not: the block's last chunk is repeated, nothing is stored)
    __device__ __forceinline__ TilePlace(int64_t d0, int64_t D) {
        const int lane = threadIdx.x & 63, left = (int)min((int64_t)64, D - d0), c = (lane & 7) * 8;
        token = lane >> 3;
        in = c < left;
        col = in ? c : (left - 1) / 8 * 8;
        n = min(8, left - col);
    }
};

// One activation's tiles: where the lane's elements are from a tile's first token and channel.  A whole tile's
// address is then the tile's (scalar) plus this, without a 64-bit product per tile and activation (first pass of the
// backward, 2 x 4096 x 2048, N = 16: 99 -> 95 us).
struct TileRow {
    int64_t at;
    __device__ __forceinline__ TileRow(const la_rows& r, const TilePlace& pl) : at(pl.token * r.token + pl.col) {}
};
// The lane's elements of the tile of `left` tokens at p (of which those behind the last repeat it).
template <typename E, bool VEC>
__device__ __forceinline__ Raw8<E> tile_load(const E* p, const TileRow& row, int64_t stride, int left, const TilePlace& pl) {
    if (left >= TT) return load8<VEC>(p + row.at, pl.n);
    return load8<VEC>(p + min(pl.token, left - 1) * stride + pl.col, pl.n);
}
// The lane's elements of token t, p at token 0 (where there are no registers for TileRows).
template <typename E, bool VEC>
__device__ __forceinline__ Raw8<E> token_load(const E* p, int64_t stride, int t, const TilePlace& pl) {
    return load8<VEC>(p + t * stride + pl.col, pl.n);
}
// The lane's 8 channels in an LDS tile [TT][64].
template <typename E>
__device__ __forceinline__ Raw8<E>* lds_chunk(E* tile) {
    return reinterpret_cast<Raw8<E>*>(tile + (threadIdx.x & 63) * 8);
}

// The same value, waited for here and unknown to the compiler from here on: the wait comes before the next
// token's loads are issued and not after them, and exponentials of the way forwards are not held on to for the
// way back, for which there are no registers.
__device__ __forceinline__ float arrived(float x) {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" : "+v"(x));
    __builtin_amdgcn_sched_barrier(0);
    return x;
}

// f(0), .., f(N - 1) with the index as a compile-time constant.
template <typename F, int... I>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
    static_for_impl(f, std::make_integer_sequence<int, N>{});
}

// c + x y^T for 4 key dims and the wave's 64 channels: key dim i is element i, the lane's channel has y.  x is in
// lanes E % 64 + i of register x[E / 64].  It is the matrix cores' 4 x 4 x 1 fp32 product: its 16 blocks of 4
// lanes are the 64 channels, and the block of x is broadcast to all of them.  One instruction in place of
// four on the vector units, which bound these kernels.
template <int E>
__device__ __forceinline__ f32x4 outer4(const float* x, float y, f32x4 c) {
    static_assert(E % 4 == 0, "a block of four lanes");
    return __builtin_amdgcn_mfma_f32_4x4x1f32(x[E / 64], y, c, 4, E % 64 / 4, 0);
}

}  // namespace la
