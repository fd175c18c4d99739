// row_ops.h -- what the kernels that work on whole rows share: 8-element accesses, sums over a row's threads, a row's
// reciprocal deviation.
#pragma once
#include "la_mixer.h"

namespace la {

// 8 adjacent elements, of which `n` exist; VEC: 16-byte words (the row is aligned and whole chunks exist).
// ONCE: a streaming load.  The forward's rows are read once and its outputs are what comes next: 16384 x 2048 bf16 to
// 8 bits, call after call, 62.6 -> 53.4 us (before the exact quotients), single launches 55.9 -> 54.6; a whole layer over
// 16384 x 2048 (norm, projections, convolution, scan) 779 -> 769.  (With the outputs streamed as well 54.6; the
// backward 35.2 -> 35.7.)
template <typename V, bool ONCE>
__device__ __forceinline__ V load_word(const V* p) {
    return ONCE ? __builtin_nontemporal_load(p) : *p;
}
template <typename E, bool VEC, bool ONCE = false>
__device__ __forceinline__ void load8(const E* p, int n, float* f) {
    if (VEC) {
        if (sizeof(E) == 2) {
            const u32x4 r = load_word<u32x4, ONCE>((const u32x4*)p);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                f[2 * i] = bits_lo_bf16(r[i]);
                f[2 * i + 1] = bits_hi_bf16(r[i]);
            }
        } else {
            const f32x4 a = load_word<f32x4, ONCE>((const f32x4*)p), b = load_word<f32x4, ONCE>((const f32x4*)p + 1);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                f[i] = a[i];
                f[4 + i] = b[i];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) f[i] = i < n ? (float)p[i] : 0.f;
    }
}
template <typename E, bool VEC>
__device__ __forceinline__ void store8(E* p, int n, const float* f) {
    if (VEC) {
        if (sizeof(E) == 2) {
            *(u32x4*)p = pack8_pairs(f);
        } else {
            *(f32x4*)p = f32x4{f[0], f[1], f[2], f[3]};
            *((f32x4*)p + 1) = f32x4{f[4], f[5], f[6], f[7]};
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < n) io<E>::st(p + i, f[i]);
    }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
    return v;
}
// Largest of non-negative values; a NaN stays one (fmaxf would drop it).
__device__ __forceinline__ float max_nan(float a, float b) { return a != a ? a : (b != b ? b : fmaxf(a, b)); }
template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int m = LANES / 2; m; m >>= 1) v = max_nan(v, __shfl_xor(v, m));
    return v;
}

// The sum over the TPR threads of a row.  `buf`: one float per wave; a barrier on either side.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* buf) {
    v = wave_sum(v);
    if (TPR == 64) return v;
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) buf[w] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 64; i++) v += buf[i];
    __syncthreads();
    return v;
}
template <int TPR>
__device__ __forceinline__ float row_max(float v, float* buf) {
    v = lanes_max<64>(v);
    if (TPR == 64) return v;
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) buf[w] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 64; i++) v = max_nan(v, buf[i]);
    __syncthreads();
    return v;
}

// 1 / sqrt(v) to about an ulp: the hardware estimate and one Newton step.  The estimate takes a subnormal v for zero:
// small ones are moved up by a power of two.
__device__ __forceinline__ float inv_sqrt(float v) {
    const bool small = v < 0x1p-100f;
    v = small ? v * 0x1p+64f : v;
    const float r = __builtin_amdgcn_rsqf(v);
    const float e = fmaf(-v * r, r, 1.f);
    const float n = fmaf(r * 0.5f, e, r);
    const float x = n == n ? n : r;  // v infinite: the estimate is exact
    return small ? x * 0x1p+32f : x;
}

// A row's reciprocal deviation, as that of the row times s: s = 1, or a power of two for rows of large values, whose own
// may lie below fp32's normal range.  A normed value is (h s) (r w), which keeps its digits.
struct RowScale {
    float r, s;
    __device__ __forceinline__ float own() const { return r * s; }
};
// 1 / sqrt(mean h^2 + eps) of a row held by TPR threads; ss: the thread's share of the sum of squares.
template <int TPR, int VPT>
__device__ __forceinline__ RowScale row_rstd(const float (&h)[VPT][8], float ss, float inv_d, float eps, float* buf) {
    ss = row_sum<TPR>(ss, buf);
    if (ss < INFINITY) return {inv_sqrt(fmaf(ss, inv_d, eps)), 1.f};
    // squares past fp32 (some value is 2^64 / sqrt(D) or more): the sum of (h 2^-96)^2, at most 2^64 D; what underflows
    // is less than 2^-70 of the sum.  All threads of the row come here.
    constexpr float S = 0x1p-96f;
    float s2 = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; i++)
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const float v = h[i][j] * S;
            s2 = fmaf(v, v, s2);
        }
    const float r = inv_sqrt(fmaf(row_sum<TPR>(s2, buf), inv_d, eps * S * S));
    // rows below 2^100: their own reciprocal, far from the subnormal numbers, so that their smallest values need no scale
    return r * S >= 0x1p-100f ? RowScale{r * S, 1.f} : RowScale{r, S};
}

// Whether rows `stride` elements apart all start on 16 bytes.
inline bool row16(const void* p, int64_t stride, size_t es) { return !p || ((uintptr_t)p % 16 == 0 && (stride * es) % 16 == 0); }

}  // namespace la
