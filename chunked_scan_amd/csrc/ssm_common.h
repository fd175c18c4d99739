// ssm_common.h -- what the selective scan's forward and backward share on the host.
#pragma once
#include <algorithm>

#include "la_mixer.h"

namespace la {

// A split of every sequence into G segments of seglen tokens (a multiple of `unit` when G > 1): as many
// as bring the channel blocks to about `waves` waves, none shorter than `least` tokens.
struct SsmPlan {
    int G;
    int64_t seglen;
};
inline SsmPlan ssm_plan(int64_t B, int64_t L, int64_t D, int64_t waves, int64_t least, int64_t unit) {
    const int64_t w = B * ((D + 63) / 64);
    const int64_t G = std::min(w > 0 ? (waves + w - 1) / w : 1, L / least);
    if (G <= 1) return {1, L};
    const int64_t seglen = ((L + G - 1) / G + unit - 1) / unit * unit;
    return {(int)((L + seglen - 1) / seglen), seglen};
}

// Packs B and C as fp32 [B, L, 2 NP] and A log2(e) as [NP, D], zeros behind N (ssm_scan.hip).
void launch_pack(const SsmArgs& a, float* bc, float* a2, int NP);

// The recurrence over a sequence's segments of one state element, x_{k+1} = 2^(rate s_k) x_k + v_k for
// k < K from x_0, done by PARTS threads: each composes its share of the steps (sum of s, result from zero), the
// maps are chained through LDS, and each applies its steps.  A block holds 64 elements, a wave per share, so
// that a step's accesses are contiguous.  at(k): where v_k is; s_at(k): where s_k is.  The thread with step k
// calls put(k, x_k, x_{k+1}).  `on`: whether the thread's element exists.
constexpr int SEG_BATCH = 16;  // loads in flight
template <int PARTS, typename V, typename S, typename Put>
__device__ __forceinline__ void segment_chain(int K, float x0, float rate, bool on, V at, S s_at, Put put) {
    __shared__ float map_y[PARTS][64], map_s[PARTS][64];
    const int el = threadIdx.x & 63, part = uniform(threadIdx.x >> 6);
    const int per = (K + PARTS - 1) / PARTS, k0 = part * per, k1 = min(k0 + per, K);
    float v[SEG_BATCH], s[SEG_BATCH];
    auto load = [&](int k) {
#pragma unroll
        for (int j = 0; j < SEG_BATCH; j++)
            if (k + j < k1) {
                v[j] = *at(k + j);
                s[j] = *s_at(k + j);
            }
    };
    float y = 0.f, sum = 0.f;
    for (int k = k0; k < k1; k += SEG_BATCH) {
        load(k);
#pragma unroll
        for (int j = 0; j < SEG_BATCH; j++)
            if (k + j < k1) {
                y = fmaf(__builtin_amdgcn_exp2f(rate * s[j]), y, v[j]);
                sum += s[j];
            }
    }
    map_y[part][el] = y;
    map_s[part][el] = sum;
    __syncthreads();
    float x = x0;
    for (int q = 0; q < part; q++) x = fmaf(__builtin_amdgcn_exp2f(rate * map_s[q][el]), x, map_y[q][el]);
    for (int k = k0; k < k1; k += SEG_BATCH) {
        if (per > SEG_BATCH) load(k);  // else the first load's values are still there
#pragma unroll
        for (int j = 0; j < SEG_BATCH; j++)
            if (k + j < k1) {
                const float next = fmaf(__builtin_amdgcn_exp2f(rate * s[j]), x, v[j]);
                if (on) put(k + j, x, next);
                x = next;
            }
    }
}
// Shares per element: 16 where there are few elements (and then many segments), else 4.
inline int segment_parts(int64_t elements) { return elements <= 8192 ? 16 : 4; }

}  // namespace la
