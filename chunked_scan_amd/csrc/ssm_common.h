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

// Whether every row of a view starts on 16 bytes.
inline bool rows16(const void* p, const la_rows& r, size_t es) {
    return !p || ((uintptr_t)p % 16 == 0 && (r.batch * es) % 16 == 0 && (r.token * es) % 16 == 0);
}

// Packs B and C as fp32 [B, L, 2 NP] and A log2(e) as [NP, D], zeros behind N (ssm_scan.hip).
void launch_pack(const SsmArgs& a, float* bc, float* a2, int NP);

}  // namespace la
