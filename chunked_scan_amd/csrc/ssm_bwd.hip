// ssm_bwd.hip -- the selective scan's backward pass.
//
// With ds_t = dy_t silu(z_t), W_t = a_t S_{t-1} = S_t - delta_t u_t B_t and the adjoint of the state
//   G_t = C_t ds_t + a_{t+1} G_{t+1}          (G after the last token: ds_out)
// the derivatives are
//   du = D ds + delta sum_n G B,   d delta = u sum_n G B + sum_n G W A,   dA = sum_t G W delta,
//   dB_t[n] = sum_d G delta u,     dC_t[n] = sum_d ds S,                  dz = dy (C S + D u) silu'(z).
//
// Passes.  Sequences are cut into G segments as in the forward.
//   1. states: per segment, in token order: the state from zero, kept every T tokens (with the sum of
//      delta up to there), and the segment's contribution sum_t (prod_{s <= t} a_s) C_t ds_t to the
//      adjoint entering it from behind; both share the exponentials.
//   2. segments: the scan over segments, forwards for states and backwards for adjoints.
//   3. main: per segment, T tokens at a time from the end: the exact state at the T tokens' start
//      (kept state + decayed incoming state of the segment), the T states recomputed into registers,
//      then the adjoint walked back through them.
//   4. sums: dB and dC over the channel blocks' partial sums, dA, dD and d dt_bias over the segments'.
//
// A lane owns a channel as in the forward, so the sums over channels cross lanes: 32 values a token (16
// key dims of dB and of dC) over 64 lanes, by halving: every exchange adds two registers into one, and
// after five of them each pair of lanes holds one value (about 70 instructions against 350 of the
// recurrence).  The main pass takes 16 key dims at a time; with more, the sums over n that du, d delta and dz
// need are carried in the workspace from one group of 16 to the next.
#include "la_mixer.h"
#include "ssm_common.h"
#include "ssm_tile.h"

namespace la {
namespace {

constexpr int T = TT;      // tokens per tile: the states at their starts are kept
constexpr int TH = T / 2;  // tokens whose states are recomputed into registers together
constexpr int NC = 16;  // key dims per group

struct BwdDev {
    const void* u;
    const void* dt;
    const void* z;
    const void* dy;
    const float* a2;  // [NP, D] rates times log2(e)
    const float* Dskip;
    const float* dt_bias;
    const float* ds_out;
    const int32_t* lengths;
    const float* bc;  // [B, L, 2 NP]
    float* hin;       // [B, G, NP, D]: states entering the segments (pass 1 writes g + 1)
    float* gout;      // [B, G, NP, D]: adjoints at the segments' ends (pass 1 writes g: its contribution)
    float* sumdt;     // [B, G, D]
    float* kept;      // [B, nk, NP, D]: states from the segment's start, every T tokens
    float* keptdt;    // [B, nk, D]
    float* acc;       // NP > 16: [3][B, L, D] sums over the groups so far
    float* dbc;       // [cb, B, L, 2 NP]
    float* dap;       // [B, G, NP, D]
    float* ddp;       // [B, G, 2, D]: dD, d dt_bias
    float* ds_in;
    void* du;
    void* ddt;
    void* dz;
    int64_t B, L, D, seglen, nk;
    int N, NP, G;
    unsigned cb;
    bool softplus;
    la_rows su, sdt, sz, sdy, sdu, sddt, sdz;
};

// Pass 1.  blockIdx.x: channel block fastest, then group of 16 key dims, segment, sequence.  Tiles as in the
// forward: tokens behind the segment's end have delta = ds = 0.
template <typename E, bool VEC>
__global__ __launch_bounds__(64) void ssm_bwd_states_kernel(BwdDev p) {
    __shared__ __align__(16) E tile[4][T * 64];  // u, dt, dy, z
    const unsigned ngr = p.NP / NC;
    unsigned r = blockIdx.x / p.cb;
    const int64_t d0 = (int64_t)(blockIdx.x % p.cb) * 64;
    const int nb = (int)(r % ngr) * NC;
    r /= ngr;
    const int g = (int)(r % p.G);
    const int64_t b = r / p.G;
    const int lane = threadIdx.x;
    const bool live = d0 + lane < p.D;
    const int64_t d = live ? d0 + lane : p.D - 1;
    const TilePlace pl(d0, p.D);
    const int t0 = (int)(g * p.seglen), t1 = min(t0 + (int)p.seglen, uniform((int)seq_len(p.lengths, b, p.L)));

    float h[NC], A2[NC], q[NC], adj[NC];
#pragma unroll
    for (int n = 0; n < NC; n++) {
        A2[n] = p.a2[(nb + n) * p.D + d];
        h[n] = 0.f;
        q[n] = 1.f;
        adj[n] = 0.f;
    }
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.f;
    const bool gate = p.z;
    const E* ub = (const E*)p.u + b * p.su.batch + d0;
    const E* xb = (const E*)p.dt + b * p.sdt.batch + d0;
    const E* yb = (const E*)p.dy + b * p.sdy.batch + d0;
    const E* zb = gate ? (const E*)p.z + b * p.sz.batch + d0 : nullptr;
    scalar_f32 row = as_scalar(p.bc + (b * p.L + t0) * (2 * p.NP) + nb);

    Raw8<E> raw[4];
    auto fetch = [&](int t) {
        const int tt = min(t + pl.token, t1 - 1);
        raw[0] = tile_load<E, VEC>(ub, p.su.token, tt, pl);
        raw[1] = tile_load<E, VEC>(xb, p.sdt.token, tt, pl);
        raw[2] = tile_load<E, VEC>(yb, p.sdy.token, tt, pl);
        if (gate) raw[3] = tile_load<E, VEC>(zb, p.sz.token, tt, pl);
    };
    float sum = 0.f;
    float* kp = p.kept + ((b * p.nk + t0 / T) * p.NP + nb) * p.D + d;
    float* kd = p.keptdt + (b * p.nk + t0 / T) * p.D + d;
    if (t0 < t1) fetch(t0);
    for (int t = t0; t < t1; t += T) {
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (i < 3 || gate) *lds_chunk(tile[i], pl) = raw[i];
        wave_lds_fence();
        float dl[T], du[T], ds[T];
#pragma unroll
        for (int j = 0; j < T; j++) dl[j] = (float)tile[1][j * 64 + lane] + bias;
        if (p.softplus) {
#pragma unroll
            for (int j = 0; j < T; j++) dl[j] = softplus<false>(dl[j], nullptr);
        }
#pragma unroll
        for (int j = 0; j < T; j++) {
            const bool in = t + j < t1;
            dl[j] = in ? dl[j] : 0.f;
            du[j] = dl[j] * (float)tile[0][j * 64 + lane];
            ds[j] = in ? (float)tile[2][j * 64 + lane] : 0.f;
        }
        if (gate) {
#pragma unroll
            for (int j = 0; j < T; j++) {
                const float z = (float)tile[3][j * 64 + lane];
                ds[j] *= z * sigmoid(z);
            }
        }
        if (t + T < t1) fetch(t + T);
        if (t > t0 && live) {
#pragma unroll
            for (int n = 0; n < NC; n++) kp[n * p.D] = h[n];
            if (nb == 0) *kd = sum;
        }
        kp += (int64_t)p.NP * p.D;
        kd += p.D;
#pragma unroll
        for (int j = 0; j < T; j++) {
#pragma unroll
            for (int n = 0; n < NC; n++) {
                const float a = __builtin_amdgcn_exp2f(dl[j] * A2[n]);
                h[n] = fmaf(a, h[n], du[j] * row[n]);
                q[n] *= a;
                adj[n] = fmaf(q[n], ds[j] * row[p.NP + n], adj[n]);
            }
            sum += dl[j];
            row += t + j + 1 < t1 ? 2 * p.NP : 0;
        }
    }
    if (!live) return;
#pragma unroll
    for (int n = 0; n < NC; n++) {
        if (g + 1 < p.G) p.hin[((b * p.G + g + 1) * p.NP + nb + n) * p.D + d] = h[n];
        p.gout[((b * p.G + g) * p.NP + nb + n) * p.D + d] = adj[n];
    }
    if (nb == 0) p.sumdt[(b * p.G + g) * p.D + d] = sum;
}

// Pass 2.  A thread owns one (b, n, d): states forwards, adjoints backwards.  hin[0] takes s_in and
// hin[g] the state entering segment g; gout[g] becomes the adjoint at segment g's end.
constexpr int PB = 32;
__global__ __launch_bounds__(256) void ssm_bwd_segments_kernel(const float* __restrict__ a2, const float* __restrict__ s_in,
                                                               const float* __restrict__ ds_out,
                                                               const float* __restrict__ sumdt, float* __restrict__ hin,
                                                               float* __restrict__ gout, int64_t total, int64_t D, int N,
                                                               int NP, int G) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const int64_t d = i % D, n = i / D % NP, b = i / (D * NP);
    const bool on = n < N;
    const int64_t io = (b * N + n) * D + d;
    const float rate = a2[n * D + d];
    const int64_t ps = (int64_t)NP * D;
    const float* sp = sumdt + b * G * D + d;
    if (blockIdx.y == 0) {
        float h = on && s_in ? s_in[io] : 0.f;
        float* pp = hin + (b * G * NP + n) * D + d;
        pp[0] = h;
        for (int g0 = 1; g0 < G; g0 += PB) {
            float v[PB], s[PB];
#pragma unroll
            for (int j = 0; j < PB; j++) {
                const int g = min(g0 + j, G - 1);
                v[j] = pp[g * ps];
                s[j] = sp[(g - 1) * D];
            }
#pragma unroll
            for (int j = 0; j < PB; j++)
                if (g0 + j < G) {
                    h = fmaf(__builtin_amdgcn_exp2f(rate * s[j]), h, v[j]);
                    pp[(g0 + j) * ps] = h;
                }
        }
    } else {
        float x = on && ds_out ? ds_out[io] : 0.f;
        float* pp = gout + (b * G * NP + n) * D + d;
        for (int g0 = G - 1; g0 >= 0; g0 -= PB) {
            float v[PB], s[PB];
#pragma unroll
            for (int j = 0; j < PB; j++) {
                const int g = max(g0 - j, 0);
                v[j] = pp[g * ps];
                s[j] = sp[g * D];
            }
#pragma unroll
            for (int j = 0; j < PB; j++)
                if (g0 - j >= 0) {
                    pp[(g0 - j) * ps] = x;
                    x = fmaf(__builtin_amdgcn_exp2f(rate * s[j]), x, v[j]);
                }
        }
    }
}

// The same value, unknown to the compiler: keeps it from holding on to exponentials of one phase for the next,
// for which there are no registers.
__device__ __forceinline__ float opaque(float x) {
    asm("" : "+v"(x));
    return x;
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}

// The sums of v[0..15] over the wave's 64 lanes: lane l returns the sum of v[l >> 2].  Four exchanges that
// halve the registers (across 32 lanes, across 16, then inside rows of 16: rotate by 8, mirror of 8), then
// two additions inside groups of four lanes.
__device__ __forceinline__ float wave_sums16(float* v) {
    const int l = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]), __float_as_uint(v[i + 8]), false, false);
        v[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[i]), __float_as_uint(v[i + 4]), false, false);
        v[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const float keep = l & 8 ? v[i + 2] : v[i], send = l & 8 ? v[i] : v[i + 2];
        v[i] = keep + dpp<0x128>(send);  // row_ror:8
    }
    const float keep = l & 4 ? v[1] : v[0], send = l & 4 ? v[0] : v[1];
    float s = keep + dpp<0x141>(send);  // row_half_mirror
    s += dpp<0x4e>(s);                  // quad_perm [2, 3, 0, 1]
    return s + dpp<0xb1>(s);            // quad_perm [1, 0, 3, 2]
}

// Pass 3.  blockIdx.x: channel block fastest, then segment, sequence.  MULTI: more than one group of 16 key dims.
// A wave per segment and channel block, at most 256 registers (two waves per SIMD): the T states of 16 key
// dims take 128 of them, so what is used once per token waits in LDS.
template <typename E, bool MULTI, bool VEC>
__global__ __launch_bounds__(64, 2) void ssm_bwd_main_kernel(BwdDev p) {
    __shared__ __align__(16) E tile[4][T * 64];  // u; dt, then d dt; dy, then du; z, then dz
    __shared__ float slope[T * 64];              // d delta / d dt
    __shared__ float hin[NC * 64], h0[NC * 64];  // the states entering the segment and the tile
    const unsigned r = blockIdx.x / p.cb;
    const unsigned cbi = blockIdx.x % p.cb;
    const int64_t d0 = (int64_t)cbi * 64;
    const int g = (int)(r % p.G);
    const int64_t b = r / p.G;
    const int lane = threadIdx.x;
    const bool live = d0 + lane < p.D;
    const int64_t d = live ? d0 + lane : p.D - 1;
    const TilePlace pl(d0, p.D);
    const int len = uniform((int)seq_len(p.lengths, b, p.L));
    const int t0 = (int)(g * p.seglen), te = (int)min(t0 + p.seglen, p.L), t1 = min(te, len);
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.f;
    const float skip = p.Dskip ? p.Dskip[d] : 0.f;
    const bool gate = p.z;
    const E* ub = (const E*)p.u + b * p.su.batch + d0;
    const E* xb = (const E*)p.dt + b * p.sdt.batch + d0;
    const E* yb = (const E*)p.dy + b * p.sdy.batch + d0;
    const E* zb = gate ? (const E*)p.z + b * p.sz.batch + d0 : nullptr;
    E* dub = (E*)p.du + b * p.sdu.batch + d0;
    E* dxb = (E*)p.ddt + b * p.sddt.batch + d0;
    E* dzb = gate ? (E*)p.dz + b * p.sdz.batch + d0 : nullptr;

    if (pl.in) {  // gradients behind the sequence's end
        const Raw8<E> zero = {};
        for (int t = max(t0, len) + pl.token; t < te; t += T) {
            store8<VEC>(dub + t * p.sdu.token + pl.col, pl.n, zero);
            store8<VEC>(dxb + t * p.sddt.token + pl.col, pl.n, zero);
            if (gate) store8<VEC>(dzb + t * p.sdz.token + pl.col, pl.n, zero);
        }
    }

    const int64_t plane = p.B * p.L * p.D;
    float dDsum = 0.f, dbsum = 0.f;
    const int groups = MULTI ? p.NP / NC : 1;
    for (int gr = 0; gr < groups; gr++) {
        const int nb = gr * NC;
        const bool first = gr == 0, last = gr == groups - 1;
        float A2[NC], adj[NC], dA[NC], kept[NC], keptdt = 0.f;
        const int64_t sg = ((b * p.G + g) * p.NP + nb) * p.D + d;
        wave_lds_fence();
#pragma unroll
        for (int n = 0; n < NC; n++) {
            A2[n] = p.a2[(nb + n) * p.D + d];
            adj[n] = p.gout[sg + n * p.D];
            hin[n * 64 + lane] = p.hin[sg + n * p.D];
            dA[n] = 0.f;
            kept[n] = 0.f;
        }
        Raw8<E> raw[4];
        auto fetch = [&](int t) {
            const int tt = min(t + pl.token, t1 - 1);
            raw[0] = tile_load<E, VEC>(ub, p.su.token, tt, pl);
            raw[1] = tile_load<E, VEC>(xb, p.sdt.token, tt, pl);
            raw[2] = tile_load<E, VEC>(yb, p.sdy.token, tt, pl);
            if (gate) raw[3] = tile_load<E, VEC>(zb, p.sz.token, tt, pl);
        };
        auto fetch_kept = [&](int t) {
            const int64_t kk = b * p.nk + t / T;
#pragma unroll
            for (int n = 0; n < NC; n++) kept[n] = t > t0 ? p.kept[(kk * p.NP + nb + n) * p.D + d] : 0.f;
            keptdt = t > t0 ? p.keptdt[kk * p.D + d] : 0.f;
        };
        scalar_f32 bcb = as_scalar(p.bc + b * p.L * (2 * p.NP) + nb);
        const int tl = t0 + (t1 - 1 - t0) / T * T;  // the segment's last tile
        if (t0 < t1) {
            fetch(tl);
            fetch_kept(tl);
        }
        for (int t = tl; t >= t0 && t0 < t1; t -= T) {
            wave_lds_fence();
#pragma unroll
            for (int i = 0; i < 4; i++)
                if (i < 3 || gate) *lds_chunk(tile[i], pl) = raw[i];
            wave_lds_fence();
            float dl[T], ds[T], hs[TH][NC], h[NC];
#pragma unroll
            for (int j = 0; j < T; j++) dl[j] = (float)tile[1][j * 64 + lane] + bias;
            if (p.softplus) {
#pragma unroll
                for (int j = 0; j < T; j++) {
                    float sl;
                    dl[j] = softplus<true>(dl[j], &sl);
                    slope[j * 64 + lane] = sl;
                }
            } else {
#pragma unroll
                for (int j = 0; j < T; j++) slope[j * 64 + lane] = 1.f;
            }
#pragma unroll
            for (int j = 0; j < T; j++) {
                const bool in = t + j < t1 && live;  // the others change no state and add nothing to a sum
                dl[j] = in ? dl[j] : 0.f;
                ds[j] = in ? (float)tile[2][j * 64 + lane] : 0.f;
            }
            // the state entering the tile
#pragma unroll
            for (int n = 0; n < NC; n++) {
                h[n] = fmaf(__builtin_amdgcn_exp2f(A2[n] * keptdt), hin[n * 64 + lane], kept[n]);
                h0[n * 64 + lane] = h[n];
            }
            // the tile's halves from the end: forwards to the half's states, then backwards through them
#pragma unroll
            for (int j0 = T - TH; j0 >= 0; j0 -= TH) {
#pragma unroll
                for (int j = 0; j < j0; j++) {
                    const float du = dl[j] * (float)tile[0][j * 64 + lane];
                    scalar_f32 row = bcb + min(t + j, t1 - 1) * (2 * p.NP);
                    const float dlj = opaque(dl[j]);
#pragma unroll
                    for (int n = 0; n < NC; n++) h[n] = fmaf(__builtin_amdgcn_exp2f(dlj * A2[n]), h[n], du * row[n]);
                }
                if (j0 == 0) {
#pragma unroll
                    for (int n = 0; n < NC; n++) h[n] = h0[n * 64 + lane];
                }
#pragma unroll
                for (int k = 0; k < TH; k++) {
                    const int j = j0 + k;
                    const float u = (float)tile[0][j * 64 + lane], du = dl[j] * u;
                    scalar_f32 row = bcb + min(t + j, t1 - 1) * (2 * p.NP);
                    float inner = 0.f;
#pragma unroll
                    for (int n = 0; n < NC; n++) {
                        h[n] = fmaf(__builtin_amdgcn_exp2f(dl[j] * A2[n]), h[n], du * row[n]);
                        hs[k][n] = h[n];
                        inner = fmaf(row[p.NP + n], h[n], inner);
                    }
                    if (gate) {
                        const float z = (float)tile[3][j * 64 + lane], sz = sigmoid(z), dyv = ds[j];
                        ds[j] *= z * sz;
                        if (MULTI) {
                            float* ap = p.acc + 2 * plane + (b * p.L + min(t + j, t1 - 1)) * p.D + d;
                            if (!first) inner += *ap;
                            if (!last && live && t + j < t1) *ap = inner;
                        }
                        if (last)
                            io<E>::st(tile[3] + j * 64 + lane, dyv * fmaf(skip, u, inner) * sz * fmaf(z, 1.f - sz, 1.f));
                    }
                }
                if (j0 == 0 && t > t0) {
                    fetch(t - T);
                    fetch_kept(t - T);
                }
#pragma unroll
                for (int k = TH - 1; k >= 0; k--) {
                    const int j = j0 + k;
                    const int tt = min(t + j, t1 - 1);
                    scalar_f32 row = bcb + tt * (2 * p.NP);
                    const float u = (float)tile[0][j * 64 + lane];
                    const float du = dl[j] * u;
                    const float dlj = opaque(dl[j]);
                    float s1 = 0.f, s2 = 0.f, v[NC];
#pragma unroll
                    for (int n = 0; n < NC; n++) v[n] = ds[j] * hs[k][n];
                    const float sc = wave_sums16(v);
#pragma unroll
                    for (int n = 0; n < NC; n++) {
                        const float gn = fmaf(ds[j], row[p.NP + n], adj[n]);
                        const float gw = gn * fmaf(-du, row[n], hs[k][n]);
                        s1 = fmaf(gn, row[n], s1);
                        s2 = fmaf(gw, A2[n], s2);
                        dA[n] = fmaf(gw, dl[j], dA[n]);
                        v[n] = gn * du;
                        adj[n] = gn * __builtin_amdgcn_exp2f(dlj * A2[n]);
                    }
                    const float sb = wave_sums16(v);
                    // lanes 4 i and 4 i + 1 write the sums of dB and dC of key dim i
                    if (t + j < t1 && (lane & 2) == 0)
                        p.dbc[((cbi * p.B + b) * p.L + tt) * (2 * p.NP) + nb + (lane >> 2) + (lane & 1) * p.NP] =
                            lane & 1 ? sc : sb;
                    if (MULTI) {
                        float* ap = p.acc + (b * p.L + tt) * p.D + d;
                        if (!first) {
                            s1 += ap[0];
                            s2 += ap[plane];
                        }
                        if (!last && live && t + j < t1) {
                            ap[0] = s1;
                            ap[plane] = s2;
                        }
                    }
                    if (last) {
                        const float dd = t + j < t1 && live ? fmaf(u, s1, s2 * LN2) * slope[j * 64 + lane] : 0.f;
                        io<E>::st(tile[2] + j * 64 + lane, fmaf(ds[j], skip, dl[j] * s1));
                        io<E>::st(tile[1] + j * 64 + lane, dd);
                        dDsum = fmaf(ds[j], u, dDsum);
                        dbsum += dd;
                    }
                }
            }
            if (last) {
                wave_lds_fence();
                const int tt = t + pl.token;
                if (pl.in && tt < t1) {
                    store8<VEC>(dub + tt * p.sdu.token + pl.col, pl.n, *lds_chunk(tile[2], pl));
                    store8<VEC>(dxb + tt * p.sddt.token + pl.col, pl.n, *lds_chunk(tile[1], pl));
                    if (gate) store8<VEC>(dzb + tt * p.sdz.token + pl.col, pl.n, *lds_chunk(tile[3], pl));
                }
            }
        }
        if (live) {
#pragma unroll
            for (int n = 0; n < NC; n++) {
                p.dap[sg + n * p.D] = dA[n];
                if (g == 0 && p.ds_in && nb + n < p.N) p.ds_in[(b * p.N + nb + n) * p.D + d] = adj[n];
            }
        }
    }
    if (live) {
        p.ddp[((b * p.G + g) * 2) * p.D + d] = dDsum;
        p.ddp[((b * p.G + g) * 2 + 1) * p.D + d] = dbsum;
    }
}

// Pass 4.  The first `nbc` blocks: dB and dC, a thread per (b, t, n) of each; the others: dA, dD and
// d dt_bias, a thread per (n or one of the two, d).
template <typename E>
__global__ __launch_bounds__(256) void ssm_bwd_sums_kernel(const float* __restrict__ dbc, const float* __restrict__ dap,
                                                           const float* __restrict__ ddp, const int32_t* lengths,
                                                           E* __restrict__ dB, E* __restrict__ dC, float* __restrict__ dA,
                                                           float* __restrict__ dD, float* __restrict__ dbias, la_rows sdb,
                                                           la_rows sdc, int64_t B, int64_t L, int64_t D, int N, int NP, int G,
                                                           unsigned cb, unsigned nbc) {
    if (blockIdx.x < nbc) {
        const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
        const int64_t row = i / (2 * NP);
        const int j = (int)(i % (2 * NP));
        if (row >= B * L) return;
        const int n = j < NP ? j : j - NP;
        if (n >= N) return;
        const int64_t b = row / L, t = row % L;
        float s = 0.f;
        if (t < seq_len(lengths, b, L)) {
            const int64_t plane = B * L * (2 * NP);
#pragma unroll 8
            for (unsigned c = 0; c < cb; c++) s += dbc[c * plane + i];
        }
        if (j < NP)
            io<E>::st(dB + b * sdb.batch + t * sdb.token + n, s);
        else
            io<E>::st(dC + b * sdc.batch + t * sdc.token + n, s);
        return;
    }
    const int64_t i = (int64_t)(blockIdx.x - nbc) * 256 + threadIdx.x;
    const int64_t n = i / D, d = i % D;
    if (n >= N + 2) return;
    const bool isA = n < N;
    const float* src = isA ? dap + n * D + d : ddp + (n - N) * D + d;
    const int64_t step = isA ? (int64_t)NP * D : 2 * D;
    float s = 0.f;
#pragma unroll 8
    for (int64_t k = 0; k < B * G; k++) s += src[k * step];
    if (isA)
        dA[d * N + n] = s;
    else if (n == N) {
        if (dD) dD[d] = s;
    } else if (dbias)
        dbias[d] = s;
}

int np_for(int N) { return (N + NC - 1) / NC * NC; }

// Segments: about 2048 waves in the main pass, none under 16 tokens.
SsmPlan bwd_plan(int64_t B, int64_t L, int64_t D) { return ssm_plan(B, L, D, 2048, 16, T); }

struct BwdWs {
    float *bc, *a2, *hin, *gout, *sumdt, *kept, *keptdt, *acc, *dbc, *dap, *ddp;
    int64_t nk;
    size_t bytes;
};
BwdWs bwd_cut(void* base, int64_t B, int64_t L, int64_t D, int N, int G) {
    WsCut c{(char*)base};
    BwdWs w;
    const int NP = np_for(N);
    const size_t seg = (size_t)(B * G) * D, tok = (size_t)(B * L);
    w.nk = (L + T - 1) / T;
    w.bc = c.take(tok * 2 * NP);
    w.a2 = c.take((size_t)NP * D);
    w.hin = c.take(seg * NP);
    w.gout = c.take(seg * NP);
    w.sumdt = c.take(seg);
    w.kept = c.take((size_t)(B * w.nk) * NP * D);
    w.keptdt = c.take((size_t)(B * w.nk) * D);
    w.acc = NP > NC ? c.take(tok * D * 3) : nullptr;
    w.dbc = c.take(tok * 2 * NP * ((D + 63) / 64));
    w.dap = c.take(seg * NP);
    w.ddp = c.take(seg * 2);
    w.bytes = c.used;
    return w;
}

template <typename E>
hipError_t launch_e(const SsmArgs& a) {
    const SsmPlan pl = bwd_plan(a.B, a.L, a.D);
    const BwdWs w = bwd_cut(a.ws, a.B, a.L, a.D, a.N, pl.G);
    BwdDev p;
    p.u = a.u; p.dt = a.dt; p.z = a.z; p.dy = a.dy; p.a2 = w.a2; p.Dskip = a.Dskip; p.dt_bias = a.dt_bias;
    p.ds_out = a.ds_out; p.lengths = a.lengths;
    p.bc = w.bc; p.hin = w.hin; p.gout = w.gout; p.sumdt = w.sumdt; p.kept = w.kept; p.keptdt = w.keptdt;
    p.acc = w.acc; p.dbc = w.dbc; p.dap = w.dap; p.ddp = w.ddp;
    p.ds_in = a.ds_in; p.du = a.du; p.ddt = a.ddt; p.dz = a.dz;
    p.B = a.B; p.L = a.L; p.D = a.D; p.seglen = pl.seglen; p.nk = w.nk;
    p.N = a.N; p.NP = np_for(a.N); p.G = pl.G;
    p.cb = (unsigned)((a.D + 63) / 64);
    p.softplus = a.softplus;
    p.su = a.su; p.sdt = a.sdt; p.sz = a.sz; p.sdy = a.sdy; p.sdu = a.sdu; p.sddt = a.sddt; p.sdz = a.sdz;
    const unsigned blocks = p.cb * (unsigned)pl.G * (unsigned)a.B;
    if (a.B > 0 && a.D > 0) {
        launch_pack(a, w.bc, w.a2, p.NP);
        const size_t es = sizeof(E);
        const bool vec = a.D % 8 == 0 && rows16(a.u, a.su, es) && rows16(a.dt, a.sdt, es) && rows16(a.z, a.sz, es) &&
                         rows16(a.dy, a.sdy, es) && rows16(a.du, a.sdu, es) && rows16(a.ddt, a.sddt, es) &&
                         rows16(a.dz, a.sdz, es);
        if (vec)
            LA_TRACED(a.tr, "ssm_bwd_states", ssm_bwd_states_kernel<E, true><<<blocks * (p.NP / NC), 64, 0, a.stream>>>(p));
        else
            LA_TRACED(a.tr, "ssm_bwd_states", ssm_bwd_states_kernel<E, false><<<blocks * (p.NP / NC), 64, 0, a.stream>>>(p));
        const int64_t total = a.B * p.NP * a.D;
        LA_TRACED(a.tr, "ssm_bwd_segments",
                  ssm_bwd_segments_kernel<<<dim3((unsigned)((total + 255) / 256), 2), 256, 0, a.stream>>>(
                      w.a2, a.s_in, a.ds_out, w.sumdt, w.hin, w.gout, total, a.D, a.N, p.NP, pl.G));
#define LA_SSM_MAIN(M, V) \
    LA_TRACED(a.tr, "ssm_bwd_main", ssm_bwd_main_kernel<E, M, V><<<blocks, 64, 0, a.stream>>>(p))
        if (p.NP > NC) {
            if (vec) LA_SSM_MAIN(true, true);
            else LA_SSM_MAIN(true, false);
        } else {
            if (vec) LA_SSM_MAIN(false, true);
            else LA_SSM_MAIN(false, false);
        }
#undef LA_SSM_MAIN
    }
    const unsigned nbc = (unsigned)((a.B * a.L * 2 * p.NP + 255) / 256);
    const unsigned nd = (unsigned)((a.D * (a.N + 2) + 255) / 256);
    if (nbc + nd > 0)
        LA_TRACED(a.tr, "ssm_bwd_sums",
                  ssm_bwd_sums_kernel<E><<<nbc + nd, 256, 0, a.stream>>>(w.dbc, w.dap, w.ddp, a.lengths, (E*)a.dB, (E*)a.dC,
                                                                         a.dA, a.dD, a.d_dt_bias, a.sdb, a.sdc, a.B, a.L,
                                                                         a.D, a.N, p.NP, pl.G, p.cb, nbc));
    return hipGetLastError();
}

}  // namespace

size_t ssm_bwd_ws(int64_t B, int64_t L, int64_t D, int N) {
    return bwd_cut(nullptr, B, L, D, N, bwd_plan(B, L, D).G).bytes;
}

hipError_t launch_ssm_scan_bwd(const SsmArgs& a) { return a.bf16 ? launch_e<__bf16>(a) : launch_e<float>(a); }

}  // namespace la
