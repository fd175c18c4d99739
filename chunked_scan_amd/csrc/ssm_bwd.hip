// ssm_bwd.hip -- the selective scan's backward pass.
//
// With ds_t = dy_t silu(z_t), W_t = a_t S_{t-1} and the adjoint of the state
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
// A lane owns a channel as in the forward.  The main pass needs a token's states again on the way back,
// which costs registers: a workgroup is NP / 8 waves on the same 64 channels, 8 key dims each, so that the
// 8 x 8 states of a tile fit beside the rest at two (fp32) or three (bf16) waves per SIMD.  What concerns a
// token and not a key dim (step size, gate, the finished gradients) is computed by one of the waves per token and
// passed through LDS.
// The sums over channels cross lanes: 16 values a token and wave (8 key dims of dB and of dC) over 64 lanes, by
// halving: every exchange adds two registers into one (about 35 instructions against 170 of the recurrence).
//
// Bound by vector issue: the decays' exponentials are formed once in pass 1 and twice in pass
// 3, which has no registers to keep them at three waves per SIMD (kept, at two waves, 330 us against 312 in the
// same session).  2 x 4096 tokens x 2048 channels, N = 16, bf16 with a gate: packing 5 us, states 98, segments 13,
// main 275 to 291 (the vector units busy 78 % of the time), sums 13.  What it must read and write is 55 us at a copy's
// rate; the kept states (0.5 N bytes per token and channel, written by pass 1 and read by pass 3, 134 MB each way) and the
// partial sums of dB and dC (N / 8 bytes, 34 MB each way) are as much again and half, under the arithmetic.
#include "la_mixer.h"
#include "ssm_common.h"
#include "ssm_tile.h"

namespace la {
namespace {

constexpr int T = TT;  // tokens per tile: the states at their starts are kept
constexpr int NW8 = 8;  // key dims per wave of the main pass

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
    float* dbc;       // [cb, B, L, 2 NP]
    float* dap;       // [B, G, NP, D]
    float* ddp;       // [B, G, NP / 8, 2, D]: dD, d dt_bias
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

// The kernel's arguments, read again from memory where they are used: held over the token loops they would
// push each other and the rows of B and C out of the scalar registers.
typedef const __attribute__((address_space(4))) BwdDev* BwdArgsPtr;
__device__ __forceinline__ BwdArgsPtr bwd_args() {
    BwdArgsPtr q = (BwdArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(q));
    return q;
}

// Pass 1.  blockIdx.x: channel block fastest, then group of NC key dims, segment, sequence.  Tiles as in the
// forward: tokens behind the segment's end have delta = ds = 0.
// NC: key dims per group, 8 or 16.
template <typename E, int NC, bool VEC>
__global__ __launch_bounds__(64, 2) void ssm_bwd_states_kernel(BwdDev p) {
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

    // key dim nb + 4 q + i is element i of h[q]
    f32x4 h[NC / 4], q[NC / 4], adj[NC / 4];
    float A2[NC];
#pragma unroll
    for (int n = 0; n < NC; n++) {
        A2[n] = p.a2[(nb + n) * p.D + d];
        h[n / 4][n % 4] = 0.f;
        q[n / 4][n % 4] = 1.f;
        adj[n / 4][n % 4] = 0.f;
    }
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.f;
    const bool gate = p.z, sp = p.softplus;
    const int NP = p.NP;
    const float* const bcb = p.bc + b * p.L * (2 * NP) + nb;

    // B and C of the tile's tokens, value j NC + n in lane (j NC + n) % 64, and the next tile's
    constexpr int BV = T * NC / 64;
    float br[BV], cr[BV], bn[BV], cn[BV];
    const TileRow row_u(p.su, pl), row_dt(p.sdt, pl), row_dy(p.sdy, pl), row_z(p.sz, pl);
    Raw8<E> raw[4];
    auto fetch = [&](int t) {
        const BwdArgsPtr q = bwd_args();
        const int left = t1 - t;
        raw[0] = tile_load<E, VEC>((const E*)q->u + b * q->su.batch + t * q->su.token + d0, row_u, q->su.token, left, pl);
        raw[1] = tile_load<E, VEC>((const E*)q->dt + b * q->sdt.batch + t * q->sdt.token + d0, row_dt, q->sdt.token, left, pl);
        raw[2] = tile_load<E, VEC>((const E*)q->dy + b * q->sdy.batch + t * q->sdy.token + d0, row_dy, q->sdy.token, left, pl);
        if (gate)
            raw[3] = tile_load<E, VEC>((const E*)q->z + b * q->sz.batch + t * q->sz.token + d0, row_z, q->sz.token, left, pl);
        const float* const rows = bcb + t * (2 * NP);
#pragma unroll
        for (int v = 0; v < BV; v++) {
            const int e = v * 64 + lane;
            const int at = left >= T ? e / NC * (2 * NP) + e % NC : min(e / NC, left - 1) * (2 * NP) + e % NC;
            bn[v] = rows[at];
            cn[v] = rows[at + NP];
        }
    };
    float sum = 0.f;
    if (t0 < t1) fetch(t0);
    for (int t = t0; t < t1; t += T) {
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (i < 3 || gate) *lds_chunk(tile[i]) = raw[i];
        wave_lds_fence();
        float dl[T], du[T], ds[T];
#pragma unroll
        for (int j = 0; j < T; j++) dl[j] = (float)tile[1][j * 64 + lane] + bias;
        if (sp) {
#pragma unroll
            for (int j = 0; j < T; j++) dl[j] = softplus(dl[j]);
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
#pragma unroll
        for (int v = 0; v < BV; v++) {
            br[v] = bn[v];
            cr[v] = cn[v];
        }
        if (t + T < t1) fetch(t + T);
        if (t > t0 && live) {
            const BwdArgsPtr q = bwd_args();
            const int64_t k = b * q->nk + t / T, D = q->D;
            float* kp = q->kept + (k * NP + nb) * D + d0;
#pragma unroll
            for (int n = 0; n < NC; n++) (kp + n * D)[lane] = h[n / 4][n % 4];
            if (nb == 0) (q->keptdt + k * D + d0)[lane] = sum;
        }
        static_for<T>([&](auto J) {
            constexpr int j = J;
            static_for<NC / 4>([&](auto Q) {
                constexpr int k = Q;
                f32x4 c;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float a = __builtin_amdgcn_exp2f(dl[j] * A2[4 * k + i]);
                    c[i] = a * h[k][i];
                    q[k][i] *= a;
                }
                h[k] = outer4<j * NC + 4 * k>(br, du[j], c);
                const f32x4 x = outer4<j * NC + 4 * k>(cr, ds[j], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int i = 0; i < 4; i++) adj[k][i] = fmaf(q[k][i], x[i], adj[k][i]);
            });
            sum += dl[j];
        });
    }
    if (!live) return;
    const BwdArgsPtr e = bwd_args();
    const int64_t D = e->D, seg = b * e->G + g;
#pragma unroll
    for (int n = 0; n < NC; n++) {
        if (g + 1 < e->G) (e->hin + ((seg + 1) * NP + nb + n) * D + d0)[lane] = h[n / 4][n % 4];
        (e->gout + (seg * NP + nb + n) * D + d0)[lane] = adj[n / 4][n % 4];
    }
    if (nb == 0) (e->sumdt + seg * D + d0)[lane] = sum;
}

// Blocks along x and z, so that the threads along one dimension stay below 2^32 (many channels and key dims).
dim3 wide_grid(int64_t blocks, unsigned y) {
    const int64_t x = std::min<int64_t>(blocks, 1 << 20);
    return dim3((unsigned)x, y, (unsigned)((blocks + x - 1) / x));
}
__device__ __forceinline__ int64_t wide_block() { return (int64_t)blockIdx.z * gridDim.x + blockIdx.x; }

// Pass 2, per (b, n, d): states forwards (blockIdx.y = 0), adjoints backwards.  hin[0] takes s_in and hin[g]
// the state entering segment g; gout[g] becomes the adjoint at segment g's end.
template <int PARTS>
__global__ __launch_bounds__(64 * PARTS) void ssm_bwd_segments_kernel(const float* __restrict__ a2, const float* __restrict__ s_in,
                                                               const float* __restrict__ ds_out, const float* sumdt,
                                                               float* hin, float* gout, int64_t total, int64_t D, int N,
                                                               int NP, int G) {
    const int64_t i0 = wide_block() * 64 + (threadIdx.x & 63);
    const bool on = i0 < total;
    const int64_t i = on ? i0 : 0;
    const int64_t d = i % D, n = i / D % NP, b = i / (D * NP);
    const int64_t io = (b * N + n) * D + d, ps = (int64_t)NP * D;
    const float rate = a2[n * D + d];
    const float* sp = sumdt + b * G * D + d;
    if (blockIdx.y == 0) {
        const float x0 = n < N && s_in ? s_in[io] : 0.f;
        float* pp = hin + (b * G * NP + n) * D + d;
        if (on && threadIdx.x < 64) pp[0] = x0;
        segment_chain<PARTS>(
            G - 1, x0, rate, on, [&](int k) { return pp + (k + 1) * ps; }, [&](int k) { return sp + k * D; },
            [&](int k, float, float next) { pp[(k + 1) * ps] = next; });
    } else {
        const float x0 = n < N && ds_out ? ds_out[io] : 0.f;
        float* pp = gout + (b * G * NP + n) * D + d;
        segment_chain<PARTS>(
            G, x0, rate, on, [&](int k) { return pp + (G - 1 - k) * ps; }, [&](int k) { return sp + (G - 1 - k) * D; },
            [&](int k, float cur, float) { pp[(G - 1 - k) * ps] = cur; });
    }
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

// Pass 3.  A workgroup of NP / 8 waves per channel block (fastest), segment and sequence.  ONE: a single wave.
// Per tile, from the segment's last: the inputs to LDS | per token (shared out over the waves): step size
// and gate | every wave: forwards to its states, backwards through them, its share of the sums over key dims
// to LDS | per token: the finished gradients.  The bars are workgroup barriers.
// Waves per SIMD: what an instance needs without spilling allows two (fp32, and single waves in unaligned rows, 175 to
// 195 registers) or three (bf16, 165 and 168).  Held to three, fp32 spills up to 26: at 2 x 2048 x 2048 N = 8
// 164 -> 142 us with two, N = 16 189 -> 173, in unaligned rows (2046 channels) 225 -> 169 and 242 -> 204; 2048 x 1024,
// N = 64, the same 152.  bf16 of more than 8 key dims in unaligned rows is faster with three and 10 registers spilled
// (2 x 2048 x 2044, N = 16: 181 us, with two 202); N = 8 there 135 -> 125 with two.
template <typename E, bool VEC, bool ONE>
__global__ __launch_bounds__(ONE ? 64 : 512, sizeof(E) == 2 && !ONE ? 3 : 2) void ssm_bwd_main_kernel(BwdDev p) {
    extern __shared__ __align__(16) char lds[];
    constexpr int NC = NW8, SLOT = T * 64;
    E* const rawt = reinterpret_cast<E*>(lds);  // [2][4][SLOT], alternating: u; dt, then d dt; dy, then du; z, then dz
    float* const dls = reinterpret_cast<float*>(lds + 2 * 4 * SLOT * sizeof(E));  // [SLOT] each:
    float* const dus = dls + SLOT;    // delta u
    float* const dss = dus + SLOT;    // ds
    float* const sums = dss + SLOT;  // [waves][3][SLOT]: sum G B, sum G W A, sum C S
    const int nw = ONE ? 1 : p.NP / NC;
    const bool sp = p.softplus;
    const int w = ONE ? 0 : uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const unsigned r = blockIdx.x / p.cb;
    const unsigned cbi = blockIdx.x % p.cb;
    const int64_t d0 = (int64_t)cbi * 64;
    const int g = (int)(r % p.G);
    const int64_t b = r / p.G;
    const bool live = d0 + lane < p.D;
    const int ln = live ? lane : (int)(p.D - 1 - d0);  // lanes behind the last channel repeat it
    const int64_t d = d0 + ln;
    const TilePlace pl(d0, p.D);
    const int len = uniform((int)seq_len(p.lengths, b, p.L));
    const int t0 = (int)(g * p.seglen), te = (int)min(t0 + p.seglen, p.L), t1 = min(te, len);
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.f;
    const float skip = p.Dskip ? p.Dskip[d] : 0.f;
    const bool gate = p.z;

    if (pl.in) {  // gradients behind the sequence's end
        const Raw8<E> zero = {};
        for (int t = max(t0, len) + w * T + pl.token; t < te; t += nw * T) {
            store8<VEC>((E*)p.du + b * p.sdu.batch + d0 + t * p.sdu.token + pl.col, pl.n, zero);
            store8<VEC>((E*)p.ddt + b * p.sddt.batch + d0 + t * p.sddt.token + pl.col, pl.n, zero);
            if (gate) store8<VEC>((E*)p.dz + b * p.sdz.batch + d0 + t * p.sdz.token + pl.col, pl.n, zero);
        }
    }

    const int nb = w * NC;
    const int64_t sg = ((b * p.G + g) * p.NP + nb) * p.D + d0;
    // key dim nb + 4 q + i is element i of adj[q], hs[.][q]
    f32x4 adj[NC / 4];
    float A2[NC], dA[NC], kept[NC], hin[NC], keptdt = 0.f;
#pragma unroll
    for (int n = 0; n < NC; n++) {
        A2[n] = (p.a2 + (nb + n) * p.D + d0)[ln];
        adj[n / 4][n % 4] = (p.gout + sg + n * p.D)[ln];
        hin[n] = (p.hin + sg + n * p.D)[ln];
        dA[n] = 0.f;
        kept[n] = 0.f;
    }
    // a wave loads the activations w, w + nw, .. of u, dt, dy, z
    const int NP = nw * NC;
    const float* const bcv = p.bc + b * p.L * (2 * NP) + nb;
    float bn, cn;  // B and C of the next tile's tokens, token j and key dim n in lane 8 j + n
    Raw8<E> raw[ONE ? 4 : 2];
    auto fetch = [&](int t) {
        const BwdArgsPtr q = bwd_args();
        const int tt = min(t + pl.token, t1 - 1);
#pragma unroll
        for (int k = 0; k < (ONE ? 4 : 2); k++) {
            const int i = w + k * nw;
            if (i == 0) raw[k] = token_load<E, VEC>((const E*)q->u + b * q->su.batch + d0, q->su.token, tt, pl);
            if (i == 1) raw[k] = token_load<E, VEC>((const E*)q->dt + b * q->sdt.batch + d0, q->sdt.token, tt, pl);
            if (i == 2) raw[k] = token_load<E, VEC>((const E*)q->dy + b * q->sdy.batch + d0, q->sdy.token, tt, pl);
            if (i == 3 && gate) raw[k] = token_load<E, VEC>((const E*)q->z + b * q->sz.batch + d0, q->sz.token, tt, pl);
        }
        const float* r = bcv + min(t + lane / NC, t1 - 1) * (2 * NP) + lane % NC;
        bn = r[0];
        cn = r[NP];
    };
    auto fetch_kept = [&](int t) {
        if (t <= t0) {
#pragma unroll
            for (int n = 0; n < NC; n++) kept[n] = 0.f;
            keptdt = 0.f;
            return;
        }
        const BwdArgsPtr q = bwd_args();
        const int64_t kk = b * q->nk + t / T, D = q->D;
        const float* kp = q->kept + (kk * q->NP + nb) * D + d0;
#pragma unroll
        for (int n = 0; n < NC; n++) kept[n] = (kp + n * D)[ln];
        keptdt = (q->keptdt + kk * D + d0)[ln];
    };
    auto barrier = [&]() {
        if (ONE) wave_lds_fence();
        else lds_barrier();
    };
    auto entry = [&](int n) -> float& { return sums[(w * 3 + n / (NC / 2)) * SLOT + n % (NC / 2) * 64 + lane]; };
    scalar_f32 bcb = as_scalar_uniform(bcv);
    // where lane 4 i of the wave adds the i-th of its 16 sums over channels
    float* const dbcb = p.dbc + (cbi * p.B + b) * p.L * (2 * NP) + nb;
    const int dbco = (lane >> 2) < NC ? lane >> 2 : NP + (lane >> 2) - NC;
    float dDsum = 0.f, dbsum = 0.f;
    const int tl = t0 + (t1 - 1 - t0) / T * T;  // the segment's last tile
    int par = 0;
    if (t0 < t1) {
        fetch(tl);
        fetch_kept(tl);
    }
    for (int t = tl; t >= t0 && t0 < t1; t -= T, par ^= 1) {
        E* const tile = rawt + par * 4 * SLOT;
#pragma unroll
        for (int k = 0; k < (ONE ? 4 : 2); k++) {
            const int i = w + k * nw;
            if (i < 3 || (i == 3 && gate)) *lds_chunk(tile + i * SLOT) = raw[k];
        }
        barrier();
        for (int j = w; j < T; j += nw) {
            const int at = j * 64 + lane;
            float dl = (float)tile[SLOT + at] + bias;
            if (sp) dl = softplus(dl);
            float ds = (float)tile[2 * SLOT + at];
            if (gate) {
                const float z = (float)tile[3 * SLOT + at];
                ds *= z * sigmoid(z);
            }
            const bool in = t + j < t1 && live;  // the others change no state and add nothing to a sum
            dl = in ? dl : 0.f;
            dls[at] = dl;
            dus[at] = dl * (float)tile[at];
            dss[at] = in ? ds : 0.f;
        }
        barrier();
        // the state entering the tile, then the tile's states
        f32x4 hs[T][NC / 4], h[NC / 4];
#pragma unroll
        for (int n = 0; n < NC; n++) h[n / 4][n % 4] = fmaf(__builtin_amdgcn_exp2f(A2[n] * keptdt), hin[n], kept[n]);
        // the way back needs it again at the tile's first token: kept where that way writes the sums of the first
        // NC / 2 tokens, which it reaches last
#pragma unroll
        for (int n = 0; n < NC; n++) entry(n) = h[n / 4][n % 4];
        const float br[1] = {bn}, cr[1] = {cn};
        if (t > t0) {
            fetch(t - T);
            fetch_kept(t - T);
        }
        // a token's step size and the row of C (forwards) or B (back), one token ahead of their use (the fences
        // keep the loads from sinking to it)
        float row[2][NC], dl_[2], du_[2], ds_[2];
        auto load_token = [&](int j, bool back) {
            scalar_f32 q = bcb + min(t + j, t1 - 1) * (2 * NP) + (back ? 0 : NP);
            const int k = j & 1;
#pragma unroll
            for (int n = 0; n < NC; n++) row[k][n] = q[n];
            dl_[k] = dls[j * 64 + lane];
            du_[k] = dus[j * 64 + lane];
            if (back) ds_[k] = dss[j * 64 + lane];
            __builtin_amdgcn_sched_barrier(0);
        };
        load_token(0, false);
        static_for<T>([&](auto J) {
            constexpr int j = J;
            const float dl = arrived(dl_[j & 1]), du = du_[j & 1];
            if (j + 1 < T) load_token(j + 1, false);
            const float* rw = row[j & 1];
            float inner = 0.f;
            static_for<NC / 4>([&](auto Q) {
                constexpr int k = Q;
                f32x4 c;
#pragma unroll
                for (int i = 0; i < 4; i++) c[i] = __builtin_amdgcn_exp2f(dl * A2[4 * k + i]) * h[k][i];
                h[k] = outer4<j * NC + 4 * k>(br, du, c);
                hs[j][k] = h[k];
#pragma unroll
                for (int i = 0; i < 4; i++) inner = fmaf(rw[4 * k + i], h[k][i], inner);
            });
            if (gate) sums[(w * 3 + 2) * SLOT + j * 64 + lane] = inner;
        });
        // and back through them
        load_token(T - 1, true);
        static_for<T>([&](auto J) {
            constexpr int j = T - 1 - J;
            const float* rw = row[j & 1];
            const float dl = arrived(dl_[j & 1]), du = du_[j & 1], ds = ds_[j & 1];
            if (j > 0) load_token(j - 1, true);
            if (j == NC / 2 - 1) {
                // this token and the ones before it write where the entering state is; half of the states are done with
                // and make room for the next tile's loads
#pragma unroll
                for (int n = 0; n < NC; n++) h[n / 4][n % 4] = entry(n);
            }
            float s1 = 0.f, s2 = 0.f, v[2 * NC];
            static_for<NC / 4>([&](auto Q) {
                constexpr int k = Q;
                const f32x4 gn = outer4<j * NC + 4 * k>(cr, ds, adj[k]);
                const f32x4 before = j > 0 ? hs[j > 0 ? j - 1 : 0][k] : h[k];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int n = 4 * k + i;
                    adj[k][i] = gn[i] * __builtin_amdgcn_exp2f(dl * A2[n]);
                    // G W as a product: with W = S_t - delta u B it would keep the roundings of S_t, which are larger
                    // than W itself where the decay is strong
                    const float gw = adj[k][i] * before[i];
                    s1 = fmaf(gn[i], rw[n], s1);
                    s2 = fmaf(gw, A2[n], s2);
                    dA[n] = fmaf(gw, dl, dA[n]);
                    // added here: left to itself the compiler adds behind the last token and holds the tile's 64
                    // products until then (2 x 4096 x 2048, N = 16, bf16: 24 registers spilled, main 333 us for 291)
                    asm volatile("" : "+v"(dA[n]));
                    v[n] = gn[i] * du;
                    v[NC + n] = ds * hs[j][k][i];
                }
            });
            sums[(w * 3) * SLOT + j * 64 + lane] = s1;
            sums[(w * 3 + 1) * SLOT + j * 64 + lane] = s2;
            const float s = wave_sums16(v);
            if (t + j < t1 && (lane & 3) == 0) (dbcb + (int64_t)(t + j) * (2 * NP))[dbco] = s;
        });
        barrier();
        for (int j = w; j < T; j += nw) {
            const int at = j * 64 + lane;
            float s1 = 0.f, s2 = 0.f, inner = 0.f;
            for (int k = 0; k < nw; k++) {
                s1 += sums[(k * 3) * SLOT + at];
                s2 += sums[(k * 3 + 1) * SLOT + at];
                if (gate) inner += sums[(k * 3 + 2) * SLOT + at];
            }
            const float u = (float)tile[at], dl = dls[at], ds = dss[at];
            float dd = t + j < t1 && live ? fmaf(u, s1, s2 * LN2) : 0.f;
            if (sp) dd *= sigmoid((float)tile[SLOT + at] + bias);  // d delta / d dt
            if (gate) {
                const float z = (float)tile[3 * SLOT + at], sz = sigmoid(z), dyv = (float)tile[2 * SLOT + at];
                io<E>::st(tile + 3 * SLOT + at, dyv * fmaf(skip, u, inner) * sz * fmaf(z, 1.f - sz, 1.f));
            }
            io<E>::st(tile + 2 * SLOT + at, fmaf(ds, skip, dl * s1));
            io<E>::st(tile + SLOT + at, dd);
            dDsum = fmaf(ds, u, dDsum);
            dbsum += dd;
        }
        wave_lds_fence();
        const int tt = t + pl.token;
        if (pl.in && tt < t1 && (ONE || pl.token % nw == w)) {  // the wave's own tokens
            const BwdArgsPtr q = bwd_args();
            store8<VEC>((E*)q->du + b * q->sdu.batch + d0 + tt * q->sdu.token + pl.col, pl.n, *lds_chunk(tile + 2 * SLOT));
            store8<VEC>((E*)q->ddt + b * q->sddt.batch + d0 + tt * q->sddt.token + pl.col, pl.n, *lds_chunk(tile + SLOT));
            if (gate)
                store8<VEC>((E*)q->dz + b * q->sdz.batch + d0 + tt * q->sdz.token + pl.col, pl.n, *lds_chunk(tile + 3 * SLOT));
        }
        if (ONE) wave_lds_fence();
    }
    if (!live) return;
    const BwdArgsPtr e = bwd_args();
    const int64_t D = e->D, seg = b * e->G + g;
    const int N = e->N;
#pragma unroll
    for (int n = 0; n < NC; n++) {
        (e->dap + (seg * NP + nb + n) * D + d0)[lane] = dA[n];
        if (g == 0 && e->ds_in && nb + n < N) (e->ds_in + (b * N + nb + n) * D + d0)[lane] = adj[n / 4][n % 4];
    }
    float* dd = e->ddp + ((seg * nw + w) * 2) * D + d0;
    dd[lane] = dDsum;
    (dd + D)[lane] = dbsum;
}

// Pass 4.  The first `nbc` blocks: dB and dC, a thread per (b, t, n) of each; the others: dA, dD and
// d dt_bias, 16 channels of one n (or of one of the two) per block, 16 threads to a channel.
template <typename E>
__global__ __launch_bounds__(256) void ssm_bwd_sums_kernel(const float* __restrict__ dbc, const float* __restrict__ dap,
                                                           const float* __restrict__ ddp, const int32_t* lengths,
                                                           E* __restrict__ dB, E* __restrict__ dC, float* __restrict__ dA,
                                                           float* __restrict__ dD, float* __restrict__ dbias, la_rows sdb,
                                                           la_rows sdc, int64_t B, int64_t L, int64_t D, int N, int NP, int G,
                                                           unsigned cb, unsigned nbc) {
    const int64_t block = wide_block();
    if (block < nbc) {
        const int64_t i = block * 256 + threadIdx.x;
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
    __shared__ float part[16][17];
    const int64_t blocks = (D + 15) / 16, k = block - nbc;
    const int64_t n = k / blocks;
    if (n >= N + 2) return;
    const int dl = threadIdx.x & 15, share = threadIdx.x >> 4;
    const int64_t d = k % blocks * 16 + dl;
    const bool isA = n < N;
    const int64_t step = isA ? (int64_t)NP * D : 2 * D, rows = isA ? B * G : B * G * (NP / NW8);
    float s = 0.f;
    if (d < D) {
        const float* src = isA ? dap + n * D + d : ddp + (n - N) * D + d;
#pragma unroll 4
        for (int64_t r = share; r < rows; r += 16) s += src[r * step];
    }
    part[share][dl] = s;
    __syncthreads();
    if (share != 0 || d >= D) return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i++) s += part[i][dl];
    if (isA)
        dA[d * N + n] = s;
    else if (n == N) {
        if (dD) dD[d] = s;
    } else if (dbias)
        dbias[d] = s;
}

int bwd_np(int N) { return (N + NW8 - 1) / NW8 * NW8; }

// Segments: about 6144 waves in the main pass (NP / 8 to a channel block), two rounds of what fits the device
// at once, none under 16 tokens.  2 x 4096 tokens x 2048 channels, N = 16, main and first pass: half as many
// waves 302 + 143 us, 6144 304 + 104, half as many again 299 + 98 (and 4 us more in the sums over segments).
SsmPlan bwd_plan(int64_t B, int64_t L, int64_t D, int NP) { return ssm_plan(B, L, D, 6144 / (NP / NW8), 16, T); }

struct BwdWs {
    float *bc, *a2, *hin, *gout, *sumdt, *kept, *keptdt, *dbc, *dap, *ddp;
    int64_t nk;
    size_t bytes;
};
BwdWs bwd_cut(void* base, int64_t B, int64_t L, int64_t D, int N, int G) {
    WsCut c{(char*)base};
    BwdWs w;
    const int NP = bwd_np(N);
    const size_t seg = (size_t)(B * G) * D, tok = (size_t)(B * L);
    w.nk = (L + T - 1) / T;
    w.bc = c.take(tok * 2 * NP);
    w.a2 = c.take((size_t)NP * D);
    w.hin = c.take(seg * NP);
    w.gout = c.take(seg * NP);
    w.sumdt = c.take(seg);
    w.kept = c.take((size_t)(B * w.nk) * NP * D);
    w.keptdt = c.take((size_t)(B * w.nk) * D);
    w.dbc = c.take(tok * 2 * NP * ((D + 63) / 64));
    w.dap = c.take(seg * NP);
    w.ddp = c.take(seg * 2 * (NP / NW8));
    w.bytes = c.used;
    return w;
}

template <typename E>
hipError_t launch_e(const SsmArgs& a) {
    const SsmPlan pl = bwd_plan(a.B, a.L, a.D, bwd_np(a.N));
    const BwdWs w = bwd_cut(a.ws, a.B, a.L, a.D, a.N, pl.G);
    BwdDev p;
    p.u = a.u; p.dt = a.dt; p.z = a.z; p.dy = a.dy; p.a2 = w.a2; p.Dskip = a.Dskip; p.dt_bias = a.dt_bias;
    p.ds_out = a.ds_out; p.lengths = a.lengths;
    p.bc = w.bc; p.hin = w.hin; p.gout = w.gout; p.sumdt = w.sumdt; p.kept = w.kept; p.keptdt = w.keptdt;
    p.dbc = w.dbc; p.dap = w.dap; p.ddp = w.ddp;
    p.ds_in = a.ds_in; p.du = a.du; p.ddt = a.ddt; p.dz = a.dz;
    p.B = a.B; p.L = a.L; p.D = a.D; p.seglen = pl.seglen; p.nk = w.nk;
    p.N = a.N; p.NP = bwd_np(a.N); p.G = pl.G;
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
#define LA_SSM_STATES(n, V)                                                                                    \
    LA_TRACED(a.tr, "ssm_bwd_states",                                                                          \
              ssm_bwd_states_kernel<E, n, V><<<blocks * (unsigned)(p.NP / n), 64, 0, a.stream>>>(p))
        if (p.NP % 16) {
            if (vec) LA_SSM_STATES(8, true);
            else LA_SSM_STATES(8, false);
        } else {
            if (vec) LA_SSM_STATES(16, true);
            else LA_SSM_STATES(16, false);
        }
#undef LA_SSM_STATES
        const int64_t total = a.B * p.NP * a.D;
        const dim3 grid = wide_grid((total + 63) / 64, 2);
#define LA_SSM_SEGMENTS(n)                                                                                       \
    LA_TRACED(a.tr, "ssm_bwd_segments", ssm_bwd_segments_kernel<n><<<grid, 64 * n, 0, a.stream>>>(               \
                                            w.a2, a.s_in, a.ds_out, w.sumdt, w.hin, w.gout, total, a.D, a.N, p.NP, pl.G))
        if (segment_parts(total) == 16) LA_SSM_SEGMENTS(16);
        else LA_SSM_SEGMENTS(4);
#undef LA_SSM_SEGMENTS
        const int nw = p.NP / NW8;
        const size_t lds = T * 64 * (2 * 4 * es + (3 + 3 * nw) * sizeof(float));
#define LA_SSM_MAIN(V, O) \
    LA_TRACED(a.tr, "ssm_bwd_main", ssm_bwd_main_kernel<E, V, O><<<blocks, 64 * nw, lds, a.stream>>>(p))
        if (nw == 1) {
            if (vec) LA_SSM_MAIN(true, true);
            else LA_SSM_MAIN(false, true);
        } else {
            if (vec) LA_SSM_MAIN(true, false);
            else LA_SSM_MAIN(false, false);
        }
#undef LA_SSM_MAIN
    }
    const unsigned nbc = (unsigned)((a.B * a.L * 2 * p.NP + 255) / 256);
    const int64_t nd = (a.D + 15) / 16 * (a.N + 2);
    if (nbc + nd > 0)
        LA_TRACED(a.tr, "ssm_bwd_sums",
                  ssm_bwd_sums_kernel<E><<<wide_grid(nbc + nd, 1), 256, 0, a.stream>>>(w.dbc, w.dap, w.ddp, a.lengths, (E*)a.dB, (E*)a.dC,
                                                                         a.dA, a.dD, a.d_dt_bias, a.sdb, a.sdc, a.B, a.L,
                                                                         a.D, a.N, p.NP, pl.G, p.cb, nbc));
    return hipGetLastError();
}

}  // namespace

size_t ssm_bwd_ws(int64_t B, int64_t L, int64_t D, int N) {
    return bwd_cut(nullptr, B, L, D, N, bwd_plan(B, L, D, bwd_np(N)).G).bytes;
}

hipError_t launch_ssm_scan_bwd(const SsmArgs& a) { return a.bf16 ? launch_e<__bf16>(a) : launch_e<float>(a); }

}  // namespace la
