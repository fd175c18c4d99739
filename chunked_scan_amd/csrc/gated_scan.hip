// gated_scan.hip -- the gated linear recurrence, its backward and its single-token form.
//
//   rho = sigma(r + r_bias), iota = sigma(i + i_bias), v = c softplus(lam) rho >= 0, a = e^-v, m = sqrt(1 - a^2)
//   h_t = a_t h_{t-1} + m_t iota_t x_t,   y_t = h_t z_t sigma(z_t)
//
// Backward, with s_t = dy_t z_t sigma(z_t) and g_t = s_t + a_{t+1} g_{t+1} the derivative by h_t:
//   dx = g m iota,  di = g m iota x (1 - iota),  dz = dy h silu'(z),
//   q  = dLoss/dv v = g (k b - v a h_{t-1}),  b = m iota x,  k = a^2 v / m^2,
//   dr = q (1 - rho),  dlam = sum q sigma(lam) / softplus(lam).
// (dm/dv = a^2 / m is infinite at v = 0; v dm/dv and so q are not: everything that follows from v goes through q.)
//
// 1 - a^2 near a = 1 loses its digits: there it is 2 a sinh(v) = 2 a v S, S = 1 + v^2/6 + v^4/120 + v^6/5040 (the next term
// is below 1.1e-8 of it for v <= 1/2), and k = a / (2 S).
#include <algorithm>
#include <initializer_list>
#include <type_traits>
#include <utility>

#include "la_mixer.h"

namespace la {
namespace {

struct GatedDev {
    const void* x;
    const void* r;
    const void* i;
    const float* lam;
    const float* r_bias;
    const float* i_bias;
    const void* z;
    const float* h_in;
    const int32_t* lengths;
    void* y;
    float* h_out;
    float* blocks;
    const float* blocks_in;
    const void* dy;
    const float* dh_out;
    void* dx;
    void* dr;
    void* di;
    void* dz;
    float* dh_in;
    float* part;  // [B * tiles, 3, D]
    float* state;
    const int32_t* slots;
    unsigned* ticket;
    uint64_t* map;         // [B, tiles, D]
    uint32_t* state_word;  // [B, tiles, D]
    uint32_t* hint;        // [B, cb, tiles]: not all ones when the tile's states are published
    int64_t L, D, tiles;   // tiles of a sequence, at least 1
    int64_t blocks_per_seq;
    unsigned cb, per_tile, total;  // channel blocks; tiles at one position; tiles in all
    int nslots, limit;
    float c;
    la_rows sx, sr, si, sz, sy, sdy, sdx, sdr, sdi, sdz;
};

// A channel's parameters: the biases times -log2 e, the largest v in base 2 (v log2 e).
struct Channel {
    float nr, ni, rate;
};
constexpr float MAX_RATE = 0x1.fffffep127f;
// A rate past fp32 is its largest value: infinity times a closed gate's zero would be NaN.  (c softplus(lam) first: c log2 e
// may be infinite where softplus is zero.)
__device__ __forceinline__ float rate_of(float lam, float c) {
    const float v = c * softplus(lam) * LOG2E;
    return v > MAX_RATE ? MAX_RATE : v;  // NaN stays
}
__device__ __forceinline__ Channel channel(const float* lam, const float* r_bias, const float* i_bias, float c, int64_t d) {
    return {r_bias ? -LOG2E * r_bias[d] : 0.f, i_bias ? -LOG2E * i_bias[d] : 0.f, rate_of(lam[d], c)};
}

// 2^-w is zero in fp32.
constexpr float NO_DECAY_LEFT = 256.f;
// With w = v log2 e, a = 2^-w.  1 - a^2 = a w p for w up to SMALL_W (v <= 1/2), where p = 2 ln2 S is a polynomial in w^2;
// above it 1 - a^2 itself has its digits.  SMALL: every w is small (a channel's rate bounds its w, so a whole wave knows).
constexpr float SMALL_W = 0.5f * LOG2E;
constexpr float P0 = 2.f * LN2, P1 = P0 * LN2 * LN2 / 6.f, P2 = P1 * LN2 * LN2 / 20.f, P3 = P2 * LN2 * LN2 / 42.f;
__device__ __forceinline__ float poly_p(float w) {
    const float w2 = w * w;
    return fmaf(w2, fmaf(w2, fmaf(w2, P3, P2), P1), P0);
}
struct Gates {
    float er, ei;               // e^-(r + r_bias), e^-(i + i_bias)
    float rho, iota, w, a, mi;  // mi = m iota
};
template <bool SMALL>
__device__ __forceinline__ Gates gates(float r, float i, const Channel& c) {
    Gates g;
    g.er = __builtin_amdgcn_exp2f(fmaf(r, -LOG2E, c.nr));
    g.ei = __builtin_amdgcn_exp2f(fmaf(i, -LOG2E, c.ni));
    g.rho = rcp(1.f + g.er);
    g.iota = rcp(1.f + g.ei);
    g.w = c.rate * g.rho;
    g.a = __builtin_amdgcn_exp2f(-g.w);
    float m2 = g.a * g.w * poly_p(g.w);
    if (!SMALL) m2 = g.w <= SMALL_W ? m2 : fmaf(-g.a, g.a, 1.f);
    g.mi = __builtin_amdgcn_sqrtf(m2) * g.iota;
    return g;
}
// rho and 1 - rho in one register: the lesser of them, negative (or -0) where that is 1 - rho.  The greater one is the
// difference from 1, which has its digits.  (2 x 4096 x 2048 bf16 forward and backward 133.4 us, 132.1 with 1 - rho a
// difference, which is nothing from r + r_bias = 17 on.)
__device__ __forceinline__ float lesser(float er, float rho) { return er < 1.f ? -(er * rho) : rho; }
__device__ __forceinline__ void both(float t, float* rho, float* shut) {
    const float u = fabsf(t), v = 1.f - u;
    const bool open = __float_as_int(t) < 0;
    *rho = open ? v : u;
    *shut = open ? u : v;
}
// k / (a ln2) = a v / (m^2 ln2): 1 / p, or a w / (1 - a^2)
__device__ __forceinline__ float input_slope(float w, float a) {
    const bool small = w <= SMALL_W;
    return (small ? 1.f : a * w) * rcp(small ? poly_p(w) : fmaf(-a, a, 1.f));
}

// ---------------------------------------------------------------------------------------------
// The scan over a sequence.  A tile is 128 tokens x 64 channels (backward 64 x 64), a workgroup's.  A tile's
// tokens map the state that enters it to the one that leaves it, h -> A h + B; its workgroup publishes (A, B) for the
// tiles behind it as soon as it has read its inputs, then looks back for the state that enters it (look_back), publishes the
// one that leaves it, and walks its tokens, whose a and b have stayed in registers.  So every input is read once, a
// sequence fills the card however few channels there are, and no tile waits for more than the tiles in flight before it.
//
// Measured, bf16 with gate (the clearing of the words among it): 1 x 16384 x 2048 forward 82 us, 335 MB at 4.1 TB/s, where
// a large copy of as many bytes takes 70; 2 x 4096 x 2048 forward 48 and backward 88 (302 MB; a copy 58 to 63).  What bounds it:
// 128 sequences of one tile, which neither clear nor wait, take 70 us, a copy's rate; sequences of two tiles 76, so clearing
// and tickets cost 6, and the look-back over 128 tiles another 6.  Arithmetic is hidden but for 2 us (4 in the backward).  Why
// this tile: 64 channels make a state word a lane in the wave that looks back; 32 and 64 tokens make more of them to fold
// (122 to 136 us where 128 took 106), 16 waves a workgroup wait for each other (97 to 134 where 8 took 98), and four channels
// a lane hold twice the registers (90 against 85).
//
// Order.  Workgroups take tiles by a ticket, those of one position in their sequences before the next position's, so
// every tile that a workgroup waits for has been taken by one that runs already, and the first of them waits for
// nothing: the waits end whatever the order of dispatch.  They are bounded all the same (chain_spin_limit polls): a
// workgroup that gives up goes on with NaN and counts it.
//
// Coherence.  A published word is its own flag: (A, B) in one 64-bit word, a state in one of 32 bits, both stored and
// loaded whole by relaxed device-scope atomics, all ones (a NaN that no result has, see word()) until then.  Nothing else
// passes between workgroups, so no fences.
//
// Results do not depend on scheduling: a state is always the left fold h_k+1 = A_k h_k + B_k from the sequence's start,
// wherever a workgroup finds it done.  An infinite state, which token by token stays one, becomes NaN where A_k underflows: a
// least A_k in its place would let states pass a complete decay.

constexpr uint32_t EMPTY = ~0u;

// Access size, tokens a lane, waves a workgroup, and the least waves a SIMD of the vector form (forward: of 2-byte types),
// whose registers fit.
template <bool BWD> struct Cfg;
template <> struct Cfg<false> { static constexpr int VEC = 2, TPT = 8, WAVES = 8, OCC = 6; };
template <> struct Cfg<true> { static constexpr int VEC = 2, TPT = 8, WAVES = 4, OCC = 3; };
template <bool BWD> constexpr int tokens_of() { return Cfg<BWD>::VEC * Cfg<BWD>::TPT * Cfg<BWD>::WAVES; }
constexpr int FWD_TOKENS = tokens_of<false>(), BWD_TOKENS = tokens_of<true>();  // tokens of a tile

// VEC adjacent elements of a row in one access.
template <typename E, int VEC> struct Row;
template <> struct Row<__bf16, 4> {
    typedef u32x2 raw;
    static __device__ __forceinline__ void get(raw r, float* f) {
        f[0] = bits_lo_bf16(r[0]); f[1] = bits_hi_bf16(r[0]); f[2] = bits_lo_bf16(r[1]); f[3] = bits_hi_bf16(r[1]);
    }
    static __device__ __forceinline__ raw put(const float* f) { return u32x2{pack2(f[0], f[1]), pack2(f[2], f[3])}; }
};
template <> struct Row<__bf16, 2> {
    typedef uint32_t raw;
    static __device__ __forceinline__ void get(raw r, float* f) { f[0] = bits_lo_bf16(r); f[1] = bits_hi_bf16(r); }
    static __device__ __forceinline__ raw put(const float* f) { return pack2(f[0], f[1]); }
};
template <> struct Row<float, 4> {
    typedef f32x4 raw;
    static __device__ __forceinline__ void get(raw r, float* f) { f[0] = r[0]; f[1] = r[1]; f[2] = r[2]; f[3] = r[3]; }
    static __device__ __forceinline__ raw put(const float* f) { return f32x4{f[0], f[1], f[2], f[3]}; }
};
template <> struct Row<float, 2> {
    typedef f32x2 raw;
    static __device__ __forceinline__ void get(raw r, float* f) { f[0] = r[0]; f[1] = r[1]; }
    static __device__ __forceinline__ raw put(const float* f) { return f32x2{f[0], f[1]}; }
};
template <typename E> struct Row<E, 1> {
    typedef E raw;
    static __device__ __forceinline__ void get(raw r, float* f) { f[0] = (float)r; }
    static __device__ __forceinline__ raw put(const float* f) { return (E)f[0]; }
};
// A token's row (a uniform address in device memory) at a lane's channels, `at` bytes behind, which fit 32 bits.
// Outputs leave by streaming stores (2 x 4096 x 2048 bf16 forward and backward 168 -> 159 us), so that the last-level cache
// keeps the forward's inputs, which the backward reads again; the backward, their last reader, takes them by streaming
// loads (134.8 -> 131.6; with ordinary stores 142).
typedef __attribute__((address_space(1))) char* GlobalRow;
__device__ __forceinline__ GlobalRow global_row(const void* p) { return (GlobalRow)(uintptr_t)p; }
template <typename E, int VEC, bool STREAM = false>
__device__ __forceinline__ typename Row<E, VEC>::raw ld(GlobalRow row, uint32_t at) {
    const auto* q = (const __attribute__((address_space(1))) typename Row<E, VEC>::raw*)(row + at);
    return STREAM ? __builtin_nontemporal_load(q) : *q;
}
template <typename E, int VEC>
__device__ __forceinline__ void st(GlobalRow row, uint32_t at, const float* f) {
    __builtin_nontemporal_store(Row<E, VEC>::put(f), (__attribute__((address_space(1))) typename Row<E, VEC>::raw*)(row + at));
}

// Waits that gave up, per device (read and cleared by gated_status).
__device__ unsigned int gated_give_ups;

// A result as a published word: any NaN as the quiet one, so that none is EMPTY.
__device__ __forceinline__ uint32_t word(float f) { return f == f ? __float_as_uint(f) : 0x7fc00000u; }
template <typename T>
__device__ __forceinline__ T peek(const T* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// Where the words of one chain (a sequence's 64 channels) stand: tile 0's, `pitch` words a tile; one hint a tile.
struct Chain {
    uint64_t* map;
    uint32_t* state;
    uint32_t* hint;
    int64_t pitch;
};
__device__ __forceinline__ void publish_map(const Chain& c, int k, float a, float b, bool on) {
    if (on) __hip_atomic_store(c.map + k * c.pitch, (uint64_t)word(b) << 32 | word(a), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish_state(const Chain& c, int k, float h, bool on) {
    if (on) __hip_atomic_store(c.state + k * c.pitch, word(h), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if ((threadIdx.x & 63) == 0) __hip_atomic_store(c.hint + k, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state that enters tile k > 0 of a lane's channel: the hints of the 64 tiles before (of those before them, if need be)
// in one access say which is the nearest whose state is on its way; from there forward through the maps of the tiles
// between.  A word that has not arrived yet, whatever its tile's hint says, is polled for.
constexpr int WINDOW = 8;  // maps loaded together
__device__ __forceinline__ float look_back(const Chain& c, int k, int limit) {
    const int lane = threadIdx.x & 63;
    int polls = 0, from = -1;
    for (;;) {
        for (int j = k - 1; j >= 0 && from < 0; j -= 64) {
            const uint64_t known = __ballot(j >= lane && peek(c.hint + max(j - lane, 0)) != EMPTY);
            if (known) from = j - __builtin_ctzll(known);
        }
        if (from >= 0 || ++polls > limit) break;
        __builtin_amdgcn_s_sleep(1);
    }
    float s = 0.f;
    if (from >= 0) {
        uint32_t h = peek(c.state + from * c.pitch);
        for (int j = from + 1; j < k; j += WINDOW) {
            uint64_t m[WINDOW];
#pragma unroll
            for (int w = 0; w < WINDOW; w++) m[w] = peek(c.map + min(j + w, k - 1) * c.pitch);
            if (j == from + 1) {
                while (!__all(h != EMPTY) && polls++ < limit) h = peek(c.state + from * c.pitch);
                s = __uint_as_float(h);
            }
#pragma unroll
            for (int w = 0; w < WINDOW; w++)
                if (j + w < k) {
                    while (!__all((uint32_t)m[w] != EMPTY) && polls++ < limit) {
                        __builtin_amdgcn_s_sleep(1);
                        m[w] = peek(c.map + (j + w) * c.pitch);
                    }
                    s = fmaf(__uint_as_float((uint32_t)m[w]), s, __uint_as_float((uint32_t)(m[w] >> 32)));
                }
        }
        if (from == k - 1) {
            while (!__all(h != EMPTY) && polls++ < limit) h = peek(c.state + from * c.pitch);
            s = __uint_as_float(h);
        }
    }
    if (polls > limit) {
        if (lane == 0) atomicAdd(&gated_give_ups, 1u);
        return __uint_as_float(0x7fc00000u);
    }
    return s;
}

// The kernel's arguments, read again from memory where they are used: held over the whole tile they would push each other
// out of the scalar registers.
typedef const __attribute__((address_space(4))) GatedDev* GatedArgsPtr;
__device__ __forceinline__ GatedArgsPtr gated_args() {
    GatedArgsPtr q = (GatedArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(q));
    return q;
}
// VEC channels' parameters as they lie in memory.  Their loads go out ahead of the rows' (which they would wait for
// otherwise: loads return in order) and without a branch: a bias that is not given is read as lam and times zero.
template <int VEC>
struct Params {
    float lam[VEC], r[VEC], i[VEC];
    float by_r, by_i;
    __device__ __forceinline__ Params(GatedArgsPtr p, int d) {
        const float *lm = p->lam, *pr = p->r_bias, *pi = p->i_bias;
        by_r = pr ? -LOG2E : 0.f;
        by_i = pi ? -LOG2E : 0.f;
        const GlobalRow l = global_row(lm), rb = global_row(pr ? pr : lm), ib = global_row(pi ? pi : lm);
        const uint32_t at = (uint32_t)d * 4u;
        typedef const __attribute__((address_space(1))) float* F;
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            lam[v] = ((F)(l + at))[v];
            r[v] = ((F)(rb + at))[v];
            i[v] = ((F)(ib + at))[v];
        }
    }
    __device__ __forceinline__ Channel channel(int v, float c) const {
        return {by_r * r[v], by_i * i[v], rate_of(lam[v], c)};
    }
};

// Keeps what is computed from these registers behind this place: else both sides of a branch's unpacking of all rows moves
// up in front of it, and its floats fill the registers.
template <typename... R>
__device__ __forceinline__ void here(R&... r) {
    (([](R& x) { asm volatile("" : "+v"(x)); }(r)), ...);
}
// Where a tile lies and what of it exists.  Its width is 64 channels whatever the access size: VEC adjacent channels a
// lane, so 64 / VEC lanes span a row and a wave holds VEC runs of TPT tokens, one behind the other.  Long narrow tiles
// keep few of them in flight on one chain, which is what a look-back has to fold.
struct Place {
    int b, d0, len;   // sequence, first channel, tokens of the sequence (2^25 at most, all of them)
    int t0;           // the wave's first token
    int k, tile, live;
    int run;          // the lane's run
    int n;            // tokens of it that exist
    int d;            // the lane's first channel; the tile's, where that does not exist (`on` false)
    bool on;
    bool full;        // all of the tile's tokens exist
    bool any;         // at least one of the wave's does
};
template <int VEC, int WAVES, int TPT>
__device__ __forceinline__ Place place_of(GatedArgsPtr p, unsigned idx, bool backward) {
    constexpr int TT = WAVES * VEC * TPT, LANES = 64 / VEC;
    const int lane = threadIdx.x & 63, wv = uniform(threadIdx.x >> 6);
    Place q;
    q.k = (int)(idx / p->per_tile);
    const unsigned rest = idx - q.k * p->per_tile;
    q.b = (int)(rest / p->cb);
    q.d0 = (int)(rest - q.b * p->cb) * 64;
    // read through the scalar cache: no launch in flight writes it
    q.len = p->lengths ? max(0, min(((const __attribute__((address_space(4))) int32_t*)(uintptr_t)p->lengths)[q.b], (int)p->L))
                       : (int)p->L;
    q.live = (q.len + TT - 1) / TT;
    q.tile = backward && q.k < q.live ? q.live - 1 - q.k : q.k;
    q.t0 = q.tile * TT + wv * (VEC * TPT);
    q.run = VEC == 1 ? 0 : lane / LANES;
    q.n = max(0, min(TPT, q.len - (q.t0 + q.run * TPT)));
    q.full = (q.tile + 1) * TT <= q.len;
    q.any = q.t0 < q.len;
    q.d = q.d0 + lane % LANES * VEC;
    q.on = q.d < p->D;
    if (!q.on) q.d = q.d0;
    return q;
}
// The rows of one operand: a uniform address and the lane's 32-bit offset (rows_on sees to the range where VEC > 1).
// Tokens that do not exist are read as the sequence's last.  FULL: all of the tile's tokens exist.
template <typename E, int VEC, int TPT, bool FULL, bool STREAM = false>
__device__ __forceinline__ void load_rows(const void* base, const __attribute__((address_space(4))) la_rows& s, const Place& q,
                                          typename Row<E, VEC>::raw (&r)[TPT]) {
    const int64_t step = s.token * (int64_t)sizeof(E);
    GlobalRow row = global_row((const E*)base + q.b * s.batch + q.t0 * s.token);
    const uint32_t at = (uint32_t)q.d * (uint32_t)sizeof(E), pitch = (uint32_t)step;
    if (FULL || VEC == 1) {
        const uint32_t own = VEC == 1 ? at : at + (uint32_t)(q.run * TPT) * pitch;
#pragma unroll
        for (int j = 0; j < TPT; j++) {
            r[j] = ld<E, VEC, STREAM>(row, own);
            if (FULL || q.t0 + j + 1 < q.len) row += step;
            asm("" : "+s"(row));  // stays a uniform address with a 32-bit offset, not one 64-bit sum a lane and token
        }
    } else {
        const int last = q.len - 1 - q.t0;
#pragma unroll
        for (int j = 0; j < TPT; j++) r[j] = ld<E, VEC, STREAM>(row, at + (uint32_t)min(q.run * TPT + j, last) * pitch);
    }
}
// An output's rows: the lane's VEC values of its j-th token.
template <typename E, int VEC, int TPT>
struct OutRows {
    GlobalRow row;
    int64_t step;
    uint32_t own;
    __device__ __forceinline__ OutRows(void* base, const __attribute__((address_space(4))) la_rows& s, const Place& q) {
        step = s.token * (int64_t)sizeof(E);
        row = global_row((E*)base + q.b * s.batch + q.t0 * s.token);
        own = (uint32_t)q.d * (uint32_t)sizeof(E);
        if (VEC > 1) own += (uint32_t)(q.run * TPT) * (uint32_t)step;
    }
    __device__ __forceinline__ void put(int j, const float* f) const {
        GlobalRow at = row + j * step;
        asm("" : "+s"(at));  // as in load_rows
        st<E, VEC>(at, own, f);
    }
};

__device__ __forceinline__ Chain chain_of(GatedArgsPtr p, const Place& q, int64_t d) {
    const int64_t first = q.b * p->tiles * p->D + d;
    return {p->map + first, p->state_word + first, p->hint + ((int64_t)q.b * p->cb + q.d0 / 64) * p->tiles, p->D};
}

// The tile of this workgroup: by ticket, or where sequences have one tile (nobody waits) by its number.
__device__ __forceinline__ unsigned take(GatedArgsPtr p, unsigned* shared) {
    if (p->tiles == 1) return blockIdx.y * gridDim.x + blockIdx.x;
    if (threadIdx.x == 0) *shared = atomicAdd(p->ticket, 1u) + 1u;  // from all ones
    lds_barrier();
    return (unsigned)uniform((int)*shared);
}

// One tile.  FULL: all of its tokens exist, and nothing asks.  Two copies, not a branch at each load: the compiler joins
// such branches again, by waiting for one side's loads where the other's go to the same registers.
template <typename E, int VEC, int WAVES, int TPT, bool FULL>
__device__ __forceinline__ void fwd_tile(GatedArgsPtr p, const Place& q, float (*map_a)[64], float (*map_b)[64]) {
    constexpr int TT = WAVES * VEC * TPT, RUNS = WAVES * VEC, LANES = 64 / VEC;
    static_assert(LA_GATED_BLOCK % TPT == 0, "a run lies in one block");
    typedef typename Row<E, VEC>::raw raw;
    const int lane = threadIdx.x & 63, wv = uniform(threadIdx.x >> 6);
    const bool gated = p->z && p->y;
    float a[TPT][VEC], bb[TPT][VEC];
    raw zr[TPT];
    if (FULL || q.any) {
        const Params<VEC> par(p, q.d);
        raw xr[TPT], rr[TPT], ir[TPT];
        load_rows<E, VEC, TPT, FULL>(p->r, p->sr, q, rr);
        load_rows<E, VEC, TPT, FULL>(p->i, p->si, q, ir);
        load_rows<E, VEC, TPT, FULL>(p->x, p->sx, q, xr);
        Channel c[VEC];
        bool small = true;
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            c[v] = par.channel(v, p->c);
            small = small && c[v].rate <= SMALL_W;
        }
        auto maps = [&](auto known) {
#pragma unroll
            for (int j = 0; j < TPT; j++) {
                float fx[VEC], fr[VEC], fi[VEC];
                here(xr[j], rr[j], ir[j]);
                Row<E, VEC>::get(xr[j], fx);
                Row<E, VEC>::get(rr[j], fr);
                Row<E, VEC>::get(ir[j], fi);
#pragma unroll
                for (int v = 0; v < VEC; v++) {
                    const Gates g = gates<decltype(known)::value>(fr[v], fi[v], c[v]);
                    a[j][v] = g.a;
                    bb[j][v] = g.mi * fx[v];
                }
            }
        };
        if (__all(small)) maps(std::true_type());
        else maps(std::false_type());
    }
    // All rows have come; said here, where it is known, so that z's are not waited for in front of the barrier: behind the
    // branches above the compiler would wait for all loads (2 x 4096 x 2048 134.4 -> 133.5 us, 1 x 16384 x 2048 82.2 -> 81.5).
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    if (gated && (FULL || q.any)) load_rows<E, VEC, TPT, FULL>(p->z, p->sz, q, zr);
    if (!FULL) {  // tokens that are not there: a = 1, no input
#pragma unroll
        for (int j = 0; j < TPT; j++)
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                a[j][v] = j < q.n ? a[j][v] : 1.f;
                bb[j][v] = j < q.n ? bb[j][v] : 0.f;
            }
    }
    const int run = wv * VEC + q.run, col = lane % LANES * VEC;
#pragma unroll
    for (int v = 0; v < VEC; v++) {
        float A = a[0][v], B = bb[0][v];
#pragma unroll
        for (int j = 1; j < TPT; j++) {
            A *= a[j][v];
            B = fmaf(a[j][v], B, bb[j][v]);
        }
        map_a[run][col + v] = A;
        map_b[run][col + v] = B;
    }
    lds_barrier();
    p = gated_args();
    if (wv == 0) {  // a lane per channel
        const int64_t D = p->D;
        const bool in = q.d0 + lane < D;
        const int64_t d = in ? q.d0 + lane : q.d0;
        const Chain chain = chain_of(p, q, d);
        const bool more = q.k + 1 < q.live;
        float h = 0.f, A = 1.f, B = 0.f;
#pragma unroll 4
        for (int k = 0; k < RUNS; k++) {
            A *= map_a[k][lane];
            B = fmaf(map_a[k][lane], B, map_b[k][lane]);
        }
        if (q.k > 0) {
            if (more) publish_map(chain, q.k, A, B, in);
            h = look_back(chain, q.k, p->limit);
        } else if (p->h_in) {
            h = p->h_in[q.b * D + d];
        }
        // the state that leaves is the same sum whether it goes to the next tile or to the caller, so that a sequence in
        // pieces of whole tiles gives the bits that it gives in one
        const float leaves = fmaf(A, h, B);
        if (more) publish_state(chain, q.k, leaves, in);
        else if (p->h_out && in) p->h_out[q.b * D + d] = leaves;
        float* blocks = p->blocks && in ? p->blocks + q.b * p->blocks_per_seq * D + d : nullptr;
#pragma unroll 4
        for (int k = 0; k < RUNS; k++) {
            const int t = q.tile * TT + k * TPT;
            if (blocks && t % LA_GATED_BLOCK == 0 && t < q.len) blocks[t / LA_GATED_BLOCK * D] = h;
            const float after = fmaf(map_a[k][lane], h, map_b[k][lane]);
            map_b[k][lane] = h;
            h = after;
        }
    }
    if (!p->y) return;
    lds_barrier();
    if (!FULL && !q.any) return;
    float h[VEC];
#pragma unroll
    for (int v = 0; v < VEC; v++) h[v] = map_b[run][col + v];
    p = gated_args();
    const OutRows<E, VEC, TPT> y(p->y, p->sy, q);
#pragma unroll
    for (int j = 0; j < TPT; j++) {
        float o[VEC];
#pragma unroll
        for (int v = 0; v < VEC; v++) o[v] = h[v] = fmaf(a[j][v], h[v], bb[j][v]);
        if (gated) {
            float z[VEC];
            Row<E, VEC>::get(zr[j], z);
#pragma unroll
            for (int v = 0; v < VEC; v++) o[v] *= z[v] * sigmoid(z[v]);
        }
        if (q.on && (FULL || j < q.n)) y.put(j, o);
    }
}
template <typename E, int VEC, int WAVES, int TPT>
__global__ __launch_bounds__(WAVES * 64, sizeof(E) == 2 && VEC > 1 ? Cfg<false>::OCC : 4) void gated_fwd_kernel(GatedDev) {
    // the runs' maps; map_b then the states that enter them
    __shared__ __align__(16) float map_a[WAVES * VEC][64], map_b[WAVES * VEC][64];
    __shared__ unsigned shared;
    GatedArgsPtr p = gated_args();
    const unsigned idx = take(p, &shared);
    if (idx >= p->total) return;
    const Place q = place_of<VEC, WAVES, TPT>(p, idx, false);
    if (q.k > 0 && q.k >= q.live) return;
    if (q.full) fwd_tile<E, VEC, WAVES, TPT, true>(p, q, map_a, map_b);
    else fwd_tile<E, VEC, WAVES, TPT, false>(p, q, map_a, map_b);
}

// Backward, 64 tokens a tile since its rows and gates stay in registers: three waves a SIMD fit (132 registers; fp32 166, two
// waves 83 us at 2 x 2048 x 2048, three 80); a fourth gains nothing (88 us with the input gates in LDS, as with three).
// fp32 at 2 x 4096 x 2048 128 us, 604 MB at 4.7 TB/s; rows that are not aligned, one channel a lane and 16 tokens: 2 x 4000 x
// 2047 bf16 162 us (2048 channels 86), fp32 215 (127).  The same from the sequence's end: the
// carry c_t = a_t g_t runs c_t = a_t (s_t + c_{t+1}) and a tile maps the carry that enters it from behind to A c + R.  The
// states h_{t-1} come from the forward's states at the tiles' starts.  Tiles behind a sequence's end write zeros.
template <typename E, int VEC, int WAVES, int TPT, bool FULL>
__device__ __forceinline__ void bwd_tile(GatedArgsPtr p, const Place& q, float (*map_a)[64], float (*map_h)[64],
                                         float (*map_c)[64]) {
    constexpr int TT = WAVES * VEC * TPT, RUNS = WAVES * VEC, LANES = 64 / VEC;
    static_assert(TT % LA_GATED_BLOCK == 0 && WAVES >= 3, "a tile starts with a block; a wave for each chain and each sum");
    typedef typename Row<E, VEC>::raw raw;
    const int lane = threadIdx.x & 63, wv = uniform(threadIdx.x >> 6);
    const bool gated = p->z != nullptr;
    float a[TPT][VEC], rho[TPT][VEC], shut[TPT][VEC], mi[TPT][VEC];  // rho: see lesser(); shut = 1 - iota
    raw xr[TPT], zr[TPT], yr[TPT];
    float rate[VEC];
    bool small = true;
    const int run = wv * VEC + q.run, col = lane % LANES * VEC;
    if (FULL || q.any) {
        const Params<VEC> par(p, q.d);
        raw rr[TPT], ir[TPT];
        load_rows<E, VEC, TPT, FULL, true>(p->r, p->sr, q, rr);
        load_rows<E, VEC, TPT, FULL, true>(p->i, p->si, q, ir);
        load_rows<E, VEC, TPT, FULL, true>(p->x, p->sx, q, xr);
        load_rows<E, VEC, TPT, FULL, true>(p->dy, p->sdy, q, yr);
        if (gated) load_rows<E, VEC, TPT, FULL, true>(p->z, p->sz, q, zr);
        Channel c[VEC];
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            c[v] = par.channel(v, p->c);
            rate[v] = c[v].rate;
            small = small && c[v].rate <= SMALL_W;
        }
        small = __all(small);
        auto maps = [&](auto known) {
#pragma unroll
            for (int j = 0; j < TPT; j++) {
                float fr[VEC], fi[VEC];
                here(rr[j], ir[j]);
                Row<E, VEC>::get(rr[j], fr);
                Row<E, VEC>::get(ir[j], fi);
#pragma unroll
                for (int v = 0; v < VEC; v++) {
                    const Gates g = gates<decltype(known)::value>(fr[v], fi[v], c[v]);
                    a[j][v] = g.a;
                    rho[j][v] = lesser(g.er, g.rho);
                    shut[j][v] = complement(g.ei, g.iota);
                    mi[j][v] = g.mi;
                }
            }
        };
        if (small) maps(std::true_type());
        else maps(std::false_type());
    }
    // s_t: the derivative that reaches h_t from y_t
    auto reach = [&](int j, float* s) {
        Row<E, VEC>::get(yr[j], s);
        if (gated) {
            float z[VEC];
            Row<E, VEC>::get(zr[j], z);
#pragma unroll
            for (int v = 0; v < VEC; v++) s[v] *= z[v] * sigmoid(z[v]);
        }
    };
    {
        float A[VEC], B[VEC], R[VEC];
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            A[v] = 1.f;
            B[v] = R[v] = 0.f;
        }
        if (FULL || q.any) {
#pragma unroll
            for (int j = 0; j < TPT; j++) {
                float fx[VEC], s[VEC];
                here(xr[j], yr[j]);
                Row<E, VEC>::get(xr[j], fx);
                reach(j, s);
#pragma unroll
                for (int v = 0; v < VEC; v++) {
                    const bool there = FULL || j < q.n;
                    a[j][v] = there ? a[j][v] : 1.f;
                    A[v] *= a[j][v];
                    R[v] = there ? fmaf(A[v], s[v], R[v]) : R[v];  // sum over t of the decays up to t times s_t
                    B[v] = there ? fmaf(a[j][v], B[v], mi[j][v] * fx[v]) : B[v];
                }
            }
        }
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            map_a[run][col + v] = A[v];
            map_h[run][col + v] = B[v];
            map_c[run][col + v] = R[v];
        }
    }
    lds_barrier();
    p = gated_args();
    if (wv < 2) {  // a lane per channel: the first wave the carry, the second the states
        const int64_t D = p->D;
        const bool in = q.d0 + lane < D;
        const int64_t d = in ? q.d0 + lane : q.d0;
        if (!FULL && q.k >= q.live) {
            if (wv == 0 && q.k == 0 && p->dh_in && in) p->dh_in[q.b * D + d] = p->dh_out ? p->dh_out[q.b * D + d] : 0.f;
        } else if (wv == 0) {
            const Chain chain = chain_of(p, q, d);
            const bool more = q.k + 1 < q.live;
            float cy = 0.f, A = 1.f, R = 0.f;
#pragma unroll 4
            for (int k = RUNS - 1; k >= 0; k--) {
                A *= map_a[k][lane];
                R = fmaf(map_a[k][lane], R, map_c[k][lane]);
            }
            if (q.k > 0) {
                if (more) publish_map(chain, q.k, A, R, in);
                cy = look_back(chain, q.k, p->limit);
            } else if (p->dh_out) {
                cy = p->dh_out[q.b * D + d];
            }
            if (more) publish_state(chain, q.k, fmaf(A, cy, R), in);
#pragma unroll 4
            for (int k = RUNS - 1; k >= 0; k--) {
                const float after = fmaf(map_a[k][lane], cy, map_c[k][lane]);
                map_c[k][lane] = cy;
                cy = after;
            }
            if (q.tile == 0 && p->dh_in && in) p->dh_in[q.b * D + d] = cy;
        } else {
            float h = 0.f;
            if (q.tile > 0) h = p->blocks_in[(q.b * p->blocks_per_seq + q.tile * (TT / LA_GATED_BLOCK)) * D + d];
            else if (p->h_in) h = p->h_in[q.b * D + d];
#pragma unroll 4
            for (int k = 0; k < RUNS; k++) {
                const float after = fmaf(map_a[k][lane], h, map_h[k][lane]);
                map_h[k][lane] = h;
                h = after;
            }
        }
    }
    lds_barrier();
    p = gated_args();
    const OutRows<E, VEC, TPT> gx(p->dx, p->sdx, q), gr(p->dr, p->sdr, q), gi(p->di, p->sdi, q), gz(p->dz, p->sdz, q);
    if (!FULL && q.on) {  // rows behind the sequence's end
        const int rows = max(0, min(TPT, (int)p->L - (q.t0 + q.run * TPT)));
        const float zero[VEC] = {};
        for (int j = 0; j < TPT; j++)
            if (j >= q.n && j < rows) {
                gx.put(j, zero);
                gr.put(j, zero);
                gi.put(j, zero);
                if (gated) gz.put(j, zero);
            }
    }
    float sq[VEC] = {}, sr[VEC] = {}, si[VEC] = {};
    if (FULL || q.any) {
        float h[VEC], cy[VEC], before[TPT][VEC], sv[TPT][VEC];
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            h[v] = map_h[run][col + v];
            cy[v] = map_c[run][col + v];
        }
#pragma unroll
        for (int j = 0; j < TPT; j++) {
            float fx[VEC], oz[VEC];
            here(xr[j], yr[j]);
            Row<E, VEC>::get(xr[j], fx);
            Row<E, VEC>::get(yr[j], sv[j]);
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                before[j][v] = h[v];
                h[v] = fmaf(a[j][v], h[v], mi[j][v] * fx[v]);
            }
            if (gated) {
                float z[VEC];
                here(zr[j]);
                Row<E, VEC>::get(zr[j], z);
#pragma unroll
                for (int v = 0; v < VEC; v++) {
                    const float sg = sigmoid(z[v]);
                    oz[v] = sv[j][v] * h[v] * sg * fmaf(z[v], 1.f - sg, 1.f);
                    sv[j][v] *= z[v] * sg;
                }
                if (q.on && (FULL || j < q.n)) gz.put(j, oz);
            }
        }
        // One copy for all decays: a second one for weak decays alone took so many registers that some spilled
        // (2 x 4096 x 2048 bf16 87 us, with strong decays 97; so 88 for both).
#pragma unroll
        for (int j = TPT - 1; j >= 0; j--) {
            if (!FULL && j >= q.n) continue;
            float fx[VEC], ox[VEC], orr[VEC], oi[VEC];
            here(xr[j]);
#pragma unroll
            for (int v = 0; v < VEC; v++) here(rho[j][v]);
            Row<E, VEC>::get(xr[j], fx);
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                float rh, rest;
                both(rho[j][v], &rh, &rest);
                const float g = sv[j][v] + cy[v], bt = mi[j][v] * fx[v];
                const float w = fminf(rate[v] * rh, NO_DECAY_LEFT);  // a = 0 there already, and w times the state may not overflow
                cy[v] = a[j][v] * g;
                const float dw = LN2 * cy[v] * fmaf(input_slope(w, a[j][v]), bt, -w * before[j][v]);
                ox[v] = g * mi[j][v];
                orr[v] = dw * rest;
                oi[v] = g * bt * shut[j][v];
                sq[v] += dw;
                sr[v] += orr[v];
                si[v] += oi[v];
            }
            if (q.on) {
                gx.put(j, ox);
                gr.put(j, orr);
                gi.put(j, oi);
            }
        }
    }
    lds_barrier();
#pragma unroll
    for (int v = 0; v < VEC; v++) {
        map_a[run][col + v] = sq[v];
        map_h[run][col + v] = sr[v];
        map_c[run][col + v] = si[v];
    }
    lds_barrier();
    p = gated_args();
    if (p->L > 0 && wv < 3 && q.d0 + lane < p->D) {  // a sum per wave
        const float(*m)[64] = wv == 0 ? map_a : wv == 1 ? map_h : map_c;
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < RUNS; k++) t += m[k][lane];
        p->part[((q.b * p->tiles + q.tile) * 3 + wv) * p->D + q.d0 + lane] = t;
    }
}
template <typename E, int VEC, int WAVES, int TPT>
__global__ __launch_bounds__(WAVES * 64, VEC > 1 ? Cfg<true>::OCC : 2) void gated_bwd_kernel(GatedDev) {
    // the runs' maps of state and carry, then what enters them; then their shares of the parameters' sums
    __shared__ __align__(16) float map_a[WAVES * VEC][64], map_h[WAVES * VEC][64], map_c[WAVES * VEC][64];
    __shared__ unsigned shared;
    GatedArgsPtr p = gated_args();
    const unsigned idx = take(p, &shared);
    if (idx >= p->total) return;
    const Place q = place_of<VEC, WAVES, TPT>(p, idx, true);
    if (q.full) bwd_tile<E, VEC, WAVES, TPT, true>(p, q, map_a, map_h, map_c);
    else bwd_tile<E, VEC, WAVES, TPT, false>(p, q, map_a, map_h, map_c);
}

// All ones: no word is published, the first ticket is 0.
__global__ __launch_bounds__(256) void gated_clear_kernel(u32x4* p, int64_t n) {
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < n; q += (int64_t)gridDim.x * 256)
        p[q] = u32x4{EMPTY, EMPTY, EMPTY, EMPTY};
}

// Sums over the rows of partial sums, 16 channels per block, 16 threads each, `chunk` rows per blockIdx.y.  `out` null:
// the parameters' derivatives of the only chunk; else one row of sums per chunk.
__global__ __launch_bounds__(256) void gated_sums_kernel(const float* __restrict__ part, int64_t D, int64_t rows, int64_t chunk,
                                                         float* __restrict__ out, const float* __restrict__ lam,
                                                         float* __restrict__ dlam, float* __restrict__ dr_bias,
                                                         float* __restrict__ di_bias) {
    __shared__ float sum[3][16][16];
    const int dl = threadIdx.x & 15, share = threadIdx.x >> 4;
    const int64_t d = (int64_t)blockIdx.x * 16 + dl;
    const int64_t r0 = blockIdx.y * chunk, r1 = min(r0 + chunk, rows);
    float s[3] = {0.f, 0.f, 0.f};
    if (d < D)
#pragma unroll 4
        for (int64_t k = r0 + share; k < r1; k += 16)
#pragma unroll
            for (int q = 0; q < 3; q++) s[q] += part[(k * 3 + q) * D + d];
#pragma unroll
    for (int q = 0; q < 3; q++) sum[q][share][dl] = s[q];
    __syncthreads();
    if (share != 0 || d >= D) return;
#pragma unroll
    for (int q = 0; q < 3; q++) {
        s[q] = 0.f;
        for (int i = 0; i < 16; i++) s[q] += sum[q][i][dl];
        if (out) out[(blockIdx.y * 3 + q) * D + d] = s[q];
    }
    if (out) return;
    // sigma / softplus tends to 1 where both underflow
    const float sp = softplus(lam[d]), sg = sigmoid(lam[d]);
    dlam[d] = s[0] * (sp > 0.f ? sg / sp : 1.f);
    if (dr_bias) dr_bias[d] = s[1];
    if (di_bias) di_bias[d] = s[2];
}

// One token: a row per wave and 64 VEC channels.  The slot and the earlier rows' slots come first, then the rows and the
// state together, then the parameters, each bias behind its own branch: a chain of waits, which bounds it (1 x 2048 takes
// 2.4 us in a graph and 11 from Python, 256 x 4096 6.7 in a graph, bf16 and fp32).
template <typename E, int VEC>
__global__ __launch_bounds__(64) void gated_step_kernel(GatedDev p) {
    const int64_t b = blockIdx.x / p.cb, d = ((int64_t)(blockIdx.x % p.cb) * 64 + threadIdx.x) * VEC;
    const int s = p.slots ? p.slots[b] : (int)b;
    if (s < 0 || s >= p.nslots) return;
    if (p.slots && earlier_row_has(p.slots, b, s)) return;
    if (d >= p.D) return;
    const uint32_t at = (uint32_t)d * (uint32_t)sizeof(E);
    auto row = [&](const void* q, const la_rows& st) { return global_row((const E*)q + b * st.batch); };
    const auto rr = ld<E, VEC>(row(p.r, p.sr), at), ri = ld<E, VEC>(row(p.i, p.si), at), rx = ld<E, VEC>(row(p.x, p.sx), at);
    typename Row<E, VEC>::raw rz = {};
    if (p.z) rz = ld<E, VEC>(row(p.z, p.sz), at);
    float* hp = p.state + (int64_t)s * p.D + d;
    const auto rh = *(const typename Row<float, VEC>::raw*)hp;
    Channel c[VEC];
#pragma unroll
    for (int v = 0; v < VEC; v++) c[v] = channel(p.lam, p.r_bias, p.i_bias, p.c, d + v);
    float fr[VEC], fi[VEC], x[VEC], z[VEC], h[VEC], y[VEC];
    Row<E, VEC>::get(rr, fr);
    Row<E, VEC>::get(ri, fi);
    Row<E, VEC>::get(rx, x);
    Row<E, VEC>::get(rz, z);
    Row<float, VEC>::get(rh, h);
#pragma unroll
    for (int v = 0; v < VEC; v++) {
        const Gates g = gates<false>(fr[v], fi[v], c[v]);
        y[v] = h[v] = fmaf(g.a, h[v], g.mi * x[v]);
        if (p.z) y[v] *= z[v] * sigmoid(z[v]);
    }
    *(typename Row<float, VEC>::raw*)hp = Row<float, VEC>::put(h);
    st<E, VEC>(row(p.y, p.sy), at, y);
}

int64_t tile_count(int64_t L, int tokens) { return std::max<int64_t>(1, (L + tokens - 1) / tokens); }

// The words that the workgroups of one launch publish, behind the ticket (none for sequences of one tile).
struct Words {
    unsigned* ticket;
    uint64_t* map;
    uint32_t* state;
    uint32_t* hint;
    size_t bytes;
};
Words words_of(void* ws, int64_t B, int64_t tiles, int64_t D) {
    WsCut w{(char*)ws};
    Words c = {};
    const size_t n = (size_t)(B * tiles * D);
    if (tiles > 1 && n > 0) {
        c.ticket = (unsigned*)w.take(1);
        c.map = (uint64_t*)w.take(2 * n);
        c.state = (uint32_t*)w.take(n);
        c.hint = (uint32_t*)w.take((size_t)(B * ((D + 63) / 64) * tiles));
    }
    c.bytes = w.used;
    return c;
}
// Workspace: the words, then the backward's partial sums and, where they are not given, the states that enter the blocks.
constexpr int64_t SUM_ROWS = 512;  // rows of partial sums added by one block
struct Cut {
    float* part;
    float* part2;  // one row per SUM_ROWS of them, where there are more
    float* blocks;
    size_t bytes;
};
Cut cut(void* ws, int64_t B, int64_t L, int64_t D, bool bwd, bool have_blocks) {
    WsCut w{(char*)ws};
    Cut c = {};
    const int64_t blocks = tile_count(L, LA_GATED_BLOCK), tiles = tile_count(L, BWD_TOKENS);
    const bool fwd = !bwd || (!have_blocks && blocks > 1);
    w.used = std::max(fwd ? words_of(nullptr, B, tile_count(L, FWD_TOKENS), D).bytes : 0,
                      bwd ? words_of(nullptr, B, tiles, D).bytes : 0);
    if (bwd) {
        const int64_t rows = B * tiles;
        c.part = w.take((size_t)(3 * rows * D));
        if (rows > SUM_ROWS) c.part2 = w.take((size_t)((rows + SUM_ROWS - 1) / SUM_ROWS * 3 * D));
        if (fwd) c.blocks = w.take((size_t)(B * blocks * D));
    }
    c.bytes = w.used;
    return c;
}

GatedDev dev(const GatedArgs& a) {
    GatedDev p = {};
    p.x = a.x; p.r = a.r; p.i = a.i; p.lam = a.lam; p.r_bias = a.r_bias; p.i_bias = a.i_bias; p.z = a.z; p.h_in = a.h_in;
    p.lengths = a.lengths; p.y = a.y; p.h_out = a.h_out; p.blocks = a.blocks; p.blocks_in = a.blocks_in; p.dy = a.dy;
    p.dh_out = a.dh_out; p.dx = a.dx; p.dr = a.dr; p.di = a.di; p.dz = a.dz; p.dh_in = a.dh_in; p.state = a.state;
    p.slots = a.slots; p.nslots = a.nslots; p.c = a.c; p.L = a.L; p.D = a.D; p.blocks_per_seq = tile_count(a.L, LA_GATED_BLOCK);
    p.sx = a.sx; p.sr = a.sr; p.si = a.si; p.sz = a.sz; p.sy = a.sy; p.sdy = a.sdy; p.sdx = a.sdx; p.sdr = a.sdr;
    p.sdi = a.sdi; p.sdz = a.sdz;
    return p;
}

// Whether all rows of the views start on `bytes`, `span` tokens apart within 31 bits.
bool rows_on(size_t bytes, size_t es, int64_t span, std::initializer_list<std::pair<const void*, la_rows>> views) {
    for (const auto& v : views)
        if (v.first && ((uintptr_t)v.first % bytes || v.second.batch * es % bytes || v.second.token * es % bytes ||
                        v.second.token * (int64_t)es * span >= (int64_t)1 << 31))
            return false;
    return true;
}

constexpr unsigned MAX_X = 1 << 20;  // workgroups along x

template <typename E, bool BWD, int VEC, int TPT>
void scan_v(const GatedArgs& a, GatedDev p) {
    constexpr int WAVES = Cfg<BWD>::WAVES;
    p.tiles = tile_count(a.L, WAVES * VEC * TPT);
    p.cb = (unsigned)((a.D + 63) / 64);
    p.per_tile = (unsigned)a.B * p.cb;
    p.total = p.per_tile * (unsigned)p.tiles;
    const Words w = words_of(a.ws, a.B, p.tiles, a.D);
    p.ticket = w.ticket; p.map = w.map; p.state_word = w.state; p.hint = w.hint; p.limit = chain_spin_limit;
    if (p.tiles > 1) {
        const int64_t n = (int64_t)(w.bytes / 16);
        LA_TRACED(a.tr, "gated_clear", gated_clear_kernel<<<(unsigned)std::min<int64_t>((n + 255) / 256, 4096), 256, 0,
                                                            a.stream>>>((u32x4*)a.ws, n));
    }
    const dim3 grid(std::min(p.total, MAX_X), (p.total + MAX_X - 1) / MAX_X);
    if constexpr (BWD)
        LA_TRACED(a.tr, "gated_scan_bwd", gated_bwd_kernel<E, VEC, WAVES, TPT><<<grid, WAVES * 64, 0, a.stream>>>(p));
    else
        LA_TRACED(a.tr, "gated_scan", gated_fwd_kernel<E, VEC, WAVES, TPT><<<grid, WAVES * 64, 0, a.stream>>>(p));
}

template <typename E>
void fwd_t(const GatedArgs& a, const GatedDev& p) {
    typedef Cfg<false> C;
    if (a.D % C::VEC == 0 && rows_on(C::VEC * sizeof(E), sizeof(E), C::VEC * C::TPT,
                                     {{p.x, p.sx}, {p.r, p.sr}, {p.i, p.si}, {p.z, p.sz}, {p.y, p.sy}}))
        scan_v<E, false, C::VEC, C::TPT>(a, p);
    else
        scan_v<E, false, 1, C::VEC * C::TPT>(a, p);
}
template <typename E>
hipError_t bwd_t(const GatedArgs& a) {
    GatedDev p = dev(a);
    const Cut c = cut(a.ws, a.B, a.L, a.D, true, a.blocks_in != nullptr);
    int64_t rows = a.B * tile_count(a.L, BWD_TOKENS);
    p.part = c.part;
    if (c.blocks && a.B > 0) {  // an empty region of a given workspace has an address too
        GatedDev f = p;
        f.y = nullptr; f.h_out = nullptr; f.blocks = c.blocks;
        fwd_t<E>(a, f);
        p.blocks_in = c.blocks;
    }
    if (a.B > 0) {
        typedef Cfg<true> C;
        if (a.D % C::VEC == 0 && rows_on(C::VEC * sizeof(E), sizeof(E), C::VEC * C::TPT,
                                         {{p.x, p.sx}, {p.r, p.sr}, {p.i, p.si}, {p.z, p.sz}, {p.dy, p.sdy}, {p.dx, p.sdx},
                                          {p.dr, p.sdr}, {p.di, p.sdi}, {p.dz, p.sdz}}))
            scan_v<E, true, C::VEC, C::TPT>(a, p);
        else
            scan_v<E, true, 1, C::VEC * C::TPT>(a, p);
    }
    const unsigned cb = (unsigned)((a.D + 15) / 16);
    const float* part = c.part;
    if (a.L == 0) rows = 0;
    if (rows > SUM_ROWS) {
        const int64_t chunks = (rows + SUM_ROWS - 1) / SUM_ROWS;
        LA_TRACED(a.tr, "gated_sums", gated_sums_kernel<<<dim3(cb, (unsigned)chunks), 256, 0, a.stream>>>(
                                          part, a.D, rows, SUM_ROWS, c.part2, nullptr, nullptr, nullptr, nullptr));
        part = c.part2;
        rows = chunks;
    }
    LA_TRACED(a.tr, "gated_sums", gated_sums_kernel<<<cb, 256, 0, a.stream>>>(part, a.D, rows, rows, nullptr, a.lam, a.dlam,
                                                                              a.dr_bias, a.di_bias));
    return hipGetLastError();
}

template <typename E, int VEC>
void step_v(const GatedArgs& a) {
    GatedDev p = dev(a);
    p.cb = (unsigned)((a.D + 64 * VEC - 1) / (64 * VEC));
    LA_TRACED(a.tr, "gated_step", gated_step_kernel<E, VEC><<<(unsigned)(a.B * p.cb), 64, 0, a.stream>>>(p));
}
// Four channels a lane where that leaves two waves a CU (256 x 4096 bf16 in a graph 6.8 us, one a lane 7.3; the floor of its
// 19 MB is 3.7), else one: a few rows are a matter of latency (1 x 2048 2.4 us), which more waves hide.
template <typename E>
hipError_t step_t(const GatedArgs& a) {
    const bool vec = a.D % 4 == 0 && a.B * ((a.D + 255) / 256) >= 512 && (uintptr_t)a.state % 16 == 0 &&
                     rows_on(4 * sizeof(E), sizeof(E), 0, {{a.x, a.sx}, {a.r, a.sr}, {a.i, a.si}, {a.z, a.sz}, {a.y, a.sy}});
    vec ? step_v<E, 4>(a) : step_v<E, 1>(a);
    return hipGetLastError();
}

}  // namespace

size_t gated_fwd_ws(int64_t B, int64_t L, int64_t D) { return cut(nullptr, B, L, D, false, false).bytes; }
size_t gated_bwd_ws(int64_t B, int64_t L, int64_t D, bool have_blocks) { return cut(nullptr, B, L, D, true, have_blocks).bytes; }

hipError_t gated_status(unsigned int* give_ups, bool clear) {
    hipError_t e = hipDeviceSynchronize();
    if (e == hipSuccess) e = hipMemcpyFromSymbol(give_ups, HIP_SYMBOL(gated_give_ups), sizeof(unsigned int));
    const unsigned int zero = 0;
    if (e == hipSuccess && clear) e = hipMemcpyToSymbol(HIP_SYMBOL(gated_give_ups), &zero, sizeof(unsigned int));
    return e;
}

hipError_t launch_gated_scan(const GatedArgs& a) {
    if (a.B == 0 || a.D == 0) return hipSuccess;
    const GatedDev p = dev(a);
    a.bf16 ? fwd_t<__bf16>(a, p) : fwd_t<float>(a, p);
    return hipGetLastError();
}
hipError_t launch_gated_scan_bwd(const GatedArgs& a) {
    if (a.D == 0) return hipSuccess;
    return a.bf16 ? bwd_t<__bf16>(a) : bwd_t<float>(a);
}
hipError_t launch_gated_step(const GatedArgs& a) {
    if (a.B == 0 || a.D == 0) return hipSuccess;
    return a.bf16 ? step_t<__bf16>(a) : step_t<float>(a);
}

}  // namespace la
