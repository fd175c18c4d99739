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
    int64_t L, D, tiles;   // tiles of a sequence
    unsigned cb, per_tile, total;  // channel blocks; tiles at one position; tiles in all
    int nslots, limit;
    float c;
    la_rows sx, sr, si, sz, sy, sdy, sdx, sdr, sdi, sdz;
};

constexpr int TILE = LA_GATED_BLOCK;

// A channel's parameters: the biases times -log2 e, the largest v.
struct Channel {
    float nr, ni, rate;
};
__device__ __forceinline__ Channel channel(const GatedDev& p, int64_t d) {
    return {p.r_bias ? -LOG2E * p.r_bias[d] : 0.f, p.i_bias ? -LOG2E * p.i_bias[d] : 0.f, p.c * softplus(p.lam[d])};
}

struct Gates {
    float rho, iota, v, a, mi;  // mi = m iota
    float s;                    // S, or 1 - a^2 where v > 1/2
};
__device__ __forceinline__ float one_minus_a2(float v, float a) {
    const float v2 = v * v;
    const float sh = fmaf(v2, fmaf(v2, fmaf(v2, 1.f / 5040.f, 1.f / 120.f), 1.f / 6.f), 1.f);
    return v <= 0.5f ? sh : fmaf(-a, a, 1.f);
}
__device__ __forceinline__ Gates gates(float r, float i, const Channel& c) {
    Gates g;
    g.rho = rcp(1.f + __builtin_amdgcn_exp2f(fmaf(r, -LOG2E, c.nr)));
    g.iota = rcp(1.f + __builtin_amdgcn_exp2f(fmaf(i, -LOG2E, c.ni)));
    g.v = c.rate * g.rho;
    g.a = __builtin_amdgcn_exp2f(g.v * -LOG2E);
    g.s = one_minus_a2(g.v, g.a);
    g.mi = __builtin_amdgcn_sqrtf(g.v <= 0.5f ? 2.f * g.a * g.v * g.s : g.s) * g.iota;
    return g;
}
// k = a^2 v / (1 - a^2)
__device__ __forceinline__ float input_slope(const Gates& g) {
    return g.v <= 0.5f ? g.a * rcp(2.f * g.s) : g.a * g.a * g.v * rcp(g.s);
}

// ---------------------------------------------------------------------------------------------
// The scan over a sequence.  A tile is 64 tokens x 64 VEC channels, a workgroup of 8 waves with 8 tokens each.  A tile's
// tokens map the state that enters it to the one that leaves it, h -> A h + B; its workgroup publishes (A, B) for the
// tiles behind it as soon as it has read its inputs, then looks back for the state that enters it (look_back), publishes the
// one that leaves it, and walks its tokens, whose a and b have stayed in registers.  So every input is read once, a
// sequence fills the card however few channels there are, and no tile waits for more than the tiles in flight before it.
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
// wherever a workgroup finds it done.

constexpr int WAVES = 8, TPT = 8;  // waves a workgroup, tokens a thread
static_assert(WAVES * TPT == TILE, "a tile is a block");
constexpr uint32_t EMPTY = ~0u;

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
// A token's row (uniform address) at a lane's channels: `at` bytes, which fit 32 bits.
template <typename E, int VEC>
__device__ __forceinline__ typename Row<E, VEC>::raw ld(const E* row, uint32_t at) {
    return *(const typename Row<E, VEC>::raw*)((const char*)row + at);
}
template <typename E, int VEC>
__device__ __forceinline__ void st(E* row, uint32_t at, const float* f) {
    *(typename Row<E, VEC>::raw*)((char*)row + at) = Row<E, VEC>::put(f);
}

// Waits that gave up, per device (read and cleared by gated_status).
__device__ unsigned int gated_give_ups;

// A result as a published word: any NaN as the quiet one, so that none is EMPTY.
__device__ __forceinline__ uint32_t word(float f) { return f == f ? __float_as_uint(f) : 0x7fc00000u; }
__device__ __forceinline__ void publish_map(uint64_t* p, float a, float b) {
    __hip_atomic_store(p, (uint64_t)word(b) << 32 | word(a), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish_state(uint32_t* p, float h) {
    __hip_atomic_store(p, word(h), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ T peek(const T* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// The state that enters tile k > 0 of a lane's channel: back to the nearest tile whose outgoing state is known for all
// lanes, then forward through the maps of those between.  map, state: tile 0's entries, `pitch` apart.
constexpr int WINDOW = 8;  // entries loaded together
__device__ __forceinline__ float look_back(const uint64_t* map, const uint32_t* state, int64_t pitch, int k, int limit) {
    int polls = 0, from = -1;
    uint32_t h = 0;
    for (;;) {
        for (int j = k - 1; j >= 0 && from < 0; j -= WINDOW) {
            uint32_t v[WINDOW];
#pragma unroll
            for (int w = 0; w < WINDOW; w++) v[w] = j >= w ? peek(state + (j - w) * pitch) : EMPTY;
#pragma unroll
            for (int w = 0; w < WINDOW; w++)
                if (from < 0 && __all(v[w] != EMPTY)) {
                    from = j - w;
                    h = v[w];
                }
        }
        if (from >= 0) break;
        if (++polls > limit) break;
        __builtin_amdgcn_s_sleep(1);
    }
    float s = __uint_as_float(h);
    for (int j = from + 1; from >= 0 && j < k; j += WINDOW) {
        uint64_t m[WINDOW];
#pragma unroll
        for (int w = 0; w < WINDOW; w++) m[w] = j + w < k ? peek(map + (j + w) * pitch) : 0;
#pragma unroll
        for (int w = 0; w < WINDOW; w++)
            if (j + w < k) {
                while (!__all((uint32_t)m[w] != EMPTY) && polls <= limit) {
                    polls++;
                    __builtin_amdgcn_s_sleep(1);
                    m[w] = peek(map + (j + w) * pitch);
                }
                s = fmaf(__uint_as_float((uint32_t)m[w]), s, __uint_as_float((uint32_t)(m[w] >> 32)));
            }
    }
    if (polls > limit) {
        if ((threadIdx.x & 63) == 0) atomicAdd(&gated_give_ups, 1u);
        return __uint_as_float(0x7fc00000u);
    }
    return s;
}

// The tile that a workgroup takes next; false when there is none.  A barrier on either side of the shared word's use.
__device__ __forceinline__ bool take(const GatedDev& p, unsigned turn, unsigned* shared, unsigned* idx) {
    if (p.tiles > 1) {
        if (threadIdx.x == 0) *shared = atomicAdd(p.ticket, 1u) + 1u;  // from all ones
        __syncthreads();
        *idx = (unsigned)uniform((int)*shared);
        __syncthreads();
    } else {
        *idx = blockIdx.x + turn * gridDim.x;
        __syncthreads();
    }
    return *idx < p.total;
}

template <typename E, int VEC>
__global__ __launch_bounds__(512) void gated_fwd_kernel(GatedDev p) {
    constexpr int CW = 64 * VEC;
    typedef typename Row<E, VEC>::raw raw;
    __shared__ float map_a[WAVES][CW], map_b[WAVES][CW];  // map_b: then the states that enter the waves' tokens
    __shared__ unsigned shared;
    const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
    unsigned idx;
    for (unsigned turn = 0; take(p, turn, &shared, &idx); turn++) {
        const int tile = (int)(idx / p.per_tile);
        const unsigned rest = idx - tile * p.per_tile;
        const int64_t b = rest / p.cb, d0 = (int64_t)(rest % p.cb) * CW;
        const int64_t len = seq_len(p.lengths, b, p.L);
        const int live = (int)((len + TILE - 1) / TILE);  // tiles with tokens
        if (tile > 0 && tile >= live) continue;
        const bool on = d0 + lane * VEC < p.D;
        const int64_t d = on ? d0 + lane * VEC : d0;
        const uint32_t at = (uint32_t)d * (uint32_t)sizeof(E);  // lanes behind the last channel do the block's first one's work
        const int64_t t0 = (int64_t)tile * TILE + w * TPT;
        const int n = (int)max((int64_t)0, min((int64_t)TPT, len - t0));
        float a[TPT][VEC], bb[TPT][VEC];
        if (n > 0) {
            const E* xp = (const E*)p.x + b * p.sx.batch + t0 * p.sx.token;
            const E* rp = (const E*)p.r + b * p.sr.batch + t0 * p.sr.token;
            const E* ip = (const E*)p.i + b * p.si.batch + t0 * p.si.token;
            raw xr[TPT], rr[TPT], ir[TPT];
#pragma unroll
            for (int j = 0; j < TPT; j++) {
                const int t = min(j, n - 1);  // behind the end: the last token's, not used
                rr[j] = ld<E, VEC>(rp + t * p.sr.token, at);
                ir[j] = ld<E, VEC>(ip + t * p.si.token, at);
                xr[j] = ld<E, VEC>(xp + t * p.sx.token, at);
            }
            Channel c[VEC];
#pragma unroll
            for (int v = 0; v < VEC; v++) c[v] = channel(p, d + v);
#pragma unroll
            for (int j = 0; j < TPT; j++) {
                float fx[VEC], fr[VEC], fi[VEC];
                Row<E, VEC>::get(xr[j], fx);
                Row<E, VEC>::get(rr[j], fr);
                Row<E, VEC>::get(ir[j], fi);
#pragma unroll
                for (int v = 0; v < VEC; v++) {
                    const Gates g = gates(fr[v], fi[v], c[v]);
                    a[j][v] = j < n ? g.a : 1.f;
                    bb[j][v] = j < n ? g.mi * fx[v] : 0.f;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < TPT; j++)
#pragma unroll
                for (int v = 0; v < VEC; v++) {
                    a[j][v] = 1.f;
                    bb[j][v] = 0.f;
                }
        }
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            float A = 1.f, B = 0.f;
#pragma unroll
            for (int j = 0; j < TPT; j++) {
                A *= a[j][v];
                B = fmaf(a[j][v], B, bb[j][v]);
            }
            map_a[w][lane * VEC + v] = A;
            map_b[w][lane * VEC + v] = B;
        }
        __syncthreads();
        if (threadIdx.x < CW) {  // whole waves: a lane per channel
            const int ch = threadIdx.x;
            const bool in = d0 + ch < p.D;
            const int64_t dc = in ? d0 + ch : d0, first = b * p.tiles * p.D + dc, own = first + tile * p.D;
            const bool more = tile + 1 < live;
            float h = 0.f;
            if (tile > 0) {
                float A = 1.f, B = 0.f;
#pragma unroll
                for (int k = 0; k < WAVES; k++) {
                    A *= map_a[k][ch];
                    B = fmaf(map_a[k][ch], B, map_b[k][ch]);
                }
                if (more && in) publish_map(p.map + own, A, B);
                h = look_back(p.map + first, p.state_word + first, p.D, tile, p.limit);
                if (more && in) publish_state(p.state_word + own, fmaf(A, h, B));
            } else {
                if (p.h_in) h = p.h_in[b * p.D + dc];
                if (more && in) {
                    float A = 1.f, B = 0.f;
#pragma unroll
                    for (int k = 0; k < WAVES; k++) {
                        A *= map_a[k][ch];
                        B = fmaf(map_a[k][ch], B, map_b[k][ch]);
                    }
                    publish_state(p.state_word + own, fmaf(A, h, B));
                }
            }
            if (p.blocks && in && tile < live) p.blocks[own] = h;
#pragma unroll
            for (int k = 0; k < WAVES; k++) {
                const float next = fmaf(map_a[k][ch], h, map_b[k][ch]);
                map_b[k][ch] = h;
                h = next;
            }
            if (p.h_out && in && !more) p.h_out[b * p.D + dc] = h;
        }
        __syncthreads();
        if (p.y && n > 0) {
            float h[VEC];
#pragma unroll
            for (int v = 0; v < VEC; v++) h[v] = map_b[w][lane * VEC + v];
            raw zr[TPT];
            if (p.z) {
                const E* zp = (const E*)p.z + b * p.sz.batch + t0 * p.sz.token;
#pragma unroll
                for (int j = 0; j < TPT; j++) zr[j] = ld<E, VEC>(zp + min(j, n - 1) * p.sz.token, at);
            }
            E* yp = (E*)p.y + b * p.sy.batch + t0 * p.sy.token;
#pragma unroll
            for (int j = 0; j < TPT; j++) {
                float o[VEC];
#pragma unroll
                for (int v = 0; v < VEC; v++) o[v] = h[v] = fmaf(a[j][v], h[v], bb[j][v]);
                if (p.z) {
                    float z[VEC];
                    Row<E, VEC>::get(zr[j], z);
#pragma unroll
                    for (int v = 0; v < VEC; v++) o[v] *= z[v] * sigmoid(z[v]);
                }
                if (on && j < n) st<E, VEC>(yp + j * p.sy.token, at, o);
            }
        }
    }
}

// Backward.  The same from the sequence's end: the carry c_t = a_t g_t runs c_t = a_t (s_t + c_{t+1}) and a tile maps the
// carry that enters it from behind to A c + R.  The states h_{t-1} come from the forward's states at the tiles'
// starts.  Tiles behind a sequence's end write zeros.
template <typename E, int VEC>
__global__ __launch_bounds__(512) void gated_bwd_kernel(GatedDev p) {
    constexpr int CW = 64 * VEC;
    typedef typename Row<E, VEC>::raw raw;
    // the waves' maps of state and carry, then what enters their tokens; then their shares of the parameters' sums
    __shared__ float map_a[WAVES][CW], map_h[WAVES][CW], map_c[WAVES][CW];
    __shared__ unsigned shared;
    const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
    unsigned idx;
    for (unsigned turn = 0; take(p, turn, &shared, &idx); turn++) {
        const int k = (int)(idx / p.per_tile);  // position from the sequence's end
        const unsigned rest = idx - k * p.per_tile;
        const int64_t b = rest / p.cb, d0 = (int64_t)(rest % p.cb) * CW;
        const int64_t len = seq_len(p.lengths, b, p.L);
        const int live = (int)((len + TILE - 1) / TILE);
        const int tile = k < live ? live - 1 - k : k;
        const bool on = d0 + lane * VEC < p.D;
        const int64_t d = on ? d0 + lane * VEC : d0;
        const uint32_t at = (uint32_t)d * (uint32_t)sizeof(E);
        const int64_t t0 = (int64_t)tile * TILE + w * TPT;
        const int n = (int)max((int64_t)0, min((int64_t)TPT, len - t0));
        const int out = (int)max((int64_t)0, min((int64_t)TPT, p.L - t0));  // rows to write
        float a[TPT][VEC], rho[TPT][VEC], iota[TPT][VEC], mi[TPT][VEC], s[TPT][VEC];
        raw xr[TPT], zr[TPT], yr[TPT];
        Channel c[VEC];
        if (n > 0) {
            const E* xp = (const E*)p.x + b * p.sx.batch + t0 * p.sx.token;
            const E* rp = (const E*)p.r + b * p.sr.batch + t0 * p.sr.token;
            const E* ip = (const E*)p.i + b * p.si.batch + t0 * p.si.token;
            const E* yp = (const E*)p.dy + b * p.sdy.batch + t0 * p.sdy.token;
            raw rr[TPT], ir[TPT];
#pragma unroll
            for (int j = 0; j < TPT; j++) {
                const int t = min(j, n - 1);
                rr[j] = ld<E, VEC>(rp + t * p.sr.token, at);
                ir[j] = ld<E, VEC>(ip + t * p.si.token, at);
                xr[j] = ld<E, VEC>(xp + t * p.sx.token, at);
                yr[j] = ld<E, VEC>(yp + t * p.sdy.token, at);
            }
            if (p.z) {
                const E* zp = (const E*)p.z + b * p.sz.batch + t0 * p.sz.token;
#pragma unroll
                for (int j = 0; j < TPT; j++) zr[j] = ld<E, VEC>(zp + min(j, n - 1) * p.sz.token, at);
            }
#pragma unroll
            for (int v = 0; v < VEC; v++) c[v] = channel(p, d + v);
#pragma unroll
            for (int j = 0; j < TPT; j++) {
                float fr[VEC], fi[VEC];
                Row<E, VEC>::get(rr[j], fr);
                Row<E, VEC>::get(ir[j], fi);
                Row<E, VEC>::get(yr[j], s[j]);
                if (p.z) {
                    float z[VEC];
                    Row<E, VEC>::get(zr[j], z);
#pragma unroll
                    for (int v = 0; v < VEC; v++) s[j][v] *= z[v] * sigmoid(z[v]);
                }
#pragma unroll
                for (int v = 0; v < VEC; v++) {
                    const Gates g = gates(fr[v], fi[v], c[v]);
                    a[j][v] = j < n ? g.a : 1.f;
                    rho[j][v] = g.rho;
                    iota[j][v] = g.iota;
                    mi[j][v] = j < n ? g.mi : 0.f;
                    s[j][v] = j < n ? s[j][v] : 0.f;
                }
            }
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                float A = 1.f, B = 0.f, R = 0.f;
#pragma unroll
                for (int j = 0; j < TPT; j++) {
                    float fx[VEC];
                    Row<E, VEC>::get(xr[j], fx);
                    A *= a[j][v];
                    B = fmaf(a[j][v], B, j < n ? mi[j][v] * fx[v] : 0.f);
                }
#pragma unroll
                for (int j = TPT - 1; j >= 0; j--) R = a[j][v] * (s[j][v] + R);
                map_a[w][lane * VEC + v] = A;
                map_h[w][lane * VEC + v] = B;
                map_c[w][lane * VEC + v] = R;
            }
        } else {
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                map_a[w][lane * VEC + v] = 1.f;
                map_h[w][lane * VEC + v] = map_c[w][lane * VEC + v] = 0.f;
            }
        }
        __syncthreads();
        if (threadIdx.x < CW) {
            const int ch = threadIdx.x;
            const bool in = d0 + ch < p.D;
            const int64_t dc = in ? d0 + ch : d0, first = b * p.tiles * p.D + dc, own = first + k * p.D;
            float cy = 0.f, h = 0.f;
            if (k < live) {
                const bool more = k + 1 < live;
                float A = 1.f, R = 0.f;
#pragma unroll
                for (int q = WAVES - 1; q >= 0; q--) {
                    A *= map_a[q][ch];
                    R = fmaf(map_a[q][ch], R, map_c[q][ch]);
                }
                if (k > 0) {
                    if (more && in) publish_map(p.map + own, A, R);
                    cy = look_back(p.map + first, p.state_word + first, p.D, k, p.limit);
                } else if (p.dh_out) {
                    cy = p.dh_out[b * p.D + dc];
                }
                if (more && in) publish_state(p.state_word + own, fmaf(A, cy, R));
                if (tile > 0) h = p.blocks_in[first + tile * p.D];
                else if (p.h_in) h = p.h_in[b * p.D + dc];
#pragma unroll
                for (int q = 0; q < WAVES; q++) {
                    const float next = fmaf(map_a[q][ch], h, map_h[q][ch]);
                    map_h[q][ch] = h;
                    h = next;
                }
#pragma unroll
                for (int q = WAVES - 1; q >= 0; q--) {
                    const float next = fmaf(map_a[q][ch], cy, map_c[q][ch]);
                    map_c[q][ch] = cy;
                    cy = next;
                }
                if (tile == 0 && p.dh_in && in) p.dh_in[b * p.D + dc] = cy;
            } else if (k == 0 && p.dh_in && in) {  // no tokens
                p.dh_in[b * p.D + dc] = p.dh_out ? p.dh_out[b * p.D + dc] : 0.f;
            }
        }
        __syncthreads();
        float sq[VEC] = {}, sr[VEC] = {}, si[VEC] = {};
        E* gx = (E*)p.dx + b * p.sdx.batch + t0 * p.sdx.token;
        E* gr = (E*)p.dr + b * p.sdr.batch + t0 * p.sdr.token;
        E* gi = (E*)p.di + b * p.sdi.batch + t0 * p.sdi.token;
        E* gz = (E*)p.dz + b * p.sdz.batch + t0 * p.sdz.token;
        if (n > 0) {
            float h[VEC], cy[VEC], before[TPT][VEC];
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                h[v] = map_h[w][lane * VEC + v];
                cy[v] = map_c[w][lane * VEC + v];
            }
#pragma unroll
            for (int j = 0; j < TPT; j++) {
                float fx[VEC];
                Row<E, VEC>::get(xr[j], fx);
#pragma unroll
                for (int v = 0; v < VEC; v++) {
                    before[j][v] = h[v];
                    h[v] = fmaf(a[j][v], h[v], mi[j][v] * fx[v]);
                }
            }
#pragma unroll
            for (int j = TPT - 1; j >= 0; j--) {
                float fx[VEC], ox[VEC], orr[VEC], oi[VEC], oz[VEC];
                Row<E, VEC>::get(xr[j], fx);
#pragma unroll
                for (int v = 0; v < VEC; v++) {
                    const float g = s[j][v] + cy[v];
                    cy[v] = a[j][v] * g;
                    Gates t;
                    t.v = c[v].rate * rho[j][v];
                    t.a = a[j][v];
                    t.s = one_minus_a2(t.v, t.a);
                    const float bt = mi[j][v] * fx[v];
                    const float q = g * fmaf(input_slope(t), bt, -t.v * t.a * before[j][v]);
                    ox[v] = g * mi[j][v];
                    orr[v] = q * (1.f - rho[j][v]);
                    oi[v] = g * bt * (1.f - iota[j][v]);
                    if (j < n) {
                        sq[v] += q;
                        sr[v] += orr[v];
                        si[v] += oi[v];
                    }
                }
                if (p.z) {
                    float z[VEC], fy[VEC];
                    Row<E, VEC>::get(zr[j], z);
                    Row<E, VEC>::get(yr[j], fy);
#pragma unroll
                    for (int v = 0; v < VEC; v++) {
                        const float sg = sigmoid(z[v]);
                        oz[v] = fy[v] * fmaf(a[j][v], before[j][v], mi[j][v] * fx[v]) * sg * fmaf(z[v], 1.f - sg, 1.f);
                    }
                }
                if (on && j < n) {
                    st<E, VEC>(gx + j * p.sdx.token, at, ox);
                    st<E, VEC>(gr + j * p.sdr.token, at, orr);
                    st<E, VEC>(gi + j * p.sdi.token, at, oi);
                    if (p.z) st<E, VEC>(gz + j * p.sdz.token, at, oz);
                }
            }
        }
        if (on) {
            float zero[VEC] = {};
            for (int j = n; j < out; j++) {
                st<E, VEC>(gx + j * p.sdx.token, at, zero);
                st<E, VEC>(gr + j * p.sdr.token, at, zero);
                st<E, VEC>(gi + j * p.sdi.token, at, zero);
                if (p.z) st<E, VEC>(gz + j * p.sdz.token, at, zero);
            }
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            map_a[w][lane * VEC + v] = sq[v];
            map_h[w][lane * VEC + v] = sr[v];
            map_c[w][lane * VEC + v] = si[v];
        }
        __syncthreads();
        if (p.tiles > 0 && threadIdx.x < CW && d0 + threadIdx.x < p.D) {
            float* row = p.part + (b * p.tiles + tile) * 3 * p.D + d0 + threadIdx.x;
            float t[3] = {};
#pragma unroll
            for (int q = 0; q < WAVES; q++) {
                t[0] += map_a[q][threadIdx.x];
                t[1] += map_h[q][threadIdx.x];
                t[2] += map_c[q][threadIdx.x];
            }
            row[0] = t[0];
            row[p.D] = t[1];
            row[2 * p.D] = t[2];
        }
    }
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

// A row per wave and 64 channels.
template <typename E>
__global__ __launch_bounds__(64) void gated_step_kernel(GatedDev p) {
    const int64_t b = blockIdx.x / p.cb, d = (int64_t)(blockIdx.x % p.cb) * 64 + threadIdx.x;
    const int s = p.slots ? p.slots[b] : (int)b;
    if (s < 0 || s >= p.nslots) return;
    if (p.slots && earlier_row_has(p.slots, b, s)) return;
    if (d >= p.D) return;
    const Channel c = channel(p, d);
    const Gates g = gates((float)((const E*)p.r)[b * p.sr.batch + d], (float)((const E*)p.i)[b * p.si.batch + d], c);
    float* st = p.state + (int64_t)s * p.D + d;
    float h = fmaf(g.a, *st, g.mi * (float)((const E*)p.x)[b * p.sx.batch + d]);
    *st = h;
    if (p.z) {
        const float z = (float)((const E*)p.z)[b * p.sz.batch + d];
        h *= z * sigmoid(z);
    }
    io<E>::st((E*)p.y + b * p.sy.batch + d, h);
}

int64_t tile_count(int64_t L) { return (L + TILE - 1) / TILE; }

// Workspace: the published words behind the ticket (none for sequences of one tile), then the backward's partial sums
// and, where they are not given, the states that enter the tiles.
constexpr int64_t SUM_ROWS = 512;  // rows of partial sums added by one block
struct Cut {
    unsigned* ticket;
    uint64_t* map;
    uint32_t* state_word;
    size_t clear;  // bytes of these three
    float* part;
    float* part2;  // one row per SUM_ROWS of them, where there are more
    float* blocks;
    size_t bytes;
};
Cut cut(void* ws, int64_t B, int64_t L, int64_t D, bool bwd, bool have_blocks) {
    WsCut w{(char*)ws};
    Cut c = {};
    const size_t n = (size_t)(B * tile_count(L) * D);
    if (tile_count(L) > 1) {
        c.ticket = (unsigned*)w.take(1);
        c.map = (uint64_t*)w.take(2 * n);
        c.state_word = (uint32_t*)w.take(n);
        c.clear = w.used;
    }
    if (bwd) {
        const int64_t rows = B * tile_count(L);
        c.part = w.take(3 * n);
        if (rows > SUM_ROWS) c.part2 = w.take((size_t)((rows + SUM_ROWS - 1) / SUM_ROWS * 3 * D));
        if (!have_blocks && tile_count(L) > 1) c.blocks = w.take(n);
    }
    c.bytes = w.used;
    return c;
}

GatedDev dev(const GatedArgs& a) {
    GatedDev p = {};
    p.x = a.x; p.r = a.r; p.i = a.i; p.lam = a.lam; p.r_bias = a.r_bias; p.i_bias = a.i_bias; p.z = a.z; p.h_in = a.h_in;
    p.lengths = a.lengths; p.y = a.y; p.h_out = a.h_out; p.blocks = a.blocks; p.blocks_in = a.blocks_in; p.dy = a.dy;
    p.dh_out = a.dh_out; p.dx = a.dx; p.dr = a.dr; p.di = a.di; p.dz = a.dz; p.dh_in = a.dh_in; p.state = a.state;
    p.slots = a.slots; p.nslots = a.nslots; p.c = a.c; p.L = a.L; p.D = a.D; p.tiles = tile_count(a.L);
    p.sx = a.sx; p.sr = a.sr; p.si = a.si; p.sz = a.sz; p.sy = a.sy; p.sdy = a.sdy; p.sdx = a.sdx; p.sdr = a.sdr;
    p.sdi = a.sdi; p.sdz = a.sdz;
    return p;
}

// Whether all rows of the views start on `bytes`.
bool rows_on(size_t bytes, size_t es, std::initializer_list<std::pair<const void*, la_rows>> views) {
    for (const auto& v : views)
        if (v.first && ((uintptr_t)v.first % bytes || v.second.batch * es % bytes || v.second.token * es % bytes)) return false;
    return true;
}

constexpr unsigned MAX_BLOCKS = 1 << 20;

template <typename E, int VEC, bool BWD>
void scan_v(const GatedArgs& a, GatedDev p, const Cut& c) {
    p.cb = (unsigned)((a.D + 64 * VEC - 1) / (64 * VEC));
    p.per_tile = (unsigned)a.B * p.cb;
    p.total = p.per_tile * (unsigned)std::max<int64_t>(1, p.tiles);
    p.ticket = c.ticket; p.map = c.map; p.state_word = c.state_word; p.limit = chain_spin_limit;
    if (c.clear) {
        const int64_t n = (int64_t)(c.clear / 16);
        LA_TRACED(a.tr, "gated_clear", gated_clear_kernel<<<(unsigned)std::min<int64_t>((n + 255) / 256, 4096), 256, 0,
                                                            a.stream>>>((u32x4*)c.ticket, n));
    }
    const unsigned blocks = std::min(p.total, MAX_BLOCKS);
    if constexpr (BWD)
        LA_TRACED(a.tr, "gated_scan_bwd", gated_bwd_kernel<E, VEC><<<blocks, 512, 0, a.stream>>>(p));
    else
        LA_TRACED(a.tr, "gated_scan", gated_fwd_kernel<E, VEC><<<blocks, 512, 0, a.stream>>>(p));
}

template <typename E>
void fwd_t(const GatedArgs& a, const GatedDev& p, const Cut& c) {
    constexpr int VEC = sizeof(E) == 2 ? 4 : 2;
    if (a.D % VEC == 0 && rows_on(VEC * sizeof(E), sizeof(E), {{p.x, p.sx}, {p.r, p.sr}, {p.i, p.si}, {p.z, p.sz}, {p.y, p.sy}}))
        scan_v<E, VEC, false>(a, p, c);
    else
        scan_v<E, 1, false>(a, p, c);
}
template <typename E>
hipError_t bwd_t(const GatedArgs& a) {
    GatedDev p = dev(a);
    const Cut c = cut(a.ws, a.B, a.L, a.D, true, a.blocks_in != nullptr);
    const int64_t rows = a.B * p.tiles;
    p.part = c.part;
    if (c.blocks) {
        GatedDev f = p;
        f.y = nullptr; f.h_out = nullptr; f.blocks = c.blocks;
        fwd_t<E>(a, f, c);
        p.blocks_in = c.blocks;
    }
    if (a.B > 0) {
        constexpr int VEC = 2;
        if (a.D % VEC == 0 && rows_on(VEC * sizeof(E), sizeof(E), {{p.x, p.sx}, {p.r, p.sr}, {p.i, p.si}, {p.z, p.sz},
                                       {p.dy, p.sdy}, {p.dx, p.sdx}, {p.dr, p.sdr}, {p.di, p.sdi}, {p.dz, p.sdz}}))
            scan_v<E, VEC, true>(a, p, c);
        else
            scan_v<E, 1, true>(a, p, c);
    }
    const float* part = c.part;
    int64_t n = rows;
    if (n > SUM_ROWS) {
        const int64_t chunks = (n + SUM_ROWS - 1) / SUM_ROWS;
        LA_TRACED(a.tr, "gated_sums", gated_sums_kernel<<<dim3((unsigned)((a.D + 15) / 16), (unsigned)chunks), 256, 0, a.stream>>>(
                                          part, a.D, n, SUM_ROWS, c.part2, nullptr, nullptr, nullptr, nullptr));
        part = c.part2;
        n = chunks;
    }
    LA_TRACED(a.tr, "gated_sums", gated_sums_kernel<<<(unsigned)((a.D + 15) / 16), 256, 0, a.stream>>>(
                                      part, a.D, n, n, nullptr, a.lam, a.dlam, a.dr_bias, a.di_bias));
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
    const Cut c = cut(a.ws, a.B, a.L, a.D, false, false);
    a.bf16 ? fwd_t<__bf16>(a, p, c) : fwd_t<float>(a, p, c);
    return hipGetLastError();
}
hipError_t launch_gated_scan_bwd(const GatedArgs& a) {
    if (a.D == 0) return hipSuccess;
    return a.bf16 ? bwd_t<__bf16>(a) : bwd_t<float>(a);
}
hipError_t launch_gated_step(const GatedArgs& a) {
    if (a.B == 0 || a.D == 0) return hipSuccess;
    GatedDev p = dev(a);
    p.cb = (unsigned)((a.D + 63) / 64);
    const unsigned blocks = (unsigned)(a.B * p.cb);
    if (a.bf16)
        LA_TRACED(a.tr, "gated_step", gated_step_kernel<__bf16><<<blocks, 64, 0, a.stream>>>(p));
    else
        LA_TRACED(a.tr, "gated_step", gated_step_kernel<float><<<blocks, 64, 0, a.stream>>>(p));
    return hipGetLastError();
}

}  // namespace la
