// short_conv.hip -- the depthwise causal convolution of 2 to 4 taps, its backward and its
// single-token form.
//
//   v_t[d] = bias[d] + sum_j w[d, j] x_{t-W+1+j}[d],   y = v or v sigmoid(v)
//
// Memory-bound: a handful of operations per element read and written.  A thread owns VEC adjacent
// channels (one 16-byte word, or one channel where rows are not 16-byte aligned) and walks a tile of
// tokens with the last W - 1 inputs in registers, so that each input is read once, plus W - 1 rows per
// tile from the neighbour's (which the cache holds).  Loads of TB tokens are in flight together.
//
// What is written once and not read here leaves the forward by a streaming store (st_once): 16384 x 2048 bf16,
// W = 4, in 26.8 us (134 MB, 5.0 TB/s; a copy of as many bytes takes 25.7), 33.0 with ordinary stores; streaming
// loads, which lose the neighbours' W - 1 rows, 28.8.  That is call after call; in a layer, whose projection and scan read
// the output next, both kinds of store take the same time (766 to 773 us for the whole prompt).  The backward keeps
// ordinary stores (28.1 and 27.9 us).
#include <algorithm>

#include "la_mixer.h"

namespace la {
namespace {

constexpr int TB = 4;  // tokens loaded together

template <typename E, int VEC> struct Vec;
template <> struct Vec<__bf16, 8> {
    typedef u32x4 raw;
    static __device__ __forceinline__ raw ld(const __bf16* p) { return *(const u32x4*)p; }
    static __device__ __forceinline__ void get(raw r, float* f) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            f[2 * i] = bits_lo_bf16(r[i]);
            f[2 * i + 1] = bits_hi_bf16(r[i]);
        }
    }
    static __device__ __forceinline__ void st(__bf16* p, const float* f) { *(u32x4*)p = pack8_pairs(f); }
    static __device__ __forceinline__ void st_once(__bf16* p, const float* f) {
        __builtin_nontemporal_store(pack8_pairs(f), (u32x4*)p);
    }
};
template <> struct Vec<__bf16, 4> {
    typedef u32x2 raw;
    static __device__ __forceinline__ raw ld(const __bf16* p) { return *(const u32x2*)p; }
    static __device__ __forceinline__ void get(raw r, float* f) {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            f[2 * i] = bits_lo_bf16(r[i]);
            f[2 * i + 1] = bits_hi_bf16(r[i]);
        }
    }
    static __device__ __forceinline__ void st(__bf16* p, const float* f) {
        *(u32x2*)p = u32x2{pack2(f[0], f[1]), pack2(f[2], f[3])};
    }
};
template <> struct Vec<float, 4> {
    typedef f32x4 raw;
    static __device__ __forceinline__ raw ld(const float* p) { return *(const f32x4*)p; }
    static __device__ __forceinline__ void get(raw r, float* f) {
#pragma unroll
        for (int i = 0; i < 4; i++) f[i] = r[i];
    }
    static __device__ __forceinline__ void st(float* p, const float* f) { *(f32x4*)p = f32x4{f[0], f[1], f[2], f[3]}; }
    static __device__ __forceinline__ void st_once(float* p, const float* f) {
        __builtin_nontemporal_store(f32x4{f[0], f[1], f[2], f[3]}, (f32x4*)p);
    }
};
template <typename E> struct Vec<E, 1> {
    typedef E raw;
    static __device__ __forceinline__ raw ld(const E* p) { return *p; }
    static __device__ __forceinline__ void get(raw r, float* f) { f[0] = (float)r; }
    static __device__ __forceinline__ void st(E* p, const float* f) { io<E>::st(p, f[0]); }
    static __device__ __forceinline__ void st_once(E* p, const float* f) { st(p, f); }
};

struct ConvDev {
    const void* x;
    const float* weight;
    const float* bias;
    const void* state_in;
    const int32_t* lengths;
    void* y;
    void* state_out;
    const void* dy;
    const void* d_state_out;
    void* dx;
    void* d_state_in;
    float* part;  // [B * tiles, W + 1, D]
    int64_t L, D;
    unsigned nvec, tiles;  // channel vectors; token tiles per sequence
    int TL;                // tokens per tile
    bool silu;
    la_rows sx, sy, sdy, sdx;
};

// The input at position p (negative: the state's), as floats.
template <typename E, int W, int VEC>
__device__ __forceinline__ void input_at(const ConvDev& c, int64_t b, int64_t pos, int64_t d, float* f) {
    typedef Vec<E, VEC> V;
    if (pos >= 0) {
        V::get(V::ld((const E*)c.x + b * c.sx.batch + pos * c.sx.token + d), f);
    } else if (c.state_in) {
        V::get(V::ld((const E*)c.state_in + (b * (W - 1) + (W - 1 + pos)) * c.D + d), f);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i++) f[i] = 0.f;
    }
}

// The taps and the bias of VEC channels: W VEC adjacent floats.
template <int W, int VEC>
__device__ __forceinline__ void load_taps(const ConvDev& c, int64_t d, float (*w)[VEC], float* bias) {
#pragma unroll
    for (int v = 0; v < VEC; v++)
#pragma unroll
        for (int j = 0; j < W; j++) w[j][v] = c.weight[(d + v) * W + j];
#pragma unroll
    for (int v = 0; v < VEC; v++) bias[v] = c.bias ? c.bias[d + v] : 0.f;
}

// A thread per (sequence, token tile, channel vector), channel vectors fastest; the sequence's last tile
// also writes state_out.  Full blocks of TB tokens, the next block's loads in flight, then the tile's rest.
template <typename E, int W, int VEC>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvDev c, unsigned total) {
    typedef Vec<E, VEC> V;
    const unsigned i = blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const int64_t d = (int64_t)(i % c.nvec) * VEC;
    const unsigned tile = i / c.nvec % c.tiles;
    const int64_t b = i / c.nvec / c.tiles;
    const int len = (int)seq_len(c.lengths, b, c.L);
    if (c.state_out && tile == c.tiles - 1) {
        for (int j = 0; j < W - 1; j++) {
            float f[VEC];
            input_at<E, W, VEC>(c, b, len - (W - 1) + j, d, f);
            V::st((E*)c.state_out + (b * (W - 1) + j) * c.D + d, f);
        }
    }
    const int t0 = tile * c.TL, t1 = min(t0 + c.TL, len);
    if (t0 >= t1) return;
    const E* xp = (const E*)c.x + b * c.sx.batch + t0 * c.sx.token + d;
    E* yp = (E*)c.y + b * c.sy.batch + t0 * c.sy.token + d;
    typename V::raw nx[TB];
    auto fetch = [&]() {
#pragma unroll
        for (int j = 0; j < TB; j++) nx[j] = V::ld(xp + j * c.sx.token);
        xp += TB * c.sx.token;
    };
    if (t0 + TB <= t1) fetch();
    float w[W][VEC], bias[VEC], x[W - 1 + TB][VEC];
#pragma unroll
    for (int j = 0; j < W - 1; j++) input_at<E, W, VEC>(c, b, t0 - (W - 1) + j, d, x[j]);
    load_taps<W, VEC>(c, d, w, bias);
    auto token = [&](int j) {
        float o[VEC];
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            float s = bias[v];
#pragma unroll
            for (int k = 0; k < W; k++) s = fmaf(w[k][v], x[j + k][v], s);
            o[v] = s;
        }
        if (c.silu)
#pragma unroll
            for (int v = 0; v < VEC; v++) o[v] *= sigmoid(o[v]);
        V::st_once(yp, o);
        yp += c.sy.token;
    };
    auto shift = [&](int n) {
#pragma unroll
        for (int j = 0; j < W - 1; j++)
#pragma unroll
            for (int v = 0; v < VEC; v++) x[j][v] = x[n + j][v];
    };
    int t = t0;
    for (; t + TB <= t1; t += TB) {
#pragma unroll
        for (int j = 0; j < TB; j++) V::get(nx[j], x[W - 1 + j]);
        if (t + 2 * TB <= t1) fetch();
#pragma unroll
        for (int j = 0; j < TB; j++) token(j);
        shift(TB);
    }
    for (; t < t1; t++) {
        V::get(V::ld(xp), x[W - 1]);
        xp += c.sx.token;
        token(0);
        shift(1);
    }
}

// Backward.  With p_t = dy_t act'(v_t) (zero outside the sequence), position s takes
//   dx_s = sum_j w[j] p_{s+W-1-j}  (+ d_state_out where s is one of the last W - 1 positions).
// A thread walks its tile's tokens t = t0 .. t1-1 and W - 1 more: at t it knows x_{t-W+1..t}, so v_t and
// p_t, and writes dx_{t-W+1}.  It owns p_t of its tile for the weight's sums; the tile that holds
// position 0 also owns the W - 1 positions before it, which are the incoming state's.  Between the first
// and the last W - 1 steps nothing is special and the loop is plain.
template <typename E, int W, int VEC>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvDev c, unsigned total) {
    typedef Vec<E, VEC> V;
    const unsigned i = blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const int64_t d = (int64_t)(i % c.nvec) * VEC;
    const unsigned tile = i / c.nvec % c.tiles;
    const int64_t b = i / c.nvec / c.tiles;
    const int len = (int)seq_len(c.lengths, b, c.L);
    const int t0 = tile * c.TL, te = (int)min((int64_t)t0 + c.TL, c.L), t1 = min(te, len);
    float w[W][VEC], bias[VEC], dw[W][VEC], db[VEC];
    float x[W - 1 + TB][VEC], p[W - 1 + TB][VEC];  // x_{t-W+1..}, p_{t-W+1..}: the last W - 1 and the block's
    load_taps<W, VEC>(c, d, w, bias);
#pragma unroll
    for (int v = 0; v < VEC; v++) {
#pragma unroll
        for (int j = 0; j < W; j++) dw[j][v] = 0.f;
        db[v] = 0.f;
    }
    const E* xb = (const E*)c.x + b * c.sx.batch + d;
    const E* yb = (const E*)c.dy + b * c.sdy.batch + d;
    E* gb = (E*)c.dx + b * c.sdx.batch + d;
    // p of the block's token j, from x[j .. j + W - 1]
    auto grad = [&](int j, typename V::raw dyr, bool in, bool own) {
        float dyv[VEC];
        V::get(dyr, dyv);
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            float g = dyv[v];
            if (c.silu) {
                float s = bias[v];
#pragma unroll
                for (int k = 0; k < W; k++) s = fmaf(w[k][v], x[j + k][v], s);
                const float sg = sigmoid(s);
                g *= sg * fmaf(s, 1.f - sg, 1.f);
            }
            g = in ? g : 0.f;
            p[W - 1 + j][v] = g;
            if (own) {
                db[v] += g;
#pragma unroll
                for (int k = 0; k < W; k++) dw[k][v] = fmaf(g, x[j + k][v], dw[k][v]);
            }
        }
    };
    // dx of position t - (W - 1), t the block's token j: p[j + k] = p_{s + k} meets tap W - 1 - k
    auto out = [&](int j, float* o) {
#pragma unroll
        for (int v = 0; v < VEC; v++) {
            o[v] = 0.f;
#pragma unroll
            for (int k = 0; k < W; k++) o[v] = fmaf(w[W - 1 - k][v], p[j + k][v], o[v]);
        }
    };
    auto shift = [&](int n) {
#pragma unroll
        for (int j = 0; j < W - 1; j++)
#pragma unroll
            for (int v = 0; v < VEC; v++) {
                x[j][v] = x[n + j][v];
                p[j][v] = p[n + j][v];
            }
    };
    const int s0 = tile == 0 ? -(W - 1) : t0, s1 = max(t1, 0);  // positions this tile writes
    // any token, one at a time
    auto step = [&](int t) {
        input_at<E, W, VEC>(c, b, min(t, len - 1), d, x[W - 1]);  // behind the end: any value, p is zero
        const bool in = t >= 0 && t < len;
        typename V::raw dyr = {};
        if (in) dyr = V::ld(yb + t * c.sdy.token);
        grad(0, dyr, in, in && t >= t0 && t < t1);
        const int s = t - (W - 1);
        if (s >= s0 && s < s1) {
            float o[VEC];
            out(0, o);
            const int so = s - (len - (W - 1));
            if (so >= 0 && c.d_state_out) {
                float f[VEC];
                V::get(V::ld((const E*)c.d_state_out + (b * (W - 1) + so) * c.D + d), f);
#pragma unroll
                for (int v = 0; v < VEC; v++) o[v] += f[v];
            }
            if (s >= 0)
                V::st(gb + s * c.sdx.token, o);
            else if (c.d_state_in)
                V::st((E*)c.d_state_in + (b * (W - 1) + (W - 1 + s)) * c.D + d, o);
        }
        shift(1);
    };
    if (s0 < t1 || tile == 0) {
        // x_{s0-W+1 .. s0-1}; below position -(W - 1) nothing reads them
#pragma unroll
        for (int j = 0; j < W - 1; j++) {
            const int pos = s0 - (W - 1) + j;
#pragma unroll
            for (int v = 0; v < VEC; v++) x[j][v] = p[j][v] = 0.f;
            if (pos >= -(W - 1)) input_at<E, W, VEC>(c, b, min(pos, len - 1), d, x[j]);
        }
        int t = s0;
        const int ta = max(s0 + W - 1, W - 1);  // from here on t - (W - 1) is a position >= 0 of this tile
        for (; t < min(ta, s1 + W - 1); t++) step(t);
        if (t + TB <= t1) {
            const E* xp = xb + t * c.sx.token;
            const E* yp = yb + t * c.sdy.token;
            E* gp = gb + (t - (W - 1)) * c.sdx.token;
            typename V::raw nx[TB], ny[TB];
            auto fetch = [&]() {
#pragma unroll
                for (int j = 0; j < TB; j++) {
                    nx[j] = V::ld(xp + j * c.sx.token);
                    ny[j] = V::ld(yp + j * c.sdy.token);
                }
                xp += TB * c.sx.token;
                yp += TB * c.sdy.token;
            };
            fetch();
            for (; t + TB <= t1; t += TB) {
                typename V::raw cy[TB];
#pragma unroll
                for (int j = 0; j < TB; j++) {
                    V::get(nx[j], x[W - 1 + j]);
                    cy[j] = ny[j];
                }
                if (t + 2 * TB <= t1) fetch();
#pragma unroll
                for (int j = 0; j < TB; j++) {
                    grad(j, cy[j], true, true);
                    float o[VEC];
                    out(j, o);
                    V::st(gp, o);
                    gp += c.sdx.token;
                }
                shift(TB);
            }
        }
        for (; t < s1 + W - 1; t++) step(t);
    }
    for (int t = max(t0, len); t < te; t++) {  // behind the sequence's end
        float zero[VEC];
#pragma unroll
        for (int v = 0; v < VEC; v++) zero[v] = 0.f;
        V::st(gb + t * c.sdx.token, zero);
    }
    float* part = c.part + ((b * c.tiles + tile) * (W + 1)) * c.D + d;
#pragma unroll
    for (int k = 0; k <= W; k++)
#pragma unroll
        for (int v = 0; v < VEC; v++) part[k * c.D + v] = k < W ? dw[k][v] : db[v];
}

// d_weight [D, W] and d_bias [D] from the tiles' sums: 16 channels of one tap (or the bias) per block, 16
// threads to a channel, each a share of the tiles.
__global__ __launch_bounds__(256) void conv_bwd_sums_kernel(const float* __restrict__ part, float* __restrict__ dw,
                                                            float* __restrict__ db, int64_t D, int W, int64_t rows) {
    __shared__ float sum[16][16];
    const int64_t cbn = (D + 15) / 16;
    const int k = (int)(blockIdx.x / cbn);
    const int dl = threadIdx.x & 15, share = threadIdx.x >> 4;
    const int64_t d = (blockIdx.x % cbn) * 16 + dl;
    float s = 0.f;
    if (d < D)
#pragma unroll 4
        for (int64_t r = share; r < rows; r += 16) s += part[(r * (W + 1) + k) * D + d];
    sum[share][dl] = s;
    __syncthreads();
    if (share != 0 || d >= D) return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i++) s += sum[i][dl];
    if (k < W)
        dw[d * W + k] = s;
    else if (db)
        db[d] = s;
}

// One token per sequence: a thread per (row, channel vector).
template <typename E, int W, int VEC>
__global__ __launch_bounds__(64) void conv_step_kernel(const E* __restrict__ x, const float* __restrict__ weight,
                                                       const float* __restrict__ bias, E* __restrict__ state,
                                                       const int32_t* __restrict__ slots, E* __restrict__ y, int64_t sx,
                                                       int64_t sy, int64_t D, unsigned nvec, unsigned cb, int nslots,
                                                       bool silu) {
    typedef Vec<E, VEC> V;
    const int64_t b = blockIdx.x / cb;
    const unsigned cv = blockIdx.x % cb * 64 + threadIdx.x;
    const int64_t slot = slots ? slots[b] : b;
    if (slot < 0 || slot >= nslots) return;
    const bool live = cv < nvec;
    const int64_t d = live ? (int64_t)cv * VEC : 0;
    E* st = state + slot * (W - 1) * D + d;
    typename V::raw old[W - 1], cur = V::ld(x + b * sx + d);
#pragma unroll
    for (int j = 0; j < W - 1; j++) old[j] = V::ld(st + j * D);
    float acc[VEC], f[VEC];
#pragma unroll
    for (int v = 0; v < VEC; v++) acc[v] = bias ? bias[d + v] : 0.f;
#pragma unroll
    for (int j = 0; j < W; j++) {
        V::get(j < W - 1 ? old[j] : cur, f);
#pragma unroll
        for (int v = 0; v < VEC; v++) acc[v] = fmaf(weight[(d + v) * W + j], f[v], acc[v]);
    }
    if (slots) {  // rows after the first that name a slot are padding
        bool dup = false;
        for (int64_t i = threadIdx.x; i < b; i += 64) dup |= slots[i] == (int32_t)slot;
        if (__any(dup)) return;
    }
    if (!live) return;
#pragma unroll
    for (int j = 0; j < W - 1; j++) *(typename V::raw*)(st + j * D) = j < W - 2 ? old[j + 1 < W - 1 ? j + 1 : j] : cur;
    if (silu)
#pragma unroll
        for (int v = 0; v < VEC; v++) acc[v] *= sigmoid(acc[v]);
    V::st(y + b * sy + d, acc);
}

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

// Tokens per thread: 16 in the forward and 32 in the backward (which writes W + 1 sums per channel and tile),
// fewer where that leaves under 2048 waves, two per SIMD.  Each tile re-reads W - 1 rows and loads the taps:
// 16384 x 2048 bf16, W = 4, ordinary stores: 8 tokens 35 us, 16 30, 32 33, 64 33; backward of 8192 x 2048: 16 tokens 38 + 8 us
// for the sums, 32 29 + 5, 64 32 + 4.
int tile_tokens(int64_t B, int64_t L, int64_t nvec, int TL) {
    while (TL > 8 && B * ((L + TL - 1) / TL) * nvec < 2048 * 64) TL /= 2;
    return TL;
}
int fwd_tile(int64_t B, int64_t L, int64_t nvec) { return tile_tokens(B, L, nvec, 16); }
int bwd_tile(int64_t B, int64_t L, int64_t nvec) { return tile_tokens(B, L, nvec, 32); }

template <typename E, int W, int VEC>
hipError_t fwd_w(const ConvArgs& a, ConvDev c) {
    c.nvec = (unsigned)(a.D / VEC);
    c.TL = fwd_tile(a.B, a.L, c.nvec);
    c.tiles = (unsigned)std::max<int64_t>(1, (a.L + c.TL - 1) / c.TL);
    const unsigned total = c.nvec * c.tiles * (unsigned)a.B;
    LA_TRACED(a.tr, "short_conv", conv_fwd_kernel<E, W, VEC><<<(total + 255) / 256, 256, 0, a.stream>>>(c, total));
    return hipGetLastError();
}
template <typename E, int W, int VEC>
hipError_t bwd_w(const ConvArgs& a, ConvDev c) {
    int64_t rows = 0;
    if (a.B > 0) {
        c.nvec = (unsigned)(a.D / VEC);
        c.TL = bwd_tile(a.B, a.L, c.nvec);
        c.tiles = (unsigned)std::max<int64_t>(1, (a.L + c.TL - 1) / c.TL);
        const unsigned total = c.nvec * c.tiles * (unsigned)a.B;
        rows = (int64_t)c.tiles * a.B;
        LA_TRACED(a.tr, "short_conv_bwd", conv_bwd_kernel<E, W, VEC><<<(total + 255) / 256, 256, 0, a.stream>>>(c, total));
    }
    LA_TRACED(a.tr, "short_conv_bwd_sums",
              conv_bwd_sums_kernel<<<(unsigned)((a.D + 15) / 16 * (W + 1)), 256, 0, a.stream>>>(c.part, a.d_weight, a.d_bias,
                                                                                              a.D, W, rows));
    return hipGetLastError();
}
template <typename E, int W, int VEC>
hipError_t step_w(const ConvArgs& a) {
    const unsigned nvec = (unsigned)(a.D / VEC), cb = (nvec + 63) / 64;
    LA_TRACED(a.tr, "short_conv_step",
              conv_step_kernel<E, W, VEC><<<cb * (unsigned)a.B, 64, 0, a.stream>>>(
                  (const E*)a.x, a.weight, a.bias, (E*)a.state, a.slots, (E*)a.y, a.sx.batch, a.sy.batch, a.D, nvec, cb,
                  a.nslots, a.silu));
    return hipGetLastError();
}

enum What { FWD, BWD, STEP };
template <typename E, int W, int VEC>
hipError_t run_w(What what, const ConvArgs& a, const ConvDev& c) {
    if constexpr (VEC == 1 || VEC == 4)
        if (what == BWD) return bwd_w<E, W, VEC>(a, c);
    if constexpr (VEC == 1 || VEC == 16 / sizeof(E))
        return what == FWD ? fwd_w<E, W, VEC>(a, c) : step_w<E, W, VEC>(a);
    return hipErrorInvalidValue;  // not reached
}
template <typename E, int VEC>
hipError_t run_v(What what, const ConvArgs& a, const ConvDev& c) {
    return a.width == 2 ? run_w<E, 2, VEC>(what, a, c) : a.width == 3 ? run_w<E, 3, VEC>(what, a, c)
                                                                       : run_w<E, 4, VEC>(what, a, c);
}
template <typename E>
hipError_t run(What what, const ConvArgs& a) {
    ConvDev c = {};
    c.x = a.x; c.weight = a.weight; c.bias = a.bias; c.state_in = a.state_in; c.lengths = a.lengths;
    c.y = a.y; c.state_out = a.state_out; c.dy = a.dy; c.d_state_out = a.d_state_out; c.dx = a.dx;
    c.d_state_in = a.d_state_in; c.part = (float*)a.ws;
    c.L = a.L; c.D = a.D; c.silu = a.silu;
    c.sx = a.sx; c.sy = a.sy; c.sdy = a.sdy; c.sdx = a.sdx;
    // 16 bytes a lane; the backward, with four times the registers per channel, 4 channels
    constexpr int VEC = 16 / sizeof(E);
    const size_t es = sizeof(E);
    const bool vec = a.D % VEC == 0 && rows16(a.x, a.sx, es) && rows16(a.y, a.sy, es) && rows16(a.dy, a.sdy, es) &&
                     rows16(a.dx, a.sdx, es) && aligned16(a.state_in) && aligned16(a.state_out) &&
                     aligned16(a.d_state_out) && aligned16(a.d_state_in) && aligned16(a.state);
    if (!vec) return run_v<E, 1>(what, a, c);
    return what == BWD ? run_v<E, 4>(what, a, c) : run_v<E, VEC>(what, a, c);
}
hipError_t run(What what, const ConvArgs& a) { return a.bf16 ? run<__bf16>(what, a) : run<float>(what, a); }

}  // namespace

// One row of W + 1 sums per token tile; the scalar form has the most threads and the longest tiles, so
// the vector form's count bounds both.
size_t short_conv_bwd_ws(int64_t B, int64_t L, int64_t D, int width) {
    const int64_t nvec = std::max<int64_t>(1, D / 4);
    const int TL = bwd_tile(B, L, nvec);
    return (size_t)(B * std::max<int64_t>(1, (L + TL - 1) / TL) * (width + 1) * D) * sizeof(float);
}

hipError_t launch_short_conv(const ConvArgs& a) { return a.B == 0 || a.D == 0 ? hipSuccess : run(FWD, a); }
hipError_t launch_short_conv_bwd(const ConvArgs& a) { return a.D == 0 ? hipSuccess : run(BWD, a); }
hipError_t launch_short_conv_step(const ConvArgs& a) { return a.B == 0 || a.D == 0 ? hipSuccess : run(STEP, a); }

}  // namespace la
