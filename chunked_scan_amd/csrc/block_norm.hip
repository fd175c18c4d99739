// block_norm.hip -- what stands between two blocks of a layer, its backward, and dropout.
//
//   n = x rp w_post (or x),  u = n act(gate) scale,  h = residual + drop(u),  y = h rq w_pre
//
// Memory-bound: every input element is read once into registers and every output written once, both norms' statistics
// and the dropped elements' places are made in between.  A row belongs to TPR threads, each holding VPT chunks of 8
// adjacent elements in fp32.  The mask is Philox4x32-10's output for the chunk's counter, one call per chunk: 16 bits an
// element, so that the generator's 20 wide products cost 8 elements, not 4; the probability is a multiple of 2^-16 for it,
// and the kept share in the scale is exact.
//
// Measured, bf16: norms, gate and scale over 16384 x 2048 63 to 68 us (335 MB, 5 TB/s, a copy's rate); their backward with
// dropout over 8191 x 2048 53 + 6 us (268 MB; fp32 over 4096 x 2048 56 us, 4.8 TB/s); dropout with a residual of 16384 x 2048 33 us (201 MB, 6.0 TB/s, of which the last-level
// cache holds a part).  A mask made by its counter costs no more than the loads hide.
#include <algorithm>

#include "la_mixer.h"
#include "row_ops.h"

namespace la {
namespace {

struct BlockDev {
    const void* x;
    const void* gate;
    const void* residual;
    const float* w_post;
    const float* scale;
    const float* w_pre;
    const uint64_t* rng;
    void* y;
    void* h;
    float* rstd_post;
    float* rstd_pre;
    const void* h_in;
    const float* rstd_post_in;
    const float* rstd_pre_in;
    const void* dy;
    const void* dh;
    void* dx;
    void* dgate;
    void* dres;
    float* part;  // [blocks, 2, D]: the sums of du xh act(gate) and of dy times the normed stream
    int64_t M, D, chunks;
    int act;
    unsigned drop;
    float keep_scale, eps, inv_d;
    int64_t sx, sg, sres, sy, sh, sdy, sdh, sdx, sdg, sdres;
};

// 8 adjacent elements as they lie in memory, of which n exist (VEC: all, on 16 bytes).  Rows that are not 16-byte aligned
// are accessed in 16 bytes all the same, which the hardware takes at any address; only a row's last elements, fewer
// than 8, are stored one by one (8000 x 2047 bf16: forward 153 us with all elements one by one, 50 so, aligned 2048 42;
// backward of 4000 rows 93, 49 and 38).  ONCE: streaming loads.
template <typename V> struct __attribute__((packed, aligned(2))) Unaligned {
    V v;
};
template <typename V, bool VEC, bool ONCE>
__device__ __forceinline__ V word_at(const void* p) {
    if (!VEC) return ((const Unaligned<V>*)p)->v;
    return load_word<V, ONCE>((const V*)p);
}
template <typename E, bool VEC> struct Chunk;
// `back`: the row has 8 elements at least, so that its last ones can be loaded with those before them and moved into
// place afterwards: put together from single loads they would be waited for where they are loaded.
template <bool VEC> struct Chunk<__bf16, VEC> {
    u32x4 r;
    template <bool ONCE = false>
    __device__ __forceinline__ void load(const __bf16* p, int n, bool back) {
        if (VEC || back) {
            r = word_at<u32x4, VEC, ONCE>(VEC ? p : p - (8 - n));
            return;
        }
        const uint16_t* e = (const uint16_t*)p;
#pragma unroll
        for (int i = 0; i < 4; i++)
            r[i] = (2 * i < n ? (uint32_t)e[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)e[2 * i + 1] << 16 : 0u);
    }
    __device__ __forceinline__ void get(float* f, int n, bool back) const {
        u32x4 t = r;
        if (!VEC && back && n < 8) {
            const int by = 8 - n;  // elements to drop in front
            if (by & 4) t = u32x4{t[2], t[3], 0, 0};
            if (by & 2) t = u32x4{t[1], t[2], t[3], 0};
            if (by & 1) t = u32x4{t[0] >> 16 | t[1] << 16, t[1] >> 16 | t[2] << 16, t[2] >> 16 | t[3] << 16, t[3] >> 16};
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            f[2 * i] = bits_lo_bf16(t[i]);
            f[2 * i + 1] = bits_hi_bf16(t[i]);
        }
    }
};
template <bool VEC> struct Chunk<float, VEC> {
    f32x4 a, b;
    template <bool ONCE = false>
    __device__ __forceinline__ void load(const float* p, int n, bool) {
        if (VEC || n == 8) {
            a = word_at<f32x4, VEC, ONCE>(p);
            b = word_at<f32x4, VEC, ONCE>(p + 4);
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            a[i] = i < n ? p[i] : 0.f;
            b[i] = 4 + i < n ? p[4 + i] : 0.f;
        }
    }
    __device__ __forceinline__ void get(float* f, int, bool) const {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            f[i] = a[i];
            f[4 + i] = b[i];
        }
    }
};
template <typename E, bool VEC, bool ONCE = false>
__device__ __forceinline__ void get8(const E* p, int n, bool back, float* f) {
    Chunk<E, VEC> c;
    c.template load<ONCE>(p, n, back);
    c.get(f, n, back);
}
template <typename E, bool VEC>
__device__ __forceinline__ void put8(E* p, int n, const float* f) {
    if (VEC) {
        store8<E, true>(p, 8, f);
    } else if (n == 8) {
        if (sizeof(E) == 2) {
            ((Unaligned<u32x4>*)p)->v = pack8_pairs(f);
        } else {
            ((Unaligned<f32x4>*)p)->v = f32x4{f[0], f[1], f[2], f[3]};
            ((Unaligned<f32x4>*)(p + 4))->v = f32x4{f[4], f[5], f[6], f[7]};
        }
    } else {
        store8<E, false>(p, n, f);
    }
}

// Philox4x32-10: ten rounds of two 32 x 32 -> 64 bit products on a 128-bit counter, the key stepped by the Weyl
// constants (Salmon, Moraes, Dror, Shaw: Parallel random numbers: as easy as 1, 2, 3; 2011).
__device__ __forceinline__ u32x4 philox(uint64_t lo, uint64_t hi, uint64_t key) {
    uint32_t c0 = (uint32_t)lo, c1 = (uint32_t)(lo >> 32), c2 = (uint32_t)hi, c3 = (uint32_t)(hi >> 32);
    uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
    for (int i = 0; i < 10; i++) {
        const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)p1;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)p0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4{c0, c1, c2, c3};
}
// The generator's key and offset, uniform.
struct Rng {
    uint64_t key, offset;
};
__device__ __forceinline__ Rng load_rng(const uint64_t* p) { return {p[0], p[1]}; }
// Bit j of the result: element j of the chunk is kept.
__device__ __forceinline__ uint32_t keep_bits(const Rng& r, int64_t chunk, uint32_t drop) {
    const u32x4 w = philox((uint64_t)chunk, r.offset, r.key);
    uint32_t k = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) k |= (((w[j >> 1] >> (16 * (j & 1))) & 0xffffu) >= drop ? 1u : 0u) << j;
    return k;
}

// The gate's factor, and with its derivative.
__device__ __forceinline__ float act(float g, int kind) {
    if (kind == LA_GATE_LINEAR) return g;
    const float s = sigmoid(g);
    return kind == LA_GATE_SIGMOID ? s : g * s;
}
__device__ __forceinline__ void act_slope(float g, int kind, float* f, float* df) {
    *f = g;
    *df = 1.f;
    if (kind == LA_GATE_LINEAR) return;
    const float e = __builtin_amdgcn_exp2f(g * -LOG2E), s = rcp(1.f + e), shut = complement(e, s);
    *f = kind == LA_GATE_SIGMOID ? s : g * s;
    *df = kind == LA_GATE_SIGMOID ? s * shut : s * fmaf(g, shut, 1.f);
}

template <typename E, int TPR, int VPT, bool VEC, bool DROP>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void block_norm_kernel(BlockDev p) {
    __shared__ float buf[16];
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
    const bool back = p.D >= 8;
    const int tid = threadIdx.x % TPR;
    const int64_t m = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
    if (m >= p.M) return;  // whole waves; TPR >= 256: whole blocks
    float v[VPT][8];
    float ss = 0.f;
    // one chunk a thread: everything is loaded before the first sum, whose wait then covers it
    constexpr bool AHEAD = VPT == 1;
    Chunk<E, VEC> gate0, res0;
    Chunk<float, VEC> post0, scale0, pre0;
    if (AHEAD) {
        const int n = (int)min((int64_t)8, p.D - (int64_t)tid * 8);
        if (n > 0) {
            if (p.gate) gate0.load((const E*)p.gate + m * p.sg + tid * 8, n, back);
            if (p.residual) res0.load((const E*)p.residual + m * p.sres + tid * 8, n, back);
            if (p.w_post) post0.load(p.w_post + tid * 8, n, back);
            if (p.scale) scale0.load(p.scale + tid * 8, n, back);
            if (p.w_pre) pre0.load(p.w_pre + tid * 8, n, back);
        }
    }
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int64_t d = (int64_t)(i * TPR + tid) * 8;
        const int n = (int)min((int64_t)8, p.D - d);
        if (n > 0) {
            get8<E, VEC, true>((const E*)p.x + m * p.sx + d, n, back, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) v[i][j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; j++) ss = fmaf(v[i][j], v[i][j], ss);
    }
    RowScale rp = {1.f, 1.f};
    if (p.w_post) {
        rp = row_rstd<TPR, VPT>(v, ss, p.inv_d, p.eps, buf);
        if (p.rstd_post && tid == 0) p.rstd_post[m] = rp.own();
    }
    Rng rng = {};
    if (DROP) rng = load_rng(p.rng);
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int64_t d = (int64_t)(i * TPR + tid) * 8;
        const int n = (int)min((int64_t)8, p.D - d);
        if (n <= 0) continue;
        float f[8];
        if (p.w_post) {
            if (AHEAD) post0.get(f, n, back);
            else get8<float, VEC>(p.w_post + d, n, back, f);
#pragma unroll
            for (int j = 0; j < 8; j++) v[i][j] = v[i][j] * rp.s * (rp.r * f[j]);
        }
        if (p.gate) {
            if (AHEAD) gate0.get(f, n, back);
            else get8<E, VEC, true>((const E*)p.gate + m * p.sg + d, n, back, f);
#pragma unroll
            for (int j = 0; j < 8; j++) v[i][j] *= act(f[j], p.act);
        }
        if (p.scale) {
            if (AHEAD) scale0.get(f, n, back);
            else get8<float, VEC>(p.scale + d, n, back, f);
#pragma unroll
            for (int j = 0; j < 8; j++) v[i][j] *= f[j];
        }
        if (DROP) {
            const uint32_t k = keep_bits(rng, m * p.chunks + (i * TPR + tid), p.drop);
#pragma unroll
            for (int j = 0; j < 8; j++) v[i][j] = (k >> j) & 1 ? v[i][j] * p.keep_scale : 0.f;
        }
        if (p.residual) {
            if (AHEAD) res0.get(f, n, back);
            else get8<E, VEC, true>((const E*)p.residual + m * p.sres + d, n, back, f);
#pragma unroll
            for (int j = 0; j < 8; j++) v[i][j] += f[j];
        }
        if (!VEC)
#pragma unroll
            for (int j = 0; j < 8; j++) v[i][j] = j < n ? v[i][j] : 0.f;
        put8<E, VEC>((E*)p.h + m * p.sh + d, n, v[i]);
#pragma unroll
        for (int j = 0; j < 8; j++) ss = fmaf(v[i][j], v[i][j], ss);
    }
    if (!p.w_pre) return;
    const RowScale rq = row_rstd<TPR, VPT>(v, ss, p.inv_d, p.eps, buf);
    if (p.rstd_pre && tid == 0) p.rstd_pre[m] = rq.own();
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int64_t d = (int64_t)(i * TPR + tid) * 8;
        const int n = (int)min((int64_t)8, p.D - d);
        if (n <= 0) continue;
        float w[8];
        if (AHEAD) pre0.get(w, n, back);
        else get8<float, VEC>(p.w_pre + d, n, back, w);
#pragma unroll
        for (int j = 0; j < 8; j++) w[j] *= v[i][j] * rq.s * rq.r;
        put8<E, VEC>((E*)p.y + m * p.sy + d, n, w);
    }
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
// The wave's sum in all lanes: lanes 1, 2 apart, the two halves of 8 and of 16 mirrored, then the four rows of 16.
__device__ __forceinline__ float wave_total(float v) {
    v = dpp_add<0xb1>(v);   // quad_perm 1 0 3 2
    v = dpp_add<0x4e>(v);   // quad_perm 2 3 0 1
    v = dpp_add<0x141>(v);  // row_half_mirror
    v = dpp_add<0x140>(v);  // row_mirror
    auto row = [&](int l) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l)); };
    return (row(0) + row(16)) + (row(32) + row(48));
}
// The sum over a row's TPR threads, of every row of the block at once.  One barrier: successive calls alternate between
// two sets of words, so a set is written again only behind the barrier that everyone reaches after reading it.
template <int TPR>
__device__ __forceinline__ float rows_total(float v, float (*buf)[16], int& set) {
    v = wave_total(v);
    if (TPR == 64) return v;
    const int w = threadIdx.x >> 6, first = w / (TPR / 64) * (TPR / 64);
    if ((threadIdx.x & 63) == 0) buf[set][w] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 64; i++) v += buf[set][first + i];
    set ^= 1;
    return v;
}

// Backward.  A block holds ROWS rows at a time and walks the rows grid-stride; each thread keeps its channels' share of the
// three parameters' sums in registers, the block's rows add theirs up at the end (LDS, one after the other) and write one
// row of `part`.  All of a row is loaded before its first sum, the next row's before this one's where the registers allow
// (2-byte types, one chunk a thread; unaligned rows up to 2048 channels): a block waits for two sums over its rows, and
// with the loads behind them it left the memory idle (8191 x 2048 bf16 with gate and dropout, 268 MB: 95.6 -> 59.6 us a
// pass, 4.5 TB/s).  Blocks of 4 waves, three of them a CU within 168 registers: at four, whose 128 spill, 68.7 us, and
// blocks of 8 waves 73.  Over 8192 channels two chunks a thread do not fit the 128 registers of 16 waves: 125 to 213 spill
// (unaligned 329 to 1127), and that bounds it: 4096 x 16384 bf16 444 us, 2.4 TB/s, fp32 905; 4096 x 9000 295 and 587.
constexpr int bwd_threads(int tpr) { return tpr > 256 ? tpr : 256; }
template <typename E, int TPR, int VPT, bool VEC, bool DROP>
__global__ __launch_bounds__(bwd_threads(TPR), TPR <= 256 || !VEC ? 3 : 4) void block_norm_bwd_kernel(BlockDev p) {
    constexpr int ROWS = bwd_threads(TPR) / TPR;
    constexpr bool AHEAD = sizeof(E) == 2 && VPT == 1 && (VEC || TPR <= 256);
    typedef Chunk<E, VEC> C;
    __shared__ float buf[2][16];
    __shared__ float acc[ROWS > 1 ? TPR * VPT * 16 : 1];
    const int tid = threadIdx.x % TPR, rw = threadIdx.x / TPR;
    const bool back = p.D >= 8;
    int set = 0;
    float sum[2][VPT][8], wq[VPT][8], ws[VPT][8];  // ws = w_post scale
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int64_t d = (int64_t)(i * TPR + tid) * 8;
        const int n = (int)min((int64_t)8, p.D - d);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            sum[0][i][j] = sum[1][i][j] = 0.f;
            wq[i][j] = ws[i][j] = 1.f;
        }
        if (n > 0) {
            if (p.w_pre) get8<float, VEC>(p.w_pre + d, n, back, wq[i]);
            if (p.w_post) get8<float, VEC>(p.w_post + d, n, back, ws[i]);
            if (p.scale) {
                float sc[8];
                get8<float, VEC>(p.scale + d, n, back, sc);
#pragma unroll
                for (int j = 0; j < 8; j++) ws[i][j] *= sc[j];
            }
        }
    }
    Rng rng = {};
    if (DROP) rng = load_rng(p.rng);
    struct Row {
        C h[VPT], dy[VPT], dh[VPT], x[VPT], g[VPT];
        float rq, rp;
    };
    auto load = [&](Row& r, int64_t m) {
        if (m >= p.M) return;
        r.rq = p.w_pre ? p.rstd_pre_in[m] : 0.f;
        r.rp = p.w_post ? p.rstd_post_in[m] : 1.f;
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int64_t d = (int64_t)(i * TPR + tid) * 8;
            const int n = (int)min((int64_t)8, p.D - d);
            if (n <= 0) continue;
            if (p.w_pre) {
                r.h[i].load((const E*)p.h_in + m * p.sh + d, n, back);
                r.dy[i].load((const E*)p.dy + m * p.sdy + d, n, back);
            }
            if (p.dh) r.dh[i].load((const E*)p.dh + m * p.sdh + d, n, back);
            r.x[i].load((const E*)p.x + m * p.sx + d, n, back);
            if (p.gate) r.g[i].load((const E*)p.gate + m * p.sg + d, n, back);
        }
    };
    const int64_t step = (int64_t)gridDim.x * ROWS;
    Row cur, next;
    load(cur, (int64_t)blockIdx.x * ROWS + rw);
    // all rows of a block take the same turns: those behind the last one only for the barriers
    for (int64_t m0 = (int64_t)blockIdx.x * ROWS; m0 < p.M; m0 += step) {
        const int64_t m = m0 + rw;
        const bool live = m < p.M;
        if (AHEAD) load(next, m + step);
        float t[VPT][8], xh[VPT][8];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int n = (int)min((int64_t)8, p.D - (int64_t)(i * TPR + tid) * 8);
            const bool there = live && n > 0;
#pragma unroll
            for (int j = 0; j < 8; j++) t[i][j] = xh[i][j] = 0.f;
            if (!there || !p.w_pre) continue;
            cur.h[i].get(xh[i], n, back);
            cur.dy[i].get(t[i], n, back);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                xh[i][j] *= cur.rq;  // the normed stream
                sum[1][i][j] = fmaf(t[i][j], xh[i][j], sum[1][i][j]);
                t[i][j] *= wq[i][j];
                dot = fmaf(t[i][j], xh[i][j], dot);
            }
        }
        if (p.w_pre) dot = rows_total<TPR>(dot, buf, set) * p.inv_d;
        float dot2 = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int64_t d = (int64_t)(i * TPR + tid) * 8;
            const int n = (int)min((int64_t)8, p.D - d);
            if (!live || n <= 0) continue;
            float f[8], g[8], o[8];
#pragma unroll
            for (int j = 0; j < 8; j++) t[i][j] = cur.rq * fmaf(-xh[i][j], dot, t[i][j]);
            if (p.dh) {
                cur.dh[i].get(f, n, back);
#pragma unroll
                for (int j = 0; j < 8; j++) t[i][j] += f[j];
            }
            if (p.dres) put8<E, VEC>((E*)p.dres + m * p.sdres + d, n, t[i]);
            uint32_t k = 0xff;
            if (DROP) k = keep_bits(rng, m * p.chunks + (i * TPR + tid), p.drop);
            cur.x[i].get(xh[i], n, back);
            if (p.gate) cur.g[i].get(g, n, back);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const bool kept = !DROP || ((k >> j) & 1);
                float a = 1.f, da = 1.f;
                if (p.gate) act_slope(g[j], p.act, &a, &da);
                xh[i][j] *= cur.rp;
                const float du = DROP ? t[i][j] * p.keep_scale : t[i][j], e = du * xh[i][j];
                o[j] = kept ? e * ws[i][j] * da : 0.f;
                sum[0][i][j] += kept ? e * a : 0.f;
                t[i][j] = kept ? du * a * ws[i][j] : 0.f;
                dot2 = fmaf(t[i][j], xh[i][j], dot2);
            }
            if (p.dgate) put8<E, VEC>((E*)p.dgate + m * p.sdg + d, n, o);
        }
        dot2 = p.w_post ? rows_total<TPR>(dot2, buf, set) * p.inv_d : 0.f;
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int64_t d = (int64_t)(i * TPR + tid) * 8;
            const int n = (int)min((int64_t)8, p.D - d);
            if (!live || n <= 0) continue;
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; j++) o[j] = p.w_post ? cur.rp * fmaf(-xh[i][j], dot2, t[i][j]) : t[i][j];
            put8<E, VEC>((E*)p.dx + m * p.sdx + d, n, o);
        }
        if (AHEAD) cur = next;
        else load(cur, m + step);
    }
    if (ROWS > 1) {
        for (int r = 0; r < ROWS; r++) {
            if (rw == r)
#pragma unroll
                for (int q = 0; q < 2; q++)
#pragma unroll
                    for (int i = 0; i < VPT; i++)
#pragma unroll
                        for (int j = 0; j < 8; j++) {
                            float* a = acc + ((q * VPT + i) * 8 + j) * TPR + tid;
                            if (r > 0) sum[q][i][j] += *a;
                            if (r < ROWS - 1) *a = sum[q][i][j];
                        }
            __syncthreads();
        }
        if (rw != ROWS - 1) return;
    }
#pragma unroll
    for (int q = 0; q < 2; q++)
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int64_t d = (int64_t)(i * TPR + tid) * 8;
            const int n = (int)min((int64_t)8, p.D - d);
            if (n > 0) put8<float, VEC>(p.part + ((int64_t)blockIdx.x * 2 + q) * p.D + d, n, sum[q][i]);
        }
}

// The parameters' derivatives: sums over the blocks' rows, 16 channels per block, 16 threads each.  blockIdx.y = 0: S = sum
// du xh act(gate), of which w_post's is S scale and scale's S w_post; 1: w_pre's.
__global__ __launch_bounds__(256) void block_norm_sums_kernel(BlockDev p, float* __restrict__ dw_post, float* __restrict__ dscale,
                                                              float* __restrict__ dw_pre, int64_t rows) {
    __shared__ float sum[16][16];
    const int dl = threadIdx.x & 15, share = threadIdx.x >> 4;
    const int64_t d = (int64_t)blockIdx.x * 16 + dl;
    if (blockIdx.y ? !dw_pre : !dw_post && !dscale) return;
    float s = 0.f;
    if (d < p.D)
#pragma unroll 4
        for (int64_t r = share; r < rows; r += 16) s += p.part[(r * 2 + blockIdx.y) * p.D + d];
    sum[share][dl] = s;
    __syncthreads();
    if (share != 0 || d >= p.D) return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i++) s += sum[i][dl];
    if (blockIdx.y) {
        dw_pre[d] = s;
    } else {
        if (dw_post) dw_post[d] = p.scale ? s * p.scale[d] : s;
        if (dscale) dscale[d] = p.w_post ? s * p.w_post[d] : s;
    }
}

// y = residual + drop(x): a thread per chunk of 8, chunks of all rows in one line.
template <typename E, bool VEC, bool DROP>
__global__ __launch_bounds__(256) void dropout_kernel(BlockDev p) {
    Rng rng = {};
    if (DROP) rng = load_rng(p.rng);
    const bool back = p.D >= 8;
    const int64_t total = p.M * p.chunks;
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < total; q += (int64_t)gridDim.x * 256) {
        const int64_t m = q / p.chunks, d = (q - m * p.chunks) * 8;
        const int n = (int)min((int64_t)8, p.D - d);
        float v[8], f[8];
        get8<E, VEC, true>((const E*)p.x + m * p.sx + d, n, back, v);
        if (DROP) {
            const uint32_t k = keep_bits(rng, q, p.drop);
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = (k >> j) & 1 ? v[j] * p.keep_scale : 0.f;
        }
        if (p.residual) {
            get8<E, VEC, true>((const E*)p.residual + m * p.sres + d, n, back, f);
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] += f[j];
        }
        put8<E, VEC>((E*)p.y + m * p.sy + d, n, v);
    }
}

// Blocks of the backward, so rows of partial sums: as many as 256 CUs hold at once (their registers allow three blocks of
// 4 waves a CU; two of 8, of which aligned rows spill 6 to 16 registers for it, unaligned ones come in two rounds; one
// of 16).
int64_t bwd_rows(int64_t M, int64_t D) { return std::min<int64_t>(D <= 2048 ? 768 : D <= 4096 ? 512 : 256, M); }

BlockDev dev(const BlockArgs& a) {
    BlockDev p = {};
    p.x = a.x; p.gate = a.gate; p.residual = a.residual; p.w_post = a.w_post; p.scale = a.scale; p.w_pre = a.w_pre;
    p.rng = a.rng; p.y = a.y; p.h = a.h; p.rstd_post = a.rstd_post; p.rstd_pre = a.rstd_pre; p.h_in = a.h_in;
    p.rstd_post_in = a.rstd_post_in; p.rstd_pre_in = a.rstd_pre_in; p.dy = a.dy; p.dh = a.dh; p.dx = a.dx;
    p.dgate = a.dgate; p.dres = a.dres; p.part = (float*)a.ws;
    p.M = a.M; p.D = a.D; p.chunks = (a.D + 7) / 8; p.act = a.act; p.drop = a.drop; p.eps = a.eps;
    p.inv_d = 1.f / (float)a.D;
    p.keep_scale = 65536.f / (float)(65536 - a.drop);
    p.sx = a.sx; p.sg = a.sg; p.sres = a.sres; p.sy = a.sy; p.sh = a.sh; p.sdy = a.sdy; p.sdh = a.sdh; p.sdx = a.sdx;
    p.sdg = a.sdg; p.sdres = a.sdres;
    return p;
}
bool vec_rows(const BlockArgs& a, size_t es) {
    auto w16 = [](const float* q) { return (uintptr_t)q % 16 == 0; };
    return a.D % 8 == 0 && row16(a.x, a.sx, es) && row16(a.gate, a.sg, es) && row16(a.residual, a.sres, es) &&
           row16(a.y, a.sy, es) && row16(a.h, a.sh, es) && row16(a.h_in, a.sh, es) && row16(a.dy, a.sdy, es) &&
           row16(a.dh, a.sdh, es) && row16(a.dx, a.sdx, es) && row16(a.dgate, a.sdg, es) && row16(a.dres, a.sdres, es) &&
           w16(a.w_post) && w16(a.scale) && w16(a.w_pre);
}

template <typename E, int TPR, int VPT, bool VEC, bool DROP>
void fwd_k(const BlockArgs& a, const BlockDev& p) {
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1, TH = TPR < 256 ? 256 : TPR;
    LA_TRACED(a.tr, "block_norm", block_norm_kernel<E, TPR, VPT, VEC, DROP>
              <<<(unsigned)((a.M + ROWS - 1) / ROWS), TH, 0, a.stream>>>(p));
}
template <typename E, int TPR, int VPT, bool VEC, bool DROP>
void bwd_k(const BlockArgs& a, const BlockDev& p) {
    constexpr int TH = bwd_threads(TPR), ROWS = TH / TPR;
    const int64_t blocks = std::min<int64_t>(bwd_rows(a.M, a.D), (a.M + ROWS - 1) / ROWS);
    if (blocks > 0)
        LA_TRACED(a.tr, "block_norm_bwd",
                  block_norm_bwd_kernel<E, TPR, VPT, VEC, DROP><<<(unsigned)blocks, TH, 0, a.stream>>>(p));
    if (a.dw_post || a.dscale || a.dw_pre)
        LA_TRACED(a.tr, "block_norm_bwd_sums", block_norm_sums_kernel<<<dim3((unsigned)((a.D + 15) / 16), 2), 256, 0, a.stream>>>(
                                                 p, a.dw_post, a.dscale, a.dw_pre, blocks));
}

template <typename E, bool VEC, bool DROP>
hipError_t run_v(const BlockArgs& a, const BlockDev& p, bool bwd) {
    const int64_t ch = (a.D + 7) / 8;
    if (!bwd) {
        // One chunk a thread, all loads ahead of the sums (16384 x 2048 bf16 with gate 69.8 -> 66.5 us against four chunks
        // in one wave; 1024 rows 8.3 -> 5.9; 64 rows 7.5 -> 3.7), but where that leaves half of the threads without one or
        // a row to 16 waves: 8192 x 1024 18.3 us in two chunks, 20.2 in one; 2048 x 8192 42 in four, 47 in one.  Few rows
        // are a matter of latency and take the most threads.
        const bool few = a.M <= 512;
        if (ch <= 64) fwd_k<E, 64, 1, VEC, DROP>(a, p);
        else if (ch <= 128 && !few) fwd_k<E, 64, 2, VEC, DROP>(a, p);
        else if (ch <= 256) fwd_k<E, 256, 1, VEC, DROP>(a, p);
        else if (ch <= 512) fwd_k<E, 512, 1, VEC, DROP>(a, p);
        else if (ch <= 1024 && !few) fwd_k<E, 256, 4, VEC, DROP>(a, p);
        else if (ch <= 1024) fwd_k<E, 1024, 1, VEC, DROP>(a, p);
        else fwd_k<E, 1024, 2, VEC, DROP>(a, p);
    } else {
        if (ch <= 64) bwd_k<E, 64, 1, VEC, DROP>(a, p);
        else if (ch <= 256) bwd_k<E, 256, 1, VEC, DROP>(a, p);
        else if (ch <= 512) bwd_k<E, 512, 1, VEC, DROP>(a, p);
        else if (ch <= 1024) bwd_k<E, 1024, 1, VEC, DROP>(a, p);
        else bwd_k<E, 1024, 2, VEC, DROP>(a, p);
    }
    return hipGetLastError();
}
template <typename E>
hipError_t run(const BlockArgs& a, bool bwd) {
    const BlockDev p = dev(a);
    const bool vec = vec_rows(a, sizeof(E)), drop = a.drop > 0;
    if (vec) return drop ? run_v<E, true, true>(a, p, bwd) : run_v<E, true, false>(a, p, bwd);
    return drop ? run_v<E, false, true>(a, p, bwd) : run_v<E, false, false>(a, p, bwd);
}

template <typename E, bool VEC>
void dropout_v(const BlockArgs& a, const BlockDev& p) {
    const unsigned blocks = (unsigned)std::min<int64_t>((a.M * p.chunks + 255) / 256, 1 << 20);
    if (a.drop > 0)
        LA_TRACED(a.tr, "dropout", dropout_kernel<E, VEC, true><<<blocks, 256, 0, a.stream>>>(p));
    else
        LA_TRACED(a.tr, "dropout", dropout_kernel<E, VEC, false><<<blocks, 256, 0, a.stream>>>(p));
}

}  // namespace

size_t block_norm_bwd_ws(int64_t M, int64_t D) { return (size_t)(bwd_rows(M, D) * 2 * D) * sizeof(float); }

hipError_t launch_block_norm(const BlockArgs& a) {
    if (a.M == 0) return hipSuccess;
    return a.bf16 ? run<__bf16>(a, false) : run<float>(a, false);
}
hipError_t launch_block_norm_bwd(const BlockArgs& a) { return a.bf16 ? run<__bf16>(a, true) : run<float>(a, true); }

hipError_t launch_dropout(const BlockArgs& a) {
    if (a.M == 0) return hipSuccess;
    const BlockDev p = dev(a);
    if (a.bf16)
        vec_rows(a, 2) ? dropout_v<__bf16, true>(a, p) : dropout_v<__bf16, false>(a, p);
    else
        vec_rows(a, 4) ? dropout_v<float, true>(a, p) : dropout_v<float, false>(a, p);
    return hipGetLastError();
}

}  // namespace la
