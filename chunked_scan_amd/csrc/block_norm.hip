// block_norm.hip -- what stands between two blocks of a layer, its backward, and dropout.
//
//   n = x rp w_post (or x),  u = n act(gate) scale,  h = residual + drop(u),  y = h rq w_pre
//
// Memory-bound: every input element is read once into registers and every output written once, both norms' statistics
// and the dropped elements' places are made in between.  A row belongs to TPR threads, each holding VPT chunks of 8
// adjacent elements in fp32.  The mask is Philox4x32-10's output for the chunk's counter, one call per chunk: 16 bits an
// element, so that the generator's 20 wide products cost 8 elements, not 4; the probability is a multiple of 2^-16 for it,
// and the kept share in the scale is exact.
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
    float* part;  // [blocks, 3, D]: dw_post, dscale, dw_pre
    int64_t M, D, chunks;
    int act;
    unsigned drop;
    float keep_scale, eps, inv_d;
    int64_t sx, sg, sres, sy, sh, sdy, sdh, sdx, sdg, sdres;
};

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
    const float s = sigmoid(g);
    *f = kind == LA_GATE_SIGMOID ? s : g * s;
    *df = kind == LA_GATE_SIGMOID ? s * (1.f - s) : s * fmaf(g, 1.f - s, 1.f);
}

template <typename E, int TPR, int VPT, bool VEC, bool DROP>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void block_norm_kernel(BlockDev p) {
    __shared__ float buf[16];
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
    const int tid = threadIdx.x % TPR;
    const int64_t m = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
    if (m >= p.M) return;  // whole waves; TPR >= 256: whole blocks
    float v[VPT][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int64_t d = (int64_t)(i * TPR + tid) * 8;
        const int n = (int)min((int64_t)8, p.D - d);
        if (n > 0) {
            load8<E, VEC, true>((const E*)p.x + m * p.sx + d, n, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) v[i][j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; j++) ss = fmaf(v[i][j], v[i][j], ss);
    }
    float rp = 1.f;
    if (p.w_post) {
        rp = row_rstd<TPR, VPT>(v, ss, p.inv_d, p.eps, buf);
        if (p.rstd_post && tid == 0) p.rstd_post[m] = rp;
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
            load8<float, VEC>(p.w_post + d, n, f);
#pragma unroll
            for (int j = 0; j < 8; j++) v[i][j] *= rp * f[j];
        }
        if (p.gate) {
            load8<E, VEC, true>((const E*)p.gate + m * p.sg + d, n, f);
#pragma unroll
            for (int j = 0; j < 8; j++) v[i][j] *= act(f[j], p.act);
        }
        if (p.scale) {
            load8<float, VEC>(p.scale + d, n, f);
#pragma unroll
            for (int j = 0; j < 8; j++) v[i][j] *= f[j];
        }
        if (DROP) {
            const uint32_t k = keep_bits(rng, m * p.chunks + (i * TPR + tid), p.drop);
#pragma unroll
            for (int j = 0; j < 8; j++) v[i][j] = (k >> j) & 1 ? v[i][j] * p.keep_scale : 0.f;
        }
        if (p.residual) {
            load8<E, VEC, true>((const E*)p.residual + m * p.sres + d, n, f);
#pragma unroll
            for (int j = 0; j < 8; j++) v[i][j] += f[j];
        }
        if (!VEC)
#pragma unroll
            for (int j = 0; j < 8; j++) v[i][j] = j < n ? v[i][j] : 0.f;
        store8<E, VEC>((E*)p.h + m * p.sh + d, n, v[i]);
#pragma unroll
        for (int j = 0; j < 8; j++) ss = fmaf(v[i][j], v[i][j], ss);
    }
    if (!p.w_pre) return;
    const float rq = row_rstd<TPR, VPT>(v, ss, p.inv_d, p.eps, buf);
    if (p.rstd_pre && tid == 0) p.rstd_pre[m] = rq;
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int64_t d = (int64_t)(i * TPR + tid) * 8;
        const int n = (int)min((int64_t)8, p.D - d);
        if (n <= 0) continue;
        float w[8];
        load8<float, VEC>(p.w_pre + d, n, w);
#pragma unroll
        for (int j = 0; j < 8; j++) w[j] *= v[i][j] * rq;
        store8<E, VEC>((E*)p.y + m * p.sy + d, n, w);
    }
}

// Backward.  Blocks walk rows grid-stride and keep their share of the three parameters' sums in registers; at the end
// a block writes one row of `part`.
template <typename E, int TPR, int VPT, bool VEC, bool DROP>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void block_norm_bwd_kernel(BlockDev p) {
    constexpr int TH = TPR < 256 ? 256 : TPR, ROWS = TH / TPR;
    __shared__ float buf[16];
    __shared__ float acc[ROWS > 1 ? TPR * VPT * 24 : 1];
    const int tid = threadIdx.x % TPR, rw = threadIdx.x / TPR;
    float sum[3][VPT][8];
#pragma unroll
    for (int q = 0; q < 3; q++)
#pragma unroll
        for (int i = 0; i < VPT; i++)
#pragma unroll
            for (int j = 0; j < 8; j++) sum[q][i][j] = 0.f;
    Rng rng = {};
    if (DROP) rng = load_rng(p.rng);
    for (int64_t m = (int64_t)blockIdx.x * ROWS + rw; m < p.M; m += (int64_t)gridDim.x * ROWS) {
        float t[VPT][8], hh[VPT][8];
        float dot = 0.f;
        const float rq = p.w_pre ? p.rstd_pre_in[m] : 0.f;
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int64_t d = (int64_t)(i * TPR + tid) * 8;
            const int n = (int)min((int64_t)8, p.D - d);
#pragma unroll
            for (int j = 0; j < 8; j++) t[i][j] = hh[i][j] = 0.f;
            if (n > 0 && p.w_pre) {
                float w[8];
                load8<E, VEC>((const E*)p.h_in + m * p.sh + d, n, hh[i]);
                load8<E, VEC>((const E*)p.dy + m * p.sdy + d, n, t[i]);
                load8<float, VEC>(p.w_pre + d, n, w);
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    hh[i][j] *= rq;
                    sum[2][i][j] = fmaf(t[i][j], hh[i][j], sum[2][i][j]);
                    t[i][j] *= w[j];
                    dot = fmaf(t[i][j], hh[i][j], dot);
                }
            }
        }
        if (p.w_pre) dot = row_sum<TPR>(dot, buf) * p.inv_d;
        // t: dresidual, then dn; hh: xh
        const float rp = p.w_post ? p.rstd_post_in[m] : 1.f;
        float dot2 = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int64_t d = (int64_t)(i * TPR + tid) * 8;
            const int n = (int)min((int64_t)8, p.D - d);
            if (n <= 0) continue;
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; j++) t[i][j] = rq * fmaf(-hh[i][j], dot, t[i][j]);
            if (p.dh) {
                load8<E, VEC>((const E*)p.dh + m * p.sdh + d, n, f);
#pragma unroll
                for (int j = 0; j < 8; j++) t[i][j] += f[j];
            }
            if (p.dres) store8<E, VEC>((E*)p.dres + m * p.sdres + d, n, t[i]);
            load8<E, VEC>((const E*)p.x + m * p.sx + d, n, hh[i]);
            uint32_t k = 0xff;
            if (DROP) {
                k = keep_bits(rng, m * p.chunks + (i * TPR + tid), p.drop);
#pragma unroll
                for (int j = 0; j < 8; j++) t[i][j] *= p.keep_scale;
            }
            float wp[8], sc[8], g[8], o[8];
#pragma unroll
            for (int j = 0; j < 8; j++) wp[j] = sc[j] = g[j] = 1.f;
            if (p.w_post) load8<float, VEC>(p.w_post + d, n, wp);
            if (p.scale) load8<float, VEC>(p.scale + d, n, sc);
            if (p.gate) load8<E, VEC>((const E*)p.gate + m * p.sg + d, n, g);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const bool kept = (k >> j) & 1;
                float a = 1.f, da = 1.f;
                if (p.gate) act_slope(g[j], p.act, &a, &da);
                hh[i][j] *= rp;
                const float du = t[i][j], un = du * hh[i][j] * wp[j], us = du * a * sc[j];
                o[j] = kept ? un * sc[j] * da : 0.f;
                sum[1][i][j] += kept ? un * a : 0.f;
                sum[0][i][j] += kept ? us * hh[i][j] : 0.f;
                t[i][j] = kept ? us * wp[j] : 0.f;
                dot2 = fmaf(t[i][j], hh[i][j], dot2);
            }
            if (p.dgate) store8<E, VEC>((E*)p.dgate + m * p.sdg + d, n, o);
        }
        dot2 = p.w_post ? row_sum<TPR>(dot2, buf) * p.inv_d : 0.f;
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int64_t d = (int64_t)(i * TPR + tid) * 8;
            const int n = (int)min((int64_t)8, p.D - d);
            if (n <= 0) continue;
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; j++) o[j] = p.w_post ? rp * fmaf(-hh[i][j], dot2, t[i][j]) : t[i][j];
            store8<E, VEC>((E*)p.dx + m * p.sdx + d, n, o);
        }
    }
    if (ROWS > 1) {
        for (int r = 0; r < ROWS; r++) {
            if (rw == r)
#pragma unroll
                for (int q = 0; q < 3; q++)
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
    for (int q = 0; q < 3; q++)
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int64_t d = (int64_t)(i * TPR + tid) * 8;
            const int n = (int)min((int64_t)8, p.D - d);
            if (n > 0) store8<float, VEC>(p.part + ((int64_t)blockIdx.x * 3 + q) * p.D + d, n, sum[q][i]);
        }
}

// The parameters' derivatives, blockIdx.y which: sums over the blocks' rows, 16 channels per block, 16 threads each.
__global__ __launch_bounds__(256) void block_norm_sums_kernel(const float* __restrict__ part, float* __restrict__ dw_post,
                                                              float* __restrict__ dscale, float* __restrict__ dw_pre,
                                                              int64_t D, int64_t rows) {
    float* out = blockIdx.y == 0 ? dw_post : blockIdx.y == 1 ? dscale : dw_pre;
    if (!out) return;
    __shared__ float sum[16][16];
    const int dl = threadIdx.x & 15, share = threadIdx.x >> 4;
    const int64_t d = (int64_t)blockIdx.x * 16 + dl;
    float s = 0.f;
    if (d < D)
#pragma unroll 4
        for (int64_t r = share; r < rows; r += 16) s += part[(r * 3 + blockIdx.y) * D + d];
    sum[share][dl] = s;
    __syncthreads();
    if (share != 0 || d >= D) return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i++) s += sum[i][dl];
    out[d] = s;
}

// y = residual + drop(x): a thread per chunk of 8, chunks of all rows in one line.
template <typename E, bool VEC, bool DROP>
__global__ __launch_bounds__(256) void dropout_kernel(BlockDev p) {
    Rng rng = {};
    if (DROP) rng = load_rng(p.rng);
    const int64_t total = p.M * p.chunks;
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < total; q += (int64_t)gridDim.x * 256) {
        const int64_t m = q / p.chunks, d = (q - m * p.chunks) * 8;
        const int n = (int)min((int64_t)8, p.D - d);
        float v[8], f[8];
        load8<E, VEC, true>((const E*)p.x + m * p.sx + d, n, v);
        if (DROP) {
            const uint32_t k = keep_bits(rng, q, p.drop);
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = (k >> j) & 1 ? v[j] * p.keep_scale : 0.f;
        }
        if (p.residual) {
            load8<E, VEC, true>((const E*)p.residual + m * p.sres + d, n, f);
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] += f[j];
        }
        store8<E, VEC>((E*)p.y + m * p.sy + d, n, v);
    }
}

constexpr int BWD_BLOCKS = 512;
int64_t bwd_rows(int64_t M) { return std::min<int64_t>(BWD_BLOCKS, M); }

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
    constexpr int TH = TPR < 256 ? 256 : TPR, ROWS = TH / TPR;
    const int64_t blocks = std::min<int64_t>(bwd_rows(a.M), (a.M + ROWS - 1) / ROWS);
    if (blocks > 0)
        LA_TRACED(a.tr, "block_norm_bwd",
                  block_norm_bwd_kernel<E, TPR, VPT, VEC, DROP><<<(unsigned)blocks, TH, 0, a.stream>>>(p));
    if (a.dw_post || a.dscale || a.dw_pre)
        LA_TRACED(a.tr, "block_norm_bwd_sums", block_norm_sums_kernel<<<dim3((unsigned)((a.D + 15) / 16), 3), 256, 0, a.stream>>>(
                                                 p.part, a.dw_post, a.dscale, a.dw_pre, a.D, blocks));
}

template <typename E, bool VEC, bool DROP>
hipError_t run_v(const BlockArgs& a, const BlockDev& p, bool bwd) {
    const int64_t ch = (a.D + 7) / 8;
    if (!bwd) {
        if (ch <= 64) fwd_k<E, 64, 1, VEC, DROP>(a, p);
        else if (ch <= 128) fwd_k<E, 64, 2, VEC, DROP>(a, p);
        else if (ch <= 256) fwd_k<E, 64, 4, VEC, DROP>(a, p);
        else if (ch <= 512) fwd_k<E, 256, 2, VEC, DROP>(a, p);
        else if (ch <= 1024) fwd_k<E, 256, 4, VEC, DROP>(a, p);
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

size_t block_norm_bwd_ws(int64_t M, int64_t D) { return (size_t)(bwd_rows(M) * 3 * D) * sizeof(float); }

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
