// add_norm.hip -- residual addition and root-mean-square norm, its 8-bit form and its backward.
//
//   h = x + residual,   r = 1 / sqrt(mean h^2 + eps),   y = h r w
//   backward, with xh = h r:   dx = r (dy w - xh mean(dy w xh)) + dh,   dw = sum over rows of dy xh
//
// Memory-bound: every input element is read once into registers and every output written once.  A row
// belongs to TPR threads (one wave for short rows, whose reductions need no barrier; four or
// sixteen for long ones), each holding VPT chunks of 8 adjacent elements in fp32.  16384 x 2048 bf16 with the sum
// kept and 8-bit output: 236 MB in 54.3 us, 4.3 TB/s, where a large copy reaches 4.8.
#include <algorithm>

#include "la_mixer.h"
#include "row_ops.h"

namespace la {
namespace {

struct NormDev {
    const void* x;
    const void* residual;
    const float* weight;
    void* y;
    uint8_t* q;
    float* scale;
    void* h;
    float* rstd;
    const void* dy;
    const void* h_in;
    const float* rstd_in;
    const void* dh;
    void* dx;
    float* part;
    int64_t M, D;
    int group;
    float eps, inv_d;
    int64_t sx, sres, sy, sh, sdy, sdh, sdx;
};

// y / s, inv its reciprocal, cut to fp32 and marked in its last bit where it is inexact, so that a conversion to e4m3
// rounds the quotient itself: rounded to nearest in fp32 first, one next to a tie of e4m3 could land on the tie or
// across it.  y inv is off by at most 2 steps, the first residual brings it within one, the second is its side's sign.
__device__ __forceinline__ float quotient(float y, float s, float inv) {
    float q = y * inv;
    q = fmaf(fmaf(-q, s, y), inv, q);
    const float rem = fmaf(-q, s, y);
    uint32_t b = __float_as_uint(q);
    b -= __uint_as_float(__float_as_uint(rem) ^ (b & 0x80000000u)) < 0.f;  // q is past y / s: the value before it
    b |= rem != 0.f;
    return __uint_as_float(b);
}
// Below TIE_NEAR where f is within 4 steps of a tie of e4m3's normal values (mantissa bits xxx1000...).
constexpr uint32_t TIE_NEAR = 8u << 12;
__device__ __forceinline__ uint32_t tie_distance(float f) { return (__float_as_uint(f) << 12) - (0x80000000u - (4u << 12)); }

// Y8: 8-bit output.  Blocks of max(TPR, 256) threads hold 256 / TPR rows when TPR = 64, else one.
template <typename E, int TPR, int VPT, bool VEC, bool Y8>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void add_norm_kernel(NormDev p) {
    __shared__ float buf[16];
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
    const int tid = threadIdx.x % TPR;
    const int64_t m = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
    if (m >= p.M) return;  // whole waves; TPR >= 256: whole blocks
    const E* x = (const E*)p.x + m * p.sx;
    const E* res = p.residual ? (const E*)p.residual + m * p.sres : nullptr;
    float h[VPT][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int64_t d = (int64_t)(i * TPR + tid) * 8;
        const int n = (int)min((int64_t)8, p.D - d);
        if (n > 0) {
            load8<E, VEC, true>(x + d, n, h[i]);
            if (res) {
                float r[8];
                load8<E, VEC, true>(res + d, n, r);
#pragma unroll
                for (int j = 0; j < 8; j++) h[i][j] += r[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) h[i][j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; j++) ss = fmaf(h[i][j], h[i][j], ss);
    }
    const RowScale rs = row_rstd<TPR, VPT>(h, ss, p.inv_d, p.eps, buf);
    if (p.rstd && tid == 0) p.rstd[m] = rs.own();
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int64_t d = (int64_t)(i * TPR + tid) * 8;
        const int n = (int)min((int64_t)8, p.D - d);
        if (n <= 0) continue;
        if (p.h) store8<E, VEC>((E*)p.h + m * p.sh + d, n, h[i]);
        float w[8];
        load8<float, VEC>(p.weight + d, n, w);
#pragma unroll
        for (int j = 0; j < 8; j++) h[i][j] = h[i][j] * rs.s * (rs.r * w[j]);
        if (!Y8)
            store8<E, VEC>((E*)p.y + m * p.sy + d, n, h[i]);
        else
#pragma unroll
            for (int j = 0; j < 8; j++) amax = max_nan(amax, fabsf(h[i][j]));
    }
    if (!Y8) return;
    if (p.group == 0) amax = row_max<TPR>(amax, buf);
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int64_t d = (int64_t)(i * TPR + tid) * 8;
        const int n = (int)min((int64_t)8, p.D - d);
        if (p.group) {  // D is a multiple of the group, so a group's lanes all exist or none does
            amax = 0.f;
            if (n > 0)
#pragma unroll
                for (int j = 0; j < 8; j++) amax = max_nan(amax, fabsf(h[i][j]));
            if (p.group == 128) amax = lanes_max<16>(amax);
            else if (p.group == 64) amax = lanes_max<8>(amax);
            else amax = lanes_max<4>(amax);
        }
        if (n <= 0) continue;
        const float top = amax / 448.f;
        const float s = top > 0.f || top != top ? top : 1.f;  // also where the quotient underflows
        if (p.group ? d % p.group == 0 : d == 0) p.scale[p.group ? m * (p.D / p.group) + d / p.group : m] = s;
        // y / s through one reciprocal per group, exact where that could miss a tie: next to one of the normal values, or
        // in e4m3's subnormal range, below 2^-6 (2^-15 of the group's largest), where the ties lie otherwise.  16384 x 2048
        // bf16 in groups of 128: 54.3 us, exact for all 56.3, for none 53.4.  A scale so small that its reciprocal would
        // overflow, or the quotient's residual not be exact, is first moved up, with y, by a power of two; in a group
        // with an infinite scale finite values give 0.
        float su = s;
        if (s < 0x1p-60f) {
            su *= 0x1p+64f;
#pragma unroll
            for (int j = 0; j < 8; j++) h[i][j] *= 0x1p+64f;
        }
        const float inv = 1.f / su;
        float f[8];
        uint32_t near = ~0u;
        float least = INFINITY;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            f[j] = h[i][j] * inv;
            near = min(near, tie_distance(f[j]));
            least = fminf(least, fabsf(f[j]));
        }
        if ((near < TIE_NEAR || least < 0x1p-6f) && su < INFINITY)
#pragma unroll
            for (int j = 0; j < 8; j++) f[j] = quotient(h[i][j], su, inv);
        uint32_t c[2];
#pragma unroll
        for (int j = 0; j < 8; j++) f[j] = __builtin_amdgcn_fmed3f(f[j], -448.f, 448.f);  // a NaN: -448
#pragma unroll
        for (int k = 0; k < 2; k++) {
            int v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * k], f[4 * k + 1], 0, false);
            c[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * k + 2], f[4 * k + 3], v, true);
        }
        uint8_t* qp = p.q + m * p.D + d;
        if (VEC) {
            *(u32x2*)qp = u32x2{c[0], c[1]};
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++)
                if (j < n) qp[j] = (uint8_t)(c[j >> 2] >> (8 * (j & 3)));
        }
    }
}

// Backward.  Blocks walk rows grid-stride and keep their share of d_weight in registers; at the end
// the block's waves add theirs up (LDS, one after the other) and write one row of `part`.
template <typename E, int TPR, int VPT, bool VEC>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void add_norm_bwd_kernel(NormDev p) {
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
    __shared__ float buf[16];
    __shared__ float acc[ROWS > 1 ? TPR * VPT * 8 : 1];
    const int tid = threadIdx.x % TPR, rw = threadIdx.x / TPR;
    float dw[VPT][8], w[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int64_t d = (int64_t)(i * TPR + tid) * 8;
        const int n = (int)min((int64_t)8, p.D - d);
#pragma unroll
        for (int j = 0; j < 8; j++) dw[i][j] = w[i][j] = 0.f;
        if (n > 0) load8<float, VEC>(p.weight + d, n, w[i]);
    }
    for (int64_t m = (int64_t)blockIdx.x * ROWS + rw; m < p.M; m += (int64_t)gridDim.x * ROWS) {
        const float r = p.rstd_in[m];
        float xh[VPT][8], dy[VPT][8];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int64_t d = (int64_t)(i * TPR + tid) * 8;
            const int n = (int)min((int64_t)8, p.D - d);
            if (n > 0) {
                load8<E, VEC>((const E*)p.h_in + m * p.sh + d, n, xh[i]);
                load8<E, VEC>((const E*)p.dy + m * p.sdy + d, n, dy[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; j++) xh[i][j] = dy[i][j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; j++) {
                xh[i][j] *= r;
                dw[i][j] = fmaf(dy[i][j], xh[i][j], dw[i][j]);
                dy[i][j] *= w[i][j];
                dot = fmaf(dy[i][j], xh[i][j], dot);
            }
        }
        dot = row_sum<TPR>(dot, buf) * p.inv_d;
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int64_t d = (int64_t)(i * TPR + tid) * 8;
            const int n = (int)min((int64_t)8, p.D - d);
            if (n <= 0) continue;
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; j++) o[j] = r * fmaf(-xh[i][j], dot, dy[i][j]);
            if (p.dh) {
                float g[8];
                load8<E, VEC>((const E*)p.dh + m * p.sdh + d, n, g);
#pragma unroll
                for (int j = 0; j < 8; j++) o[j] += g[j];
            }
            store8<E, VEC>((E*)p.dx + m * p.sdx + d, n, o);
        }
    }
    if (ROWS > 1) {
        for (int k = 0; k < ROWS; k++) {
            if (rw == k)
#pragma unroll
                for (int i = 0; i < VPT; i++)
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        float* a = acc + (i * 8 + j) * TPR + tid;
                        if (k > 0) dw[i][j] += *a;
                        if (k < ROWS - 1) *a = dw[i][j];
                    }
            __syncthreads();
        }
        if (rw != ROWS - 1) return;
    }
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int64_t d = (int64_t)(i * TPR + tid) * 8;
        const int n = (int)min((int64_t)8, p.D - d);
        if (n > 0) store8<float, VEC>(p.part + blockIdx.x * p.D + d, n, dw[i]);
    }
}

// d_weight[d] = sum over the blocks' rows: 16 channels per block, 16 threads each.
__global__ __launch_bounds__(256) void add_norm_bwd_sums_kernel(const float* __restrict__ part, float* __restrict__ dw,
                                                                int64_t D, int64_t rows) {
    __shared__ float sum[16][16];
    const int dl = threadIdx.x & 15, share = threadIdx.x >> 4;
    const int64_t d = (int64_t)blockIdx.x * 16 + dl;
    float s = 0.f;
    if (d < D)
#pragma unroll 4
        for (int64_t r = share; r < rows; r += 16) s += part[r * D + d];
    sum[share][dl] = s;
    __syncthreads();
    if (share != 0 || d >= D) return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i++) s += sum[i][dl];
    dw[d] = s;
}

constexpr int BWD_BLOCKS = 512;
int64_t bwd_rows(int64_t M) { return std::min<int64_t>(BWD_BLOCKS, M); }  // blocks, so rows of partial sums

template <typename E, int TPR, int VPT, bool VEC>
void fwd_k(const NormArgs& a, const NormDev& p) {
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1, TH = TPR < 256 ? 256 : TPR;
    const unsigned blocks = (unsigned)((a.M + ROWS - 1) / ROWS);
    if (a.q)
        LA_TRACED(a.tr, "add_norm_q8", add_norm_kernel<E, TPR, VPT, VEC, true><<<blocks, TH, 0, a.stream>>>(p));
    else
        LA_TRACED(a.tr, "add_norm", add_norm_kernel<E, TPR, VPT, VEC, false><<<blocks, TH, 0, a.stream>>>(p));
}
template <typename E, int TPR, int VPT, bool VEC>
void bwd_k(const NormArgs& a, const NormDev& p) {
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1, TH = TPR < 256 ? 256 : TPR;
    const int64_t blocks = std::min<int64_t>(bwd_rows(a.M), (a.M + ROWS - 1) / ROWS);
    if (blocks > 0)
        LA_TRACED(a.tr, "add_norm_bwd", add_norm_bwd_kernel<E, TPR, VPT, VEC><<<(unsigned)blocks, TH, 0, a.stream>>>(p));
    LA_TRACED(a.tr, "add_norm_bwd_sums", add_norm_bwd_sums_kernel<<<(unsigned)((a.D + 15) / 16), 256, 0, a.stream>>>(
                                             p.part, a.d_weight, a.D, blocks));
}

// Threads per row by the row's chunks of 8: a wave up to 4 chunks a lane (D <= 2048), four waves to
// 8192, sixteen to the limit of 16384 (beyond it the backward's registers would not hold a row).
template <typename E, bool VEC>
hipError_t run_v(const NormArgs& a, const NormDev& p, bool bwd) {
    const int64_t ch = (a.D + 7) / 8;
#define LA_NORM_CASE(T_, V_) (bwd ? bwd_k<E, T_, V_, VEC>(a, p) : fwd_k<E, T_, V_, VEC>(a, p))
    if (ch <= 64) LA_NORM_CASE(64, 1);
    else if (ch <= 128) LA_NORM_CASE(64, 2);
    else if (ch <= 256) LA_NORM_CASE(64, 4);
    else if (ch <= 512) LA_NORM_CASE(256, 2);
    else if (ch <= 1024) LA_NORM_CASE(256, 4);
    else LA_NORM_CASE(1024, 2);
#undef LA_NORM_CASE
    return hipGetLastError();
}
template <typename E>
hipError_t run(const NormArgs& a, bool bwd) {
    NormDev p = {};
    p.x = a.x; p.residual = a.residual; p.weight = a.weight; p.y = a.y; p.q = a.q; p.scale = a.scale; p.h = a.h;
    p.rstd = a.rstd; p.dy = a.dy; p.h_in = a.h_in; p.rstd_in = a.rstd_in; p.dh = a.dh; p.dx = a.dx;
    p.part = (float*)a.ws;
    p.M = a.M; p.D = a.D; p.group = a.group; p.eps = a.eps; p.inv_d = 1.f / (float)a.D;
    p.sx = a.sx; p.sres = a.sres; p.sy = a.sy; p.sh = a.sh; p.sdy = a.sdy; p.sdh = a.sdh; p.sdx = a.sdx;
    const size_t es = sizeof(E);
    const bool vec = a.D % 8 == 0 && row16(a.x, a.sx, es) && row16(a.residual, a.sres, es) && row16(a.y, a.sy, es) &&
                     row16(a.h, a.sh, es) && row16(a.h_in, a.sh, es) && row16(a.dy, a.sdy, es) &&
                     row16(a.dh, a.sdh, es) && row16(a.dx, a.sdx, es) && (uintptr_t)a.weight % 16 == 0 &&
                     (uintptr_t)a.q % 8 == 0;
    return vec ? run_v<E, true>(a, p, bwd) : run_v<E, false>(a, p, bwd);
}

}  // namespace

size_t add_norm_bwd_ws(int64_t M, int64_t D) { return (size_t)(bwd_rows(M) * D) * sizeof(float); }

hipError_t launch_add_norm(const NormArgs& a) {
    if (a.M == 0) return hipSuccess;
    return a.bf16 ? run<__bf16>(a, false) : run<float>(a, false);
}
hipError_t launch_add_norm_bwd(const NormArgs& a) { return a.bf16 ? run<__bf16>(a, true) : run<float>(a, true); }

}  // namespace la
