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
    float* part;  // [rows, 3, D]
    float* state;
    const int32_t* slots;
    int64_t L, D, tiles;
    unsigned cb;
    int nslots;
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
__device__ __forceinline__ Gates gates(float r, float i, const Channel& c) {
    Gates g;
    g.rho = rcp(1.f + __builtin_amdgcn_exp2f(fmaf(r, -LOG2E, c.nr)));
    g.iota = rcp(1.f + __builtin_amdgcn_exp2f(fmaf(i, -LOG2E, c.ni)));
    g.v = c.rate * g.rho;
    g.a = __builtin_amdgcn_exp2f(g.v * -LOG2E);
    const float v2 = g.v * g.v;
    const float sh = fmaf(v2, fmaf(v2, fmaf(v2, 1.f / 5040.f, 1.f / 120.f), 1.f / 6.f), 1.f);
    const float direct = fmaf(-g.a, g.a, 1.f);
    const bool small = g.v <= 0.5f;
    g.s = small ? sh : direct;
    g.mi = __builtin_amdgcn_sqrtf(small ? 2.f * g.a * g.v * sh : direct) * g.iota;
    return g;
}
// k = a^2 v / (1 - a^2)
__device__ __forceinline__ float input_slope(const Gates& g) {
    return g.v <= 0.5f ? g.a * rcp(2.f * g.s) : g.a * g.a * g.v * rcp(g.s);
}

// A thread per (sequence, channel).
template <typename E>
__global__ __launch_bounds__(64) void gated_fwd_kernel(GatedDev p) {
    const int64_t d = (int64_t)(blockIdx.x % p.cb) * 64 + threadIdx.x, b = blockIdx.x / p.cb;
    if (d >= p.D) return;
    const int64_t len = seq_len(p.lengths, b, p.L);
    const Channel c = channel(p, d);
    float h = p.h_in ? p.h_in[b * p.D + d] : 0.f;
    for (int64_t t = 0; t < len; t++) {
        if (p.blocks && t % TILE == 0) p.blocks[(b * p.tiles + t / TILE) * p.D + d] = h;
        const Gates g = gates((float)((const E*)p.r)[b * p.sr.batch + t * p.sr.token + d],
                              (float)((const E*)p.i)[b * p.si.batch + t * p.si.token + d], c);
        h = fmaf(g.a, h, g.mi * (float)((const E*)p.x)[b * p.sx.batch + t * p.sx.token + d]);
        if (p.y) {
            float o = h;
            if (p.z) {
                const float z = (float)((const E*)p.z)[b * p.sz.batch + t * p.sz.token + d];
                o *= z * sigmoid(z);
            }
            io<E>::st((E*)p.y + b * p.sy.batch + t * p.sy.token + d, o);
        }
    }
    if (p.h_out) p.h_out[b * p.D + d] = h;
}

// A thread per (sequence, channel): a block of tokens at a time from the last, its states made again into LDS.
template <typename E>
__global__ __launch_bounds__(64) void gated_bwd_kernel(GatedDev p) {
    __shared__ float before[TILE][64];
    const int64_t d = (int64_t)(blockIdx.x % p.cb) * 64 + threadIdx.x, b = blockIdx.x / p.cb;
    if (d >= p.D) return;
    const int64_t len = seq_len(p.lengths, b, p.L);
    const Channel c = channel(p, d);
    float carry = p.dh_out ? p.dh_out[b * p.D + d] : 0.f;
    float sq = 0.f, sr = 0.f, si = 0.f;
    for (int64_t t = len; t < p.L; t++) {
        io<E>::st((E*)p.dx + b * p.sdx.batch + t * p.sdx.token + d, 0.f);
        io<E>::st((E*)p.dr + b * p.sdr.batch + t * p.sdr.token + d, 0.f);
        io<E>::st((E*)p.di + b * p.sdi.batch + t * p.sdi.token + d, 0.f);
        if (p.z) io<E>::st((E*)p.dz + b * p.sdz.batch + t * p.sdz.token + d, 0.f);
    }
    auto at = [&](const void* q, const la_rows& s, int64_t t) { return (float)((const E*)q)[b * s.batch + t * s.token + d]; };
    for (int64_t t0 = (len - 1) / TILE * TILE; len > 0 && t0 >= 0; t0 -= TILE) {
        float h = t0 > 0 ? p.blocks_in[(b * p.tiles + t0 / TILE) * p.D + d] : p.h_in ? p.h_in[b * p.D + d] : 0.f;
        const int n = (int)min((int64_t)TILE, len - t0);
        for (int j = 0; j < n; j++) {
            before[j][threadIdx.x] = h;
            const Gates g = gates(at(p.r, p.sr, t0 + j), at(p.i, p.si, t0 + j), c);
            h = fmaf(g.a, h, g.mi * at(p.x, p.sx, t0 + j));
        }
        for (int j = n - 1; j >= 0; j--) {
            const int64_t t = t0 + j;
            const Gates g = gates(at(p.r, p.sr, t), at(p.i, p.si, t), c);
            const float bb = g.mi * at(p.x, p.sx, t), hp = before[j][threadIdx.x];
            float s = at(p.dy, p.sdy, t);
            if (p.z) {
                const float z = at(p.z, p.sz, t), sg = sigmoid(z);
                io<E>::st((E*)p.dz + b * p.sdz.batch + t * p.sdz.token + d,
                          s * fmaf(g.a, hp, bb) * sg * fmaf(z, 1.f - sg, 1.f));
                s *= z * sg;
            }
            const float gt = s + carry;
            carry = g.a * gt;
            const float q = gt * fmaf(input_slope(g), bb, -g.v * g.a * hp);
            const float dr = q * (1.f - g.rho), di = gt * bb * (1.f - g.iota);
            sq += q;
            sr += dr;
            si += di;
            io<E>::st((E*)p.dx + b * p.sdx.batch + t * p.sdx.token + d, gt * g.mi);
            io<E>::st((E*)p.dr + b * p.sdr.batch + t * p.sdr.token + d, dr);
            io<E>::st((E*)p.di + b * p.sdi.batch + t * p.sdi.token + d, di);
        }
    }
    if (p.dh_in) p.dh_in[b * p.D + d] = carry;
    p.part[(b * 3 + 0) * p.D + d] = sq;
    p.part[(b * 3 + 1) * p.D + d] = sr;
    p.part[(b * 3 + 2) * p.D + d] = si;
}

// The parameters' derivatives: sums over the rows of partial sums, 16 channels per block, 16 threads each.
__global__ __launch_bounds__(256) void gated_bwd_sums_kernel(const float* __restrict__ part, const float* __restrict__ lam,
                                                             float* __restrict__ dlam, float* __restrict__ dr_bias,
                                                             float* __restrict__ di_bias, int64_t D, int64_t rows) {
    __shared__ float sum[3][16][16];
    const int dl = threadIdx.x & 15, share = threadIdx.x >> 4;
    const int64_t d = (int64_t)blockIdx.x * 16 + dl;
    float s[3] = {0.f, 0.f, 0.f};
    if (d < D)
        for (int64_t k = share; k < rows; k += 16)
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
    }
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

struct BwdCut {
    float* blocks;
    float* part;
    size_t bytes;
};
BwdCut bwd_cut(void* ws, int64_t B, int64_t L, int64_t D, bool have_blocks) {
    WsCut w{(char*)ws};
    BwdCut c;
    c.blocks = !have_blocks && tile_count(L) > 1 ? w.take((size_t)(B * tile_count(L) * D)) : nullptr;
    c.part = w.take((size_t)(B * 3 * D));
    c.bytes = w.used;
    return c;
}

GatedDev dev(const GatedArgs& a) {
    GatedDev p = {};
    p.x = a.x; p.r = a.r; p.i = a.i; p.lam = a.lam; p.r_bias = a.r_bias; p.i_bias = a.i_bias; p.z = a.z; p.h_in = a.h_in;
    p.lengths = a.lengths; p.y = a.y; p.h_out = a.h_out; p.blocks = a.blocks; p.blocks_in = a.blocks_in; p.dy = a.dy;
    p.dh_out = a.dh_out; p.dx = a.dx; p.dr = a.dr; p.di = a.di; p.dz = a.dz; p.dh_in = a.dh_in; p.state = a.state;
    p.slots = a.slots; p.nslots = a.nslots; p.c = a.c; p.L = a.L; p.D = a.D; p.tiles = tile_count(a.L);
    p.cb = (unsigned)((a.D + 63) / 64);
    p.sx = a.sx; p.sr = a.sr; p.si = a.si; p.sz = a.sz; p.sy = a.sy; p.sdy = a.sdy; p.sdx = a.sdx; p.sdr = a.sdr;
    p.sdi = a.sdi; p.sdz = a.sdz;
    return p;
}

template <typename E>
void fwd_t(const GatedArgs& a, const GatedDev& p) {
    LA_TRACED(a.tr, "gated_scan", gated_fwd_kernel<E><<<(unsigned)(a.B * p.cb), 64, 0, a.stream>>>(p));
}
template <typename E>
hipError_t bwd_t(const GatedArgs& a) {
    GatedDev p = dev(a);
    const BwdCut c = bwd_cut(a.ws, a.B, a.L, a.D, a.blocks_in != nullptr);
    p.part = c.part;
    if (c.blocks) {
        GatedDev f = p;
        f.y = nullptr; f.h_out = nullptr; f.blocks = c.blocks;
        fwd_t<E>(a, f);
        p.blocks_in = c.blocks;
    }
    if (a.B > 0) LA_TRACED(a.tr, "gated_bwd", gated_bwd_kernel<E><<<(unsigned)(a.B * p.cb), 64, 0, a.stream>>>(p));
    LA_TRACED(a.tr, "gated_bwd_sums", gated_bwd_sums_kernel<<<(unsigned)((a.D + 15) / 16), 256, 0, a.stream>>>(
                                          c.part, a.lam, a.dlam, a.dr_bias, a.di_bias, a.D, a.B));
    return hipGetLastError();
}

}  // namespace

size_t gated_fwd_ws(int64_t, int64_t, int64_t) { return 0; }
size_t gated_bwd_ws(int64_t B, int64_t L, int64_t D, bool have_blocks) { return bwd_cut(nullptr, B, L, D, have_blocks).bytes; }

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
    const GatedDev p = dev(a);
    const unsigned blocks = (unsigned)(a.B * p.cb);
    if (a.bf16)
        LA_TRACED(a.tr, "gated_step", gated_step_kernel<__bf16><<<blocks, 64, 0, a.stream>>>(p));
    else
        LA_TRACED(a.tr, "gated_step", gated_step_kernel<float><<<blocks, 64, 0, a.stream>>>(p));
    return hipGetLastError();
}

}  // namespace la
