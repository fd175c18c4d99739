// ssm_scan.hip -- the selective scan forward, and its single-token form.
//
//   S_t[n,d] = exp(delta_t[d] A[d,n]) S_{t-1}[n,d] + delta_t[d] u_t[d] B_t[n],   y_t[d] = sum_n C_t[n] S_t[n,d]
//
// The decay differs per (n, d) and per token, so no factorisation turns the pair weights into a
// matrix product; the work is, per (t, n, d): a product and an exponential for the decay, a product
// and a fused multiply-add for the state, one more for the output.  That bounds the operator by
// vector issue, not by memory (N = 16: 16 exponentials against 8 bytes moved per (t, d)).
//
// Layout.  A lane owns one channel and keeps its N states and its N rates A log2(e) in registers.
// B_t and C_t are the same for every channel, so they are read through the scalar cache and enter the
// arithmetic as scalar operands; a first launch packs them as fp32 [B, L, 2 NP] (NP = N rounded up
// to a size with a kernel, zeros behind N), which takes any stride, type and alignment out of the inner loop.
//
// Split.  A sequence gives only D / 64 waves, the device wants a few per SIMD.  Sequences are
// cut into G segments: a first pass runs segments 0..G-2 from zero and keeps their end states and sums
// of delta (a segment's total decay is exp(A sum delta)), a scan over the segments turns them into
// every segment's incoming state, and the second pass runs all segments from those.  The first
// pass costs (G - 1) / G of one more recurrence without the output sum.
#include "la_mixer.h"
#include "ssm_common.h"

namespace la {
namespace {

constexpr int TB = 8;  // tokens per block of loads

struct FwdDev {
    const void* u;
    const void* dt;
    const void* z;
    const float* A;
    const float* Dskip;
    const float* dt_bias;
    const float* bc;     // [B, L, 2 NP]
    const float* hin;    // [B, G, N, D] states entering the segments; null: zero (G = 1)
    const int32_t* lengths;
    void* y;
    float* s_out;
    float* part;  // state pass: hin, written at g + 1
    float* sumdt; // state pass: [B, G, D]
    int64_t L, D, seglen;
    int N, G;
    unsigned cb, ng;  // channel blocks; segments this launch runs
    bool softplus;
    la_rows su, sdt, sz, sy;
};

template <typename T>
__global__ __launch_bounds__(256) void pack_bc_kernel(const T* __restrict__ Bm, const T* __restrict__ Cm, la_rows sb,
                                                      la_rows sc, float* __restrict__ bc, int64_t rows, int64_t L, int N,
                                                      int NP) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t r = i / (2 * NP);
    if (r >= rows) return;
    const int j = (int)(i % (2 * NP));
    const int64_t b = r / L, t = r % L;
    float v = 0.f;
    if (j < NP) {
        if (j < N) v = io<T>::ld(Bm + b * sb.batch + t * sb.token + j);
    } else if (j - NP < N) {
        v = io<T>::ld(Cm + b * sc.batch + t * sc.token + (j - NP));
    }
    bc[i] = v;
}

template <typename T, int NP, bool STATE>
__global__ __launch_bounds__(64) void ssm_fwd_kernel(FwdDev p) {
    // blocks: channel block fastest, then segment, then sequence
    const unsigned r = blockIdx.x / p.cb;
    const int g = (int)(r % p.ng);
    const int64_t b = r / p.ng;
    const int64_t d0 = (int64_t)(blockIdx.x % p.cb) * 64;
    const bool live = d0 + threadIdx.x < p.D;
    const int lane = live ? threadIdx.x : 0;  // idle lanes repeat the block's first channel and write nothing
    const int64_t d = d0 + lane;

    float h[NP], A2[NP];
#pragma unroll
    for (int n = 0; n < NP; n++) {
        A2[n] = n < p.N ? p.A[d * p.N + n] * LOG2E : 0.f;
        h[n] = !STATE && p.hin && n < p.N ? p.hin[((b * p.G + g) * p.N + n) * p.D + d] : 0.f;
    }
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.f;
    const float skip = !STATE && p.Dskip ? p.Dskip[d] : 0.f;
    const int64_t len = seq_len(p.lengths, b, p.L);
    const int64_t t0 = g * p.seglen, t1 = min(t0 + p.seglen, len);
    const bool gate = !STATE && p.z;

    const T* ub = (const T*)p.u + b * p.su.batch + d0;
    const T* xb = (const T*)p.dt + b * p.sdt.batch + d0;
    const T* zb = gate ? (const T*)p.z + b * p.sz.batch + d0 : nullptr;
    T* yb = STATE ? nullptr : (T*)p.y + b * p.sy.batch + d0;
    scalar_f32 bcb = as_scalar(p.bc + b * p.L * (2 * NP));

    T un[TB], xn[TB], zn[TB];
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int j = 0; j < TB; j++) {
            const int64_t tt = min(t + j, t1 - 1);
            un[j] = ub[tt * p.su.token + lane];
            xn[j] = xb[tt * p.sdt.token + lane];
            if (gate) zn[j] = zb[tt * p.sz.token + lane];
        }
    };
    float sum = 0.f;
    if (t0 < t1) fetch(t0);
    for (int64_t t = t0; t < t1; t += TB) {
        float dl[TB], du[TB], uu[TB], zz[TB];
#pragma unroll
        for (int j = 0; j < TB; j++) {
            const float x = (float)xn[j] + bias;
            dl[j] = p.softplus ? softplus<false>(x, nullptr) : x;
            uu[j] = (float)un[j];
            du[j] = dl[j] * uu[j];
            if (gate) zz[j] = (float)zn[j];
        }
        if (t + TB < t1) fetch(t + TB);
        const int nt = (int)min((int64_t)TB, t1 - t);
#pragma unroll
        for (int j = 0; j < TB; j++) {
            if (j < nt) {
                scalar_f32 row = bcb + (t + j) * (2 * NP);
                float acc[2] = {skip * uu[j], 0.f};
#pragma unroll
                for (int n = 0; n < NP; n++) {
                    const float a = __builtin_amdgcn_exp2f(dl[j] * A2[n]);
                    h[n] = fmaf(a, h[n], du[j] * row[n]);
                    if (!STATE) acc[n & 1] = fmaf(row[NP + n], h[n], acc[n & 1]);
                }
                if (STATE) {
                    sum += dl[j];
                } else {
                    float v = acc[0] + acc[1];
                    if (gate) v *= zz[j] * sigmoid(zz[j]);
                    if (live) io<T>::st(yb + (t + j) * p.sy.token + lane, v);
                }
            }
        }
    }
    if (!live) return;
    if (STATE) {
#pragma unroll
        for (int n = 0; n < NP; n++)
            if (n < p.N) p.part[((b * p.G + g + 1) * p.N + n) * p.D + d] = h[n];
        p.sumdt[(b * p.G + g) * p.D + d] = sum;
    } else if (p.s_out && g == p.G - 1) {
#pragma unroll
        for (int n = 0; n < NP; n++)
            if (n < p.N) p.s_out[(b * p.N + n) * p.D + d] = h[n];
    }
}

// States entering the segments from the segments' own end states: slot 0 takes s_in, slot g + 1
// (holding segment g's end state from zero) adds the decayed state that entered segment g.  A thread
// owns one (b, n, d); its loads are issued PB segments ahead of the chain.
constexpr int PB = 8;
__global__ __launch_bounds__(256) void ssm_segments_kernel(const float* __restrict__ A, const float* __restrict__ s_in,
                                                           const float* __restrict__ sumdt, float* __restrict__ part,
                                                           int64_t total, int64_t D, int N, int G) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const int64_t d = i % D, n = i / D % N, b = i / (D * N);
    const float a2 = A[d * N + n] * LOG2E;
    float h = s_in ? s_in[i] : 0.f;
    float* pp = part + (b * G * N + n) * D + d;
    const float* sp = sumdt + b * G * D + d;
    const int64_t ps = (int64_t)N * D;
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
                h = fmaf(__builtin_amdgcn_exp2f(a2 * s[j]), h, v[j]);
                pp[(g0 + j) * ps] = h;
            }
    }
}

int np_for(int N) { return N <= 8 ? 8 : N <= 16 ? 16 : N <= 24 ? 24 : N <= 32 ? 32 : N <= 48 ? 48 : 64; }

// Segments: about 2048 waves, none under 64 tokens.
SsmPlan fwd_plan(int64_t B, int64_t L, int64_t D) { return ssm_plan(B, L, D, 2048, 64, TB); }

struct FwdWs {
    float *bc, *part, *sumdt;
    size_t bytes;
};
FwdWs fwd_cut(void* base, int64_t B, int64_t L, int64_t D, int N, int G) {
    WsCut c{(char*)base};
    FwdWs w;
    w.bc = c.take((size_t)(B * L) * 2 * np_for(N));
    w.part = G > 1 ? c.take((size_t)(B * G) * N * D) : nullptr;
    w.sumdt = G > 1 ? c.take((size_t)(B * G) * D) : nullptr;
    w.bytes = c.used;
    return w;
}

template <typename T, int NP>
void launch_np(const SsmArgs& a, FwdDev p, const SsmPlan& pl) {
    p.cb = (unsigned)((a.D + 63) / 64);
    if (pl.G > 1) {
        p.ng = pl.G - 1;
        LA_TRACED(a.tr, "ssm_state", ssm_fwd_kernel<T, NP, true><<<p.cb * p.ng * (unsigned)a.B, 64, 0, a.stream>>>(p));
        const int64_t total = a.B * a.N * a.D;
        LA_TRACED(a.tr, "ssm_segments", ssm_segments_kernel<<<(unsigned)((total + 255) / 256), 256, 0, a.stream>>>(
                                            a.A, a.s_in, p.sumdt, p.part, total, a.D, a.N, pl.G));
    }
    p.ng = pl.G;
    LA_TRACED(a.tr, "ssm_out", ssm_fwd_kernel<T, NP, false><<<p.cb * p.ng * (unsigned)a.B, 64, 0, a.stream>>>(p));
}

template <typename T>
hipError_t launch_t(const SsmArgs& a) {
    const SsmPlan pl = fwd_plan(a.B, a.L, a.D);
    const FwdWs w = fwd_cut(a.ws, a.B, a.L, a.D, a.N, pl.G);
    const int NP = np_for(a.N);
    FwdDev p;
    p.u = a.u; p.dt = a.dt; p.z = a.z; p.A = a.A; p.Dskip = a.Dskip; p.dt_bias = a.dt_bias;
    p.bc = w.bc;
    p.hin = pl.G > 1 ? w.part : a.s_in;
    p.lengths = a.lengths; p.y = a.y; p.s_out = a.s_out;
    p.part = w.part; p.sumdt = w.sumdt;
    p.L = a.L; p.D = a.D; p.seglen = pl.seglen; p.N = a.N; p.G = pl.G;
    p.softplus = a.softplus;
    p.su = a.su; p.sdt = a.sdt; p.sz = a.sz; p.sy = a.sy;
    launch_pack_bc(a, w.bc, NP);
    switch (NP) {
        case 8: launch_np<T, 8>(a, p, pl); break;
        case 16: launch_np<T, 16>(a, p, pl); break;
        case 24: launch_np<T, 24>(a, p, pl); break;
        case 32: launch_np<T, 32>(a, p, pl); break;
        case 48: launch_np<T, 48>(a, p, pl); break;
        default: launch_np<T, 64>(a, p, pl); break;
    }
    return hipGetLastError();
}

// ---------------------------------------------------------------------------------------------
// One token per sequence.  A lane owns one channel of one row; it reads and writes the state of its
// slot once, 256 contiguous bytes per wave and key dim.  B and C are loaded once per wave, lane n
// holding B[n] and C[n], and broadcast by lane reads.  `first_use`: rows that name a slot an earlier
// row names are padding, so that no two rows write one state.
__device__ __forceinline__ bool earlier_row_has(const int32_t* slots, int64_t b, int32_t s) {
    bool dup = false;
    for (int64_t i = threadIdx.x & 63; i < b; i += 64) dup |= slots[i] == s;
    return __any(dup);
}

template <typename T, int NP>
__global__ __launch_bounds__(64) void ssm_step_kernel(const T* __restrict__ u, const T* __restrict__ dt,
                                                      const float* __restrict__ A, const T* __restrict__ Bm,
                                                      const T* __restrict__ Cm, const float* __restrict__ Dskip,
                                                      const T* __restrict__ z, const float* __restrict__ dt_bias,
                                                      float* __restrict__ state, const int32_t* __restrict__ slots,
                                                      T* __restrict__ y, int64_t su, int64_t sdt, int64_t sb, int64_t sc,
                                                      int64_t sz, int64_t sy, int64_t D, unsigned cb, int N, int nslots, bool sp) {
    const int64_t b = blockIdx.x / cb;
    const int64_t d0 = (int64_t)(blockIdx.x % cb) * 64;
    const bool live = d0 + threadIdx.x < D;
    const int64_t d = live ? d0 + threadIdx.x : d0;
    const int64_t slot = slots ? slots[b] : b;
    if (slot < 0 || slot >= nslots) return;
    const int n0 = threadIdx.x < N ? threadIdx.x : N - 1;
    const float bl = (float)Bm[b * sb + n0], cl = (float)Cm[b * sc + n0];
    float* st = state + slot * N * D + d;
    float h[NP], a2[NP];
#pragma unroll
    for (int n = 0; n < NP; n++) {
        h[n] = n < N ? st[(int64_t)n * D] : 0.f;
        a2[n] = n < N ? A[d * N + n] * LOG2E : 0.f;
    }
    const float uu = (float)u[b * su + d];
    const float x = (float)dt[b * sdt + d] + (dt_bias ? dt_bias[d] : 0.f);
    const float zz = z ? (float)z[b * sz + d] : 0.f;
    float acc = Dskip ? Dskip[d] * uu : 0.f;
    const float delta = sp ? softplus<false>(x, nullptr) : x;
    const float du = delta * uu;
#pragma unroll
    for (int n = 0; n < NP; n++)
        if (n < N) {
            const float bn = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(bl), n));
            const float cn = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(cl), n));
            h[n] = fmaf(__builtin_amdgcn_exp2f(delta * a2[n]), h[n], du * bn);
            acc = fmaf(cn, h[n], acc);
        }
    if (slots && earlier_row_has(slots, b, (int32_t)slot)) return;
    if (!live) return;
#pragma unroll
    for (int n = 0; n < NP; n++)
        if (n < N) st[(int64_t)n * D] = h[n];
    if (z) acc *= zz * sigmoid(zz);
    io<T>::st(y + b * sy + d, acc);
}

template <typename T, int NP>
void step_np(const SsmArgs& a) {
    const unsigned cb = (unsigned)((a.D + 63) / 64);
    LA_TRACED(a.tr, "ssm_step",
              ssm_step_kernel<T, NP><<<cb * (unsigned)a.B, 64, 0, a.stream>>>(
                  (const T*)a.u, (const T*)a.dt, a.A, (const T*)a.Bm, (const T*)a.Cm, a.Dskip, (const T*)a.z, a.dt_bias,
                  a.state, a.slots, (T*)a.y, a.su.batch, a.sdt.batch, a.sb.batch, a.sc.batch, a.sz.batch, a.sy.batch, a.D, cb,
                  a.N, a.nslots, a.softplus));
}
template <typename T>
hipError_t step_t(const SsmArgs& a) {
    switch (np_for(a.N)) {
        case 8: step_np<T, 8>(a); break;
        case 16: step_np<T, 16>(a); break;
        case 24: step_np<T, 24>(a); break;
        case 32: step_np<T, 32>(a); break;
        case 48: step_np<T, 48>(a); break;
        default: step_np<T, 64>(a); break;
    }
    return hipGetLastError();
}

template <typename T>
void pack_t(const SsmArgs& a, float* bc, int NP) {
    const int64_t n = a.B * a.L * 2 * NP;
    if (n == 0) return;
    LA_TRACED(a.tr, "ssm_pack", pack_bc_kernel<T><<<(unsigned)((n + 255) / 256), 256, 0, a.stream>>>(
                                    (const T*)a.Bm, (const T*)a.Cm, a.sb, a.sc, bc, a.B * a.L, a.L, a.N, NP));
}

}  // namespace

void launch_pack_bc(const SsmArgs& a, float* bc, int NP) { a.bf16 ? pack_t<__bf16>(a, bc, NP) : pack_t<float>(a, bc, NP); }

size_t ssm_fwd_ws(int64_t B, int64_t L, int64_t D, int N) {
    return fwd_cut(nullptr, B, L, D, N, fwd_plan(B, L, D).G).bytes;
}

hipError_t launch_ssm_scan(const SsmArgs& a) {
    if (a.B == 0 || a.D == 0) return hipSuccess;
    return a.bf16 ? launch_t<__bf16>(a) : launch_t<float>(a);
}

hipError_t launch_ssm_step(const SsmArgs& a) {
    if (a.B == 0 || a.D == 0) return hipSuccess;
    return a.bf16 ? step_t<__bf16>(a) : step_t<float>(a);
}

}  // namespace la
