// ssm_scan.hip -- the selective scan forward, and its single-token form.
//
//   S_t[n,d] = exp(delta_t[d] A[d,n]) S_{t-1}[n,d] + delta_t[d] u_t[d] B_t[n],   y_t[d] = sum_n C_t[n] S_t[n,d]
//
// The decay differs per (n, d) and per token, so no factorisation turns the pair weights into a
// matrix product; the work is, per (t, n, d): a product and an exponential for the decay, a product
// and a fused multiply-add for the state, one more for the output, and per (t, d) a softplus and a gate.  That
// bounds the operator by vector issue, not by memory: a wave's exponential takes 8 cycles, its product or
// multiply-add 4, and both passes below keep the vector units busy 78 % of the time.
//
// Layout.  A lane owns one channel and keeps its N states and its N rates A log2(e) in registers.  Activations
// come and go through LDS (ssm_tile.h).  B_t and C_t are the same for every channel; a first launch packs them
// as fp32 [B, L, 2 NP] (NP = N rounded up to a size with a kernel, zeros behind N), which takes any stride, type
// and alignment out of the inner loop.  C's rows are scalar operands.  B's enter through the matrix cores' outer
// product in the output pass (as scalar operands its rows and C's wait for each other; through LDS it takes the
// same time), through LDS reads in the state pass, which has no other scalar loads to wait for: at the sizes below
// 121 us, 127 through the matrix cores or as scalar operands (3 x 333 x 200, where latency counts: 8.9 and 8.1).
//
// Split.  A sequence gives only D / 64 waves, the device wants a few per SIMD.  Sequences are
// cut into G segments: a first pass runs segments 0..G-2 from zero and keeps their end states and sums
// of delta (a segment's total decay is exp(A sum delta)), a scan over the segments turns them into
// every segment's incoming state, and the second pass runs all segments from those.  The first
// pass costs (G - 1) / G of one more recurrence without the output sum.
//
// 16384 tokens x 2048 channels, N = 16, bf16 with a gate: packing 5 us, states 121, segments 12, outputs 143.  Without
// the exponentials of the decays, and the waits for them, the state pass takes 50 us less, without the softplus 19; the
// output pass has the gate's sigmoid and the output sum besides.  What it reads and writes is 268 MB, 56 us at a copy's
// rate.
#include "la_mixer.h"
#include "ssm_common.h"
#include "ssm_tile.h"

namespace la {
namespace {

struct FwdDev {
    const void* u;
    const void* dt;
    const void* z;
    const float* Dskip;
    const float* dt_bias;
    const float* bc;     // [B, L, 2 NP]
    const float* a2;     // [NP, D] rates times log2(e)
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

// The first launch: B and C as fp32 [B, L, 2 NP] and A log2(e) as [NP, D] (channels contiguous, so that a
// wave's loads of its rates coalesce), zeros behind N.
template <typename T>
__global__ __launch_bounds__(256) void pack_kernel(const T* __restrict__ Bm, const T* __restrict__ Cm,
                                                   const float* __restrict__ A, la_rows sb, la_rows sc,
                                                   float* __restrict__ bc, float* __restrict__ a2, int64_t rows, int64_t L,
                                                   int64_t D, int N, int NP, unsigned nbc) {
    if (blockIdx.x >= nbc) {
        const int64_t i = (int64_t)(blockIdx.x - nbc) * 256 + threadIdx.x;
        const int64_t n = i / D, d = i % D;
        if (n < NP) a2[i] = n < N ? A[d * N + n] * LOG2E : 0.f;
        return;
    }
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

// The kernel's arguments, read again from memory where they are used: held over the token loop they would push
// each other and the rows of B and C out of the scalar registers (5 x 777 x 1000 fp32, N = 24: 29 -> 24 us a pass).
typedef const __attribute__((address_space(4))) FwdDev* FwdArgsPtr;
__device__ __forceinline__ FwdArgsPtr fwd_args() {
    FwdArgsPtr q = (FwdArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(q));
    return q;
}

// STATE: the first pass (a segment's end state from zero and its sum of delta), else the second.  VEC: rows are
// 16-byte aligned and whole 8-channel chunks.  Tokens of a tile behind the segment's end repeat its last row
// with delta = 0 (decay 1, input 0): they leave the state alone and are not stored.
template <typename E, int NP, bool STATE, bool VEC>
__global__ __launch_bounds__(64, 2) void ssm_fwd_kernel(FwdDev p) {
    constexpr int NS = STATE ? 2 : 3;
    constexpr int BV = TT * NP / 64;
    __shared__ __align__(16) E tile[STATE ? 2 : 4][TT * 64];  // u, dt, z, y
    __shared__ __align__(16) float brow[STATE ? TT * NP : 4];  // first pass: B of the tile's tokens
    // blocks: channel block fastest, then segment, then sequence
    const unsigned r = blockIdx.x / p.cb;
    const int g = (int)(r % p.ng);
    const int64_t b = r / p.ng;
    const int64_t d0 = (int64_t)(blockIdx.x % p.cb) * 64;
    const int lane = threadIdx.x;
    const bool live = d0 + lane < p.D;
    const int64_t d = live ? d0 + lane : p.D - 1;  // lanes behind the last channel repeat it
    const TilePlace pl(d0, p.D);

    // key dim 4 q + i is element i of h[q]
    f32x4 h[NP / 4];
    float A2[NP];
#pragma unroll
    for (int n = 0; n < NP; n++) {
        A2[n] = p.a2[n * p.D + d];
        h[n / 4][n % 4] = 0.f;
    }
    if (!STATE && p.hin) {
#pragma unroll
        for (int n = 0; n < NP; n++) {
            const float v = p.hin[((b * p.G + g) * p.N + min(n, p.N - 1)) * p.D + d];
            h[n / 4][n % 4] = n < p.N ? v : 0.f;
        }
    }
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.f;
    const float skip = !STATE && p.Dskip ? p.Dskip[d] : 0.f;
    const int t0 = (int)(g * p.seglen), t1 = min(t0 + (int)p.seglen, uniform((int)seq_len(p.lengths, b, p.L)));
    const bool gate = !STATE && p.z;
    const bool sp = p.softplus;
    const float* const bcb = p.bc + b * p.L * (2 * NP);
    scalar_f32 rowc = as_scalar(bcb + t0 * (2 * NP) + NP);

    Raw8<E> raw[NS];
    float br[BV], bn[BV];  // B of the tile's tokens, value j NP + n in lane (j NP + n) % 64, and the next tile's
    auto fetch = [&](int t) {
        const FwdArgsPtr q = fwd_args();
        const int tt = min(t + pl.token, t1 - 1);
        raw[0] = token_load<E, VEC>((const E*)q->u + b * q->su.batch + d0, q->su.token, tt, pl);
        raw[1] = token_load<E, VEC>((const E*)q->dt + b * q->sdt.batch + d0, q->sdt.token, tt, pl);
        if (gate) raw[NS - 1] = token_load<E, VEC>((const E*)q->z + b * q->sz.batch + d0, q->sz.token, tt, pl);
#pragma unroll
        for (int v = 0; v < BV; v++) {
            const int e = v * 64 + lane;
            bn[v] = bcb[min(t + e / NP, t1 - 1) * (2 * NP) + e % NP];
        }
    };
    float sum = 0.f;
    if (t0 < t1) fetch(t0);
    for (int t = t0; t < t1; t += TT) {
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < NS; i++)
            if (i < 2 || gate) *lds_chunk(tile[i]) = raw[i];
        if (STATE)
#pragma unroll
            for (int v = 0; v < BV; v++) brow[v * 64 + lane] = bn[v];
        wave_lds_fence();
        float dl[TT], du[TT], out[TT];
#pragma unroll
        for (int j = 0; j < TT; j++) dl[j] = (float)tile[1][j * 64 + lane] + bias;
        if (sp) {
#pragma unroll
            for (int j = 0; j < TT; j++) dl[j] = softplus(dl[j]);
        }
#pragma unroll
        for (int j = 0; j < TT; j++) {
            const float u = (float)tile[0][j * 64 + lane];
            dl[j] = t + j < t1 ? dl[j] : 0.f;
            du[j] = dl[j] * u;
            out[j] = skip * u;
        }
#pragma unroll
        for (int v = 0; v < BV; v++) br[v] = bn[v];
        if (t + TT < t1) fetch(t + TT);
        static_for<TT>([&](auto J) {
            constexpr int j = J;
            static_for<NP / 4>([&](auto Q) {
                constexpr int q = Q;
                f32x4 c;
#pragma unroll
                for (int i = 0; i < 4; i++) c[i] = __builtin_amdgcn_exp2f(dl[j] * A2[4 * q + i]) * h[q][i];
                if (STATE) {
                    const f32x4 bq = *(const f32x4*)(brow + j * NP + 4 * q);
#pragma unroll
                    for (int i = 0; i < 4; i++) h[q][i] = fmaf(bq[i], du[j], c[i]);
                } else {
                    h[q] = outer4<j * NP + 4 * q>(br, du[j], c);
                }
            });
            if (STATE) {
                sum += dl[j];
            } else {
                float acc = 0.f;
#pragma unroll
                for (int n = 0; n < NP; n++) {
                    if (n & 1) acc = fmaf(rowc[n], h[n / 4][n % 4], acc);
                    else out[j] = fmaf(rowc[n], h[n / 4][n % 4], out[j]);
                }
                out[j] += acc;
                rowc += t + j + 1 < t1 ? 2 * NP : 0;
            }
        });
        if (STATE) continue;
        if (gate) {
#pragma unroll
            for (int j = 0; j < TT; j++) {
                const float z = (float)tile[2][j * 64 + lane];
                out[j] *= z * sigmoid(z);
            }
        }
#pragma unroll
        for (int j = 0; j < TT; j++) io<E>::st(tile[3] + j * 64 + lane, out[j]);
        wave_lds_fence();
        if (pl.in && t + pl.token < t1) {
            const FwdArgsPtr q = fwd_args();
            store8<VEC>((E*)q->y + b * q->sy.batch + d0 + (t + pl.token) * q->sy.token + pl.col, pl.n,
                        *lds_chunk(tile[3]));
        }
    }
    if (!live) return;
    const FwdArgsPtr e = fwd_args();
    const int64_t D = e->D;
    const int N = e->N;
    if (STATE) {
        float* part = e->part + (b * e->G + g + 1) * N * D + d0;
#pragma unroll
        for (int n = 0; n < NP; n++)
            if (n < N) (part + n * D)[lane] = h[n / 4][n % 4];
        (e->sumdt + (b * e->G + g) * D + d0)[lane] = sum;
    } else if (e->s_out && g == e->G - 1) {
        float* so = e->s_out + b * N * D + d0;
#pragma unroll
        for (int n = 0; n < NP; n++)
            if (n < N) (so + n * D)[lane] = h[n / 4][n % 4];
    }
}

// States entering the segments from the segments' own end states: slot 0 takes s_in, slot g + 1
// (holding segment g's end state from zero) adds the decayed state that entered segment g.
template <int PARTS>
__global__ __launch_bounds__(64 * PARTS) void ssm_segments_kernel(const float* __restrict__ a2, const float* __restrict__ s_in,
                                                           const float* sumdt, float* part, int64_t total, int64_t D,
                                                           int N, int G) {
    const int64_t i0 = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
    const bool on = i0 < total;
    const int64_t i = on ? i0 : 0;
    const int64_t d = i % D, n = i / D % N, b = i / (D * N);
    const float x0 = s_in ? s_in[i] : 0.f;
    float* pp = part + (b * G * N + n) * D + d;
    const float* sp = sumdt + b * G * D + d;
    const int64_t ps = (int64_t)N * D;
    if (on && threadIdx.x < 64) pp[0] = x0;
    segment_chain<PARTS>(
        G - 1, x0, a2[n * D + d], on, [&](int k) { return pp + (k + 1) * ps; }, [&](int k) { return sp + k * D; },
        [&](int k, float, float next) { pp[(k + 1) * ps] = next; });
}

int fwd_np(int N) { return N <= 8 ? 8 : N <= 16 ? 16 : N <= 24 ? 24 : N <= 32 ? 32 : N <= 48 ? 48 : 64; }

// Segments: about 4096 waves, none under 16 tokens.
SsmPlan fwd_plan(int64_t B, int64_t L, int64_t D) { return ssm_plan(B, L, D, 4096, 16, TT); }

struct FwdWs {
    float *bc, *a2, *part, *sumdt;
    size_t bytes;
};
FwdWs fwd_cut(void* base, int64_t B, int64_t L, int64_t D, int N, int G) {
    WsCut c{(char*)base};
    FwdWs w;
    w.bc = c.take((size_t)(B * L) * 2 * fwd_np(N));
    w.a2 = c.take((size_t)fwd_np(N) * D);
    w.part = G > 1 ? c.take((size_t)(B * G) * N * D) : nullptr;
    w.sumdt = G > 1 ? c.take((size_t)(B * G) * D) : nullptr;
    w.bytes = c.used;
    return w;
}

template <typename T, int NP, bool VEC>
void launch_np(const SsmArgs& a, FwdDev p, const SsmPlan& pl) {
    p.cb = (unsigned)((a.D + 63) / 64);
    if (pl.G > 1) {
        p.ng = pl.G - 1;
        LA_TRACED(a.tr, "ssm_state", ssm_fwd_kernel<T, NP, true, VEC><<<p.cb * p.ng * (unsigned)a.B, 64, 0, a.stream>>>(p));
        const int64_t total = a.B * a.N * a.D;
#define LA_SSM_SEGMENTS(n)                                                                                    \
    LA_TRACED(a.tr, "ssm_segments", ssm_segments_kernel<n><<<(unsigned)((total + 63) / 64), 64 * n, 0, a.stream>>>( \
                                        p.a2, a.s_in, p.sumdt, p.part, total, a.D, a.N, pl.G))
        if (segment_parts(total) == 16) LA_SSM_SEGMENTS(16);
        else LA_SSM_SEGMENTS(4);
#undef LA_SSM_SEGMENTS
    }
    p.ng = pl.G;
    LA_TRACED(a.tr, "ssm_out", ssm_fwd_kernel<T, NP, false, VEC><<<p.cb * p.ng * (unsigned)a.B, 64, 0, a.stream>>>(p));
}

template <typename T>
hipError_t launch_t(const SsmArgs& a) {
    const SsmPlan pl = fwd_plan(a.B, a.L, a.D);
    const FwdWs w = fwd_cut(a.ws, a.B, a.L, a.D, a.N, pl.G);
    const int NP = fwd_np(a.N);
    FwdDev p;
    p.u = a.u; p.dt = a.dt; p.z = a.z; p.Dskip = a.Dskip; p.dt_bias = a.dt_bias;
    p.bc = w.bc;
    p.a2 = w.a2;
    p.hin = pl.G > 1 ? w.part : a.s_in;
    p.lengths = a.lengths; p.y = a.y; p.s_out = a.s_out;
    p.part = w.part; p.sumdt = w.sumdt;
    p.L = a.L; p.D = a.D; p.seglen = pl.seglen; p.N = a.N; p.G = pl.G;
    p.softplus = a.softplus;
    p.su = a.su; p.sdt = a.sdt; p.sz = a.sz; p.sy = a.sy;
    launch_pack(a, w.bc, w.a2, NP);
    const bool vec = a.D % 8 == 0 && rows16(a.u, a.su, sizeof(T)) && rows16(a.dt, a.sdt, sizeof(T)) &&
                     rows16(a.z, a.sz, sizeof(T)) && rows16(a.y, a.sy, sizeof(T));
#define LA_SSM_NP(n) (vec ? launch_np<T, n, true>(a, p, pl) : launch_np<T, n, false>(a, p, pl))
    switch (NP) {
        case 8: LA_SSM_NP(8); break;
        case 16: LA_SSM_NP(16); break;
        case 24: LA_SSM_NP(24); break;
        case 32: LA_SSM_NP(32); break;
        case 48: LA_SSM_NP(48); break;
        default: LA_SSM_NP(64); break;
    }
#undef LA_SSM_NP
    return hipGetLastError();
}

// ---------------------------------------------------------------------------------------------
// One token per sequence.  A lane owns one channel and reads and writes its state once, 256 contiguous bytes
// per wave and key dim; with many rows a wave takes R of them one after the other, the next row's loads in
// flight, so that its rates (A's rows, N floats apart from lane to lane) are loaded once for all of them.
// B and C are loaded once per wave and row, lane n holding B[n] and C[n], and broadcast by lane reads.
struct StepDev {
    const void* u;
    const void* dt;
    const void* Bm;
    const void* Cm;
    const void* z;
    const float* A;
    const float* Dskip;
    const float* dt_bias;
    float* state;
    const int32_t* slots;
    void* y;
    int64_t su, sdt, sb, sc, sz, sy, B, D;
    unsigned cb;
    int N, nslots, R;
    bool softplus;
};

// A4: A's rows are 16-byte aligned (N a multiple of 4).
template <typename T, int NP, bool A4>
__global__ __launch_bounds__(64) void ssm_step_kernel(StepDev p) {
    const int64_t d0 = (int64_t)(blockIdx.x % p.cb) * 64;
    const bool live = d0 + threadIdx.x < p.D;
    const int64_t d = live ? d0 + threadIdx.x : p.D - 1;
    const int64_t b0 = (int64_t)(blockIdx.x / p.cb) * p.R, b1 = min(b0 + p.R, p.B);
    const int n0 = threadIdx.x < p.N ? threadIdx.x : p.N - 1;

    float h[NP], nb, nc, nu, nx, nz = 0.f;
    int slot;
    auto fetch = [&](int64_t b) {
        slot = p.slots ? uniform(p.slots[b]) : (int)b;
        const bool ok = slot >= 0 && slot < p.nslots;
        const float* st = p.state + (int64_t)(ok ? slot : 0) * p.N * p.D + d;
        if (ok)
#pragma unroll
            for (int n = 0; n < NP; n++) h[n] = st[min(n, p.N - 1) * p.D];
        nb = (float)((const T*)p.Bm)[b * p.sb + n0];
        nc = (float)((const T*)p.Cm)[b * p.sc + n0];
        nu = (float)((const T*)p.u)[b * p.su + d];
        nx = (float)((const T*)p.dt)[b * p.sdt + d];
        if (p.z) nz = (float)((const T*)p.z)[b * p.sz + d];
    };
    fetch(b0);
    float a2[NP];
    const float* ar = p.A + d * p.N;
#pragma unroll
    for (int n = 0; n < NP; n += 4) {
        if (A4) {
            const f32x4 v = *(const f32x4*)(ar + min(n, p.N - 4));
#pragma unroll
            for (int i = 0; i < 4; i++) a2[n + i] = v[i] * LOG2E;
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) a2[n + i] = ar[min(n + i, p.N - 1)] * LOG2E;
        }
    }
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.f, skip = p.Dskip ? p.Dskip[d] : 0.f;
    for (int64_t b = b0; b < b1; b++) {
        float cur[NP];
#pragma unroll
        for (int n = 0; n < NP; n++) cur[n] = h[n];
        const float bl = nb, cl = nc, u = nu, x = nx + bias, z = nz;
        const int s = slot;
        if (b + 1 < b1) fetch(b + 1);
        if (s < 0 || s >= p.nslots) continue;
        if (p.slots && earlier_row_has(p.slots, b, s)) continue;
        const float delta = p.softplus ? softplus(x) : x;
        const float du = delta * u;
        float acc = skip * u;
#pragma unroll
        for (int n = 0; n < NP; n++)
            if (n < p.N) {
                const float bn = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(bl), n));
                const float cn = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(cl), n));
                cur[n] = fmaf(__builtin_amdgcn_exp2f(delta * a2[n]), cur[n], du * bn);
                acc = fmaf(cn, cur[n], acc);
            }
        if (p.z) acc *= z * sigmoid(z);
        if (live) {
            float* st = p.state + (int64_t)s * p.N * p.D + d;
#pragma unroll
            for (int n = 0; n < NP; n++)
                if (n < p.N) st[(int64_t)n * p.D] = cur[n];
            io<T>::st((T*)p.y + b * p.sy + d, acc);
        }
    }
}

// Rows per wave: one until there are 4096 waves, then up to 4 (256 rows x 4096, N = 16, in one session: 1 row 27.9 us,
// 2 26.1, 4 25.7; 8 and 16 rows take 3 and 16 us more than 4).
int step_rows(int64_t B, int64_t cb) { return (int)std::min<int64_t>(4, std::max<int64_t>(1, B * cb / 4096)); }

template <typename T, int NP>
void step_np(const SsmArgs& a) {
    StepDev p;
    p.u = a.u; p.dt = a.dt; p.Bm = a.Bm; p.Cm = a.Cm; p.z = a.z; p.A = a.A; p.Dskip = a.Dskip; p.dt_bias = a.dt_bias;
    p.state = a.state; p.slots = a.slots; p.y = a.y;
    p.su = a.su.batch; p.sdt = a.sdt.batch; p.sb = a.sb.batch; p.sc = a.sc.batch; p.sz = a.sz.batch; p.sy = a.sy.batch;
    p.B = a.B; p.D = a.D; p.cb = (unsigned)((a.D + 63) / 64); p.N = a.N; p.nslots = a.nslots; p.softplus = a.softplus;
    p.R = step_rows(a.B, p.cb);
    const unsigned blocks = p.cb * (unsigned)((a.B + p.R - 1) / p.R);
    if (a.N % 4 == 0 && (uintptr_t)a.A % 16 == 0)
        LA_TRACED(a.tr, "ssm_step", ssm_step_kernel<T, NP, true><<<blocks, 64, 0, a.stream>>>(p));
    else
        LA_TRACED(a.tr, "ssm_step", ssm_step_kernel<T, NP, false><<<blocks, 64, 0, a.stream>>>(p));
}
template <typename T>
hipError_t step_t(const SsmArgs& a) {
    switch (fwd_np(a.N)) {
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
void pack_t(const SsmArgs& a, float* bc, float* a2, int NP) {
    const unsigned nbc = (unsigned)((a.B * a.L * 2 * NP + 255) / 256), na = (unsigned)((a.D * NP + 255) / 256);
    LA_TRACED(a.tr, "ssm_pack", pack_kernel<T><<<nbc + na, 256, 0, a.stream>>>((const T*)a.Bm, (const T*)a.Cm, a.A, a.sb,
                                                                               a.sc, bc, a2, a.B * a.L, a.L, a.D, a.N, NP,
                                                                               nbc));
}

}  // namespace

void launch_pack(const SsmArgs& a, float* bc, float* a2, int NP) {
    a.bf16 ? pack_t<__bf16>(a, bc, a2, NP) : pack_t<float>(a, bc, a2, NP);
}

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
