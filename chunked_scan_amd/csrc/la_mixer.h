// la_mixer.h -- host-side interface and device helpers of the selective state space layer (the short convolution, the
// selective scan, the residual norm) and of the gated recurrent layer (the gated recurrence, the norms around a block,
// dropout).  Launchers get validated arguments.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "la_chunk.h"
#include "la_device.h"
#include "la_internal.h"

namespace la {

struct ConvArgs {
    const void* x;
    const float* weight;
    const float* bias;
    const void* state_in;
    const int32_t* lengths;
    void* y;
    void* state_out;
    // backward
    const void* dy;
    const void* d_state_out;
    void* dx;
    float* d_weight;
    float* d_bias;
    void* d_state_in;
    void* ws;
    // step
    void* state;
    const int32_t* slots;
    int nslots;
    int64_t B, L, D;
    int width;
    bool bf16, silu;
    la_rows sx, sy, sdy, sdx;  // resolved strides
    hipStream_t stream;
    Tracer* tr;
};
hipError_t launch_short_conv(const ConvArgs& a);
size_t short_conv_bwd_ws(int64_t B, int64_t L, int64_t D, int width);
hipError_t launch_short_conv_bwd(const ConvArgs& a);
hipError_t launch_short_conv_step(const ConvArgs& a);

struct SsmArgs {
    const void* u;
    const void* dt;
    const float* A;
    const void* Bm;
    const void* Cm;
    const float* Dskip;
    const void* z;
    const float* dt_bias;
    const float* s_in;
    const int32_t* lengths;
    void* y;
    float* s_out;
    // backward
    const void* dy;
    const float* ds_out;
    void* du;
    void* ddt;
    float* dA;
    void* dB;
    void* dC;
    float* dD;
    void* dz;
    float* d_dt_bias;
    float* ds_in;
    void* ws;
    // step
    float* state;
    const int32_t* slots;
    int nslots;
    int64_t B, L, D;
    int N;
    bool bf16, softplus;
    la_rows su, sdt, sb, sc, sz, sy, sdy, sdu, sddt, sdb, sdc, sdz;  // resolved strides
    hipStream_t stream;
    Tracer* tr;
};
size_t ssm_fwd_ws(int64_t B, int64_t L, int64_t D, int N);
hipError_t launch_ssm_scan(const SsmArgs& a);
size_t ssm_bwd_ws(int64_t B, int64_t L, int64_t D, int N);
hipError_t launch_ssm_scan_bwd(const SsmArgs& a);
hipError_t launch_ssm_step(const SsmArgs& a);

struct NormArgs {
    const void* x;
    const void* residual;
    const float* weight;
    void* y;
    uint8_t* q;
    float* scale;
    void* h;
    float* rstd;
    // backward
    const void* dy;
    const void* h_in;
    const float* rstd_in;
    const void* dh;
    void* dx;
    float* d_weight;
    void* ws;
    int64_t M, D;
    int group;
    float eps;
    bool bf16;
    int64_t sx, sres, sy, sh, sdy, sdh, sdx;  // resolved strides
    hipStream_t stream;
    Tracer* tr;
};
hipError_t launch_add_norm(const NormArgs& a);
size_t add_norm_bwd_ws(int64_t M, int64_t D);
hipError_t launch_add_norm_bwd(const NormArgs& a);

struct GatedArgs {
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
    // backward
    const float* blocks_in;
    const void* dy;
    const float* dh_out;
    void* dx;
    void* dr;
    void* di;
    float* dlam;
    float* dr_bias;
    float* di_bias;
    void* dz;
    float* dh_in;
    void* ws;
    // step
    float* state;
    const int32_t* slots;
    int nslots;
    int64_t B, L, D;
    float c;
    bool bf16;
    la_rows sx, sr, si, sz, sy, sdy, sdx, sdr, sdi, sdz;  // resolved strides
    hipStream_t stream;
    Tracer* tr;
};
size_t gated_fwd_ws(int64_t B, int64_t L, int64_t D);
hipError_t launch_gated_scan(const GatedArgs& a);
size_t gated_bwd_ws(int64_t B, int64_t L, int64_t D, bool have_blocks);
hipError_t launch_gated_scan_bwd(const GatedArgs& a);
hipError_t launch_gated_step(const GatedArgs& a);
// as chain_status, of the gated recurrence's waits
hipError_t gated_status(unsigned int* give_ups, bool clear);

struct BlockArgs {
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
    // backward
    const void* h_in;
    const float* rstd_post_in;
    const float* rstd_pre_in;
    const void* dy;
    const void* dh;
    void* dx;
    void* dgate;
    void* dres;
    float* dw_post;
    float* dscale;
    float* dw_pre;
    void* ws;
    int64_t M, D;
    int act;
    unsigned drop;  // T: dropped where 16 random bits are below it
    float eps;
    bool bf16;
    int64_t sx, sg, sres, sy, sh, sdy, sdh, sdx, sdg, sdres;  // resolved strides
    hipStream_t stream;
    Tracer* tr;
};
hipError_t launch_block_norm(const BlockArgs& a);
size_t block_norm_bwd_ws(int64_t M, int64_t D);
hipError_t launch_block_norm_bwd(const BlockArgs& a);
hipError_t launch_dropout(const BlockArgs& a);

// Whether every row of a view starts on 16 bytes.
inline bool rows16(const void* p, const la_rows& r, size_t es) {
    return !p || ((uintptr_t)p % 16 == 0 && (r.batch * es) % 16 == 0 && (r.token * es) % 16 == 0);
}

// A workspace cut into 256-byte aligned regions.
struct WsCut {
    char* base;
    size_t used = 0;
    float* take(size_t floats) {
        float* p = base ? reinterpret_cast<float*>(base + used) : nullptr;
        used += (floats * sizeof(float) + 255) & ~(size_t)255;
        return p;
    }
};

// ---------------------------------------------------------------------------------------------
// device helpers

// A float array read through the scalar cache (uniform addresses, data that no launch in flight writes).
typedef const __attribute__((address_space(4))) float* scalar_f32;
__device__ __forceinline__ scalar_f32 as_scalar(const float* p) { return (scalar_f32)(uintptr_t)p; }
// The same for an address that the compiler does not see to be uniform (one that depends on the wave's number).
__device__ __forceinline__ scalar_f32 as_scalar_uniform(const float* p) {
    const uint64_t a = (uint64_t)(uintptr_t)p;
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));
    return (scalar_f32)(uintptr_t)(((uint64_t)hi << 32) | lo);
}

// A value that is the same in all lanes, moved to a scalar register.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

__device__ __forceinline__ float rcp(float x) { return __builtin_amdgcn_rcpf(x); }

// 1 / (1 + e^-x): the hardware's base-2 exponential and reciprocal, about 1 ulp each.  For x far
// below zero e^-x overflows to infinity and the result is 0.
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + __builtin_amdgcn_exp2f(x * -LOG2E)); }

// 1 - s for s = sigma(x) = 1 / (1 + e), e = e^-x: e s where s is the greater part, since the difference keeps none of the
// digits of what is left next to 1.  (e infinite: s = 0, and the difference is exact.)
__device__ __forceinline__ float complement(float e, float s) { return e < 1.f ? e * s : 1.f - s; }

// delta = log(1 + e^x) = max(x, 0) + log1p(y), y = e^-|x| in [0, 1].  Step sizes of 1e-3 are ordinary,
// so log1p needs its relative accuracy near y = 0, which log2(1 + y) loses (2^-24 / y).  With
// s = y / (2 + y) <= 1/3, log1p(y) = 2 atanh(s) = s P(s^2); the degree-4 P below was fitted at the
// Chebyshev nodes of s^2 in [0, 1/9].  The fit is within 8e-9 of it relative to the value; evaluated in fp32, P is
// within 7e-8 and the product s P within 1.3e-7, before the ulps of y and of the reciprocal.
__device__ __forceinline__ float softplus(float x) {
    const float y = __builtin_amdgcn_exp2f(-fabsf(x) * LOG2E);
    const float s = y * rcp(2.f + y);
    const float v = s * s;
    float p = 0x1.20822cp-2f;
    p = fmaf(p, v, 0x1.1e532ep-2f);
    p = fmaf(p, v, 0x1.99dac0p-2f);
    p = fmaf(p, v, 0x1.5554e0p-1f);
    p = fmaf(p, v, 2.f);
    return fmaf(s, p, fmaxf(x, 0.f));
}

// Two values rounded to bf16, nearest even, in one instruction; and eight.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}
__device__ __forceinline__ u32x4 pack8_pairs(const float* f) {
    return u32x4{pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])};
}

__device__ __forceinline__ int64_t seq_len(const int32_t* lengths, int64_t b, int64_t L) {
    if (!lengths) return L;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : (n < L ? n : L);
}

// Rows that name a slot an earlier row names are padding, so that no two rows write one state.  Every wave looks
// through the earlier rows' slots, which is quadratic in the rows: nothing at a few thousand; 65536 rows of 64 channels
// take 1.15 ms, 0.09 without slots.
__device__ __forceinline__ bool earlier_row_has(const int32_t* slots, int64_t b, int32_t s) {
    bool dup = false;
    for (int64_t i = threadIdx.x & 63; i < b; i += 64) dup |= slots[i] == s;
    return __any(dup);
}

}  // namespace la
