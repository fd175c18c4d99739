// la_mixer_api.hip -- the C ABI of the selective state space layer (declared in include/la_chunk.h):
// short convolution, selective scan, residual norm.  As in la_api.hip every argument is validated on the
// host before the first HIP call; validation order: shape pointer, sizes, limits, dtype, required
// pointers, strides, workspace, aliasing; the first failure is returned.
#include <math.h>
#include <stdint.h>

#include "la_chunk.h"
#include "la_internal.h"
#include "la_mixer.h"
#include "la_views.h"

using namespace la::api;

namespace {

// ---------------------------------------------------------------- convolution

la_status conv_shape(const la_conv_shape* s, bool step) {
    if (!s) return LA_ERR_NULL;
    const la_status st = sizes_ok(s, step ? 1 : s->L);
    if (st != LA_OK) return st;
    if (step && s->nslots < 0) return LA_ERR_SHAPE;
    if (s->width < 2 || s->width > 4 || (step && mul(s->nslots, s->D) > kMaxElems)) return LA_ERR_UNSUPPORTED;
    if (!dtype_ok(s->dtype)) return LA_ERR_DTYPE;
    if (s->silu != 0 && s->silu != 1) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

la::ConvArgs conv_args(const la_conv_shape* s, int64_t L) {
    la::ConvArgs a = {};
    a.B = s->B; a.L = L; a.D = s->D; a.width = s->width;
    a.bf16 = s->dtype == LA_BF16; a.silu = s->silu != 0; a.nslots = s->nslots;
    a.sx = resolve(s->x, L, s->D); a.sy = resolve(s->y, L, s->D);
    a.sdy = resolve(s->dy, L, s->D); a.sdx = resolve(s->dx, L, s->D);
    a.stream = (hipStream_t)s->stream;
    return a;
}

// ---------------------------------------------------------------- scan

la_status ssm_shape(const la_ssm_shape* s, bool step) {
    if (!s) return LA_ERR_NULL;
    const la_status st = sizes_ok(s, step ? 1 : s->L);
    if (st != LA_OK) return st;
    if (s->N < 1 || (step && s->nslots < 0)) return LA_ERR_SHAPE;
    if (s->N > 64 || (step && mul(mul(s->nslots, s->D), s->N) > kMaxElems)) return LA_ERR_UNSUPPORTED;
    if (!dtype_ok(s->dtype)) return LA_ERR_DTYPE;
    if (s->softplus != 0 && s->softplus != 1) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

la::SsmArgs ssm_args(const la_ssm_shape* s, int64_t L) {
    la::SsmArgs a = {};
    a.B = s->B; a.L = L; a.D = s->D; a.N = s->N;
    a.bf16 = s->dtype == LA_BF16; a.softplus = s->softplus != 0; a.nslots = s->nslots;
    a.su = resolve(s->u, L, s->D); a.sdt = resolve(s->dt, L, s->D); a.sz = resolve(s->z, L, s->D);
    a.sy = resolve(s->y, L, s->D); a.sb = resolve(s->b, L, s->N); a.sc = resolve(s->c, L, s->N);
    a.sdy = resolve(s->dy, L, s->D); a.sdu = resolve(s->du, L, s->D); a.sddt = resolve(s->ddt, L, s->D);
    a.sdz = resolve(s->dz, L, s->D); a.sdb = resolve(s->db, L, s->N); a.sdc = resolve(s->dc, L, s->N);
    a.stream = (hipStream_t)s->stream;
    return a;
}

// ---------------------------------------------------------------- norm

la_status norm_shape(const la_norm_shape* s) {
    if (!s) return LA_ERR_NULL;
    if (s->M < 0 || s->D < 1 || !(s->eps > 0.f) || !isfinite(s->eps) || s->reserved != 0) return LA_ERR_SHAPE;
    if (s->D > 16384 || s->M > kMaxNormRows || mul(s->M, s->D) > kMaxNormElems) return LA_ERR_UNSUPPORTED;
    if (!dtype_ok(s->dtype)) return LA_ERR_DTYPE;
    for (int64_t st : {s->x_stride, s->residual_stride, s->y_stride, s->h_stride, s->dy_stride, s->dh_stride, s->dx_stride})
        if (st < 0 || st > kMaxSpan || mul(s->M, st) > kMaxSpan) return LA_ERR_SHAPE;
    return LA_OK;
}

la::NormArgs norm_args(const la_norm_shape* s) {
    la::NormArgs a = {};
    auto st = [&](int64_t v) { return v ? v : s->D; };
    a.M = s->M; a.D = s->D; a.group = s->group; a.eps = s->eps; a.bf16 = s->dtype == LA_BF16;
    a.sx = st(s->x_stride); a.sres = st(s->residual_stride); a.sy = st(s->y_stride); a.sh = st(s->h_stride);
    a.sdy = st(s->dy_stride); a.sdh = st(s->dh_stride); a.sdx = st(s->dx_stride);
    a.stream = (hipStream_t)s->stream;
    return a;
}
la_status norm_fwd(const void* x, const void* residual, const float* weight, void* y, uint8_t* q, float* scale, void* h,
                   float* rstd, const la_norm_shape* s, bool q8) {
    la_status st = norm_shape(s);
    if (st != LA_OK) return st;
    if (q8) {
        if (s->group != 0 && s->group != 32 && s->group != 64 && s->group != 128) return LA_ERR_UNSUPPORTED;
        if (s->group && s->D % s->group) return LA_ERR_SHAPE;
    }
    if (s->M > 0 && (!x || !weight || (q8 ? !q || !scale : !y))) return LA_ERR_NULL;
    la::NormArgs a = norm_args(s);
    const size_t es = esize(s->dtype);
    const View vx = mat(x, s->M, a.sx, s->D, es), vr = mat(residual, s->M, a.sres, s->D, es), vw = flat(weight, s->D * 4);
    const View vy = mat(y, s->M, a.sy, s->D, es), vh = mat(h, s->M, a.sh, s->D, es), vs = flat(rstd, s->M * 4);
    const View vq = flat(q, s->M * s->D), vc = flat(scale, s->M * 4 * (s->group ? s->D / s->group : 1));
    const View in[] = {vx, vr, vw};
    const View out[] = {vy, vs, vq, vc};
    if (clash(in, out)) return LA_ERR_ALIAS;
    if (self_overlap(vh) || overlap(vh, vw) || overlap(vh, vy) || overlap(vh, vs) || overlap(vh, vq) || overlap(vh, vc) ||
        clash_inplace(vh, vx) || clash_inplace(vh, vr))
        return LA_ERR_ALIAS;
    // in place over one of the two while it partly overlaps the other is a clash already
    if ((st = check_trace(s->trace)) != LA_OK) return st;
    la::Tracer tr = make_tracer(s->trace, s->stream);
    a.x = x; a.residual = residual; a.weight = weight; a.y = y; a.q = q; a.scale = scale; a.h = h; a.rstd = rstd;
    a.tr = &tr;
    return from_hip(la::launch_add_norm(a));
}

}  // namespace

extern "C" {

la_status la_short_conv(const void* x, const float* weight, const float* bias, const void* state_in, const int32_t* lengths,
                        void* y, void* state_out, const la_conv_shape* s) {
    la_status st = conv_shape(s, false);
    if (st != LA_OK) return st;
    const int64_t n = s->B * s->L * s->D;
    if (n > 0 && (!x || !weight || !y)) return LA_ERR_NULL;
    if (!rows_ok(s, s->x, s->L) || !rows_ok(s, s->y, s->L)) return LA_ERR_SHAPE;
    la::ConvArgs a = conv_args(s, s->L);
    const size_t es = esize(s->dtype);
    const int64_t nst = s->B * (s->width - 1) * s->D * (int64_t)es;
    const View in[] = {rows(x, a.sx, s->B, s->L, s->D, es), flat(weight, s->D * s->width * 4), flat(bias, s->D * 4),
                       flat(state_in, nst), flat(lengths, s->B * 4)};
    const View out[] = {rows(y, a.sy, s->B, s->L, s->D, es), flat(state_out, nst)};
    if (clash(in, out)) return LA_ERR_ALIAS;
    if ((st = check_trace(s->trace)) != LA_OK) return st;
    la::Tracer tr = make_tracer(s->trace, s->stream);
    if (n == 0 && !(state_out && nst > 0)) return LA_OK;
    if (!weight) return LA_ERR_NULL;
    a.x = x; a.weight = weight; a.bias = bias; a.state_in = state_in; a.lengths = lengths; a.y = y; a.state_out = state_out;
    a.tr = &tr;
    return from_hip(la::launch_short_conv(a));
}

int64_t la_short_conv_bwd_workspace(const la_conv_shape* s) {
    const la_status st = conv_shape(s, false);
    if (st != LA_OK) return st;
    return (int64_t)la::short_conv_bwd_ws(s->B, s->L, s->D, s->width);
}

la_status la_short_conv_bwd(const void* x, const float* weight, const float* bias, const void* state_in,
                            const int32_t* lengths, const void* dy, const void* d_state_out, void* dx, float* d_weight,
                            float* d_bias, void* d_state_in, void* workspace, uint64_t workspace_bytes,
                            const la_conv_shape* s) {
    la_status st = conv_shape(s, false);
    if (st != LA_OK) return st;
    const int64_t n = s->B * s->L * s->D;
    if (n > 0 && (!x || !dy || !dx)) return LA_ERR_NULL;
    if (s->D > 0 && (!weight || !d_weight)) return LA_ERR_NULL;
    if (!rows_ok(s, s->x, s->L) || !rows_ok(s, s->dy, s->L) || !rows_ok(s, s->dx, s->L)) return LA_ERR_SHAPE;
    const size_t need = la::short_conv_bwd_ws(s->B, s->L, s->D, s->width);
    if (ws_bad(workspace, workspace_bytes, need)) return LA_ERR_WORKSPACE;
    la::ConvArgs a = conv_args(s, s->L);
    const size_t es = esize(s->dtype);
    const int64_t nst = s->B * (s->width - 1) * s->D * (int64_t)es;
    const View in[] = {rows(x, a.sx, s->B, s->L, s->D, es), flat(weight, s->D * s->width * 4), flat(bias, s->D * 4),
                       flat(state_in, nst), flat(lengths, s->B * 4), rows(dy, a.sdy, s->B, s->L, s->D, es),
                       flat(d_state_out, nst)};
    const View out[] = {rows(dx, a.sdx, s->B, s->L, s->D, es), flat(d_weight, s->D * s->width * 4), flat(d_bias, s->D * 4),
                        flat(d_state_in, nst), flat(workspace, (int64_t)need)};
    if (clash(in, out)) return LA_ERR_ALIAS;
    if ((st = check_trace(s->trace)) != LA_OK) return st;
    la::Tracer tr = make_tracer(s->trace, s->stream);
    a.x = x; a.weight = weight; a.bias = bias; a.state_in = state_in; a.lengths = lengths; a.dy = dy;
    a.d_state_out = d_state_out; a.dx = dx; a.d_weight = d_weight; a.d_bias = d_bias; a.d_state_in = d_state_in;
    a.ws = workspace;
    a.tr = &tr;
    return from_hip(la::launch_short_conv_bwd(a));
}

la_status la_short_conv_step(const void* x, const float* weight, const float* bias, void* state, const int32_t* slots,
                             void* y, const la_conv_shape* s) {
    la_status st = conv_shape(s, true);
    if (st != LA_OK) return st;
    if (!slots && s->nslots < s->B) return LA_ERR_SHAPE;
    const int64_t n = s->B * s->D;
    if (n > 0 && (!x || !weight || !y || (!state && s->nslots > 0))) return LA_ERR_NULL;
    if (!rows_ok(s, s->x, 1) || !rows_ok(s, s->y, 1)) return LA_ERR_SHAPE;
    la::ConvArgs a = conv_args(s, 1);
    const size_t es = esize(s->dtype);
    const View in[] = {rows(x, a.sx, s->B, 1, s->D, es), flat(weight, s->D * s->width * 4), flat(bias, s->D * 4),
                       flat(slots, s->B * 4)};
    const View out[] = {rows(y, a.sy, s->B, 1, s->D, es), flat(state, (int64_t)s->nslots * (s->width - 1) * s->D * (int64_t)es)};
    if (clash(in, out)) return LA_ERR_ALIAS;
    if ((st = check_trace(s->trace)) != LA_OK) return st;
    la::Tracer tr = make_tracer(s->trace, s->stream);
    a.x = x; a.weight = weight; a.bias = bias; a.state = state; a.slots = slots; a.y = y;
    a.tr = &tr;
    return from_hip(la::launch_short_conv_step(a));
}

int64_t la_ssm_workspace(const la_ssm_shape* s, int32_t backward) {
    const la_status st = ssm_shape(s, false);
    if (st != LA_OK) return st;
    return (int64_t)(backward ? la::ssm_bwd_ws(s->B, s->L, s->D, s->N) : la::ssm_fwd_ws(s->B, s->L, s->D, s->N));
}

la_status la_ssm_scan(const void* u, const void* dt, const float* A, const void* Bm, const void* Cm, const float* Dskip,
                      const void* z, const float* dt_bias, const float* s_in, const int32_t* lengths, void* y, float* s_out,
                      void* workspace, uint64_t workspace_bytes, const la_ssm_shape* s) {
    la_status st = ssm_shape(s, false);
    if (st != LA_OK) return st;
    const int64_t n = s->B * s->L * s->D;
    if (n > 0 && (!u || !dt || !Bm || !Cm || !y)) return LA_ERR_NULL;
    if (s->B * s->D > 0 && !A) return LA_ERR_NULL;
    for (const la_rows& r : {s->u, s->dt, s->b, s->c, s->z, s->y})
        if (!rows_ok(s, r, s->L)) return LA_ERR_SHAPE;
    const size_t need = la::ssm_fwd_ws(s->B, s->L, s->D, s->N);
    if (ws_bad(workspace, workspace_bytes, need)) return LA_ERR_WORKSPACE;
    la::SsmArgs a = ssm_args(s, s->L);
    const size_t es = esize(s->dtype);
    const int64_t B = s->B, L = s->L, D = s->D, N = s->N, nst = B * N * D * 4;
    const View in[] = {rows(u, a.su, B, L, D, es), rows(dt, a.sdt, B, L, D, es), flat(A, D * N * 4),
                       rows(Bm, a.sb, B, L, N, es), rows(Cm, a.sc, B, L, N, es), flat(Dskip, D * 4),
                       rows(z, a.sz, B, L, D, es), flat(dt_bias, D * 4), flat(s_in == s_out ? nullptr : s_in, nst),
                       flat(lengths, B * 4)};
    const View out[] = {rows(y, a.sy, B, L, D, es), flat(s_out, nst), flat(workspace, (int64_t)need)};
    if (clash(in, out)) return LA_ERR_ALIAS;
    if ((st = check_trace(s->trace)) != LA_OK) return st;
    la::Tracer tr = make_tracer(s->trace, s->stream);
    a.u = u; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dskip = Dskip; a.z = z; a.dt_bias = dt_bias; a.s_in = s_in;
    a.lengths = lengths; a.y = y; a.s_out = s_out; a.ws = workspace;
    a.tr = &tr;
    return from_hip(la::launch_ssm_scan(a));
}

la_status la_ssm_scan_bwd(const void* u, const void* dt, const float* A, const void* Bm, const void* Cm,
                          const float* Dskip, const void* z, const float* dt_bias, const float* s_in,
                          const int32_t* lengths, const void* dy, const float* ds_out, void* du, void* ddt, float* dA,
                          void* dB, void* dC, float* dD, void* dz, float* d_dt_bias, float* ds_in, void* workspace,
                          uint64_t workspace_bytes, const la_ssm_shape* s) {
    la_status st = ssm_shape(s, false);
    if (st != LA_OK) return st;
    const int64_t B = s->B, L = s->L, D = s->D, N = s->N, nst = B * N * D * 4;
    if (B * L * D > 0 && (!u || !dt || !Bm || !Cm || !dy || !du || !ddt || (z && !dz))) return LA_ERR_NULL;
    if (B * L > 0 && (!dB || !dC)) return LA_ERR_NULL;
    if (D > 0 && (!A || !dA)) return LA_ERR_NULL;
    for (const la_rows& r : {s->u, s->dt, s->b, s->c, s->z, s->dy, s->du, s->ddt, s->db, s->dc, s->dz})
        if (!rows_ok(s, r, s->L)) return LA_ERR_SHAPE;
    const size_t need = la::ssm_bwd_ws(B, L, D, s->N);
    if (ws_bad(workspace, workspace_bytes, need)) return LA_ERR_WORKSPACE;
    la::SsmArgs a = ssm_args(s, L);
    const size_t es = esize(s->dtype);
    const View in[] = {rows(u, a.su, B, L, D, es), rows(dt, a.sdt, B, L, D, es), flat(A, D * N * 4),
                       rows(Bm, a.sb, B, L, N, es), rows(Cm, a.sc, B, L, N, es), flat(Dskip, D * 4),
                       rows(z, a.sz, B, L, D, es), flat(dt_bias, D * 4), flat(s_in, nst), flat(lengths, B * 4),
                       rows(dy, a.sdy, B, L, D, es), flat(ds_out, nst)};
    const View out[] = {rows(du, a.sdu, B, L, D, es), rows(ddt, a.sddt, B, L, D, es), flat(dA, D * N * 4),
                        rows(dB, a.sdb, B, L, N, es), rows(dC, a.sdc, B, L, N, es), flat(dD, D * 4),
                        rows(z ? dz : nullptr, a.sdz, B, L, D, es), flat(d_dt_bias, D * 4), flat(ds_in, nst),
                        flat(workspace, (int64_t)need)};
    if (clash(in, out)) return LA_ERR_ALIAS;
    if ((st = check_trace(s->trace)) != LA_OK) return st;
    la::Tracer tr = make_tracer(s->trace, s->stream);
    a.u = u; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dskip = Dskip; a.z = z; a.dt_bias = dt_bias; a.s_in = s_in;
    a.lengths = lengths; a.dy = dy; a.ds_out = ds_out; a.du = du; a.ddt = ddt; a.dA = dA; a.dB = dB; a.dC = dC; a.dD = dD;
    a.dz = dz; a.d_dt_bias = d_dt_bias; a.ds_in = ds_in; a.ws = workspace;
    a.tr = &tr;
    return from_hip(la::launch_ssm_scan_bwd(a));
}

la_status la_ssm_step(const void* u, const void* dt, const float* A, const void* Bm, const void* Cm, const float* Dskip,
                      const void* z, const float* dt_bias, float* state, const int32_t* slots, void* y,
                      const la_ssm_shape* s) {
    la_status st = ssm_shape(s, true);
    if (st != LA_OK) return st;
    if (!slots && s->nslots < s->B) return LA_ERR_SHAPE;
    const int64_t B = s->B, D = s->D, N = s->N;
    if (B * D > 0 && (!u || !dt || !A || !Bm || !Cm || !y || (!state && s->nslots > 0))) return LA_ERR_NULL;
    for (const la_rows& r : {s->u, s->dt, s->b, s->c, s->z, s->y})
        if (!rows_ok(s, r, 1)) return LA_ERR_SHAPE;
    la::SsmArgs a = ssm_args(s, 1);
    const size_t es = esize(s->dtype);
    const View in[] = {rows(u, a.su, B, 1, D, es), rows(dt, a.sdt, B, 1, D, es), flat(A, D * N * 4),
                       rows(Bm, a.sb, B, 1, N, es), rows(Cm, a.sc, B, 1, N, es), flat(Dskip, D * 4),
                       rows(z, a.sz, B, 1, D, es), flat(dt_bias, D * 4), flat(slots, B * 4)};
    const View out[] = {rows(y, a.sy, B, 1, D, es), flat(state, s->nslots * N * D * 4)};
    if (clash(in, out)) return LA_ERR_ALIAS;
    if ((st = check_trace(s->trace)) != LA_OK) return st;
    la::Tracer tr = make_tracer(s->trace, s->stream);
    a.u = u; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dskip = Dskip; a.z = z; a.dt_bias = dt_bias; a.state = state;
    a.slots = slots; a.y = y;
    a.tr = &tr;
    return from_hip(la::launch_ssm_step(a));
}

la_status la_add_norm(const void* x, const void* residual, const float* weight, void* y, void* h, float* rstd,
                      const la_norm_shape* s) {
    return norm_fwd(x, residual, weight, y, nullptr, nullptr, h, rstd, s, false);
}

la_status la_add_norm_q8(const void* x, const void* residual, const float* weight, void* q, float* scale, void* h,
                         float* rstd, const la_norm_shape* s) {
    return norm_fwd(x, residual, weight, nullptr, (uint8_t*)q, scale, h, rstd, s, true);
}

int64_t la_add_norm_bwd_workspace(const la_norm_shape* s) {
    const la_status st = norm_shape(s);
    if (st != LA_OK) return st;
    return (int64_t)la::add_norm_bwd_ws(s->M, s->D);
}

la_status la_add_norm_bwd(const void* dy, const void* h, const float* weight, const float* rstd, const void* dh, void* dx,
                          float* d_weight, void* workspace, uint64_t workspace_bytes, const la_norm_shape* s) {
    la_status st = norm_shape(s);
    if (st != LA_OK) return st;
    if (!weight || !d_weight || (s->M > 0 && (!dy || !h || !rstd || !dx))) return LA_ERR_NULL;
    const size_t need = la::add_norm_bwd_ws(s->M, s->D);
    if (ws_bad(workspace, workspace_bytes, need)) return LA_ERR_WORKSPACE;
    la::NormArgs a = norm_args(s);
    const size_t es = esize(s->dtype);
    const View vdy = mat(dy, s->M, a.sdy, s->D, es), vdh = mat(dh, s->M, a.sdh, s->D, es);
    const View vdx = mat(dx, s->M, a.sdx, s->D, es);
    const View in[] = {mat(h, s->M, a.sh, s->D, es), flat(weight, s->D * 4), flat(rstd, s->M * 4), vdy, vdh};
    const View out[] = {flat(d_weight, s->D * 4), flat(workspace, (int64_t)need)};
    if (clash(in, out)) return LA_ERR_ALIAS;
    if (self_overlap(vdx) || clash_inplace(vdx, vdy) || clash_inplace(vdx, vdh)) return LA_ERR_ALIAS;
    for (const View& v : {in[0], in[1], in[2], out[0], out[1]})
        if (overlap(vdx, v)) return LA_ERR_ALIAS;
    if ((st = check_trace(s->trace)) != LA_OK) return st;
    la::Tracer tr = make_tracer(s->trace, s->stream);
    a.dy = dy; a.h_in = h; a.weight = weight; a.rstd_in = rstd; a.dh = dh; a.dx = dx; a.d_weight = d_weight; a.ws = workspace;
    a.tr = &tr;
    return from_hip(la::launch_add_norm_bwd(a));
}

}  // extern "C"
