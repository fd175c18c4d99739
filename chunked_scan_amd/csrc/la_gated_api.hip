// la_gated_api.hip -- the C ABI of the gated recurrent layer (declared in include/la_chunk.h): the gated recurrence, the norms
// around a block, dropout.  Validation as in la_mixer_api.hip: everything on the host before the first HIP call, in
// the order shape pointer, sizes, limits, dtype, required pointers, strides, workspace, aliasing.
#include <math.h>
#include <stdint.h>

#include "la_chunk.h"
#include "la_internal.h"
#include "la_mixer.h"
#include "la_views.h"

using namespace la::api;

namespace {

// ---------------------------------------------------------------- recurrence

la_status gated_shape(const la_gated_shape* s, bool step) {
    if (!s) return LA_ERR_NULL;
    const la_status st = sizes_ok(s, step ? 1 : s->L);
    if (st != LA_OK) return st;
    if (!(s->c > 0.f) || !isfinite(s->c) || s->reserved != 0 || (step && s->nslots < 0)) return LA_ERR_SHAPE;
    if (step && mul(s->nslots, s->D) > kMaxElems) return LA_ERR_UNSUPPORTED;
    if (!dtype_ok(s->dtype)) return LA_ERR_DTYPE;
    return LA_OK;
}

la::GatedArgs gated_args(const la_gated_shape* s, int64_t L) {
    la::GatedArgs a = {};
    a.B = s->B; a.L = L; a.D = s->D; a.c = s->c; a.bf16 = s->dtype == LA_BF16; a.nslots = s->nslots;
    a.sx = resolve(s->x, L, s->D); a.sr = resolve(s->r, L, s->D); a.si = resolve(s->i, L, s->D);
    a.sz = resolve(s->z, L, s->D); a.sy = resolve(s->y, L, s->D); a.sdy = resolve(s->dy, L, s->D);
    a.sdx = resolve(s->dx, L, s->D); a.sdr = resolve(s->dr, L, s->D); a.sdi = resolve(s->di, L, s->D);
    a.sdz = resolve(s->dz, L, s->D);
    a.stream = (hipStream_t)s->stream;
    return a;
}
int64_t block_bytes(const la_gated_shape* s) {
    return s->B * ((s->L + LA_GATED_BLOCK - 1) / LA_GATED_BLOCK) * s->D * 4;
}

// ---------------------------------------------------------------- norms and dropout

la_status block_shape(const la_block_shape* s, bool dropout) {
    if (!s) return LA_ERR_NULL;
    if (s->M < 0 || s->D < 1) return LA_ERR_SHAPE;
    if (!(s->p >= 0.f && s->p <= 1.f - 0x1p-16f)) return LA_ERR_SHAPE;
    if (!dropout && (!(s->eps > 0.f) || !isfinite(s->eps))) return LA_ERR_SHAPE;
    if ((!dropout && s->D > 16384) || s->M > kMaxNormRows || s->D > kMaxNormElems || mul(s->M, s->D) > kMaxNormElems)
        return LA_ERR_UNSUPPORTED;
    if (!dropout && (s->act < LA_GATE_LINEAR || s->act > LA_GATE_SILU)) return LA_ERR_UNSUPPORTED;
    if (!dtype_ok(s->dtype)) return LA_ERR_DTYPE;
    for (int64_t st : {s->x_stride, s->gate_stride, s->residual_stride, s->y_stride, s->h_stride, s->dy_stride, s->dh_stride,
                       s->dx_stride, s->dgate_stride, s->dresidual_stride})
        if (st < 0 || st > kMaxSpan || mul(s->M, st) > kMaxSpan) return LA_ERR_SHAPE;
    return LA_OK;
}

la::BlockArgs block_args(const la_block_shape* s) {
    la::BlockArgs a = {};
    auto st = [&](int64_t v) { return v ? v : s->D; };
    a.M = s->M; a.D = s->D; a.act = s->act; a.eps = s->eps; a.bf16 = s->dtype == LA_BF16;
    a.drop = (unsigned)(s->p * 65536.f + 0.5f);
    a.sx = st(s->x_stride); a.sg = st(s->gate_stride); a.sres = st(s->residual_stride); a.sy = st(s->y_stride);
    a.sh = st(s->h_stride); a.sdy = st(s->dy_stride); a.sdh = st(s->dh_stride); a.sdx = st(s->dx_stride);
    a.sdg = st(s->dgate_stride); a.sdres = st(s->dresidual_stride);
    a.stream = (hipStream_t)s->stream;
    return a;
}
la_status rng_ok(const la::BlockArgs& a, const uint64_t* rng) {
    if (a.M == 0 || a.drop == 0) return LA_OK;
    return !rng ? LA_ERR_NULL : (uintptr_t)rng % 8 != 0 ? LA_ERR_SHAPE : LA_OK;
}
View rng_view(const la::BlockArgs& a, const uint64_t* rng) { return flat(a.drop > 0 ? rng : nullptr, 16); }

}  // namespace

extern "C" {

int64_t la_gated_scan_workspace(const la_gated_shape* s, int32_t backward) {
    const la_status st = gated_shape(s, false);
    if (st != LA_OK) return st;
    if (backward < 0 || backward > 2) return LA_ERR_UNSUPPORTED;
    return (int64_t)(backward ? la::gated_bwd_ws(s->B, s->L, s->D, backward == 2) : la::gated_fwd_ws(s->B, s->L, s->D));
}

la_status la_gated_scan(const void* x, const void* r, const void* i, const float* lam, const float* r_bias,
                        const float* i_bias, const void* z, const float* h_in, const int32_t* lengths, void* y,
                        float* h_out, float* h_blocks, void* workspace, uint64_t workspace_bytes,
                        const la_gated_shape* s) {
    la_status st = gated_shape(s, false);
    if (st != LA_OK) return st;
    const int64_t B = s->B, L = s->L, D = s->D, nst = B * D * 4;
    if (B * L * D > 0 && (!x || !r || !i || !y)) return LA_ERR_NULL;
    if (B * D > 0 && !lam) return LA_ERR_NULL;
    for (const la_rows& v : {s->x, s->r, s->i, s->z, s->y})
        if (!rows_ok(s, v, L)) return LA_ERR_SHAPE;
    const size_t need = la::gated_fwd_ws(B, L, D);
    if (ws_bad(workspace, workspace_bytes, need)) return LA_ERR_WORKSPACE;
    la::GatedArgs a = gated_args(s, L);
    const size_t es = esize(s->dtype);
    const View in[] = {rows(x, a.sx, B, L, D, es), rows(r, a.sr, B, L, D, es), rows(i, a.si, B, L, D, es), flat(lam, D * 4),
                       flat(r_bias, D * 4), flat(i_bias, D * 4), rows(z, a.sz, B, L, D, es),
                       flat(h_in == h_out ? nullptr : h_in, nst), flat(lengths, B * 4)};
    const View out[] = {rows(y, a.sy, B, L, D, es), flat(h_out, nst), flat(h_blocks, block_bytes(s)),
                        flat(workspace, (int64_t)need)};
    if (clash(in, out)) return LA_ERR_ALIAS;
    if ((st = check_trace(s->trace)) != LA_OK) return st;
    la::Tracer tr = make_tracer(s->trace, s->stream);
    a.x = x; a.r = r; a.i = i; a.lam = lam; a.r_bias = r_bias; a.i_bias = i_bias; a.z = z; a.h_in = h_in;
    a.lengths = lengths; a.y = y; a.h_out = h_out; a.blocks = h_blocks; a.ws = workspace;
    a.tr = &tr;
    return from_hip(la::launch_gated_scan(a));
}

la_status la_gated_scan_bwd(const void* x, const void* r, const void* i, const float* lam, const float* r_bias,
                            const float* i_bias, const void* z, const float* h_in, const int32_t* lengths,
                            const float* h_blocks, const void* dy, const float* dh_out, void* dx, void* dr, void* di,
                            float* dlam, float* dr_bias, float* di_bias, void* dz, float* dh_in, void* workspace,
                            uint64_t workspace_bytes, const la_gated_shape* s) {
    la_status st = gated_shape(s, false);
    if (st != LA_OK) return st;
    const int64_t B = s->B, L = s->L, D = s->D, nst = B * D * 4;
    if (B * L * D > 0 && (!x || !r || !i || !dy || !dx || !dr || !di || (z && !dz))) return LA_ERR_NULL;
    if (D > 0 && (!lam || !dlam)) return LA_ERR_NULL;
    for (const la_rows& v : {s->x, s->r, s->i, s->z, s->dy, s->dx, s->dr, s->di, s->dz})
        if (!rows_ok(s, v, L)) return LA_ERR_SHAPE;
    const size_t need = la::gated_bwd_ws(B, L, D, h_blocks != nullptr);
    if (ws_bad(workspace, workspace_bytes, need)) return LA_ERR_WORKSPACE;
    la::GatedArgs a = gated_args(s, L);
    const size_t es = esize(s->dtype);
    const View in[] = {rows(x, a.sx, B, L, D, es), rows(r, a.sr, B, L, D, es), rows(i, a.si, B, L, D, es), flat(lam, D * 4),
                       flat(r_bias, D * 4), flat(i_bias, D * 4), rows(z, a.sz, B, L, D, es), flat(h_in, nst),
                       flat(lengths, B * 4), flat(h_blocks, block_bytes(s)), rows(dy, a.sdy, B, L, D, es),
                       flat(dh_out, nst)};
    const View out[] = {rows(dx, a.sdx, B, L, D, es), rows(dr, a.sdr, B, L, D, es), rows(di, a.sdi, B, L, D, es),
                        flat(dlam, D * 4), flat(dr_bias, D * 4), flat(di_bias, D * 4),
                        rows(z ? dz : nullptr, a.sdz, B, L, D, es), flat(dh_in, nst), flat(workspace, (int64_t)need)};
    if (clash(in, out)) return LA_ERR_ALIAS;
    if ((st = check_trace(s->trace)) != LA_OK) return st;
    la::Tracer tr = make_tracer(s->trace, s->stream);
    a.x = x; a.r = r; a.i = i; a.lam = lam; a.r_bias = r_bias; a.i_bias = i_bias; a.z = z; a.h_in = h_in;
    a.lengths = lengths; a.blocks_in = h_blocks; a.dy = dy; a.dh_out = dh_out; a.dx = dx; a.dr = dr; a.di = di;
    a.dlam = dlam; a.dr_bias = dr_bias; a.di_bias = di_bias; a.dz = dz; a.dh_in = dh_in; a.ws = workspace;
    a.tr = &tr;
    return from_hip(la::launch_gated_scan_bwd(a));
}

la_status la_gated_step(const void* x, const void* r, const void* i, const float* lam, const float* r_bias,
                        const float* i_bias, const void* z, float* state, const int32_t* slots, void* y,
                        const la_gated_shape* s) {
    la_status st = gated_shape(s, true);
    if (st != LA_OK) return st;
    if (!slots && s->nslots < s->B) return LA_ERR_SHAPE;
    const int64_t B = s->B, D = s->D;
    if (B * D > 0 && (!x || !r || !i || !lam || !y || (!state && s->nslots > 0))) return LA_ERR_NULL;
    for (const la_rows& v : {s->x, s->r, s->i, s->z, s->y})
        if (!rows_ok(s, v, 1)) return LA_ERR_SHAPE;
    la::GatedArgs a = gated_args(s, 1);
    const size_t es = esize(s->dtype);
    const View in[] = {rows(x, a.sx, B, 1, D, es), rows(r, a.sr, B, 1, D, es), rows(i, a.si, B, 1, D, es), flat(lam, D * 4),
                       flat(r_bias, D * 4), flat(i_bias, D * 4), rows(z, a.sz, B, 1, D, es), flat(slots, B * 4)};
    const View out[] = {rows(y, a.sy, B, 1, D, es), flat(state, s->nslots * D * 4)};
    if (clash(in, out)) return LA_ERR_ALIAS;
    if ((st = check_trace(s->trace)) != LA_OK) return st;
    la::Tracer tr = make_tracer(s->trace, s->stream);
    a.x = x; a.r = r; a.i = i; a.lam = lam; a.r_bias = r_bias; a.i_bias = i_bias; a.z = z; a.state = state; a.slots = slots;
    a.y = y;
    a.tr = &tr;
    return from_hip(la::launch_gated_step(a));
}

la_status la_block_norm(const void* x, const void* gate, const void* residual, const float* w_post, const float* scale,
                        const float* w_pre, const uint64_t* rng, void* y, void* h, float* rstd_post, float* rstd_pre,
                        const la_block_shape* s) {
    la_status st = block_shape(s, false);
    if (st != LA_OK) return st;
    la::BlockArgs a = block_args(s);
    if (s->M > 0 && (!x || !h || (w_pre && !y))) return LA_ERR_NULL;
    if ((st = rng_ok(a, rng)) != LA_OK) return st;
    if (!w_pre) y = nullptr, rstd_pre = nullptr;
    if (!w_post) rstd_post = nullptr;
    const size_t es = esize(s->dtype);
    const int64_t M = s->M, D = s->D;
    const View vx = mat(x, M, a.sx, D, es), vr = mat(residual, M, a.sres, D, es), vh = mat(h, M, a.sh, D, es);
    const View in[] = {vx, vr, mat(gate, M, a.sg, D, es), flat(w_post, D * 4), flat(scale, D * 4), flat(w_pre, D * 4),
                       rng_view(a, rng)};
    const View out[] = {mat(y, M, a.sy, D, es), flat(rstd_post, M * 4), flat(rstd_pre, M * 4)};
    if (clash(in, out)) return LA_ERR_ALIAS;
    if (self_overlap(vh) || clash_inplace(vh, vx) || clash_inplace(vh, vr)) return LA_ERR_ALIAS;
    for (const View& v : {in[2], in[3], in[4], in[5], in[6], out[0], out[1], out[2]})
        if (overlap(vh, v)) return LA_ERR_ALIAS;
    if ((st = check_trace(s->trace)) != LA_OK) return st;
    la::Tracer tr = make_tracer(s->trace, s->stream);
    a.x = x; a.gate = gate; a.residual = residual; a.w_post = w_post; a.scale = scale; a.w_pre = w_pre; a.rng = rng; a.y = y;
    a.h = h; a.rstd_post = rstd_post; a.rstd_pre = rstd_pre;
    a.tr = &tr;
    return from_hip(la::launch_block_norm(a));
}

int64_t la_block_norm_bwd_workspace(const la_block_shape* s) {
    const la_status st = block_shape(s, false);
    if (st != LA_OK) return st;
    return (int64_t)la::block_norm_bwd_ws(s->M, s->D);
}

la_status la_block_norm_bwd(const void* x, const void* gate, const void* h, const float* w_post, const float* scale,
                            const float* w_pre, const uint64_t* rng, const float* rstd_post, const float* rstd_pre,
                            const void* dy, const void* dh, void* dx, void* dgate, void* dresidual, float* dw_post,
                            float* dscale, float* dw_pre, void* workspace, uint64_t workspace_bytes,
                            const la_block_shape* s) {
    la_status st = block_shape(s, false);
    if (st != LA_OK) return st;
    la::BlockArgs a = block_args(s);
    if (!w_pre) dy = nullptr, h = nullptr, rstd_pre = nullptr, dw_pre = nullptr;
    if (!w_post) rstd_post = nullptr, dw_post = nullptr;
    if (!scale) dscale = nullptr;
    if (!gate) dgate = nullptr;
    if ((w_post && !dw_post) || (scale && !dscale) || (w_pre && !dw_pre)) return LA_ERR_NULL;
    if (s->M > 0 && (!x || !dx || (gate && !dgate) || (w_post && !rstd_post) || (w_pre && (!dy || !h || !rstd_pre))))
        return LA_ERR_NULL;
    if ((st = rng_ok(a, rng)) != LA_OK) return st;
    const size_t need = la::block_norm_bwd_ws(s->M, s->D);
    if (ws_bad(workspace, workspace_bytes, need)) return LA_ERR_WORKSPACE;
    const size_t es = esize(s->dtype);
    const int64_t M = s->M, D = s->D;
    const View vdy = mat(dy, M, a.sdy, D, es), vdh = mat(dh, M, a.sdh, D, es), vdr = mat(dresidual, M, a.sdres, D, es);
    const View in[] = {mat(x, M, a.sx, D, es), mat(gate, M, a.sg, D, es), mat(h, M, a.sh, D, es), flat(w_post, D * 4),
                       flat(scale, D * 4), flat(w_pre, D * 4), rng_view(a, rng), flat(rstd_post, M * 4),
                       flat(rstd_pre, M * 4), vdy, vdh};
    const View out[] = {mat(dx, M, a.sdx, D, es), mat(dgate, M, a.sdg, D, es), flat(dw_post, D * 4), flat(dscale, D * 4),
                        flat(dw_pre, D * 4), flat(workspace, (int64_t)need)};
    if (clash(in, out)) return LA_ERR_ALIAS;
    if (self_overlap(vdr) || clash_inplace(vdr, vdy) || clash_inplace(vdr, vdh)) return LA_ERR_ALIAS;
    for (int k = 0; k < 9; k++)
        if (overlap(vdr, in[k])) return LA_ERR_ALIAS;
    for (const View& v : out)
        if (overlap(vdr, v)) return LA_ERR_ALIAS;
    if ((st = check_trace(s->trace)) != LA_OK) return st;
    la::Tracer tr = make_tracer(s->trace, s->stream);
    a.x = x; a.gate = gate; a.h_in = h; a.w_post = w_post; a.scale = scale; a.w_pre = w_pre; a.rng = rng;
    a.rstd_post_in = rstd_post; a.rstd_pre_in = rstd_pre; a.dy = dy; a.dh = dh; a.dx = dx; a.dgate = dgate;
    a.dres = dresidual; a.dw_post = dw_post; a.dscale = dscale; a.dw_pre = dw_pre; a.ws = workspace;
    a.tr = &tr;
    return from_hip(la::launch_block_norm_bwd(a));
}

la_status la_dropout(const void* x, const void* residual, const uint64_t* rng, void* y, const la_block_shape* s) {
    la_status st = block_shape(s, true);
    if (st != LA_OK) return st;
    la::BlockArgs a = block_args(s);
    if (s->M > 0 && (!x || !y)) return LA_ERR_NULL;
    if ((st = rng_ok(a, rng)) != LA_OK) return st;
    const size_t es = esize(s->dtype);
    const View vx = mat(x, s->M, a.sx, s->D, es), vr = mat(residual, s->M, a.sres, s->D, es), vy = mat(y, s->M, a.sy, s->D, es);
    if (self_overlap(vy) || clash_inplace(vy, vx) || clash_inplace(vy, vr) || overlap(vy, rng_view(a, rng))) return LA_ERR_ALIAS;
    if ((st = check_trace(s->trace)) != LA_OK) return st;
    la::Tracer tr = make_tracer(s->trace, s->stream);
    a.x = x; a.residual = residual; a.rng = rng; a.y = y;
    a.tr = &tr;
    return from_hip(la::launch_dropout(a));
}

}  // extern "C"
