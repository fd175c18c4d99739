"""The gated recurrence, the norms around a block and dropout on the GPU against their fp64 forms (gated_ref.py, whose
bounds on the roundings are the tolerances, with half a step of the stored type), at the sizes, strides and masks where
they can go wrong."""
import numpy as np
import pytest
import torch

import gated_ref as G
import mixer_ref as R
from chunked_scan_amd import binding as la
from gpu_util import note
from test_gpu_mixer import BF, F32, SENTINEL, Draw, check_tail, cut, ints, nan_tail

pytestmark = pytest.mark.gpu


def keep3(n, B, L):
    return torch.from_numpy(G.keep_of(n, B, L)[..., None]).cuda()


def nonan(t):
    return None if t is None else np.nan_to_num(R.f64(t))


# ------------------------------------------------------------------------------------ recurrence

SCAN = [  # B, L, D, lengths, strided, z, biases, h_in, lam's middle
    (1, 1, 64, None, False, True, True, False, -5.0),
    (2, 9, 64, [9, 4], False, True, True, True, -5.0),
    (3, 67, 40, [67, 0, 1], False, False, True, True, -5.0),
    (1, 63, 3, None, False, True, False, True, -4.0),
    (2, 64, 130, [64, 63], True, True, True, False, -5.0),
    (2, 65, 256, None, False, True, True, True, -5.0),
    (1, 200, 258, None, True, False, True, True, -6.0),
    (2, 333, 65, [300, 17], True, True, False, True, -4.0),
    (2, 129, 520, [130, -2], False, True, True, True, -5.0),
    (1, 0, 32, None, False, True, True, True, -5.0),
    (3, 0, 8, [0, 0, 0], False, False, True, True, -5.0),
    (1, 517, 64, None, False, True, True, True, -2.0),
    (2, 260, 72, [64, 128], False, True, True, True, 2.0),     # strong decay; ends on a block's end
    (1, 1500, 7, [1499], False, False, True, True, -12.0),     # hardly any decay
    (4, 700, 1024, [700, 640, 1, 0], False, True, True, True, -5.0),
]


def scan_inputs(case, dtype, seed):
    B, L, D, lengths, strided, z, biases, h_in, mid = case
    g = Draw(seed)
    make = g.wide if strided else g.normal
    a = dict(x=make(B, L, D, dtype=dtype))
    ri = g.normal(B, L, 2 * D + 3, dtype=dtype)  # an odd pitch: rows at every alignment
    a["r"], a["i"] = (ri[..., :D], ri[..., D + 3 :]) if strided else (ri[..., :D].contiguous(), ri[..., D + 3 :].contiguous())
    a["lam"] = mid + g.normal(D, std=0.7)
    a["rb"], a["ib"] = (g.normal(D), g.normal(D)) if biases else (None, None)
    a["z"] = make(B, L, D, dtype=dtype) if z else None
    a["h_in"] = g.normal(B, D) if h_in else None
    a["dy"], a["dh_out"] = make(B, L, D, dtype=dtype), g.normal(B, D)
    n = cut(lengths, L)
    for k in ("x", "r", "i", "z", "dy"):
        if a[k] is not None:
            nan_tail(a[k], n)
    return a, n


def scan_kw(a, lengths):
    return dict(r_bias=a["rb"], i_bias=a["ib"], z=a["z"], h_in=a["h_in"], lengths=ints(lengths))


def scan_ref(a, n, c):
    return [nonan(a[k]) for k in ("x", "r", "i", "lam", "rb", "ib", "z", "h_in")] + [n, c]


GRADS = ("dx", "dr", "di", "dlam", "dr_bias", "di_bias", "dz", "dh_in")


def check_grads(got, ref, dtype, n):
    for name, t, r in zip(GRADS, got, ref):
        assert (t is None) == (r is None), name
        if t is None:
            continue
        if t.dim() == 3:
            check_tail(t, n, 0.0, name)
        G.close(t, *r, dtype if t.dim() == 3 else F32, name)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", SCAN, ids=str)
def test_scan_forward_and_backward(case, dtype):
    B, L, D, lengths, strided, z, biases, h_in, mid = case
    note(f"gated scan {case} {dtype}")
    c = 8.0 if mid < 0 else 3.0
    a, n = scan_inputs(case, dtype, 200 + L)
    kw = scan_kw(a, lengths)
    args = [a[k] for k in ("x", "r", "i", "lam")]
    wide = torch.full((B, L, D + 16), SENTINEL, dtype=dtype, device="cuda")
    y = wide[..., 8 : 8 + D] if strided else wide[..., :D].contiguous()
    nb = -(-L // 64)
    blocks = torch.full((B, nb, D), SENTINEL, device="cuda")
    got, h, blk = la.la_gated_scan(*args, c=c, y=y, h_blocks=blocks, **kw)
    ry, rh, (rb, eb), _ = G.scan(*scan_ref(a, n, c))
    check_tail(got, n, SENTINEL, "y")
    if strided:
        assert (wide[..., :8] == SENTINEL).all() and (wide[..., 8 + D :] == SENTINEL).all()
    G.close(torch.where(keep3(n, B, L), got, torch.zeros_like(got)), *ry, dtype, "y")
    G.close(h, *rh, F32, "h_out")
    none = torch.from_numpy(np.isnan(rb)).cuda()
    assert (blk[none] == SENTINEL).all()
    G.close(torch.where(none, torch.zeros_like(blk), blk), np.nan_to_num(rb), np.nan_to_num(eb), F32, "h_blocks")
    if h_in:  # the state written over the incoming one
        s = a["h_in"].clone()
        _, h2, none_ = la.la_gated_scan(*args, c=c, h_out=s, **dict(kw, h_in=s))
        assert none_ is None and h2.data_ptr() == s.data_ptr() and torch.equal(s, h)

    ref = G.scan_bwd(*scan_ref(a, n, c), nonan(a["dy"]), R.f64(a["dh_out"]))
    ref = [None if (k in ("dr_bias", "di_bias") and not biases) or (k == "dh_in" and not h_in) else v
           for k, v in zip(GRADS, ref)]
    once = la.la_gated_scan_bwd(*args, a["dy"], dh_out=a["dh_out"], h_blocks=blk, c=c, **kw)
    check_grads(once, ref, dtype, n)
    again = la.la_gated_scan_bwd(*args, a["dy"], dh_out=a["dh_out"], c=c, **kw)  # the states made again
    for s, t in zip(once, again):
        assert (s is None) == (t is None) and (s is None or torch.equal(s, t))


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,D,S,slots,z", [(1, 64, 1, None, True), (3, 40, 5, [4, 0, 2], False), (4, 70, 4, [1, -1, 9, 3], True),
                                           (5, 1030, 6, [2, 5, 2, 0, 5], True), (2, 3, 2, None, False), (2, 2048, 2, [1, 0], True)])
def test_step(B, D, S, slots, z, dtype):
    note(f"gated step {B} {D} {S} {slots} {dtype}")
    a, _ = scan_inputs((B, 1, D, None, True, z, True, False, -5.0), dtype, 7)
    one = {k: (v[:, 0] if v is not None and v.dim() == 3 else v) for k, v in a.items()}
    state = Draw(8).normal(S, D)
    before = state.clone()
    y = torch.full((B, D), SENTINEL, dtype=dtype, device="cuda")
    la.la_gated_step(one["x"], one["r"], one["i"], a["lam"], state, r_bias=a["rb"], i_bias=a["ib"], z=one["z"],
                     slots=ints(slots), y=y)
    seen = set()
    for b, s in enumerate(range(B) if slots is None else slots):
        if s < 0 or s >= S or s in seen:
            assert (y[b] == SENTINEL).all()
            continue
        seen.add(s)
        ref = [None if v is None else (v[b : b + 1] if v.ndim == 3 else v) for v in scan_ref(a, None, 8.0)[:7]]
        ry, rh, _, _ = G.scan(*ref, R.f64(before[s])[None], None, 8.0)
        G.close(y[b], ry[0][0, 0], ry[1][0, 0], dtype, "y")
        G.close(state[s], rh[0][0], rh[1][0], F32, "state")
    for s in set(range(S)) - seen:
        assert torch.equal(state[s], before[s])


def test_steps_equal_a_scan():
    note("gated steps against a scan")
    a, _ = scan_inputs((3, 70, 96, None, False, True, True, True, -5.0), F32, 17)
    y, h, _ = la.la_gated_scan(a["x"], a["r"], a["i"], a["lam"], **scan_kw(a, None))
    state = a["h_in"].clone()
    for t in range(70):
        o = la.la_gated_step(a["x"][:, t], a["r"][:, t], a["i"][:, t], a["lam"], state, r_bias=a["rb"], i_bias=a["ib"],
                             z=a["z"][:, t])
        # the same operations in another order: each state's bound twice, about 4 roundings a token at most
        assert (o - y[:, t]).abs().max() <= 2 * 4 * 70 * 2.0 ** -24 * y.abs().max()
    assert (state - h).abs().max() <= 2 * 4 * 70 * 2.0 ** -24 * h.abs().max()


def test_scan_backward_against_differences():
    """Central differences of the forward on the GPU in every argument, along random directions."""
    note("gated scan differences")
    a, _ = scan_inputs((2, 150, 40, [150, 77], False, True, True, True, -4.0), F32, 23)
    lengths = [150, 77]
    for k in ("x", "r", "i", "z", "dy"):
        a[k] = torch.nan_to_num(a[k])
    g = Draw(24)

    def loss(b):
        y = torch.zeros(2, 150, 40, device="cuda")
        y, h, _ = la.la_gated_scan(b["x"], b["r"], b["i"], b["lam"], y=y, **scan_kw(b, lengths))
        return float((y.double() * a["dy"].double()).sum() + (h.double() * a["dh_out"].double()).sum())

    grads = dict(zip(("x", "r", "i", "lam", "rb", "ib", "z", "h_in"),
                     la.la_gated_scan_bwd(a["x"], a["r"], a["i"], a["lam"], a["dy"], dh_out=a["dh_out"], **scan_kw(a, lengths))))
    for k, gr in grads.items():
        v, e = g.normal(*a[k].shape), 1e-2
        up, dn = (loss(dict(a, **{k: a[k] + s * e * v})) for s in (1, -1))
        diff = (up - dn) / (2 * e)
        want = float((gr.double() * v.double()).sum())
        scale = float((gr.double().abs() * v.double().abs()).sum())
        # e^2 of the third derivatives, and the loss's fp32 roundings over e
        assert abs(diff - want) <= 1e-2 * scale / np.sqrt(v.numel()) + 1e-3 * scale, (k, diff, want, scale)


def test_gradient_slices_and_held_states():
    """Gradients into slices of wide buffers touch nothing beside them; r = -infinity holds the state."""
    note("gated gradient slices")
    a, n = scan_inputs((2, 75, 72, [75, 20], False, True, True, True, -5.0), BF, 31)
    args = [a[k] for k in ("x", "r", "i", "lam", "dy")]
    kw = dict(scan_kw(a, n), dh_out=a["dh_out"])
    ref = la.la_gated_scan_bwd(*args, **kw)
    B, L, D = 2, 75, 72
    uz = torch.full((B, L, 2 * D + 8), SENTINEL, dtype=BF, device="cuda")
    ri = torch.full((B, L, 2 * D + 8), SENTINEL, dtype=BF, device="cuda")
    got = la.la_gated_scan_bwd(*args, **kw, dx=uz[..., :D], dz=uz[..., D : 2 * D], dr=ri[..., :D], di=ri[..., D : 2 * D])
    for s, t in zip(ref, got):
        assert torch.equal(s, t)
    assert (uz[..., 2 * D :] == SENTINEL).all() and (ri[..., 2 * D :] == SENTINEL).all()

    a["r"][:, 10:12] = float("-inf")
    x, r, i, lam, dy = args
    y, h, _ = la.la_gated_scan(x, r, i, lam, **dict(scan_kw(a, n), z=None))
    assert torch.equal(y[:, 10], y[:, 9]) and torch.equal(y[:, 11], y[:, 9])
    got = la.la_gated_scan_bwd(x, r, i, lam, dy, **dict(kw, z=None))
    assert (got[0][:, 10:12] == 0).all() and (got[1][:, 10:12] == 0).all() and (got[2][:, 10:12] == 0).all()
    for t in got:
        assert t is None or torch.isfinite(t).all()


# ------------------------------------------------------------------------------------ norms around a block

BLOCK = [(1, 8), (3, 64), (5, 1000), (2, 7), (4, 130), (9, 2048), (2, 2056), (3, 4096), (1, 8200), (2, 16384), (700, 96),
         (0, 64), (2, 1), (1030, 40), (6, 5000)]


def block_inputs(M, D, dtype, seed, act="silu", post=True, pre=True, scale=True, res=True, strided=False):
    g = Draw(seed)
    make = g.wide if strided else g.normal
    a = dict(x=make(M, D, std=3.0, dtype=dtype), gate=None if act is None else make(M, D, dtype=dtype),
             res=make(M, D, std=2.0, dtype=dtype) if res else None, w_post=1 + g.normal(D, std=0.2) if post else None,
             scale=g.uniform(D, lo=-0.5, hi=0.5) if scale else None, w_pre=1 + g.normal(D, std=0.2) if pre else None)
    a["dy"], a["dh"] = make(M, D, dtype=dtype), make(M, D, dtype=dtype)
    return a


def rng_of(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def check_block(a, act, p, dtype, M, D, dh=True, seed=-5, offset=2 ** 40 + 3):
    rng = rng_of(seed, offset) if p else None
    kept, f = G.keep(seed, offset, M, D, p) if p else (None, 1.0)
    kw = dict(w_post=a["w_post"], w_pre=a["w_pre"], gate=a["gate"], act=act or "linear", scale=a["scale"], p=p, rng=rng)
    y, h, rp, rq = la.la_block_norm(a["x"], a["res"], eps=1e-5, **kw)
    ref = [R.f64(a[k]) for k in ("x", "gate", "res", "w_post", "scale", "w_pre")]
    want = G.block(*ref, act, 1e-5, kept, f)
    for name, t, r, dt in (("y", y, want[0], dtype), ("h", h, want[1], dtype), ("rp", rp, want[2], F32), ("rq", rq, want[3], F32)):
        assert (t is None) == (r is None), name
        if t is not None:
            G.close(t, *r, dt, name)
    pre = a["w_pre"] is not None
    out = la.la_block_norm_bwd(a["x"], h if pre else None, a["dy"] if pre else None, a["dh"] if dh else None, rstd_post=rp,
                               rstd_pre=rq, **kw)
    want = G.block_bwd(R.f64(a["x"]), R.f64(a["gate"]), R.f64(h), *[R.f64(a[k]) for k in ("w_post", "scale", "w_pre")], act,
                       R.f64(rp), R.f64(rq), R.f64(a["dy"]), R.f64(a["dh"]) if dh else None, kept, f)
    for name, t, r in zip(("dx", "dresidual", "dgate", "dw_post", "dw_pre", "dscale"), out, want):
        assert (t is None) == (r is None), name
        if t is not None:
            G.close(t, *r, dtype if t.dim() == 2 else F32, name)
    return (y, h, rp, rq), out, kw


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,D", BLOCK)
def test_block_forward_and_backward(M, D, dtype):
    note(f"block norm {M} {D} {dtype}")
    a = block_inputs(M, D, dtype, M + D)
    if M > 1:
        a["x"][1] = 0.0  # a row of zeros
        a["res"][1] = 0.0
    check_block(a, "silu", 0.0, dtype, M, D)
    check_block(a, "silu", 0.3, dtype, M, D)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("act", [None, "linear", "sigmoid", "silu"])
@pytest.mark.parametrize("post,pre,scale,res,dh", [(True, True, True, True, True), (False, True, True, True, True),
                                                   (True, False, True, True, True), (False, False, False, False, True),
                                                   (True, True, False, False, False), (False, True, False, True, False)])
def test_block_parts(act, post, pre, scale, res, dh, dtype):
    """Every part left out in turn, strided rows, with and without dropout."""
    note(f"block parts {act} {post} {pre} {scale} {res} {dh} {dtype}")
    for D in (72, 1001):
        a = block_inputs(6, D, dtype, 11, act, post, pre, scale, res, strided=True)
        check_block(a, act, 0.0, dtype, 6, D, dh)
        check_block(a, act, 0.5, dtype, 6, D, dh)


def test_block_in_place():
    note("block norm in place")
    a = block_inputs(5, 264, BF, 3)
    (y, h, rp, rq), out, kw = check_block(a, "silu", 0.2, BF, 5, 264)
    for k in ("x", "res"):
        t = {q: (v.clone() if v is not None else None) for q, v in a.items()}
        y2, h2, _, _ = la.la_block_norm(t["x"], t["res"], h=t[k], **kw)
        assert h2.data_ptr() == t[k].data_ptr() and torch.equal(h2, h) and torch.equal(y2, y)
    for k in ("dy", "dh"):
        t = {q: (v.clone() if v is not None else None) for q, v in a.items()}
        got = la.la_block_norm_bwd(t["x"], h, t["dy"], t["dh"], rstd_post=rp, rstd_pre=rq, dresidual=t[k], **kw)
        assert got[1].data_ptr() == t[k].data_ptr()
        for s, q in zip(got, out):
            assert torch.equal(s, q)


@pytest.mark.parametrize("D", [72, 2048, 4096, 9000])
def test_block_of_values_whose_squares_overflow(D):
    note(f"block norm of large values {D}")
    a = block_inputs(4, D, F32, 9)
    a["x"][1] *= 1e30
    a["res"][2] *= 1e30
    check_block(a, "silu", 0.25, F32, 4, D)


def test_block_dropped_values_that_are_not_finite():
    """What is dropped leaves no trace, whatever it holds."""
    note("block norm, dropped infinities")
    M, D, p = 6, 520, 0.5
    a = block_inputs(M, D, F32, 13, post=False)
    kept, _ = G.keep(-5, 2 ** 40 + 3, M, D, p)
    gone = torch.from_numpy(~kept).cuda()
    clean = dict(a, x=a["x"].masked_fill(gone, 1.0), gate=a["gate"].masked_fill(gone, 1.0))
    first, out, kw = check_block(clean, "silu", p, F32, M, D)
    for value in (float("inf"), float("nan")):
        x, gate = a["x"].masked_fill(gone, value), a["gate"].masked_fill(gone, value)
        kw2 = dict(kw, gate=gate)
        got = la.la_block_norm(x, a["res"], **kw2)
        for s, t in zip(first, got):
            assert (s is None) == (t is None) and (s is None or torch.equal(s, t))
        back = la.la_block_norm_bwd(x, got[1], a["dy"], a["dh"], rstd_pre=got[3], **kw2)
        for s, t in zip(out, back):
            assert (s is None) == (t is None) and (s is None or torch.equal(s, t))
        y = la.la_dropout(x, kw["rng"], p)
        assert (y[gone] == 0).all() and torch.isfinite(y).all()


# ------------------------------------------------------------------------------------ dropout


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,D,strided", [(1, 8, False), (3, 64, True), (5, 1001, False), (1, 1, False), (777, 24, False),
                                         (2, 40000, True), (0, 5, False), (4, 6, True)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1 - 2.0 ** -16])
def test_dropout(M, D, strided, p, dtype):
    note(f"dropout {M} {D} {strided} {p} {dtype}")
    g = Draw(M + D)
    make = g.wide if strided else g.normal
    x, res = make(M, D, dtype=dtype), make(M, D, dtype=dtype)
    for seed, offset in ((0, 0), (-1, 2 ** 63 - 1), (2 ** 40 + 17, 9)):
        kept, f = G.keep(seed, offset, M, D, p)
        rng = rng_of(seed, offset)
        y = la.la_dropout(x, rng, p)
        want = np.where(kept, R.f64(x) * f, 0)
        assert torch.equal(y == 0, torch.from_numpy(~kept).cuda() | (x == 0))
        G.close(y, want, np.abs(want) * 2, dtype, "y")
        y = la.la_dropout(x, rng, p, res)
        G.close(y, want + R.f64(res), np.abs(want) * 2 + np.abs(want + R.f64(res)), dtype, "sum")
        for k in (0, 1):
            t = (x.clone(), res.clone())
            assert torch.equal(la.la_dropout(t[0], rng, p, t[1], y=t[k]), y) and torch.equal(t[k], y)
