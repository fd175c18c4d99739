"""The gated recurrent layer's operators and the residual norm where their numbers are extreme (rows near the type's largest
value, gates that are all but open, rates past fp32's range, infinities), on empty batches, and on the paths that only
large batches take, against the fp64 forms of gated_ref.py."""
import ctypes

import numpy as np
import pytest
import torch

import gated_ref as G
import mixer_ref as R
from chunked_scan_amd import binding as la
from chunked_scan_amd import pipeline
from gpu_util import note
from test_gpu_gated import block_inputs, check_block, check_grads, nonan, rng_of, scan_inputs, scan_kw, scan_ref
from test_gpu_gated_layer import layer
from test_gpu_mixer import BF, F32, SENTINEL, Draw

pytestmark = pytest.mark.gpu

# ------------------------------------------------------------------------------------ rows near the largest value


def huge_rows(M, D, dtype, seed):
    """Rows of 1e37, 1e38 and 3e38 times a factor in 0.5..1, signs in turn."""
    t = Draw(seed).uniform(M, D, lo=0.5, hi=1.0) * torch.tensor([1e37, 1e38, 3e38], device="cuda").repeat(M)[:M, None]
    return (t * (1 - 2 * (torch.arange(D, device="cuda") % 2))).to(dtype)


def check_rstd(got, ref, D):
    """D / 8 + 32 roundings (a lane's share of a row's sum, the lanes'), and half a step of fp32's subnormal numbers."""
    assert (np.abs(R.f64(got) - ref) <= (D / 8 + 32) * R.U * ref + 2.0 ** -150).all()


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 1001, 2048, 16384])
def test_norms_of_rows_near_the_largest_value(D, dtype):
    note(f"norms of rows near the largest value {D} {dtype}")
    M, eps = 6, 1e-5
    for big in ("x", "res"):
        a = block_inputs(M, D, dtype, 21)
        a[big] = huge_rows(M, D, dtype, 22)
        if big == "x":  # the post-norm brings small rows down further still
            a["w_post"][: D // 2] *= 1e-6
            a["res"] = None
        (y, h, rp, rq), _, _ = check_block(a, "silu", 0.0, dtype, M, D)
        _, (hr, _), rpr, rqr = G.block(*[R.f64(a[k]) for k in ("x", "gate", "res", "w_post", "scale", "w_pre")], "silu", eps)
        check_rstd(rp, rpr[0], D)
        if big == "res":  # u is below half a step of the stream
            check_rstd(rq, rqr[0], D)
            assert np.abs(R.f64(y)).max() > 0.5
    x, w = huge_rows(M, D, dtype, 23), 1 + Draw(24).normal(D, std=0.2)
    w[: D // 2] *= 1e-6
    x64, w64 = R.f64(x), R.f64(w)
    r = 1 / np.sqrt((x64 ** 2).mean(1, keepdims=True) + eps)
    y, _, rstd = la.la_add_norm(x, w)
    G.close(y, x64 * r * w64, np.abs(x64 * r * w64) * (D / 8 + 36), dtype, "y")
    check_rstd(rstd, r[:, 0], D)
    q, scale, _, rstd = la.la_add_norm_q8(x, w)
    # e4m3: half a step of 2^-4 of the value in its normal range, of 2^-9 of the scale below it
    want, s = x64 * r * w64, R.f64(scale)
    tol = np.abs(want) * (2.0 ** -4 + (D / 8 + 40) * R.U) + s * 2.0 ** -10 * 1.01
    assert (np.abs(R.f64(q.float()) * s - want) <= tol).all()
    check_rstd(rstd, r[:, 0], D)


# ------------------------------------------------------------------------------------ gates that are all but open

# sigma(-v) next to zero is a small number in its own right.  With e = exp(-v), 1 - sigma(v) = e sigma(v): e's relative bound
# 2 (|r| + |b|) + 2, and the sum, the reciprocal and the product; so gated_ref's bound of sigma, and one rounding where it is
# taken as a difference from 1 (there it is above 1/2).


def open_gates_ref(a, c):
    """[(value, bound)] of dr, di, dr_bias, di_bias without output gate and lengths, relative to 1 - rho and 1 - iota."""
    x, r, i, lam, rb, ib, _, h_in, _, _ = scan_ref(a, None, c)
    g, _, _, _, _, before, e_before, H_before, b = G.scan(x, r, i, lam, rb, ib, None, h_in, None, c)[3]
    dy = R.f64(a["dy"])
    carry, ec = np.zeros_like(h_in), np.zeros_like(h_in)
    gs, eg, Gm = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
    C = np.abs(carry)
    for t in range(x.shape[1] - 1, -1, -1):
        gs[:, t], Gm[:, t] = dy[:, t] + carry, np.abs(dy[:, t]) + C
        eg[:, t] = ec + 4 * Gm[:, t]
        at = g.a[:, t]
        carry, C, ec = at * gs[:, t], at * Gm[:, t], at * (eg[:, t] + (g.k_a[:, t] + 1) * Gm[:, t])
    co_r, co_i, ab = R.sig(-(r + rb)), R.sig(-(i + ib)), np.abs(b)
    q = gs * (g.slope * b - g.v * g.a * before)
    eq = eg * (g.slope * ab + g.v * g.a * H_before) + Gm * (
        g.slope * ab * (g.k_slope + g.k_mi + 4) + g.v * g.a * (e_before + (g.k_v + g.k_a + 5) * H_before))
    Q = Gm * (g.slope * ab + g.v * g.a * H_before)
    dr = (q * co_r, co_r * (eq + Q * (g.k_rho + 3)))
    di = (gs * b * co_i, ab * co_i * (eg + Gm * (g.k_mi + g.k_iota + 6)))
    n = x.shape[0] * x.shape[1] + 8
    return [dr, di, (dr[0].sum((0, 1)), dr[1].sum((0, 1)) + n * (Q * co_r).sum((0, 1))),
            (di[0].sum((0, 1)), di[1].sum((0, 1)) + n * (ab * Gm * co_i).sum((0, 1)))]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,L,D", [(40, 1, 64), (2, 70, 130), (1, 200, 65)])
def test_scan_gradients_of_gates_that_are_all_but_open(B, L, D, dtype):
    """r + r_bias and i + i_bias from -20 to 40: the gates' gradients keep their digits however close to 1 a gate is."""
    note(f"gated scan: open gates {B} {L} {D} {dtype}")
    a, _ = scan_inputs((B, L, D, None, False, False, True, True, -5.0), dtype, 51)
    g = Draw(52)
    for k in ("r", "i"):
        a[k] = g.uniform(B, L, D, lo=-20.0, hi=38.0).to(dtype)
    got = la.la_gated_scan_bwd(*[a[k] for k in ("x", "r", "i", "lam", "dy")], **scan_kw(a, None))
    names = ("dr", "di", "dr_bias", "di_bias")
    for name, t, ref in zip(names, (got[1], got[2], got[4], got[5]), open_gates_ref(a, 8.0)):
        G.close(t, *ref, dtype if t.dim() == 3 else F32, name)
    # and where sigma's complement leaves fp32 there is no value but zero
    a["r"].fill_(200.0), a["i"].fill_(200.0)
    got = la.la_gated_scan_bwd(*[a[k] for k in ("x", "r", "i", "lam", "dy")], **scan_kw(a, None))
    assert (got[1] == 0).all() and (got[2] == 0).all() and all(torch.isfinite(t).all() for t in got if t is not None)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 1001])
def test_norm_gradients_of_gates_that_are_all_but_open(D, dtype):
    note(f"block norm: open gates {D} {dtype}")
    M = 5
    a = block_inputs(M, D, dtype, 53)
    a["gate"] = Draw(54).uniform(M, D, lo=-20.0, hi=40.0).to(dtype)
    _, h, rp, rq = la.la_block_norm(a["x"], a["res"], w_post=a["w_post"], w_pre=a["w_pre"], gate=a["gate"], act="sigmoid",
                                    scale=a["scale"])
    got = la.la_block_norm_bwd(a["x"], h, a["dy"], a["dh"], w_post=a["w_post"], w_pre=a["w_pre"], gate=a["gate"],
                               act="sigmoid", scale=a["scale"], rstd_post=rp, rstd_pre=rq)[2]
    # du n scale, which the linear gate's derivative is; times s (1 - s), each with the gate's relative bound
    v, e = G.block_bwd(R.f64(a["x"]), R.f64(a["gate"]), R.f64(h), *[R.f64(a[k]) for k in ("w_post", "scale", "w_pre")], "linear",
                       R.f64(rp), R.f64(rq), R.f64(a["dy"]), R.f64(a["dh"]))[2]
    gate = R.f64(a["gate"])
    slope = R.sig(gate) * R.sig(-gate)
    G.close(got, v * slope, (e + np.abs(v) * (4 * np.abs(gate) + 20)) * slope, dtype, "dgate")


# ------------------------------------------------------------------------------------ rates past fp32's range


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 65])
def test_rates_beyond_the_range(D, dtype):
    """c softplus(lam) up to infinity in fp32 for finite c and lam: the decay is complete (a = 0, m = 1) where the gate is
    open, a closed gate holds the state, and every gradient is finite."""
    note(f"gated scan: rates beyond the range {D} {dtype}")
    B, L = 2, 150
    a, _ = scan_inputs((B, L, D, None, False, True, True, True, -5.0), dtype, 61)
    a["lam"] = torch.tensor([3e38, 1e38, 3e37, 1e30, 1e20, 200.0, -3.0], device="cuda").repeat(D)[:D].contiguous()
    a["x"] = a["x"] * 1e6
    a["h_in"] = a["h_in"] * 1e9
    a["r"][:, 10:14] = float("-inf")
    a["r"][:, 130:] = float("-inf")
    kw, args = scan_kw(a, None), [a[k] for k in ("x", "r", "i", "lam")]
    y, h, _ = la.la_gated_scan(*args, **kw)
    ref = scan_ref(a, None, 8.0)
    ref[1] = np.where(np.isneginf(R.f64(a["r"])), -np.inf, ref[1])  # scan_ref takes infinities to large numbers
    with np.errstate(invalid="ignore", over="ignore"):
        ry, rh, _, _ = G.scan(*ref)
    live = np.broadcast_to(R.f64(a["lam"]) < 1e3, ry[0].shape)
    # a complete decay has no roundings in its exponent: the state is iota x of the last open token, or the incoming one
    open_ = ~np.isneginf(R.f64(a["r"]))
    want, s = np.zeros_like(ry[0]), R.f64(a["h_in"])
    iota = R.sig(ref[2] + ref[5])
    for t in range(L):
        s = np.where(open_[:, t], iota[:, t] * ref[0][:, t], s)
        want[:, t] = s
    k_iota = 2 * (np.abs(ref[2]) + np.abs(ref[5])) + 10
    z, kz = G.silu_of(ref[6])
    held = np.maximum.accumulate(np.where(open_, np.arange(L)[None, :, None], 0), 1)
    ks = np.take_along_axis(k_iota, held, 1)
    G.close(y, np.where(live, ry[0], want * z), np.where(live, ry[1], np.abs(want * z) * (ks + kz + 4)), dtype, "y")
    assert torch.isfinite(h).all()
    # bf16 rows of dy times states of 1e9 stay in range
    got = la.la_gated_scan_bwd(*args, a["dy"], dh_out=a["dh_out"], **kw)
    full = torch.from_numpy(~live[0, 0]).cuda()
    for t in got:
        assert torch.isfinite(t).all()
    # v dL/dv is zero at a complete decay, and zero where the state is held
    assert (got[1][..., full] == 0).all() and (got[3][full] == 0).all() and (got[4][full] == 0).all()
    state = a["h_in"].clone()
    one = [t[:, 10].contiguous() for t in (a["x"], a["r"], a["i"])]
    la.la_gated_step(*one, a["lam"], state, r_bias=a["rb"], i_bias=a["ib"])
    assert torch.equal(state, a["h_in"])
    # a large c and a softplus that is zero: no decay
    h = la.la_gated_scan(*args[:3], torch.full_like(a["lam"], -200.0), c=3e38, **kw)[1]
    assert torch.equal(h, a["h_in"])


# ------------------------------------------------------------------------------------ the layer's generator


def test_layer_backward_after_the_generator_moved_on():
    """One generator for several layers, its offset advanced in place behind each forward: a layer's backward drops what
    its own forward dropped."""
    note("gated layer: the generator moves on")
    B, L, D, Dm, W = 2, 40, 32, 48, 4
    p, proj, backwards = layer(D, Dm, W, 71, dropout=0.4)
    g = Draw(72)
    n, res, dy, dh = (g.normal(B, L, Dm) for _ in range(4))
    grads = []
    for step in (0, 1):
        rng, saved = rng_of(3, 100), {}
        pipeline.gated_prompt(p, n, res, *proj, rng=rng, saved=saved)
        rng[1] += step
        grads.append(pipeline.gated_backward(p, saved, dy, dh, **backwards(F32)))
    for k, t in grads[0].items():
        assert (t is None) == (grads[1][k] is None) and (t is None or torch.equal(t, grads[1][k])), k


# ------------------------------------------------------------------------------------ empty batches


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("L", [5, 100, 200])
def test_empty_batch_with_a_workspace(L, dtype):
    """No sequences, and a workspace that the caller has from other calls: the parameters' derivatives are zero."""
    note(f"gated scan backward: empty batch {L} {dtype}")
    D = 72
    lam = torch.zeros(D, device="cuda")
    sums = [torch.full((D,), SENTINEL, device="cuda") for _ in range(3)]
    ws = torch.full((1 << 16,), 7, dtype=torch.uint8, device="cuda")
    shp = la.GatedShape(0, L, D, 0 if dtype == F32 else 1, 8.0)
    shp.stream = torch.cuda.current_stream().cuda_stream
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    none = ctypes.c_void_p(None)
    lib = la.lib()
    assert lib.la_gated_scan_workspace(ctypes.byref(shp), 1) == 0
    st = lib.la_gated_scan(none, none, none, p(lam), none, none, none, none, none, none, none, none, p(ws), 1 << 16,
                           ctypes.byref(shp))
    assert st == 0
    st = lib.la_gated_scan_bwd(none, none, none, p(lam), p(lam), p(lam), none, none, none, none, none, none, none, none, none,
                               p(sums[0]), p(sums[1]), p(sums[2]), none, none, p(ws), 1 << 16, ctypes.byref(shp))
    assert st == 0
    torch.cuda.synchronize()
    assert all((t == 0).all() for t in sums) and (ws == 7).all()


# ------------------------------------------------------------------------------------ infinities


@pytest.mark.parametrize("D", [64, 65])
def test_infinity_stays_in_its_channel(D):
    """An infinite x or state leaves its channel infinite or NaN from that token on, forward and in the states handed on;
    what came before it and every other channel keeps its bits."""
    note(f"gated scan: infinity {D}")
    B, L = 2, 700
    a, _ = scan_inputs((B, L, D, None, False, False, True, True, -1.0), F32, 81)
    args, kw = lambda x: (x, a["r"], a["i"], a["lam"]), scan_kw(a, None)  # noqa: E731
    y, h, _ = la.la_gated_scan(*args(a["x"]), **kw)
    for where in ("x", "h_in"):
        x, s = a["x"].clone(), a["h_in"].clone()
        bad = torch.zeros_like(y, dtype=torch.bool)
        if where == "x":
            x[1, 140, 33] = float("inf")
            bad[1, 140:, 33] = True
        else:
            s[1, 33] = float("-inf")
            bad[1, :, 33] = True
        y2, h2, _ = la.la_gated_scan(*args(x), **dict(kw, h_in=s))
        assert not torch.isfinite(y2[bad]).any() and torch.equal(y2[~bad], y[~bad])
        assert not torch.isfinite(h2[1, 33]) and int((~torch.isfinite(h2)).sum()) == 1
        got = la.la_gated_scan_bwd(*args(x), a["dy"], **dict(kw, h_in=s))
        ref = la.la_gated_scan_bwd(*args(a["x"]), a["dy"], **kw)
        for t, q in zip(got, ref):  # other channels, also in the sums over sequences
            if t is not None:
                keep = torch.arange(D, device="cuda") != 33
                assert torch.equal(t[..., keep], q[..., keep])
    state = a["h_in"].clone()
    state[1, 33] = float("inf")
    la.la_gated_step(a["x"][:, 0], a["r"][:, 0], a["i"][:, 0], a["lam"], state, r_bias=a["rb"], i_bias=a["ib"])
    assert not torch.isfinite(state[1, 33]) and int((~torch.isfinite(state)).sum()) == 1


# ------------------------------------------------------------------------------------ large batches


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,D", [(3500, 96), (3500, 41), (1700, 1000), (900, 2047), (600, 4095), (600, 4096), (300, 8191), (300, 8192),
                                 (300, 8200), (300, 16384), (300, 9001)])
def test_block_of_more_rows_than_blocks(M, D, dtype):
    """The backward's blocks walk several rows each (at most 768, 512 or 256 blocks by width), and the forward takes its forms
    for many rows; the parameters' sums against the fp64 form."""
    note(f"block norm of many rows {M} {D} {dtype}")
    a = block_inputs(M, D, dtype, M + D)
    check_block(a, "silu", 0.0, dtype, M, D)
    check_block(a, "sigmoid", 0.3, dtype, M, D)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,D", [(600, 1024), (600, 5000), (600, 600)])
def test_block_of_two_chunks_a_thread(M, D, dtype):
    note(f"block norm, wide rows in many {M} {D} {dtype}")
    a = block_inputs(M, D, dtype, M + D)
    check_block(a, "silu", 0.3, dtype, M, D)


def check_sums(got, ref, a):
    """dlam, dr_bias and di_bias as sums of the fp64 form's own terms, bound by the terms' bounds and by the roundings of
    the sum, which is no chain over all tokens: 16 of a lane's, 8 runs of a tile, 32 and 16 of 512 rows, and up to 17 behind
    them, 100 in all; sigma / softplus 24 more."""
    (dr, er), (di, ei) = ref[1:3]
    co = R.sig(-(R.f64(a["r"]) + R.f64(a["rb"])))
    with np.errstate(invalid="ignore"):
        q, eq = np.nan_to_num(dr / co), np.nan_to_num(er / co)
    lam = R.f64(a["lam"])
    for t, v, e, k, by in ((got[3], q, eq, 124, R.sig(lam) / G.softplus(lam)), (got[4], dr, er, 100, 1.0), (got[5], di, ei, 100, 1.0)):
        G.close(t, by * v.sum((0, 1)), by * (e.sum((0, 1)) + k * np.abs(v).sum((0, 1))), F32, "sums")


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", [(3, 64 * 171 + 5, 5, None, False, False, True, True, -3.0),
                                  (20, 64 * 60 + 9, 6, None, False, False, True, True, -3.0),
                                  (700, 70, 8, [70, 0, 3, 64, 65] * 140, False, True, True, True, -3.0)], ids=lambda c: str(c[:3]))
def test_scan_sums_of_many_partial_rows(case, dtype):
    """More than 512 rows of partial sums (a row per sequence and 64 tokens: 516, 1220, 1400), so that they are added in
    two steps; the last step's share is not a whole one."""
    note(f"gated scan: many partial rows {case[:3]} {dtype}")
    a, n = scan_inputs(case, dtype, 91)
    got = la.la_gated_scan_bwd(*[a[k] for k in ("x", "r", "i", "lam", "dy")], dh_out=a["dh_out"], **scan_kw(a, case[3]))
    ref = G.scan_bwd(*scan_ref(a, n, 8.0), nonan(a["dy"]), R.f64(a["dh_out"]))
    check_grads(got, ref, dtype, n)
    check_sums(got, ref, a)
    # a few rows alone, at the ends of the first step's shares: none of them can be lost in the others' bounds
    B, L = case[:2]
    tiles = -(-L // 64)
    last = B * tiles - 1
    rows = [k for k in (0, 15, 16, 511, 512, 527, 528, 1023, 1024, last - 1, last) if k <= last]
    mask = torch.zeros(B * tiles, dtype=torch.bool)
    mask[rows] = True
    mask = mask.view(B, tiles, 1).expand(B, tiles, 64).reshape(B, tiles * 64)[:, :L, None].cuda()
    a["dy"] = torch.where(mask, a["dy"], torch.zeros_like(a["dy"]))
    got = la.la_gated_scan_bwd(*[a[k] for k in ("x", "r", "i", "lam", "dy")], **scan_kw(a, case[3]))
    check_sums(got, G.scan_bwd(*scan_ref(a, n, 8.0), nonan(a["dy"]), None), a)
