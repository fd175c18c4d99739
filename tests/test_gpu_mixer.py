"""The short convolution, the selective scan and the residual norm on the GPU against their fp64 forms
(mixer_ref.py), at the sizes, strides and masks where they can go wrong, alone and together.

Tolerances: half a step of the stored type, plus K 2^-24 of the sum of the terms' absolute values, where K counts
the roundings that can reach a value.  Convolution: W + 4 taps and sums and about 24 for the hardware
exponential and reciprocal (each about 1 ulp on an argument rounded once, |argument| < 12).  Scan: every token
multiplies a state by a decay whose exponent carries about 8 roundings, so after L tokens K = 8 L, plus 64
for the step size, the gate and the sum over the state (64 terms at most, in fp32); sums over D channels
or B L tokens add one rounding a term.  Norm: D / 8 for a lane's share of a row's sum, plus 32.
"""
import dataclasses
import itertools

import numpy as np
import pytest
import torch

import mixer_ref as R
from chunked_scan_amd import binding as la
from chunked_scan_amd import pipeline
from gpu_util import note

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SENTINEL = 7.0


class Draw:
    def __init__(self, seed):
        self.g = torch.Generator()
        self.g.manual_seed(seed)

    def normal(self, *shape, std=1.0, dtype=F32):
        return (torch.randn(shape, generator=self.g) * std).to(dtype).cuda()

    def uniform(self, *shape, lo=0.0, hi=1.0):
        return (torch.rand(shape, generator=self.g) * (hi - lo) + lo).cuda()

    def wide(self, *shape, std=1.0, dtype=F32, extra=24, at=8):
        """The same through a slice of a wider buffer."""
        buf = self.normal(*shape[:-1], shape[-1] + extra, std=std, dtype=dtype)
        return buf[..., at : at + shape[-1]]


def cut(lengths, L):
    return None if lengths is None else [min(max(int(n), 0), L) for n in lengths]


def ints(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")


def check_tail(t, lengths, value, what):
    """Rows behind every sequence's end hold ``value``."""
    if lengths is not None:
        for i, n in enumerate(lengths):
            assert (t[i, n:] == value).all(), (what, i)


def nan_tail(t, lengths):
    """NaN in the rows behind every sequence's end: no result may see them."""
    if lengths is not None:
        for i, n in enumerate(lengths):
            t[i, n:] = float("nan")


# ------------------------------------------------------------------------------------ convolution

CONV = [  # B, L, D, W, lengths, strided, state, bias, silu
    (1, 1, 8, 2, None, False, False, True, True),
    (2, 5, 64, 4, None, False, True, True, True),
    (3, 67, 40, 3, [67, 0, 1], False, True, False, True),
    (2, 130, 72, 4, [129, 2], True, True, True, False),
    (1, 300, 7, 4, None, False, True, True, True),      # D not a whole vector
    (2, 33, 24, 4, [40, -3], True, False, True, True),  # lengths outside 0..L are cut
    (4, 1, 16, 4, [1, 0, 1, 1], False, True, True, True),
    (1, 0, 16, 3, None, False, True, True, True),
    (2, 700, 520, 4, None, True, True, True, True),
]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv_forward_and_backward(case, dtype):
    B, L, D, W, lengths, strided, state, bias, act = case
    note(f"conv {case} {dtype}")
    g = Draw(10 + L)
    make = g.wide if strided else g.normal
    x, dy = make(B, L, D, dtype=dtype), make(B, L, D, dtype=dtype)
    w, b = g.normal(D, W, std=0.6), g.normal(D) if bias else None
    st = g.normal(B, W - 1, D, dtype=dtype) if state else None
    dso = g.normal(B, W - 1, D, dtype=dtype)
    n = cut(lengths, L)
    nan_tail(x, n)
    nan_tail(dy, n)
    wide = torch.full((B, L, D + 16), SENTINEL, dtype=dtype, device="cuda")
    y = wide[..., 8 : 8 + D] if strided else wide[..., :D].contiguous()
    got, so = la.la_short_conv(x, w, b, st, lengths=ints(lengths), silu=act, y=y, want_state=True)
    xn = np.nan_to_num(R.f64(x))
    ref, ref_so = R.conv(xn, R.f64(w), R.f64(b), R.f64(st), n, act)
    mag, _ = R.conv(np.abs(xn), np.abs(R.f64(w)), None if b is None else np.abs(R.f64(b)), None if st is None else np.abs(R.f64(st)), n, False)
    check_tail(got, n, SENTINEL, "y")
    keep = np.ones((B, L, 1), bool) if n is None else (np.arange(L)[None] < np.array(n)[:, None])[..., None]
    K = W + 28
    R.close(torch.where(torch.from_numpy(keep).cuda(), got, torch.zeros_like(got)), ref, mag, K, dtype, "y")
    assert np.array_equal(R.f64(so), ref_so), "state_out"
    if strided:
        assert (wide[..., :8] == SENTINEL).all() and (wide[..., 8 + D :] == SENTINEL).all()

    dx = torch.full((B, L, D + 16), SENTINEL, dtype=dtype, device="cuda")[..., 8 : 8 + D] if strided else None
    dx, dw, db, ds = la.la_short_conv_bwd(x, w, dy, b, st, dso, lengths=ints(lengths), silu=act, dx=dx)
    args = (xn, R.f64(w), R.f64(b), R.f64(st), n, act, np.nan_to_num(R.f64(dy)), R.f64(dso))
    r, m = R.conv_bwd(*args), R.conv_bwd(*args, mag=True)
    check_tail(dx, n, 0.0, "dx")
    R.close(dx, r[0], m[0], 2 * K, dtype, "dx")
    R.close(dw, r[1], m[1], 2 * K + B * L, F32, "dw")
    if bias:
        R.close(db, r[2], m[2], 2 * K + B * L, F32, "db")
    if state:
        R.close(ds, r[3], m[3], 2 * K, dtype, "ds")


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,D,W,S,slots", [(1, 8, 2, 1, None), (3, 40, 4, 5, [4, 0, 2]), (4, 7, 3, 4, [1, -1, 9, 3]),
                                           (5, 640, 4, 6, [2, 5, 2, 0, 5])])
def test_conv_step(B, D, W, S, slots, dtype):
    note(f"conv step {B} {D} {W} {S} {slots} {dtype}")
    g = Draw(3)
    x, w, b = g.wide(B, D, dtype=dtype), g.normal(D, W, std=0.6), g.normal(D)
    state = g.normal(S, W - 1, D, dtype=dtype)
    before = state.clone()
    y = torch.full((B, D), SENTINEL, dtype=dtype, device="cuda")
    la.la_short_conv_step(x, w, state, b, slots=ints(slots), y=y)
    at = list(range(B)) if slots is None else slots
    seen = set()
    for i, s in enumerate(at):
        if s < 0 or s >= S or s in seen:  # padding: out of the pool, or named by an earlier row
            assert (y[i] == SENTINEL).all()
            continue
        seen.add(s)
        args = (R.f64(x[i])[None, None], R.f64(w), R.f64(b), R.f64(before[s])[None], None)
        ref, so = R.conv(*args, True)
        mag, _ = R.conv(*[np.abs(v) if v is not None else None for v in args], False)
        R.close(y[i], ref[0, 0], mag[0, 0], W + 28, dtype, "y")
        assert np.array_equal(R.f64(state[s]), so[0])
    for s in set(range(S)) - seen:
        assert torch.equal(state[s], before[s])


# ------------------------------------------------------------------------------------ scan

SCAN = [  # B, L, D, N, lengths, strided, gate, skip, bias, s_in, softplus
    (1, 1, 64, 16, None, False, True, True, True, False, True),
    (2, 9, 64, 16, [9, 4], False, True, True, True, True, True),
    (3, 67, 40, 8, [67, 0, 1], False, False, True, True, True, True),
    (1, 200, 70, 16, None, True, True, True, True, True, True),    # split over segments, two channel blocks
    (2, 333, 65, 24, [300, 17], True, True, False, False, True, True),
    (2, 150, 130, 17, [151, -2], False, True, True, True, False, True),
    (1, 129, 3, 1, None, False, False, False, True, True, True),
    (1, 140, 64, 64, [139], False, True, True, True, True, True),
    (2, 72, 33, 48, None, True, False, True, False, False, False),
    (2, 64, 16, 32, [64, 63], False, True, True, True, True, False),
    (1, 0, 32, 16, None, False, True, True, True, True, True),
    (1, 517, 64, 16, None, False, True, True, True, False, True),
]


def scan_inputs(case, dtype, seed):
    B, L, D, N, lengths, strided, gate, skip, bias, s_in, sp = case
    g = Draw(seed)
    make = g.wide if strided else g.normal
    a = dict(u=make(B, L, D, dtype=dtype), A=-g.uniform(D, N, lo=0.5, hi=N + 1.0))
    if sp:
        a["dt"] = make(B, L, D, std=0.5, dtype=dtype)
        a["dt_bias"] = g.uniform(D, lo=-6.0, hi=-1.0) if bias else None
    else:  # step sizes given as they are
        wide = g.uniform(B, L, D + 24, lo=0.001, hi=0.2).to(dtype)
        a["dt"] = wide[..., 8 : 8 + D] if strided else wide[..., :D].contiguous()
        a["dt_bias"] = g.uniform(D, lo=0.0, hi=0.1) if bias else None
    bc = g.normal(B, L, 2 * N + 5, dtype=dtype)  # odd offsets: 2-byte aligned rows in bf16
    a["B"], a["C"] = bc[..., 5 : 5 + N], bc[..., 5 + N :]
    a["D"] = g.normal(D) if skip else None
    a["z"] = make(B, L, D, dtype=dtype) if gate else None
    a["s_in"] = g.normal(B, N, D) if s_in else None
    a["dy"] = make(B, L, D, dtype=dtype)
    a["ds_out"] = g.normal(B, N, D)
    n = cut(lengths, L)
    for k in ("u", "dt", "B", "C", "z", "dy"):
        if a[k] is not None:
            nan_tail(a[k], n)
    return a, n


def ref_args(a, n, sp):
    f = {k: (None if v is None else np.nan_to_num(R.f64(v))) for k, v in a.items()}
    return (f["u"], f["dt"], f["A"], f["B"], f["C"], f["D"], f["z"], f["dt_bias"], f["s_in"], n, sp), f["dy"], f["ds_out"]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", SCAN, ids=str)
def test_scan_forward_and_backward(case, dtype):
    B, L, D, N, lengths, strided, gate, skip, bias, s_in, sp = case
    note(f"scan {case} {dtype}")
    a, n = scan_inputs(case, dtype, 100 + L)
    args, dy, ds_out = ref_args(a, n, sp)
    kw = {k: a[k] for k in ("D", "z", "dt_bias", "s_in")}
    wide = torch.full((B, L, D + 16), SENTINEL, dtype=dtype, device="cuda")
    y = wide[..., 8 : 8 + D] if strided else wide[..., :D].contiguous()
    got, so = la.la_ssm_scan(a["u"], a["dt"], a["A"], a["B"], a["C"], y=y, lengths=ints(lengths), softplus=sp, **kw)
    ref, ref_so, _ = R.scan(*args)
    mag, mag_so, _ = R.scan(*args, mag=True)
    check_tail(got, n, SENTINEL, "y")
    if strided:
        assert (wide[..., :8] == SENTINEL).all() and (wide[..., 8 + D :] == SENTINEL).all()
    keep = np.ones((B, L, 1), bool) if n is None else (np.arange(L)[None] < np.array(n)[:, None])[..., None]
    K = 8 * L + 64
    R.close(torch.where(torch.from_numpy(keep).cuda(), got, torch.zeros_like(got)), ref, mag, K, dtype, "y")
    R.close(so, ref_so, mag_so, K, F32, "s_out")
    # the state written over the incoming one
    if s_in:
        s = a["s_in"].clone()
        kw2 = dict(kw, s_in=s)
        _, so2 = la.la_ssm_scan(a["u"], a["dt"], a["A"], a["B"], a["C"], s_out=s, lengths=ints(lengths), softplus=sp, **kw2)
        assert so2.data_ptr() == s.data_ptr() and torch.equal(s, so)

    grads = la.la_ssm_scan_bwd(a["u"], a["dt"], a["A"], a["B"], a["C"], a["dy"], ds_out=a["ds_out"], lengths=ints(lengths),
                               softplus=sp, **kw)
    r, m = R.scan_bwd(*args, dy, ds_out), R.scan_bwd(*args, dy, ds_out, mag=True)
    names = ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "d_dt_bias", "ds_in")
    extra = dict(dA=B * L, dB=D, dC=D, dD=B * L, d_dt_bias=B * L)
    for k, (name, gt) in enumerate(zip(names, grads)):
        none = dict(dD=not skip, dz=not gate, d_dt_bias=not bias, ds_in=not s_in).get(name, False)
        assert (gt is None) == none, name
        if gt is None:
            continue
        t = F32 if name in ("dA", "dD", "d_dt_bias", "ds_in") else dtype
        if gt.dim() == 3 and name != "ds_in":
            check_tail(gt, n, 0.0, name)
        R.close(gt, r[k], m[k], 2 * K + extra.get(name, 0), t, name)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,D,N,S,slots,gate", [(1, 64, 16, 1, None, True), (3, 40, 8, 5, [4, 0, 2], False),
                                                (4, 70, 17, 4, [1, -1, 9, 3], True), (5, 130, 64, 6, [2, 5, 2, 0, 5], True),
                                                (2, 3, 1, 2, None, False), (2, 64, 48, 2, [1, 0], True)])
def test_scan_step(B, D, N, S, slots, gate, dtype):
    note(f"scan step {B} {D} {N} {S} {slots} {dtype}")
    a, _ = scan_inputs((B, 1, D, N, None, True, gate, True, True, False, True), dtype, 5)
    one = {k: (v[:, 0] if v is not None and k in ("u", "dt", "B", "C", "z") else v) for k, v in a.items()}
    state = Draw(6).normal(S, N, D)
    before = state.clone()
    y = torch.full((B, D), SENTINEL, dtype=dtype, device="cuda")
    la.la_ssm_step(one["u"], one["dt"], a["A"], one["B"], one["C"], state, D=a["D"], z=one["z"], dt_bias=a["dt_bias"],
                   slots=ints(slots), y=y)
    seen = set()
    for i, s in enumerate(range(B) if slots is None else slots):
        if s < 0 or s >= S or s in seen:
            assert (y[i] == SENTINEL).all()
            continue
        seen.add(s)
        row = {k: (v[i : i + 1] if v is not None and k in ("u", "dt", "B", "C", "z") else v) for k, v in a.items()}
        row["s_in"] = before[s : s + 1]
        args, _, _ = ref_args(row, None, True)
        ref, so, _ = R.scan(*args)
        mag, mso, _ = R.scan(*args, mag=True)
        R.close(y[i], ref[0, 0], mag[0, 0], 72, dtype, "y")
        R.close(state[s], so[0], mso[0], 72, F32, "state")
    for s in set(range(S)) - seen:
        assert torch.equal(state[s], before[s])


def test_scan_backward_against_differences():
    """<gradient, direction> against the difference of the forward's own fp32 outputs.  With step e the
    truncation is e^2/6 of a third derivative and the rounding 2^-24 of the loss's magnitude over e: e = 2^-6
    leaves both below 1e-3 of the directional derivative's magnitude here."""
    case = (2, 90, 64, 16, [90, 31], False, True, True, True, True, True)
    note("scan differences")
    a, n = scan_inputs(case, F32, 77)
    for k in ("u", "dt", "B", "C", "z", "dy"):
        a[k] = torch.nan_to_num(a[k]).contiguous()
    names = ["u", "dt", "A", "B", "C", "D", "z", "dt_bias", "s_in"]
    lens = ints(n)

    def loss(v):
        y = torch.zeros_like(v["u"])
        y, s = la.la_ssm_scan(v["u"], v["dt"], v["A"], v["B"], v["C"], D=v["D"], z=v["z"], dt_bias=v["dt_bias"],
                              s_in=v["s_in"], lengths=lens, y=y)
        return float((y.double() * a["dy"].double()).sum() + (s.double() * a["ds_out"].double()).sum())

    gr = la.la_ssm_scan_bwd(*(a[k] for k in ("u", "dt", "A", "B", "C")), a["dy"], D=a["D"], z=a["z"], dt_bias=a["dt_bias"],
                            s_in=a["s_in"], ds_out=a["ds_out"], lengths=lens)
    grads = dict(zip(("u", "dt", "A", "B", "C", "D", "z", "dt_bias", "s_in"), gr))
    g = Draw(8)
    for k in names:
        v = g.normal(*a[k].shape)
        e = 2.0 ** -6
        up, dn = dict(a), dict(a)
        up[k], dn[k] = a[k] + e * v, a[k] - e * v
        diff = (loss(up) - loss(dn)) / (2 * e)
        want = float((grads[k].double() * v.double()).sum())
        scale = float((grads[k].double().abs() * v.double().abs()).sum())
        assert abs(diff - want) <= 1e-2 * scale / np.sqrt(v.numel()) + 1e-3 * scale, (k, diff, want, scale)


def test_gradients_into_slices_of_wide_buffers():
    """du and dz as the halves of one buffer, ddt, dB and dC as slices of another: the same values as dense outputs,
    and nothing beside the slices is touched."""
    note("gradient slices")
    case = (2, 75, 72, 16, [75, 20], False, True, True, True, True, True)
    a, n = scan_inputs(case, BF, 31)
    kw = dict(D=a["D"], z=a["z"], dt_bias=a["dt_bias"], s_in=a["s_in"], ds_out=a["ds_out"], lengths=ints(n))
    args = [a[k] for k in ("u", "dt", "A", "B", "C", "dy")]
    ref = la.la_ssm_scan_bwd(*args, **kw)
    B, L, D, N = 2, 75, 72, 16
    xz = torch.full((B, L, 2 * D + 8), SENTINEL, dtype=BF, device="cuda")
    dbc = torch.full((B, L, D + 2 * N + 8), SENTINEL, dtype=BF, device="cuda")
    got = la.la_ssm_scan_bwd(*args, **kw, du=xz[..., :D], dz=xz[..., D : 2 * D], ddt=dbc[..., :D], dB=dbc[..., D : D + N],
                             dC=dbc[..., D + N : D + 2 * N])
    for r, t in zip(ref, got):
        assert torch.equal(r, t)
    assert (xz[..., 2 * D :] == SENTINEL).all() and (dbc[..., D + 2 * N :] == SENTINEL).all()


def test_offsets_beyond_32_bits():
    """Sequences, rows and slots more than 2^32 bytes and 2^31 elements apart give what they give close together."""
    note("large offsets")
    far = (1 << 31) + 64
    g = Draw(71)
    L, D, N = 20, 64, 16
    buf = torch.empty(far + L * D + D * N, dtype=BF, device="cuda")

    def spread(t):
        """t [2, ...] with its second entry far behind the first."""
        inner = t[0].numel()
        v = buf.as_strided(t.shape, (far,) + tuple(t[0].stride()))
        assert inner <= buf.numel() - far
        v.copy_(t)
        return v

    x, w = g.normal(2, L, D, dtype=BF), g.normal(D, 4, std=0.5)
    want, _ = la.la_short_conv(x, w)
    got, _ = la.la_short_conv(spread(x), w)
    assert torch.equal(want, got)
    out = buf.as_strided(x.shape, (far, D, 1))
    buf.zero_()
    la.la_short_conv(x, w, y=out)
    assert torch.equal(want, out)
    a, _ = scan_inputs((2, L, D, N, None, False, False, True, True, False, True), BF, 72)
    args = lambda u: (u, a["dt"], a["A"], a["B"], a["C"])  # noqa: E731
    kw = dict(D=a["D"], dt_bias=a["dt_bias"])
    want = la.la_ssm_scan(*args(a["u"]), **kw)
    got = la.la_ssm_scan(*args(spread(a["u"])), **kw)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    want = la.la_ssm_scan_bwd(*args(a["u"]), a["dy"], **kw)
    got = la.la_ssm_scan_bwd(*args(spread(a["u"])), a["dy"], **kw)
    for r, t in zip(want, got):
        assert r is None or torch.equal(r, t)
    rows, nw = g.normal(2, 512, dtype=BF), 1 + g.normal(512, std=0.1)
    want = la.la_add_norm(rows, nw)
    got = la.la_add_norm(spread(rows), nw)
    assert torch.equal(want[0], got[0]) and torch.equal(want[2], got[2])
    del buf, got, out
    S = (1 << 31) // (N * D) + 3  # the last slots start behind 2^31 elements
    pool = torch.empty(S, N, D, device="cuda")
    st = g.normal(2, N, D)
    pool[0], pool[S - 1] = st[0], st[1]
    one = [v[:, 0] if v.dim() == 3 else v for v in args(a["u"])]
    y0 = la.la_ssm_step(*one, st, **kw)
    y1 = la.la_ssm_step(*one, pool, slots=ints([0, S - 1]), **kw)
    assert torch.equal(y0, y1) and torch.equal(pool[S - 1], st[1]) and torch.equal(pool[0], st[0])


def test_scan_backward_of_the_most_channels():
    """The widest batch there is, at a state size that takes the sums past 2^32 threads: channels from the start, the
    middle and the end against the oracle on those channels alone (what is summed over channels is left out)."""
    note("scan backward, 2^25 channels")
    D, N = 1 << 25, 33
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    rnd = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    u, dt, dy = rnd(1, 1, D), rnd(1, 1, D), rnd(1, 1, D)
    Bm, C = rnd(1, 1, N), rnd(1, 1, N)
    A = torch.rand(D, N, generator=g, device="cuda").neg_()
    s_in = torch.rand(1, N, D, generator=g, device="cuda")
    du, ddt, dA, _, _, _, _, _, ds_in = la.la_ssm_scan_bwd(u, dt, A, Bm, C, dy, s_in=s_in)
    at = torch.cat([torch.arange(k, k + 70) for k in (0, (1 << 24) - 3, D - 70)]).cuda()
    pick = lambda t: R.f64(t[..., at])  # noqa: E731
    args = (pick(u), pick(dt), R.f64(A[at]), R.f64(Bm), R.f64(C), None, None, None, pick(s_in), None, True, pick(dy),
            np.zeros((1, N, 210)))
    r, m = R.scan_bwd(*args), R.scan_bwd(*args, mag=True)
    for name, got, k in (("du", du[..., at], 0), ("ddt", ddt[..., at], 1), ("dA", dA[at], 2), ("ds_in", ds_in[..., at], 8)):
        R.close(got, r[k], m[k], 8 + 64, F32, name)


# ------------------------------------------------------------------------------------ norm

NORM = [(1, 8, False), (3, 64, False), (5, 1000, False), (2, 7, False), (4, 130, True), (9, 2048, False), (2, 2056, True),
        (3, 4096, False), (1, 8200, False), (2, 16384, False), (700, 96, False), (0, 64, False), (2, 1, False)]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,D,strided", NORM)
@pytest.mark.parametrize("add", [True, False])
def test_norm_forward_and_backward(M, D, strided, add, dtype):
    note(f"norm {M} {D} {strided} {add} {dtype}")
    g = Draw(M + D)
    make = g.wide if strided else g.normal
    x, res = make(M, D, dtype=dtype), make(M, D, std=2.0, dtype=dtype) if add else None
    w = 1 + g.normal(D, std=0.2)
    if M > 1:
        x[1] = 0.0  # a row of zeros: 1 / sqrt(eps) times zero
        if add:
            res[1] = 0.0
    y, h, r = la.la_add_norm(x, w, res, eps=1e-5)
    ry, rh, rr = R.norm(R.f64(x), R.f64(res), R.f64(w), 1e-5)
    K = D / 8 + 32
    R.close(y, ry, np.abs(ry), K, dtype, "y")
    R.close(h, rh, np.abs(rh), 1, dtype, "h")
    R.close(r, rr, np.abs(rr), K, F32, "rstd")
    if not add:
        assert h is x
    # the sum written over the residual, and over x
    if add and M:
        for over in ("res", "x"):
            x2, r2 = x.clone(), res.clone()
            y2, h2, _ = la.la_add_norm(x2, w, r2, eps=1e-5, h=r2 if over == "res" else x2)
            assert torch.equal(y2, y) and torch.equal(h2, h)
    dy, dh = make(M, D, dtype=dtype), g.normal(M, D, dtype=dtype) if add else None
    dx, dw = la.la_add_norm_bwd(dy, h, w, r, dh)
    args = (R.f64(dy), R.f64(h), R.f64(w), R.f64(r), R.f64(dh))
    (rx, rw), (mx, mw) = R.norm_bwd(*args), R.norm_bwd(*args, mag=True)
    R.close(dx, rx, mx, K, dtype, "dx")
    R.close(dw, rw, mw, K + M, F32, "dw")
    if add and M:
        dx2, _ = la.la_add_norm_bwd(dy, h, w, r, dh, dx=dh)
        assert dx2.data_ptr() == dh.data_ptr() and torch.equal(dx2, dx)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,D,group", [(1, 128, 0), (3, 256, 32), (2, 64, 64), (5, 2048, 128), (4, 1000, 0), (2, 4224, 128),
                                       (3, 16384, 0), (2, 7, 0), (6, 96, 32)])
def test_norm_q8(M, D, group, dtype):
    note(f"norm q8 {M} {D} {group} {dtype}")
    g = Draw(D)
    x, res, w = g.normal(M, D, dtype=dtype), g.normal(M, D, dtype=dtype), 1 + g.normal(D, std=0.2)
    if M > 1:
        x[1] = 0.0
        res[1] = 0.0
    if M > 2:
        x[2] *= 1e-22  # y of about 1e-20: a subnormal scale is not reached, a tiny one is
        res[2] = 0.0
    q, s, h, r = la.la_add_norm_q8(x, w, res, group=group)
    ry, rh, rr = R.norm(R.f64(x), R.f64(res), R.f64(w), 1e-5)
    K = D / 8 + 32
    R.close(h, rh, np.abs(rh), 1, dtype, "h")
    R.close(r, rr, np.abs(rr), K, F32, "rstd")
    gs = group or D
    amax = np.abs(ry).reshape(M, D // gs, gs).max(2)
    rs = np.where(amax > 0, amax / 448, 1.0)
    R.close(s, rs, rs, K + 2, F32, "scale")
    # value(q) against y / scale: half a step (2^-4 of the value, 2^-10 below the normal range) and K roundings
    v = ry / np.repeat(rs, gs, 1).reshape(M, D)
    got = q.to(torch.float32).cpu().double().numpy()
    tol = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) + (K + 4) * R.U * np.abs(v)
    assert (np.abs(got - v) <= tol).all(), np.abs(got - v).max()
    assert np.abs(got).max() <= 448


def test_norm_nonfinite_rows_stay_apart():
    note("norm non-finite rows")
    g = Draw(1)
    x, w = g.normal(6, 256), 1 + g.normal(256, std=0.1)
    clean, _, _ = la.la_add_norm(x, w)
    cq, cs, _, _ = la.la_add_norm_q8(x, w, group=64)
    x[1, 3], x[4, 200] = float("nan"), float("inf")
    y, _, r = la.la_add_norm(x, w)
    q, s, _, _ = la.la_add_norm_q8(x, w, group=64)
    for i in (0, 2, 3, 5):
        assert torch.equal(y[i], clean[i]) and torch.equal(s[i], cs[i])
        assert torch.equal(q[i].view(torch.uint8), cq[i].view(torch.uint8))
    assert torch.isnan(y[1]).all() and torch.isnan(r[1]) and torch.isnan(s[1]).all()
    assert not torch.isfinite(s[4, 3])


# ------------------------------------------------------------------------------------ together


def layer(D, N, W, seed, q8=None):
    """(params, project_in, project_dbc, weights): a layer whose two projections are fp32 products."""
    g = Draw(seed)
    p = pipeline.SelectiveParams(1 + g.normal(D, std=0.1), g.normal(D, W, std=0.5), g.normal(D, std=0.1),
                                 -g.uniform(D, N, lo=0.5, hi=8.0), g.normal(D), g.uniform(D, lo=-5.0, hi=-2.0), q8_group=q8)
    wx, wp = g.normal(D, 2 * D, std=D ** -0.5), g.normal(D, D + 2 * N, std=D ** -0.5)

    def project_in(y):
        if q8 is not None:  # dequantised: value times its group's scale
            q, scale = y
            y = (q.float().view(q.shape[0], scale.shape[1], -1) * scale[:, :, None]).view(q.shape)
        xz = (y.float() @ wx).to(torch.bfloat16 if q8 is not None else y.dtype)
        return xz[..., :D], xz[..., D:]

    def project_dbc(v):
        t = (v.float() @ wp).to(v.dtype)
        return t[..., :D], t[..., D : D + N], t[..., D + N :]

    return p, project_in, project_dbc, wx, wp


def test_layer_prompt_then_tokens_equals_one_prompt():
    """A padded batch of prompts of unequal lengths, then single tokens from its states in a pool, gives what each
    sequence gives as one prompt.  In fp32, where the two orders differ by roundings: 8 L + 64 of 2^-24, and as much
    again for each of the two fp32 projections between (sums of D = 64)."""
    note("layer: prompts, then tokens")
    B, L, D, N, W, T = 3, 150, 64, 16, 4, 6
    p, pin, pdbc, _, _ = layer(D, N, W, 40)
    g = Draw(41)
    x, res = g.normal(B, L + T, D), g.normal(B, L + T, D)
    lens = [150, 3, 97]
    o, _, cs, so = pipeline.selective_prompt(p, x[:, :L].contiguous(), res[:, :L].contiguous(), pin, pdbc, lengths=ints(lens))
    conv_pool, pool = torch.zeros(5, W - 1, D, device="cuda"), torch.zeros(5, N, D, device="cuda")
    at = torch.tensor([4, 0, 2], device="cuda")
    conv_pool[at], pool[at] = cs, so
    slots = at.to(torch.int32)
    rows = []
    for k in range(T):
        xt = torch.stack([x[i, lens[i] + k] for i in range(B)])
        rt = torch.stack([res[i, lens[i] + k] for i in range(B)])
        rows.append(pipeline.selective_token(p, xt, rt, pin, pdbc, conv_pool, pool, slots)[0])
    for i in range(B):
        n = lens[i] + T
        one, _, c1, s1 = pipeline.selective_prompt(p, x[i : i + 1, :n].contiguous(), res[i : i + 1, :n].contiguous(), pin, pdbc)
        tol = 3 * (8 * n + 64) * R.U * float(one.abs().max()) * 8
        assert float((one[0, : lens[i]] - o[i, : lens[i]]).abs().max()) <= tol
        for k in range(T):
            assert float((one[0, lens[i] + k] - rows[k][i]).abs().max()) <= tol, (i, k)
        assert float((s1[0] - pool[at[i]]).abs().max()) <= 3 * (8 * n + 64) * R.U * float(s1.abs().max()) * 8
        assert float((c1[0] - conv_pool[at[i]]).abs().max()) <= 64 * 3 * R.U * float(c1.abs().max()) * 8


def test_layer_in_pieces_equals_one_prompt():
    """A prompt in two pieces, the second from the first's states, against the whole; 8-bit norm output.  Rows are
    normed, quantised and projected one by one, so only the scan's order of sums differs: in bf16 a state that
    differs by a rounding of fp32 may move an output to the neighbouring bf16 value, one step of 2^-7 relative."""
    note("layer: pieces, 8 bits")
    B, L, D, N, W = 2, 260, 128, 16, 4
    p, pin, pdbc, _, _ = layer(D, N, W, 44, q8=32)
    g = Draw(45)
    x, res = g.normal(B, L, D, dtype=BF), g.normal(B, L, D, dtype=BF)
    o, h, cs, so = pipeline.selective_prompt(p, x, res, pin, pdbc)
    k = 101
    a = pipeline.selective_prompt(p, x[:, :k].contiguous(), res[:, :k].contiguous(), pin, pdbc)
    b = pipeline.selective_prompt(p, x[:, k:].contiguous(), res[:, k:].contiguous(), pin, pdbc, conv_state=a[2], s_in=a[3])
    got = torch.cat([a[0], b[0]], 1).double()
    ref = o.double()
    assert ((got - ref).abs() <= 2.0 ** -7 * ref.abs() + 3 * (8 * L + 64) * R.U * float(ref.abs().max()) * 8).all()
    assert torch.equal(torch.cat([a[1], b[1]], 1), h) and torch.equal(b[2], cs)
    assert float((b[3] - so).abs().max()) <= 3 * (8 * L + 64) * R.U * float(so.abs().max()) * 8


@pytest.mark.parametrize("B,L", [(0, 5), (2, 0)])
def test_layer_of_no_tokens(B, L):
    """An empty batch and prompts of no tokens: states pass through, gradients of the parameters are zero."""
    note(f"layer: {B} prompts of {L}")
    D, N, W = 64, 16, 4
    p, pin, pdbc, _, _ = layer(D, N, W, 60)
    g = Draw(61)
    x, cs, s = g.normal(B, L, D), g.normal(B, W - 1, D), g.normal(B, N, D)
    saved = {}
    o, h, c1, s1 = pipeline.selective_prompt(p, x, x, pin, pdbc, conv_state=cs, s_in=s, saved=saved)
    assert o.shape == (B, L, D) and h.shape == (B, L, D) and torch.equal(c1, cs) and torch.equal(s1, s)
    gr = pipeline.selective_backward(p, saved, o, lambda ddt, dB, dC: ddt, lambda du, dz: du.reshape(B * L, D),
                                     d_conv_state=cs, ds_out=s)
    assert gr["dx"].shape == (B, L, D) and torch.equal(gr["conv_state"], cs) and torch.equal(gr["s_in"], s)
    for k in ("norm_weight", "conv_weight", "conv_bias", "A", "skip", "dt_bias"):
        assert (gr[k] == 0).all(), k


def test_layer_gradients_against_differences():
    """selective_backward's gradients of a scalar against differences of selective_prompt itself, in fp32, along one
    random direction per argument (the step and the bound as in the scan's own test)."""
    note("layer: gradients")
    B, L, D, N, W = 2, 70, 64, 16, 4
    p, pin, pdbc, wx, wp = layer(D, N, W, 47)
    g = Draw(48)
    lens = ints([70, 33])
    a = dict(x=g.normal(B, L, D), res=g.normal(B, L, D), cs=g.normal(B, W - 1, D), s=g.normal(B, N, D))
    live = (torch.arange(L, device="cuda")[None] < lens[:, None])[..., None]
    dy, dh = g.normal(B, L, D) * live, g.normal(B, L, D)
    dcs, ds = g.normal(B, W - 1, D), g.normal(B, N, D)
    names = dict(norm_weight="norm_weight", conv_weight="conv_weight", conv_bias="conv_bias", A="A", skip="skip", dt_bias="dt_bias")

    def loss(a, p):
        o, h, c, s = pipeline.selective_prompt(p, a["x"], a["res"], pin, pdbc, conv_state=a["cs"], s_in=a["s"], lengths=lens)
        o = torch.where(live, o, torch.zeros_like(o))
        return float(sum((t.double() * d.double()).sum() for t, d in ((o, dy), (h, dh), (c, dcs), (s, ds))))

    saved = {}
    pipeline.selective_prompt(p, a["x"], a["res"], pin, pdbc, conv_state=a["cs"], s_in=a["s"], lengths=lens, saved=saved)
    gr = pipeline.selective_backward(
        p, saved, dy, lambda ddt, dB, dC: torch.cat([ddt, dB, dC], -1) @ wp.t(),
        lambda du, dz: torch.cat([du, dz], -1).view(B * L, -1) @ wx.t(), dh=dh, d_conv_state=dcs, ds_out=ds)
    want = dict(x=gr["dx"], res=gr["dx"], cs=gr["conv_state"], s=gr["s_in"])
    e = 2.0 ** -7
    for k in list(a) + list(names):
        base = a[k] if k in a else getattr(p, k)
        grad = want[k] if k in a else gr[names[k]]
        v = g.normal(*base.shape)
        vals = []
        for sign in (1, -1):
            if k in a:
                vals.append(loss(dict(a, **{k: base + sign * e * v}), p))
            else:
                vals.append(loss(a, dataclasses.replace(p, **{k: base + sign * e * v})))
        diff = (vals[0] - vals[1]) / (2 * e)
        dot = float((grad.double() * v.double()).sum())
        scale = float((grad.double().abs() * v.double().abs()).sum())
        assert abs(diff - dot) <= 1e-2 * scale / np.sqrt(v.numel()) + 1e-3 * scale, (k, diff, dot, scale)


def test_layer_in_a_graph_and_on_two_streams():
    """The layer captured and replayed with new inputs, eager work between the replays; and on two streams at once."""
    note("layer: graph and streams")
    B, L, D, N, W = 2, 300, 128, 16, 4
    p, pin, pdbc, wx, wp = layer(D, N, W, 50)
    g = Draw(51)
    xs = [(g.normal(B, L, D, dtype=BF), g.normal(B, L, D, dtype=BF), g.normal(B, L, D, dtype=BF)) for _ in range(4)]
    zero = torch.zeros(B, N, D, device="cuda")

    def both(x, res, dy):
        saved = {}
        out = pipeline.selective_prompt(p, x, res, pin, pdbc, s_in=zero, saved=saved)
        gr = pipeline.selective_backward(
            p, saved, dy, lambda ddt, dB, dC: (torch.cat([ddt, dB, dC], -1).float() @ wp.t()).to(BF),
            lambda du, dz: (torch.cat([du, dz], -1).view(B * L, -1).float() @ wx.t()).to(BF), dh=x)
        return list(out) + [t for t in gr.values() if t is not None]

    eager = [both(*x) for x in xs]
    torch.cuda.synchronize()
    ins = [t.clone() for t in xs[0]]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both(*ins)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both(*ins)
    for k in (1, 2, 3, 0):
        for t, v in zip(ins, xs[k]):
            t.copy_(v)
        graph.replay()
        other = both(*xs[(k + 1) % 4])  # eager work between replays
        torch.cuda.synchronize()
        for a, b in zip(outs, eager[k]):
            assert torch.equal(a, b)
        for a, b in zip(other, eager[(k + 1) % 4]):
            assert torch.equal(a, b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for st, x in ((s1, xs[1]), (s2, xs[2])):
        with torch.cuda.stream(st):
            got.append(both(*x))
    torch.cuda.synchronize()
    for a, b in itertools.chain(zip(got[0], eager[1]), zip(got[1], eager[2])):
        assert torch.equal(a, b)


def test_stream_argument():
    """``stream=`` enqueues and allocates on that stream."""
    note("stream argument")
    g = Draw(60)
    x, w = g.normal(64, 256, dtype=BF), 1 + g.normal(256, std=0.1)
    want, _, _ = la.la_add_norm(x, w)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    y, _, _ = la.la_add_norm(x, w, stream=st)
    st.synchronize()
    assert torch.equal(y, want)


def test_traced_kernels():
    note("traces")
    g = Draw(61)
    timer = la.KernelTimer()
    x, w = g.normal(2, 40, 64, dtype=BF), g.normal(64, 4)
    la.la_short_conv_bwd(x, w, x.clone(), timer=timer)
    torch.cuda.synchronize()
    names = [n for n, ms in timer.harvest()]
    assert names == ["short_conv_bwd", "short_conv_bwd_sums"]


def test_token_step_in_two_graphs():
    """Single tokens captured into two graphs of one memory pool, replayed in turn with other inputs and other slots (a
    padding row and a slot named twice among them), eager steps on a second pool of states between: every replay gives
    what the eager step gives."""
    note("token: graphs")
    D, N, W, S = 128, 16, 4, 6
    p, pin, pdbc, _, _ = layer(D, N, W, 70)
    g = Draw(71)
    pools = [g.normal(S, W - 1, D), g.normal(S, N, D)]
    mine = [t.clone() for t in pools]
    shapes = [3, 5]
    graphs, bufs, mem = [], [], None
    for B in shapes:
        b = dict(x=g.normal(B, D), res=g.normal(B, D), slots=torch.full((B,), -1, dtype=torch.int32, device="cuda"))
        pipeline.selective_token(p, b["x"], b["res"], pin, pdbc, *mine, b["slots"])  # all padding: changes no state
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, pool=mem):
            b["y"], b["h"] = pipeline.selective_token(p, b["x"], b["res"], pin, pdbc, *mine, b["slots"])
        mem = mem or gr.pool()
        graphs.append(gr)
        bufs.append(b)
    for t, m in zip(pools, mine):
        assert torch.equal(t, m)
    turns = [(0, [4, 0, 2]), (1, [5, 1, -1, 3, 1]), (0, [0, 0, 9]), (1, [0, 1, 2, 3, 4]), (0, [5, 4, 3])]
    for k, slots in turns:
        b = bufs[k]
        x, res = g.normal(*b["x"].shape), g.normal(*b["x"].shape)
        for name, v in (("x", x), ("res", res), ("slots", ints(slots))):
            b[name].copy_(v)
        graphs[k].replay()
        y, h = pipeline.selective_token(p, x, res, pin, pdbc, *pools, ints(slots))
        torch.cuda.synchronize()
        live = [i for i, s in enumerate(slots) if 0 <= s < S and s not in slots[:i]]
        assert torch.equal(b["y"][live], y[live]) and torch.equal(b["h"], h)
        for t, m in zip(pools, mine):
            assert torch.equal(t, m)


def test_scan_on_a_given_stream():
    """stream= for calls with workspaces: two at once on two streams, outputs and scratch of their own."""
    note("scan: stream argument")
    case = (2, 333, 72, 16, None, False, True, True, True, True, True)
    sets = [scan_inputs(case, BF, 80 + i)[0] for i in range(2)]
    args = lambda a: [a[k] for k in ("u", "dt", "A", "B", "C")]  # noqa: E731
    kw = lambda a: {k: a[k] for k in ("D", "z", "dt_bias", "s_in")}  # noqa: E731
    want = [(la.la_ssm_scan(*args(a), **kw(a)), la.la_ssm_scan_bwd(*args(a), a["dy"], **kw(a))) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [(la.la_ssm_scan(*args(a), **kw(a), stream=s), la.la_ssm_scan_bwd(*args(a), a["dy"], **kw(a), stream=s))
           for a, s in zip(sets, streams)]
    torch.cuda.synchronize()
    for w, v in zip(want, got):
        for a, b in zip(w[0] + w[1], v[0] + v[1]):
            assert torch.equal(a, b)
