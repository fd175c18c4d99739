"""The short convolution, the selective scan and the residual norm where the ordinary cases of test_gpu_mixer.py do not
look: values next to a tie of the 8-bit output, strong decays, values at the ends of fp32's range, padding that is
not finite, and the sizes from which the kernels take their wide forms."""
import numpy as np
import pytest
import torch

import mixer_ref as R
from chunked_scan_amd import binding as la
from chunked_scan_amd import pipeline
from gpu_util import note
from test_gpu_mixer import BF, F32, Draw, cut, ints, layer

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------ norm


def e4m3(v):
    """The nearest e4m3 value, ties to even, of values given in fp64.  A quotient of two fp32 numbers that is not a
    tie of e4m3 differs from it by 2^-29 of its size at least (24 bits against 24 + 5), so fp64's rounding of the
    quotient never makes one."""
    a = np.minimum(np.abs(v), 448.0)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -6))), -6) - 3)
    return np.round(a / step) * step * np.sign(v)


@pytest.mark.parametrize("group", [0, 128])
def test_norm_q8_rounds_the_quotient_itself(group):
    """The codes are the nearest ones to y / scale, y being what la_add_norm gives in fp32 and scale the returned one:
    values within a few fp32 steps of every tie of e4m3, normal and subnormal, at scales over many octaves, are
    rounded to the right side of it."""
    note(f"norm q8 at ties {group}")
    ties = [(m + 0.5) * 2.0 ** -9 for m in range(8)]
    ties += [(8 + m + 0.5) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8) if (8 + m + 0.5) * 2.0 ** (e - 3) < 448]
    base = np.array(ties, np.float32) / np.float32(448.0)
    near = np.concatenate([(base.view(np.int32) + k).view(np.float32) for k in range(-4, 5)])
    near = near[: len(near) // 127 * 127].reshape(-1, 127)  # every group of 128 leads with its largest, 1
    w = torch.from_numpy(np.concatenate([np.ones((len(near), 1), np.float32), near], 1).reshape(-1)).cuda()
    D, M = w.numel(), 96
    g = Draw(5)
    # rows of one value a: r = 1 / sqrt(a^2 + eps), so y / weight moves over many octaves as a falls below sqrt(eps)
    a = torch.exp2(g.uniform(M, lo=-110.0, hi=3.0))
    x = (a[:, None] * torch.where(g.uniform(M, D) < 0.5, -1.0, 1.0)).contiguous()
    y, _, _ = la.la_add_norm(x, w)
    q, s, _, _ = la.la_add_norm_q8(x, w, group=group)
    y, s = y.cpu().numpy(), s.cpu().numpy()
    same = s == np.abs(y).reshape(M, -1, group or D).max(2) / np.float32(448.0)
    assert same.all(), (same.size, same.sum())
    v = y.astype(np.float64) / np.repeat(s.astype(np.float64), group or D, 1)
    same = q.to(F32).cpu().double().numpy() == e4m3(v)
    assert same.all(), (same.size, same.sum())


@pytest.mark.parametrize("group", [0, 32])
def test_norm_q8_scale_that_underflows(group):
    """Where the largest |y| / 448 is zero in fp32 the scale is 1 and the codes are zero, also for values that are not
    zero themselves (subnormal ones); next to such a group an ordinary one."""
    note(f"norm q8 underflow {group}")
    w = torch.full((64,), 1e-44, device="cuda")
    if group:
        w[32:] = 1.0
    x = Draw(9).normal(5, 64)
    q, s, _, _ = la.la_add_norm_q8(x, w, group=group)
    tiny = 32 if group else 64
    assert (s[:, 0] == 1).all() and (q[:, :tiny].float() == 0).all()
    if group:
        assert (s[:, 1] < 1).all() and (q[:, 32:].float().abs().amax(1) == 448).all()


def test_norm_with_a_subnormal_eps():
    """Rows of zeros and a row of ones with an eps below fp32's normal range: 1 / sqrt(eps) is finite, and zeros stay
    zeros.  K as in test_gpu_mixer.py."""
    note("norm: subnormal eps")
    eps = float(np.float32(1e-40))
    x = torch.zeros(3, 64, device="cuda")
    x[1] = 1.0
    w = 1 + Draw(2).normal(64, std=0.1)
    y, _, r = la.la_add_norm(x, w, eps=eps)
    ry, _, rr = R.norm(R.f64(x), None, R.f64(w), eps)
    R.close(y, ry, np.abs(ry), 64 / 8 + 32, F32, "y")
    R.close(r, rr, np.abs(rr), 64 / 8 + 32, F32, "rstd")


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [7, 64, 4096, 16384])
def test_norm_of_values_whose_squares_overflow(D, dtype):
    """Rows of 1e19 to 1e37 between ordinary ones: the statistics hold, forward, 8 bits and backward.  K as in
    test_gpu_mixer.py."""
    note(f"norm: large values {D} {dtype}")
    g = Draw(D)
    M = 6
    scale = torch.tensor([1.0, 1e25, 1.0, 1e36, 1e19, 1e30], device="cuda")[:, None]
    x, w = (g.normal(M, D) * scale).to(dtype), 1 + g.normal(D, std=0.2)
    y, h, r = la.la_add_norm(x, w)
    ry, _, rr = R.norm(R.f64(x), None, R.f64(w), 1e-5)
    K = D / 8 + 32
    R.close(y, ry, np.abs(ry), K, dtype, "y")
    assert (np.abs(R.f64(r) - rr) <= (K + 1) * R.U * rr).all()
    q, s, _, r8 = la.la_add_norm_q8(x, w)
    assert torch.equal(r8, r)
    top = np.abs(ry).max(1, keepdims=True) / 448
    assert (np.abs(R.f64(s) - top) <= (K + 3) * R.U * top).all()
    dy = g.normal(M, D, dtype=dtype)
    dx, dw = la.la_add_norm_bwd(dy, h, w, r)
    args = (R.f64(dy), R.f64(h), R.f64(w), R.f64(r), None)
    (rx, rw), (mx, mw) = R.norm_bwd(*args), R.norm_bwd(*args, mag=True)
    R.close(dx, rx, mx, K, dtype, "dx")
    R.close(dw, rw, mw, K + M, F32, "dw")


# ------------------------------------------------------------------------------------ scan


def scan_bwd_bounds(a, s_in, ds_out):
    """dA [D, N] and ddt [L, D] of one sequence in fp64, each with a bound on what fp32 arithmetic that forms them as the
    formulas say may be off by.  Errors are carried through the recurrences to first order, u = 2^-24: a step size
    is off by 8 u of itself; a decay exp(delta A) by 8 u plus the rounding of its exponent, (8 + L) u |delta A| with up to
    L step sizes summed before the product, and by 2^-126 where it leaves fp32's normal range; every sum or product
    by u of its result, a sum over N or L terms by as many."""
    f = {k: R.f64(v) for k, v in a.items()}
    u = R.U
    L, D = f["u"].shape[1:]
    N = f["A"].shape[1]
    A = f["A"].T
    S, E = R.f64(s_in)[0], np.zeros((N, D))
    kept = []
    for t in range(L):
        x = f["dt"][0, t] + f["dt_bias"]
        dl = R.softplus(x)
        dec, b = np.exp(dl * A), f["B"][0, t][:, None] * (dl * f["u"][0, t])
        rho = (8 + (8 + L) * np.abs(dl * A)) * u
        kept.append((S, E, x, dl, dec, rho))
        E = dec * E + np.abs(S) * (dec * rho + 2.0 ** -126) + 11 * u * np.abs(b)
        S = dec * S + b
        E = E + u * np.abs(S)
    G, F = R.f64(ds_out)[0], np.zeros((N, D))
    dA, dAe = np.zeros((N, D)), np.zeros((N, D))
    ddt, ddte = np.zeros((L, D)), np.zeros((L, D))
    for t in range(L - 1, -1, -1):
        S, E, x, dl, dec, rho = kept[t]
        B = f["B"][0, t][:, None]
        z, dy = f["z"][0, t], f["dy"][0, t]
        c = f["C"][0, t][:, None] * (dy * R.silu(z))
        F = F + 16 * u * np.abs(c)
        G = G + c
        F = F + u * np.abs(G)
        gw = G * dec * S
        gwe = F * dec * np.abs(S) + np.abs(G) * (np.abs(S) * (dec * rho + 2.0 ** -126) + dec * E) + 4 * u * np.abs(gw)
        dA += gw * dl
        dAe += (gwe + (L + 10) * u * np.abs(gw)) * dl
        ut = f["u"][0, t]
        terms, termse = G * B * ut + gw * A, F * np.abs(B * ut) + gwe * np.abs(A)
        termse = termse + (N + 8) * u * (np.abs(G * B * ut) + np.abs(gw * A))
        sg = R.sig(x)
        ddt[t], ddte[t] = terms.sum(0) * sg, termse.sum(0) * sg + 8 * u * np.abs(terms.sum(0) * sg)
        G, F = G * dec, F * dec + np.abs(G) * (dec * rho + 2.0 ** -126) + u * np.abs(G * dec)
    return dA.T, 1.01 * dAe.T, ddt, 1.01 * ddte


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,most", [(8, 12.0), (8, 32.0), (16, 32.0), (24, 60.0), (64, 64.0)])
def test_scan_backward_under_strong_decay(N, most, dtype):
    """Step sizes around 1.3 and rates to -most: a token leaves next to nothing of the state before it, and the
    derivatives that go through that remainder keep their relative accuracy, element by element.  (mixer_ref.scan_bwd's
    magnitudes are too wide to see that: they also hold for the remainder formed as S_t - delta u B.)"""
    note(f"scan backward: strong decay {N} {most} {dtype}")
    g = Draw(90 + N)
    L, D = 40, 72
    a = dict(u=g.normal(1, L, D, dtype=dtype), dt=g.normal(1, L, D, std=0.5, dtype=dtype),
             A=-g.uniform(D, N, lo=0.5, hi=most), B=g.normal(1, L, N, dtype=dtype), C=g.normal(1, L, N, dtype=dtype),
             D=g.normal(D), z=g.normal(1, L, D, dtype=dtype), dt_bias=g.uniform(D, lo=0.5, hi=1.5))
    s_in, ds_out = g.normal(1, N, D), g.normal(1, N, D)
    a["dy"] = g.normal(1, L, D, dtype=dtype)
    _, ddt, dA, *_ = la.la_ssm_scan_bwd(a["u"], a["dt"], a["A"], a["B"], a["C"], a["dy"], D=a["D"], z=a["z"],
                                        dt_bias=a["dt_bias"], s_in=s_in, ds_out=ds_out)
    rA, eA, rdt, edt = scan_bwd_bounds(a, s_in, ds_out)
    for name, got, ref, err, t in (("dA", dA, rA, eA, F32), ("ddt", ddt[0], rdt, edt, dtype)):
        off = np.abs(R.f64(got) - ref)
        bad = ~(off <= R.HALF[t] * np.abs(ref) + err * (1 + R.HALF[t]))
        assert not bad.any(), (name, int(bad.sum()), bad.size, float((off / (np.abs(ref) + 1e-300))[bad].max()))


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_scan_with_step_sizes_of_zero(dtype):
    """dt of minus infinity and of the type's lowest value through softplus: a step size of zero, which leaves the state
    alone and whose derivatives are zero; forward, backward and one token.  K as in test_gpu_mixer.py."""
    note(f"scan: step sizes of zero {dtype}")
    B, L, D, N = 2, 70, 72, 16
    g = Draw(33)
    u, dy, z = (g.normal(B, L, D, dtype=dtype) for _ in range(3))
    dt, Bm, C = g.normal(B, L, D, std=0.5, dtype=dtype), g.normal(B, L, N, dtype=dtype), g.normal(B, L, N, dtype=dtype)
    dt[0, 5:9], dt[:, 30, ::2], dt[1, 40:] = -float("inf"), torch.finfo(dtype).min, -float("inf")
    A, bias, skip = -g.uniform(D, N, lo=0.5, hi=8.0), g.uniform(D, lo=-4.0, hi=0.0), g.normal(D)
    s_in, ds_out = g.normal(B, N, D), g.normal(B, N, D)
    kw = dict(D=skip, z=z, dt_bias=bias, s_in=s_in)
    y, so = la.la_ssm_scan(u, dt, A, Bm, C, **kw)
    got = la.la_ssm_scan_bwd(u, dt, A, Bm, C, dy, ds_out=ds_out, **kw)
    args = (R.f64(u), R.f64(dt), R.f64(A), R.f64(Bm), R.f64(C), R.f64(skip), R.f64(z), R.f64(bias), R.f64(s_in), None, True)
    K = 8 * L + 64
    (ry, rs, _), (my, ms, _) = R.scan(*args), R.scan(*args, mag=True)
    R.close(y, ry, my, K, dtype, "y")
    R.close(so, rs, ms, K, F32, "s_out")
    r, m = R.scan_bwd(*args, R.f64(dy), R.f64(ds_out)), R.scan_bwd(*args, R.f64(dy), R.f64(ds_out), mag=True)
    extra = dict(dA=B * L, dB=D, dC=D, dD=B * L, d_dt_bias=B * L)
    for k, name in enumerate(("du", "ddt", "dA", "dB", "dC", "dD", "dz", "d_dt_bias", "ds_in")):
        t = F32 if name in ("dA", "dD", "d_dt_bias", "ds_in") else dtype
        R.close(got[k], r[k], m[k], 2 * K + extra.get(name, 0), t, name)
    assert (got[1][0, 5:9] == 0).all() and (got[1][1, 40:] == 0).all()
    st = s_in.clone()
    la.la_ssm_step(u[:, 5], dt[:, 50], A, Bm[:, 5], C[:, 5], st, D=skip, z=z[:, 5], dt_bias=bias)
    assert torch.equal(st[1], s_in[1])


# ------------------------------------------------------------------------------------ together


@pytest.mark.parametrize("value", [float("nan"), float("inf")], ids=["nan", "inf"])
@pytest.mark.parametrize("q8", [None, 0, 32])
def test_layer_with_padding_that_is_not_finite(q8, value):
    """Rows behind a sequence's length hold NaN or infinities, as in a batch of uninitialised memory: outputs, states
    and every derivative, the projections' own (products over all rows) among them, are what they are with zeros
    there."""
    note(f"layer: padding of {value}, q8 {q8}")
    B, L, D, N, W = 3, 40, 64, 16, 4
    p, pin, pdbc, wx, wp = layer(D, N, W, 47, q8=q8)
    g = Draw(48)
    lens = [40, -1, 17]
    live = (torch.arange(L)[None] < torch.tensor(lens)[:, None])[..., None].cuda()
    x, res, dy, dh = (g.normal(B, L, D) for _ in range(4))
    taken = []

    def project_in(y):
        taken.append(y if q8 is None else (y[0].float().view(B * L, y[1].shape[1], -1) * y[1][:, :, None]).view(B * L, D))
        return pin(y)

    def run(fill):
        put = lambda t: torch.where(live, t, torch.full_like(t, fill))  # noqa: E731
        e = torch.float32 if q8 is None else torch.bfloat16
        saved = {}
        o, h, c, s = pipeline.selective_prompt(p, put(x).to(e), put(res).to(e), project_in, pdbc, lengths=ints(lens), saved=saved)
        d_in = []

        def in_backward(du, dz):
            d_in.append(torch.cat([du, dz], -1).view(B * L, -1).float())
            return (d_in[0] @ wx.t()).to(e)

        dbc_backward = lambda ddt, dB, dC: (torch.cat([ddt, dB, dC], -1).float() @ wp.t()).to(e)  # noqa: E731
        gr = pipeline.selective_backward(p, saved, put(dy).to(e), dbc_backward, in_backward, dh=dh.to(e))
        out = [torch.where(live, h, torch.zeros_like(h)), o, c, s, taken[-1].float().t() @ d_in[0]]
        return out + [gr[k] for k in sorted(gr) if gr[k] is not None]

    want, got = run(0.0), run(value)
    for k, (a, b) in enumerate(zip(want, got)):
        assert torch.isfinite(b).all() and torch.equal(a, b), k


# ------------------------------------------------------------------------------------ the wide forms


def chosen(D, n=24, seed=3):
    """n channels: the ends, and some between (channels do not meet in the convolution or the scan's states)."""
    rng = np.random.default_rng(seed)
    return torch.from_numpy(np.unique(np.concatenate([[0, 1, D - 2, D - 1], rng.integers(0, D, n - 4)]))).cuda()


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,L,D,W,lengths", [
    (1, 1100, 16384, 4, None),            # vectors: tiles of 16 tokens forward, 32 back, a remainder of 12
    (2, 1077, 4095, 3, [1077, 530]),      # one channel a thread
    (2, 1077, 8192, 2, [-5, 1061]),
    (40, 33, 16384, 4, None),             # a tile and a token
])
def test_conv_in_long_tiles(B, L, D, W, lengths, dtype):
    """Sizes from which a thread walks 16 tokens forward and 32 back, on some of the channels."""
    note(f"conv in long tiles {B} {L} {D} {W} {lengths} {dtype}")
    g = torch.Generator(device="cuda")
    g.manual_seed(L + D)
    rnd = lambda *s, e=F32: torch.randn(s, generator=g, device="cuda").to(e)  # noqa: E731
    x, dy = rnd(B, L, D, e=dtype), rnd(B, L, D, e=dtype)
    w, b, st, dso = rnd(D, W) * 0.6, rnd(D), rnd(B, W - 1, D, e=dtype), rnd(B, W - 1, D, e=dtype)
    n = cut(lengths, L)
    y, so = la.la_short_conv(x, w, b, st, lengths=ints(lengths), y=torch.zeros_like(x), want_state=True)
    got = la.la_short_conv_bwd(x, w, dy, b, st, dso, lengths=ints(lengths))
    at = chosen(D)
    p = lambda t: R.f64(t[..., at])  # noqa: E731
    args = (p(x), R.f64(w[at]), R.f64(b[at]), p(st), n, True)
    K = W + 28
    ref, ref_so = R.conv(*args)
    mag, _ = R.conv(*[np.abs(v) if i < 4 else v for i, v in enumerate(args[:5])], False)
    R.close(y[..., at], ref, mag, K, dtype, "y")
    assert np.array_equal(p(so), ref_so)
    r, m = R.conv_bwd(*args, p(dy), p(dso)), R.conv_bwd(*args, p(dy), p(dso), mag=True)
    R.close(got[0][..., at], r[0], m[0], 2 * K, dtype, "dx")
    R.close(got[1][at], r[1], m[1], 2 * K + B * L, F32, "dw")
    R.close(got[2][at], r[2], m[2], 2 * K + B * L, F32, "db")
    R.close(got[3][..., at], r[3], m[3], 2 * K, dtype, "d_state")


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,D,N,gate", [(258, 4096, 16, True), (300, 2100, 17, False), (515, 2048, 8, True), (1100, 700, 24, True)])
def test_scan_step_of_many_rows(B, D, N, gate, dtype):
    """Several rows a wave: slots outside the pool, repeated ones next to each other and in other waves, a last wave
    with fewer rows, on some of the channels."""
    note(f"scan step of many rows {B} {D} {N} {dtype}")
    rng = np.random.default_rng(B)
    S = B + 7
    slots = rng.permutation(S)[:B].astype(np.int64)
    slots[1], slots[2], slots[5] = slots[0], -1, S  # neighbours of one wave
    slots[B - 1], slots[B - 2], slots[77] = slots[3], slots[B - 3], -(1 << 31)
    g = torch.Generator(device="cuda")
    g.manual_seed(B)
    rnd = lambda *s, e=F32: torch.randn(s, generator=g, device="cuda").to(e)  # noqa: E731
    u, dt, z = rnd(B, D, e=dtype), rnd(B, D, e=dtype), rnd(B, 2 * D, e=dtype)[:, D:] if gate else None
    Bm, C = rnd(B, N, e=dtype), rnd(B, N, e=dtype)
    A = -8 * torch.rand(D, N, generator=g, device="cuda") - 0.5
    skip, bias, state = rnd(D), rnd(D) - 3, rnd(S, N, D)
    before = state.clone()
    y = torch.full((B, D), 7.0, dtype=dtype, device="cuda")
    la.la_ssm_step(u, dt, A, Bm, C, state, D=skip, z=z, dt_bias=bias, slots=ints(slots.tolist()), y=y)
    first = {}
    for i, s in enumerate(slots):
        if 0 <= s < S:
            first.setdefault(int(s), i)
    rows = torch.tensor(sorted(first.values()), device="cuda")
    rest = torch.tensor(sorted(set(range(B)) - set(first.values())), device="cuda")
    assert len(rest) == 6 and (y[rest] == 7.0).all()
    untouched = torch.tensor(sorted(set(range(S)) - set(first)), device="cuda")
    assert torch.equal(state[untouched], before[untouched])
    at = chosen(D)
    sl = torch.from_numpy(slots).cuda()[rows]
    p = lambda t: None if t is None else R.f64(t[rows][:, at])[:, None]  # noqa: E731
    args = (p(u), p(dt), R.f64(A[at]), R.f64(Bm[rows])[:, None], R.f64(C[rows])[:, None], R.f64(skip[at]), p(z),
            R.f64(bias[at]), R.f64(before[sl][..., at]), None, True)
    ref, so, _ = R.scan(*args)
    mag, mso, _ = R.scan(*args, mag=True)
    R.close(y[rows][:, at], ref[:, 0], mag[:, 0], 72, dtype, "y")
    R.close(state[sl][..., at], so, mso, 72, F32, "state")


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,L,D,N,lengths", [
    (1, 1296, 600, 16, None),         # more than 8192 states, 81 segments of 16 tokens: 4 shares of 20
    (2, 1152, 300, 16, [1151, 1000]), # 72 segments: 4 shares of 18
    (1, 4800, 64, 16, None),          # few states, 300 segments: 16 shares of 19
    (3, 60, 700, 8, [60, 0, 33]),     # more than 8192 states, 3 segments
])
def test_scan_over_many_segments(B, L, D, N, lengths, dtype):
    """The scan over segments with shares of more than 16, which are loaded twice, forward and backward."""
    note(f"scan over many segments {B} {L} {D} {N} {lengths} {dtype}")
    g = torch.Generator(device="cuda")
    g.manual_seed(L)
    rnd = lambda *s, e=F32: torch.randn(s, generator=g, device="cuda").to(e)  # noqa: E731
    u, dt, dy = rnd(B, L, D, e=dtype), 0.5 * rnd(B, L, D), rnd(B, L, D, e=dtype)
    dt = dt.to(dtype)
    Bm, C = rnd(B, L, N, e=dtype), rnd(B, L, N, e=dtype)
    A = -4 * torch.rand(D, N, generator=g, device="cuda") - 0.05
    skip, bias, s_in, ds_out = rnd(D), rnd(D) - 4, rnd(B, N, D), rnd(B, N, D)
    n = cut(lengths, L)
    kw = dict(D=skip, dt_bias=bias, s_in=s_in, lengths=ints(lengths))
    y, so = la.la_ssm_scan(u, dt, A, Bm, C, y=torch.zeros_like(u), **kw)
    got = la.la_ssm_scan_bwd(u, dt, A, Bm, C, dy, ds_out=ds_out, **kw)
    args = (R.f64(u), R.f64(dt), R.f64(A), R.f64(Bm), R.f64(C), R.f64(skip), None, R.f64(bias), R.f64(s_in), n, True)
    K = 8 * L + 64
    ref, ref_so, _ = R.scan(*args)
    mag, mag_so, _ = R.scan(*args, mag=True)
    R.close(y, ref, mag, K, dtype, "y")
    R.close(so, ref_so, mag_so, K, F32, "s_out")
    r, m = R.scan_bwd(*args, R.f64(dy), R.f64(ds_out)), R.scan_bwd(*args, R.f64(dy), R.f64(ds_out), mag=True)
    extra = dict(dA=B * L, dB=D, dC=D, dD=B * L, d_dt_bias=B * L)
    for k, name in enumerate(("du", "ddt", "dA", "dB", "dC", "dD", "dz", "d_dt_bias", "ds_in")):
        if name != "dz":
            t = F32 if name in ("dA", "dD", "d_dt_bias", "ds_in") else dtype
            R.close(got[k], r[k], m[k], 2 * K + extra.get(name, 0), t, name)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,D", [(2051, 512), (4500, 63), (2500, 1024), (700, 4096), (1030, 2056), (530, 16384)])
def test_norm_backward_of_many_rows(M, D, dtype):
    """More rows than one turn of the workgroups takes."""
    note(f"norm backward of many rows {M} {D} {dtype}")
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    rnd = lambda *s, e=F32: torch.randn(s, generator=g, device="cuda").to(e)  # noqa: E731
    h, dy, dh = 2 * rnd(M, D), rnd(M, D, e=dtype), rnd(M, D, e=dtype)
    h, w = h.to(dtype), 1 + 0.2 * rnd(D)
    _, _, r = la.la_add_norm(h, w)
    dx, dw = la.la_add_norm_bwd(dy, h, w, r, dh)
    args = (R.f64(dy), R.f64(h), R.f64(w), R.f64(r), R.f64(dh))
    (rx, rw), (mx, mw) = R.norm_bwd(*args), R.norm_bwd(*args, mag=True)
    K = D / 8 + 32
    R.close(dx, rx, mx, K, dtype, "dx")
    R.close(dw, rw, mw, K + M, F32, "dw")


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_longest_sequences(dtype):
    """2^24 tokens, the most there may be, at the largest state size: the last ones against the oracle.  Step sizes of
    at least softplus(-0.1 - 0.5) = 0.43 and rates of at most -2 leave e^-0.86 a token, so that of what lies
    more than 200 tokens back nothing is left in fp64 next to the tolerance."""
    note(f"longest sequences {dtype}")
    L, D, N, W, T, back = 1 << 24, 3, 64, 4, 300, 200
    g = torch.Generator(device="cuda")
    g.manual_seed(24)
    rnd = lambda *s, e=F32: torch.randn(s, generator=g, device="cuda").to(e)  # noqa: E731
    uni = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    u, dy = rnd(1, L, D, e=dtype), rnd(1, L, D, e=dtype)
    dt = (uni(1, L, D) - 0.5).to(dtype)
    w, b = rnd(D, W), rnd(D)
    y, so = la.la_short_conv(u, w, b, want_state=True)
    dx = la.la_short_conv_bwd(u, w, dy, b)[0]
    p = lambda t: R.f64(t[:, L - T :])  # noqa: E731
    args = (p(u), R.f64(w), R.f64(b), None, None, True)
    ref, ref_so = R.conv(*args)
    mag, _ = R.conv(*[None if v is None else np.abs(v) for v in args[:4]], None, False)
    R.close(y[:, L - T + W :], ref[:, W:], mag[:, W:], W + 28, dtype, "conv")
    assert np.array_equal(R.f64(so), ref_so)
    r, m = R.conv_bwd(*args, p(dy), None), R.conv_bwd(*args, p(dy), None, mag=True)
    R.close(dx[:, L - T + W :], r[0][:, W:], m[0][:, W:], 2 * (W + 28), dtype, "conv dx")
    del y, dx
    Bm, C = rnd(1, L, N, e=dtype), rnd(1, L, N, e=dtype)
    A, bias, skip, ds_out = -2 - 2 * uni(D, N), uni(D) * 0.1 - 0.1, rnd(D), rnd(1, N, D)
    kw = dict(D=skip, dt_bias=bias)
    y, so = la.la_ssm_scan(u, dt, A, Bm, C, **kw)
    got = la.la_ssm_scan_bwd(u, dt, A, Bm, C, dy, ds_out=ds_out, **kw)
    args = (p(u), p(dt), R.f64(A), p(Bm), p(C), R.f64(skip), None, R.f64(bias), None, None, True)
    (ry, rs, _), (my, ms, _) = R.scan(*args), R.scan(*args, mag=True)
    K = 8 * T + 64
    R.close(y[:, L - T + back :], ry[:, back:], my[:, back:], K, dtype, "y")
    R.close(so, rs, ms, K, F32, "s_out")
    r, m = R.scan_bwd(*args, p(dy), R.f64(ds_out)), R.scan_bwd(*args, p(dy), R.f64(ds_out), mag=True)
    for k, name, extra in ((0, "du", 0), (1, "ddt", 0), (3, "dB", D), (4, "dC", D)):
        R.close(got[k][:, L - T + back :], r[k][:, back:], m[k][:, back:], 2 * K + extra, dtype, name)


def test_most_sequences():
    """2^20 sequences, the most there may be: rows from the start, the middle and the end give what they give alone (one
    segment either way, so bit for bit), forward, backward and one token; so does the convolution."""
    note("most sequences")
    B, L, D, N, W = 1 << 20, 2, 32, 16, 4
    g = torch.Generator(device="cuda")
    g.manual_seed(20)
    rnd = lambda *s, e=BF: torch.randn(s, generator=g, device="cuda").to(e)  # noqa: E731
    at = torch.cat([torch.arange(k, k + 40) for k in (0, (1 << 19) - 7, B - 40)]).cuda()
    u, dt, z, dy, Bm, C = (rnd(B, L, n) for n in (D, D, D, D, N, N))
    A, skip, bias = -torch.rand(D, N, generator=g, device="cuda") - 0.1, rnd(D, e=F32), rnd(D, e=F32) - 3
    s_in, lens = rnd(B, N, D, e=F32), torch.randint(0, L + 1, (B,), generator=g, device="cuda", dtype=torch.int32)

    def scan(pick, back):
        a = [pick(t) for t in (u, dt)] + [A, pick(Bm), pick(C)]
        kw = dict(D=skip, z=pick(z), dt_bias=bias, s_in=pick(s_in), lengths=pick(lens))
        if back:
            r = la.la_ssm_scan_bwd(*a, pick(dy), ds_out=pick(s_in), **kw)
            return [r[k] for k in (0, 1, 3, 4, 6, 8)]  # what is not summed over sequences
        return la.la_ssm_scan(*a, y=torch.zeros_like(a[0]), **kw)

    for back in (False, True):
        for k, (one, all_) in enumerate(zip(scan(lambda t: t[at], back), scan(lambda t: t, back))):
            assert torch.equal(one, all_[at]), (back, k)
    w, b, st = rnd(D, W, e=F32), rnd(D, e=F32), rnd(B, W - 1, D)
    conv = lambda pick: la.la_short_conv(pick(u), w, b, pick(st), lengths=pick(lens), y=torch.zeros_like(pick(u)), want_state=True)  # noqa: E731
    for one, all_ in zip(conv(lambda t: t[at]), conv(lambda t: t)):
        assert torch.equal(one, all_[at])
    one, all_ = (la.la_short_conv_bwd(p(u), w, p(dy), b, p(st), p(st), lengths=p(lens)) for p in (lambda t: t[at], lambda t: t))
    assert torch.equal(one[0], all_[0][at]) and torch.equal(one[3], all_[3][at])
    pools = [s_in[at].clone(), s_in], [st[at].clone(), st]
    y = [la.la_ssm_step(p(u)[:, 0], p(dt)[:, 0], A, p(Bm)[:, 0], p(C)[:, 0], s, D=skip, z=p(z)[:, 0], dt_bias=bias)
         for p, s in zip((lambda t: t[at], lambda t: t), pools[0])]
    assert torch.equal(y[0], y[1][at]) and torch.equal(pools[0][0], s_in[at])
    y = [la.la_short_conv_step(p(u)[:, 1], w, s, b) for p, s in zip((lambda t: t[at], lambda t: t), pools[1])]
    assert torch.equal(y[0], y[1][at]) and torch.equal(pools[1][0], st[at])


@pytest.mark.parametrize("M,D", [(1 << 25, 8), (1 << 25, 3), ((1 << 22) + 5, 2048), ((1 << 19) + 3, 16384)])
def test_norm_of_the_most_rows(M, D):
    """2^25 rows, and rows past 2^33 elements: rows from the start, the middle and the end give what they give alone; the
    backward's dx likewise, and d_weight of repeated rows is the repeated rows' sum.  Each of 512 workgroups adds at most
    M / 512 + 1 rows one after the other, then come at most 4 + 32 + 16 partial sums: K = M / 512 + 64 on top of a
    term's own roundings, 8."""
    note(f"norm of the most rows {M} {D}")
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    R_ = 4096
    few = torch.randn(R_, D, generator=g, device="cuda").to(BF)
    w = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    reps = -(-M // R_)
    x = few.repeat(reps, 1)[:M]
    y1, _, r1 = la.la_add_norm(few, w)
    y, _, r = la.la_add_norm(x, w)
    at = torch.cat([torch.arange(k, k + 40) for k in (0, M // 2 - 7, M - 40)]).cuda()
    assert torch.equal(y[at], y1[at % R_]) and torch.equal(r, r1.repeat(reps)[:M])
    del y
    q1, s1, _, _ = la.la_add_norm_q8(few, w)
    q, s, _, _ = la.la_add_norm_q8(x, w)
    assert torch.equal(q[at].view(torch.uint8), q1[at % R_].view(torch.uint8)) and torch.equal(s, s1.repeat(reps, 1)[:M])
    del q
    dx, dw = la.la_add_norm_bwd(x, x, w, r)
    dx2, _ = la.la_add_norm_bwd(few, few, w, r1)
    assert torch.equal(dx[at], dx2[at % R_])
    xh = R.f64(few) * R.f64(r1)[:, None]
    times = np.full((R_, 1), M // R_) + (np.arange(R_)[:, None] < M % R_)
    R.close(dw, (R.f64(few) * xh * times).sum(0), (np.abs(R.f64(few) * xh) * times).sum(0), M / 512 + 72, F32, "dw")


def test_padded_layer_in_a_graph():
    """A padded batch, forward and backward, captured once and replayed with other inputs and other lengths, NaN in the
    padding, eager work between the replays: every replay gives what the eager call gives."""
    note("padded layer in a graph")
    B, L, D, N, W = 3, 150, 64, 16, 4
    p, pin, pdbc, wx, wp = layer(D, N, W, 57)
    g = Draw(58)

    def inputs(lens):
        live = (torch.arange(L)[None] < torch.tensor(lens)[:, None])[..., None].cuda()
        t = [torch.where(live, g.normal(B, L, D), torch.full((), float("nan"), device="cuda")) for _ in range(3)]
        return t + [g.normal(B, L, D), ints(lens)]

    def both(x, res, dy, dh, lens):
        saved = {}
        out = pipeline.selective_prompt(p, x, res, pin, pdbc, lengths=lens, saved=saved)
        gr = pipeline.selective_backward(p, saved, dy, lambda ddt, dB, dC: torch.cat([ddt, dB, dC], -1) @ wp.t(),
                                         lambda du, dz: torch.cat([du, dz], -1).view(B * L, -1) @ wx.t(), dh=dh)
        return [out[0], out[2], out[3]] + [t for t in gr.values() if t is not None]

    sets = [inputs(n) for n in ([150, 3, 97], [0, 150, 40], [1, 2, 149], [150, 150, 150])]
    eager = [both(*s) for s in sets]
    bufs = [t.clone() for t in sets[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(*bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both(*bufs)
    for k in (1, 2, 3, 0, 2):
        for t, v in zip(bufs, sets[k]):
            t.copy_(v)
        graph.replay()
        other = both(*sets[(k + 1) % 4])
        torch.cuda.synchronize()
        for i, (a, b, c, d) in enumerate(zip(outs, eager[k], other, eager[(k + 1) % 4])):
            assert torch.isfinite(b).all() and torch.equal(a, b) and torch.equal(c, d), (k, i)
