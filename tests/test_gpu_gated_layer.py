"""The gated recurrent layer's operators together, as pipeline.gated_prompt, gated_backward and gated_token run them; in
graphs, on streams, with waits that give up; and the operators at the largest sizes and far offsets."""
import dataclasses

import numpy as np
import pytest
import torch

import gated_ref as G
import mixer_ref as R
from chunked_scan_amd import binding as la
from chunked_scan_amd import pipeline
from gpu_util import note
from test_gpu_gated import GRADS, check_grads, nonan, rng_of, scan_inputs, scan_kw, scan_ref
from test_gpu_mixer import BF, F32, SENTINEL, Draw, ints

pytestmark = pytest.mark.gpu


def layer(D, Dm, W, seed, dropout=0.0, gate=True):
    """Parameters and projections: n [rows, Dm] -> (u, z) [rows, D]; v -> (r, i); o [rows, D] -> (x, gate) [rows, Dm]."""
    g = Draw(seed)
    p = pipeline.GatedParams(conv_weight=g.normal(D, W, std=0.5), conv_bias=g.normal(D, std=0.1), lam=g.normal(D) - 4,
                             r_bias=g.normal(D, std=0.3), i_bias=g.normal(D, std=0.3), w_post=1 + g.normal(Dm, std=0.1),
                             scale=g.uniform(Dm, lo=0.2, hi=1.0), w_pre=1 + g.normal(Dm, std=0.1), dropout=dropout)
    wi, wg, wo = (g.normal(a, b, std=a ** -0.5) for a, b in ((Dm, 2 * D), (D, 2 * D), (D, 2 * Dm if gate else Dm)))

    def halves(t, n):
        return t[..., :n], t[..., n:]

    def project_in(n):
        return halves((n.float() @ wi).to(n.dtype), D)

    def project_gates(v):
        return halves((v.float() @ wg).to(v.dtype), D)

    def project_out(o):
        t = (o.float() @ wo).to(o.dtype)
        return halves(t, Dm) if gate else (t, None)

    def backwards(dt):
        return dict(out_backward=lambda dx, dg: ((torch.cat([dx, dg], -1) if gate else dx).float() @ wo.t()).to(dt),
                    gates_backward=lambda dr, di: (torch.cat([dr, di], -1).float() @ wg.t()).to(dt),
                    in_backward=lambda du, dz: (torch.cat([du, dz], -1).flatten(0, 1).float() @ wi.t()).to(dt))

    return p, (project_in, project_gates, project_out), backwards


def test_layer_prompt_then_tokens_equals_one_prompt():
    """A padded batch of prompts of unequal lengths, then single tokens from its states in pools, gives what each
    sequence gives as one prompt.  In fp32, where the orders differ by roundings: 4 a token in the state and 64 in the
    rest, and as much again for each of the three fp32 projections (sums of 64 to 96 terms), on values that the two norms
    scale by up to 8 of their largest."""
    note("gated layer: prompts, then tokens")
    B, L, D, Dm, W, T = 3, 150, 64, 96, 4, 6
    p, proj, _ = layer(D, Dm, W, 140)
    g = Draw(141)
    x, res = g.normal(B, L + T, Dm), g.normal(B, L + T, Dm)
    lens = [150, 3, 97]
    y, h, cs, so = pipeline.gated_prompt(p, x[:, :L].contiguous(), res[:, :L].contiguous(), *proj, lengths=ints(lens))
    conv_pool, pool = torch.zeros(5, W - 1, D, device="cuda"), torch.zeros(5, D, device="cuda")
    at = torch.tensor([4, 0, 2], device="cuda")
    conv_pool[at], pool[at] = cs, so
    slots = at.to(torch.int32)
    rows = []
    for k in range(T):
        xt = torch.stack([x[i, lens[i] + k] for i in range(B)])
        rt = torch.stack([res[i, lens[i] + k] for i in range(B)])
        rows.append(pipeline.gated_token(p, xt, rt, *proj, conv_pool, pool, slots))
    for i in range(B):
        n = lens[i] + T
        one, h1, c1, s1 = pipeline.gated_prompt(p, x[i : i + 1, :n].contiguous(), res[i : i + 1, :n].contiguous(), *proj)
        tol = lambda t: 4 * (4 * n + 64) * R.U * float(t.abs().max()) * 8  # noqa: E731
        assert float((one[0, : lens[i]] - y[i, : lens[i]]).abs().max()) <= tol(one)
        assert float((h1[0, : lens[i]] - h[i, : lens[i]]).abs().max()) <= tol(h1)
        for k in range(T):
            assert float((one[0, lens[i] + k] - rows[k][0][i]).abs().max()) <= tol(one), (i, k)
            assert float((h1[0, lens[i] + k] - rows[k][1][i]).abs().max()) <= tol(h1), (i, k)
        assert float((s1[0] - pool[at[i]]).abs().max()) <= tol(s1)
        assert float((c1[0] - conv_pool[at[i]]).abs().max()) <= tol(c1)


def test_layer_in_pieces_equals_one_prompt():
    """Pieces that end where a tile ends take the same states in the same order: the same bits, also in bf16."""
    note("gated layer: pieces")
    B, L, D, Dm, W = 2, 400, 128, 128, 4
    p, proj, _ = layer(D, Dm, W, 144)
    g = Draw(145)
    x, res = g.normal(B, L, D, dtype=BF), g.normal(B, L, D, dtype=BF)
    y, h, cs, so = pipeline.gated_prompt(p, x, res, *proj)
    k = 256
    a = pipeline.gated_prompt(p, x[:, :k].contiguous(), res[:, :k].contiguous(), *proj)
    b = pipeline.gated_prompt(p, x[:, k:].contiguous(), res[:, k:].contiguous(), *proj, conv_state=a[2], h_in=a[3])
    assert torch.equal(torch.cat([a[1], b[1]], 1), h) and torch.equal(torch.cat([a[0], b[0]], 1), y)
    assert torch.equal(b[2], cs) and torch.equal(b[3], so)


@pytest.mark.parametrize("B,L", [(0, 5), (2, 0)])
def test_layer_of_no_tokens(B, L):
    note(f"gated layer of no tokens {B} {L}")
    D, Dm, W = 32, 40, 4
    p, proj, backwards = layer(D, Dm, W, 146)
    g = Draw(147)
    x, h0, c0 = g.normal(B, L, Dm), g.normal(B, D), g.normal(B, W - 1, D)
    saved = {}
    y, h, cs, so = pipeline.gated_prompt(p, x, x, *proj, conv_state=c0, h_in=h0, saved=saved)
    assert y.shape == h.shape == (B, L, Dm) and torch.equal(so, h0) and torch.equal(cs, c0)
    dc, dh = g.normal(B, W - 1, D), g.normal(B, D)
    gr = pipeline.gated_backward(p, saved, x, x, **backwards(F32), d_conv_state=dc, dh_out=dh)
    assert torch.equal(gr["conv_state"], dc) and torch.equal(gr["h_in"], dh)
    for k in ("lam", "r_bias", "i_bias", "w_post", "w_pre", "scale", "conv_weight", "conv_bias"):
        assert (gr[k] == 0).all(), k


@pytest.mark.parametrize("gate", [True, False])
def test_layer_gradients_against_differences(gate):
    """gated_backward's gradients of a scalar against differences of gated_prompt itself, in fp32 with dropout, along one
    random direction per argument (the step and the bound as in the recurrence's own test)."""
    note(f"gated layer: gradients {gate}")
    B, L, D, Dm, W = 2, 140, 64, 48, 4
    p, proj, backwards = layer(D, Dm, W, 148, dropout=0.2, gate=gate)
    g = Draw(149)
    lens, rng = ints([140, 33]), rng_of(7, 9)
    a = dict(n=g.normal(B, L, Dm), res=g.normal(B, L, Dm), cs=g.normal(B, W - 1, D), h_in=g.normal(B, D))
    live = (torch.arange(L, device="cuda")[None] < lens[:, None])[..., None]
    dy, dh = g.normal(B, L, Dm) * live, g.normal(B, L, Dm) * live
    dcs, ds = g.normal(B, W - 1, D), g.normal(B, D)
    names = ["conv_weight", "conv_bias", "lam", "r_bias", "i_bias", "w_post", "w_pre", "scale"]

    def loss(a, p):
        y, h, c, s = pipeline.gated_prompt(p, a["n"], a["res"], *proj, conv_state=a["cs"], h_in=a["h_in"], lengths=lens, rng=rng)
        return float(sum((t.double() * d.double()).sum() for t, d in ((y, dy), (h, dh), (c, dcs), (s, ds))))

    saved = {}
    pipeline.gated_prompt(p, a["n"], a["res"], *proj, conv_state=a["cs"], h_in=a["h_in"], lengths=lens, rng=rng, saved=saved)
    gr = pipeline.gated_backward(p, saved, dy, dh, **backwards(F32), d_conv_state=dcs, dh_out=ds)
    want = dict(n=gr["dn"], res=gr["dresidual"], cs=gr["conv_state"], h_in=gr["h_in"])
    e = 2.0 ** -8
    for k in list(a) + names:
        base = a[k] if k in a else getattr(p, k)
        grad = want[k] if k in a else gr[k]
        v = g.normal(*base.shape)
        vals = [loss(dict(a, **{k: base + s * e * v}), p) if k in a else loss(a, dataclasses.replace(p, **{k: base + s * e * v}))
                for s in (1, -1)]
        diff = (vals[0] - vals[1]) / (2 * e)
        dot = float((grad.double() * v.double()).sum())
        scale = float((grad.double().abs() * v.double().abs()).sum())
        assert abs(diff - dot) <= 1e-2 * scale / np.sqrt(v.numel()) + 1e-3 * scale, (k, diff, dot, scale)


def run_both(p, proj, backwards, dt, n, res, dy, dh, lens, rng):
    saved = {}
    out = pipeline.gated_prompt(p, n, res, *proj, lengths=lens, rng=rng, saved=saved)
    gr = pipeline.gated_backward(p, saved, dy, dh, **backwards(dt))
    return list(out) + [t for t in gr.values() if t is not None]


def test_padded_layer_in_a_graph():
    """A padded batch with dropout, forward and backward, captured once and replayed with other inputs, lengths and seeds,
    NaN in the padding, eager work between the replays: every replay gives what the eager call gives, all of it finite."""
    note("padded gated layer in a graph")
    B, L, D, Dm, W = 3, 300, 64, 96, 4
    p, proj, backwards = layer(D, Dm, W, 157, dropout=0.25)
    g = Draw(158)

    def inputs(lens, seed):
        live = (torch.arange(L)[None] < torch.tensor(lens)[:, None])[..., None].cuda()
        t = [torch.where(live, g.normal(B, L, Dm), torch.full((), float("nan"), device="cuda")) for _ in range(4)]
        return t + [ints(lens), rng_of(seed, 5)]

    sets = [inputs(n, k) for k, n in enumerate(([300, 3, 97], [0, 300, 140], [1, 129, 299], [300, 300, 300]))]
    both = lambda s: run_both(p, proj, backwards, F32, *s)  # noqa: E731
    eager = [both(s) for s in sets]
    bufs = [t.clone() for t in sets[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both(bufs)
    for k in (1, 2, 3, 0, 2):
        for t, v in zip(bufs, sets[k]):
            t.copy_(v)
        graph.replay()
        other = both(sets[(k + 1) % 4])
        torch.cuda.synchronize()
        for i, (a, b, c, d) in enumerate(zip(outs, eager[k], other, eager[(k + 1) % 4])):
            assert torch.isfinite(b).all() and torch.equal(a, b) and torch.equal(c, d), (k, i)
    assert la.la_chain_status() == 0


def test_many_tiles_on_many_streams():
    """Recurrences whose workgroups wait for each other, four at once on four streams, again and again: the bits of the
    call that runs alone."""
    note("gated scans on streams")
    sets = []
    for k, case in enumerate([(2, 1500, 520, None, False, True, True, True, -5.0), (1, 3000, 130, None, False, False, True, False, -6.0),
                              (4, 700, 257, [700, 1, 0, 399], False, True, True, True, -4.0),
                              (1, 2049, 1024, None, False, True, True, True, -5.0)]):
        a, n = scan_inputs(case, BF if k % 2 else F32, 300 + k)
        B, L, D = case[:3]
        # rows behind a sequence's end are left as they were: the same zeros for every call
        sets.append((a, dict(scan_kw(a, n)), torch.zeros(B, L, D, dtype=a["x"].dtype, device="cuda")))

    def one(a, kw, y):
        out = la.la_gated_scan(a["x"], a["r"], a["i"], a["lam"], y=y.clone(), **kw)[:2]
        return list(out) + [t for t in la.la_gated_scan_bwd(a["x"], a["r"], a["i"], a["lam"], a["dy"], dh_out=a["dh_out"], **kw)
                            if t is not None]

    want = [one(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(one(*s))
        torch.cuda.synchronize()
        for w, t in zip(want, got):
            for a, b in zip(w, t):
                assert torch.equal(a, b)
    assert la.la_chain_status() == 0


def test_stream_argument_and_traces():
    note("gated stream argument")
    a, n = scan_inputs((2, 333, 72, None, False, True, True, True, -5.0), BF, 90)
    kw = scan_kw(a, None)
    args = [a[k] for k in ("x", "r", "i", "lam")]
    want = la.la_gated_scan(*args, **kw)[0]
    rng = rng_of(1, 2)
    x = Draw(1).normal(64, 256, dtype=BF)
    wd, wn = la.la_dropout(x, rng, 0.5), la.la_block_norm(x, w_pre=a["lam"].new_ones(256), p=0.5, rng=rng)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    timer = la.KernelTimer()
    y = la.la_gated_scan(*args, stream=st, **kw)[0]
    d, nn = la.la_dropout(x, rng, 0.5, stream=st), la.la_block_norm(x, w_pre=a["lam"].new_ones(256), p=0.5, rng=rng, stream=st)
    st.synchronize()
    assert torch.equal(y, want) and torch.equal(d, wd) and torch.equal(nn[0], wn[0])
    la.la_gated_scan_bwd(*args, a["dy"], timer=timer, **kw)
    torch.cuda.synchronize()
    assert [k for k, _ in timer.harvest()] == ["gated_clear", "gated_scan", "gated_clear", "gated_scan_bwd", "gated_sums"]
    with pytest.raises(ValueError, match="stream is on|must be"):
        la.la_dropout(x, rng.cpu(), 0.5)


def test_waits_that_give_up():
    """With a poll limit of zero a workgroup whose incoming state is not there at once goes on with NaN: no value is
    wrong but not NaN, the give-ups are counted, and the next call at the default limit is whole again."""
    note("gated scan: waits that give up")
    a, _ = scan_inputs((2, 4000, 512, None, False, False, True, True, -5.0), F32, 95)
    args, kw = [a[k] for k in ("x", "r", "i", "lam")], scan_kw(a, None)
    y, h, _ = la.la_gated_scan(*args, **kw)
    grads = la.la_gated_scan_bwd(*args, a["dy"], **kw)
    assert la.la_chain_status() == 0
    default = la.la_set_chain_spin_limit(0)
    try:
        y0, h0, _ = la.la_gated_scan(*args, **kw)
        grads0 = la.la_gated_scan_bwd(*args, a["dy"], **kw)
        torch.cuda.synchronize()
    finally:
        la.la_set_chain_spin_limit(default)
    lost = False
    for t, t0 in zip([y, h, *grads[:3]], [y0, h0, *grads0[:3]]):
        assert ((t == t0) | torch.isnan(t0)).all()
        lost = lost or bool(torch.isnan(t0).any())
    if lost:
        with pytest.raises(la.LaError, match="LA_ERR_TIMEOUT"):
            la.la_chain_status()
    assert la.la_chain_status() == 0
    y1, h1, _ = la.la_gated_scan(*args, **kw)
    assert torch.equal(y, y1) and torch.equal(h, h1)


def test_strong_and_dead_decay():
    """Decays from none at all (softplus below fp32's range) to complete ones, in one call: everything finite and within
    the bounds."""
    note("gated scan: decays of every size")
    a, n = scan_inputs((2, 200, 72, [200, 65], False, True, True, True, -5.0), F32, 97)
    a["lam"] = torch.linspace(-110.0, 30.0, 72, device="cuda")
    kw = scan_kw(a, n)
    args = [a[k] for k in ("x", "r", "i", "lam")]
    y, h, _ = la.la_gated_scan(*args, y=torch.zeros_like(a["x"]), **kw)
    ref = scan_ref(a, n, 8.0)
    ry, rh, _, _ = G.scan(*ref)
    G.close(y, *ry, F32, "y")
    G.close(h, *rh, F32, "h")
    got = la.la_gated_scan_bwd(*args, a["dy"], dh_out=a["dh_out"], **kw)
    for t in got:
        assert torch.isfinite(t).all()
    want = G.scan_bwd(*ref, nonan(a["dy"]), R.f64(a["dh_out"]))
    # lam <= -80: v = 8 softplus(lam) rho < 8 e^-80 = 1.5e-34 and subnormal below -87, where the hardware takes it for zero.  The
    # input's factor is sqrt(2 v) < 1.8e-17 there, and so are, times a few, the derivatives of x, r and i and the sums of 200
    # tokens at most: compared with 1e-17 and 1e-15
    live = (a["lam"] > -80).cpu().numpy()
    for name, t, r in zip(GRADS, got, want):
        v, e = r
        if t.dim() == 3:
            e = e + 1e-17 / R.U * ~live
        if t.dim() == 1:
            assert np.abs(R.f64(t)[~live]).max() <= 1e-15
            G.close(t[torch.from_numpy(live).cuda()], v[live], e[live], F32, name)
        else:
            G.close(t, v, e, F32, name)


def test_nan_stays_in_its_channel():
    note("gated scan: NaN")
    a, _ = scan_inputs((2, 300, 130, None, False, False, True, True, -5.0), F32, 98)
    args, kw = lambda x: (x, a["r"], a["i"], a["lam"]), scan_kw(a, None)  # noqa: E731
    y, h, _ = la.la_gated_scan(*args(a["x"]), **kw)
    x = a["x"].clone()
    x[1, 140, 77] = float("nan")
    y2, h2, _ = la.la_gated_scan(*args(x), **kw)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[1, 140:, 77] = True
    assert torch.isnan(y2[bad]).all() and torch.equal(y2[~bad], y[~bad])
    assert torch.isnan(h2[1, 77]) and int(torch.isnan(h2).sum()) == 1


def test_offsets_beyond_32_bits():
    """Sequences, rows and slots more than 2^32 bytes apart give what they give close together; tokens too far apart for
    32-bit offsets take the form that has none."""
    note("gated: large offsets")
    far = (1 << 31) + 64
    g = Draw(171)
    L, D = 200, 64
    buf = torch.empty(far + L * D * 2, dtype=BF, device="cuda")

    def spread(t):
        v = buf.as_strided(t.shape, (far,) + tuple(t[0].stride()))
        v.copy_(t)
        return v

    a, _ = scan_inputs((2, L, D, None, False, False, True, True, -5.0), BF, 172)
    kw = scan_kw(a, None)
    run = lambda x: la.la_gated_scan(x, a["r"], a["i"], a["lam"], **kw)[:2]  # noqa: E731
    back = lambda x: la.la_gated_scan_bwd(x, a["r"], a["i"], a["lam"], a["dy"], **kw)  # noqa: E731
    want, wgrad = run(a["x"]), back(a["x"])
    sx = spread(a["x"])
    for s, t in zip(want + tuple(wgrad), run(sx) + tuple(back(sx))):
        assert s is None or torch.equal(s, t)
    rows, w = g.normal(2, 512, dtype=BF), 1 + g.normal(512, std=0.1)
    want = la.la_block_norm(rows, w_post=w, w_pre=w)
    got = la.la_block_norm(spread(rows), w_post=w, w_pre=w)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    rng = rng_of(3, 4)
    assert torch.equal(la.la_dropout(rows, rng, 0.5), la.la_dropout(spread(rows), rng, 0.5))
    # 20 tokens 2^27 elements apart: two runs of 8 reach past 2^31 bytes
    step = 1 << 27
    xs, big = g.normal(1, 20, D, dtype=BF), torch.empty(19 * step + D, dtype=BF, device="cuda")
    v = big.as_strided((1, 20, D), (0, step, 1))
    v.copy_(xs)
    c = lambda t: t[:1, :20].contiguous()  # noqa: E731
    kw = dict(r_bias=a["rb"], i_bias=a["ib"])
    one = la.la_gated_scan(xs, c(a["r"]), c(a["i"]), a["lam"], **kw)
    two = la.la_gated_scan(v, c(a["r"]), c(a["i"]), a["lam"], **kw)
    # another order of products within a tile: two runs of 8 tokens against one of 16
    assert float((one[0].double() - two[0].double()).abs().max()) <= (2.0 ** -7 + 200 * R.U) * float(one[0].abs().max())
    del buf, big, v, sx
    S = (1 << 31) // D + 3
    pool = torch.empty(S, D, device="cuda")
    st = g.normal(2, D)
    pool[0], pool[S - 1] = st[0], st[1]
    args = [t[:, 0].contiguous() for t in (a["x"], a["r"], a["i"])] + [a["lam"]]
    y0 = la.la_gated_step(*args, st)
    y1 = la.la_gated_step(*args, pool, slots=ints([0, S - 1]))
    assert torch.equal(y0, y1) and torch.equal(pool[S - 1], st[1]) and torch.equal(pool[0], st[0])


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_longest_sequence(dtype):
    """2^24 tokens of one sequence: the last block's tokens from the state that entered it, forward and backward, against
    the oracle; the state that enters the first tile's end against a short call."""
    note(f"gated scan of 2^24 tokens {dtype}")
    L, D, tail = 1 << 24, 6, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, r, i, dy = rnd(1, L, D), rnd(1, L, D), rnd(1, L, D), rnd(1, L, D)
    lam, dh = torch.randn(D, generator=g, device="cuda") - 5, torch.randn(1, D, generator=g, device="cuda")
    y, h, blocks = la.la_gated_scan(x, r, i, lam, want_blocks=True)
    cut = lambda t: nonan(t[:, -tail:])  # noqa: E731
    h0 = R.f64(blocks[:, -1])
    args = (cut(x), cut(r), cut(i), R.f64(lam), None, None, None, h0, None, 8.0)
    ry, rh, _, _ = G.scan(*args)
    G.close(y[:, -tail:], *ry, dtype, "y")
    G.close(h, *rh, F32, "h")
    y2, _, b2 = la.la_gated_scan(x[:, :300].contiguous(), r[:, :300].contiguous(), i[:, :300].contiguous(), lam, want_blocks=True)
    assert torch.equal(y2[:, :256], y[:, :256]) and torch.equal(b2[:, :5], blocks[:, :5])
    got = la.la_gated_scan_bwd(x, r, i, lam, dy, dh_out=dh, h_blocks=blocks)
    want = G.scan_bwd(*args, cut(dy), R.f64(dh))
    for name, t, w in zip(GRADS[:3], got, want):
        G.close(t[:, -tail:], *w, dtype, name)
    assert torch.isfinite(got[3]).all()
    del y, blocks, y2
    again = la.la_gated_scan_bwd(x, r, i, lam, dy, dh_out=dh)
    for s, t in zip(got, again):
        assert s is None or torch.equal(s, t)
    assert la.la_chain_status() == 0


def test_most_sequences_and_channels():
    note("gated scan: 2^20 sequences, 2^25 channels")
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    for B, L, D in ((1 << 20, 3, 32), (1, 2, 1 << 25)):
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        x, r, i, dy = (rnd(B, L, D).to(BF) for _ in range(4))
        lam, h_in, dh = rnd(D) - 5, rnd(B, D), rnd(B, D)
        y, h, _ = la.la_gated_scan(x, r, i, lam, h_in=h_in)
        got = la.la_gated_scan_bwd(x, r, i, lam, dy, h_in=h_in, dh_out=dh)
        at = torch.tensor([0, 1, B // 2, B - 1] if B > 1 else [0], device="cuda")
        ch = torch.arange(D, device="cuda") if B > 1 else torch.cat([torch.arange(k, k + 70) for k in (0, (1 << 24) - 3, D - 70)]).cuda()
        pick = lambda t: R.f64(t[at][..., ch])  # noqa: E731
        args = (pick(x), pick(r), pick(i), R.f64(lam[ch]), None, None, None, pick(h_in), None, 8.0)
        ry, rh, _, _ = G.scan(*args)
        G.close(y[at][..., ch], *ry, BF, "y")
        G.close(h[at][..., ch], *rh, F32, "h")
        want = G.scan_bwd(*args, pick(dy), pick(dh))
        for name, t, w in zip(GRADS, got, want):
            if t is not None and name not in ("dlam",):
                G.close(t[at][..., ch], *w, F32 if name == "dh_in" else BF, name)
        if B == 1:  # one sequence: the parameter's sum is these channels' own
            G.close(got[3][ch], *want[3], F32, "dlam")
        del x, r, i, dy, y, h, got


def test_block_and_dropout_of_the_most_rows():
    """2^25 rows of 8 values; a row of 2^32 and 9 values (dropout)."""
    note("block norm and dropout: the most rows")
    M, D = 1 << 25, 8
    few = Draw(9).normal(4096, D, dtype=BF)
    x = few.repeat(M // 4096, 1)
    rng, w = rng_of(11, 12), torch.ones(D, device="cuda")
    y, h, rp, rq = la.la_block_norm(x, x, w_post=w, w_pre=w, p=0.5, rng=rng)
    at = [0, 1, 4095, M // 2 + 5, M - 2, M - 1]
    kept, f = G.keep(11, 12, 6, D, 0.5, rows=at)
    rows = torch.tensor(at, device="cuda")
    ref = G.block(R.f64(x[rows]), None, R.f64(x[rows]), np.ones(D), None, np.ones(D), "linear", 1e-5, kept, f)
    for t, r, dt in ((y, ref[0], BF), (h, ref[1], BF), (rp, ref[2], F32), (rq, ref[3], F32)):
        G.close(t[rows], *r, dt)
    dx, dres, _, dwp, dwq, _ = la.la_block_norm_bwd(x, h, x, None, w_post=w, w_pre=w, p=0.5, rng=rng, rstd_post=rp, rstd_pre=rq)
    ref = G.block_bwd(R.f64(x[rows]), None, R.f64(h[rows]), np.ones(D), None, np.ones(D), "linear", R.f64(rp[rows]),
                      R.f64(rq[rows]), R.f64(x[rows]), None, kept, f)
    G.close(dx[rows], *ref[0], BF, "dx")
    G.close(dres[rows], *ref[1], BF, "dresidual")
    assert torch.isfinite(dwp).all() and torch.isfinite(dwq).all()
    del x, y, h, dx, dres
    D = (1 << 32) + 9
    x = torch.ones(1, D, dtype=BF, device="cuda")
    y = la.la_dropout(x, rng, 0.25, y=x)
    for first in (0, 1 << 31, D // 8 * 8 - 64):
        n = min(72, D - first)
        nc = np.arange(first // 8, first // 8 + 9, dtype=np.uint64)
        ctr = np.stack([nc & np.uint64(0xFFFFFFFF), nc >> np.uint64(32), np.full_like(nc, 12), np.zeros_like(nc)], -1)
        wd = G.philox(ctr, (11, 0))
        bits = np.stack([wd & 0xFFFF, wd >> 16], -1).reshape(-1)[:n]
        assert np.array_equal(R.f64(y[0, first : first + n]) != 0, bits >= 16384), first
    share = float((y[0, : 1 << 30] != 0).double().mean())
    assert abs(share - 0.75) < 5 * (0.75 * 0.25 / 2 ** 30) ** 0.5


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,D", [(3, 9), (5, 1001), (600, 515), (7, 2047), (4, 4095), (3, 8201)])
def test_in_place_rows_of_every_alignment(M, D, dtype):
    """Rows whose last elements are loaded with those before them, updated in place: the bits of separate outputs, and
    nothing between the rows is touched."""
    note(f"in place {M} {D} {dtype}")
    g = Draw(M + D)
    p, rng = 0.25, rng_of(3, 4)
    wide = {k: g.normal(M, D + 3, dtype=dtype) for k in ("x", "gate", "res", "dy", "dh")}
    w = {k: 1 + g.normal(D, std=0.2) for k in ("w_post", "w_pre", "scale")}

    def views():
        t = {k: v.clone() for k, v in wide.items()}
        return t, {k: v[:, 1 : D + 1] for k, v in t.items()}

    def untouched(t, k):
        assert torch.equal(t[k][:, :1], wide[k][:, :1]) and torch.equal(t[k][:, D + 1 :], wide[k][:, D + 1 :])

    _, v = views()
    kw = dict(gate=v["gate"], p=p, rng=rng, **w)
    y, h, rp, rq = la.la_block_norm(v["x"], v["res"], **kw)
    out = la.la_block_norm_bwd(v["x"], h, v["dy"], v["dh"], rstd_post=rp, rstd_pre=rq, **kw)
    drop = la.la_dropout(v["x"], rng, p, v["res"])
    for k in ("x", "res"):
        t, v = views()
        y2, h2, _, _ = la.la_block_norm(v["x"], v["res"], h=v[k], **kw)
        assert torch.equal(h2, h) and torch.equal(y2, y)
        untouched(t, k)
        t, v = views()
        assert torch.equal(la.la_dropout(v["x"], rng, p, v["res"], y=v[k]), drop)
        untouched(t, k)
    for k in ("dy", "dh"):
        t, v = views()
        got = la.la_block_norm_bwd(v["x"], h, v["dy"], v["dh"], rstd_post=rp, rstd_pre=rq, dresidual=v[k], **kw)
        for a, b in zip(got, out):
            assert torch.equal(a, b)
        untouched(t, k)
