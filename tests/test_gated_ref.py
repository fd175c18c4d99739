"""The fp64 forms of gated_ref.py against what does not share their code: published outputs of the generator, central
differences, closed forms.  CPU only."""
import numpy as np
import pytest

import gated_ref as R

RNG = np.random.default_rng


def test_generator_known_answers():
    """Outputs that Salmon et al. publish with the generator: counter and key all zero, all one, digits of pi."""
    for ctr, key, want in (
            ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
            ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
            ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
             [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1])):
        assert R.philox(np.array(ctr, dtype=np.uint64), key).tolist() == want


def test_mask_share_and_independence():
    a, f = R.keep(3, 5, 400, 1000, 0.25)
    assert f == 4 / 3
    # 400000 draws of a Bernoulli(3/4): five deviations of the mean
    assert abs(a.mean() - 0.75) < 5 * np.sqrt(0.75 * 0.25 / a.size)
    for other in (R.keep(4, 5, 400, 1000, 0.25)[0], R.keep(3, 6, 400, 1000, 0.25)[0]):
        assert abs((a == other).mean() - (0.75 ** 2 + 0.25 ** 2)) < 5 * np.sqrt(0.25 / a.size)
    assert np.array_equal(a[7:9], R.keep(3, 5, 2, 1000, 0.25, rows=[7, 8])[0])
    assert R.keep(3, 5, 9, 13, 0.0)[0].all()


def scan_case(seed, z=True, h_in=True, lengths=None, B=2, L=7, D=3):
    g = RNG(seed)
    n = lambda *s: g.standard_normal(s)  # noqa: E731
    return dict(x=n(B, L, D), r=n(B, L, D), i=n(B, L, D), lam=n(D) - 1, rb=n(D), ib=n(D), z=n(B, L, D) if z else None,
                h_in=n(B, D) if h_in else None), lengths, n(B, L, D), n(B, D)


@pytest.mark.parametrize("z", [True, False])
@pytest.mark.parametrize("lengths", [None, [7, 3], [0, 9]])
def test_scan_derivatives_against_differences(z, lengths):
    a, lengths, dy, dh = scan_case(1, z, True, lengths)
    keys = ["x", "r", "i", "lam", "rb", "ib", "z", "h_in"]

    def loss(b):
        (y, _), (h, _), _, _ = R.scan(*[b[k] for k in keys], lengths, 4.0)
        return (y * dy).sum() + (h * dh).sum()

    got = dict(zip(keys, R.scan_bwd(*[a[k] for k in keys], lengths, 4.0, dy, dh)))
    g = RNG(9)
    for k in keys:
        if a[k] is None:
            assert got[k] is None
            continue
        v, e = g.standard_normal(a[k].shape), 1e-5
        up, dn = (loss(dict(a, **{k: a[k] + s * e * v})) for s in (1, -1))
        want = (got[k][0] * v).sum()
        # second-order differences: e^2 of a third derivative of order one, and 1e-16 / e of rounding of a loss of order ten
        assert abs((up - dn) / (2 * e) - want) < 1e-8 * (1 + abs(want)), k


def test_scan_closed_forms():
    a, _, _, _ = scan_case(2, z=False)
    keys = ["x", "r", "i", "lam", "rb", "ib", "z", "h_in"]
    held = dict(a, r=np.full_like(a["r"], -np.inf))  # a = 1, no input: the state stays
    (y, _), (h, _), _, _ = R.scan(*[held[k] for k in keys], None, 8.0)
    assert np.array_equal(h, a["h_in"]) and np.array_equal(y, np.broadcast_to(a["h_in"][:, None], y.shape))
    lost = dict(a, lam=np.full_like(a["lam"], 400.0))  # a = 0: the gated input alone
    (y, _), _, _, _ = R.scan(*[lost[k] for k in keys], None, 8.0)
    assert np.allclose(y, a["x"] / (1 + np.exp(-(a["i"] + a["ib"]))), rtol=1e-14)
    # two pieces are one
    whole = R.scan(*[a[k] for k in keys], None, 8.0)
    first = R.scan(*[v[:, :4] if v is not None and v.ndim == 3 else v for v in (a[k] for k in keys)], None, 8.0)
    rest = dict(a, h_in=first[1][0])
    second = R.scan(*[v[:, 4:] if v is not None and v.ndim == 3 else v for v in (rest[k] for k in keys)], None, 8.0)
    assert np.array_equal(np.concatenate([first[0][0], second[0][0]], 1), whole[0][0])


@pytest.mark.parametrize("kind", ["none", "linear", "sigmoid", "silu"])
@pytest.mark.parametrize("post,pre,drop", [(True, True, False), (True, True, True), (False, True, True), (True, False, False),
                                           (False, False, True)])
def test_block_derivatives_against_differences(kind, post, pre, drop):
    g = RNG(5)
    M, D, eps = 3, 11, 1e-3
    n = lambda *s: g.standard_normal(s)  # noqa: E731
    a = dict(x=n(M, D), gate=None if kind == "none" else n(M, D), res=n(M, D), w_post=1 + n(D) if post else None,
             scale=n(D), w_pre=1 + n(D) if pre else None)
    kept, f = R.keep(1, 2, M, D, 0.4) if drop else (None, 1.0)
    dy, dh = n(M, D), n(M, D)

    def forward(b):
        return R.block(*[b[k] for k in ("x", "gate", "res", "w_post", "scale", "w_pre")], kind, eps, kept, f)

    def loss(b):
        y, h, _, _ = forward(b)
        return (h[0] * dh).sum() + (0 if y is None else (y[0] * dy).sum())

    _, h, rp, rq = forward(a)
    out = R.block_bwd(a["x"], a["gate"], h[0], a["w_post"], a["scale"], a["w_pre"], kind, rp and rp[0], rq and rq[0],
                      dy if pre else None, dh, kept, f)
    for k, got in zip(("x", "res", "gate", "w_post", "w_pre", "scale"), out):
        if a[k] is None:
            assert got is None, k
            continue
        v, e = n(*a[k].shape), 1e-5
        up, dn = (loss(dict(a, **{k: a[k] + s * e * v})) for s in (1, -1))
        want = (got[0] * v).sum()
        assert abs((up - dn) / (2 * e) - want) < 1e-7 * (1 + abs(want)), (k, (up - dn) / (2 * e), want)
