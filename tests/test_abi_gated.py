"""Argument checks of the gated recurrent layer's entry points (gated recurrence, norms around a block, dropout) that
need no GPU: struct layouts, status codes, workspace sizes, and a seeded fuzz.  Validation happens on the host before
any HIP call; the pointers are fake addresses, never dereferenced.
"""
import ctypes
import random

import pytest
import torch

from chunked_scan_amd import binding as B
from test_abi_mixer import A, ALIAS, DTYPE, I32, I64, LAUNCH, NULL, OK, P, SHAPE, UNSUP, WORKSPACE, no_gpu


@pytest.fixture(scope="module")
def lib():
    return B.lib()


def test_struct_layouts():
    # offsets follow the C layout in include/la_chunk.h
    assert (B.GatedShape.dtype.offset, B.GatedShape.c.offset, B.GatedShape.nslots.offset, B.GatedShape.x.offset,
            B.GatedShape.dy.offset, B.GatedShape.stream.offset) == (24, 28, 32, 40, 120, 200)
    assert (B.BlockShape.dtype.offset, B.BlockShape.act.offset, B.BlockShape.eps.offset, B.BlockShape.p.offset,
            B.BlockShape.x_stride.offset, B.BlockShape.stream.offset) == (16, 20, 24, 28, 32, 112)
    assert [ctypes.sizeof(s) for s in (B.GatedShape, B.BlockShape)] == [216, 128]


def gated_shape(**kw):
    s = B.GatedShape(2, 200, 64, B.LA_BF16, 8.0)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


SCAN = ["x", "r", "i", "lam", "rb", "ib", "z", "h_in", "lengths", "y", "h_out", "blocks", "ws"]
BWD = SCAN[:9] + ["blocks", "dy", "dh_out", "dx", "dr", "di", "dlam", "drb", "dib", "dz", "dh_in", "ws"]
STEP = ["x", "r", "i", "lam", "rb", "ib", "z", "state", "slots", "y"]


def scan(lib, s, n=None, bwd=False, **kw):
    names = BWD if bwd else SCAN
    at = {k: A[i] for i, k in enumerate(names)}
    at["lengths"] = 0
    at.update(kw)
    mode = 0 if not bwd else 2 if at["blocks"] else 1
    n = lib.la_gated_scan_workspace(ctypes.byref(s), mode) if n is None else n
    fn = lib.la_gated_scan_bwd if bwd else lib.la_gated_scan
    return fn(*[P(at[k]) for k in names], max(n, 0), ctypes.byref(s))


@pytest.mark.parametrize("bwd", [False, True])
def test_scan_validation(lib, bwd):
    fn = lib.la_gated_scan_bwd if bwd else lib.la_gated_scan
    names = BWD if bwd else SCAN
    nan, inf = float("nan"), float("inf")
    assert fn(*([None] * len(names)), 0, None) == NULL
    for bad in (dict(B=-1), dict(L=-1), dict(D=-1), dict(c=0.0), dict(c=-1.0), dict(c=nan), dict(c=inf), dict(reserved=1),
                dict(x=B.Rows(-1, 64)), dict(i=B.Rows(0, -1)), dict(z=B.Rows(1 << 42, 1 << 42))):
        assert scan(lib, gated_shape(**bad), bwd=bwd) == SHAPE, bad
    for bad in (dict(L=(1 << 24) + 1), dict(B=1 << 40), dict(D=1 << 62), dict(B=(1 << 20) + 1)):
        assert scan(lib, gated_shape(**bad), bwd=bwd) == UNSUP, bad
    assert scan(lib, gated_shape(dtype=2), bwd=bwd) == DTYPE
    for k in ["x", "r", "i", "lam"] + (["dy", "dx", "dr", "di", "dlam", "dz"] if bwd else ["y"]):
        assert scan(lib, gated_shape(), bwd=bwd, **{k: 0}) == NULL, k
    s = gated_shape()
    for mode, blocks in ((0, 1),) if not bwd else ((2, A[30]), (1, 0)):
        need = lib.la_gated_scan_workspace(ctypes.byref(s), mode)
        assert need > 0
        kw = dict(blocks=blocks) if bwd else {}
        assert scan(lib, s, n=need - 1, bwd=bwd, **kw) == WORKSPACE
        assert scan(lib, s, ws=0, n=need, bwd=bwd, **kw) == WORKSPACE
        assert scan(lib, s, ws=A[-1] + 8, n=need, bwd=bwd, **kw) == WORKSPACE
    outs = BWD[12:20] if bwd else ["y", "h_out", "blocks"]
    at = {k: A[i] for i, k in enumerate(names)}
    for o in outs + ["ws"]:
        for i in names:
            if i in (o, "lengths") or (i, o) == ("h_in", "h_out"):
                continue
            assert scan(lib, s, bwd=bwd, **{o: at[i]}) == ALIAS, (o, i)
    if bwd:
        # without z its derivative is neither required nor looked at
        assert scan(lib, gated_shape(B=0), bwd=True, z=0, dz=A[0], lam=0) == NULL
    else:
        assert scan(lib, s, h_out=A[7] + 4) == ALIAS       # over h_in, but not the same
        nothing = {k: 0 for k in SCAN}
        for empty in (dict(D=0), dict(B=0)):
            assert scan(lib, gated_shape(**empty), **nothing) == OK
    for mode in (0, 1, 2):
        assert lib.la_gated_scan_workspace(None, mode) == NULL
        assert lib.la_gated_scan_workspace(ctypes.byref(gated_shape(c=0.0)), mode) == SHAPE
    for mode in (-1, 3):
        assert lib.la_gated_scan_workspace(ctypes.byref(s), mode) == UNSUP
    assert lib.la_gated_scan_workspace(ctypes.byref(gated_shape(L=128)), 0) == 0


def test_step_validation(lib):
    def call(s, **kw):
        at = {k: A[i] for i, k in enumerate(STEP)}
        at.update(kw)
        return lib.la_gated_step(*[P(at[k]) for k in STEP], ctypes.byref(s))

    assert lib.la_gated_step(*([None] * 11)) == NULL
    assert call(gated_shape(nslots=-1)) == SHAPE
    assert call(gated_shape(nslots=1), slots=0) == SHAPE       # no slots: nslots >= B
    for k in ("x", "r", "i", "lam", "state", "y"):
        assert call(gated_shape(nslots=4), **{k: 0}) == NULL, k
    for k in STEP:
        if k != "y":
            assert call(gated_shape(nslots=4), y=A[STEP.index(k)]) == ALIAS, k
        if k != "state":
            assert call(gated_shape(nslots=4), state=A[STEP.index(k)]) == ALIAS, k
    assert call(gated_shape(nslots=4, y=B.Rows(63, 0))) == ALIAS
    assert call(gated_shape(nslots=(1 << 31) - 1, D=1 << 25, B=1)) == UNSUP
    assert call(gated_shape(B=0, nslots=0), **{k: 0 for k in STEP}) == OK


def block_shape(**kw):
    s = B.BlockShape(8, 256, B.LA_BF16, 2, 1e-5, 0.25)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


FWD = ["x", "gate", "res", "w_post", "scale", "w_pre", "rng", "y", "h", "rp", "rq"]
BACK = ["x", "gate", "h", "w_post", "scale", "w_pre", "rng", "rp", "rq", "dy", "dh", "dx", "dgate", "dres", "dwp", "dsc",
        "dwq", "ws"]


def block(lib, s, **kw):
    at = {k: A[i] for i, k in enumerate(FWD)}
    at.update(kw)
    return lib.la_block_norm(*[P(at[k]) for k in FWD], ctypes.byref(s))


def back(lib, s, n=None, **kw):
    at = {k: A[i] for i, k in enumerate(BACK)}
    at.update(kw)
    n = lib.la_block_norm_bwd_workspace(ctypes.byref(s)) if n is None else n
    return lib.la_block_norm_bwd(*[P(at[k]) for k in BACK], max(n, 0), ctypes.byref(s))


def drop(lib, s, x=A[0], res=A[1], rng=A[2], y=A[3]):
    return lib.la_dropout(P(x), P(res), P(rng), P(y), ctypes.byref(s))


def test_block_validation(lib):
    nan, inf = float("nan"), float("inf")
    assert lib.la_block_norm(*([None] * 12)) == NULL and lib.la_block_norm_bwd(*([None] * 18), 0, None) == NULL
    assert lib.la_dropout(*([None] * 5)) == NULL and lib.la_block_norm_bwd_workspace(None) == NULL
    for f in (block, back, drop):
        for bad in (dict(M=-1), dict(D=0), dict(p=-0.1), dict(p=1.0), dict(p=nan), dict(x_stride=-1), dict(dgate_stride=1 << 60)):
            assert f(lib, block_shape(**bad)) == SHAPE, bad
        for bad in (dict(M=1 << 26), dict(M=1 << 25, D=16384)):
            assert f(lib, block_shape(**bad)) == UNSUP, bad
        assert f(lib, block_shape(dtype=7)) == DTYPE
        assert f(lib, block_shape(), rng=0) == NULL
        assert f(lib, block_shape(), rng=A[31] + 4) == SHAPE    # not on 8 bytes
    for f in (block, back):
        for bad in (dict(eps=0.0), dict(eps=nan), dict(eps=inf)):
            assert f(lib, block_shape(**bad)) == SHAPE, bad
        for bad in (dict(D=16385), dict(act=3), dict(act=-1)):
            assert f(lib, block_shape(**bad)) == UNSUP, bad
    for k in ("x", "h", "y"):
        assert block(lib, block_shape(), **{k: 0}) == NULL, k
    for k in ("x", "dx", "dgate", "dwp", "dsc", "dwq", "rp", "rq", "dy", "h"):
        assert back(lib, block_shape(), **{k: 0}) == NULL, k
    need = lib.la_block_norm_bwd_workspace(ctypes.byref(block_shape()))
    assert need > 0 and back(lib, block_shape(), n=need - 1) == WORKSPACE and back(lib, block_shape(), ws=0, n=need) == WORKSPACE
    for o in ("y", "rp", "rq"):
        for i in FWD:
            if i != o:
                assert block(lib, block_shape(), **{o: A[FWD.index(i)]}) == ALIAS, (o, i)
    assert block(lib, block_shape(), h=A[0] + 2) == ALIAS              # in place means the same rows
    assert block(lib, block_shape(h_stride=512), h=A[2]) == ALIAS      # ... and the same stride
    for i in ("gate", "w_post", "scale", "w_pre", "rng"):
        assert block(lib, block_shape(), h=A[FWD.index(i)]) == ALIAS, i
    for o in ("dx", "dgate", "dres", "dwp", "dsc", "dwq", "ws"):
        for i in BACK:
            if i != o and not (o == "dres" and i in ("dy", "dh")):
                assert back(lib, block_shape(), **{o: A[BACK.index(i)]}) == ALIAS, (o, i)
    assert back(lib, block_shape(), dres=A[9] + 2) == ALIAS
    assert drop(lib, block_shape(), y=A[0] + 2) == ALIAS and drop(lib, block_shape(y_stride=512), y=A[1]) == ALIAS
    assert drop(lib, block_shape(), y=A[2]) == ALIAS and drop(lib, block_shape(y_stride=255)) == ALIAS
    for f in (block, back, drop):
        zero = {k: 0 for k in dict(block=FWD, back=[b for b in BACK if b not in ("w_post", "scale", "w_pre")],
                                   drop=["x", "res", "rng", "y"])[f.__name__]}
        if f is not back:
            assert f(lib, block_shape(M=0), **zero) == OK
    # parts that are not there are not looked at
    gone = dict(w_pre=0, y=A[0], rq=A[0])
    assert block(lib, block_shape(M=0), x=0, gate=0, res=0, w_post=0, scale=0, rng=0, h=0, rp=0, **gone) == OK


@no_gpu
def test_valid_calls_reach_the_device(lib):
    assert scan(lib, gated_shape()) == LAUNCH and scan(lib, gated_shape(), bwd=True) == LAUNCH
    assert scan(lib, gated_shape(), bwd=True, blocks=0, z=0, dz=A[0]) == LAUNCH
    assert scan(lib, gated_shape(), h_out=A[7]) == LAUNCH              # over h_in
    assert block(lib, block_shape()) == LAUNCH and back(lib, block_shape()) == LAUNCH
    assert block(lib, block_shape(), h=A[0]) == LAUNCH and block(lib, block_shape(), h=A[2]) == LAUNCH
    assert back(lib, block_shape(), dres=A[9]) == LAUNCH and back(lib, block_shape(), dres=A[10]) == LAUNCH
    assert block(lib, block_shape(p=0.0), rng=0) == LAUNCH
    assert block(lib, block_shape(p=1e-6), rng=0) == LAUNCH            # nearest multiple of 2^-16: zero
    assert drop(lib, block_shape()) == LAUNCH and drop(lib, block_shape(), y=A[0]) == LAUNCH
    assert drop(lib, block_shape(), y=A[1]) == LAUNCH and drop(lib, block_shape(p=1 - 2.0 ** -16)) == LAUNCH
    assert drop(lib, block_shape(M=4, D=1 << 30)) == LAUNCH
    # two halves of one wide buffer do not overlap
    half = dict(x_stride=512, y_stride=512)
    assert drop(lib, block_shape(**half), y=A[0] + 512) == LAUNCH and drop(lib, block_shape(**half), y=A[0] + 510) == ALIAS


@no_gpu
@pytest.mark.parametrize("seed", range(4))
def test_validation_fuzz(lib, seed):
    """Every entry point returns a documented status for any shape; under the host-sanitized build an overflow or a
    bad read on the way is a failure."""
    rng = random.Random(seed)
    codes = {OK, NULL, SHAPE, DTYPE, ALIAS, UNSUP, LAUNCH, WORKSPACE}

    def pick(ordinary, extreme):
        return rng.choice(extreme) if rng.random() < 0.12 else rng.choice(ordinary)

    def rows():
        return B.Rows(0, 0) if rng.random() < 0.7 else B.Rows(pick([64, 4096, 1 << 20], I64), pick([64, 128], I64))

    seen = set()
    for _ in range(1200):
        b, ln, d = pick([1, 2, 5], I64), pick([1, 7, 300], I64), pick([8, 64, 100], I64)
        dt = pick([0, 1], [2, -1])
        g = B.GatedShape(b, ln, d, dt, pick([8.0], [0.0, float("inf")]), pick([8], I32), pick([0], I32), *[rows() for _ in range(10)])
        n = B.BlockShape(b, d, dt, pick([0, 1, 2], I32), pick([1e-5], [0.0]), pick([0.0, 0.5], [1.0, -1.0]),
                         *[pick([0], I64) for _ in range(10)])
        ptr = [P(A[i] if rng.random() < 0.95 else 0) for i in range(24)]
        got = [lib.la_gated_scan(*ptr[:13], 1 << 50, ctypes.byref(g)), lib.la_gated_scan_bwd(*ptr[:21], 1 << 50, ctypes.byref(g)),
               lib.la_gated_step(*ptr[:10], ctypes.byref(g)), lib.la_block_norm(*ptr[:11], ctypes.byref(n)),
               lib.la_block_norm_bwd(*ptr[:18], 1 << 40, ctypes.byref(n)), lib.la_dropout(*ptr[:4], ctypes.byref(n))]
        assert set(got) <= codes, got
        seen |= {(i, r) for i, r in enumerate(got)}
        for w in [lib.la_gated_scan_workspace(ctypes.byref(g), m) for m in (0, 1, 2)] + [lib.la_block_norm_bwd_workspace(ctypes.byref(n))]:
            assert w >= 0 or w in codes
    for i in range(6):
        assert (i, LAUNCH) in seen, i
        assert len({r for k, r in seen if k == i}) >= 4, i


def test_binding_refusals():
    x, v = torch.zeros(2, 8, 16), torch.zeros(16)
    with pytest.raises(ValueError, match="device tensor"):
        B.la_gated_scan(x, x, x, v)
    with pytest.raises(ValueError, match="dims"):
        B.la_gated_scan(x[0], x[0], x[0], v)
    with pytest.raises(ValueError, match="device tensor"):
        B.la_gated_scan_bwd(x, x, x, v, x)
    with pytest.raises(ValueError, match="device tensor"):
        B.la_gated_step(x[:, 0], x[:, 0], x[:, 0], v, torch.zeros(4, 16))
    with pytest.raises(ValueError, match="unsupported dtype"):
        B.la_block_norm(x[0].double())
    with pytest.raises(ValueError, match="act must be"):
        B.la_block_norm(x[0], act="gelu")
    with pytest.raises(ValueError, match="device tensor"):
        B.la_dropout(x[0], None, 0.0)
