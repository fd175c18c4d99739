"""Argument checks of the selective state space layer's entry points (short convolution, selective scan,
residual norm) that need no GPU: struct layouts, status codes, workspace sizes, and a seeded fuzz.
Validation happens on the host before any HIP call; the pointers are fake addresses, never dereferenced.
"""
import ctypes
import os
import random

import pytest
import torch

from chunked_scan_amd import binding as B

OK, NULL, SHAPE, DTYPE, ALIAS, UNSUP, LAUNCH, DECAY, WORKSPACE = 0, -1, -2, -3, -4, -5, -6, -7, -8
no_gpu = pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="fake device addresses: only without a GPU")
P = ctypes.c_void_p
A = [0x10000000000 * (i + 1) for i in range(32)]  # far apart


@pytest.fixture(scope="module")
def lib():
    return B.lib()


def test_struct_layouts():
    # offsets follow the C layout in include/la_chunk.h
    assert ctypes.sizeof(B.Rows) == 16
    assert (B.ConvShape.width.offset, B.ConvShape.x.offset, B.ConvShape.stream.offset) == (24, 40, 104)
    assert (B.SsmShape.N.offset, B.SsmShape.u.offset, B.SsmShape.dy.offset, B.SsmShape.stream.offset) == (24, 40, 136, 232)
    assert (B.NormShape.dtype.offset, B.NormShape.eps.offset, B.NormShape.x_stride.offset,
            B.NormShape.stream.offset) == (16, 24, 32, 88)
    assert [ctypes.sizeof(s) for s in (B.ConvShape, B.SsmShape, B.NormShape)] == [120, 248, 104]


def conv_shape(**kw):
    s = B.ConvShape(2, 16, 64, 4, B.LA_BF16, 1, 0)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def conv(lib, s, x=A[0], w=A[1], b=A[2], st=A[3], ln=None, y=A[4], so=A[5]):
    return lib.la_short_conv(P(x), P(w), P(b), P(st), P(ln), P(y), P(so), ctypes.byref(s))


def conv_bwd(lib, s, x=A[0], dy=A[6], dx=A[7], dw=A[8], db=A[9], ds=A[10], ws=A[11], n=None, dso=None):
    n = lib.la_short_conv_bwd_workspace(ctypes.byref(s)) if n is None else n
    return lib.la_short_conv_bwd(P(x), P(A[1]), P(A[2]), P(A[3]), None, P(dy), P(dso), P(dx), P(dw), P(db), P(ds), P(ws),
                                 max(n, 0), ctypes.byref(s))


def test_conv_validation(lib):
    assert lib.la_short_conv(*([None] * 8)) == NULL
    assert lib.la_short_conv_bwd_workspace(None) == NULL
    for bad in (dict(B=-1), dict(L=-1), dict(D=-1), dict(x=B.Rows(-1, 64)), dict(y=B.Rows(1024, 1 << 42))):
        assert conv(lib, conv_shape(**bad)) == SHAPE, bad
    for bad in (dict(width=1), dict(width=5), dict(silu=2), dict(B=(1 << 20) + 1), dict(L=1 << 40), dict(D=1 << 60)):
        assert conv(lib, conv_shape(**bad)) == UNSUP, bad
    assert conv(lib, conv_shape(dtype=2)) == DTYPE
    assert conv(lib, conv_shape(), x=0) == NULL
    assert conv(lib, conv_shape(), w=0) == NULL
    assert conv(lib, conv_shape(), y=0) == NULL
    n = 2 * 16 * 64 * 2
    assert conv(lib, conv_shape(), y=A[0] + n - 2) == ALIAS
    assert conv(lib, conv_shape(), so=A[0]) == ALIAS
    assert conv(lib, conv_shape(), y=A[3] + 2) == ALIAS       # over the incoming state
    assert conv(lib, conv_shape(), so=A[3]) == ALIAS          # the state is not updated in place
    assert conv(lib, conv_shape(y=B.Rows(1024, 63))) == ALIAS  # rows of y overlap each other
    assert conv(lib, conv_shape(y=B.Rows(1000, 64))) == ALIAS
    # two halves of one wide buffer do not overlap; shifted by one element they do
    half = dict(x=B.Rows(16 * 128, 128), y=B.Rows(16 * 128, 128))
    assert conv(lib, conv_shape(**half), y=A[0] + 126) == ALIAS
    assert conv(lib, conv_shape(**half), y=A[0] + 2) == ALIAS
    # nothing to do
    assert conv(lib, conv_shape(B=0), x=0, w=0, b=0, st=0, y=0, so=0) == OK
    assert conv(lib, conv_shape(D=0), x=0, w=0, b=0, st=0, y=0, so=0) == OK
    assert conv(lib, conv_shape(L=0), x=0, w=0, b=0, st=0, y=0, so=0) == OK


def test_conv_bwd_validation(lib):
    s = conv_shape()
    need = lib.la_short_conv_bwd_workspace(ctypes.byref(s))
    assert need > 0
    assert conv_bwd(lib, s, n=need - 1) == WORKSPACE
    assert conv_bwd(lib, s, ws=0, n=need) == WORKSPACE
    assert conv_bwd(lib, s, ws=A[11] + 8, n=need) == WORKSPACE
    for k in ("x", "dy", "dx", "dw"):
        assert conv_bwd(lib, s, **{k: 0}) == NULL, k
    assert conv_bwd(lib, s, dx=A[6]) == ALIAS
    assert conv_bwd(lib, s, dw=A[1]) == ALIAS
    assert conv_bwd(lib, s, db=A[8] + 4) == ALIAS
    assert conv_bwd(lib, s, ws=A[7]) == ALIAS
    assert lib.la_short_conv_bwd_workspace(ctypes.byref(conv_shape(width=9))) == UNSUP


@no_gpu
def test_interleaved_halves_pass_validation(lib):
    half = dict(x=B.Rows(16 * 128, 128), y=B.Rows(16 * 128, 128))
    assert conv(lib, conv_shape(**half), y=A[0] + 128) == LAUNCH   # reaches HIP: no device here
    assert conv(lib, conv_shape(**half), y=A[0] - 128) == LAUNCH
    assert conv(lib, conv_shape(B=1, **half), y=A[0] + 128) == LAUNCH
    # sequences laid out token by token: [L, B, D] memory seen as [B, L, D]
    assert conv(lib, conv_shape(y=B.Rows(64, 128))) == LAUNCH


def test_conv_step_validation(lib):
    def call(s, x=A[0], st=A[3], sl=A[4], y=A[5], w=A[1]):
        return lib.la_short_conv_step(P(x), P(w), None, P(st), P(sl), P(y), ctypes.byref(s))

    assert lib.la_short_conv_step(*([None] * 7)) == NULL
    assert call(conv_shape(nslots=-1)) == SHAPE
    assert call(conv_shape(nslots=1), sl=0) == SHAPE           # no slots: nslots >= B
    assert call(conv_shape(nslots=4), st=0) == NULL
    assert call(conv_shape(nslots=4), y=A[0]) == ALIAS
    assert call(conv_shape(nslots=4), y=A[3] + 64) == ALIAS
    assert call(conv_shape(nslots=4, y=B.Rows(63, 0))) == ALIAS
    assert call(conv_shape(nslots=4), st=A[4]) == ALIAS        # the pool over the slots
    assert call(conv_shape(B=0, nslots=4), x=0, y=0) == OK


def ssm_shape(**kw):
    s = B.SsmShape(2, 16, 64, 16, B.LA_BF16, 1, 0)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


SCAN = ["u", "dt", "A", "B", "C", "D", "z", "bias", "s_in", "lengths", "y", "s_out", "ws"]
BWD = SCAN[:10] + ["dy", "ds_out", "du", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "ds_in", "ws"]


def scan(lib, s, n=None, bwd=False, **kw):
    names = BWD if bwd else SCAN
    at = {k: A[i] for i, k in enumerate(names)}
    at["lengths"] = 0
    at.update(kw)
    n = lib.la_ssm_workspace(ctypes.byref(s), int(bwd)) if n is None else n
    fn = lib.la_ssm_scan_bwd if bwd else lib.la_ssm_scan
    return fn(*[P(at[k]) for k in names], max(n, 0), ctypes.byref(s))


@pytest.mark.parametrize("bwd", [False, True])
def test_scan_validation(lib, bwd):
    fn = lib.la_ssm_scan_bwd if bwd else lib.la_ssm_scan
    names = BWD if bwd else SCAN
    assert fn(*([None] * len(names)), 0, None) == NULL
    for bad in (dict(B=-1), dict(L=-1), dict(D=-1), dict(N=0), dict(N=-3), dict(u=B.Rows(-1, 64)), dict(b=B.Rows(0, -1))):
        assert scan(lib, ssm_shape(**bad), bwd=bwd) == SHAPE, bad
    for bad in (dict(N=65), dict(softplus=2), dict(L=(1 << 24) + 1), dict(B=1 << 40), dict(D=1 << 62)):
        assert scan(lib, ssm_shape(**bad), bwd=bwd) == UNSUP, bad
    assert scan(lib, ssm_shape(dtype=-1), bwd=bwd) == DTYPE
    needed = ["u", "dt", "A", "B", "C"] + (["dy", "du", "ddt", "dA", "dB", "dC", "dz"] if bwd else ["y"])
    for k in needed:
        assert scan(lib, ssm_shape(), bwd=bwd, **{k: 0}) == NULL, k
    s = ssm_shape()
    need = lib.la_ssm_workspace(ctypes.byref(s), int(bwd))
    assert need > 0
    assert scan(lib, s, n=need - 1, bwd=bwd) == WORKSPACE
    assert scan(lib, s, ws=0, n=need, bwd=bwd) == WORKSPACE
    assert scan(lib, s, ws=A[12] + 4, n=need, bwd=bwd) == WORKSPACE
    outs = ["du", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "ds_in"] if bwd else ["y", "s_out"]
    at = {k: A[i] for i, k in enumerate(names)}
    for o in outs:
        for i in names:
            if i in (o, "lengths") or (i, o) == ("s_in", "s_out"):
                continue
            assert scan(lib, s, bwd=bwd, **{o: at[i]}) == ALIAS, (o, i)
    if not bwd:
        assert scan(lib, s, s_out=A[8] + 4) == ALIAS       # s_out over s_in, but not the same
        assert scan(lib, ssm_shape(D=0), u=0, dt=0, A=0, B=0, C=0, D=0, z=0, bias=0, s_in=0, y=0, s_out=0) == OK
    assert lib.la_ssm_workspace(None, 0) == NULL
    assert lib.la_ssm_workspace(ctypes.byref(ssm_shape(N=65)), 1) == UNSUP


def test_scan_step_validation(lib):
    names = ["u", "dt", "A", "B", "C", "D", "z", "bias", "state", "slots", "y"]

    def call(s, **kw):
        at = {k: A[i] for i, k in enumerate(names)}
        at.update(kw)
        return lib.la_ssm_step(*[P(at[k]) for k in names], ctypes.byref(s))

    assert lib.la_ssm_step(*([None] * 12)) == NULL
    assert call(ssm_shape(nslots=-2)) == SHAPE
    assert call(ssm_shape(nslots=1), slots=0) == SHAPE
    for k in ("u", "dt", "A", "B", "C", "y", "state"):
        assert call(ssm_shape(nslots=4), **{k: 0}) == NULL, k
    for k in names:
        if k != "y":
            assert call(ssm_shape(nslots=4), y=A[names.index(k)]) == ALIAS, k
    assert call(ssm_shape(B=0, nslots=0), u=0, state=0, y=0) == OK


def norm_shape(**kw):
    s = B.NormShape(8, 256, B.LA_BF16, 0, 1e-5, 0)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def test_norm_validation(lib):
    def fwd(s, x=A[0], r=A[1], w=A[2], y=A[3], h=A[4], rs=A[5]):
        return lib.la_add_norm(P(x), P(r), P(w), P(y), P(h), P(rs), ctypes.byref(s))

    def q8(s, x=A[0], r=A[1], w=A[2], q=A[3], sc=A[4], h=A[5], rs=A[6]):
        return lib.la_add_norm_q8(P(x), P(r), P(w), P(q), P(sc), P(h), P(rs), ctypes.byref(s))

    def bwd(s, dy=A[0], h=A[1], w=A[2], rs=A[3], dh=A[4], dx=A[5], dw=A[6], ws=A[7], n=None):
        n = lib.la_add_norm_bwd_workspace(ctypes.byref(s)) if n is None else n
        return lib.la_add_norm_bwd(P(dy), P(h), P(w), P(rs), P(dh), P(dx), P(dw), P(ws), max(n, 0), ctypes.byref(s))

    nan, inf = float("nan"), float("inf")
    for f in (fwd, q8, bwd):
        for bad in (dict(M=-1), dict(D=0), dict(eps=0.0), dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(reserved=1),
                    dict(h_stride=-1), dict(dx_stride=1 << 60)):
            assert f(norm_shape(**bad)) == SHAPE, bad
        for bad in (dict(D=16385), dict(M=1 << 26), dict(M=1 << 25, D=16384)):
            assert f(norm_shape(**bad)) == UNSUP, bad
        assert f(norm_shape(dtype=5)) == DTYPE
    assert lib.la_add_norm(*([None] * 7)) == NULL and lib.la_add_norm_q8(*([None] * 8)) == NULL
    for k in ("x", "w", "y"):
        assert fwd(norm_shape(), **{k: 0}) == NULL
    for k in ("x", "w", "q", "sc"):
        assert q8(norm_shape(), **{k: 0}) == NULL
    for k in ("dy", "h", "w", "rs", "dx", "dw"):
        assert bwd(norm_shape(), **{k: 0}) == NULL
    assert q8(norm_shape(group=16)) == UNSUP and q8(norm_shape(D=96, group=64)) == SHAPE
    assert fwd(norm_shape(), y=A[0]) == ALIAS and fwd(norm_shape(), y=A[4] + 16) == ALIAS
    assert fwd(norm_shape(), h=A[1] + 2) == ALIAS             # in place means the same rows
    assert fwd(norm_shape(h_stride=512), h=A[1]) == ALIAS     # ... and the same stride
    assert fwd(norm_shape(h_stride=255)) == ALIAS
    assert q8(norm_shape(), sc=A[3] + 4) == ALIAS and q8(norm_shape(), rs=A[4]) == ALIAS
    assert bwd(norm_shape(), dx=A[1]) == ALIAS                # dx may be dy or dh, not h
    assert bwd(norm_shape(), dx=A[0] + 2) == ALIAS and bwd(norm_shape(), dw=A[2]) == ALIAS
    need = lib.la_add_norm_bwd_workspace(ctypes.byref(norm_shape()))
    assert need > 0 and bwd(norm_shape(), n=need - 1) == WORKSPACE and bwd(norm_shape(), ws=0, n=need) == WORKSPACE
    assert fwd(norm_shape(M=0), x=0, w=0, y=0) == OK


def test_trace_validation(lib):
    t = B.Trace()
    t.capacity = 17
    s = conv_shape()
    s.trace = ctypes.pointer(t)
    assert conv(lib, s) == SHAPE
    t.capacity = 1
    assert conv(lib, s) == NULL


I64 = [0, 1, 2, 3, 7, 64, 100, 16384, -1, -(1 << 40), (1 << 31) - 1, 1 << 40, 1 << 62, (1 << 63) - 1, -(1 << 63)]
I32 = [0, 1, 2, 4, 16, 64, 128, -1, (1 << 31) - 1, -(1 << 31)]


@no_gpu
@pytest.mark.parametrize("seed", range(4))
def test_validation_fuzz(lib, seed):
    """Every entry point returns a documented status for any shape; under the host-sanitized build an overflow or a
    bad read on the way is a failure."""
    rng = random.Random(seed)
    codes = {OK, NULL, SHAPE, DTYPE, ALIAS, UNSUP, LAUNCH, WORKSPACE}

    def pick(ordinary, extreme):
        return rng.choice(extreme) if rng.random() < 0.15 else rng.choice(ordinary)

    def rows():
        return B.Rows(0, 0) if rng.random() < 0.7 else B.Rows(pick([64, 4096, 1 << 20], I64), pick([64, 128], I64))

    seen = set()
    for _ in range(1500):
        b, ln, d = pick([1, 2, 5], I64), pick([1, 7, 300], I64), pick([8, 64, 100], I64)
        dt = pick([0, 1], [2, -1])
        c = B.ConvShape(b, ln, d, pick([2, 3, 4], I32), dt, pick([0, 1], I32), pick([8], I32), rows(), rows(), rows(), rows())
        s = B.SsmShape(b, ln, d, pick([1, 16, 64], I32), dt, pick([0, 1], I32), pick([8], I32), *[rows() for _ in range(12)])
        n = B.NormShape(b, d, dt, pick([0, 32, 64, 128], I32), pick([1e-5], [0.0, float("nan")]), pick([0], I32),
                        *[pick([0], I64) for _ in range(7)])
        ptr = [P(A[i] if rng.random() < 0.95 else 0) for i in range(24)]
        got = [lib.la_short_conv(*ptr[:7], ctypes.byref(c)), lib.la_short_conv_bwd(*ptr[:12], 1 << 40, ctypes.byref(c)),
               lib.la_short_conv_step(*ptr[:6], ctypes.byref(c)), lib.la_ssm_scan(*ptr[:13], 1 << 50, ctypes.byref(s)),
               lib.la_ssm_scan_bwd(*ptr[:22], 1 << 50, ctypes.byref(s)), lib.la_ssm_step(*ptr[:11], ctypes.byref(s)),
               lib.la_add_norm(*ptr[:6], ctypes.byref(n)), lib.la_add_norm_q8(*ptr[:7], ctypes.byref(n)),
               lib.la_add_norm_bwd(*ptr[:8], 1 << 40, ctypes.byref(n))]
        assert set(got) <= codes, got
        seen |= {(i, r) for i, r in enumerate(got)}
        for w in (lib.la_short_conv_bwd_workspace(ctypes.byref(c)), lib.la_ssm_workspace(ctypes.byref(s), 0),
                  lib.la_ssm_workspace(ctypes.byref(s), 1), lib.la_add_norm_bwd_workspace(ctypes.byref(n))):
            assert w >= 0 or w in codes
    for i in range(9):
        assert (i, LAUNCH) in seen or (i, OK) in seen, i
        assert len({r for k, r in seen if k == i}) >= 4, i


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(2, 8, 16), torch.zeros(16, 4)
    with pytest.raises(ValueError, match="device tensor"):
        B.la_short_conv(x, w)
    with pytest.raises(ValueError, match="dims"):
        B.la_short_conv(x[0], w)
    with pytest.raises(ValueError, match="device tensor"):
        B.la_short_conv_step(x[:, 0], w, torch.zeros(4, 3, 16))
    with pytest.raises(ValueError, match="device tensor"):
        B.la_ssm_scan(x, x, torch.zeros(16, 4), x, x)
    with pytest.raises(ValueError, match="unsupported dtype"):
        B.la_add_norm(x[0].double(), torch.zeros(16))
    with pytest.raises(ValueError, match="group"):
        B.la_add_norm_q8(x[0], torch.zeros(16), group=48)
