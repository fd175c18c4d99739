"""Plain fp64 forms of the gated recurrence, the norms around a block and counter-based dropout (numpy), their
derivatives by formula, and bounds on the roundings of an fp32 evaluation.

Every bound is in units of U = 2^-24 and is carried along with the value by the rule of each operation: a value v with
bound e, multiplied by a factor with relative bound k, has bound (e + k |v|) times the factor, and sums add.  Relative
bounds of the elementary steps, from the hardware's exponential, reciprocal and roots (1 ulp, so 2 U, each):
  sigma(r + b): two products and a sum in the exponent move it by 2 (|r| + |b|) U, then the exponential, a sum and
    a reciprocal: 2 (|r| + |b|) + 6;
  softplus: its polynomial's 1.3e-7 (3 U), the ulps of the exponential and of the reciprocal and a product: 10;
  v = c softplus rho: both and two products;   a = e^-v: v times (v's bound + 2), plus 2, and 2^-126 absolutely;
  1 - a^2 = 2 a v S: a's and v's and 8;   or directly (v > 1/2): 2 a^2 (a's bound + 1) / (1 - a^2) + 1;   its root: half and 3.
A state is carried by a product and a sum per token, and in segments by one product more: 4 U per token of H, the
recurrence of the terms' absolute values.
"""
import numpy as np

from mixer_ref import HALF, U, dsilu, dsilu_mag, f64, sig  # noqa: F401


def close(got, ref, err, dtype, what="", terms=0, mag=None):
    """got within half a step of its type and ``err`` U (with ``terms`` more roundings of ``mag``) of ref."""
    g = f64(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    e = err if mag is None else err + terms * mag
    tol = HALF[dtype] * np.abs(ref) + e * U * (1 + HALF[dtype]) + 1e-37
    bad = ~(np.abs(g - ref) <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(g - ref) / tol, 0)), ref.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, worst at {i}: {g[i]} against {ref[i]}, "
                             f"tolerance {tol[i]:.3e}")


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


class Gates:
    """rho, iota, v, a, m and their relative bounds in U."""

    def __init__(self, r, i, lam, rb, ib, c):
        rb = 0 if rb is None else rb
        ib = 0 if ib is None else ib
        fin = lambda t: np.where(np.isfinite(t), t, 0)  # noqa: E731
        self.rho, self.iota = sig(r + rb), sig(i + ib)
        self.k_rho, self.k_iota = 2 * (np.abs(fin(r)) + np.abs(rb)) + 6, 2 * (np.abs(fin(i)) + np.abs(ib)) + 6
        self.v = c * softplus(lam) * self.rho
        self.k_v = self.k_rho + 12
        self.a = np.exp(-self.v)
        # an exponential below fp32's normal range is flushed to zero: 2^-126 absolutely, whatever a is
        self.k_a = self.v * (self.k_v + 2) + 2 + 2.0 ** -126 / U / np.maximum(self.a, 1e-250)
        m2 = -np.expm1(-2 * self.v)
        self.m = np.sqrt(m2)
        safe = np.where(m2 > 0, m2, 1)
        direct = 2 * self.a ** 2 * (self.k_a + 1) / safe + 1
        self.k_m = np.where(self.v <= 0.5, self.k_a + self.k_v + 8, direct) / 2 + 3
        self.mi = self.m * self.iota
        self.k_mi = self.k_m + self.k_iota + 1
        # k = a^2 v / m^2
        self.slope = np.where(m2 > 0, self.a ** 2 * self.v / safe, 0.5)
        self.k_slope = np.where(self.v <= 0.5, self.k_a + 10, 2 * self.k_a + self.k_v + direct + 6)


def keep_of(lengths, B, L):
    n = np.full(B, L) if lengths is None else np.clip(np.asarray(lengths), 0, L)
    return np.arange(L)[None] < n[:, None]


def silu_of(z):
    """silu(z) and its relative bound."""
    return z * sig(z), 2 * np.abs(z) + 8


def scan(x, r, i, lam, rb, ib, z, h_in, lengths, c):
    """((y, bound), (h_out, bound), blocks, kept): y zero behind a sequence's end; blocks (value, bound) [B, ceil(L/64), D]
    with NaN where no token is; kept: what scan_bwd takes."""
    B, L, D = x.shape
    g = Gates(r, i, lam, rb, ib, c)
    live = keep_of(lengths, B, L)
    h = np.zeros((B, D)) if h_in is None else h_in.copy()
    H, e = np.abs(h), np.zeros((B, D))
    hs, He, befores = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
    es, e_befores, H_befores = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
    nb = -(-L // 64)
    blocks, eblocks = np.full((B, nb, D), np.nan), np.full((B, nb, D), np.nan)
    b = g.mi * x
    for t in range(L):
        on = live[:, t, None]
        if t % 64 == 0:
            blocks[:, t // 64], eblocks[:, t // 64] = np.where(on, h, np.nan), np.where(on, e, np.nan)
        befores[:, t], e_befores[:, t], H_befores[:, t] = h, e, H
        a, bt = g.a[:, t], b[:, t]
        e2 = a * (e + g.k_a[:, t] * H) + (g.k_mi[:, t] + 1) * np.abs(bt)
        H2 = a * H + np.abs(bt)
        h = np.where(on, a * h + bt, h)
        e = np.where(on, e2 + 4 * H2, e)
        H = np.where(on, H2, H)
        hs[:, t], es[:, t], He[:, t] = h, e, H
    on = live[..., None]
    if z is None:
        y, ey = hs, es
    else:
        s, ks = silu_of(z)
        y, ey = hs * s, np.abs(s) * (es + (ks + 1) * He)
    return (np.where(on, y, 0), np.where(on, ey, 0)), (h, e), (blocks, eblocks), (g, live, hs, es, He, befores, e_befores,
                                                                              H_befores, b)


def scan_bwd(x, r, i, lam, rb, ib, z, h_in, lengths, c, dy, dh_out):
    """[(value, bound)] of dx, dr, di, dlam, dr_bias, di_bias, dz, dh_in."""
    B, L, D = x.shape
    g, live, hs, es, He, before, e_before, H_before, b = scan(x, r, i, lam, rb, ib, z, h_in, lengths, c)[3]
    on = live[..., None]
    dy = np.where(on, dy, 0)
    if z is None:
        ds, eds = dy, np.zeros_like(dy)
        dz = None
    else:
        s, ks = silu_of(z)
        ds, eds = dy * s, np.abs(dy * s) * (ks + 1)
        dz = (dy * hs * dsilu(z), np.abs(dy) * (es * np.abs(dsilu(z)) + He * dsilu_mag(z) * (2 * np.abs(z) + 12)))
    carry = np.zeros((B, D)) if dh_out is None else dh_out.copy()
    ec, C = np.zeros((B, D)), np.abs(carry)
    gs, eg, G = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
    for t in range(L - 1, -1, -1):
        o = live[:, t, None]
        gt, Gt = ds[:, t] + carry, np.abs(ds[:, t]) + C
        et = eds[:, t] + ec + 4 * Gt
        gs[:, t], eg[:, t], G[:, t] = np.where(o, gt, 0), np.where(o, et, 0), np.where(o, Gt, 0)
        a = g.a[:, t]
        carry = np.where(o, a * gt, carry)
        ec = np.where(o, a * (et + (g.k_a[:, t] + 1) * Gt), ec)
        C = np.where(o, a * Gt, C)
    dx = (gs * g.mi, g.mi * (eg + (g.k_mi + 1) * G))
    ab = np.abs(b)
    di = (gs * b * (1 - g.iota), ab * (1 - g.iota) * (eg + (g.k_mi + 3) * G) + ab * G * (g.k_iota * g.iota + 1))
    q = gs * (g.slope * b - g.v * g.a * before)
    inner = g.slope * ab + g.v * g.a * H_before
    eq = eg * inner + G * (g.slope * ab * (g.k_slope + g.k_mi + 4)
                           + g.v * g.a * (e_before + (g.k_v + g.k_a + 4) * H_before))
    Q = G * inner
    dr = (q * (1 - g.rho), eq * (1 - g.rho) + Q * (g.k_rho * g.rho + 2))
    n = B * L + 8
    total = lambda v, e, mag: (v.sum((0, 1)), e.sum((0, 1)) + n * mag.sum((0, 1)))  # noqa: E731
    ratio = sig(lam) / softplus(lam)
    dlam = tuple(t * ratio for t in total(q, eq + 24 * Q, Q))
    return [dx, dr, di, dlam, total(*dr, Q), total(*di, ab * G), dz, (carry, ec)]


# ------------------------------------------------------------------------------- random numbers


def philox(ctr, key):
    """Philox4x32-10 of counters [..., 4] and key (two 32-bit words): [..., 4] uint32."""
    u = np.uint64
    c = [np.asarray(ctr)[..., k].astype(u) for k in range(4)]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(10):
        p0, p1 = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        lo = u(0xFFFFFFFF)
        c = [(p1 >> u(32)) ^ c[1] ^ u(k0), p1 & lo, (p0 >> u(32)) ^ c[3] ^ u(k1), p0 & lo]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, -1).astype(np.uint32)


def keep(seed, offset, M, D, p, rows=None):
    """(kept elements [M, D], the kept ones' factor); ``rows``: the rows' numbers, where they are not 0..M-1."""
    T = int(p * 65536 + 0.5)
    seed, offset = seed % 2 ** 64, offset % 2 ** 64
    nc = (D + 7) // 8
    m = np.arange(M, dtype=np.uint64) if rows is None else np.asarray(rows, dtype=np.uint64)
    n = (m[:, None] * np.uint64(nc) + np.arange(nc, dtype=np.uint64)[None])
    ctr = np.stack([n & np.uint64(0xFFFFFFFF), n >> np.uint64(32), np.full_like(n, offset & 0xFFFFFFFF),
                    np.full_like(n, offset >> 32)], -1)
    w = philox(ctr, (seed & 0xFFFFFFFF, seed >> 32))
    bits = np.stack([w & 0xFFFF, w >> 16], -1).reshape(len(m), nc * 8)[:, :D]
    return bits >= T, 65536 / (65536 - T)


# ------------------------------------------------------------------------------- norms


def act_of(gate, kind):
    """act, its derivative, and the bounds of both (relative to |act|, absolute for the derivative)."""
    if gate is None:
        return 1.0, 0.0, 0.0, 0.0
    if kind == "linear":
        return gate, np.ones_like(gate), 0.0, 0.0
    s, k = sig(gate), 2 * np.abs(gate) + 8
    if kind == "sigmoid":
        return s, s * (1 - s), k, s * ((1 - s) * (k + 2) + s * (k + 1))
    return gate * s, dsilu(gate), k + 1, dsilu_mag(gate) * (2 * k + 4)


def _rstd(v, err, eps):
    """1 / sqrt(mean v^2 + eps) and its relative bound: a lane's share of the sum, the lanes', and v's own bounds."""
    D = v.shape[1]
    ms = (v ** 2).mean(1, keepdims=True) + eps
    return 1 / np.sqrt(ms), D / 8 + 32 + (np.abs(v) * err).mean(1, keepdims=True) / ms


def block(x, gate, res, w_post, scale, w_pre, kind, eps, kept=None, factor=1.0):
    """(y, h, rp, rq), each (value, bound) or None."""
    n, en, rp = x, np.zeros_like(x), None
    if w_post is not None:
        r, k = _rstd(x, 0 * x, eps)
        n = x * r * w_post
        en = np.abs(n) * (k + 2)
        rp = (r[:, 0], r[:, 0] * k[:, 0])
    a, _, ka, _ = act_of(gate, kind)
    u = n * a
    eu = np.abs(a) * (en + (ka + 1) * np.abs(n))
    if scale is not None:
        u, eu = u * scale, np.abs(scale) * (eu + np.abs(u))
    if kept is not None:
        u, eu = np.where(kept, u * factor, 0), np.where(kept, factor * (eu + 2 * np.abs(u)), 0)
    h = u if res is None else u + res
    eh = eu + np.abs(h)
    if w_pre is None:
        return None, (h, eh), rp, None
    r, k = _rstd(h, eh, eps)
    y = h * r * w_pre
    return (y, np.abs(r * w_pre) * (eh + (k + 2) * np.abs(h))), (h, eh), rp, (r[:, 0], r[:, 0] * k[:, 0])


def block_bwd(x, gate, h, w_post, scale, w_pre, kind, rp, rq, dy, dh, kept=None, factor=1.0):
    """(value, bound) or None of dx, dresidual, dgate, dw_post, dw_pre, dscale."""
    M, D = x.shape
    terms = D / 8 + 16
    one = np.ones_like(x)
    dres, eres, dwq = np.zeros_like(x), np.zeros_like(x), None
    if w_pre is not None:
        hh = h * rq[:, None]
        t = dy * w_pre
        dot, dmag = (t * hh).mean(1, keepdims=True), np.abs(t * hh).mean(1, keepdims=True)
        dres = rq[:, None] * (t - hh * dot)
        eres = np.abs(rq[:, None]) * (4 * np.abs(t) + np.abs(hh) * (np.abs(dot) * 4 + dmag * (terms + 4)))
        dwq = ((dy * hh).sum(0), (M + 8) * np.abs(dy * hh).sum(0))
    if dh is not None:
        eres = eres + np.abs(dres) + np.abs(dh)
        dres = dres + dh
    du, edu = (dres, eres) if kept is None else (np.where(kept, dres * factor, 0),
                                                np.where(kept, factor * (eres + 2 * np.abs(dres)), 0))
    a, da, ka, eda = act_of(gate, kind)
    a = a * one
    xh = x * rp[:, None] if w_post is not None else x
    wp, sc = (one if w is None else w * one for w in (w_post, scale))
    n = xh * wp
    mag = np.abs(du * n)
    dgate = None
    if gate is not None:
        dgate = (du * n * sc * da, np.abs(n * sc) * (edu * np.abs(da) + np.abs(du) * (eda + 6 * np.abs(da))))
    dsc = None
    if scale is not None:
        dsc = ((du * n * a).sum(0), (np.abs(n * a) * edu + mag * np.abs(a) * (ka + 6)).sum(0)
               + (M + 8) * (mag * np.abs(a)).sum(0))
    dn, edn = du * a * sc, np.abs(a * sc) * (edu + np.abs(du) * (ka + 3))
    if w_post is None:
        return (dn, edn), (dres, eres), dgate, None, dwq, dsc
    dwp = ((dn * xh).sum(0), (np.abs(xh) * (edn + 2 * np.abs(dn))).sum(0) + (M + 8) * np.abs(dn * xh).sum(0))
    t, et = dn * wp, np.abs(wp) * (edn + np.abs(dn))
    dot, dmag = (t * xh).mean(1, keepdims=True), np.abs(t * xh).mean(1, keepdims=True)
    edot = (np.abs(xh) * et).mean(1, keepdims=True) + dmag * (terms + 3)
    dx = rp[:, None] * (t - xh * dot)
    edx = np.abs(rp[:, None]) * (et + 4 * np.abs(t) + np.abs(xh) * (edot + 4 * np.abs(dot)))
    return (dx, edx), (dres, eres), dgate, dwp, dwq, dsc
