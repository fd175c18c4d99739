"""Plain fp64 forms of the short convolution, the selective scan and the residual norm (numpy, token by
token), their derivatives by formula, and the magnitudes that rounding errors are measured against.

With ``mag=True`` every sum is taken over the absolute values of its terms: a computation of the same sums
in fp32, in any order, is off by at most K 2^-24 of that magnitude, K the length of the longest chain of
roundings that reaches a value.  Storing a result rounds it by at most half a step of its type.
"""
import numpy as np
import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
U = 2.0 ** -24


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def close(got, ref, mag, K, dtype=torch.float32, what=""):
    """got within half a step of its type plus K roundings of the magnitude."""
    g = f64(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    tol = HALF[dtype] * np.abs(ref) + K * U * mag * (1 + HALF[dtype]) + 1e-37
    bad = ~(np.abs(g - ref) <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(g - ref) / tol, 0)), ref.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, worst at {i}: {g[i]} against {ref[i]}, "
                             f"tolerance {tol[i]:.3e}")


def sig(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


def silu(x):
    return x * sig(x)


def dsilu(x):
    s = sig(x)
    return s * (1 + x * (1 - s))


def dsilu_mag(x):
    """silu'(x) = s + s x (1 - s) is a sum of two terms that cancel near x = -1.28: its roundings are relative to
    their absolute values' sum, not to the value."""
    s = sig(x)
    return s * (1 + np.abs(x) * (1 - s))


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def conv(x, w, b, state, lengths, act):
    """(y, state_out) with y zero behind a sequence's end."""
    B, L, D = x.shape
    W = w.shape[1]
    y, so = np.zeros_like(x), np.zeros((B, W - 1, D))
    for i in range(B):
        n = L if lengths is None else lengths[i]
        xs = np.concatenate([np.zeros((W - 1, D)) if state is None else state[i], x[i, :n]])
        for t in range(n):
            v = (w.T * xs[t : t + W]).sum(0) + (0 if b is None else b)
            y[i, t] = silu(v) if act else v
        so[i] = xs[n:]
    return y, so


def conv_bwd(x, w, b, state, lengths, act, dy, dso, mag=False):
    """(dx, dw, db, dstate)."""
    B, L, D = x.shape
    W = w.shape[1]
    a = np.abs if mag else (lambda v: v)
    dx, dw, db, ds = np.zeros_like(x), np.zeros_like(w), np.zeros(D), np.zeros((B, W - 1, D))
    for i in range(B):
        n = L if lengths is None else lengths[i]
        xs = np.concatenate([np.zeros((W - 1, D)) if state is None else state[i], x[i, :n]])
        g = np.zeros_like(xs)
        for t in range(n):
            v = (w.T * xs[t : t + W]).sum(0) + (0 if b is None else b)
            # silu' moves by at most |its second derivative| <= 1/2 per unit of v: the error of v counts too
            p = a(dy[i, t]) * (1.0 if not act else dsilu_mag(v) if mag else dsilu(v))
            if mag and act:
                p = p + np.abs(dy[i, t]) * ((np.abs(w.T) * np.abs(xs[t : t + W])).sum(0) + (0 if b is None else np.abs(b)))
            g[t : t + W] += a(w.T) * p
            dw += (a(xs[t : t + W]) * p).T
            db += p
        if dso is not None:
            g[n:] += a(dso[i])
        dx[i, :n], ds[i] = g[W - 1 :], g[: W - 1]
    return dx, dw, db, ds


def scan(u, dt, A, Bm, C, D, z, bias, s_in, lengths, sp, mag=False):
    """(y, s_out, kept): kept[i] = the states before each token and after the last."""
    a = np.abs if mag else (lambda v: v)
    B, L, Dn = u.shape
    N = A.shape[1]
    y, so, kept = np.zeros_like(u), np.zeros((B, N, Dn)), []
    for i in range(B):
        n = L if lengths is None else lengths[i]
        h = np.zeros((N, Dn)) if s_in is None else a(s_in[i]).copy()
        ks = [h]
        for t in range(n):
            x = dt[i, t] + (0 if bias is None else bias)
            dl = softplus(x) if sp else x
            h = np.exp(dl * A.T) * h + a(Bm[i, t])[:, None] * a(dl * u[i, t])
            v = (a(C[i, t])[:, None] * h).sum(0) + (0 if D is None else a(D * u[i, t]))
            y[i, t] = v if z is None else v * a(silu(z[i, t]))
            ks.append(h)
        so[i] = h
        kept.append(ks)
    return y, so, kept


def scan_bwd(u, dt, A, Bm, C, D, z, bias, s_in, lengths, sp, dy, ds_out, mag=False):
    """(du, ddt, dA, dB, dC, dD, dz, dbias, ds_in)."""
    a = np.abs if mag else (lambda v: v)
    _, _, kept = scan(u, dt, A, Bm, C, D, z, bias, s_in, lengths, sp, mag)
    B, L, Dn = u.shape
    N = A.shape[1]
    du, ddt, dz = np.zeros_like(u), np.zeros_like(u), np.zeros_like(u)
    dA, dB, dC = np.zeros_like(A), np.zeros_like(Bm), np.zeros_like(C)
    dD, dbias, ds_in = np.zeros(Dn), np.zeros(Dn), np.zeros((B, N, Dn))
    Dv = np.zeros(Dn) if D is None else a(D)
    for i in range(B):
        n = L if lengths is None else lengths[i]
        g = np.zeros((N, Dn)) if ds_out is None else a(ds_out[i]).copy()
        for t in range(n - 1, -1, -1):
            x = dt[i, t] + (0 if bias is None else bias)
            dl = softplus(x) if sp else x
            ut, b, c = a(u[i, t]), a(Bm[i, t])[:, None], a(C[i, t])[:, None]
            before, after = kept[i][t], kept[i][t + 1]
            zt = None if z is None else z[i, t]
            ds = a(dy[i, t]) if z is None else a(dy[i, t] * silu(zt))
            e = np.exp(dl * A.T)
            g = g + c * ds
            gw = g * e * before
            if mag:  # the kernels form e * before as after - delta u B
                gw = g * (after + b * a(dl * u[i, t]))
            gb = (g * b).sum(0)
            dd = gb * ut + (gw * a(A.T)).sum(0)
            du[i, t] = ds * Dv + gb * a(dl)
            ddt[i, t] = dd * (sig(x) if sp else 1.0)
            dA += (gw * a(dl)).T
            dB[i, t] = (g * a(dl * u[i, t])).sum(1)
            dC[i, t] = (after * ds).sum(1)
            dD += ds * ut
            if z is not None:
                inner = (c * after).sum(0) + Dv * ut
                dz[i, t] = a(dy[i, t]) * (dsilu_mag(zt) if mag else dsilu(zt)) * inner
            dbias += ddt[i, t]
            g = g * e
        ds_in[i] = g
    return du, ddt, dA, dB, dC, dD, dz, dbias, ds_in


def norm(x, res, w, eps):
    h = x if res is None else x + res
    r = 1 / np.sqrt((h * h).mean(1) + eps)
    return h * r[:, None] * w, h, r


def norm_bwd(dy, h, w, r, dh, mag=False):
    a = np.abs if mag else (lambda v: v)
    xh = a(h) * r[:, None]
    p = a(dy) * a(w)
    m = (p * xh).mean(1, keepdims=True)
    dx = r[:, None] * (p + xh * m if mag else p - xh * m)
    if dh is not None:
        dx = dx + a(dh)
    return dx, (a(dy) * xh).sum(0)
