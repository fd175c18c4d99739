"""Benchmark cases of the selective state space operators: the short causal convolution, the selective
scan and the residual root-mean-square norm, for prompts, training and single tokens.

Each case names an operator (``op``) and its sizes.  ``run`` computes it in plain torch operations (``own``
false) or through the library's entry points (``own`` true); ``exact`` computes it in 64 bits, token by token.

Layouts: activations [B, L, D] (channels contiguous), the scan's B and C [B, L, N], the scan's state
[B, N, D] float32, the convolution's state [B, W - 1, D] (oldest input first), parameters float32.
"""
import math

import torch

own = False

EPS = 1e-5


def listed():
    return [
        # a prompt at the per-device shape (16 heads of 128 channels, 16384 tokens) through the convolution; the
        # input is one half of a projection's output, the gate the other half
        dict(name="conv_prompt", op="conv", B=1, L=16384, D=2048, W=4, dtype="bf16", ragged=False),
        # continued, padded prompts of unequal lengths at an odd width, in fp32
        dict(name="conv_ragged_f32", op="conv", B=5, L=777, D=1000, W=3, dtype="f32", ragged=True),
        # the convolution in training: forward and backward
        dict(name="conv_train", op="conv_train", B=2, L=4096, D=2048, W=4, dtype="bf16", ragged=False),
        # one new token of each of 64 running requests, their states in a pool of slots
        dict(name="conv_step", op="conv_step", B=64, D=2048, W=4, S=96, dtype="bf16"),
        # the selective scan over the same prompt
        dict(name="scan_prompt", op="scan", B=1, L=16384, D=2048, N=16, dtype="bf16", gate=True, ragged=False),
        # continued, padded prompts at an odd width and state size, in fp32
        dict(name="scan_ragged_f32", op="scan", B=5, L=777, D=1000, N=24, dtype="f32", gate=False, ragged=True),
        # a training step of the scan: forward and backward
        dict(name="scan_train", op="scan_train", B=2, L=4096, D=2048, N=16, dtype="bf16", gate=True, ragged=False),
        # a small, odd training step with incoming and outgoing state derivatives
        dict(name="scan_train_odd_f32", op="scan_train", B=3, L=333, D=200, N=16, dtype="f32", gate=False, ragged=True),
        # one new token of one request: latency
        dict(name="scan_step_one", op="scan_step", B=1, D=2048, N=16, S=1, dtype="bf16", gate=True),
        # one new token of each of 256 running requests
        dict(name="scan_step_many", op="scan_step", B=256, D=4096, N=16, S=300, dtype="bf16", gate=True),
        # the norm before a mixer with an 8-bit output for its projection, a prompt's tokens
        dict(name="norm_q8", op="norm_q8", M=16384, D=2048, dtype="bf16", group=128),
        # the norm's backward in training
        dict(name="norm_train", op="norm_bwd", M=8191, D=2048, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_train", "conv_step", "scan", "scan_train", "scan_step", "norm", "norm_q8", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    D = _log(rng, 64, 4096)
    if rng.random() < 0.5:
        D = max(64, D // 64 * 64)
    c = dict(op=op, D=D, dtype=dtype)
    if op.endswith("step"):
        c["B"] = _log(rng, 1, 256)
        c["S"] = c["B"] + rng.randrange(0, 64)
    elif op.startswith("norm"):
        c["M"] = _log(rng, 1, 16384)
        if op == "norm_q8":
            c["D"] = max(128, D // 128 * 128)
            c["group"] = rng.choice([0, 32, 64, 128])
    else:
        c["B"] = rng.choice([1, 2, 3, 4, 5, 8])
        # at most a quarter of the largest listed scan's tokens times channels, a tenth in training
        most = 16384 * 2048 // (8 if op == "scan_train" else 4)
        c["L"] = max(1, min(_log(rng, 1, 16384), most // (c["B"] * c["D"])))
        c["ragged"] = rng.random() < 0.5
    if op.startswith("conv"):
        c["W"] = rng.choice([2, 3, 4])
    if op.startswith("scan"):
        c["N"] = rng.choice([8, 16, 16, 16, 24, 32])
        c["gate"] = rng.random() < 0.7
    return c


def _dt(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, D = _dt(case), case["D"]

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    s = dict(case=case)
    op = case["op"]
    if op.startswith("norm"):
        M = case["M"]
        s["weight"] = 1 + normal(D, std=0.1)
        if op == "norm_bwd":
            s["h"] = normal(M, D, std=2.0, dtype=dt)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
            s["dy"], s["dh"] = normal(M, D, dtype=dt), normal(M, D, dtype=dt)
        else:
            s["x"], s["res"] = normal(M, D, dtype=dt), normal(M, D, std=2.0, dtype=dt)
        return s
    B = case["B"]
    step = op.endswith("step")
    if step:
        # which slot of the pool each request holds
        s["slots"] = torch.randperm(case["S"], generator=g, device="cuda")[:B].to(torch.int32)
    elif case["ragged"]:
        s["lengths"] = (uniform(B) * (case["L"] + 1)).to(torch.int32).clamp_(0, case["L"])
    rows = (B,) if step else (B, case["L"])
    if op.startswith("conv"):
        W = case["W"]
        # the first half of the projection's output rows; the second half is the scan's gate
        s["x"] = normal(*rows, 2 * D, dtype=dt)[..., :D]
        s["weight"] = normal(D, W, std=W ** -0.5)
        s["bias"] = normal(D, std=0.1)
        if step:
            s["state"] = normal(case["S"], W - 1, D, dtype=dt)
        elif op == "conv_train" or case["ragged"]:
            s["state_in"] = normal(B, W - 1, D, dtype=dt)
        if not step:
            s["y"] = torch.zeros(*rows, D, dtype=dt, device="cuda")
        if op == "conv_train":
            s["dy"] = normal(*rows, D, dtype=dt)
            s["d_state_out"] = normal(B, W - 1, D, dtype=dt)
        return s
    N = case["N"]
    # u: what leaves the convolution; dt: a projection's output around a bias whose softplus is log-uniform in
    # [0.001, 0.1]; A: -1..-N per channel, a little apart; B and C: slices of one projection's output
    x = normal(*rows, D)
    s["u"] = (x * torch.sigmoid(x)).to(dt)
    s["dt"] = normal(*rows, D, std=0.5, dtype=dt)
    step0 = torch.exp(uniform(D, lo=math.log(1e-3), hi=math.log(1e-1)))
    s["dt_bias"] = step0 + torch.log(-torch.expm1(-step0))
    s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(normal(D, N, std=0.05))
    bc = normal(*rows, 64 + 2 * N, dtype=dt)
    s["B"], s["C"] = bc[..., 64 : 64 + N], bc[..., 64 + N :]
    s["D"] = 1 + normal(D, std=0.1)
    if case["gate"]:
        s["z"] = normal(*rows, 2 * D, dtype=dt)[..., D:]
    if step:
        s["state"] = normal(case["S"], N, D, std=0.2)
    else:
        s["y"] = torch.zeros(*rows, D, dtype=dt, device="cuda")
        if op == "scan_train" or case["ragged"]:
            s["s_in"] = normal(B, N, D, std=0.2)
    if op == "scan_train":
        s["dy"] = normal(*rows, D, dtype=dt)
        s["ds_out"] = normal(B, N, D)
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    from chunked_scan_amd import binding as la

    op = s["case"]["op"]
    get = s.get
    if op == "conv":
        return la.la_short_conv(s["x"], s["weight"], s["bias"], get("state_in"), lengths=get("lengths"), y=s["y"],
                                want_state=True)
    if op == "conv_train":
        y, state = la.la_short_conv(s["x"], s["weight"], s["bias"], s["state_in"], lengths=get("lengths"), y=s["y"],
                                    want_state=True)
        return (y, state) + tuple(la.la_short_conv_bwd(s["x"], s["weight"], s["dy"], s["bias"], s["state_in"],
                                                       s["d_state_out"], lengths=get("lengths")))
    if op == "conv_step":
        return la.la_short_conv_step(s["x"], s["weight"], s["state"], s["bias"], slots=s["slots"]), s["state"]
    if op.startswith("scan"):
        a = (s["u"], s["dt"], s["A"], s["B"], s["C"])
        kw = dict(D=s["D"], z=get("z"), dt_bias=s["dt_bias"])
        if op == "scan_step":
            return la.la_ssm_step(*a, s["state"], slots=s["slots"], **kw), s["state"]
        kw.update(s_in=get("s_in"), lengths=get("lengths"))
        out = la.la_ssm_scan(*a, y=s["y"], **kw)
        if op == "scan_train":
            out = tuple(out) + tuple(la.la_ssm_scan_bwd(*a, s["dy"], ds_out=s["ds_out"], **kw))
        return out
    if op == "norm":
        return la.la_add_norm(s["x"], s["weight"], s["res"], eps=EPS)
    if op == "norm_q8":
        return la.la_add_norm_q8(s["x"], s["weight"], s["res"], eps=EPS, group=s["case"]["group"])
    return la.la_add_norm_bwd(s["dy"], s["h"], s["weight"], s["rstd"], s["dh"])


# ------------------------------------------------------------------------------- the plain form


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _recur(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from zero, by doubling."""
    s, L = 1, a.shape[1]
    while s < L:
        b = torch.cat([b[:, :s], b[:, s:] + a[:, s:] * b[:, :-s]], 1)
        a = torch.cat([a[:, :s], a[:, s:] * a[:, :-s]], 1)
        s *= 2
    return b


def _mask(s, L, dev):
    if s.get("lengths") is None:
        return None
    return (torch.arange(L, device=dev)[None, :] < s["lengths"][:, None])[:, :, None]


def _conv_plain(s):
    x, w, b = s["x"].float(), s["weight"], s["bias"]
    B, L, D = x.shape
    W = w.shape[1]
    st = s["state_in"].float() if s.get("state_in") is not None else x.new_zeros(B, W - 1, D)
    xp = torch.cat([st, x], 1)
    win = xp.unfold(1, W, 1)  # [B, L, D, W]
    pre = (win * w).sum(-1) + b
    n = s["lengths"].long() if s.get("lengths") is not None else torch.full((B,), L, device=x.device)
    at = n[:, None] + torch.arange(W - 1, device=x.device)
    state = torch.gather(xp, 1, at[:, :, None].expand(B, W - 1, D))
    return pre, win, state, at


def _plain(s):
    case = s["case"]
    op, dt = case["op"], _dt(case)
    if op in ("conv", "conv_train"):
        pre, win, state, at = _conv_plain(s)
        B, L, D = pre.shape
        W = s["weight"].shape[1]
        m = _mask(s, L, pre.device)
        sig = torch.sigmoid(pre)
        y = pre * sig
        if m is not None:
            y = torch.where(m, y, torch.zeros_like(y))
        out = (y.to(dt), state.to(dt))
        if op == "conv":
            return out
        dpre = s["dy"].float() * sig * (1 + pre * (1 - sig))
        if m is not None:
            dpre = torch.where(m, dpre, torch.zeros_like(dpre))
        pad = torch.cat([dpre.new_zeros(B, W - 1, D), dpre, dpre.new_zeros(B, W - 1, D)], 1)
        dxp = (pad.unfold(1, W, 1) * s["weight"].flip(1)).sum(-1)  # [B, W - 1 + L, D]
        dxp = dxp.scatter_add(1, at[:, :, None].expand(B, W - 1, D), s["d_state_out"].float())
        dw = (dpre[..., None] * win).sum((0, 1))
        return out + (dxp[:, W - 1 :].to(dt), dw, dpre.sum((0, 1)), dxp[:, : W - 1].to(dt))
    if op == "conv_step":
        at = s["slots"].long()
        win = torch.cat([s["state"][at].float(), s["x"].float()[:, None]], 1)  # [B, W, D]
        pre = (win * s["weight"].t()).sum(1) + s["bias"]
        s["state"][at] = win[:, 1:].to(dt)
        return (pre * torch.sigmoid(pre)).to(dt), s["state"]
    if op == "scan_step":
        at = s["slots"].long()
        u, delta = s["u"].float(), _softplus(s["dt"].float() + s["dt_bias"])
        h = torch.exp(delta[:, None] * s["A"].t()) * s["state"][at]
        h = h + (delta * u)[:, None] * s["B"].float()[:, :, None]
        s["state"][at] = h
        y = (h * s["C"].float()[:, :, None]).sum(1) + s["D"] * u
        if s.get("z") is not None:
            z = s["z"].float()
            y = y * z * torch.sigmoid(z)
        return y.to(dt), s["state"]
    if op in ("scan", "scan_train"):
        u, x = s["u"].float(), s["dt"].float() + s["dt_bias"]
        Bn, L, D = u.shape
        m = _mask(s, L, u.device)
        delta = _softplus(x)
        if m is not None:
            delta = torch.where(m, delta, torch.zeros_like(delta))
        Bm, C = s["B"].float()[..., None], s["C"].float()[..., None]
        A = s["A"].t()
        a = torch.exp(delta[:, :, None] * A)  # [B, L, N, D]
        b = (delta * u)[:, :, None] * Bm
        if s.get("s_in") is not None:
            b[:, 0] += a[:, 0] * s["s_in"]
        h = _recur(a, b)
        del b
        inner = (h * C).sum(2) + s["D"] * u
        z = s["z"].float() if s.get("z") is not None else None
        sig = torch.sigmoid(z) if z is not None else None
        y = inner if z is None else inner * z * sig
        if m is not None:
            y = torch.where(m, y, torch.zeros_like(y))
        out = (y.to(dt), h[:, -1].clone())
        if op == "scan":
            return out
        dy = s["dy"].float()
        if m is not None:
            dy = torch.where(m, dy, torch.zeros_like(dy))
        ds = dy if z is None else dy * z * sig
        dz = None if z is None else (dy * inner * sig * (1 + z * (1 - sig))).to(dt)
        c = (ds[:, :, None] * C).flip(1)
        c[:, 0] += s["ds_out"]
        g = _recur(torch.cat([torch.ones_like(a[:, :1]), a.flip(1)[:, :-1]], 1), c).flip(1)
        del c
        ds_in = a[:, 0] * g[:, 0]
        w = a * torch.cat([s["s_in"][:, None], h[:, :-1]], 1) * g
        del a
        gb = (g * Bm).sum(2)
        if m is not None:
            gb = torch.where(m, gb, torch.zeros_like(gb))
            w = torch.where(m[..., None], w, torch.zeros_like(w))
        du = ds * s["D"] + gb * delta
        ddt = (gb * u + (w * A).sum(2)) * torch.sigmoid(x)
        dA = (w * delta[:, :, None]).sum((0, 1)).t().contiguous()
        dB = (g * (delta * u)[:, :, None]).sum(3)
        dC = (h * ds[:, :, None]).sum(3)
        return out + (du.to(dt), ddt.to(dt), dA, dB.to(dt), dC.to(dt), (ds * u).sum((0, 1)), dz, ddt.sum((0, 1)), ds_in)
    w = s["weight"]
    if op == "norm_bwd":
        xh = s["h"].float() * s["rstd"][:, None]
        dy = s["dy"].float()
        dxh = dy * w
        dx = s["rstd"][:, None] * (dxh - xh * (dxh * xh).mean(1, keepdim=True)) + s["dh"].float()
        return dx.to(dt), (dy * xh).sum(0)
    h = s["x"].float() + s["res"].float()
    rstd = torch.rsqrt(h.square().mean(1) + EPS)
    y = h * rstd[:, None] * w
    if op == "norm":
        return y.to(dt), h.to(dt), rstd
    grp = case["group"] or case["D"]
    yg = y.view(y.shape[0], -1, grp)
    amax = yg.abs().amax(2)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    q = (yg / scale[..., None]).clamp(-448.0, 448.0).view_as(y).to(torch.float8_e4m3fn)
    return q, scale, h.to(dt), rstd


# ------------------------------------------------------------------------------- in 64 bits


def work(case):
    """Bytes: each input read once, each output written once.  Flops: an exponential, a product or a sum is one."""
    op, D = case["op"], case["D"]
    e = 4 if case["dtype"] == "f32" else 2
    if op.startswith("norm"):
        n = case["M"] * D
        if op == "norm_bwd":
            return dict(bytes=n * e * 4 + case["M"] * 4 + D * 8, flops=n * 11)
        if op == "norm_q8":
            groups = D // case["group"] if case["group"] else 1
            return dict(bytes=n * (3 * e + 1) + case["M"] * 4 * (1 + groups) + D * 4, flops=n * 8)
        return dict(bytes=n * e * 4 + case["M"] * 4 + D * 4, flops=n * 5)
    B, L = case["B"], case.get("L", 1)
    n = B * L * D
    if op.startswith("conv"):
        W = case["W"]
        par, st = D * (W + 1) * 4, B * (W - 1) * D * e
        if op == "conv_step":
            return dict(bytes=2 * n * e + 2 * st + par, flops=n * (2 * W + 5))
        if op == "conv":
            return dict(bytes=2 * n * e + st * (2 if case["ragged"] else 1) + par, flops=n * (2 * W + 5))
        # the forward reads x and writes y; the backward reads x and dy and writes dx
        return dict(bytes=5 * n * e + 5 * st + 3 * par, flops=n * (8 * W + 20))
    N, z = case["N"], int(case["gate"])
    par, st, bc = D * (N + 2) * 4, B * N * D * 4, 2 * B * L * N * e
    if op == "scan_step":
        return dict(bytes=(3 + z) * n * e + 2 * st + par + bc, flops=n * (7 * N + 15))
    if op == "scan":
        return dict(bytes=(3 + z) * n * e + st * (2 if case["ragged"] else 1) + par + bc, flops=n * (7 * N + 15))
    # forward, then: u, dt, z, dy, B, C in, du, ddt, dz, dB, dC out; the states once more
    return dict(bytes=(3 + z + 5 + 2 * z) * n * e + 5 * st + 3 * par + 3 * bc, flops=n * (28 * N + 40))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {k: (v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v) for k, v in s.items()}
    silu = lambda t: t / (1 + torch.exp(-t))  # noqa: E731
    dsilu = lambda t: (1 + torch.exp(-t) * (1 + t)) / (1 + torch.exp(-t)).square()  # noqa: E731
    soft = lambda t: torch.where(t > 0, t + torch.log1p(torch.exp(-t.abs())), torch.log1p(torch.exp(t)))  # noqa: E731
    if op.startswith("norm"):
        if op == "norm_bwd":
            r = d["rstd"][:, None]
            p = d["dy"] * d["weight"]
            dot = (p * d["h"]).sum(1, keepdim=True) / case["D"]
            return p * r - d["h"] * r ** 3 * dot + d["dh"], (d["dy"] * d["h"] * r).sum(0)
        h = d["x"] + d["res"]
        ms = h.pow(2).sum(1) / case["D"] + EPS
        y = h * d["weight"] / ms.sqrt()[:, None]
        if op == "norm":
            return y, h, 1 / ms.sqrt()
        grp = case["group"] or case["D"]
        amax = y.reshape(y.shape[0], -1, grp).abs().max(2).values
        return None, amax / 448, h, 1 / ms.sqrt()
    if op.startswith("conv"):
        x, w = d["x"], d["weight"]
        W = w.shape[1]
        if op == "conv_step":
            at = s["slots"].long()
            win = [d["state"][at, j] for j in range(W - 1)] + [x]
            pre = d["bias"] + sum(w[:, j] * win[j] for j in range(W))
            state = d["state"].clone()
            for j in range(W - 1):
                state[at, j] = win[j + 1]
            return silu(pre), state
        Bn, L, D = x.shape
        lens = s["lengths"].tolist() if s.get("lengths") is not None else [L] * Bn
        y, dx = torch.zeros_like(x), torch.zeros_like(x)
        state = torch.zeros(Bn, W - 1, D, dtype=x.dtype, device=x.device)
        dw, db, dst = torch.zeros_like(w), torch.zeros_like(d["bias"]), torch.zeros_like(state)
        for i, n in enumerate(lens):
            xs = torch.zeros(W - 1 + n, D, dtype=x.dtype, device=x.device)
            if d.get("state_in") is not None:
                xs[: W - 1] = d["state_in"][i]
            xs[W - 1 :] = x[i, :n]
            pre = d["bias"] + sum(w[:, j] * xs[j : j + n] for j in range(W))
            y[i, :n], state[i] = silu(pre), xs[n:]
            if op == "conv_train":
                dp = d["dy"][i, :n] * dsilu(pre)
                dxs = torch.zeros_like(xs)
                for j in range(W):
                    dxs[j : j + n] += w[:, j] * dp
                    dw[:, j] += (dp * xs[j : j + n]).sum(0)
                dxs[n:] += d["d_state_out"][i]
                db += dp.sum(0)
                dx[i, :n], dst[i] = dxs[W - 1 :], dxs[: W - 1]
        return (y, state) if op == "conv" else (y, state, dx, dw, db, dst)
    A = d["A"].t()
    if op == "scan_step":
        at = s["slots"].long()
        delta = soft(d["dt"] + d["dt_bias"])
        h = torch.exp(delta[:, None, :] * A) * d["state"][at] + d["B"][:, :, None] * (delta * d["u"])[:, None, :]
        y = (d["C"][:, None, :] @ h)[:, 0] + d["D"] * d["u"]
        state = d["state"].clone()
        state[at] = h
        return (y if d.get("z") is None else y * silu(d["z"])), state
    u, x = d["u"], d["dt"] + d["dt_bias"]
    Bn, L, D = u.shape
    delta = soft(x)
    live = torch.ones(Bn, L, dtype=torch.bool, device=u.device)
    if s.get("lengths") is not None:
        live = torch.arange(L, device=u.device)[None] < s["lengths"][:, None]
    h = d["s_in"].clone() if d.get("s_in") is not None else torch.zeros(Bn, case["N"], D, dtype=u.dtype, device=u.device)
    inner = torch.zeros_like(u)
    kept = []
    for t in range(L):
        on = live[:, t, None, None]
        new = torch.exp(delta[:, t, None] * A) * h + d["B"][:, t, :, None] * (delta[:, t] * u[:, t])[:, None]
        if op == "scan_train":
            kept.append(h)
        h = torch.where(on, new, h)
        inner[:, t] = (d["C"][:, t, :, None] * h).sum(1) + d["D"] * u[:, t]
    z = d.get("z")
    y = (inner if z is None else inner * silu(z)) * live[..., None]
    if op == "scan":
        return y, h
    dy = d["dy"] * live[..., None]
    ds = dy if z is None else dy * silu(z)
    dz = None if z is None else dy * inner * dsilu(z)
    s_last, g = h, d["ds_out"].clone()
    du, dd = torch.zeros_like(u), torch.zeros_like(u)
    dA = torch.zeros_like(A)
    dB, dC = torch.zeros_like(d["B"]), torch.zeros_like(d["C"])
    after = s_last
    for t in range(L - 1, -1, -1):
        on = live[:, t, None, None]
        before = kept.pop()
        a = torch.exp(delta[:, t, None] * A)
        g = torch.where(on, g + d["C"][:, t, :, None] * ds[:, t, None], g)
        lg = torch.where(on, g, torch.zeros_like(g))
        gah = lg * a * before
        gb = (lg * d["B"][:, t, :, None]).sum(1)
        du[:, t] = ds[:, t] * d["D"] + gb * delta[:, t]
        dd[:, t] = gb * u[:, t] + (gah * A).sum(1)
        dA += (gah * delta[:, t, None]).sum(0)
        dB[:, t] = (lg * (delta[:, t] * u[:, t])[:, None]).sum(2)
        dC[:, t] = (after * ds[:, t, None]).sum(2)
        g = torch.where(on, g * a, g)
        after = before
    ddt = dd / (1 + torch.exp(-x))
    return y, s_last, du, ddt, dA.t().contiguous(), dB, dC, (ds * u).sum((0, 1)), dz, ddt.sum((0, 1)), g
