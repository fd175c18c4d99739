"""Benchmark cases of a gated recurrent layer's operators: the gated linear recurrence (prompts, training, single
tokens), the norms after and before a block with its gate, residual scale and residual sum, and dropout from a
counter-based generator.

Each case names an operator (``op``) and its sizes.  ``run`` computes it in plain torch operations (``own``
false) or through the library's entry points (``own`` true); ``exact`` computes it in 64 bits.

Layouts: activations [B, L, D] or [M, D] (channels contiguous), the recurrence's state [B, D] float32, parameters
float32, the generator's seed and offset int64 [2].
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
C = 8.0  # the recurrence's log-decay is -C softplus(lam) times its gate


def listed():
    return [
        # a prompt at the per-device shape (16 heads of 128 channels, 16384 tokens) through the recurrence
        dict(name="scan_prompt", op="scan", B=1, L=16384, D=2048, dtype="bf16", gate=True, ragged=False),
        # continued, padded prompts of unequal lengths at an odd width, in fp32
        dict(name="scan_ragged_f32", op="scan", B=5, L=777, D=1000, dtype="f32", gate=False, ragged=True),
        # a training step of the recurrence: forward and backward
        dict(name="scan_train", op="scan_train", B=2, L=4096, D=2048, dtype="bf16", gate=True, ragged=False),
        # a small, odd training step with incoming and outgoing state derivatives
        dict(name="scan_train_odd_f32", op="scan_train", B=3, L=333, D=200, dtype="f32", gate=False, ragged=True),
        # one new token of one request: latency
        dict(name="step_one", op="step", B=1, D=2048, S=1, dtype="bf16", gate=True),
        # one new token of each of 256 running requests, their states in a pool of slots
        dict(name="step_many", op="step", B=256, D=4096, S=300, dtype="bf16", gate=True),
        # what stands between two blocks over a prompt: norm after the one, its gate and scale, residual, norm before
        # the next
        dict(name="norm_prompt", op="norm", M=16384, D=2048, dtype="bf16", act="silu", post=True, p=0.0),
        # the same for one token of each of 64 running requests
        dict(name="norm_token", op="norm", M=64, D=2048, dtype="bf16", act="silu", post=True, p=0.0),
        # its backward in training, with the branch's dropout
        dict(name="norm_train", op="norm_bwd", M=8191, D=2048, dtype="bf16", act="silu", post=True, p=0.1),
        # a small, odd one in fp32
        dict(name="norm_train_odd_f32", op="norm_bwd", M=333, D=1000, dtype="f32", act="sigmoid", post=True, p=0.1),
        # dropout of a branch on its way into the residual stream, a training batch
        dict(name="dropout_residual", op="dropout", M=16384, D=2048, dtype="bf16", p=0.1, residual=True),
        # a small, odd one in fp32
        dict(name="dropout_odd_f32", op="dropout", M=777, D=1001, dtype="f32", p=0.25, residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_train", "scan_train", "step", "norm", "norm_bwd", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    D = _log(rng, 64, 4096)
    if rng.random() < 0.5:
        D = max(64, D // 64 * 64)
    c = dict(op=op, D=D, dtype=dtype)
    if op == "step":
        c["B"] = _log(rng, 1, 256)
        c["S"] = c["B"] + rng.randrange(0, 64)
        c["gate"] = rng.random() < 0.7
    elif op.startswith("scan"):
        c["B"] = rng.choice([1, 2, 3, 4, 5, 8])
        # at most half of the largest listed scan's tokens times channels, a quarter in training
        most = 16384 * 2048 // (4 if op == "scan_train" else 2)
        c["L"] = max(1, min(_log(rng, 1, 16384), most // (c["B"] * c["D"])))
        c["gate"] = rng.random() < 0.7
        c["ragged"] = rng.random() < 0.5
    else:
        most = 16384 * 2048 // (4 if op == "norm_bwd" else 2)
        c["M"] = max(1, min(_log(rng, 1, 16384), most // D))
        c["p"] = rng.choice([0.1, 0.25, 0.5] if op == "dropout" else [0.0, 0.1, 0.25])
        if op == "dropout":
            c["residual"] = rng.random() < 0.6
        else:
            c["act"] = rng.choice(["none", "linear", "sigmoid", "silu", "silu"])  # none: no gate
            c["post"] = rng.random() < 0.7
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
    if "M" in case:
        M = case["M"]
        if case["p"] > 0:
            s["rng"] = torch.randint(0, 2 ** 62, (2,), generator=g, device="cuda")  # seed, offset
        if op == "dropout":
            s["x"] = normal(M, D, dtype=dt)
            s["res"] = normal(M, D, std=2.0, dtype=dt) if case["residual"] else None
            return s
        s["x"] = normal(M, D, std=3.0, dtype=dt)
        # the gate is the second half of a projection's output rows
        s["gate"] = normal(M, 2 * D, dtype=dt)[:, D:] if case["act"] != "none" else None
        s["w_post"] = 1 + normal(D, std=0.1) if case["post"] else None
        s["w_pre"] = 1 + normal(D, std=0.1)
        s["scale"] = uniform(D, lo=0.05, hi=0.5)
        if op == "norm":
            s["res"] = normal(M, D, std=2.0, dtype=dt)
            return s
        # what the forward leaves for the backward: the residual stream and the rows' reciprocal deviations
        s["h"] = normal(M, D, std=2.0, dtype=dt)
        s["rstd_pre"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
        s["rstd_post"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS) if case["post"] else None
        s["dy"], s["dh"] = normal(M, D, dtype=dt), normal(M, D, dtype=dt)
        return s
    B = case["B"]
    step = op == "step"
    if step:
        # which slot of the pool each request holds
        s["slots"] = torch.randperm(case["S"], generator=g, device="cuda")[:B].to(torch.int32)
    elif case["ragged"]:
        s["lengths"] = (uniform(B) * (case["L"] + 1)).to(torch.int32).clamp_(0, case["L"])
    rows = (B,) if step else (B, case["L"])
    # x: a convolution's output; r and i: the halves of one projection's output; lam: a decay at an open gate that is
    # uniform in [0.9, 0.999]
    s["x"] = normal(*rows, D, dtype=dt)
    ri = normal(*rows, 2 * D, dtype=dt)
    s["r"], s["i"] = ri[..., :D], ri[..., D:]
    s["lam"] = torch.log(torch.expm1(-torch.log(uniform(D, lo=0.9, hi=0.999)) / C))
    s["r_bias"], s["i_bias"] = normal(D, std=0.5), normal(D, std=0.5)
    if case["gate"]:
        s["z"] = normal(*rows, 2 * D, dtype=dt)[..., D:]
    if step:
        s["state"] = normal(case["S"], D)
        return s
    s["y"] = torch.zeros(*rows, D, dtype=dt, device="cuda")
    if op == "scan_train" or case["ragged"]:
        s["h_in"] = normal(B, D)
    if op == "scan_train":
        s["dy"] = normal(*rows, D, dtype=dt)
        s["dh_out"] = normal(B, D)
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    from chunked_scan_amd import binding as la

    case, get = s["case"], s.get
    op = case["op"]
    if op == "dropout":
        return la.la_dropout(s["x"], s["rng"], case["p"], s["res"])
    if op.startswith("norm"):
        kw = dict(w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"], scale=s["scale"], p=case["p"], rng=get("rng"),
                  act="linear" if case["act"] == "none" else case["act"])
        if op == "norm":
            return la.la_block_norm(s["x"], s["res"], eps=EPS, **kw)
        return la.la_block_norm_bwd(s["x"], s["h"], s["dy"], s["dh"], rstd_post=s["rstd_post"], rstd_pre=s["rstd_pre"],
                                    **kw)
    a = (s["x"], s["r"], s["i"], s["lam"])
    kw = dict(r_bias=s["r_bias"], i_bias=s["i_bias"], z=get("z"), c=C)
    if op == "step":
        return la.la_gated_step(*a, s["state"], slots=s["slots"], **kw), s["state"]
    kw.update(h_in=get("h_in"), lengths=get("lengths"))
    if op == "scan":
        return la.la_gated_scan(*a, y=s["y"], **kw)[:2]
    # the states that enter every 64 tokens, kept for the backward
    y, h_out, blocks = la.la_gated_scan(*a, y=s["y"], want_blocks=True, **kw)
    return (y, h_out) + tuple(la.la_gated_scan_bwd(*a, s["dy"], dh_out=s["dh_out"], h_blocks=blocks, **kw))


# ------------------------------------------------------------------------------- the plain form


def _recur(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from zero, by doubling."""
    s, L = 1, a.shape[1]
    while s < L:
        b = torch.cat([b[:, :s], b[:, s:] + a[:, s:] * b[:, :-s]], 1)
        a = torch.cat([a[:, :s], a[:, s:] * a[:, :-s]], 1)
        s *= 2
    return b


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _keep(s, M, D):
    """Which elements dropout keeps, times 1 / (share kept): Philox4x32-10 with key ``seed`` on the counters
    (row * ceil(D / 8) + d / 8, offset), 16 bits of its output for each of 8 channels; an element is dropped where its bits
    are below p 65536."""
    seed, offset = s["rng"][0], s["rng"][1]
    nc, mask = (D + 7) // 8, 0xFFFFFFFF
    n = torch.arange(M * nc, device="cuda")
    c0, c1 = n & mask, n >> 32
    c2, c3 = (offset & mask).expand_as(n), ((offset >> 32) & mask).expand_as(n)
    k0, k1 = seed & mask, (seed >> 32) & mask
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # the low 64 bits, whatever the sign
        c0, c1, c2, c3 = ((p1 >> 32) & mask) ^ c1 ^ k0, p1 & mask, ((p0 >> 32) & mask) ^ c3 ^ k1, p0 & mask
        k0, k1 = (k0 + 0x9E3779B9) & mask, (k1 + 0xBB67AE85) & mask
    words = torch.stack([c0, c1, c2, c3], 1)
    bits = torch.stack([words & 0xFFFF, words >> 16], 2).view(M, nc * 8)[:, :D]
    t = int(s["case"]["p"] * 65536 + 0.5)
    return bits >= t, 65536.0 / (65536 - t)


def _drop(s, v):
    if s["case"]["p"] == 0:
        return v
    keep, scale = _keep(s, *v.shape)
    return torch.where(keep, v * scale, torch.zeros_like(v))


def _act(s, like):
    """The gate's factor and its derivative."""
    if s["gate"] is None:
        return torch.ones_like(like), None
    g = s["gate"].float()
    if s["case"]["act"] == "linear":
        return g, torch.ones_like(g)
    sig = torch.sigmoid(g)
    if s["case"]["act"] == "sigmoid":
        return sig, sig * (1 - sig)
    return g * sig, sig * (1 + g * (1 - sig))


def _plain_norm(s):
    case, dt = s["case"], _dt(s["case"])
    x = s["x"].float()
    act, dact = _act(s, x)
    if case["op"] == "norm":
        rp = torch.rsqrt(x.square().mean(1) + EPS) if case["post"] else None
        n = x * rp[:, None] * s["w_post"] if case["post"] else x
        h = s["res"].float() + _drop(s, n * act * s["scale"])
        rq = torch.rsqrt(h.square().mean(1) + EPS)
        return (h * rq[:, None] * s["w_pre"]).to(dt), h.to(dt), rp, rq
    rp, rq = s["rstd_post"], s["rstd_pre"]
    dy = s["dy"].float()
    hh = s["h"].float() * rq[:, None]
    t = dy * s["w_pre"]
    dres = rq[:, None] * (t - hh * (t * hh).mean(1, keepdim=True)) + s["dh"].float()
    du = _drop(s, dres)
    xh = x * rp[:, None] if case["post"] else x
    n = xh * s["w_post"] if case["post"] else x
    dscale = (du * n * act).sum(0)
    dgate = (du * n * s["scale"] * dact).to(dt) if dact is not None else None
    dn = du * act * s["scale"]
    dx, dw_post = dn, None
    if case["post"]:
        t = dn * s["w_post"]
        dx = rp[:, None] * (t - xh * (t * xh).mean(1, keepdim=True))
        dw_post = (dn * xh).sum(0)
    return dx.to(dt), dres.to(dt), dgate, dw_post, (dy * hh).sum(0), dscale


def _plain(s):
    case = s["case"]
    op, dt = case["op"], _dt(case)
    if op == "dropout":
        v = _drop(s, s["x"].float())
        return (v if s["res"] is None else v + s["res"].float()).to(dt)
    if op.startswith("norm"):
        return _plain_norm(s)
    x = s["x"].float()
    rt, it = torch.sigmoid(s["r"].float() + s["r_bias"]), torch.sigmoid(s["i"].float() + s["i_bias"])
    la = -C * _softplus(s["lam"]) * rt
    a = torch.exp(la)
    m = torch.sqrt(-torch.expm1(2 * la))
    z = s["z"].float() if s.get("z") is not None else None
    sig = torch.sigmoid(z) if z is not None else None
    if op == "step":
        at = s["slots"].long()
        h = a * s["state"][at] + m * it * x
        s["state"][at] = h
        return (h if z is None else h * z * sig).to(dt), s["state"]
    Bn, L, D = x.shape
    live = None
    b = m * it * x
    if s.get("lengths") is not None:
        live = (torch.arange(L, device=x.device)[None, :] < s["lengths"][:, None])[:, :, None]
        a, b = torch.where(live, a, torch.ones_like(a)), torch.where(live, b, torch.zeros_like(b))
    if s.get("h_in") is not None:
        b[:, 0] += a[:, 0] * s["h_in"]
    h = _recur(a, b)
    y = h if z is None else h * z * sig
    if live is not None:
        y = torch.where(live, y, torch.zeros_like(y))
    out = (y.to(dt), h[:, -1].clone())
    if op == "scan":
        return out
    dy = s["dy"].float()
    if live is not None:
        dy = torch.where(live, dy, torch.zeros_like(dy))
    ds = (dy if z is None else dy * z * sig).flip(1)
    ds[:, 0] += s["dh_out"]
    g = _recur(torch.cat([torch.ones_like(a[:, :1]), a.flip(1)[:, :-1]], 1), ds).flip(1)
    dh_in = a[:, 0] * g[:, 0]
    if live is not None:
        g = torch.where(live, g, torch.zeros_like(g))
    before = torch.cat([s["h_in"][:, None], h[:, :-1]], 1)
    q = g * (la * a * before - a * a * (la / m) * it * x)  # la times the loss's derivative by la
    dr, di = q * (1 - rt), g * m * x * it * (1 - it)
    dz = None if z is None else (dy * h * sig * (1 + z * (1 - sig))).to(dt)
    dlam = q.sum((0, 1)) * torch.sigmoid(s["lam"]) / _softplus(s["lam"])
    return out + ((g * m * it).to(dt), dr.to(dt), di.to(dt), dlam, dr.sum((0, 1)), di.sum((0, 1)), dz, dh_in)


def work(case):
    """Bytes: each input read once, each output written once; a training pass is two calls, each with its own.
    Flops: an exponential, a root, a product or a sum is one."""
    op, D = case["op"], case["D"]
    e = 4 if case["dtype"] == "f32" else 2
    if op == "dropout":
        n = case["M"] * D
        return dict(bytes=n * e * (3 if case["residual"] else 2) + 16, flops=n * 10)
    if op.startswith("norm"):
        n, g, q = case["M"] * D, int(case["act"] != "none"), int(case["post"])
        drop = 8 if case["p"] > 0 else 0
        if op == "norm":
            return dict(bytes=n * e * (4 + g) + case["M"] * 4 * (1 + q) + D * 4 * (2 + q), flops=n * (10 + 6 * g + 4 * q + drop))
        return dict(bytes=n * e * (6 + 2 * g) + case["M"] * 4 * (1 + q) + 2 * D * 4 * (2 + q),
                    flops=n * (20 + 14 * g + 8 * q + drop))
    n, z, st = case["B"] * case.get("L", 1) * D, int(case["gate"]), case["B"] * D * 4
    if op == "step":
        return dict(bytes=(4 + z) * n * e + 2 * st + 12 * D, flops=n * 30)
    if op == "scan":
        return dict(bytes=(4 + z) * n * e + st * (2 if case["ragged"] else 1) + 12 * D, flops=n * 30)
    return dict(bytes=(4 + z + 7 + 2 * z) * n * e + 5 * st + 36 * D, flops=n * 110)


# ------------------------------------------------------------------------------- in 64 bits


def _philox_keep(seed, offset, M, D, t):
    """The kept elements, on the host in unsigned 64-bit arithmetic."""
    u = np.uint64
    low, word = u(0xFFFFFFFF), u(32)
    nc = (D + 7) // 8
    n = np.arange(M * nc, dtype=u)
    ctr = [n & low, n >> word, np.full_like(n, offset & 0xFFFFFFFF), np.full_like(n, offset >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = ctr[0] * u(0xD2511F53), ctr[2] * u(0xCD9E8D57)
        ctr = [(b >> word) ^ ctr[1] ^ u(key[0]), b & low, (a >> word) ^ ctr[3] ^ u(key[1]), a & low]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    bits = np.empty((M, nc, 8), dtype=np.uint16)
    for k in range(4):
        bits[:, :, 2 * k] = (ctr[k] & u(0xFFFF)).astype(np.uint16).reshape(M, nc)
        bits[:, :, 2 * k + 1] = (ctr[k] >> u(16)).astype(np.uint16).reshape(M, nc)
    return torch.from_numpy(bits.reshape(M, nc * 8)[:, :D] >= t).cuda()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {k: (v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v) for k, v in s.items()}
    x = d["x"]
    logistic = lambda t: 1 / (1 + torch.exp(-t))  # noqa: E731

    if "M" in case:
        factor = torch.ones_like(x)
        if case["p"] > 0:
            t = int(case["p"] * 65536 + 0.5)
            key, offset = s["rng"].tolist()
            factor = _philox_keep(key, offset, *x.shape, t).double() * (65536 / (65536 - t))
        if op == "dropout":
            return x * factor + (d["res"] if d["res"] is not None else 0)
        D = case["D"]
        act, slope = torch.ones_like(x), None
        if case["act"] == "linear":
            act, slope = d["gate"], torch.ones_like(x)
        elif case["act"] == "sigmoid":
            act = logistic(d["gate"])
            slope = act * logistic(-d["gate"])
        elif case["act"] == "silu":
            act = d["gate"] * logistic(d["gate"])
            slope = logistic(d["gate"]) + act * logistic(-d["gate"])
        w_post = d["w_post"] if case["post"] else torch.ones(D, dtype=x.dtype, device=x.device)
        if op == "norm":
            dev = ((x * x).sum(1) / D + EPS).sqrt()
            n = x * w_post / dev[:, None] if case["post"] else x
            h = d["res"] + factor * n * act * d["scale"]
            dq = ((h * h).sum(1) / D + EPS).sqrt()
            return h * d["w_pre"] / dq[:, None], h, (1 / dev if case["post"] else None), 1 / dq
        r = d["rstd_pre"][:, None]
        t = d["dy"] * d["w_pre"]
        dres = d["dh"] + r * t - r ** 3 * d["h"] * ((t * d["h"]).sum(1, keepdim=True) / D)
        du = dres * factor
        p = d["rstd_post"][:, None] if case["post"] else torch.ones_like(r)
        xh = x * p
        dgate = None if slope is None else du * xh * w_post * d["scale"] * slope
        dscale = (du * xh * w_post * act).sum(0)
        t = du * act * d["scale"] * w_post
        dx = p * (t - xh * ((t * xh).sum(1, keepdim=True) / D)) if case["post"] else t
        dw_post = (du * act * d["scale"] * xh).sum(0) if case["post"] else None
        return dx, dres, dgate, dw_post, (d["dy"] * d["h"] * r).sum(0), dscale

    soft = torch.log1p(torch.exp(d["lam"]))
    rt, it = logistic(d["r"] + d["r_bias"]), logistic(d["i"] + d["i_bias"])
    la = -C * soft * rt
    a = torch.exp(la)
    m = (-torch.expm1(2 * la)).sqrt()
    z = d.get("z")
    silu = None if z is None else z * logistic(z)
    if op == "step":
        at = s["slots"].long()
        h = a * d["state"][at] + m * it * x
        state = d["state"].clone()
        state[at] = h
        return (h if z is None else h * silu), state
    Bn, L, D = x.shape
    lens = s["lengths"] if s.get("lengths") is not None else torch.full((Bn,), L, device=x.device)
    live = torch.arange(L, device=x.device)[None] < lens[:, None]
    h = d["h_in"].clone() if d.get("h_in") is not None else torch.zeros(Bn, D, dtype=x.dtype, device=x.device)
    after, before = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(L):
        before[:, t] = h
        h = torch.where(live[:, t, None], a[:, t] * h + m[:, t] * it[:, t] * x[:, t], h)
        after[:, t] = h
    on = live[..., None].double()
    y = after * on if z is None else after * silu * on
    if op == "scan":
        return y, h
    dy = d["dy"] * on
    ds = dy if z is None else dy * silu
    dz = None if z is None else dy * after * (logistic(z) + silu * logistic(-z))
    g, gs = d["dh_out"].clone(), torch.zeros_like(x)
    for t in range(L - 1, -1, -1):
        gs[:, t] = (g + ds[:, t]) * on[:, t]
        g = torch.where(live[:, t, None], a[:, t] * gs[:, t], g)
    dla = gs * (a * before - it * x * a * a / m)
    dr = dla * la * (1 - rt)
    di = gs * m * x * it * (1 - it)
    dlam = (dla * rt).sum((0, 1)) * -C * logistic(d["lam"])
    return y, h, gs * m * it, dr, di, dlam, dr.sum((0, 1)), di.sum((0, 1)), dz, g
