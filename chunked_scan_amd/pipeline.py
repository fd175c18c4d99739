"""One device's share of ZeCO causal linear attention, composed from the four C-ABI calls.

Nothing here computes: each function only sequences library calls (and allocates their
buffers when the caller does not pass them).  The structure follows the linear-decomposition
identity of the review page "ZeCO: Zero Communication Overhead Sequence Parallelism for Linear
Attention" (pith_extraction.key_machinery): local work runs from a zero state, the incoming
state is folded into the state by the All-Scan update and into the outputs by a rank-dk
correction.

``device_step``   -- one device holding one segment, given the state S_recv it receives.  The
                     segment is cut into G sub-segments, each treated as one more device of the
                     same identity: the local forward of every sub-segment from a zero state (one
                     launch, no second pass over K and V), then one inclusive scan over
                     [S_recv, S_loc,1, ..., S_loc,G] that yields every sub-segment's exact incoming
                     state (its last entry is the All-Scan update S_out = Lambda S_recv + S_loc),
                     then one correction pass O += (Q * cumulative decay) S_in over every
                     sub-segment.  With G = 1 this is the plain form: local forward, two-entry scan,
                     correction by S_recv.  Without decay there is no decay to prepare (Lambda = 1,
                     cumulative decay = 1): the scan runs as a plain sum.  Head decay: Lambda from
                     the closed form, the cumulative decay formed inside the correction.  Gate
                     decay: the forward itself emits Q * cumulative decay and Lambda
                     (la_chunk_fwd_decayed), and the correction adds a plain product.
``ExactStep``     -- the same outputs and S_out from one la_chunk_fwd call that starts from S_recv: the
                     library splits the segment into sub-segments itself, scans their local states
                     with S_recv as the first entry and runs every sub-segment's outputs from its
                     exact incoming state (no correction pass); ``schedule`` picks the library's
                     separate passes or its chained single launch.
``RecvFirstStep`` -- the decomposed step with S_recv taken in at the start of the first sub-segment:
                     the segment is cut into G segments of one segmented forward, the first of
                     which starts from S_recv (it is then exact), the others from zero; the scan
                     over their G local states yields every incoming state, and the correction
                     covers sub-segments 1..G-1 only.  It saves the first sub-segment's correction
                     and one scan entry, at the price of a local forward that needs S_recv.
``segmented_forward`` -- P devices emulated on one GPU: the local forward of all P segments in
                     one launch, the P-entry state scan, and the correction of segments 1..P-1.

The selective state space layer, whose decay comes from an input-dependent step size, is sequenced likewise
around the caller's two projections (which are not part of the library):

``selective_prompt`` -- residual norm, projection to the mixer's input and gate, short convolution, projection
                     to step size, B and C, selective scan, for a (padded) batch of prompts or for the next
                     piece of one.
``selective_token``  -- the same for one token of each of several running sequences, whose convolution and scan
                     states live in pools.
``selective_backward`` -- the prompt's operators in reverse, the projections' own backward left to the caller.

The gated recurrent layer, whose state is one value per channel, likewise, from one pre-norm's output to the next one's:

``gated_prompt``   -- projection to the recurrence's input and output gate, short convolution, projection to the
                     recurrence's gates, gated recurrence, projection back, then the norm after the block, its gate, residual
                     scale, dropout, the residual sum and the norm before the next block.
``gated_token``    -- the same for one token of each of several running sequences, states in pools.
``gated_backward`` -- the prompt's operators in reverse.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Callable, Optional, Tuple

import torch

from .binding import (la_add_norm, la_add_norm_bwd, la_add_norm_q8, la_block_norm, la_block_norm_bwd, la_chunk_fwd,
                      la_chunk_fwd_decayed, la_cumdecay, la_gated_scan, la_gated_scan_bwd, la_gated_step, la_short_conv,
                      la_short_conv_bwd, la_short_conv_step, la_ssm_scan, la_ssm_scan_bwd, la_ssm_step, la_state_correct,
                      la_state_scan)


def _tile_flags(B, H, L, nseg, dev):
    """Per-64-token-tile liveness flags of q * cumulative decay, one int32 per tile of each segment."""
    return torch.empty((B, H, nseg, (L // nseg + 63) // 64), dtype=torch.int32, device=dev)


def _forward(step, s_in, s_out, totals, nseg, timers):
    """The local forward and the decay quantities the scan and the correction need."""
    B, H, L, dk, dv = step.shape
    kw = dict(mode=step.mode, nseg=nseg, chunk=step.chunk, gate_norm=step.gate_norm,
              subseg_chunks=step.subseg_chunks)
    if step.mode == "gate":
        la_chunk_fwd_decayed(step.q, step.k, step.v, step.decay, s_in, step.o, s_out, step.qd, totals,
                             step.live, timer=timers.get("fwd"), **kw)
        return
    la_chunk_fwd(step.q, step.k, step.v, step.decay, s_in, step.o, s_out, timer=timers.get("fwd"), **kw)
    if step.mode == "head":
        la_cumdecay(step.decay, B, H, L, dk, mode="head", nseg=nseg, total=totals, want_cum=False,
                    timer=timers.get("cum"))


def _correct(step, s_recv, nseg, seg_begin, timers):
    """O += (Q * cumulative decay) S_recv; in gate mode Q * cum is the forward's q_decayed, and the
    tiles where it is exactly zero (the cumulative decay has underflowed) are skipped."""
    if step.mode == "gate":
        la_state_correct(step.qd, None, s_recv, step.o, mode="none", nseg=nseg, seg_begin=seg_begin,
                         tile_live=step.live, timer=timers.get("corr"))
    else:
        la_state_correct(step.q, step.decay if step.mode == "head" else None, s_recv, step.o, mode=step.mode,
                         nseg=nseg, seg_begin=seg_begin, timer=timers.get("corr"))


def subsegments(B: int, H: int, L: int, target_units: int = 0, min_len: int = 256, dk: int = 128) -> int:
    """Sub-segments per sequence for a device step: about ``target_units`` (b,h,sub-segment) units
    in all, each at least ``min_len`` tokens; G must divide L, and lengths that are whole 64-token
    chunks are preferred.  By default 256 units (one workgroup per compute unit) at dk = 128 and
    512 below: the small-head kernels are latency-bound and several of their workgroups share a
    compute unit (B1 H16 L16k, G = 16 -> 32: dk = 64 step 61.9 -> 54.4 us, dk = 32 41.1 -> 40.4 us;
    G = 64 gains no more at dk = 32, where its 65-entry scan leaves the scan's vector form)."""
    if target_units <= 0:
        target_units = 256 if dk >= 128 else 512
    want = max(1, -(-target_units // max(1, B * H)))
    cands = [g for g in range(1, want + 1) if L % g == 0 and (g == 1 or L // g >= min_len)]
    whole = [g for g in cands if (L // g) % 64 == 0]
    return max(whole or cands)


class DeviceStep:
    """Buffers and call sequence of one device step; ``run()`` may be timed or graph-captured.
    ``subseg`` fixes the number G of sub-segments (0 = ``subsegments()``)."""

    def __init__(self, q, k, v, decay, s_recv, *, mode: str, chunk: int = 64, gate_norm: float = 16.0,
                 subseg_chunks: int = 0, subseg: int = 0):
        B, H, L, dk = q.shape
        dv = v.shape[-1]
        dev = q.device
        G = subseg or subsegments(B, H, L, dk=dk)
        if L % G:
            raise ValueError(f"{G} sub-segments do not divide L = {L}")
        self.q, self.k, self.v, self.decay = q, k, v, decay
        self.mode, self.chunk, self.gate_norm, self.subseg_chunks = mode, chunk, gate_norm, subseg_chunks
        self.G = G
        self.shape = (B, H, L, dk, dv)
        self.o = torch.empty((B, H, L, dv), dtype=q.dtype, device=dev)
        # scan buffer: slot 0 = incoming state (what the previous device sends), slots 1..G = local
        # states of the sub-segments; after the scan slot p is the incoming state of sub-segment p
        # and slot G the outgoing state
        self.states = torch.zeros((B, H, G + 1, dk, dv), dtype=torch.float32, device=dev)
        if s_recv is not None:
            self.states[:, :, 0].copy_(s_recv)
        self.totals = torch.ones((B, H, G + 1, dk), dtype=torch.float32, device=dev)
        self.qd = torch.empty_like(q) if mode == "gate" else None  # q times its cumulative decay
        self.live = _tile_flags(B, H, L, G, dev) if mode == "gate" else None

    def run(self, timers: Optional[dict] = None):
        """One step.  ``timers`` optionally maps "fwd", "cum", "scan", "corr" to KernelTimers."""
        t = timers or {}
        G = self.G
        _forward(self, None, self.states[:, :, 1:], self.totals[:, :, 1:], G, t)
        la_state_scan(self.states, self.totals if self.mode != "none" else None, self.states, timer=t.get("scan"))
        _correct(self, self.states[:, :, 0:G], G, 0, t)
        return self.o, self.states[:, :, G]


class ExactStep:
    """One device step as a single exact forward from S_recv (la_chunk_fwd with s_in = S_recv);
    ``run()`` may be timed or graph-captured.  Returns (o, s_out [B,H,dk,dv])."""

    def __init__(self, q, k, v, decay, s_recv, *, mode: str, chunk: int = 64, gate_norm: float = 16.0,
                 subseg_chunks: int = 0, schedule: str = "auto"):
        B, H, L, dk = q.shape
        dv = v.shape[-1]
        self.q, self.k, self.v, self.decay, self.s_recv = q, k, v, decay, s_recv
        self.mode, self.chunk, self.gate_norm = mode, chunk, gate_norm
        self.subseg_chunks, self.schedule = subseg_chunks, schedule
        self.shape = (B, H, L, dk, dv)
        self.o = torch.empty((B, H, L, dv), dtype=q.dtype, device=q.device)
        self.s_out = torch.empty((B, H, 1, dk, dv), dtype=torch.float32, device=q.device)

    def run(self, timers: Optional[dict] = None):
        """One step.  ``timers`` optionally maps "fwd" to a KernelTimer."""
        t = timers or {}
        la_chunk_fwd(self.q, self.k, self.v, self.decay, self.s_recv, self.o, self.s_out, mode=self.mode,
                     chunk=self.chunk, gate_norm=self.gate_norm, subseg_chunks=self.subseg_chunks,
                     schedule=self.schedule, timer=t.get("fwd"))
        return self.o, self.s_out[:, :, 0]


class RecvFirstStep:
    """One device step as a segmented forward over G sub-segments whose first starts from S_recv;
    ``run()`` may be timed or graph-captured.  Returns (o, s_out [B,H,dk,dv])."""

    def __init__(self, q, k, v, decay, s_recv, *, mode: str, chunk: int = 64, gate_norm: float = 16.0,
                 subseg_chunks: int = 0, subseg: int = 0):
        B, H, L, dk = q.shape
        G = subseg or subsegments(B, H, L, dk=dk)
        if L % G:
            raise ValueError(f"{G} sub-segments do not divide L = {L}")
        self.G = self.nseg = G
        self.seg = SegmentedForward(q, k, v, decay, s_recv, mode=mode, nseg=G, chunk=chunk, gate_norm=gate_norm,
                                    subseg_chunks=subseg_chunks)
        self.live = self.seg.live  # gate mode: the forward's tile flags of q * cumulative decay

    def run(self, timers: Optional[dict] = None):
        """One step.  ``timers`` optionally maps "fwd", "cum", "scan", "corr" to KernelTimers."""
        o, states = self.seg.run(timers)
        return o, states[:, :, -1]


def device_step(q, k, v, decay, s_recv, *, mode: str, chunk: int = 64, gate_norm: float = 16.0,
                subseg_chunks: int = 0, subseg: int = 0):
    """Returns (o, s_out) of one device that receives s_recv (None = zero)."""
    return DeviceStep(q, k, v, decay, s_recv, mode=mode, chunk=chunk, gate_norm=gate_norm,
                      subseg_chunks=subseg_chunks, subseg=subseg).run()


class SegmentedForward:
    """P segments (P emulated devices) of each (b,h) sequence on one GPU; ``run()`` is one pass."""

    def __init__(self, q, k, v, decay, s_in, *, mode: str, nseg: int, chunk: int = 64, gate_norm: float = 16.0,
                 subseg_chunks: int = 0):
        B, H, L, dk = q.shape
        dv = v.shape[-1]
        dev = q.device
        self.q, self.k, self.v, self.decay, self.s_in = q, k, v, decay, s_in
        self.mode, self.nseg, self.chunk, self.gate_norm = mode, nseg, chunk, gate_norm
        self.subseg_chunks = subseg_chunks
        self.shape = (B, H, L, dk, dv)
        self.o = torch.empty((B, H, L, dv), dtype=q.dtype, device=dev)
        self.states = torch.empty((B, H, nseg, dk, dv), dtype=torch.float32, device=dev)
        self.totals = torch.empty((B, H, nseg, dk), dtype=torch.float32, device=dev)
        self.qd = torch.empty_like(q) if mode == "gate" else None  # q times its cumulative decay
        self.live = _tile_flags(B, H, L, nseg, dev) if mode == "gate" else None

    def run(self, timers: Optional[dict] = None):
        """One pass.  ``timers`` optionally maps "fwd", "cum", "scan", "corr" to KernelTimers."""
        P = self.nseg
        t = timers or {}
        _forward(self, self.s_in, self.states, self.totals, P, t)
        la_state_scan(self.states, self.totals if self.mode != "none" else None, self.states, timer=t.get("scan"))
        if P > 1:
            _correct(self, self.states[:, :, : P - 1], P, 1, t)
        return self.o, self.states


def segmented_forward(q, k, v, decay, s_in, *, mode: str, nseg: int, chunk: int = 64, gate_norm: float = 16.0,
                      subseg_chunks: int = 0):
    """Returns (o, out_states [B,H,P,dk,dv]); out_states[:, :, -1] is the final state."""
    return SegmentedForward(q, k, v, decay, s_in, mode=mode, nseg=nseg, chunk=chunk, gate_norm=gate_norm,
                            subseg_chunks=subseg_chunks).run()


@dataclass
class SelectiveParams:
    """A selective layer's own parameters, all float32: norm_weight [Dm]; conv_weight [D, W], conv_bias [D] or
    None; A [D, N]; skip [D] or None; dt_bias [D] or None.  q8_group: None (the norm's output in the
    activations' type) or the elements per scale of an 8-bit output (la_add_norm_q8's group)."""
    norm_weight: torch.Tensor
    conv_weight: torch.Tensor
    conv_bias: Optional[torch.Tensor]
    A: torch.Tensor
    skip: Optional[torch.Tensor] = None
    dt_bias: Optional[torch.Tensor] = None
    eps: float = 1e-5
    q8_group: Optional[int] = None


def _norm_in(p: SelectiveParams, x, residual, pad=None):
    """(what the input projection takes, h, rstd): the normed rows, or (q, scale) in 8 bits; those of ``pad``, a mask
    [rows, 1], are zero."""
    if p.q8_group is None:
        y, h, rstd = la_add_norm(x, p.norm_weight, residual, eps=p.eps)
        return (y if pad is None else y.masked_fill_(pad, 0)), h, rstd
    q, scale, h, rstd = la_add_norm_q8(x, p.norm_weight, residual, eps=p.eps, group=p.q8_group)
    if pad is not None:
        q.view(torch.uint8).masked_fill_(pad, 0)
        scale.masked_fill_(pad, 1)
    return (q, scale), h, rstd


def _padding(lengths, B, L, device):
    """Which of B L rows lie behind their sequence's length: [B L, 1], or None."""
    if lengths is None:
        return None
    return (torch.arange(L, device=device)[None] >= lengths[:, None]).view(B * L, 1)


def selective_prompt(p: SelectiveParams, x: torch.Tensor, residual: Optional[torch.Tensor],
                     project_in: Callable, project_dbc: Callable, *, conv_state: Optional[torch.Tensor] = None,
                     s_in: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                     saved: Optional[dict] = None) -> Tuple[torch.Tensor, ...]:
    """One layer over x [B, L, Dm] (residual the same or None).  project_in maps the normed rows [B L, Dm] (or
    (q, scale)) to (u, z): two [B L, D] tensors, the gate z possibly None, usually the halves of one
    product.  project_dbc maps the convolved [B, L, D] to (dt, B, C): [B, L, D], [B, L, N], [B, L, N].
    Rows of x and residual behind a sequence's length may hold anything: what project_in takes is zero there.
    conv_state [B, W-1, D] and s_in [B, N, D]: states of the tokens before, or None.  Returns (y [B, L, D],
    zero behind a sequence's length, h [B, L, Dm] the residual stream, conv_state, s_out).  `saved`, a dict, receives what
    selective_backward takes."""
    B, L, Dm = x.shape
    rows = lambda t: None if t is None else t.reshape(B * L, Dm)  # noqa: E731
    y, h, rstd = _norm_in(p, rows(x), rows(residual), _padding(lengths, B, L, x.device))
    u, z = (None if t is None else t.unflatten(0, (B, L)) for t in project_in(y))
    # rows behind a sequence's length are not written: they are zero here (as the normed ones are), so that a product
    # over all rows (the projections' weight derivatives) stays finite whatever the padding holds
    blank = lambda: None if lengths is None else torch.zeros(u.shape, dtype=u.dtype, device=u.device)  # noqa: E731
    v, conv_out = la_short_conv(u, p.conv_weight, p.conv_bias, conv_state, lengths=lengths, y=blank(), want_state=True)
    dt, Bm, C = project_dbc(v)
    o, s_out = la_ssm_scan(v, dt, p.A, Bm, C, D=p.skip, z=z, dt_bias=p.dt_bias, s_in=s_in, lengths=lengths, y=blank())
    if saved is not None:
        saved.update(h=h, rstd=rstd, u=u, z=z, v=v, dt=dt, B=Bm, C=C, conv_state=conv_state, s_in=s_in, lengths=lengths)
    return o, h.view(B, L, Dm), conv_out, s_out


def selective_backward(p: SelectiveParams, saved: dict, dy: torch.Tensor, dbc_backward: Callable,
                       in_backward: Callable, *, dh: Optional[torch.Tensor] = None,
                       d_conv_state: Optional[torch.Tensor] = None, ds_out: Optional[torch.Tensor] = None) -> dict:
    """Backward of selective_prompt from dy [B, L, D], dh [B, L, Dm] (the residual stream's derivative) and those of
    the returned states.  dbc_backward maps (ddt, dB, dC) to the convolved tensor's part of the derivative
    [B, L, D]; in_backward maps (du, dz), zero behind a sequence's length, to the normed rows' [B L, Dm].  Returns
    dx (of x and residual alike; behind a length dh) and the parameters' and incoming states' derivatives by name."""
    s = saved
    B, L, _ = s["u"].shape
    dv, ddt, dA, dB, dC, dskip, dz, d_dt_bias, ds_in = la_ssm_scan_bwd(
        s["v"], s["dt"], p.A, s["B"], s["C"], dy, D=p.skip, z=s["z"], dt_bias=p.dt_bias, s_in=s["s_in"], ds_out=ds_out,
        lengths=s["lengths"])
    dv += dbc_backward(ddt, dB, dC)
    du, dcw, dcb, d_conv = la_short_conv_bwd(s["u"], p.conv_weight, dv, p.conv_bias, s["conv_state"], d_conv_state,
                                             lengths=s["lengths"])
    dn = in_backward(du, dz)
    h, rstd, pad = s["h"], s["rstd"], _padding(s["lengths"], B, L, dy.device)
    if pad is not None:  # the normed padding rows were zero: dn is zero there and what they hold may not meet it
        h, rstd = h.masked_fill(pad, 0), rstd.masked_fill(pad[:, 0], 1)
    dx, dnw = la_add_norm_bwd(dn, h, p.norm_weight, rstd, None if dh is None else dh.reshape(dn.shape))
    return dict(dx=dx.view(B, L, dn.shape[1]), norm_weight=dnw, conv_weight=dcw, conv_bias=dcb, A=dA, skip=dskip,
                dt_bias=d_dt_bias, conv_state=d_conv, s_in=ds_in)


def selective_token(p: SelectiveParams, x: torch.Tensor, residual: Optional[torch.Tensor], project_in: Callable,
                    project_dbc: Callable, conv_pool: torch.Tensor, state_pool: torch.Tensor,
                    slots: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """One layer over one token of each of B sequences, x [B, Dm]; conv_pool [S, W-1, D] and state_pool
    [S, N, D] are updated in place at the rows' slots.  Returns (y [B, D], h [B, Dm]).  Rows that are padding (a
    slot outside the pools, or one that an earlier row names) have undefined y."""
    y, h, _ = _norm_in(p, x, residual)
    u, z = project_in(y)
    v = la_short_conv_step(u, p.conv_weight, conv_pool, p.conv_bias, slots=slots)
    dt, Bm, C = project_dbc(v)
    return la_ssm_step(v, dt, p.A, Bm, C, state_pool, D=p.skip, z=z, dt_bias=p.dt_bias, slots=slots), h


@dataclass
class GatedParams:
    """A gated recurrent layer's own parameters, all float32: conv_weight [D, W], conv_bias [D] or None; lam [D], r_bias
    and i_bias [D] or None, c the log-decay's scale; w_post and scale [Dm] or None (the norm after the block and the
    residual scale), w_pre [Dm] or None (the norm before the next block); act the output gate's activation, dropout the
    share of the branch that is dropped."""
    conv_weight: torch.Tensor
    conv_bias: Optional[torch.Tensor]
    lam: torch.Tensor
    r_bias: Optional[torch.Tensor] = None
    i_bias: Optional[torch.Tensor] = None
    c: float = 8.0
    w_post: Optional[torch.Tensor] = None
    scale: Optional[torch.Tensor] = None
    w_pre: Optional[torch.Tensor] = None
    act: str = "silu"
    dropout: float = 0.0
    eps: float = 1e-5

    def scan(self):
        return dict(r_bias=self.r_bias, i_bias=self.i_bias, c=self.c)

    def norms(self):
        return dict(w_post=self.w_post, w_pre=self.w_pre, scale=self.scale, act=self.act)


def _blank_rows(t: Optional[torch.Tensor], pad):
    """``t`` [rows, n] with the rows of ``pad``, a mask [rows, 1], zero; ``t`` itself without a mask."""
    return t if t is None or pad is None else t.masked_fill(pad, 0)


def gated_prompt(p: GatedParams, n: torch.Tensor, residual: Optional[torch.Tensor], project_in: Callable,
                 project_gates: Callable, project_out: Callable, *, conv_state: Optional[torch.Tensor] = None,
                 h_in: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                 rng: Optional[torch.Tensor] = None, saved: Optional[dict] = None) -> Tuple[torch.Tensor, ...]:
    """One layer over n [B, L, Dm], the normed rows (a layer's y or the first norm's), and the residual stream (the same
    shape, or None).  project_in maps n's rows [B L, Dm] to (u, z): two [B L, D] tensors, z possibly None; project_gates
    the convolved [B, L, D] to (r, i): two [B, L, D]; project_out the recurrence's rows [B L, D] to (x, gate): two
    [B L, Dm], gate possibly None.  Rows of n and residual behind a sequence's length may hold anything and count as
    zero.  conv_state [B, W-1, D] and h_in [B, D]: states of the tokens before, or None; rng: dropout's seed and
    offset, which may be changed in place after the call (`saved` holds a copy).  Returns (y [B, L, Dm] the next layer's n
    or None without w_pre, h [B, L, Dm] the residual stream, conv_state, h_out).  `saved`, a dict, receives what
    gated_backward takes."""
    B, L, Dm = n.shape
    pad = _padding(lengths, B, L, n.device)
    rows = lambda t: None if t is None else t.reshape(B * L, Dm)  # noqa: E731
    u, z = (None if t is None else t.unflatten(0, (B, L)) for t in project_in(_blank_rows(rows(n), pad)))
    # rows behind a sequence's length are not written: they are zero here, so that a product over all rows stays finite
    blank = lambda: None if lengths is None else torch.zeros(u.shape, dtype=u.dtype, device=u.device)  # noqa: E731
    v, conv_out = la_short_conv(u, p.conv_weight, p.conv_bias, conv_state, lengths=lengths, silu=False, y=blank(),
                                want_state=True)
    r, i = project_gates(v)
    o, h_out, blocks = la_gated_scan(v, r, i, p.lam, z=z, h_in=h_in, lengths=lengths, y=blank(),
                                     want_blocks=saved is not None, **p.scan())
    x, gate = project_out(o.view(B * L, u.shape[2]))
    y, h, rstd_post, rstd_pre = la_block_norm(x, _blank_rows(rows(residual), pad), gate=gate, p=p.dropout, rng=rng,
                                              eps=p.eps, **p.norms())
    if saved is not None:
        if rng is not None:
            rng = rng.clone()  # what it holds now: the caller may move on to the next layer's offset in place
        saved.update(u=u, z=z, v=v, r=r, i=i, conv_state=conv_state, h_in=h_in, lengths=lengths, blocks=blocks, x=x,
                     gate=gate, h=h, rstd_post=rstd_post, rstd_pre=rstd_pre, rng=rng)
    return None if y is None else y.view(B, L, Dm), h.view(B, L, Dm), conv_out, h_out


def gated_backward(p: GatedParams, saved: dict, dy: Optional[torch.Tensor], dh: Optional[torch.Tensor],
                   out_backward: Callable, gates_backward: Callable, in_backward: Callable, *,
                   d_conv_state: Optional[torch.Tensor] = None, dh_out: Optional[torch.Tensor] = None) -> dict:
    """Backward of gated_prompt from dy [B, L, Dm] (None without w_pre), dh [B, L, Dm] (the residual stream's derivative,
    or None) and those of the returned states; rows behind a sequence's length count as zero.  out_backward maps
    (dx, dgate) [B L, Dm] to the recurrence's rows' derivative [B L, D]; gates_backward (dr, di) to the convolved tensor's
    part [B, L, D]; in_backward (du, dz), zero behind a sequence's length, to n's rows' [B L, Dm].  Returns dn and
    dresidual and the parameters' and incoming states' derivatives by name."""
    s = saved
    B, L, D = s["u"].shape
    Dm = s["x"].shape[1]
    pad = _padding(s["lengths"], B, L, s["x"].device)
    rows = lambda t: _blank_rows(None if t is None else t.reshape(B * L, Dm), pad)  # noqa: E731
    dx, dres, dgate, dw_post, dw_pre, dscale = la_block_norm_bwd(
        s["x"], s["h"] if p.w_pre is not None else None, rows(dy), rows(dh), gate=s["gate"], p=p.dropout, rng=s["rng"],
        rstd_post=s["rstd_post"], rstd_pre=s["rstd_pre"], **p.norms())
    do = out_backward(dx, dgate).view(B, L, D)
    dv, dr, di, dlam, dr_bias, di_bias, dz, dh_in = la_gated_scan_bwd(
        s["v"], s["r"], s["i"], p.lam, do, z=s["z"], h_in=s["h_in"], lengths=s["lengths"], h_blocks=s["blocks"],
        dh_out=dh_out, **p.scan())
    dv += gates_backward(dr, di)
    du, dcw, dcb, d_conv = la_short_conv_bwd(s["u"], p.conv_weight, dv, p.conv_bias, s["conv_state"], d_conv_state,
                                             lengths=s["lengths"], silu=False)
    dn = in_backward(du, dz)
    return dict(dn=dn.view(B, L, Dm), dresidual=dres.view(B, L, Dm), conv_weight=dcw, conv_bias=dcb, lam=dlam,
                r_bias=dr_bias, i_bias=di_bias, w_post=dw_post, w_pre=dw_pre, scale=dscale, conv_state=d_conv, h_in=dh_in)


def gated_token(p: GatedParams, n: torch.Tensor, residual: Optional[torch.Tensor], project_in: Callable,
                project_gates: Callable, project_out: Callable, conv_pool: torch.Tensor, state_pool: torch.Tensor,
                slots: Optional[torch.Tensor] = None) -> Tuple[Optional[torch.Tensor], torch.Tensor]:
    """One layer over one token of each of B sequences, n [B, Dm], without dropout; conv_pool [S, W-1, D] and state_pool
    [S, D] are updated in place at the rows' slots.  Returns (y [B, Dm] or None, h [B, Dm]).  Rows that are padding (a
    slot outside the pools, or one that an earlier row names) have undefined y and h."""
    u, z = project_in(n)
    v = la_short_conv_step(u, p.conv_weight, conv_pool, p.conv_bias, slots=slots, silu=False)
    r, i = project_gates(v)
    x, gate = project_out(la_gated_step(v, r, i, p.lam, state_pool, z=z, slots=slots, **p.scan()))
    return la_block_norm(x, residual, gate=gate, eps=p.eps, **p.norms())[:2]
