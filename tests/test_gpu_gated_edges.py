"""The gated recurrent layer's operators and the residual norm where their numbers are extreme, against the fp64 forms of
gated_ref.py."""
import numpy as np
import pytest
import torch

import gated_ref as G
import mixer_ref as R
from chunked_scan_amd import binding as la
from gpu_util import note
from test_gpu_gated import block_inputs, check_block
from test_gpu_mixer import BF, F32, Draw

pytestmark = pytest.mark.gpu

# ------------------------------------------------------------------------------------ rows near the largest value


def huge_rows(M, D, dtype, seed):
    """Rows of 1e37, 1e38 and 3e38 times a factor in 0.5..1, signs in turn."""
    t = Draw(seed).uniform(M, D, lo=0.5, hi=1.0) * torch.tensor([1e37, 1e38, 3e38], device="cuda").repeat(M)[:M, None]
    return (t * (1 - 2 * (torch.arange(D, device="cuda") % 2))).to(dtype)


def check_rstd(got, ref, D):
    """D / 8 + 32 roundings (a lane's share of a row's sum, the lanes'), and half a step of fp32's subnormal numbers."""
    assert (np.abs(R.f64(got) - ref) <= (D / 8 + 32) * R.U * ref + 2.0 ** -150).all()


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 1001, 2048, 16384])
def test_norms_of_rows_near_the_largest_value(D, dtype):
    note(f"norms of rows near the largest value {D} {dtype}")
    M, eps = 6, 1e-5
    for big in ("x", "res"):
        a = block_inputs(M, D, dtype, 21)
        a[big] = huge_rows(M, D, dtype, 22)
        if big == "x":  # the post-norm brings small rows down further still
            a["w_post"][: D // 2] *= 1e-6
            a["res"] = None
        (y, h, rp, rq), _, _ = check_block(a, "silu", 0.0, dtype, M, D)
        _, (hr, _), rpr, rqr = G.block(*[R.f64(a[k]) for k in ("x", "gate", "res", "w_post", "scale", "w_pre")], "silu", eps)
        check_rstd(rp, rpr[0], D)
        if big == "res":  # u is below half a step of the stream
            check_rstd(rq, rqr[0], D)
            assert np.abs(R.f64(y)).max() > 0.5
    x, w = huge_rows(M, D, dtype, 23), 1 + Draw(24).normal(D, std=0.2)
    w[: D // 2] *= 1e-6
    x64, w64 = R.f64(x), R.f64(w)
    r = 1 / np.sqrt((x64 ** 2).mean(1, keepdims=True) + eps)
    y, _, rstd = la.la_add_norm(x, w)
    G.close(y, x64 * r * w64, np.abs(x64 * r * w64) * (D / 8 + 36), dtype, "y")
    check_rstd(rstd, r[:, 0], D)
    q, scale, _, rstd = la.la_add_norm_q8(x, w)
    # e4m3: half a step of 2^-4 of the value in its normal range, of 2^-9 of the scale below it
    want, s = x64 * r * w64, R.f64(scale)
    tol = np.abs(want) * (2.0 ** -4 + (D / 8 + 40) * R.U) + s * 2.0 ** -10 * 1.01
    assert (np.abs(R.f64(q.float()) * s - want) <= tol).all()
    check_rstd(rstd, r[:, 0], D)
