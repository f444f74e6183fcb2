"""The block norm's gate far from zero, where a sigmoid is next to 0 or 1; the
other tolerances as in test_block_norm.py."""

import pytest
import torch

from hybrid_ssm_sliding_b200 import _lib as L
from hybrid_ssm_sliding_b200 import build as B
from hybrid_ssm_sliding_b200 import ops
from tests.test_block_norm import BF16, EPS, F32, HALF, bwd64, gpu, make


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


@pytest.mark.gpu
@pytest.mark.parametrize("yt", [F32, BF16])
def test_gate_gradients_far_out(lib, yt):
    """dgate = dt t (1 - s) where the sigmoid s has come to 1 (or 0): its error
    is a part of itself.  The exponential of |x| is off by |x| 2^-23 of itself (the
    product with log2 e and the instruction), the quotient and the products by a
    few 2^-23: below (|x| + 16) 2^-23 of dgate, and dr's own error in dt."""
    rows, C = 40, 512
    p = gpu(make(rows, C, F32, yt, True, True, True, seed=11))
    far = torch.linspace(-40, 40, C).repeat(rows, 1)
    p["gate"] = far.to(yt).cuda()
    dr = torch.randn((rows, C), generator=torch.Generator().manual_seed(12)).cuda()
    rsy = torch.rsqrt(p["y"].float().square().mean(1) + EPS)
    out = ops.block_norm_bwd(None, p["r"], None, None, dr_out=dr, y=p["y"], w_post=p["w_post"], rstd_post=rsy,
                             gate=p["gate"], alpha=p["alpha"])
    x = p["gate"].double()
    t = p["y"].double() * rsy.double()[:, None] * p["w_post"].double()
    want = p["alpha"].double() * dr.double() * t * torch.special.expit(x) * torch.special.expit(-x)
    tol = ((x.abs() + 16) * 2.0 ** -23 + HALF[yt]) * want.abs() + 2.0 ** -140
    assert float(((out["dgate"].double() - want).abs() / tol).max()) <= 1
    # and the other gradients with such gates
    w2, mag = bwd64(None, p["r"], None, None, dr, p["y"], p["w_post"], rsy, p["gate"], p["alpha"])
    for k in ("dy", "dalpha", "dw_post"):
        col = w2[k].dim() == 1
        bound = (2.0 ** -16 if col else 2.0 ** -17) * mag[k] + (0 if col else HALF[yt]) * w2[k].abs()
        assert float(((out[k].double() - w2[k]).abs() - bound).max()) <= 0, k


@pytest.mark.gpu
def test_gates_past_the_exponential(lib):
    """Gates beyond what exp holds: the sigmoid is 0 or 1 and dgate 0; NaN stays NaN."""
    p = gpu(make(4, 64, F32, F32, False, True, False, seed=13))
    p["gate"][0], p["gate"][1], p["gate"][2, ::2], p["gate"][2, 1::2] = 1e30, -1e30, float("inf"), float("-inf")
    p["gate"][3] = float("nan")
    dr = torch.ones_like(p["r"])
    out = ops.block_norm_bwd(None, p["r"], None, None, dr_out=dr, y=p["y"], gate=p["gate"])
    assert float(out["dgate"][:3].abs().max()) == 0
    assert torch.equal(out["dy"][0], dr[0]) and float(out["dy"][1].abs().max()) == 0
    assert torch.equal(out["dy"][2, ::2], dr[2, ::2]) and float(out["dy"][2, 1::2].abs().max()) == 0
    assert torch.isnan(out["dy"][3]).all() and torch.isnan(out["dgate"][3]).all()
