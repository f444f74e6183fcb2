"""Sliding-window attention where some rows of a warp find a much larger score in a later key tile than in the first and
others do not: the accumulator is rescaled for the former only.  Tolerances: the output's half step (2^-8 in
bf16) and the weights' (2^-8; 2^-11 for scores up to 2^8, whose fp32 sums carry 2^-20) against sum p |v|."""

import math

import pytest
import torch

from hybrid_ssm_sliding_b200 import _lib as L
from hybrid_ssm_sliding_b200 import build as B
from hybrid_ssm_sliding_b200 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


def swa64(q, k, v, W):
    q, k, v = (t[0].double().transpose(0, 1) for t in (q, k, v))
    n, grp = q.shape[1], q.shape[0] // k.shape[0]
    k, v = (t.repeat_interleave(grp, 0) for t in (k, v))
    i = torch.arange(n, device=q.device)
    see = (i[None] <= i[:, None]) & (i[None] > i[:, None] - W)
    p = torch.softmax((q @ k.transpose(1, 2) * q.shape[-1] ** -0.5).masked_fill(~see, -math.inf), -1)
    return (p @ v).transpose(0, 1)[None], (p @ v.abs()).transpose(0, 1)[None]


@pytest.mark.parametrize("by", [1.0, 4.0, 12.0])
@pytest.mark.parametrize("d", [64, 16, 32])
@pytest.mark.parametrize("group", [2, 1, 4, 8, 16])
def test_rows_of_a_warp_rescale_apart(group, d, by):
    n, W = 700, 400
    g = torch.Generator(device="cuda").manual_seed(400 + group + d)
    q, k, v = (torch.randn((1, n, h, d), generator=g, device="cuda") for h in (2 * group, 2, 2))
    q, k, v = (q * by).to(torch.bfloat16), k.to(torch.bfloat16), v.to(torch.bfloat16)
    o = ops.swa_fwd(q, k, v, W).double()
    assert ops.get_status() == L.SAMBA_OK
    want, mag = swa64(q, k, v, W)
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -11) * mag
    assert float(((o - want).abs() - tol).max()) <= 0


def test_one_row_of_a_warp():
    """A row alone, found by going through its inputs on the host."""
    g = torch.Generator().manual_seed(306)
    q, k, v = (torch.randn((1, 300, h, 64), generator=g).to(torch.bfloat16).cuda() for h in (4, 2, 2))
    q[..., 3] = 1.0
    o = ops.swa_fwd(q, k, v, 90).double()
    assert ops.get_status() == L.SAMBA_OK
    want, mag = swa64(q, k, v, 90)
    assert float(((o - want).abs() - 2.0 ** -8 * want.abs() - (2.0 ** -8 + 2.0 ** -13) * mag).max()) <= 0
