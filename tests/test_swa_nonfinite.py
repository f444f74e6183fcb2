"""Sliding-window attention where scores are not finite: a row that sees a key or query of NaN or infinity is NaN, as
its softmax is; every other row stays what it was.  Tolerances: the output's half
step (2^-8 in bf16) and the weights' (2^-8, and 2^-13 for scores and exponentials) against sum p |v|."""

import math

import pytest
import torch

from hybrid_ssm_sliding_b200 import _lib as L
from hybrid_ssm_sliding_b200 import build as B
from hybrid_ssm_sliding_b200 import ops

pytestmark = pytest.mark.gpu

LEN, HQ, HKV, W = 300, 4, 2, 90


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


def inputs(d, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn((1, LEN, h, d), generator=g).to(torch.bfloat16) for h in (HQ, HKV, HKV)]


def swa64(q, k, v):
    q, k, v = (t[0].double().transpose(0, 1) for t in (q, k, v))
    k, v = (t.repeat_interleave(HQ // HKV, 0) for t in (k, v))
    i = torch.arange(LEN)
    see = (i[None] <= i[:, None]) & (i[None] > i[:, None] - W)
    p = torch.softmax((q @ k.transpose(1, 2) * q.shape[-1] ** -0.5).masked_fill(~see, -math.inf), -1)
    return (p @ v).transpose(0, 1)[None], (p @ v.abs()).transpose(0, 1)[None]


def check(q, k, v, rows=slice(None)):
    lse = torch.empty((1, HQ, LEN), device="cuda")
    o = ops.swa_fwd(q.cuda(), k.cuda(), v.cuda(), W, lse=lse).cpu().double()[:, rows]
    assert ops.get_status() == L.SAMBA_OK
    want, mag = (t[:, rows] for t in swa64(q, k, v))
    assert torch.equal(torch.isnan(o), torch.isnan(want))
    assert torch.equal(torch.isnan(lse.cpu().transpose(1, 2))[:, rows], torch.isnan(want).any(-1))
    bad = (o - want).abs() > 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -13) * mag
    assert not bool((bad & ~torch.isnan(want)).any())


@pytest.mark.parametrize("d", [16, 32, 64])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_a_visible_key_that_is_not_finite(d, bad):
    for p in (*range(16), 128 + 15, 256 + 14):
        q, k, v = inputs(d, 300 + p)
        q[..., 3] = 1.0
        k[0, p, 0, 3] = float(bad)
        check(q, k, v)


@pytest.mark.parametrize("d", [16, 32, 64])
def test_a_query_that_is_not_finite(d):
    q, k, v = inputs(d, 320)
    q[0, 0, 1, 2], q[0, 131, 3, 0], q[0, 299, 2, 1] = float("nan"), float("inf"), float("-inf")
    check(q, k, v)


@pytest.mark.parametrize("d", [16, 32, 64])
def test_hidden_values_of_any_size_weigh_nothing(d):
    q, k, v = inputs(d, 330)
    v[0, 286], v[0, 287] = 2.0 ** 127, -(2.0 ** 126)   # hidden from the rows before,
    v[0, 14], v[0, 15] = -(2.0 ** 127), 2.0 ** 126     # and from those W and more behind
    check(q, k, v, slice(15 + W, 286))
