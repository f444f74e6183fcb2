"""Kernels that read tensor memory by whole warps, at sizes whose last rows end inside a warp: every output once, nothing
behind it.  GEMM: half a bf16 step, 2^-8, and fp32 sums of 2^-20 of sum |a b|.  SWA backward: the roundings of P, dS and o (2^-8 each
of the sum of the terms' sizes, 2^-7 with the fp32 sums) and of the result."""

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


@pytest.mark.parametrize("M", [33, 47, 129, 161])
@pytest.mark.parametrize("N", [40, 200, 296])
def test_gemm_rows_that_end_inside_a_warp(M, N):
    K = 96
    g = torch.Generator(device="cuda").manual_seed(500 + M + N)
    a, w = (torch.randn((r, K), generator=g, device="cuda").to(torch.bfloat16) for r in (M, N))
    pool = torch.full((M + 3, N), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.gemm(a, w, outs=[(pool[:M, :24], 0, 24, None), (pool[:M, 24:], 24, N, None)])
    assert ops.get_status() == L.SAMBA_OK
    want, mag = a.double() @ w.double().T, a.double().abs() @ w.double().abs().T
    assert float(((pool[:M].double() - want).abs() - 2.0 ** -8 * want.abs() - 2.0 ** -20 * mag).max()) <= 0
    assert bool((pool[M:] == 7).all())


@pytest.mark.parametrize("n", [1, 45, 131, 257])
@pytest.mark.parametrize("d,group", [(64, 1), (64, 8), (32, 2), (16, 4)])
def test_swa_backward_rows_that_end_inside_a_warp(n, d, group):
    W, Hkv = 70, 2
    g = torch.Generator(device="cuda").manual_seed(510 + n + d)
    q, k, v, do = (torch.randn((1, n, h, d), generator=g, device="cuda").to(torch.bfloat16)
                   for h in (Hkv * group, Hkv, Hkv, Hkv * group))
    lse = torch.empty((1, Hkv * group, n), device="cuda")
    o = ops.swa_fwd(q, k, v, W, lse=lse)
    dq, dk, dv = ops.swa_bwd(do, q, k, v, o, lse, W)
    assert ops.get_status() == L.SAMBA_OK
    Q, K, V, G = (t[0].double().transpose(0, 1) for t in (q, k, v, do))
    K, V = (t.repeat_interleave(group, 0) for t in (K, V))
    i = torch.arange(n, device="cuda")
    see = (i[None] <= i[:, None]) & (i[None] > i[:, None] - W)
    sc = d ** -0.5
    p = torch.softmax((Q @ K.transpose(1, 2) * sc).masked_fill(~see, -math.inf), -1)
    dp, D = G @ V.transpose(1, 2), (G * (p @ V)).sum(-1, keepdim=True)
    ds = p * (dp - D)
    big = p * (G.abs() @ V.abs().transpose(1, 2) + (G.abs() * (p @ V.abs())).sum(-1, keepdim=True))

    def per_kv(t):
        return t.unflatten(0, (Hkv, group)).sum(1)

    for got, want, mag in ((dq, ds @ K * sc, big @ K.abs() * sc),
                           (dk, per_kv(ds.transpose(1, 2) @ Q) * sc, per_kv(big.transpose(1, 2) @ Q.abs()) * sc),
                           (dv, per_kv(p.transpose(1, 2) @ G), per_kv(p.transpose(1, 2) @ G.abs()))):
        err = (got[0].double().transpose(0, 1) - want).abs() - 2.0 ** -8 * want.abs() - 2.0 ** -7 * mag
        assert float(err.max()) <= 0
