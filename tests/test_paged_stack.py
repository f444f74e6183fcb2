"""The new operators as they are used together: a stack of SWA layers over
paged caches with the norms, gates and residual sums between them, prompts in
one call and then in chunks and tokens; and gradients through two blocks.

Tolerances.  The residual stream's increments pass, a block, the roundings to
bf16 of n, of qkv, of the rotated q and k, of the probabilities, of o, of y
and of the gate: eight of at most 2^-8 of their values, which the linear maps
(of variance-keeping random weights) and the softmax's average leave at that
size, so two blocks stay below 16 * 2^-8 = 2^-4 of the increments' root mean
square even if all add up; 8 bits add 2^-4 of the cached values a block.  Means
of absolute errors are held to that."""

import pytest
import torch

from hybrid_ssm_sliding_b200 import _lib as L
from hybrid_ssm_sliding_b200 import build as B
from hybrid_ssm_sliding_b200 import layers, ops
from tests._paged import rotated64

pytestmark = pytest.mark.gpu

DM, HQ, HKV, D, P, W = 256, 8, 2, 64, 32, 150


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


def make_blocks(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def vec(by, plus):
        return torch.randn((DM,), generator=g, device="cuda") * by + plus

    out = []
    for i in range(n):
        gate = (torch.randn((DM, DM), generator=g, device="cuda") / DM ** 0.5).to(torch.bfloat16)
        out.append(layers.BlockWeights(layer=layers.random_swa_weights(DM, HQ, HKV, D, W, seed + 10 + i), w_pre=vec(0.1, 1.0),
                                       w_post=vec(0.1, 1.0), gate_proj=gate if i % 2 == 0 else None,
                                       alpha=vec(0.1, 0.7)))
    return out, vec(0.1, 1.0)


def stack64(r, lens, blocks, w_final, freqs, eps=1e-6):
    """The stack in 64 bits, without roundings in between: r [sum lens, DM]."""
    r = r.double()

    def rms(x, w):
        return x / torch.sqrt((x * x).mean(1, keepdim=True) + eps) * w.double()

    for w in blocks:
        n = rms(r, w.w_pre)
        qkv = n @ w.layer.qkv_proj.double().T
        y, at = [], 0
        for ln in lens:
            x = qkv[at:at + ln]
            pos = torch.arange(ln, device=r.device)
            q = rotated64(x[:, :HQ * D].unflatten(1, (HQ, D)), pos, freqs, False).transpose(0, 1)
            k = rotated64(x[:, HQ * D:(HQ + HKV) * D].unflatten(1, (HKV, D)), pos, freqs, False).transpose(0, 1)
            v = x[:, (HQ + HKV) * D:].unflatten(1, (HKV, D)).transpose(0, 1)
            k, v = k.repeat_interleave(HQ // HKV, 0), v.repeat_interleave(HQ // HKV, 0)
            see = (pos[None] <= pos[:, None]) & (pos[None] > pos[:, None] - W)
            p = torch.softmax((q @ k.transpose(1, 2) * D ** -0.5).masked_fill(~see, float("-inf")), -1)
            y.append((p @ v).transpose(0, 1).reshape(ln, HQ * D))
            at += ln
        y = rms(torch.cat(y) @ w.layer.o_proj.double().T, w.w_post) * w.alpha.double()
        if w.gate_proj is not None:
            y = y * torch.sigmoid(n @ w.gate_proj.double().T)
        r = r + y
    return r, rms(r, w_final)


@pytest.mark.parametrize("e4m3", [False, True])
def test_prompts_chunks_and_tokens_through_a_stack(e4m3):
    lens = [230, 1, 97]
    cuts = [[0, 100, 229, 230], [0, 0, 0, 1], [0, 64, 96, 97]]  # three calls: chunks (one sequence idle twice), then a token each
    blocks, w_final = make_blocks(2, seed=1)
    freqs = 10000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
    g = torch.Generator(device="cuda").manual_seed(2)
    r = torch.randn((sum(lens), DM), generator=g, device="cuda")
    need = [-(-n // P) for n in lens]
    table = torch.zeros((3, max(need)), dtype=torch.int32)
    perm = torch.randperm(sum(need), generator=torch.Generator().manual_seed(3)).to(torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    first = [0, lens[0], lens[0] + lens[1]]
    caches = [ops.PagedKv.empty(sum(need), HKV, P, D, dtype=dtype) for _ in blocks]
    got_r, got_n = torch.empty_like(r), torch.empty((sum(lens), DM), device="cuda")
    for step in range(3):
        new = [c[step + 1] - c[step] for c in cuts]
        rows = torch.cat([torch.arange(first[b] + cuts[b][step], first[b] + cuts[b][step + 1]) for b in range(3)]).cuda()
        start = torch.tensor([0, *new]).cumsum(0).to(torch.int32).cuda()
        kv = torch.tensor([c[step + 1] for c in cuts], dtype=torch.int32, device="cuda")
        batch = ops.PagedBatch(start, kv, table.cuda(), max(new), int(kv.max()))
        a, n = layers.paged_stack(r[rows].contiguous(), blocks, w_final, caches, batch, freqs=freqs)
        got_r[rows], got_n[rows] = a, n.float()
    assert ops.get_status() == L.SAMBA_OK
    want_r, want_n = stack64(r, lens, blocks, w_final, freqs)
    step = want_r - r.double()
    size = float(step.square().mean().sqrt())
    tol = 2.0 ** -4 + (2 * 2.0 ** -4 if e4m3 else 0)
    assert float((got_r.double() - want_r).abs().mean()) <= tol * size
    assert float((got_n.double() - want_n).abs().mean()) <= tol * size + 2.0 ** -8 * float(want_n.abs().mean())


def test_gradients_through_two_blocks():
    """Two joins with an elementwise block between them, forward and backward
    by the operators, against autograd of the same in 64 bits.  Each gradient
    passes at most eight roundings of 2^-8 on its way."""
    M, C = 600, 512
    g = torch.Generator(device="cuda").manual_seed(5)

    def n(*shape, dtype=torch.bfloat16, by=1.0, plus=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * by + plus).to(dtype)

    f32 = torch.float32
    r0, gate = n(M, C, dtype=f32), [n(M, C) for _ in range(2)]
    pre = [n(C, dtype=f32, by=0.1, plus=1.0) for _ in range(3)]
    post = [n(C, dtype=f32, by=0.1, plus=1.0) for _ in range(2)]
    alpha = [n(C, dtype=f32, by=0.1, plus=0.7) for _ in range(2)]
    scale = [n(C, dtype=f32) for _ in range(2)]         # the blocks: y = n * scale
    dn, dr = n(M, C), n(M, C, dtype=f32)
    stat = [[torch.empty((M,), device="cuda") for _ in range(2)] for _ in range(3)]
    _, x = ops.block_norm_fwd(r0, pre[0], n_dtype=torch.bfloat16, rstd_pre=stat[0][0])
    r, ys = r0, []
    rs = [r0]
    for i in range(2):
        ys.append((x.float() * scale[i]).to(torch.bfloat16))
        r, x = ops.block_norm_fwd(r, pre[i + 1], y=ys[i], w_post=post[i], gate=gate[i], alpha=alpha[i],
                                  rstd_pre=stat[i + 1][0], rstd_post=stat[i + 1][1])
        rs.append(r)
    got, d_n, d_r = {}, dn, dr
    for i in (1, 0):
        out = ops.block_norm_bwd(d_n, rs[i + 1], pre[i + 1], stat[i + 1][0], dr_out=d_r, y=ys[i], w_post=post[i],
                                 rstd_post=stat[i + 1][1], gate=gate[i], alpha=alpha[i])
        got |= {f"pre{i + 1}": out["dw_pre"], f"post{i}": out["dw_post"], f"gate{i}": out["dgate"], f"alpha{i}": out["dalpha"]}
        d_n, d_r = (out["dy"].float() * scale[i]).to(torch.bfloat16), out["dr"]
    out = ops.block_norm_bwd(d_n, r0, pre[0], stat[0][0], dr_out=d_r)
    got |= {"pre0": out["dw_pre"], "r": out["dr"]}
    assert ops.get_status() == L.SAMBA_OK

    leaf = {"r": r0, **{f"pre{i}": v for i, v in enumerate(pre)}, **{f"post{i}": v for i, v in enumerate(post)},
            **{f"gate{i}": v for i, v in enumerate(gate)}, **{f"alpha{i}": v for i, v in enumerate(alpha)}}
    leaf = {k: v.double().requires_grad_() for k, v in leaf.items()}

    def rms(v, w):
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * w

    r, x = leaf["r"], rms(leaf["r"], leaf["pre0"])
    for i in range(2):
        y = rms(x * scale[i].double(), leaf[f"post{i}"])
        r = r + leaf[f"alpha{i}"] * torch.sigmoid(leaf[f"gate{i}"]) * y
        x = rms(r, leaf[f"pre{i + 1}"])
    ((x * dn.double()).sum() + (r * dr.double()).sum()).backward()
    for k, v in leaf.items():
        size = float(v.grad.square().mean().sqrt())
        assert float((got[k].double() - v.grad).abs().mean()) <= 8 * 2.0 ** -8 * size, k
