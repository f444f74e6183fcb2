"""Pages that several calls fill, call by call against the definitions in 64
bits: codes, scales and outputs after every chunk, and the end against the
same prompt in one call."""

import copy

import pytest
import torch

from hybrid_ssm_sliding_b200 import _lib as L
from hybrid_ssm_sliding_b200 import build as B
from hybrid_ssm_sliding_b200 import layers, ops
from tests._paged import E4M3, Case
from tests.test_paged import BF16_HALF, E4M3_HALF, check_append, check_attn, make_freqs
from tests.test_paged_stack import D, DM, HKV, HQ, P, W, make_blocks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


def part_of(c, cache, lo, hi, q=None):
    """The case of rows lo[b] .. hi[b] of each sequence over the pool as it is."""
    s = copy.copy(c)
    rows = torch.cat([torch.arange(c.start[b] + lo[b], c.start[b] + hi[b]) for b in range(len(lo))])
    s.new, s.past, s.kv = [b - a for a, b in zip(lo, hi)], list(lo), list(hi)
    s.start = [0]
    for n in s.new:
        s.start.append(s.start[-1] + n)
    s.T, s.max_q, s.max_kv = s.start[-1], max(s.new), max(s.kv)
    s.q, s.k, s.v = (c.q if q is None else q)[rows], c.k[rows], c.v[rows]
    s.kc, s.vc = cache.k.cpu(), cache.v.cpu()
    s.ks, s.vs = (None, None) if cache.k_scale is None else (cache.k_scale.cpu(), cache.v_scale.cpu())
    return s, rows


def batch_of(s):
    i32 = dict(dtype=torch.int32, device="cuda")
    return ops.PagedBatch(torch.tensor(s.start, **i32), torch.tensor(s.kv, **i32), s.table.cuda(), s.max_q, s.max_kv)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,page,window", [(64, 32, 100), (128, 16, 0), (16, 128, 0)])
def test_chunks_and_tokens_step_by_step(d, page, window, e4m3):
    """Rows that grow along the prompt, so that pages begun in one call get larger scales in the next."""
    lens = [150, 61]
    cuts = [[0, 33, 100, 147, 148, 149, 150], [0, 1, 30, 30, 31, 60, 61]]
    c = Case(lens, [0, 0], 8, 2, d, page, e4m3, seed=200 + d)
    grow = torch.exp2(torch.cat([torch.linspace(-3, 3, n) for n in lens]))[:, None, None]
    c.k, c.v = (c.k.float() * grow).to(torch.bfloat16), (c.v.float() * grow).to(torch.bfloat16)
    fr = make_freqs(d).cuda()
    ends = []
    for steps in ([[0, n] for n in lens], cuts):
        cache, _ = c.gpu()
        grown = 0
        for lo, hi in zip(zip(*[x[:-1] for x in steps]), zip(*[x[1:] for x in steps])):
            s, rows = part_of(c, cache, lo, hi)
            batch = batch_of(s)
            qr = ops.kv_append(s.q.cuda(), s.k.cuda(), s.v.cuda(), cache, batch, freqs=fr)
            check_append(s, d, False, qr.cpu(), cache)
            if e4m3:
                page_b = {int(s.table[b, a // page]) for b, a in enumerate(lo) if a % page and hi[b] > a}
                grown += sum(bool((cache.k_scale[g].cpu() > s.ks[g]).any()) for g in page_b)
            full = torch.zeros_like(c.q)
            full[rows] = qr.cpu()
            t, _ = part_of(c, cache, lo, hi, q=full)
            o = ops.paged_attn(qr, cache, batch, window=window)
            check_attn(t, window, o)
        assert ops.get_status() == L.SAMBA_OK
        ends.append(cache)
        assert grown > 0 or not e4m3 or steps is not cuts
    one, many = ends
    used = torch.cat([c.table[b, :-(-n // page)] for b, n in enumerate(lens)]).long().cuda()
    seen = torch.zeros((c.pages, page), dtype=torch.bool)
    for b, n in enumerate(lens):
        for p in range(n):
            seen[int(c.table[b, p // page]), p % page] = True
    seen = seen[:, None, :, None].cuda()
    for x, y, sx, sy in ((one.k, many.k, one.k_scale, many.k_scale), (one.v, many.v, one.v_scale, many.v_scale)):
        if not e4m3:
            assert bool(((x == y) | ~seen).all())
            continue
        assert torch.equal(sx[used], sy[used])          # the largest need of a page, however it came
        scale = sx.double()[..., None, None]
        a, b = x.double() * scale, y.double() * sy.double()[..., None, None]
        # both are roundings of one value; the chunks' were rounded again at each growth, by half a step of a step then
        # at most as large as the last one: six growths here
        tol = 7 * (E4M3_HALF * torch.maximum(a.abs(), b.abs()) + 2.0 ** -10 * scale)
        assert bool((((a - b).abs() <= tol) | ~seen).all())


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_layer_over_its_own_cache(e4m3):
    """paged_swa_layer in chunks and tokens: bit for bit its projections, append and
    attention called apart, whose attention is held to 64 bits element by element."""
    w = make_blocks(1, seed=21)[0][0].layer
    n, cuts = 140, [0, 70, 71, 100, 139, 140]
    h = torch.randn((n, DM), generator=torch.Generator(device="cuda").manual_seed(22), device="cuda").to(torch.bfloat16)
    fr = make_freqs(D).cuda()
    c = Case([n], [0], HQ, HKV, D, P, e4m3, seed=24)
    cache, other = (ops.PagedKv.empty(c.pages, HKV, P, D, dtype=E4M3 if e4m3 else torch.bfloat16) for _ in range(2))
    for lo, hi in zip(cuts, cuts[1:]):
        qkv = ops.gemm(h[lo:hi], w.qkv_proj)
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([HQ * D, HKV * D, HKV * D], 1))
        s, _ = part_of(c, other, [lo], [hi])
        batch = batch_of(s)
        out = layers.paged_swa_layer(h[lo:hi], w, cache, batch, freqs=fr)
        s.q, s.k, s.v = q.cpu(), k.cpu(), v.cpu()
        qr = ops.kv_append(q, k, v, other, batch, freqs=fr)
        check_append(s, D, False, qr.cpu(), other)
        o = ops.paged_attn(qr, other, batch, window=W)
        full = torch.zeros((n, HQ, D), dtype=torch.bfloat16)
        full[lo:hi] = qr.cpu()
        check_attn(part_of(c, other, [lo], [hi], q=full)[0], W, o)
        assert torch.equal(out, ops.gemm(o.flatten(1), w.o_proj))
        for x, y in ((cache.k, other.k), (cache.v, other.v), (cache.k_scale, other.k_scale), (cache.v_scale, other.v_scale)):
            assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert ops.get_status() == L.SAMBA_OK
