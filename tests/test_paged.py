"""The paged cache on the GPU: samba_kv_append and samba_paged_attn against
their definitions in 64 bits, at the sizes and batches where they can go
wrong; refusals; captured and replayed, on other streams, with bad batches.

Tolerances.  Rotation: the turn is rounded to fp32 (2^-25 of a turn, 2^-22.3
in the angle) and the sine, cosine and products add a few 2^-24, together
below 2^-20 of |x| + |y| of the pair, before the result is rounded once: half
a step is 2^-8 of the value in bf16, 2^-4 in e4m3 (2^-10 of the page's scale
in its subnormal range).  Attention: the output's half step, 2^-8 of it; the
probabilities' rounding (2^-8 in bf16, 2^-11 in f16 for an 8-bit cache) and
the scores' (fp32 sums of up to 128 terms and an exponential of relative
error about 2^-20 times a score below 64, under 2^-13) against sum p |v|; and
f16 probabilities below 2^-14 lose up to 2^-25 each of sum |v|."""

import pytest
import torch

from hybrid_ssm_sliding_b200 import _lib as L
from hybrid_ssm_sliding_b200 import build as B
from hybrid_ssm_sliding_b200 import ops
from tests._paged import E4M3, Case, append64, attend64

pytestmark = pytest.mark.gpu

BF16_HALF, E4M3_HALF = 2.0 ** -8, 2.0 ** -4


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


def make_freqs(rot):
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) if rot else None


def run_append(c, rot, inter, packed=False):
    freqs = make_freqs(rot)
    cache, batch = c.gpu()
    if packed:  # q, k and v as column ranges of one matrix
        m = torch.cat([t.flatten(1) for t in (c.q, c.k, c.v)], 1).cuda()
        nq, nk = c.Hq * c.d, c.Hkv * c.d
        q, k, v = (t.unflatten(1, (-1, c.d)) for t in (m[:, :nq], m[:, nq:nq + nk], m[:, nq + nk:]))
    else:
        q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    out = torch.full(c.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ops.kv_append(q, k, v, cache, batch, freqs=None if freqs is None else freqs.cuda(), interleaved=inter, q_out=out)
    assert ops.get_status() == L.SAMBA_OK
    return out.cpu(), cache


def check_append(c, rot, inter, got_q, cache):
    want, stored = append64(c, make_freqs(rot), inter)
    q = got_q.double()
    live = torch.zeros(c.T, dtype=torch.bool)
    live[c.start[0]:c.start[-1]] = True
    assert torch.equal(q[~live], torch.full_like(q[~live], 7.0))  # rows of no sequence stay as they were
    pair = c.q.double().abs().amax(-1, keepdim=True) * 2
    err = (q - want["q"]).abs() - (BF16_HALF * want["q"].abs() + 2.0 ** -20 * pair)
    assert float(err[live].max()) <= 0
    for which, pool, scale in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale)):
        x = pool.cpu().double()
        if c.e4m3:
            s = scale.cpu().double()
            assert torch.equal(s, want[which + "_scale"]), which
            x = x * s[..., None, None]
        if which == "v" or rot == 0:  # nothing but one rounding
            assert torch.equal(x, want["v"] if which == "v" else want["k"].to(torch.bfloat16).double() if not c.e4m3
                               else want["k"])
            continue
        exact = want["k"].clone()     # unrounded where this call stored
        touched = torch.zeros(exact.shape, dtype=torch.bool)
        for w, pg, o, rows in stored:
            if w == "k":
                exact[pg, :, o:o + rows.shape[1]] = rows
                touched[pg, :, o:o + rows.shape[1]] = True
        tol = (E4M3_HALF if c.e4m3 else BF16_HALF) * exact.abs() + 2.0 ** -20 * 2 * exact.abs().amax(-1, keepdim=True)
        if c.e4m3:
            tol = tol + 2.0 ** -10 * want["k_scale"][..., None, None]
        assert float(((x - exact).abs() - tol)[touched].max()) <= 0
        assert torch.equal(x[~touched], exact[~touched])   # the rest as before, or re-rounded to a grown scale


APPEND = [
    # new, past, Hq, Hkv, d, P, rot, inter
    ([1], [0], 1, 1, 16, 16, 16, False),
    ([1, 1, 1, 1], [0, 15, 16, 999], 8, 2, 64, 16, 64, False),
    ([0, 3, 0, 70, 0], [5, 14, 0, 33, 900], 4, 4, 32, 32, 16, True),
    ([129, 1, 64], [127, 255, 64], 32, 4, 64, 64, 64, False),
    ([300, 255], [0, 257], 16, 1, 128, 256, 128, True),
    ([17, 40], [3, 130], 6, 3, 128, 128, 64, False),
    ([33, 2], [1, 62], 3, 3, 64, 64, 0, False),
    ([1] * 40, list(range(0, 400, 10)), 4, 2, 32, 16, 32, False),
    ([300, 5], [0, 251], 1, 1, 128, 256, 128, False),
    ([7, 40], [12, 0], 300, 1, 128, 64, 128, False),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"{len(c[0])}x{max(c[0])}_h{c[2]}.{c[3]}_d{c[4]}_p{c[5]}_r{c[6]}")
def test_append_matches_its_definition(case, e4m3):
    new, past, Hq, Hkv, d, P, rot, inter = case
    c = Case(new, past, Hq, Hkv, d, P, e4m3, seed=len(new) + d + P, pad=3, slack=2)
    q, cache = run_append(c, rot, inter)
    check_append(c, rot, inter, q, cache)


@pytest.mark.parametrize("e4m3", [False, True])
def test_append_takes_column_ranges_and_far_positions(e4m3):
    c = Case([2, 5], [255, 70], 8, 2, 64, 256, e4m3, seed=3, pad=1).shift(3905)  # positions about 10^6
    q, cache = run_append(c, 64, False, packed=True)
    check_append(c, 64, False, q, cache)


@pytest.mark.parametrize("e4m3", [False, True])
def test_append_without_queries_and_in_place(e4m3):
    c = Case([9, 30], [3, 20], 2, 2, 32, 16, e4m3, seed=4)
    want, ref = run_append(c, 32, False)
    cache, batch = c.gpu()
    fr = make_freqs(32).cuda()
    assert ops.kv_append(None, c.k.cuda(), c.v.cuda(), cache, batch, freqs=fr) is None
    q = c.q.cuda()
    ops.kv_append(q, c.k.cuda(), c.v.cuda(), c.gpu()[0], batch, freqs=fr, q_out=q)
    assert torch.equal(q.cpu(), want)
    assert torch.equal(cache.k.view(torch.uint8), ref.k.view(torch.uint8))
    assert torch.equal(cache.v.view(torch.uint8), ref.v.view(torch.uint8))


def test_append_grows_a_scale_token_by_token():
    """Tokens of growing size one call at a time: earlier codes are re-rounded
    whenever the page's scale grows; zeros, NaN and infinities keep it."""
    c = Case([1], [0], 1, 1, 16, 16, True, seed=5)
    cache, _ = c.gpu()
    cache.k_scale.fill_(float("nan"))  # an uninitialised pool
    pg = int(c.table[0, 0])
    rows = torch.randn((8, 1, 16), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    rows *= torch.tensor([1.0, 0.0, 2.0, 2.0 ** 20, 1.0, 2.0 ** -40, 3.0, 2.0 ** 21], dtype=torch.bfloat16)[:, None, None]
    rows[4, 0, 3], rows[4, 0, 5] = float("nan"), float("-inf")
    want, scale = torch.zeros(16, 16, dtype=torch.float64), 0.0
    from tests._paged import e4m3_64, pow2_scale
    for t in range(8):
        batch = ops.PagedBatch(torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                               torch.tensor([t + 1], dtype=torch.int32, device="cuda"), c.table.cuda(), 1, 16)
        x = rows[t:t + 1].cuda()
        ops.kv_append(None, x, x, cache, batch)
        r = rows[t, 0].double()
        fin = r[torch.isfinite(r)].abs().max()
        now = max(scale, pow2_scale(float(fin)))
        want[:t] = e4m3_64(want[:t] / now) * now
        want[t] = e4m3_64(r / now) * now
        scale = now
        got = cache.k[pg, 0].cpu().double() * float(cache.k_scale[pg, 0])
        assert float(cache.k_scale[pg, 0]) == scale, t
        assert torch.equal(torch.nan_to_num(got[:t + 1], nan=12345.0), torch.nan_to_num(want[:t + 1], nan=12345.0)), t
    assert ops.get_status() == L.SAMBA_OK


def test_append_beyond_the_largest_and_smallest_scale():
    c = Case([2], [0], 1, 1, 16, 16, True, seed=7)
    cache, batch = c.gpu()
    x = torch.zeros((2, 1, 16), dtype=torch.bfloat16)
    x[0, 0, 0] = 2.0 ** 100
    k = torch.full((2, 1, 16), 2.0 ** -80, dtype=torch.bfloat16)
    ops.kv_append(None, k.cuda(), x.cuda(), cache, batch)
    pg = int(c.table[0, 0])
    assert float(cache.v_scale[pg, 0]) == 2.0 ** 30 and float(cache.v[pg, 0, 0, 0]) == 448.0
    assert float(cache.k_scale[pg, 0]) == 2.0 ** -60 and float(cache.k[pg, 0, :2].float().abs().max()) == 0.0


# ------------------------------------------------------------------ attention
def check_attn(c, window, o, scale=None):
    want, mag = attend64(c, window, scale)
    o = o.cpu().double()
    live = torch.zeros(c.T, dtype=torch.bool)
    live[c.start[0]:c.start[-1]] = True
    assert torch.equal(o[~live], torch.full_like(o[~live], 7.0))
    vsum = max(float(c.seq_values(b, "v").abs().sum(1).max()) for b in range(len(c.new)) if c.kv[b])
    tol = BF16_HALF * want.abs() + ((2.0 ** -11 if c.e4m3 else BF16_HALF) + 2.0 ** -13) * mag
    if c.e4m3:
        tol = tol + 2.0 ** -25 * vsum
    bad = (o - want).abs() - tol
    assert float(bad[live].max()) <= 0, float((o - want)[live].abs().max())


def run_attn(c, window, **kw):
    cache, batch = c.gpu()
    o = torch.full(c.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ops.paged_attn(c.q.cuda(), cache, batch, window=window, o=o, **kw)
    assert ops.get_status() == L.SAMBA_OK
    return o


ATTN = [
    # new, past, Hq, Hkv, d, P, window
    ([1], [0], 1, 1, 16, 16, 0),
    ([1, 1, 1], [0, 127, 128], 8, 1, 64, 16, 0),
    ([1, 1, 0, 1], [3000, 17, 40, 2047], 32, 4, 64, 64, 2048),
    ([1], [5000], 16, 1, 128, 128, 0),
    ([1, 1], [300, 1000], 4, 4, 128, 16, 100),
    ([1] * 9, [0, 1, 2, 15, 16, 31, 32, 255, 256], 6, 2, 32, 256, 1),
    ([2, 5, 1], [700, 0, 64], 8, 4, 64, 32, 300),
    ([3, 1], [1200, 9], 16, 1, 32, 16, 0),
    ([130, 1, 0, 77], [0, 500, 9, 250], 8, 2, 64, 64, 0),
    ([257, 64], [100, 383], 4, 4, 128, 32, 128),
    ([200, 3], [0, 129], 16, 1, 16, 128, 33),
    ([333], [0], 10, 2, 32, 16, 0),
    ([129, 128, 127], [1, 0, 385], 32, 4, 64, 256, 2048),
    ([70], [1000], 3, 3, 128, 64, 0),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("case", ATTN, ids=lambda c: f"{len(c[0])}x{max(c[0])}_{max(c[1])}_h{c[2]}.{c[3]}_d{c[4]}_p{c[5]}_w{c[6]}")
def test_attention_matches_its_definition(case, e4m3):
    new, past, Hq, Hkv, d, P, window = case
    c = Case(new, past, Hq, Hkv, d, P, e4m3, seed=11 + len(new) + d + P, pad=2, slack=3)
    check_attn(c, window, run_attn(c, window))


MANY = [
    # new, past, Hq, Hkv, d, P, window: rows and heads enough that no key tiles are split off
    ([130] * 9, [1700, 1500, 0, 1601, 1024, 900, 1151, 1407, 1279], 18, 18, 64, 64, 0),
    ([129] * 9, [1200] * 9, 18, 18, 16, 16, 0),
    ([257] * 9, [1300] * 9, 18, 18, 128, 128, 1200),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("case", MANY, ids=lambda c: f"d{c[4]}_p{c[5]}_w{c[6]}")
def test_attention_over_many_key_tiles(case, e4m3):
    """More key tiles a block than any of its rings holds."""
    new, past, Hq, Hkv, d, P, window = case
    c = Case(new, past, Hq, Hkv, d, P, e4m3, seed=5 + d, slack=2)
    check_attn(c, window, run_attn(c, window))


LOOSE = [
    # new, past, Hq, Hkv, d, P, window, max_kv
    ([1], [0], 4, 2, 64, 16, 0, 400000),
    ([1, 1, 0, 1, 1], [4000, 17, 300, 31, 700], 8, 1, 64, 64, 0, 300000),
    ([1] * 7, [5, 64, 900, 33, 1500, 0, 31], 16, 2, 128, 16, 0, 60000),
    ([1, 2, 0, 2], [700, 95, 3, 1200], 8, 2, 32, 32, 0, 900000),
    ([3, 1, 2], [250, 640, 1000], 12, 4, 64, 128, 90, 200000),
    ([4, 4], [2000, 3], 16, 1, 16, 256, 0, 2000000),
    ([1] * 130, [11 * i % 97 for i in range(130)], 2, 2, 32, 16, 0, 30000),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("case", LOOSE, ids=lambda c: f"{len(c[0])}x{max(c[0])}_h{c[2]}.{c[3]}_d{c[4]}_p{c[5]}_w{c[6]}")
def test_attention_under_loose_bounds(case, e4m3):
    """Bounds far above the lengths: the positions are shared out end to end
    (or over many splits), most of them to nobody."""
    new, past, Hq, Hkv, d, P, window, max_kv = case
    c = Case(new, past, Hq, Hkv, d, P, e4m3, seed=80 + len(new) + d, pad=1)
    c.max_kv = max_kv
    check_attn(c, window, run_attn(c, window))


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_with_large_scores_and_own_scale(e4m3, new):
    """Scores of some hundred: the running maximum moves often, and most
    probabilities are zero."""
    c = Case([new, new], [700, 90], 8, 2, 64, 16, e4m3, seed=21)
    c.q = (c.q.float() * 8).to(torch.bfloat16)
    cache, batch = c.gpu()
    o = ops.paged_attn(c.q.cuda(), cache, batch, scale=0.25)
    want, mag = attend64(c, 0, 0.25)
    # a score up to 2^11 carries fp32 sums' 2^-22 of its terms: an exponent off by 2^-10
    tol = BF16_HALF * want.abs() + (BF16_HALF + 2.0 ** -9) * mag
    assert float(((o.cpu().double() - want).abs() - tol).max()) <= 0


@pytest.mark.parametrize("new", [1, 33])
@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_ignores_what_is_masked(e4m3, new):
    """NaN and infinities behind the last position, before the window and in
    pages of nobody change nothing."""
    c = Case([new, new], [150, 100], 8, 2, 64, 16, e4m3, seed=22)
    window = 60
    want = run_attn(c, window)
    cache, batch = c.gpu()
    visible = torch.zeros((c.pages, c.P), dtype=torch.bool)
    for b in range(2):
        for p in range(max(0, c.past[b] - window + 1), c.kv[b]):
            visible[int(c.table[b, p // c.P]), p % c.P] = True
    hidden = ~visible[:, None, :, None].expand(c.kc.shape).cuda()
    for t in (cache.k, cache.v):
        bad = torch.full(t.shape, float("nan"), device="cuda")
        bad[..., ::2] = float("inf")
        t.copy_(torch.where(hidden, bad.to(t.dtype).float(), t.float()).to(t.dtype))
    o = ops.paged_attn(c.q.cuda(), cache, batch, window=window)
    assert torch.equal(o, want)


def test_attention_with_pages_of_very_different_scales():
    """An all-zero page (the smallest scale) beside pages of large values."""
    c = Case([1], [63], 4, 1, 64, 16, True, seed=23)
    ids = c.table[0, :4].long()
    c.vs[ids[0]], c.vs[ids[1]], c.vs[ids[2]] = 2.0 ** -60, 2.0 ** 20, 2.0 ** -20
    c.vc[ids[0]] = torch.zeros_like(c.vc[ids[0]].float()).to(E4M3)
    c.ks[ids[3]] = 2.0 ** -60
    want, mag = attend64(c, 0)
    o = run_attn(c, 0).cpu().double()
    tol = BF16_HALF * want.abs() + (2.0 ** -11 + 2.0 ** -13) * mag + 2.0 ** -25 * float(c.seq_values(0, "v").abs().sum(1).max())
    assert float(((o - want).abs() - tol).max()) <= 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("new", [1, 150])
def test_attention_is_the_same_captured_and_replayed(e4m3, new):
    """A captured append and attention, replayed after the batch, the inputs
    and the cache were changed in place, on a side stream."""
    c = Case([new, new, 0], [200, 9, 40], 8, 2, 64, 32, e4m3, seed=24, slack=4)
    cache, batch = c.gpu()
    saved = [None if t is None else t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    fr = make_freqs(64).cuda()
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    q_out, o = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty((max(16, ops.paged_attn_workspace_size(batch, cache, 8, 90)),), dtype=torch.uint8, device="cuda")

    def step():
        ops.kv_append(q, k, v, cache, batch, freqs=fr, q_out=q_out)
        ops.paged_attn(q_out, cache, batch, window=90, o=o, workspace=ws)

    def restore():
        for t, s in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), saved):
            if t is not None:
                t.copy_(s)

    def vary():  # one more and two fewer positions before the new rows
        batch.kv_len.add_(torch.tensor([1, -2, 3], dtype=torch.int32, device="cuda"))
        q.mul_(-1)

    step()
    first = o.clone()
    restore()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    o.fill_(0)
    graph.replay()
    assert torch.equal(o, first)
    restore()
    vary()
    step()
    second = o.clone()
    restore()
    o.fill_(0)
    graph.replay()
    assert torch.equal(o, second) and not torch.equal(first, second)
    assert ops.get_status() == L.SAMBA_OK


def test_calls_on_two_streams_at_once():
    cs = [Case([1] * 8, [900 + 50 * i] * 8, 32, 4, 64, 64, True, seed=30 + i) for i in range(2)]
    want = [run_attn(c, 0) for c in cs]
    state = [c.gpu() for c in cs]
    qs = [c.q.cuda() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            outs[i].append(ops.paged_attn(qs[i], *state[i], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


def test_bad_batches_are_reported_and_skipped():
    c = Case([1, 2, 1], [40, 30, 17], 4, 2, 32, 16, False, seed=40)
    want = run_attn(c, 0)

    def run(start=None, kv=None, table=None):
        cache, batch = c.gpu()
        start = c.start if start is None else start
        kv = c.kv if kv is None else kv
        table = c.table if table is None else table
        batch = ops.PagedBatch(torch.tensor(start, dtype=torch.int32, device="cuda"),
                               torch.tensor(kv, dtype=torch.int32, device="cuda"), table.cuda(), 2, 64)
        q = c.q.cuda()
        o = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        ops.paged_attn(q, cache, batch, o=o)
        a = ops.get_status()
        k0 = cache.k.clone()
        qo = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        ops.kv_append(q, c.k.cuda(), c.v.cuda(), cache, batch, q_out=qo)
        return o, qo, a, ops.get_status(), (cache.k != k0).flatten(1).any(1).cpu()

    o, qo, a, b, _ = run()
    assert torch.equal(o, want) and a == b == L.SAMBA_OK
    for kv in ([c.kv[0], 65, c.kv[2]], [c.kv[0], 1, c.kv[2]], [c.kv[0], -4, c.kv[2]]):  # past the bound, below its rows
        o, qo, a, b, hit = run(kv=kv)
        assert a == b == L.SAMBA_ERR_BATCH
        assert torch.equal(o[[0, 3]], want[[0, 3]]) and float((o[1:3] - 7).abs().max()) == 0
        assert float((qo[1:3] - 7).abs().max()) == 0
        assert not hit[c.table[1][c.table[1] >= 0].long()].any()
    o, qo, a, b, hit = run(start=[0, 1, 3, 9])                  # past the rows
    assert a == b == L.SAMBA_ERR_BATCH and torch.equal(o[:3], want[:3]) and float((o[3] - 7).abs().max()) == 0
    t = c.table.clone()
    t[1, 1] = c.pages                                            # no such page
    o, qo, a, b, hit = run(table=t)
    assert a == L.SAMBA_ERR_BATCH and torch.equal(o[[0, 3]], want[[0, 3]])
    assert ops.get_status() == L.SAMBA_OK                        # read and cleared


def test_a_cache_past_32_bit_offsets():
    """Pages whose byte offset is beyond 2^32."""
    P, Hkv, d = 256, 8, 128
    pages = (2 ** 32) // (P * Hkv * d * 2) + 9
    k = torch.zeros((pages, Hkv, P, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    c = Case([40], [300], 16, Hkv, d, P, False, seed=50)
    ids = torch.tensor([pages - 1, 3, pages - 2], dtype=torch.int32)
    k[ids[:2].long().cuda()] = c.kc[c.table[0, :2].long()].cuda()
    v[ids[:2].long().cuda()] = c.vc[c.table[0, :2].long()].cuda()
    cache = ops.PagedKv(k, v)
    batch = ops.PagedBatch(torch.tensor([0, 40], dtype=torch.int32, device="cuda"),
                           torch.tensor([340], dtype=torch.int32, device="cuda"), ids[None].cuda(), 40, 400)
    o = ops.paged_attn(c.q.cuda(), cache, batch)
    assert torch.equal(o, run_attn(c, 0))
    ops.kv_append(None, c.k.cuda(), c.v.cuda(), cache, batch)
    assert torch.equal(k[3, :, 300 - 256:340 - 256].transpose(0, 1).cpu(), c.k)
    assert ops.get_status() == L.SAMBA_OK


def test_refusals():
    c = Case([2], [10], 4, 2, 32, 16, True, seed=60)
    cache, batch = c.gpu()
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    fr = make_freqs(32).cuda()
    with pytest.raises(TypeError):
        ops.kv_append(q.float(), k, v, cache, batch)
    with pytest.raises(ValueError):
        ops.kv_append(q, k[:1], v, cache, batch)
    with pytest.raises(ValueError):
        ops.kv_append(q, k[:, :1], v, cache, batch)
    with pytest.raises(ValueError):
        ops.kv_append(q.transpose(0, 1).contiguous().transpose(0, 1), k, v, cache, batch)
    with pytest.raises(TypeError):
        ops.kv_append(q, k, v, cache, batch, freqs=fr.float())
    with pytest.raises(L.SambaError):
        ops.kv_append(q, k, v, cache, batch, freqs=make_freqs(48).cuda())  # past the head
    with pytest.raises(ValueError):
        ops.kv_append(q.cpu(), k, v, cache, batch)
    with pytest.raises(ValueError):
        ops.PagedKv(cache.k, cache.v)                                     # 8 bits without scales
    with pytest.raises(TypeError):
        ops.PagedKv(cache.k.float(), cache.v.float())
    with pytest.raises(ValueError):
        ops.PagedBatch(batch.q_start[:1], batch.kv_len, batch.block_table, 1, 12)
    with pytest.raises(TypeError):
        ops.PagedBatch(batch.q_start.long(), batch.kv_len, batch.block_table, 1, 12)
    with pytest.raises(ValueError):
        ops.paged_attn(q[..., :16], cache, batch)
    with pytest.raises(L.SambaError) as e:
        ops.paged_attn(torch.zeros((2, 5, 32), dtype=torch.bfloat16, device="cuda"), cache, batch)
    assert e.value.code == L.SAMBA_ERR_INVALID_ARG
    with pytest.raises(L.SambaError) as e:
        ops.paged_attn(q, cache, batch, window=-1)
    assert e.value.code == L.SAMBA_ERR_INVALID_ARG
    big = Case([1], [2000], 4, 2, 32, 16, False, seed=61)
    bc, bb = big.gpu()
    need = ops.paged_attn_workspace_size(bb, bc, 4)
    assert need > 0
    with pytest.raises(L.SambaError) as e:
        ops.paged_attn(big.q.cuda(), bc, bb, workspace=torch.empty((need - 1,), dtype=torch.uint8, device="cuda"))
    assert e.value.code == L.SAMBA_ERR_WORKSPACE
    assert ops.get_status() == L.SAMBA_OK


def test_empty_calls():
    c = Case([0, 0], [10, 3], 4, 2, 32, 16, False, seed=62)
    cache, batch = c.gpu()
    q = torch.empty((0, 4, 32), dtype=torch.bfloat16, device="cuda")
    kv = torch.empty((0, 2, 32), dtype=torch.bfloat16, device="cuda")
    assert ops.kv_append(q, kv, kv, cache, batch).shape == q.shape
    assert ops.paged_attn(q, cache, batch).shape == q.shape
    pad = torch.full((3, 4, 32), 7.0, dtype=torch.bfloat16, device="cuda")   # rows, but no sequence has any
    before = cache.k.clone()
    ops.kv_append(pad, pad[:, :2].contiguous(), pad[:, :2].contiguous(), cache, batch, q_out=pad)
    assert torch.equal(ops.paged_attn(pad, cache, batch, o=pad.clone()), pad)
    assert torch.equal(cache.k, before) and ops.get_status() == L.SAMBA_OK


@pytest.mark.parametrize("e4m3", [False, True])
def test_prompt_in_chunks_and_tokens_equals_one_prompt(e4m3):
    """A prompt appended and attended at once, in chunks, and token by token
    at its end: bf16 caches are bit for bit the same; an 8-bit page's earlier
    rows may be re-rounded as its scale grows (half a step of the larger scale)."""
    n, Hq, Hkv, d, P = 150, 8, 2, 64, 32
    one = Case([n], [0], Hq, Hkv, d, P, e4m3, seed=70)
    fr = make_freqs(d).cuda()
    q, k, v = one.q.cuda(), one.k.cuda(), one.v.cuda()
    outs, pools = [], []
    for cuts in ([0, n], [0, 33, 100, n - 3, n - 2, n - 1, n]):
        cache, _ = one.gpu()
        parts = []
        for a, b in zip(cuts, cuts[1:]):
            batch = ops.PagedBatch(torch.tensor([0, b - a], dtype=torch.int32, device="cuda"),
                                   torch.tensor([b], dtype=torch.int32, device="cuda"), one.table.cuda(), b - a, b)
            qr = ops.kv_append(q[a:b], k[a:b], v[a:b], cache, batch, freqs=fr)
            parts.append(ops.paged_attn(qr, cache, batch, window=100))
        outs.append(torch.cat(parts).double())
        pools.append(cache)
    if not e4m3:
        assert torch.equal(pools[0].k, pools[1].k) and torch.equal(pools[0].v, pools[1].v)
        # the two differ by their outputs' rounding and the probabilities' (2^-8 each, twice)
        assert float((outs[0] - outs[1]).abs().max()) <= 4 * BF16_HALF * float(v.double().abs().max())
    else:
        # keys off by up to 2^-4 a step, |q.k| scale below 64 d^-1/2: values bound the outputs
        assert torch.isfinite(outs[0]).all() and float((outs[0] - outs[1]).abs().mean()) <= 2.0 ** -4 * float(
            v.double().abs().max())
    assert ops.get_status() == L.SAMBA_OK
