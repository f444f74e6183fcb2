"""The paged cache's kernels where a warp, a tile or a call is not of one piece:
row tiles that end inside a warp, products that share tensor memory, values
that are not finite, weights far below the largest, batches out of order.
Tolerances as in test_paged.py; what a test adds to them stands at the test."""

import math

import pytest
import torch

from hybrid_ssm_sliding_b200 import _lib as L
from hybrid_ssm_sliding_b200 import build as B
from hybrid_ssm_sliding_b200 import ops
from tests._paged import Case, attend64, rotated64
from tests.test_paged import BF16_HALF, check_attn, make_freqs, run_attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


PARTIAL = [
    # new, past, Hq, Hkv, d, P: rows of a kv head that end inside a warp's 32
    ([71], [0], 1, 1, 16, 16),
    ([69, 129, 0, 161], [40, 3, 7, 300], 6, 6, 64, 32),
    ([33, 46], [900, 5], 15, 5, 32, 128),
    ([130, 67], [1, 260], 4, 2, 128, 64),
    ([65] * 40, [200 + i for i in range(40)], 8, 8, 64, 64),   # units for every SM: no splits
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("case", PARTIAL, ids=lambda c: f"{len(c[0])}x{max(c[0])}_d{c[4]}")
def test_chunk_tiles_that_end_inside_a_warp(case, e4m3):
    """Lanes without a row store nothing, and a call repeats itself bit for bit."""
    c = Case(*case, e4m3, seed=90 + case[4], pad=2)
    o = run_attn(c, 0)
    check_attn(c, 0, o)
    assert all(torch.equal(run_attn(c, 0), o) for _ in range(3))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window", [0, 700])
def test_wide_heads_where_scores_and_weights_share_columns(e4m3, window):
    """A head dimension of 128: the next key tile's scores go where the weights
    of this one are being multiplied.  Many tiles, two chains a block, no splits."""
    c = Case([140] * 20, [1024 + 37 * i for i in range(20)], 16, 8, 128, 64, e4m3, seed=95)
    o = run_attn(c, window)
    check_attn(c, window, o)
    assert all(torch.equal(run_attn(c, window), o) for _ in range(5))


# ------------------------------------------------- what is not finite
NEW = {"few rows": 3, "chunk": 150}


def check_nonfinite(c, window, o):
    """NaN where the definition in 64 bits has it, the usual bound elsewhere."""
    want, mag = attend64(c, window)
    o = o.cpu().double()
    assert torch.equal(torch.isnan(o), torch.isnan(want))
    fine = ~torch.isnan(want)
    vsum = max(float(c.seq_values(b, "v").abs().sum(1).max()) for b in range(len(c.new)))
    tol = BF16_HALF * want.abs() + ((2.0 ** -11 if c.e4m3 else BF16_HALF) + 2.0 ** -13) * mag
    tol = tol + (2.0 ** -25 * vsum if c.e4m3 else 0)
    assert not bool(((o - want).abs() > tol)[fine].any())


def poison_key(c, b, p, bad, head=0):
    """Element 5 of the key at position p of sequence b."""
    x = c.kc.float()
    x[int(c.table[b, p // c.P]), head, p % c.P, 5] = bad
    c.kc = x.to(c.kc.dtype)


@pytest.mark.parametrize("which", NEW)
@pytest.mark.parametrize("e4m3,d,bad", [(False, 64, "nan"), (False, 64, "inf"), (False, 128, "nan"), (False, 128, "-inf"),
                                        (True, 64, "nan"), (True, 16, "nan"), (True, 128, "nan")])
def test_a_visible_key_that_is_not_finite(e4m3, d, bad, which):
    """At every position modulo 16: rows that see it become NaN, whichever kernel
    takes them, and the others stay; a row that sees nothing else included."""
    n = NEW[which]
    for p in range(16):
        c = Case([n, n], [0, 40], 4, 2, d, 16, e4m3, seed=100 + p)
        c.q[c.start[0]:, :, 5] = 1.0                        # the score has the key's sign
        poison_key(c, 0, p, float(bad))
        poison_key(c, 1, 16 + p, float(bad), head=1)
        check_nonfinite(c, 0, run_attn(c, 0))
        check_nonfinite(c, 3, run_attn(c, 3))


@pytest.mark.parametrize("which", NEW)
@pytest.mark.parametrize("e4m3", [False, True])
def test_a_whole_split_of_nan_keys(e4m3, which):
    """Splits that see only NaN, and rows whose later key tiles are all hidden."""
    n = NEW[which]
    for lo, hi in ((0, 700), (1500, 2600), (4990, 5000)):
        c = Case([n], [5000], 2, 1, 64, 64, e4m3, seed=120 + n)
        x = c.kc.float()
        for p in range(lo, hi):
            x[int(c.table[0, p // 64]), 0, p % 64] = float("nan")
        c.kc = x.to(c.kc.dtype)
        for window in (0, 2000, 5):
            check_nonfinite(c, window, run_attn(c, window))


@pytest.mark.parametrize("which", NEW)
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
def test_a_query_that_is_not_finite(bad, e4m3, which):
    """Its row and head become NaN, no other."""
    n = NEW[which]
    c = Case([n, 1], [70, 9], 4, 2, 64, 32, e4m3, seed=130)
    c.q[c.start[0] + n - 2, 1, 7], c.q[c.start[1], 3, 0] = float(bad), float(bad)
    check_nonfinite(c, 0, run_attn(c, 0))
    check_nonfinite(c, 30, run_attn(c, 30))


@pytest.mark.parametrize("which", NEW)
def test_hidden_values_of_any_size_weigh_nothing(which):
    """bf16 values of 2^127 at positions that some rows do not see: exactly nothing of them reaches those rows."""
    n = NEW[which]
    c = Case([n], [300], 4, 2, 64, 64, False, seed=140)
    x = c.vc.float()
    last = c.kv[0] - 1
    x[int(c.table[0, last // 64]), :, last % 64] = 2.0 ** 127   # the last position: only the last row sees it
    c.vc = x.to(torch.bfloat16)
    for window in (0, 100):
        o, (want, mag) = run_attn(c, window).cpu().double(), attend64(c, window)
        tol = BF16_HALF * want.abs() + (BF16_HALF + 2.0 ** -13) * mag
        assert float(((o - want).abs() - tol)[:n - 1].max()) <= 0


# ------------------------------------------------- weights far below the largest
def lost_weights(c, window):
    """What f16 weights may lose of each output, in 64 bits: a weight times its value's scale is held relative to a
    row's largest at 2^7 or more, so each is off by at most half of f16's smallest step, 2^-25 there (what it
    loses above is half a step of itself, and counted with the sum of p |v|)."""
    tol = torch.zeros((c.T, c.Hq, c.d), dtype=torch.float64)
    grp = c.Hq // c.Hkv
    for b, n in enumerate(c.new):
        k, v = c.seq_values(b, "k"), c.seq_values(b, "v")
        page = c.table[b, torch.arange(c.kv[b]) // c.P].long()
        vs = c.vs.double()[page].T.repeat_interleave(grp, 0)[:, None, :]                     # [Hq, 1, kv]
        q = c.q[c.start[b]:c.start[b + 1]].double().transpose(0, 1)
        key, pos = torch.arange(c.kv[b]), torch.arange(c.past[b], c.kv[b])
        see = key[None] <= pos[:, None]
        if window:
            see &= key[None] + window > pos[:, None]
        s = torch.einsum("hnd,hkd->hnk", q, k.repeat_interleave(grp, 0)) * c.d ** -0.5
        w = torch.where(see, torch.exp(s) * vs, torch.zeros((), dtype=torch.float64))
        w = w / w.amax(-1, keepdim=True) * 2.0 ** 7
        codes = v.abs().repeat_interleave(grp, 0) / vs.transpose(1, 2)
        lost = 2.0 ** -25 * see.double() @ codes / (w / vs).sum(-1, keepdim=True)
        tol[c.start[b]:c.start[b + 1]] = lost.transpose(0, 1)
    return tol


@pytest.mark.parametrize("which", NEW)
@pytest.mark.parametrize("apart", [10, 20, 26, 40])
def test_small_scales_beside_a_large_one(apart, which):
    """A page of a value scale 2^apart times the others', zero in half of its
    elements: there the others' values are the answer."""
    n = NEW[which]
    c = Case([n, n], [79, 700], 8, 2, 64, 16, True, seed=150 + apart)
    c.vs = c.vs * 2.0 ** -16                                # all within 2^-60 .. 2^30
    for b in range(2):
        pg = int(c.table[b, 1])
        c.vs[pg] = c.vs[pg] * 2.0 ** apart
        x = c.vc.float()
        x[pg, :, :, ::2] = 0
        c.vc = x.to(torch.float8_e4m3fn)
    for window in (0, 0 if n == 150 else 75):
        o = run_attn(c, window).cpu().double()
        want, mag = attend64(c, window)
        tol = BF16_HALF * want.abs() + (2.0 ** -11 + 2.0 ** -13) * mag + lost_weights(c, window)
        assert float(((o - want).abs() / tol).max()) <= 1


# ------------------------------------------------- batches out of order
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("value", [999, -5, -2 ** 31, 2 ** 31 - 1, 0, 40])
@pytest.mark.parametrize("B", [5, 300])
def test_an_entry_of_q_start_out_of_range_costs_its_neighbours_only(B, value, e4m3):
    """The sequences on both sides of the entry fail; every other one gets its keys, values and
    rotated queries, as from a batch without the fault, and attends them."""
    new = [(3, 1, 17, 2, 0)[b % 5] for b in range(B)]
    bad = B // 2                                                   # the entry between sequences bad - 1 and bad
    c = Case(new, [(b * 7) % 40 for b in range(B)], 4, 2, 32, 16, e4m3, seed=160 + B)
    fr, q, k, v = make_freqs(32).cuda(), c.q.cuda(), c.k.cuda(), c.v.cuda()
    res = []
    for broken in (False, True):
        cache, batch = c.gpu()
        if broken:
            batch.q_start[bad] = value
        before = cache.k.view(torch.uint8).clone()
        qo, o = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
        ops.kv_append(q, k, v, cache, batch, freqs=fr, q_out=qo)
        assert ops.get_status() == (L.SAMBA_ERR_BATCH if broken else L.SAMBA_OK)
        ops.paged_attn(qo, cache, batch, o=o)
        assert ops.get_status() == (L.SAMBA_ERR_BATCH if broken else L.SAMBA_OK)
        pools = [t.view(torch.uint8).clone() if t.dtype != torch.float32 else t.clone()
                 for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]
        res.append((qo, o, pools))
    (q0, o0, p0), (q1, o1, p1) = res
    start = [*c.start[:bad], value, *c.start[bad + 1:]]
    for b in range(B):
        rows = slice(c.start[b], c.start[b + 1])
        pages = c.table[b, :-(-c.kv[b] // c.P)].long().cuda()
        if b in (bad - 1, bad):
            assert start[b] < 0 or not 0 <= start[b + 1] - start[b] <= c.max_q     # out of range
            assert bool((q1[rows] == 7).all()) and bool((o1[rows] == 7).all())
            assert torch.equal(p1[0][pages], before[pages])
        else:
            assert torch.equal(q0[rows], q1[rows]) and torch.equal(o0[rows], o1[rows]), b
            assert all(torch.equal(x[pages], y[pages]) for x, y in zip(p0, p1)), b


# ------------------------------------------------- angles
@pytest.mark.parametrize("inter", [False, True])
def test_rotation_next_to_quarter_turns(inter):
    """Angles within 2^-22 turns a position of quarter turns, one element of each pair zero: what is left is x times
    a sine or cosine down to 2^-20, held to a part of itself.  The sine and cosine
    are off by 2^-23 of themselves, their turn's rest adds one rounding and the
    product one (2^-24 each), then the result is rounded once."""
    n, d = 97, 64
    c = Case([n], [0], 2, 2, d, 32, False, seed=170)
    j = torch.arange(d // 2, dtype=torch.float64)
    turns = 0.25 + 2.0 ** -22 * (1 + 0.137 * j) * torch.where(j.long() % 2 == 0, 1.0, -1.0)
    freqs = turns * 2 * math.pi
    hi = slice(1, d, 2) if inter else slice(d // 2, d)
    c.q[..., hi], c.k[..., hi] = 0, 0
    cache, batch = c.gpu()
    q = ops.kv_append(c.q.cuda(), c.k.cuda(), c.v.cuda(), cache, batch, freqs=freqs.cuda(), interleaved=inter)
    rows = torch.cat([cache.k[int(pg)].transpose(0, 1) for pg in c.table[0, :4]])[:n]
    for x, got in ((c.q, q), (c.k, rows)):
        want = rotated64(x, torch.arange(n), freqs, inter)
        # position * angle in 64 bits carries 2^-52 of up to 152 radians itself: 2^-44
        tol = (BF16_HALF + 2.0 ** -22) * want.abs() + 2.0 ** -44 * x.double().abs().amax(-1, keepdim=True)
        assert float(((got.cpu().double() - want).abs() - tol).max()) <= 0
    assert ops.get_status() == L.SAMBA_OK
