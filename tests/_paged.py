"""Paged-cache test helpers: batches of ragged sequences and the 64-bit
definitions of samba_kv_append and samba_paged_attn."""

import math
import random

import torch

from hybrid_ssm_sliding_b200 import ops

E4M3 = torch.float8_e4m3fn


def e4m3_64(x):
    """Nearest e4m3 value of each x (float64, ties to even, saturating; NaN stays)."""
    a = x.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.sign(x) * torch.round(a / step) * step


def pow2_scale(amax):
    """Smallest 2^k >= 2^-60 with amax <= 448 2^k, at most 2^30 (amax: a Python float)."""
    if amax == 0.0:
        return 2.0 ** -60
    m, e = math.frexp(amax)           # amax = m 2^e, 448 = 0.875 2^9
    return 2.0 ** max(-60, min(30, e - 9 if m <= 0.875 else e - 8))


class Case:
    """Sequences with `new[b]` new tokens after `past[b]` earlier ones, in
    pages in shuffled order; `pad` rows before and behind the sequences."""

    def __init__(self, new, past, Hq, Hkv, d, P, e4m3, seed, pad=0, extra_pages=3, slack=0):
        g = torch.Generator(device="cpu")
        g.manual_seed(seed)
        self.new, self.past, self.Hq, self.Hkv, self.d, self.P, self.e4m3 = new, past, Hq, Hkv, d, P, e4m3
        self.kv = [a + b for a, b in zip(new, past)]
        self.T = sum(new) + 2 * pad
        self.start = [pad]
        for n in new:
            self.start.append(self.start[-1] + n)
        cols = max(-(-x // P) for x in self.kv) + 1
        need = [-(-x // P) for x in self.kv]
        self.pages = sum(need) + extra_pages
        ids = list(range(self.pages))
        random.Random(seed).shuffle(ids)
        self.table = torch.full((len(new), cols), -1, dtype=torch.int32)  # unused entries hold nonsense
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
            at += n
        self.q = torch.randn((self.T, Hq, d), generator=g).to(torch.bfloat16)
        self.k = torch.randn((self.T, Hkv, d), generator=g).to(torch.bfloat16)
        self.v = torch.randn((self.T, Hkv, d), generator=g).to(torch.bfloat16)
        shape = (self.pages, Hkv, P, d)
        spread = torch.exp2(torch.randint(-3, 4, shape[:2], generator=g).float())
        x = torch.randn(shape, generator=g) * spread[..., None, None]
        y = torch.randn(shape, generator=g) * spread.flip(0)[..., None, None]
        if e4m3:
            self.ks = torch.tensor([[pow2_scale(float(x[i, h].abs().max())) for h in range(Hkv)] for i in range(self.pages)])
            self.vs = torch.tensor([[pow2_scale(float(y[i, h].abs().max())) for h in range(Hkv)] for i in range(self.pages)])
            self.kc = (x / self.ks[..., None, None]).to(E4M3)
            self.vc = (y / self.vs[..., None, None]).to(E4M3)
        else:
            self.ks = self.vs = None
            self.kc, self.vc = x.to(torch.bfloat16), y.to(torch.bfloat16)
        self.max_q, self.max_kv = max(new) + slack, max(self.kv) + 7 * slack

    def shift(self, cols):
        """The same rows `cols` pages further on (whose earlier pages nobody holds)."""
        self.past = [p + cols * self.P for p in self.past]
        self.kv = [p + cols * self.P for p in self.kv]
        self.table = torch.cat((torch.full((len(self.new), cols), -1, dtype=torch.int32), self.table), 1)
        self.max_kv += cols * self.P
        return self

    def gpu(self):
        """(cache, batch) on the GPU."""
        c = [None if t is None else t.cuda() for t in (self.kc, self.vc, self.ks, self.vs)]
        cache = ops.PagedKv(*c)
        batch = ops.PagedBatch(torch.tensor(self.start, dtype=torch.int32, device="cuda"),
                               torch.tensor(self.kv, dtype=torch.int32, device="cuda"), self.table.cuda(), self.max_q,
                               self.max_kv)
        return cache, batch

    def values(self, which):
        """The pool's values in 64 bits."""
        x, s = (self.kc, self.ks) if which == "k" else (self.vc, self.vs)
        return x.double() if s is None else x.double() * s.double()[..., None, None]

    def seq_values(self, b, which):
        """Keys or values of sequence b: [Hkv, kv_len, d] in 64 bits."""
        n = -(-self.kv[b] // self.P)
        x = self.values(which)[self.table[b, :n].long()]
        return x.transpose(0, 1).reshape(self.Hkv, n * self.P, self.d)[:, :self.kv[b]]


def rotated64(x, pos, freqs, inter):
    """x [n, H, d] (any type) rotated by pos [n] in 64 bits."""
    x = x.double().clone()
    if freqs is None:
        return x
    a = pos.double()[:, None] * freqs.double()
    co, si = torch.cos(a)[:, None], torch.sin(a)[:, None]
    h = freqs.numel()
    lo, hi = (x[..., 0:2 * h:2], x[..., 1:2 * h:2]) if inter else (x[..., :h], x[..., h:2 * h])
    u, w = lo * co - hi * si, hi * co + lo * si
    if inter:
        x[..., 0:2 * h:2], x[..., 1:2 * h:2] = u, w
    else:
        x[..., :h], x[..., h:2 * h] = u, w
    return x


def append64(c: Case, freqs, inter):
    """samba_kv_append's results in 64 bits: rotated queries, the pools' values
    and scales, and the unrounded values that were stored ({(which, page): rows})."""
    out = {"q": c.q.double(), "k": c.values("k"), "v": c.values("v")}
    if c.e4m3:
        out["k_scale"], out["v_scale"] = c.ks.double().clone(), c.vs.double().clone()
    stored = []
    for b, n in enumerate(c.new):
        s, p0 = c.start[b], c.past[b]
        pos = torch.arange(p0, p0 + n)
        out["q"][s:s + n] = rotated64(c.q[s:s + n], pos, freqs, inter)
        for which, x in (("k", rotated64(c.k[s:s + n], pos, freqs, inter)), ("v", c.v[s:s + n].double())):
            at = p0
            while at < p0 + n:
                end = min(p0 + n, (at // c.P + 1) * c.P)
                pg, o = int(c.table[b, at // c.P]), at % c.P
                rows = x[at - p0:end - p0].transpose(0, 1)
                stored.append((which, pg, o, rows))
                if not c.e4m3:
                    out[which][pg, :, o:o + end - at] = rows
                else:
                    sc = out[which + "_scale"]
                    for h in range(c.Hkv):
                        fin = rows[h][torch.isfinite(rows[h])]
                        now = pow2_scale(float(fin.abs().max()) if fin.numel() else 0.0)
                        if o:
                            now = max(now, float(sc[pg, h]))
                            codes = out[which][pg, h, :o] / now
                            out[which][pg, h, :o] = e4m3_64(codes) * now
                        out[which][pg, h, o:o + end - at] = e4m3_64(rows[h] / now) * now
                        out[which][pg, h, o + end - at:] *= now / float(sc[pg, h])  # codes of nobody stay
                        sc[pg, h] = now
                at = end
    return out, stored


def attend64(c: Case, window, scale=None):
    """samba_paged_attn in 64 bits: o [T, Hq, d] (zero in rows of no sequence)
    and the sum of p |v| of each output."""
    o = torch.zeros((c.T, c.Hq, c.d), dtype=torch.float64)
    mag = torch.zeros_like(o)
    grp = c.Hq // c.Hkv
    scale = scale or c.d ** -0.5
    for b, n in enumerate(c.new):
        if n == 0:
            continue
        k, v = c.seq_values(b, "k"), c.seq_values(b, "v")
        q = c.q[c.start[b]:c.start[b + 1]].double().transpose(0, 1)        # [Hq, n, d]
        key, pos = torch.arange(c.kv[b]), torch.arange(c.past[b], c.kv[b])
        hide = key[None] > pos[:, None]
        if window:
            hide |= key[None] + window <= pos[:, None]
        a = torch.einsum("hnd,hkd->hnk", q, k.repeat_interleave(grp, 0)) * scale
        p = torch.softmax(a.masked_fill(hide, -math.inf), -1)
        vv = torch.where(hide.all(0)[:, None], torch.zeros_like(v), v).repeat_interleave(grp, 0)
        o[c.start[b]:c.start[b + 1]] = (p @ vv).transpose(0, 1)
        mag[c.start[b]:c.start[b + 1]] = (p @ vv.abs()).transpose(0, 1)
    return o, mag
