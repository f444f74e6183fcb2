"""The serving and training operators around the mixers, as they are measured: their cases, their plain forms in
elementary torch operations and, where ``own`` is true, the calls of the framework's kernels.

* append: rotated keys and values of prompts or single tokens into a paged cache (bf16, or e4m3 with one power-of-two
  scale for each page and kv head), and the rotated queries;
* attend: attention of those queries over the cache, causal, over a window or over everything;
* join / join_bwd: the norms after a block and before the next one with the gate, the residual scale and the residual
  sum between them, and their gradients.
"""

import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token for each of 16 sequences, the serving loop's batch and heads, 8-bit cache
        dict(name="append tokens e4m3", op="append", seqs=16, past_lo=3900, past_hi=4100, new_lo=1, new_hi=1, heads_q=32,
             heads_kv=4, dim=64, page=64, e4m3=True, rot=64, inter=False, lens=1),
        # one new token for each of 160 sequences far into long contexts, bf16 cache of small pages
        dict(name="append tokens bf16", op="append", seqs=160, past_lo=0, past_hi=200000, new_lo=1, new_hi=1, heads_q=32,
             heads_kv=8, dim=128, page=16, e4m3=False, rot=64, inter=True, lens=2, table=8),
        # a batch of ragged prompts into an 8-bit cache
        dict(name="append prompts e4m3", op="append", seqs=9, past_lo=0, past_hi=0, new_lo=900, new_hi=6500, heads_q=32,
             heads_kv=4, dim=64, page=64, e4m3=True, rot=64, inter=False, lens=3),
        # chunks of prompts that go on from any position, bf16 cache
        dict(name="append chunks bf16", op="append", seqs=7, past_lo=0, past_hi=5000, new_lo=33, new_hi=2049, heads_q=16,
             heads_kv=16, dim=128, page=32, e4m3=False, rot=128, inter=False, lens=4),
        # a decode step of the serving loop: 16 sequences, window of 2048
        dict(name="attend tokens e4m3", op="attend", seqs=16, past_lo=3900, past_hi=4100, new_lo=1, new_hi=1, heads_q=32,
             heads_kv=4, dim=64, page=64, e4m3=True, window=2048, lens=5),
        # one sequence with a long context: the work is split over the keys
        dict(name="attend long bf16", op="attend", seqs=1, past_lo=131000, past_hi=131000, new_lo=1, new_hi=1, heads_q=32,
             heads_kv=8, dim=128, page=16, e4m3=False, window=0, lens=6),
        # a large ragged batch of decode steps over everything, 8-bit cache
        dict(name="attend ragged e4m3", op="attend", seqs=64, past_lo=500, past_hi=32000, new_lo=1, new_hi=1, heads_q=32,
             heads_kv=4, dim=64, page=32, e4m3=True, window=0, lens=7),
        # chunks of prompts over their window, 8-bit cache
        dict(name="attend chunks e4m3", op="attend", seqs=5, past_lo=100, past_hi=6000, new_lo=200, new_hi=1500, heads_q=32,
             heads_kv=4, dim=64, page=64, e4m3=True, window=2048, lens=8),
        # a decode step between two blocks: the smallest call
        dict(name="join tokens", op="join", rows=16, width=2048, r32=False, y32=False, post=True, gate=True, alpha=True),
        # a prompt between two blocks, the residual held in 32 bits
        dict(name="join prompt", op="join", rows=32768, width=2048, r32=True, y32=False, post=True, gate=True, alpha=True),
        # a small training step without the norm after the block, an odd row count
        dict(name="join gradient small", op="join_bwd", rows=1023, width=4096, r32=False, y32=False, post=False, gate=False,
             alpha=False),
        # the training step's 8 sequences of 4096 tokens with every part
        dict(name="join gradient", op="join_bwd", rows=32768, width=2048, r32=True, y32=False, post=True, gate=True,
             alpha=True),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm uniform."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "join", "join_bwd"])
    if op in ("join", "join_bwd"):
        c = dict(op=op, rows=_log(rng, 1, 20000), width=8 * _log(rng, 32, 1024), r32=rng.random() < 0.5,
                 y32=rng.random() < 0.25, post=rng.random() < 0.6, gate=rng.random() < 0.6, alpha=rng.random() < 0.6)
        c["rows"] = max(1, min(c["rows"], 24_000_000 // c["width"]))
        return c
    dim = rng.choice([64, 64, 128, 32])
    hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, seqs=0, past_lo=0, past_hi=0, new_lo=1, new_hi=1, heads_q=hkv * rng.choice([1, 2, 4, 8]), heads_kv=hkv,
             dim=dim, page=rng.choice([16, 32, 64, 128]), e4m3=rng.random() < 0.6, lens=rng.randrange(1 << 20))
    if rng.random() < 0.6:  # single tokens
        c["seqs"] = _log(rng, 1, 128)
        c["past_hi"] = _log(rng, 1, min(60000, 1_000_000 // c["seqs"]))
    else:
        c["seqs"] = _log(rng, 1, 8)
        c["new_hi"] = _log(rng, 2, 6000 // c["seqs"])
        c["past_hi"] = _log(rng, 1, 6000)
    if op == "append":
        c["rot"] = rng.choice([dim, dim, dim // 2, 0])
        c["inter"] = rng.random() < 0.3
    else:
        c["window"] = rng.choice([0, 2048, _log(rng, 1, 4000)])
    return c


def _lens(c):
    """New tokens and tokens before them, for each sequence: sizes, so they go by the case alone."""
    r = random.Random(c["lens"])
    return [(r.randint(c["new_lo"], c["new_hi"]), r.randint(c["past_lo"], c["past_hi"])) for _ in range(c["seqs"])]


# ----------------------------------------------------------------- the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _pow2_scale(amax):
    """The smallest power of two s >= 2^-60 with amax <= 448 s, at most 2^30."""
    m, e = torch.frexp(amax)
    k = torch.where(m <= 0.875, e - 9, e - 8)
    k = torch.where(amax > 0, k, torch.full_like(k, -60)).clamp(-60, 30)
    return torch.ldexp(torch.ones_like(amax), k)


def _code(x):
    return x.clamp(-448.0, 448.0).to(E4M3)


def _cache(shape, e4m3, g):
    """A pool's content: what earlier tokens left there."""
    x = torch.randn(shape, generator=g, device="cuda") * torch.exp(0.7 * torch.randn(shape[:2] + (1, 1), generator=g, device="cuda"))
    if not e4m3:
        return x.to(torch.bfloat16), None
    s = _pow2_scale(x.abs().amax((2, 3)))
    return _code(x / s[:, :, None, None]), s


def prepare(case, seed):
    c, g, dev = case, _gen(seed), "cuda"

    def normal(*shape, dtype=torch.bfloat16, by=1.0):
        return (torch.randn(shape, generator=g, device=dev) * by).to(dtype)

    if c["op"] in ("join", "join_bwd"):
        M, C = c["rows"], c["width"]
        rt, yt = (torch.float32 if c["r32"] else torch.bfloat16), (torch.float32 if c["y32"] else torch.bfloat16)
        s = dict(c=c, r=normal(M, C, dtype=rt, by=2.0), y=normal(M, C, dtype=yt, by=0.5),
                 w_pre=1 + 0.2 * normal(C, dtype=torch.float32),
                 w_post=1 + 0.2 * normal(C, dtype=torch.float32) if c["post"] else None,
                 gate=normal(M, C, dtype=yt) if c["gate"] else None,
                 alpha=0.5 + 0.1 * normal(C, dtype=torch.float32) if c["alpha"] else None)
        if c["op"] == "join_bwd":
            # r is the forward's residual sum here; a training step has the row statistics from its forward
            s["rstd_pre"] = torch.rsqrt(s["r"].float().square().mean(1) + EPS)
            s["rstd_post"] = torch.rsqrt(s["y"].float().square().mean(1) + EPS) if c["post"] else None
            s["dn"], s["dr"] = normal(M, C, dtype=yt), normal(M, C, dtype=rt)
        return s

    lens = _lens(c)
    P, Hq, Hkv, d = c["page"], c["heads_q"], c["heads_kv"], c["dim"]
    new, past = [n for n, _ in lens], [p for _, p in lens]
    T, kv = sum(new), [a + b for a, b in lens]
    width = -(-max(kv) // P)
    q_start = torch.tensor([0] + new, device=dev).cumsum(0).to(torch.int32)
    kv_len = torch.tensor(kv, device=dev, dtype=torch.int32)
    if c.get("table"):
        # only the pages that the call touches are held here, so a pool of long contexts stays small
        first = [p // P for p in past]
        need = [(l + P - 1) // P - f for l, f in zip(kv, first)]
    else:
        first, need = [0] * len(kv), [(l + P - 1) // P for l in kv]
    pages = sum(need) + sum(need) // 8 + 2
    perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32).cpu()
    table = torch.full((len(kv), width), -1, dtype=torch.int32)
    at = 0
    for b, (f, n) in enumerate(zip(first, need)):
        table[b, f:f + n] = perm[at:at + n]
        at += n
    k, ks = _cache((pages, Hkv, P, d), c["e4m3"], g)
    v, vs = _cache((pages, Hkv, P, d), c["e4m3"], g)
    s = dict(c=c, k=k, v=v, ks=ks, vs=vs, q_start=q_start, kv_len=kv_len, table=table.to(dev), T=T, max_q=max(new),
             max_kv=max(kv))
    if c["op"] == "append":
        # the projection's output: q, k and v are column ranges of one matrix
        qkv = normal(T, (Hq + 2 * Hkv) * d)
        s["q"] = qkv[:, :Hq * d].unflatten(1, (Hq, d))
        s["nk"] = qkv[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
        s["nv"] = qkv[:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d))
        R = c["rot"]
        s["freqs"] = 10000.0 ** (-torch.arange(0, R, 2, device=dev, dtype=torch.float64) / R) if R else None
    else:
        s["q"] = normal(T, Hq, d)
    if own:
        from hybrid_ssm_sliding_b200 import ops

        s["cache"] = ops.PagedKv(k, v, ks, vs)
        s["batch"] = ops.PagedBatch(q_start, kv_len, s["table"], max_q=s["max_q"], max_kv=s["max_kv"])
        if c["op"] == "attend":
            n = ops.paged_attn_workspace_size(s["batch"], s["cache"], Hq, c["window"])
            s["ws"] = torch.empty((max(n, 16),), dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------ the plain forms
def _rows(s):
    """Sequence and position of each row."""
    t = torch.arange(s["T"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["q_start"], t, right=True) - 1
    n = s["q_start"][1:] - s["q_start"][:-1]
    return seq, (s["kv_len"] - n)[seq].long() + (t - s["q_start"][seq]).long()


def _rotate(x, pos, freqs, inter):
    """x [T, H, d] in 32 bits, its first 2 len(freqs) elements of each head rotated by position."""
    if freqs is None:
        return x
    a = pos.double()[:, None] * freqs
    co, si = a.cos().float()[:, None], a.sin().float()[:, None]
    R = 2 * freqs.numel()
    p, q = (x[..., 0:R:2], x[..., 1:R:2]) if inter else (x[..., :R // 2], x[..., R // 2:R])
    u, w = p * co - q * si, q * co + p * si
    new = torch.stack((u, w), -1).flatten(-2) if inter else torch.cat((u, w), -1)
    return torch.cat((new, x[..., R:]), -1)


def _store(cache, scale, x, page, off, start):
    """Writes x [T, Hkv, d] (32 bits) to rows `off` of pages `page`; `start`: each row's first offset in its page."""
    if scale is None:
        cache[page, :, off] = x.to(cache.dtype)
        return
    amax = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(2), "amax")
    first = torch.full((scale.shape[0],), cache.shape[2], device="cuda", dtype=torch.long)
    first.index_reduce_(0, page, start, "amin")
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, page, True)
    old = torch.where((first > 0)[:, None], scale, torch.zeros_like(scale))
    now = torch.maximum(_pow2_scale(amax), old)
    t = touched.nonzero()[:, 0]
    before = torch.arange(cache.shape[2], device="cuda")[None, :] < first[t][:, None]
    was = cache[t]
    again = _code(was.float() * (old[t] / now[t])[:, :, None, None])
    keep = before[:, None, :, None]
    cache[t] = torch.where(keep, again.float(), was.float()).to(E4M3)
    cache[page, :, off] = _code(x / now[page][:, :, None])
    scale[t] = now[t]


def _append(s):
    c, P = s["c"], s["c"]["page"]
    seq, pos = _rows(s)
    q = _rotate(s["q"].float(), pos, s["freqs"], c["inter"]).to(torch.bfloat16)
    k = _rotate(s["nk"].float(), pos, s["freqs"], c["inter"])
    page, off = s["table"][seq, pos // P].long(), pos % P
    n = s["q_start"][1:] - s["q_start"][:-1]
    first = (s["kv_len"] - n)[seq].long()
    start = torch.where(pos // P == first // P, first % P, torch.zeros_like(first))
    _store(s["k"], s["ks"], k, page, off, start)
    _store(s["v"], s["vs"], s["nv"].float(), page, off, start)
    return q


def _attend(s):
    c, P, d, Hkv = s["c"], s["c"]["page"], s["c"]["dim"], s["c"]["heads_kv"]
    grp, B, W = c["heads_q"] // Hkv, c["seqs"], c["window"]
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    kv = s["kv_len"].long()
    low = (kv - n - W + 1).clamp(min=0) if W else torch.zeros_like(kv)
    np_ = min(s["table"].shape[1], -(-(W + s["max_q"]) // P) + 1) if W else s["table"].shape[1]
    col = (low // P)[:, None] + torch.arange(np_, device="cuda")
    ids = s["table"].gather(1, col.clamp(max=s["table"].shape[1] - 1)).clamp(min=0).long()

    def values(x, sc):
        x = x[ids].float()
        x = x if sc is None else x * sc[ids][..., None, None]
        return x.transpose(1, 2).reshape(B, Hkv, np_ * P, d)

    at = (col[:, :, None] * P + torch.arange(P, device="cuda")).reshape(B, np_ * P)
    i = torch.arange(s["max_q"], device="cuda")
    row = (s["q_start"][:-1].long()[:, None] + i).clamp(max=s["T"] - 1)
    q = s["q"][row].float().reshape(B, s["max_q"], Hkv, grp, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, grp * s["max_q"], d)
    pos = (kv - n)[:, None] + i
    see = (at[:, None, :] <= pos[:, :, None]) & (at < kv[:, None])[:, None, :]
    if W:
        see &= at[:, None, :] > pos[:, :, None] - W
    see = see[:, None, None]
    sc = (q @ values(s["k"], s["ks"]).transpose(2, 3)).reshape(B, Hkv, grp, s["max_q"], np_ * P) * d ** -0.5
    sc = sc.masked_fill(~see, -math.inf)
    p = torch.exp(sc - sc.amax(-1, keepdim=True).clamp(min=-3e38))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = p.reshape(B, Hkv, grp * s["max_q"], -1) @ values(s["v"], s["vs"])
    o = o.reshape(B, Hkv, grp, s["max_q"], d).permute(0, 3, 1, 2, 4).reshape(B, s["max_q"], Hkv * grp, d)
    return o[i[None, :] < n[:, None]].to(torch.bfloat16)


def _join(s):
    r, t = s["r"].float(), s["y"].float()
    if s["w_post"] is not None:
        t = t * torch.rsqrt(t.square().mean(1, keepdim=True) + EPS) * s["w_post"]
    if s["gate"] is not None:
        t = t / (1 + torch.exp(-s["gate"].float()))
    if s["alpha"] is not None:
        t = t * s["alpha"]
    r = r + t
    rstd = torch.rsqrt(r.square().mean(1, keepdim=True) + EPS)
    return r.to(s["r"].dtype), (r * rstd * s["w_pre"]).to(s["y"].dtype)


def _join_bwd(s):
    x = s["r"].float() * s["rstd_pre"][:, None]
    dn = s["dn"].float()
    out = {"dw_pre": (dn * x).sum(0)}
    dx = dn * s["w_pre"]
    g = s["dr"].float() + s["rstd_pre"][:, None] * (dx - x * (dx * x).mean(1, keepdim=True))
    out["dr"] = g.to(s["r"].dtype)
    yh = s["y"].float()
    t = yh
    if s["w_post"] is not None:
        yh = yh * s["rstd_post"][:, None]
        t = yh * s["w_post"]
    du = g if s["alpha"] is None else g * s["alpha"]
    dt = du
    if s["gate"] is not None:
        sg = 1 / (1 + torch.exp(-s["gate"].float()))
        out["dgate"] = (du * t * sg * (1 - sg)).to(s["y"].dtype)
        dt, t = du * sg, t * sg
    if s["alpha"] is not None:
        out["dalpha"] = (g * t).sum(0)
    if s["w_post"] is not None:
        out["dw_post"] = (dt * yh).sum(0)
        dt = dt * s["w_post"]
        dt = s["rstd_post"][:, None] * (dt - yh * (dt * yh).mean(1, keepdim=True))
    out["dy"] = dt.to(s["y"].dtype)
    return out


# -------------------------------------------------------------------- a pass
def run(state):
    s, op = state, state["c"]["op"]
    if own:
        from hybrid_ssm_sliding_b200 import ops

        if op == "append":
            q = ops.kv_append(s["q"], s["nk"], s["nv"], s["cache"], s["batch"], freqs=s["freqs"],
                              interleaved=s["c"]["inter"])
        elif op == "attend":
            return {"o": ops.paged_attn(s["q"], s["cache"], s["batch"], window=s["c"]["window"], workspace=s["ws"])}
        elif op == "join":
            r, n = ops.block_norm_fwd(s["r"], s["w_pre"], y=s["y"], w_post=s["w_post"], gate=s["gate"], alpha=s["alpha"],
                                      eps=EPS)
            return {"r": r, "n": n}
        else:
            out = ops.block_norm_bwd(s["dn"], s["r"], s["w_pre"], s["rstd_pre"], dr_out=s["dr"], y=s["y"],
                                     w_post=s["w_post"], rstd_post=s["rstd_post"], gate=s["gate"], alpha=s["alpha"])
            return {k: v for k, v in out.items() if v is not None}
    elif op == "append":
        q = _append(s)
    elif op == "attend":
        return {"o": _attend(s)}
    elif op == "join":
        return dict(zip(("r", "n"), _join(s)))
    else:
        return _join_bwd(s)
    out = {"q": q, "k": s["k"], "v": s["v"]}
    return out if s["ks"] is None else {**out, "k_scale": s["ks"], "v_scale": s["vs"]}


# ---------------------------------------------------------------- the floor
def work(case):
    c = case
    if c["op"] in ("join", "join_bwd"):
        n, C = c["rows"] * c["width"], c["width"]
        r, y = (4 if c["r32"] else 2), (4 if c["y32"] else 2)
        vec = 4 * C * (1 + c["post"] + c["alpha"])
        if c["op"] == "join":
            return {"bytes": n * (2 * r + 2 * y + (y if c["gate"] else 0)) + vec, "flops": 12 * n}
        stats = 4 * c["rows"] * (1 + c["post"])
        # read dn, dr, r, y (, gate); write dr, dy (, dgate)
        return {"bytes": n * (3 * r + 3 * y + (2 * y if c["gate"] else 0)) + 2 * vec + stats, "flops": 30 * n}
    lens, d, Hq, Hkv = _lens(c), c["dim"], c["heads_q"], c["heads_kv"]
    T, el = sum(n for n, _ in lens), (1 if c["e4m3"] else 2)
    if c["op"] == "append":
        return {"bytes": T * d * (4 * Hq + 4 * Hkv + 2 * el * Hkv), "flops": 4 * T * d * (Hq + Hkv)}
    W, keys, pairs = c["window"], 0, 0
    for n, p in lens:
        lo = max(0, p - W + 1) if W else 0
        keys += n + p - lo
        pairs += sum(min(W, p + i + 1) for i in range(n)) if W else n * p + n * (n + 1) // 2
    return {"bytes": 2 * el * keys * Hkv * d + 4 * T * Hq * d, "flops": 4 * d * Hq * pairs}


# ------------------------------------------------------- 64 bits, from the definitions
def _e4m3_64(x):
    """The nearest e4m3 value of each x (64 bits, ties to even), at most 448 in size."""
    a = x.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    e = torch.where(torch.exp2(e) > a.clamp(min=2.0 ** -6), e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= a.clamp(min=2.0 ** -6), e + 1, e)
    step = torch.exp2(e - 3)
    return torch.sign(x) * torch.round(a / step) * step


def _exact_append(s):
    c = s["c"]
    P, R = c["page"], c["rot"]
    start, kv, table = s["q_start"].tolist(), s["kv_len"].tolist(), s["table"].tolist()
    out = {"q": s["q"].double(), "k": s["k"].double(), "v": s["v"].double()}
    if s["ks"] is not None:
        out |= {"k_scale": s["ks"].double(), "v_scale": s["vs"].double()}
    nk = s["nk"].double()
    T = s["T"]
    pos = torch.zeros(T, dtype=torch.float64, device="cuda")
    for b, l in enumerate(kv):
        n = start[b + 1] - start[b]
        pos[start[b]:start[b + 1]] = torch.arange(l - n, l, device="cuda", dtype=torch.float64)
    for j in range(R // 2):
        a = pos * 10000.0 ** (-2.0 * j / R)
        lo, hi = (2 * j, 2 * j + 1) if c["inter"] else (j, j + R // 2)
        co, si = torch.cos(a)[:, None], torch.sin(a)[:, None]
        for x in (out["q"], nk):
            u, w = x[:, :, lo].clone(), x[:, :, hi].clone()
            x[:, :, lo], x[:, :, hi] = u * co - w * si, u * si + w * co
    for name, x in (("k", nk), ("v", s["nv"].double())):
        cache, scale = out[name], out.get(name + "_scale")
        for b, l in enumerate(kv):
            p0, t0 = l - (start[b + 1] - start[b]), start[b]
            at = p0
            while at < l:
                end = min(l, (at // P + 1) * P)
                pg, o = table[b][at // P], at % P
                rows = x[t0 + at - p0:t0 + end - p0].transpose(0, 1)  # [Hkv, rows, d]
                if scale is None:
                    cache[pg, :, o:o + end - at] = rows
                else:
                    big = rows.abs().amax((1, 2))
                    k = torch.ceil(torch.log2((big / 448.0).clamp(2.0 ** -60, 2.0 ** 30)))
                    now = torch.exp2(k)
                    if o:
                        now = torch.maximum(now, scale[pg])
                        by = (scale[pg] / now)[:, None, None]
                        cache[pg, :, :o] = _e4m3_64(cache[pg, :, :o] * by)
                    cache[pg, :, o:o + end - at] = _e4m3_64(rows / now[:, None, None])
                    scale[pg] = now
                at = end
    return out


def _exact_attend(s):
    c = s["c"]
    P, d, Hkv, W = c["page"], c["dim"], c["heads_kv"], c["window"]
    grp = c["heads_q"] // Hkv
    start, kv = s["q_start"].tolist(), s["kv_len"].tolist()
    o = torch.zeros(s["T"], c["heads_q"], d, dtype=torch.float64, device="cuda")
    for b, l in enumerate(kv):
        n = start[b + 1] - start[b]
        lo = max(0, l - n - W + 1) if W else 0
        ids = s["table"][b, lo // P:-(-l // P)].long()

        def values(x, sc):
            x = x[ids].double()
            x = x if sc is None else x * sc[ids].double()[:, :, None, None]
            return x.transpose(0, 1).reshape(Hkv, -1, d)[:, lo % P:lo % P + l - lo]

        k, v = values(s["k"], s["ks"]), values(s["v"], s["vs"])
        key = torch.arange(lo, l, device="cuda")
        pos = torch.arange(l - n, l, device="cuda")
        hide = key[None] > pos[:, None]
        if W:
            hide |= key[None] + W <= pos[:, None]
        for h in range(c["heads_q"]):
            q = s["q"][start[b]:start[b + 1], h].double()
            a = (q @ k[h // grp].T / math.sqrt(d)).masked_fill(hide, -math.inf)
            o[start[b]:start[b + 1], h] = torch.softmax(a, 1) @ v[h // grp]
    return {"o": o}


def _exact_join(s, grad):
    f = lambda k: None if s.get(k) is None else s[k].double()  # noqa: E731
    r, y, gate, alpha, wp, wq = f("r"), f("y"), f("gate"), f("alpha"), f("w_post"), f("w_pre")
    sig = 1.0 if gate is None else torch.special.expit(gate)
    al = 1.0 if alpha is None else alpha
    if not grad:
        t = y if wp is None else wp * y / torch.sqrt((y * y).mean(1, keepdim=True) + EPS)
        r = r + al * sig * t
        return {"r": r, "n": wq * r / torch.sqrt((r * r).mean(1, keepdim=True) + EPS)}
    C = r.shape[1]
    a, dn = f("rstd_pre")[:, None], f("dn")
    proj = (dn * wq * r).sum(1, keepdim=True) / C
    g = f("dr") + a * dn * wq - a ** 3 * r * proj
    out = {"dr": g, "dw_pre": (a * r * dn).sum(0)}
    if wp is None:
        t, dt = y, al * sig * g
        out["dy"] = dt
    else:
        e = f("rstd_post")[:, None]
        t, dt = y * e * wp, al * sig * g
        out["dw_post"] = (dt * y * e).sum(0)
        out["dy"] = e * dt * wp - e ** 3 * y * (dt * wp * y).sum(1, keepdim=True) / C
    if gate is not None:
        out["dgate"] = al * g * t * sig * (1 - sig)
    if alpha is not None:
        out["dalpha"] = (g * sig * t).sum(0)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return _exact_append(s) if op == "append" else _exact_attend(s) if op == "attend" else _exact_join(s, op == "join_bwd")
