"""The block norm (samba_block_norm_fwd / _bwd): the 64-bit formulas against
differences (CPU), and the kernels against the formulas (GPU).

Tolerances.  Every output is rounded once: half a step is 2^-8 of a bf16
value.  In fp32 a row's sum of up to 8192 terms goes through 8 additions a
thread and two trees (under 2^-20), the reciprocal root, exponential and fast
quotient add a few 2^-22 (the exponential of |x| < 16 under 2^-20), so an
output's terms carry below 2^-17 of their sizes.  Column sums add each
block's rows in turn, below 256 here, and the blocks: below 2^-16 of the sum
of their terms' sizes."""

import pytest
import torch

from hybrid_ssm_sliding_b200 import _lib as L
from hybrid_ssm_sliding_b200 import build as B
from hybrid_ssm_sliding_b200 import ops

EPS = 1e-6
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def fwd64(r, y=None, w_pre=None, w_post=None, gate=None, alpha=None):
    """(r', n, rstd_pre, rstd_post, |r| + |added term|) in 64 bits."""
    d = lambda t: None if t is None else t.double()  # noqa: E731
    r, y, w_pre, w_post, gate, alpha = map(d, (r, y, w_pre, w_post, gate, alpha))
    rsy, mag = None, r.abs()
    if y is not None:
        u = y
        if w_post is not None:
            rsy = 1 / torch.sqrt((y * y).mean(1) + EPS)
            u = u * rsy[:, None] * w_post
        if gate is not None:
            u = u * torch.special.expit(gate)
        if alpha is not None:
            u = u * alpha
        mag = mag + u.abs()
        r = r + u
    rs = 1 / torch.sqrt((r * r).mean(1) + EPS)
    return r, None if w_pre is None else r * rs[:, None] * w_pre, rs, rsy, mag


def bwd64(dn, r, w_pre, rs, dr_out, y, w_post, rsy, gate, alpha):
    """The gradients in 64 bits, and the sizes their rounding errors scale with."""
    d = lambda t: None if t is None else t.double()  # noqa: E731
    dn, r, w_pre, rs, dr_out, y, w_post, rsy, gate, alpha = map(d, (dn, r, w_pre, rs, dr_out, y, w_post, rsy, gate, alpha))
    out, mag = {}, {}
    g, gm = torch.zeros_like(r), torch.zeros_like(r)
    if dr_out is not None:
        g, gm = dr_out, dr_out.abs()
    if dn is not None:
        x, a = r * rs[:, None], rs[:, None]
        t = dn * w_pre
        g = g + a * (t - x * (t * x).mean(1, keepdim=True))
        gm = gm + a * (t.abs() + x.abs() * (t * x).abs().mean(1, keepdim=True))
        out["dw_pre"], mag["dw_pre"] = (dn * x).sum(0), (dn * x).abs().sum(0)
    out["dr"], mag["dr"] = g, gm
    if y is not None:
        b = torch.ones_like(r[:, :1]) if w_post is None else rsy[:, None]
        yh = y * b
        w = 1.0 if w_post is None else w_post
        s = torch.ones_like(r) if gate is None else torch.special.expit(gate)
        al = 1.0 if alpha is None else alpha
        t = yh * w
        dt, dtm = al * g * s, abs(al) * gm * s if isinstance(al, float) else al.abs() * gm * s
        if gate is not None:
            out["dgate"], mag["dgate"] = dt * t * (1 - s), dtm * t.abs()
        if alpha is not None:
            out["dalpha"], mag["dalpha"] = (g * s * t).sum(0), (gm * s * t.abs()).sum(0)
        if w_post is not None:
            out["dw_post"], mag["dw_post"] = (dt * yh).sum(0), (dtm * yh.abs()).sum(0)
            p, pm = dt * w, dtm * w.abs()
            out["dy"] = b * (p - yh * (p * yh).mean(1, keepdim=True))
            mag["dy"] = b * (pm + yh.abs() * (pm * yh.abs()).mean(1, keepdim=True))
        else:
            out["dy"], mag["dy"] = dt, dtm
    return out, mag


def make(rows, C, rt, yt, post, gate, alpha, seed, device="cpu"):
    g = torch.Generator().manual_seed(seed)

    def n(*shape, dtype=torch.float32, by=1.0, plus=0.0):
        return (torch.randn(shape, generator=g) * by + plus).to(dtype).to(device)

    return dict(r=n(rows, C, dtype=rt, by=2.0), y=n(rows, C, dtype=yt, by=0.5), w_pre=n(C, by=0.2, plus=1.0),
                w_post=n(C, by=0.2, plus=1.0) if post else None, gate=n(rows, C, dtype=yt, by=2.0) if gate else None,
                alpha=n(C, by=0.1, plus=0.5) if alpha else None)


@pytest.mark.parametrize("post,gate,alpha", [(False, False, False), (True, True, True), (True, False, True), (False, True, False)])
def test_formulas_match_differences(post, gate, alpha):
    """d(sum dn n + dr' r') along a random direction of every input, central
    differences in 64 bits: error about h^2 = 1e-10 of the third derivative
    and 1e-16 / h = 1e-11, against 1e-7 allowed."""
    p = {k: None if v is None else v.double() for k, v in
         make(3, 16, torch.float64, torch.float64, post, gate, alpha, seed=1).items()}
    g = torch.Generator().manual_seed(2)
    dn, dr = (torch.randn((3, 16), generator=g, dtype=torch.float64) for _ in range(2))

    def loss(q):
        r, n, *_ = fwd64(q["r"], q["y"], q["w_pre"], q["w_post"], q["gate"], q["alpha"])
        return float((dn * n).sum() + (dr * r).sum())

    r1, _, rs, rsy, _ = fwd64(p["r"], p["y"], p["w_pre"], p["w_post"], p["gate"], p["alpha"])
    out, _ = bwd64(dn, r1, p["w_pre"], rs, dr, p["y"], p["w_post"], rsy, p["gate"], p["alpha"])
    for key, grad in (("r", "dr"), ("y", "dy"), ("w_pre", "dw_pre"), ("w_post", "dw_post"), ("gate", "dgate"), ("alpha", "dalpha")):
        if p[key] is None:
            continue
        v = torch.randn(p[key].shape, generator=g, dtype=torch.float64)
        h = 1e-5
        up, down = dict(p), dict(p)
        up[key], down[key] = p[key] + h * v, p[key] - h * v
        want = (loss(up) - loss(down)) / (2 * h)
        assert abs(float((out[grad] * v).sum()) - want) <= 1e-7 * max(1.0, abs(want)), key


F32, BF16 = torch.float32, torch.bfloat16
SHAPES = [  # rows, width, r, y, post, gate, alpha
    (1, 8, BF16, BF16, True, True, True),
    (5, 264, F32, BF16, True, False, True),
    (4000, 256, BF16, BF16, False, True, False),
    (16, 2048, BF16, BF16, True, True, True),
    (2049, 2048, F32, BF16, True, True, True),
    (1300, 1000, F32, F32, True, True, False),
    (777, 4096, BF16, F32, False, False, False),
    (700, 4104, BF16, BF16, True, True, True),
    (333, 8192, F32, F32, True, True, True),
    (3000, 64, F32, BF16, False, False, True),
]


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def gpu(p):
    return {k: None if v is None else v.cuda() for k, v in p.items()}


@pytest.mark.gpu
@pytest.mark.parametrize("case", SHAPES, ids=lambda c: f"{c[0]}x{c[1]}")
def test_forward_matches_the_formula(lib, case):
    rows, C = case[:2]
    p = gpu(make(*case, seed=rows + C))
    rp, rq = torch.full((rows,), 7.0, device="cuda"), torch.full((rows,), 7.0, device="cuda")
    r, n = ops.block_norm_fwd(p["r"], p["w_pre"], y=p["y"], w_post=p["w_post"], gate=p["gate"], alpha=p["alpha"],
                              rstd_pre=rp, rstd_post=rq if case[4] else None)
    assert ops.get_status() == L.SAMBA_OK
    wr, wn, rs, rsy, mag = fwd64(p["r"], p["y"], p["w_pre"], p["w_post"], p["gate"], p["alpha"])
    assert float(((r.double() - wr).abs() - HALF[r.dtype] * wr.abs() - 2.0 ** -17 * mag).max()) <= 0
    nm = mag * rs[:, None] * p["w_pre"].double().abs()
    assert float(((n.double() - wn).abs() - HALF[n.dtype] * wn.abs() - 2.0 ** -16 * nm).max()) <= 0
    # the sums of squares move by twice their terms' error
    cond = (mag * mag).mean(1) * rs * rs
    assert float(((rp.double() - rs).abs() - 2.0 ** -16 * rs * cond).max()) <= 0
    if case[4]:
        assert float(((rq.double() - rsy).abs() - 2.0 ** -17 * rsy).max()) <= 0


@pytest.mark.gpu
@pytest.mark.parametrize("parts", ["both", "dn", "dr"])
@pytest.mark.parametrize("case", SHAPES, ids=lambda c: f"{c[0]}x{c[1]}")
def test_backward_matches_the_formula(lib, case, parts):
    rows, C, rt, yt = case[:4]
    p = gpu(make(*case, seed=rows + C + 1))
    g = torch.Generator().manual_seed(rows)
    dn = torch.randn((rows, C), generator=g).to(yt).cuda() if parts != "dr" else None
    dr = torch.randn((rows, C), generator=g).to(rt).cuda() if parts != "dn" else None
    rs = torch.rsqrt(p["r"].float().square().mean(1) + EPS)
    rsy = torch.rsqrt(p["y"].float().square().mean(1) + EPS) if case[4] else None
    out = ops.block_norm_bwd(dn, p["r"], p["w_pre"], rs, dr_out=dr, y=p["y"], w_post=p["w_post"], rstd_post=rsy,
                             gate=p["gate"], alpha=p["alpha"])
    assert ops.get_status() == L.SAMBA_OK
    want, mag = bwd64(dn, p["r"], p["w_pre"], rs, dr, p["y"], p["w_post"], rsy, p["gate"], p["alpha"])
    assert {k for k, v in out.items() if v is not None} == set(want)
    for k, w in want.items():
        col = w.dim() == 1
        tol = (2.0 ** -16 if col else 2.0 ** -17) * mag[k] + (0 if col else HALF[out[k].dtype]) * w.abs()
        err = (out[k].double() - w).abs()
        assert float((err - tol).max()) <= 0, (k, float((err / mag[k].clamp(min=1e-30)).max()))
    again = ops.block_norm_bwd(dn, p["r"], p["w_pre"], rs, dr_out=dr, y=p["y"], w_post=p["w_post"], rstd_post=rsy,
                               gate=p["gate"], alpha=p["alpha"])
    assert all(torch.equal(out[k], again[k]) for k in want)  # the sums' order is fixed


@pytest.mark.gpu
def test_the_norm_before_the_first_block(lib):
    p = gpu(make(300, 512, BF16, BF16, False, False, False, seed=3))
    rs = torch.empty((300,), device="cuda")
    r, n = ops.block_norm_fwd(p["r"].view(3, 100, 512), p["w_pre"], n_dtype=F32, rstd_pre=rs)
    assert r.data_ptr() == p["r"].data_ptr() and n.dtype == F32 and n.shape == (3, 100, 512)
    _, wn, ws, _, _ = fwd64(p["r"], w_pre=p["w_pre"])
    assert float(((n.double().view(300, 512) - wn).abs() - 2.0 ** -17 * wn.abs()).max()) <= 0
    dn = torch.ones((300, 512), device="cuda")
    out = ops.block_norm_bwd(dn, p["r"], p["w_pre"], rs)
    want, mag = bwd64(dn, p["r"], p["w_pre"], rs, None, None, None, None, None, None)
    assert out["dy"] is None and out["dalpha"] is None
    assert float(((out["dr"].double() - want["dr"]).abs() - HALF[BF16] * want["dr"].abs() - 2.0 ** -17 * mag["dr"]).max()) <= 0
    r2, n2 = ops.block_norm_fwd(p["r"], y=p["y"])  # the sum alone
    assert n2 is None
    assert torch.equal(r2, (p["r"].float() + p["y"].float()).to(BF16))


@pytest.mark.gpu
def test_extreme_rows_and_gates(lib):
    """Rows of zeros, of large and of tiny values, gates far out, NaN in one row."""
    p = gpu(make(6, 128, F32, BF16, True, True, True, seed=4))
    p["y"][0] = 0
    p["r"][1], p["y"][1] = 0, 0
    p["y"][2] *= 1e15
    p["y"][3] *= 1e-15
    p["gate"][4, ::2], p["gate"][4, 1::2] = 1000.0, -1000.0
    p["y"][5, 7] = float("nan")
    rs, rsy = torch.empty((6,), device="cuda"), torch.empty((6,), device="cuda")
    r, n = ops.block_norm_fwd(p["r"], p["w_pre"], y=p["y"], w_post=p["w_post"], gate=p["gate"], alpha=p["alpha"],
                              rstd_pre=rs, rstd_post=rsy)
    wr, wn, ws, wsy, mag = fwd64(p["r"], p["y"], p["w_pre"], p["w_post"], p["gate"], p["alpha"])
    assert float((r[:5].double() - wr[:5]).abs().max()) <= 2.0 ** -17 * float(mag[:5].max())
    assert float(((n[:5].double() - wn[:5]).abs() - 2.0 ** -8 * wn[:5].abs() - 2.0 ** -16).max()) <= 0
    assert float(n[1].float().abs().max()) == 0 and torch.isnan(n[5]).all()
    out = ops.block_norm_bwd(torch.ones_like(n), r, p["w_pre"], rs, y=p["y"], w_post=p["w_post"], rstd_post=rsy,
                             gate=p["gate"], alpha=p["alpha"])
    assert all(torch.isfinite(out[k][:5].float()).all() for k in ("dr", "dy", "dgate"))
    assert torch.isnan(out["dy"][5]).all()


@pytest.mark.gpu
def test_in_place_residual_and_zero_rows(lib):
    p = gpu(make(500, 1024, F32, BF16, True, False, True, seed=5))
    want, n = ops.block_norm_fwd(p["r"], p["w_pre"], y=p["y"], w_post=p["w_post"], alpha=p["alpha"])
    r = p["r"].clone()
    got, n2 = ops.block_norm_fwd(r, p["w_pre"], y=p["y"], w_post=p["w_post"], alpha=p["alpha"], r_out=r)
    assert got.data_ptr() == r.data_ptr() and torch.equal(r, want) and torch.equal(n, n2)
    e = torch.empty((0, 64), device="cuda")
    w = torch.ones((64,), device="cuda")
    r0, n0 = ops.block_norm_fwd(e, w, y=e.bfloat16())
    assert r0.shape == n0.shape == (0, 64)
    out = ops.block_norm_bwd(n0, r0, w, torch.empty((0,), device="cuda"), y=e.bfloat16(), alpha=w)
    assert float(out["dw_pre"].abs().max()) == 0 and float(out["dalpha"].abs().max()) == 0


@pytest.mark.gpu
def test_captured_replayed_and_on_two_streams(lib):
    ps = [gpu(make(900 + 300 * i, 2048, F32, BF16, True, True, True, seed=6 + i)) for i in range(2)]

    def both(p, stream=None):
        m = p["r"].shape[0]
        rs, rsy = torch.empty((m,), device="cuda"), torch.empty((m,), device="cuda")
        r, n = ops.block_norm_fwd(p["r"], p["w_pre"], y=p["y"], w_post=p["w_post"], gate=p["gate"], alpha=p["alpha"],
                                  rstd_pre=rs, rstd_post=rsy, stream=stream)
        out = ops.block_norm_bwd(n, r, p["w_pre"], rs, dr_out=r, y=p["y"], w_post=p["w_post"], rstd_post=rsy,
                                 gate=p["gate"], alpha=p["alpha"], stream=stream)
        return {"r": r, "n": n, **out}

    want = [both(p) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = []
    for s, p in zip(streams, ps):
        with torch.cuda.stream(s):
            got.append(both(p))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(a[k], b[k]) for k in a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both(ps[0])
    ps[0]["y"].mul_(2.0)
    ps[0]["gate"].neg_()
    graph.replay()
    torch.cuda.synchronize()
    fresh = both(ps[0])
    assert all(torch.equal(held[k], fresh[k]) for k in fresh)
    assert ops.get_status() == L.SAMBA_OK


@pytest.mark.gpu
def test_refusals(lib):
    p = gpu(make(4, 64, F32, BF16, True, True, True, seed=8))
    r, w = p["r"], p["w_pre"]
    with pytest.raises(TypeError):
        ops.block_norm_fwd(r.double(), w)
    with pytest.raises(ValueError):
        ops.block_norm_fwd(r.t(), w)
    with pytest.raises(TypeError):
        ops.block_norm_fwd(r, w.bfloat16())
    with pytest.raises(ValueError):
        ops.block_norm_fwd(r, w, y=p["y"][:2])
    with pytest.raises(TypeError):
        ops.block_norm_fwd(r, w, y=p["y"], gate=p["gate"].float())
    with pytest.raises(L.SambaError):
        ops.block_norm_fwd(r, w, alpha=p["alpha"])          # no y
    with pytest.raises(L.SambaError):
        ops.block_norm_fwd(r[:, :4].contiguous(), w[:4].contiguous())
    with pytest.raises(ValueError):
        ops.block_norm_fwd(r.cpu(), w)
    rs = torch.ones((4,), device="cuda")
    with pytest.raises(ValueError):
        ops.block_norm_bwd(None, r, w, rs)
    with pytest.raises(ValueError):
        ops.block_norm_bwd(p["y"], r, w, rs, y=p["y"], w_post=w)
    with pytest.raises(ValueError):
        ops.block_norm_bwd(p["y"], r, w, rs[:3])
    with pytest.raises(L.SambaError) as e:
        ops.block_norm_bwd(p["y"], r, w, rs, workspace=torch.empty((32,), dtype=torch.uint8, device="cuda"))
    assert e.value.code == L.SAMBA_ERR_WORKSPACE
