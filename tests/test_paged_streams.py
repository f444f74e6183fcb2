"""Calls on a stream that is not the current one: what they allocate on the way is not handed out
before that stream is done with it, nor taken from memory that the current
stream is still to write.  Results are compared bit for bit with the same call
on the current stream."""

import pytest
import torch

from hybrid_ssm_sliding_b200 import _lib as L
from hybrid_ssm_sliding_b200 import build as B
from hybrid_ssm_sliding_b200 import layers, ops
from tests._paged import Case
from tests.test_paged import make_freqs
from tests.test_paged_stack import make_blocks

pytestmark = pytest.mark.gpu

T, HQ, HKV, D, P, DM = 300, 8, 2, 64, 32, 256  # heads and widths of make_blocks
CLOCKS = 20_000_000                            # about ten milliseconds


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


def _scribble(n=48):
    """Takes the current stream's free memory in pieces of every size used here and fills it."""
    held = []
    for size in (T * DM * 2, T * DM * 4, T * HQ * D * 2, T * (HQ + 2 * HKV) * D * 2, 4096, 1 << 22):
        held += [torch.full((size,), 0xff, dtype=torch.uint8, device="cuda") for _ in range(n)]
    return held


def _stack():
    blocks, w_final = make_blocks(2, seed=3)
    r = torch.randn((T, DM), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    c = Case([T], [0], HQ, HKV, D, P, False, seed=5)
    fr = make_freqs(D).cuda()
    batch = c.gpu()[1]
    ws = torch.empty((1 << 22,), dtype=torch.uint8, device="cuda")

    def run(stream=None):
        caches = [ops.PagedKv.empty(c.pages, HKV, P, D) for _ in blocks]
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        out = layers.paged_stack(r, blocks, w_final, caches, batch, freqs=fr, workspace=ws, stream=stream)
        return (*out, *[x.k for x in caches], *[x.v for x in caches])
    return run


def _ops():
    c = Case([1, T - 1], [3000, 40], HQ, HKV, D, P, True, seed=6)
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    fr = make_freqs(D).cuda()
    n = lambda *s: torch.randn(s, generator=torch.Generator(device="cuda").manual_seed(7), device="cuda")  # noqa: E731
    r, y, w, al = n(T, DM), n(T, DM).bfloat16(), n(DM), n(DM) + 1

    pool, batch = c.gpu()

    def run(stream=None):
        cache = ops.PagedKv(*[t.clone() for t in (pool.k, pool.v, pool.k_scale, pool.v_scale)])
        rs, rsy = torch.empty((T,), device="cuda"), torch.empty((T,), device="cuda")
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        qr = ops.kv_append(q, k, v, cache, batch, freqs=fr, stream=stream)
        o = ops.paged_attn(qr, cache, batch, stream=stream)
        r1, n1 = ops.block_norm_fwd(r, w, y=y, w_post=w, gate=y, alpha=al, rstd_pre=rs, rstd_post=rsy, stream=stream)
        g = ops.block_norm_bwd(n1, r1, w, rs, dr_out=r1, y=y, w_post=w, rstd_post=rsy, gate=y, alpha=al, stream=stream)
        return (qr, o, cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale, r1, n1, rs, rsy,
                *g.values())  # (the inputs too: the caller keeps them)
    return run


@pytest.mark.parametrize("make", [_stack, _ops], ids=["stack", "ops"])
def test_memory_of_a_call_is_kept_until_its_stream_is_done(make):
    run = make()
    want = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(CLOCKS)       # the call's kernels come after this
        got = run(side)
        held = _scribble()                  # before them, on the current stream
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del held, got
    assert ops.get_status() == L.SAMBA_OK


@pytest.mark.parametrize("make", [_stack, _ops], ids=["stack", "ops"])
def test_memory_that_the_current_stream_is_to_write_is_not_taken(make):
    run = make()
    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    plain = side.wait_stream

    def wait_then_scribble(other):
        plain(other)                        # the call's inputs are there
        torch.cuda._sleep(CLOCKS)           # then the current stream has more to do: writes
        _scribble()                         # to memory that it has given back by the time of the call

    side.wait_stream = wait_then_scribble
    got = run(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert ops.get_status() == L.SAMBA_OK


@pytest.mark.parametrize("make", [_stack, _ops], ids=["stack", "ops"])
def test_outputs_freed_by_the_caller_are_not_reused_under_it(make):
    """The caller's stream still reads the outputs when it lets them go; the next
    call on the side stream must not write there."""
    run = make()
    want = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    got = run(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(CLOCKS)
    read = [t.clone() for t in got]
    del got
    with torch.cuda.stream(side):
        held = _scribble()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(read, want))
    del held


@pytest.mark.parametrize("make", [_stack, _ops], ids=["stack", "ops"])
def test_a_call_on_a_stream_that_joins_a_capture(make):
    """Captured on one stream, called on another that was forked from it."""
    run = make()
    want = [t.clone() for t in run()]
    first, side = torch.cuda.Stream(), torch.cuda.Stream()
    run(side)                               # what a first call loads is loaded
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(first), torch.cuda.graph(graph, stream=first):
        got = run(side)
        first.wait_stream(side)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert ops.get_status() == L.SAMBA_OK
    same = [torch.equal(a, b) for a, b in zip(got, want)]
    assert all(same), same
