"""The paged cache's kernels where a warp, a tile or a call is not of one piece:
row tiles that end inside a warp, products that share tensor memory, values
that are not finite, weights far below the largest, batches out of order.
Tolerances as in test_paged.py; what a test adds to them stands at the test."""

import pytest
import torch

from hybrid_ssm_sliding_b200 import _lib as L
from hybrid_ssm_sliding_b200 import build as B
from hybrid_ssm_sliding_b200 import ops
from tests._paged import Case
from tests.test_paged import check_attn, run_attn

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
