"""Runs the paged cache's, the paged attention's and the block norm's calls and
saves their outputs (a helper of tests/test_debug_paged.py, run in a child
process so that the library can be chosen with SAMBA_LIBRARY).

    python tests/_debug_paged_cases.py OUT.npz"""

import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from hybrid_ssm_sliding_b200 import ops  # noqa: E402
from tests._paged import Case  # noqa: E402


def main(path):
    out = {}
    freqs = 10000.0 ** (-torch.arange(0, 32, 2, dtype=torch.float64, device="cuda") / 32)
    for e4m3 in (False, True):
        for i, (new, past, d, P) in enumerate((([1, 1, 0], [900, 40, 3], 64, 16), ([300, 1, 77], [0, 500, 130], 64, 64),
                                               ([130], [1500], 128, 32), ([2, 3], [70, 1200], 32, 256))):
            c = Case(new, past, 8, 2, d, P, e4m3, seed=90 + i, pad=1)
            cache, batch = c.gpu()
            key = f"{i}{'e' if e4m3 else 'b'}_"
            q = torch.zeros(c.q.shape, dtype=torch.bfloat16, device="cuda")
            ops.kv_append(c.q.cuda(), c.k.cuda(), c.v.cuda(), cache, batch, freqs=freqs, q_out=q)
            out[key + "q"], out[key + "k"] = q, cache.k.float()
            for window in (0, 50):
                out[key + f"o{window}"] = ops.paged_attn(q, cache, batch, window=window, o=torch.zeros_like(q))
            if ops.get_status() != 0:
                raise SystemExit(f"{key}: status set")
    g = torch.Generator(device="cuda").manual_seed(1)
    for rows, C in ((5, 264), (3000, 2048), (700, 8192)):
        r = torch.randn((rows, C), generator=g, device="cuda")
        y, gate = (torch.randn((rows, C), generator=g, device="cuda").bfloat16() for _ in range(2))
        w = torch.rand((C,), generator=g, device="cuda") + 0.5
        rs, rsy = (torch.empty((rows,), device="cuda") for _ in range(2))
        r1, n = ops.block_norm_fwd(r, w, y=y, w_post=w, gate=gate, alpha=w, rstd_pre=rs, rstd_post=rsy)
        grads = ops.block_norm_bwd(n, r1, w, rs, dr_out=r, y=y, w_post=w, rstd_post=rsy, gate=gate, alpha=w)
        out |= {f"norm{C}_{k}": v for k, v in {"r": r1, "n": n, **grads}.items()}
        if ops.get_status() != 0:
            raise SystemExit(f"norm {rows} x {C}: status set")
    np.savez(path, **{k: v.detach().float().cpu().numpy() for k, v in out.items()})


if __name__ == "__main__":
    main(sys.argv[1])
