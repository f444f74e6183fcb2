"""The debug build (every global output store's index checked on the device)
runs the paged and block norm calls with no check firing, and gives the
release build's results but for roundings."""

import os
import subprocess
import sys

import numpy as np
import pytest

from hybrid_ssm_sliding_b200 import build as B

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _run(tmp_path, which):
    out = str(tmp_path / f"{which}.npz")
    env = dict(os.environ)
    env.pop("SAMBA_LIBRARY", None)
    if which == "debug":
        env["SAMBA_LIBRARY"] = "debug"
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "_debug_paged_cases.py"), out], env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, f"{which} build: {r.stdout[-2000:]}{r.stderr[-4000:]}"
    return np.load(out)


def test_debug_build_runs_clean_and_matches_release(tmp_path):
    B.build()
    B.build(debug=True)
    rel, dbg = _run(tmp_path, "release"), _run(tmp_path, "debug")
    assert set(rel.files) == set(dbg.files)
    for k in rel.files:
        # contraction of products and sums may differ between the builds: a bf16 step at most
        scale = float(np.max(np.abs(np.nan_to_num(rel[k])))) or 1.0
        assert np.array_equal(np.isnan(rel[k]), np.isnan(dbg[k])), k
        assert float(np.max(np.abs(np.nan_to_num(rel[k]) - np.nan_to_num(dbg[k])))) <= 2.0 ** -7 * scale, k
