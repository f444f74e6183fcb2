"""CPU checks of the paged cache's and the block norm's C entry points: bad
arguments are refused on the host, before any launch."""

import ctypes

import pytest

from hybrid_ssm_sliding_b200 import _lib as L
from hybrid_ssm_sliding_b200 import build as B

F = 0x90000  # a 16-byte aligned dummy address; never followed on refused calls
INV, UNS, WSP = L.SAMBA_ERR_INVALID_ARG, L.SAMBA_ERR_UNSUPPORTED, L.SAMBA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def _set(a, over):
    for k, v in over.items():
        o, *rest = k.split("__")
        if rest:
            setattr(getattr(a, o), rest[0], v)
        else:
            setattr(a, o, v)
    return a


def _paged(a):
    a.kv.k = a.kv.v = F
    a.kv.num_pages, a.kv.page_size, a.kv.heads_kv, a.kv.head_dim, a.kv.dtype = 10, 16, 2, 64, L.SAMBA_BF16
    a.batch.q_start = a.batch.kv_len = a.batch.block_table = F
    a.batch.batch, a.batch.rows, a.batch.max_pages, a.batch.max_q, a.batch.max_kv = 3, 5, 4, 2, 64
    return a


PAGED = [
    (dict(kv__k=None), INV), (dict(kv__v=F + 8), INV), (dict(kv__num_pages=0), INV), (dict(kv__page_size=48), UNS),
    (dict(kv__head_dim=80), UNS), (dict(kv__dtype=0), UNS), (dict(kv__dtype=2), INV),
    (dict(kv__k_scale=F, kv__v_scale=F), INV), (dict(kv__num_pages=2 ** 30), UNS), (dict(kv__heads_kv=0), INV),
    (dict(batch__batch=70000), UNS), (dict(batch__rows=-1), INV), (dict(batch__rows=2 ** 30), UNS),
    (dict(batch__max_kv=2 ** 30), UNS), (dict(batch__q_start=None), INV), (dict(batch__block_table=None), INV),
]


def _append():
    a = _paged(L.KvAppendArgs())
    a.q = a.k = a.v = a.freqs = F
    a.q_out = F + 16
    a.ldq, a.ldk, a.ldv, a.heads_q, a.rot_dim = 8 * 64, 128, 128, 8, 64
    return a


@pytest.mark.parametrize("over,code", PAGED + [
    (dict(k=None), INV), (dict(v=F + 4), INV), (dict(q=None), INV), (dict(q_out=None), INV), (dict(heads_q=0), INV),
    (dict(ldq=500), INV), (dict(ldk=132), INV), (dict(ldv=64), INV), (dict(rot_dim=24), INV), (dict(rot_dim=80), INV),
    (dict(rot_dim=0), INV), (dict(freqs=None), INV), (dict(q_out=F, ldq=1024), INV),
])
def test_append_refuses(lib, over, code):
    assert lib.samba_kv_append(ctypes.byref(_set(_append(), over)), None) == code
    assert lib.samba_last_error().decode().startswith("samba_kv_append")


def _attn():
    a = _paged(L.PagedAttnArgs())
    a.q = a.o = F
    a.heads_q, a.window = 8, 0
    return a


@pytest.mark.parametrize("over,code", PAGED + [
    (dict(q=None), INV), (dict(o=None), INV), (dict(o=F + 8), INV), (dict(heads_q=7), INV), (dict(heads_q=34), UNS),
    (dict(window=-1), INV), (dict(window=2 ** 30), UNS), (dict(workspace=F + 4, workspace_bytes=1 << 30), INV),
    (dict(batch__max_q=2 ** 29), UNS),
])
def test_attention_refuses(lib, over, code):
    assert lib.samba_paged_attn(ctypes.byref(_set(_attn(), over)), None) == code
    assert lib.samba_last_error().decode().startswith("samba_paged_attn")


def test_attention_refuses_a_short_workspace(lib):
    a = _set(_attn(), dict(batch__max_kv=100000, batch__max_pages=7000, batch__max_q=1))
    need = lib.samba_paged_attn_workspace_size(ctypes.byref(a))
    assert need > 0
    assert lib.samba_paged_attn(ctypes.byref(a), None) == WSP
    a.workspace, a.workspace_bytes = F, need - 1
    assert lib.samba_paged_attn(ctypes.byref(a), None) == WSP
    assert lib.samba_paged_attn_workspace_size(ctypes.byref(_set(_attn(), dict(kv__head_dim=7)))) == 2 ** 64 - 1


def test_null_structs(lib):
    for f in (lib.samba_kv_append, lib.samba_paged_attn, lib.samba_block_norm_fwd, lib.samba_block_norm_bwd):
        assert f(None, None) == INV


def _fwd():
    a = L.BlockNormArgs()
    a.r = a.y = a.w_pre = a.w_post = a.gate = a.alpha = a.r_out = a.n = a.rstd_pre = a.rstd_post = F
    a.rows, a.width, a.r_dtype, a.y_dtype, a.eps = 4, 256, L.SAMBA_F32, L.SAMBA_BF16, 1e-6
    return a


@pytest.mark.parametrize("over,code", [
    (dict(r=None), INV), (dict(n=None), INV), (dict(w_pre=None), INV), (dict(r_out=None), INV), (dict(y=None), INV),
    (dict(y=None, r_out=None), INV), (dict(w_post=None), INV), (dict(width=250), INV), (dict(width=0), INV),
    (dict(width=8200), UNS), (dict(rows=-1), INV), (dict(rows=2 ** 31), UNS), (dict(r_dtype=2), UNS),
    (dict(y_dtype=5), UNS), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(gate=F + 2), INV),
    (dict(n=None, w_pre=None), INV),
])
def test_norm_refuses(lib, over, code):
    assert lib.samba_block_norm_fwd(ctypes.byref(_set(_fwd(), over)), None) == code


def _bwd(lib):
    a = L.BlockNormBwdArgs()
    for f, _ in L.BlockNormBwdArgs._fields_[:17]:
        setattr(a, f, F)
    a.rows, a.width, a.r_dtype, a.y_dtype = 4, 256, L.SAMBA_F32, L.SAMBA_BF16
    a.workspace_bytes = lib.samba_block_norm_bwd_workspace_size(4, 256)
    return a


@pytest.mark.parametrize("over,code", [
    (dict(dr=None), INV), (dict(dn=None, dr_out=None), INV), (dict(r=None), INV), (dict(rstd_pre=None), INV),
    (dict(dw_pre=None), INV), (dict(dn=None), INV), (dict(dy=None), INV), (dict(dgate=None), INV), (dict(gate=None), INV),
    (dict(dalpha=None), INV), (dict(dw_post=None), INV), (dict(rstd_post=None), INV), (dict(y=None, dy=None), INV),
    (dict(width=12), INV), (dict(width=16384), UNS), (dict(y_dtype=2), UNS), (dict(dy=F + 8), INV),
    (dict(workspace=None), WSP), (dict(workspace_bytes=16), WSP), (dict(workspace=F + 8), INV),
])
def test_norm_backward_refuses(lib, over, code):
    assert lib.samba_block_norm_bwd(ctypes.byref(_set(_bwd(lib), over)), None) == code


def test_norm_backward_workspace_size(lib):
    size = lib.samba_block_norm_bwd_workspace_size
    assert size(0, 256) == 0 and size(4, 0) == 0
    # two planes of column sums for each group of rows (one of 2048 elements, eight of 256)
    assert size(1, 2048) == 2 * 2048 * 4 and size(8, 256) == 2 * 256 * 4
