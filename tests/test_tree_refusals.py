"""Host-side refusals of the drafted-tree calls (CPU only: nothing is launched)."""
import ctypes

import pytest
import torch

import mla_latent_kv_06_gb300 as mla
from mla_latent_kv_06_gb300 import _build
from workload import TINY

P = ctypes.c_void_p(256)
GLM_D = mla.MlaDims(64, 192, 64, 512, 256, 0.0, 0.0)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return mla.load()


def _decode(lib, d=GLM_D, dtype=1, B=1, S=2, q=P, Lc=P, T_cap=16, T=P, parent=P, kv_b=P, out_dtype=0, out=P):
    return lib.mla_decode_tree(ctypes.byref(d), dtype, B, S, q, Lc, P, T_cap, T, parent, kv_b, out_dtype, out, None, 0, None)


def test_decode_tree(lib):
    assert _decode(lib, S=65, T_cap=100) == mla.MLA_ERR_UNSUPPORTED and b"64" in lib.mla_last_error()
    for bad in (dict(S=0), dict(B=0), dict(S=17), dict(dtype=7), dict(out_dtype=2), dict(q=None), dict(Lc=None), dict(T=None),
                dict(parent=None), dict(kv_b=None), dict(out=None), dict(out=ctypes.c_void_p(8)),
                dict(d=mla.MlaDims(64, 192, 63, 512, 256, 0.0, 0.0))):
        assert _decode(lib, **bad) == mla.MLA_ERR_INVALID, bad
    for table, ps, pages, want in ((None, 128, 2, mla.MLA_ERR_INVALID), (P, 0, 2, mla.MLA_ERR_INVALID),
                                   (P, 1 << 8, 1 << 24, mla.MLA_ERR_UNSUPPORTED)):
        assert lib.mla_decode_tree_paged(ctypes.byref(GLM_D), 1, 1, 2, P, P, P, pages, ps, table, 2, P, P, P, 0, P, None, 0,
                                         None) == want
    assert lib.mla_decode_tree_workspace_size(ctypes.byref(GLM_D), 1, 1, 65, 100) == 0
    assert lib.mla_decode_tree_workspace_size(ctypes.byref(GLM_D), 1, 1, 8, 100) > 0
    tiny = mla.MlaDims(4, 16, 8, 32, 16, 0.0, 0.0)
    assert lib.mla_decode_tree_workspace_size(ctypes.byref(tiny), 0, 1, 4, 64) == 0      # one split of the keys
    assert lib.mla_decode_tree_workspace_size(ctypes.byref(tiny), 0, 1, 8, 100000) > 0   # several


def test_append_tree(lib):
    def call(B=1, S=2, comp=P, T_cap=16, parent=P, eps=1e-6):
        return lib.mla_cache_append_tree(ctypes.byref(GLM_D), 1, B, S, comp, P, eps, T_cap, P, parent, P, P, None)
    assert call(S=65, T_cap=100) == mla.MLA_ERR_UNSUPPORTED
    for bad in (dict(S=0), dict(B=0), dict(S=17), dict(comp=None), dict(parent=None), dict(eps=-1.0)):
        assert call(**bad) == mla.MLA_ERR_INVALID, bad
    assert lib.mla_cache_append_tree_paged(ctypes.byref(GLM_D), 1, 1, 2, P, P, 1e-6, P, P, 4, 16, None, 2, P, P,
                                           None) == mla.MLA_ERR_INVALID


def test_verify(lib):
    def call(B=1, S=2, V=8, p=P, p_row=8, p_batch=24, q=P, q_row=8, q_batch=24, tokens=P, parent=P, u=P, path=P, n=P, token=P):
        return lib.mla_tree_verify(B, S, V, p, p_row, p_batch, q, q_row, q_batch, tokens, parent, u, path, n, token, None)
    assert call(S=65) == mla.MLA_ERR_UNSUPPORTED
    for bad in (dict(B=0), dict(S=0), dict(V=0), dict(p=None), dict(tokens=None), dict(parent=None), dict(u=None),
                dict(path=None), dict(n=None), dict(token=None), dict(p_row=7), dict(q_row=7), dict(p_batch=-1),
                dict(q_batch=-1), dict(V=(1 << 30) + 1), dict(B=(1 << 24) + 1)):
        assert call(**bad) == mla.MLA_ERR_INVALID, bad


def test_commit(lib):
    arr, hole = (ctypes.c_void_p * 2)(1 << 20, 2 << 20), (ctypes.c_void_p * 2)(1 << 20, None)
    size, zero = (ctypes.c_int * 2)(1024, 128), (ctypes.c_int * 2)(1024, 0)

    def call(n=2, cache=arr, rb=size, B=1, S=2, T_cap=16, T=P, path=P, n_acc=P, T_out=ctypes.c_void_p(1024)):
        return lib.mla_tree_commit(n, cache, rb, B, S, T_cap, T, path, n_acc, T_out, None)
    assert call(S=65, T_cap=100) == mla.MLA_ERR_UNSUPPORTED
    for bad in (dict(n=0), dict(cache=None), dict(rb=None), dict(cache=hole), dict(rb=zero), dict(B=0), dict(B=65536), dict(S=0),
                dict(S=17), dict(T=None), dict(path=None), dict(n_acc=None), dict(T_out=P)):
        assert call(**bad) == mla.MLA_ERR_INVALID, bad
    assert lib.mla_tree_commit_paged(2, arr, size, 1, 2, 4, 16, None, 2, P, P, P, None, None) == mla.MLA_ERR_INVALID


@pytest.mark.parametrize("second,row_bytes,B,bad", [(1 << 20, 128, 1, True), ((1 << 20) + 16 * 1024 - 1, 128, 1, True),
                                                    ((1 << 20) - 16 * 128 + 1, 128, 1, True),
                                                    ((1 << 20) + 16 * 1024, 128, 2, True)])
@pytest.mark.parametrize("paged", [False, True])
def test_commit_refuses_caches_that_overlap(lib, second, row_bytes, B, bad, paged):
    """The same cache twice, or caches of 16 rows per sequence that share bytes, would have rows moved twice."""
    arr, size = (ctypes.c_void_p * 2)(1 << 20, second), (ctypes.c_int * 2)(1024, row_bytes)
    x, y, z = (ctypes.c_void_p(i << 30) for i in (1, 2, 3))
    if paged:
        rc = lib.mla_tree_commit_paged(2, arr, size, B, 2, 4 * B, 4, ctypes.c_void_p(5 << 30), 4, x, y, z, None, None)
    else:
        rc = lib.mla_tree_commit(2, arr, size, B, 2, 16, x, y, z, None, None)
    assert rc == mla.MLA_ERR_INVALID and b"overlaps" in lib.mla_last_error()


def test_commit_refuses_a_late_overlap(lib):
    """Among many caches, out of order, only the last one overlaps: with an early or a late one."""
    n = 300
    x, y, z = (ctypes.c_void_p(i << 40) for i in (1, 2, 3))
    for twin in (7, 200):
        at = [(1 << 20) + 16 * 1024 * ((37 * i) % n) for i in range(n)]
        at.append(at[twin])
        rc = lib.mla_tree_commit(n + 1, (ctypes.c_void_p * (n + 1))(*at), (ctypes.c_int * (n + 1))(*[1024] * (n + 1)), 1, 2, 16,
                                 x, y, z, None, None)
        assert rc == mla.MLA_ERR_INVALID and b"cache 300 overlaps" in lib.mla_last_error()


def test_commit_refuses_lengths_over_its_arguments(lib):
    arr, size = (ctypes.c_void_p * 1)(1 << 20), (ctypes.c_int * 1)(1024)
    B, S, T, path, n = 3, 4, 1 << 30, 2 << 30, 3 << 30
    for at in (T, T + 8, T - 8, path, path + 4 * B * S - 4, n, n - 4):
        rc = lib.mla_tree_commit(1, arr, size, B, S, 16, ctypes.c_void_p(T), ctypes.c_void_p(path), ctypes.c_void_p(n),
                                 ctypes.c_void_p(at), None)
        assert rc == mla.MLA_ERR_INVALID and b"T_out" in lib.mla_last_error(), at


def test_binding_refuses_on_the_host(lib):
    """Wrong shapes, types and places are found before the library is called."""
    B, S, V = 2, 3, 5
    p, tok, u = torch.rand(B, S + 1, V), torch.zeros(B, S, dtype=torch.int32), torch.rand(B, S + 1)
    par = torch.full((B, S), -1, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        mla.tree_verify(p, p, tok, par, u)
    with pytest.raises(ValueError, match="shape"):
        mla.tree_verify(p[:, 1:], None, tok, par, u)
    with pytest.raises(TypeError):
        mla.tree_verify(p.double(), None, tok, par, u)
    with pytest.raises(TypeError):
        mla.tree_verify(p, None, tok.long(), par, u)
    with pytest.raises(ValueError, match="contiguous"):
        mla.tree_verify(p.transpose(1, 2).contiguous().transpose(1, 2), None, tok, par, u)
    with pytest.raises(ValueError):
        mla.CacheRows([])
    with pytest.raises(ValueError, match="GPU"):
        mla.CacheRows([torch.zeros(1, 4, 8)])
    with pytest.raises(ValueError, match="shape"):
        mla.CacheRows([torch.zeros(1, 4, 8), torch.zeros(1, 5, 8)])
    q = torch.zeros(B, S, TINY.H, TINY.qk_head)
    Lc, Rc = torch.zeros(B, 8, TINY.kv_lora), torch.zeros(B, 8, TINY.qk_rope)
    kv_b, T = torch.zeros(TINY.H, TINY.qk_nope + TINY.v_head, TINY.kv_lora), torch.full((B,), 8, dtype=torch.int32)
    for change, error in ((dict(), ValueError), (dict(T=T.long()), TypeError), (dict(parent=par[:, :2]), ValueError),
                          (dict(q=q[:, :, :3]), ValueError), (dict(kv_b=kv_b[:, 1:]), ValueError),
                          (dict(Rc=Rc[:, 1:]), ValueError), (dict(out_dtype=torch.float16), TypeError)):
        args = dict(q=q, Lc=Lc, Rc=Rc, T=T, parent=par, kv_b=kv_b, dims=TINY)
        args.update(change)
        with pytest.raises(error):
            mla.decode_tree(**args)
    comp, ln = torch.zeros(B, S, TINY.kv_lora + TINY.qk_rope), torch.ones(TINY.kv_lora)
    with pytest.raises(ValueError, match="GPU"):
        mla.cache_append_tree(comp, ln, T, par, Lc, Rc, TINY, 1e-6)
    with pytest.raises(ValueError):
        mla.cache_append_tree(comp[:, :, 1:], ln, T, par, Lc, Rc, TINY, 1e-6)


@pytest.mark.parametrize("dims,dtype", [(GLM_D, 1), (mla.MlaDims(1, 2, 2, 1, 1, 0.0, 0.0), 0)])
def test_decode_tree_refuses_capacities_at_the_end_of_int32(lib, dims, dtype):
    """Key indices step by up to 256 past a sequence's length in int32."""
    top = (1 << 31) - 1
    for cap in (top, top - 1022):
        assert _decode(lib, d=dims, dtype=dtype, T_cap=cap) == mla.MLA_ERR_UNSUPPORTED, cap
        assert lib.mla_decode_tree_workspace_size(ctypes.byref(dims), dtype, 1, 2, cap) == 0
    assert lib.mla_decode_tree_workspace_size(ctypes.byref(dims), dtype, 1, 2, top - 1023) > 0
    table_pages = (top - 127) // 128  # a capacity of 2^31 - 128 rows
    assert lib.mla_decode_tree_paged(ctypes.byref(dims), dtype, 1, 2, P, P, P, 4, 128, P, table_pages, P, P, P, 0, P, None, 0,
                                     None) == mla.MLA_ERR_UNSUPPORTED
