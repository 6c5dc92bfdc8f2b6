"""Host-side refusals of decode_shared_paged (CPU only: nothing is launched)."""
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


def _call(lib, d=GLM_D, dtype=1, B=2, S=2, q=P, Lc=P, num_pages=9, page=128, table=P, max_pages=4, T=P, shared=256, parent=None, kv_b=P,
          out_dtype=0, out=P):
    return lib.mla_decode_shared_paged(ctypes.byref(d), dtype, B, S, q, Lc, P, num_pages, page, table, max_pages, T, shared, parent, kv_b,
                                       out_dtype, out, None, 0, None)


def test_arguments(lib):
    for bad in (dict(B=0), dict(S=0), dict(dtype=5), dict(out_dtype=2), dict(q=None), dict(Lc=None), dict(table=None), dict(T=None),
                dict(kv_b=None), dict(out=None), dict(out=ctypes.c_void_p(264)), dict(shared=-1), dict(shared=511),
                dict(shared=(1 << 31) - 1), dict(num_pages=0), dict(page=0), dict(max_pages=0),
                dict(d=mla.MlaDims(64, 192, 63, 512, 256, 0.0, 0.0))):
        assert _call(lib, **bad) == mla.MLA_ERR_INVALID, bad
    assert _call(lib, S=3, shared=510) == mla.MLA_ERR_INVALID and b"fit" in lib.mla_last_error()
    assert _call(lib, B=8193, S=1) == mla.MLA_ERR_UNSUPPORTED
    assert _call(lib, B=200, S=41) == mla.MLA_ERR_UNSUPPORTED and b"8192" in lib.mla_last_error()
    assert _call(lib, S=65) == mla.MLA_ERR_UNSUPPORTED and b"64" in lib.mla_last_error()
    assert _call(lib, max_pages=((1 << 31) - 127) // 128) == mla.MLA_ERR_UNSUPPORTED
    assert _call(lib, num_pages=1 << 25) == mla.MLA_ERR_UNSUPPORTED
    assert _call(lib, B=300, S=1, max_pages=(1 << 30) // 128) == mla.MLA_ERR_UNSUPPORTED and b"behind" in lib.mla_last_error()


def test_workspace_size(lib):
    def size(d=GLM_D, dtype=1, B=4, S=1, cap=4096, shared=1024):
        return lib.mla_decode_shared_workspace_size(ctypes.byref(d), dtype, B, S, cap, shared)
    assert size() > 0 and size(shared=0) > 0 and size(shared=4095) > 0
    for none in (dict(B=0), dict(S=0), dict(S=65), dict(B=8193), dict(shared=-1), dict(shared=4096), dict(cap=0), dict(cap=(1 << 31) - 1000)):
        assert size(**none) == 0, none
    tiny = mla.MlaDims(4, 16, 8, 32, 16, 0.0, 0.0)
    assert size(d=tiny, dtype=0, B=400, cap=64, shared=32) == 0  # one split of the keys


def test_binding(lib):
    B, S = 2, 1
    q = torch.zeros(B, S, TINY.H, TINY.qk_head)
    L, R = torch.zeros(5, 16, TINY.kv_lora), torch.zeros(5, 16, TINY.qk_rope)
    kv_b, T = torch.zeros(TINY.H, TINY.qk_nope + TINY.v_head, TINY.kv_lora), torch.full((B,), 20, dtype=torch.int32)
    table = torch.zeros(B, 2, dtype=torch.int32)
    for change, error in ((dict(), ValueError), (dict(T=T.long()), TypeError), (dict(table=table[:1]), ValueError),
                          (dict(table=table.long()), TypeError), (dict(q=q[..., :3]), ValueError), (dict(kv_b=kv_b[:, 1:]), ValueError),
                          (dict(R=R[:, 1:]), ValueError), (dict(out_dtype=torch.float16), TypeError), (dict(kv_b=kv_b.bfloat16()), TypeError),
                          (dict(parent=table), ValueError)):
        a = dict(q=q, L=L, R=R, table=table, T=T, kv_b=kv_b, out_dtype=None, parent=None)
        a.update(change)
        with pytest.raises(error):
            mla.decode_shared_paged(a["q"], a["L"], a["R"], a["table"], a["T"], 16, a["kv_b"], TINY, out_dtype=a["out_dtype"],
                                    parent=a["parent"])
