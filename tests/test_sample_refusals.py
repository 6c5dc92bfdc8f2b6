"""Host-side refusals of the sampling calls (CPU only: nothing is launched)."""
import ctypes

import pytest
import torch

import mla_latent_kv_06_gb300 as mla
from mla_latent_kv_06_gb300 import _build


def _at(x):
    return ctypes.c_void_p(x)


LOGITS, SET, U, TOKEN, PROBS = (_at(i << 30) for i in range(1, 6))


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return mla.load()


def _call(lib, B=2, N=3, V=100, dtype=0, logits=LOGITS, l_row=100, l_batch=300, temperature=SET, top_k=None, top_p=None,
          min_p=None, per_row=0, u=U, token=TOKEN, probs=PROBS, p_row=100, p_batch=300):
    return lib.mla_sample(B, N, V, dtype, logits, l_row, l_batch, temperature, top_k, top_p, min_p, per_row, u, token, probs,
                          p_row, p_batch, None)


def test_arguments(lib):
    for bad in (dict(B=0), dict(N=0), dict(V=0), dict(B=(1 << 24) + 1, N=1), dict(dtype=2), dict(logits=None),
                dict(token=None, u=None, probs=None), dict(u=None), dict(token=None), dict(l_row=99), dict(l_row=-1, N=1),
                dict(l_batch=-1), dict(l_row=1 << 41), dict(l_batch=1 << 41), dict(p_row=99), dict(p_batch=299), dict(p_batch=-1),
                dict(p_row=1 << 41, B=1), dict(logits=_at((1 << 30) + 2)), dict(logits=_at((1 << 30) + 1), dtype=1),
                dict(probs=_at((5 << 30) + 2)), dict(l_row=(1 << 37) + 1), dict(u=_at((3 << 30) + 1)), dict(token=_at((4 << 30) + 2)),
                dict(temperature=_at((2 << 30) + 2)), dict(top_k=_at((2 << 30) + 1)), dict(top_p=_at((2 << 30) + 3)),
                dict(min_p=_at((2 << 30) + 2))):
        assert _call(lib, **bad) == mla.MLA_ERR_INVALID, bad
    assert _call(lib, V=327681, l_row=327681, p_row=327681, p_batch=1 << 20) == mla.MLA_ERR_UNSUPPORTED
    assert b"327680" in lib.mla_last_error()


@pytest.mark.parametrize("who,where", [
    ("token", (1 << 30) + 4 * 599), ("token", (1 << 30) - 20), ("token", (3 << 30) + 20), ("token", (2 << 30) + 4),
    ("token", (5 << 30) + 4 * 599), ("probs", (1 << 30) + 4 * 599), ("probs", (1 << 30) - 4 * 599), ("probs", (2 << 30) - 4 * 599),
    ("probs", (3 << 30) + 20)])
def test_overlaps(lib, who, where):
    """Tokens or probabilities of one row written over what another row reads."""
    assert _call(lib, **{who: _at(where)}) == mla.MLA_ERR_INVALID and b"overlap" in lib.mla_last_error()


def test_settings_per_row_reach_further(lib):
    assert _call(lib, per_row=1, token=_at((2 << 30) + 4 * 5)) == mla.MLA_ERR_INVALID
    assert _call(lib, top_k=_at(7 << 30), per_row=1, token=_at((7 << 30) + 20)) == mla.MLA_ERR_INVALID


def test_binding(lib):
    x, u, t = torch.randn(2, 5), torch.rand(2), torch.ones(2)
    with pytest.raises(ValueError, match="GPU"):
        mla.sample(x, u)
    with pytest.raises(ValueError, match="GPU"):
        mla.sample_probs(x)
    with pytest.raises(ValueError, match="needed"):
        mla.sample(x, None)
    with pytest.raises(ValueError):
        mla.sample(x[0], u)
    with pytest.raises(TypeError):
        mla.sample(x.double(), u)
    with pytest.raises(ValueError, match="contiguous"):
        mla.sample(torch.randn(5, 2).T, u)
    with pytest.raises(ValueError, match="temperature"):
        mla.sample(x, u, temperature=torch.ones(3))
    with pytest.raises(ValueError, match="u has shape"):
        mla.sample(x, torch.rand(3))
    y = torch.randn(2, 3, 5)
    with pytest.raises(ValueError, match="all per"):
        mla.sample_probs(y, temperature=torch.ones(2), top_p=torch.ones(2, 3))
    with pytest.raises(ValueError, match="probs"):
        mla.sample_probs(y, probs=torch.empty(2, 3, 4))
