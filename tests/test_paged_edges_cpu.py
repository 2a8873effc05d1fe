"""Calls at the edge of what the paged-cache wrappers accept, without a GPU:
tensors that the library would misread are refused before it sees them."""
import pytest
import torch

from hybrid_linear_attention_arl2_b200 import arl2


def _rows(**kw):
    return arl2._token_rows(8, torch.float32, -1, [(name, t, t.shape[1]) for name, t in kw.items()])


def test_rows_broadcast_over_tokens_are_refused():
    """A view of stride 0 over tokens has the storage of one row, one of a pitch below a row's width rows that
    overlap: the library's pitch of 0 means contiguous, so neither may pass for it."""
    one = torch.zeros(1, 4, 8)
    assert _rows(q=one) == (0, 1)
    assert _rows(q=one.expand(1, 4, 8)) == (0, 1)
    wide = torch.zeros(6 * 96)
    for t in (one.expand(6, 4, 8), wide.as_strided((6, 4, 8), (24, 8, 1)), wide.as_strided((6, 4, 8), (8, 8, 1))):
        with pytest.raises(ValueError):
            _rows(q=t)
        with pytest.raises(ValueError):
            _rows(q=t, k=torch.zeros(6, 2, 8))
        with pytest.raises(ValueError):
            _rows(q=torch.zeros(6, 2, 8), k=t)
    # the pitch holds the widest tensor's row, not the first one's
    with pytest.raises(ValueError):
        _rows(k=wide.as_strided((6, 1, 8), (16, 8, 1)), q=wide.as_strided((6, 4, 8), (16, 8, 1)))
    # a view of one row for all tokens beside a strided one of the same pitch
    assert _rows(q=wide.as_strided((6, 4, 8), (96, 8, 1)), k=wide.as_strided((6, 1, 8), (96, 8, 1), 32)) == (96, 6)


def test_host_tensors_are_refused(monkeypatch):
    """The library takes device memory: tensors of the host never reach it."""
    def reached(*a):
        raise AssertionError("the library was called")

    monkeypatch.setattr(arl2, "load_library", reached)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    q, pool = torch.zeros(3, 4, 8), torch.zeros(2, 4, 8, 8)
    for kw in ({}, dict(q_out=torch.empty_like(q), k_out=torch.empty_like(q))):
        with pytest.raises(ValueError):
            arl2.qk_norm_rope(arl2.QKPrep([]), q, q, **kw)
    with pytest.raises(ValueError):
        arl2.PagedKVLayer(4, 4, 8, arl2.ARL2_F32, pool, pool.clone())
