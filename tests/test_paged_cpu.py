"""The paged-cache entry points without a GPU: host-side refusals, and pins of
their oracle against formulas written another way."""
import ctypes

import numpy as np
import pytest
import torch

from hybrid_linear_attention_arl2_b200 import arl2, build
from oracle import paged_oracle as po

MB = 1 << 20
A, B, C, D, E, F = (i * (MB << 4) for i in range(1, 7))  # fake 16-byte-aligned addresses, never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return arl2.load_library()


def _prep(axes=(), theta=1e4, halves=0, eps=1e-6, w_q=None, w_k=None):
    return arl2.arl2_qk_prep(len(axes), (ctypes.c_int32 * 3)(*axes), halves, theta, eps, w_q, w_k)


def _rope(lib, prep=None, dtype=arl2.ARL2_BF16, heads=4, kv_heads=2, d=128, tokens=0, q=A, k=B, ld=0, pos=E, q_out=C,
          k_out=D, ld_out=0):
    prep = _prep((d,) if d % 2 == 0 else ()) if prep is None else prep
    return lib.arl2_qk_norm_rope(ctypes.addressof(prep), dtype, heads, kv_heads, d, tokens, q, k, ld, pos, q_out, k_out,
                                 ld_out, None)


def test_norm_rope_refusals(lib):
    INV, UNS = 1, 2
    assert _rope(lib) == 0                                    # no tokens: nothing to do
    assert lib.arl2_qk_norm_rope(None, 1, 4, 2, 128, 0, A, B, 0, E, C, D, 0, None) == INV
    for kw, want in [(dict(heads=0), INV), (dict(tokens=-1), INV), (dict(dtype=7), UNS), (dict(d=256), UNS),
                     (dict(d=12), UNS), (dict(d=0), INV), (dict(dtype=arl2.ARL2_F32, d=6), UNS),
                     (dict(ld=4 * 128 - 8), INV), (dict(ld=4 * 128 + 4), INV), (dict(ld_out=8), INV),
                     (dict(tokens=1 << 31), UNS)]:
        assert _rope(lib, **kw) == want, kw
    for prep, want in [(_prep((3,)), INV), (_prep((0,)), INV), (_prep((64, 66)), INV), (_prep((8,), theta=0.5), INV),
                       (_prep((8,), theta=float("nan")), INV), (_prep((8,), eps=-1.0), INV),
                       (_prep((8,), eps=float("inf")), INV), (_prep((8,), halves=2), INV), (_prep((8,), w_q=A), INV),
                       (_prep((8,), w_q=A + 4, w_k=B), INV), (_prep((8,), halves=1), UNS)]:
        assert _rope(lib, prep) == want
    # pointers and overlaps, 10 tokens of 4 + 2 heads of 128 bf16
    for kw in [dict(q=None), dict(k_out=None), dict(pos=None), dict(q=A + 8), dict(q_out=B), dict(q_out=A + 1024),
               dict(k_out=A + 1024), dict(q_out=C, k_out=C + 9 * 1024), dict(q_out=E), dict(k_out=E - 16),
               dict(ld=768, k=A + 1024, q_out=A, k_out=D),           # in place with another pitch
               dict(ld=768, k=A + 1024, ld_out=768, q_out=A, k_out=A + 1024 + 256)]:
        assert _rope(lib, tokens=10, **kw) == INV, kw


def test_paged_init_refusals(lib):
    h = ctypes.c_void_p()

    def init(H=8, hk=2, d=128, page=16, n=100, dtype=arl2.ARL2_BF16, scale=0.0, k=A, v=D):
        cfg = arl2.arl2_paged_config(H, hk, d, page, n, dtype, scale)
        return lib.arl2_paged_init(ctypes.byref(cfg), k, v, None, ctypes.byref(h))

    assert lib.arl2_paged_init(None, A, B, None, ctypes.byref(h)) == 1
    for kw, want in [(dict(H=0), 1), (dict(H=7), 1), (dict(H=130, hk=2), 2), (dict(d=64), 2), (dict(d=132), 2),
                     (dict(dtype=arl2.ARL2_F32, d=30), 2), (dict(dtype=9), 2), (dict(page=12), 2), (dict(page=0), 1),
                     (dict(page=8192), 2), (dict(n=0), 1), (dict(n=1 << 28), 2), (dict(scale=-1.0), 1),
                     (dict(scale=float("nan")), 1), (dict(k=None), 1), (dict(v=D + 8), 1), (dict(v=A + MB // 2), 1)]:
        assert init(**kw) == want, kw
        assert h.value is None


def test_foreign_paged_handles(lib):
    bogus = ctypes.c_void_p(0x1000)
    b = arl2.arl2_paged_batch(0, 0, 0, 0, 0, None, None, None)
    for h in (None, bogus):
        assert lib.arl2_paged_append(h, ctypes.addressof(b), None, None, A, B, 0, None, None, None) == 1
        assert lib.arl2_paged_attend(h, ctypes.addressof(b), A, 0, 0, B, None, None) == 1
        assert lib.arl2_paged_weights(h, ctypes.addressof(b), A, 0, 0, B, 1.0, C, D, 0, None) == 1
        assert lib.arl2_paged_evict(h, ctypes.addressof(b), A, 8, 4, 0, 0, B, 1, C, D, E, None) == 1
        assert lib.arl2_paged_last_error(h) == 1
        assert lib.arl2_paged_device_bytes(h) == -1
        assert lib.arl2_paged_set_wait_limit(h, 1) == 1
        assert lib.arl2_paged_destroy(h) == 1
    assert arl2.arl2_status_string(9).startswith("a page")


def test_wrapper_refusals():
    """The Python wrappers refuse tensors that the library would misread."""
    t = torch.zeros(6, 4, 8)
    ok = lambda **kw: arl2._token_rows(8, torch.float32, -1, [(name, x, 4) for name, x in kw.items()])
    wide = torch.zeros(6, 96)
    assert ok(q=t, k=t) == (0, 6)
    assert ok(q=wide[:, :32].unflatten(1, (4, 8)), k=wide[:, 32:64].unflatten(1, (4, 8))) == (96, 6)
    assert ok(q=wide[:1, :32].unflatten(1, (4, 8)), k=t[:1]) == (0, 1)
    for kw in [dict(q=t[:, :2]), dict(q=t.double()), dict(q=t, k=t[:5]), dict(q=t.transpose(0, 1)[:, :4]),
               dict(q=torch.zeros(6, 4, 16)[..., ::2]), dict(q=wide[:, :32].unflatten(1, (4, 8)), k=t),
               dict(q=torch.zeros(6, 8, 4).transpose(1, 2))]:
        with pytest.raises(ValueError):
            ok(**kw)
    with pytest.raises(ValueError):
        arl2.QKPrep([2, 2, 2, 2])
    with pytest.raises(ValueError):
        arl2.QKPrep([8], w_q=torch.ones(8))
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError):
        arl2.PagedBatch(i32(2), i32(2), i32(2, 3), tokens=0, max_q=0, max_kv=0)
    with pytest.raises(ValueError):
        arl2.PagedBatch(i32(3), i32(2).long(), i32(2, 3), tokens=0, max_q=0, max_kv=0)
    with pytest.raises(ValueError):
        arl2.PagedBatch(i32(3), i32(2), i32(3, 3), tokens=0, max_q=0, max_kv=0)


# ------------------------------------------------------------------ oracle pins
def test_oracle_norm_rope_pins():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 2, 16))
    w = rng.standard_normal(16)
    zero = np.zeros((5, 2), int)
    y = po.norm_rope(x, w, zero, (8, 4))
    assert np.allclose(y, x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 1e-6) * w)
    # a rotation by complex numbers, lengths kept, channels past R left alone
    pos = rng.integers(-50, 50, (5, 2))
    for halves in (False, True):
        y = po.norm_rope(x, None, pos, (8, 4), theta=100.0, halves=halves)
        assert np.array_equal(y[..., 12:], x[..., 12:]) and np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        z = (x[..., :6] + 1j * x[..., 6:12]) if halves else (x[..., 0:12:2] + 1j * x[..., 1:12:2])
        f = np.concatenate([np.outer(pos[:, 0], 100.0 ** (-np.arange(4) / 4)), np.outer(pos[:, 1], 100.0 ** (-np.arange(2) / 2))], 1)
        z = z * np.exp(1j * f)[:, None]
        got = (y[..., :6] + 1j * y[..., 6:12]) if halves else (y[..., 0:12:2] + 1j * y[..., 1:12:2])
        assert np.allclose(got, z)


def test_oracle_attention_pins():
    rng = np.random.default_rng(4)
    hk, page, d, H = 2, 4, 8, 4
    kp, vp = rng.standard_normal((2, 9, hk, page, d))
    tables = np.array([[4, 0, 7], [2, 8, -1]])
    seqs = [(5, 10), (3, 7)]
    q = rng.standard_normal((8, H, d))
    for mask in (0, 1, 2):
        o, lse, _ = po.attend(q, kp, vp, seqs, tables, mask)
        at = 0
        for b, (n, kv) in enumerate(seqs):
            j = np.arange(kv)
            K = torch.tensor(kp[tables[b][j // page], :, j % page]).transpose(0, 1).repeat_interleave(2, 0)
            V = torch.tensor(vp[tables[b][j // page], :, j % page]).transpose(0, 1).repeat_interleave(2, 0)
            i = np.arange(n)
            see = np.ones((n, kv), bool) if mask == 0 else ((j - (kv - n)) // mask)[None] <= (i // mask)[:, None]
            Q = torch.tensor(q[at:at + n]).transpose(0, 1)
            ref = torch.nn.functional.scaled_dot_product_attention(Q, K, V, torch.tensor(see))
            assert np.allclose(o[at:at + n], ref.transpose(0, 1).numpy())
            # the weights of a row sum to one, so those of a call to its rows
            at += n
        w = po.weights(q, kp, lse, np.zeros((2, hk, 10)), seqs, tables, mask, 1.0)
        assert np.allclose(w.sum((1, 2)), [5 * H, 3 * H])
    assert po.visible(5, 3, 1) == [0, 0, 1, 2, 3] and po.visible(5, 9, 2) == [6, 6, 8, 8, 9]
    o, lse, _ = po.attend(q[:5], kp, vp, [(5, 3)], tables[:1], 1)
    assert not o[:2].any() and np.isinf(lse[:2]).all()


def test_oracle_keep_pins():
    w = np.array([0.0, 5.0, 1.0, np.nan, 1.0, -0.0, 0.0, 9.0, 1.0, 2.0])
    assert po.keep(w, 10, 10, 1, 1) == list(range(10))
    assert po.keep(w, 10, 4, 1, 1) == [0, 1, 7, 9]
    assert po.keep(w, 10, 5, 1, 1) == [0, 1, 2, 7, 9]
    assert po.keep(w, 10, 8, 1, 1) == [0, 1, 2, 4, 5, 7, 8, 9]
    assert po.keep(w, 10, 9, 1, 1) == [0, 1, 2, 4, 5, 6, 7, 8, 9]
    assert po.keep(w, 10, 3, 2, 1) == [0, 1, 9]
