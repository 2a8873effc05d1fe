"""Thin ctypes binding of libarl2.so (C ABI in include/arl2.h).

The functions named ``arl2_*`` mirror the C entry points one to one and only
marshal arguments: torch tensors become device pointers, a torch stream
becomes a ``cudaStream_t``.  ``HybridLayer`` and ``KVLayer`` wrap a handle
for convenience.  Every step of the hot path runs in the library's CUDA
kernels; there is no fallback -- importing works without a GPU, but any call
that needs the library raises if ``libarl2.so`` is missing.
"""
from __future__ import annotations

import ctypes
import os
import re

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libarl2.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "arl2.h")

ARL2_F32, ARL2_BF16 = 0, 1
ARL2_INTRA_ONLY, ARL2_INTER_ONLY = 1, 2

STATUS = {
    0: "ARL2_OK", 1: "ARL2_ERR_INVALID_ARGUMENT", 2: "ARL2_ERR_UNSUPPORTED",
    3: "ARL2_ERR_OUT_OF_MEMORY", 4: "ARL2_ERR_CUDA", 5: "ARL2_ERR_TIMEOUT", 6: "ARL2_ERR_NO_DEVICE",
    7: "ARL2_ERR_SCRATCH_LIMIT",
    8: "ARL2_ERR_BOUNDS",
    9: "ARL2_ERR_PAGE",
}
ARL2_NOALLOC_SCRATCH_BYTES = 16 << 20


class Arl2Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}")


class arl2_config(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("tokens_per_frame", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float), ("corr_scale", ctypes.c_float), ("flags", ctypes.c_uint32),
    ]


class arl2_qk_prep(ctypes.Structure):
    _fields_ = [
        ("n_axes", ctypes.c_int32), ("axis_dim", ctypes.c_int32 * 3), ("halves", ctypes.c_int32),
        ("theta", ctypes.c_float), ("eps", ctypes.c_float), ("w_q", ctypes.c_void_p), ("w_k", ctypes.c_void_p),
    ]


class arl2_paged_config(ctypes.Structure):
    _fields_ = [
        ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float),
    ]


class arl2_paged_batch(ctypes.Structure):
    _fields_ = [
        ("n_seqs", ctypes.c_int32), ("tokens", ctypes.c_int32), ("max_q", ctypes.c_int32),
        ("max_kv", ctypes.c_int32), ("pages_ld", ctypes.c_int32),
        ("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("pages", ctypes.c_void_p),
    ]


_VP, _I32, _I64, _U64, _F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_float
_SIGS = {
    "arl2_state_init": (_I32, [ctypes.POINTER(arl2_config), _VP, _VP, _VP, _VP, ctypes.POINTER(_VP)]),
    "arl2_frame_query": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP]),
    "arl2_frame_commit": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
    "arl2_frame_query_strided": (_I32, [_VP, _VP, _VP, _VP, _I64, _VP, _VP]),
    "arl2_frame_commit_strided": (_I32, [_VP, _VP, _VP, _VP, _I64, _VP, _VP, _VP, _VP]),
    "arl2_token_query": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
    "arl2_token_commit": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
    "arl2_state_get": (_I32, [_VP, _VP, ctypes.POINTER(_I64), _VP]),
    "arl2_state_set": (_I32, [_VP, _VP, _I64, _VP]),
    "arl2_last_error": (_I32, [_VP]),
    "arl2_state_device_bytes": (_I64, [_VP]),
    "arl2_state_set_wait_limit": (_I32, [_VP, _U64]),
    "arl2_state_destroy": (_I32, [_VP]),
    "arl2_kv_init": (_I32, [ctypes.POINTER(arl2_config), _I32, _VP, ctypes.POINTER(_VP)]),
    "arl2_kv_query": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP]),
    "arl2_kv_commit": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP]),
    "arl2_kv_query_strided": (_I32, [_VP, _VP, _VP, _VP, _I64, _VP, _VP]),
    "arl2_kv_commit_strided": (_I32, [_VP, _VP, _VP, _VP, _I64, _VP, _VP]),
    "arl2_kv_frames": (_I64, [_VP]),
    "arl2_kv_device_bytes": (_I64, [_VP]),
    "arl2_kv_last_error": (_I32, [_VP]),
    "arl2_kv_destroy": (_I32, [_VP]),
    "arl2_qk_norm_rope": (_I32, [_VP, _I32, _I32, _I32, _I32, _I64, _VP, _VP, _I64, _VP, _VP, _VP, _I64, _VP]),
    "arl2_paged_init": (_I32, [ctypes.POINTER(arl2_paged_config), _VP, _VP, _VP, ctypes.POINTER(_VP)]),
    "arl2_paged_append": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP, _I64, _VP, _VP, _VP]),
    "arl2_paged_attend": (_I32, [_VP, _VP, _VP, _I64, _I32, _VP, _VP, _VP]),
    "arl2_paged_weights": (_I32, [_VP, _VP, _VP, _I64, _I32, _VP, _F32, _VP, _VP, _I64, _VP]),
    "arl2_paged_evict": (_I32, [_VP, _VP, _VP, _I64, _I32, _I32, _I32, _VP, _I32, _VP, _VP, _VP, _VP]),
    "arl2_paged_last_error": (_I32, [_VP]),
    "arl2_paged_device_bytes": (_I64, [_VP]),
    "arl2_paged_set_wait_limit": (_I32, [_VP, _U64]),
    "arl2_paged_destroy": (_I32, [_VP]),
    "arl2_block_init": (_I32, [ctypes.POINTER(arl2_config), _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.POINTER(_VP)]),
    "arl2_block_query": (_I32, [_VP, _VP, _VP, _VP]),
    "arl2_block_commit": (_I32, [_VP, _VP, _VP, _VP]),
    "arl2_block_layer": (_VP, [_VP]),
    "arl2_block_destroy": (_I32, [_VP]),
    "arl2_state_write_noalloc": (_I32, [ctypes.POINTER(arl2_config), _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                        _VP]),
    "arl2_selftest_wait_timeout": (_I32, [_U64, _VP]),
    "arl2_selftest_exp2": (_I32, [_VP, _VP, _I64, _VP]),
    "arl2_gemm_bf16": (_I32, [_VP, _I64, _VP, _I64, _VP, _I64, _I64, _I64, _I64, _VP]),
    "arl2_attn_partition": (_I32, [_I32, _I32, _I32, _I32, _I32, _VP, _I32, _VP, _VP, _VP]),
    "arl2_status_string": (ctypes.c_char_p, [_I32]),
    "arl2_abi_version": (_I32, []),
    "arl2_debug_bounds_enabled": (_I32, []),
}

_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libarl2.so; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libarl2.so not built at {path}; run python -m hybrid_linear_attention_arl2_b200.build")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def declared_symbols(header: str = HEADER) -> list[str]:
    """Entry points declared in include/arl2.h."""
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(arl2_[a-z0-9_]+)\s*\(", text)))


# ---------------------------------------------------------------- marshalling
def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, what: str) -> None:
    if status != 0:
        raise Arl2Error(status, what)


def make_config(batch, heads, head_dim, tokens, dtype, softmax_scale=0.0, corr_scale=-1.0, flags=0):
    return arl2_config(batch, heads, head_dim, tokens, dtype, softmax_scale, corr_scale, flags)


# ---------------------------------------------------------------- C entry points
def arl2_state_init(cfg: arl2_config, phi_q, phi_k, phi_v, stream=None) -> int:
    h = _VP()
    _check(load_library().arl2_state_init(ctypes.byref(cfg), _ptr(phi_q), _ptr(phi_k), _ptr(phi_v),
                                          _stream(stream), ctypes.byref(h)), "arl2_state_init")
    return h.value


def arl2_frame_query(h, q, k, v, o, stream=None) -> None:
    _check(load_library().arl2_frame_query(h, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _stream(stream)),
           "arl2_frame_query")


def arl2_frame_commit(h, q, k, v, alpha, beta, o, stream=None) -> None:
    _check(load_library().arl2_frame_commit(h, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(o),
                                            _stream(stream)), "arl2_frame_commit")


def arl2_frame_query_strided(h, q, k, v, ld, o, stream=None) -> None:
    _check(load_library().arl2_frame_query_strided(h, _ptr(q), _ptr(k), _ptr(v), int(ld), _ptr(o), _stream(stream)),
           "arl2_frame_query_strided")


def arl2_frame_commit_strided(h, q, k, v, ld, alpha, beta, o, stream=None) -> None:
    _check(load_library().arl2_frame_commit_strided(h, _ptr(q), _ptr(k), _ptr(v), int(ld), _ptr(alpha), _ptr(beta),
                                                    _ptr(o), _stream(stream)), "arl2_frame_commit_strided")


def arl2_token_query(h, q, k, v, alpha_tok, beta, o, stream=None) -> None:
    _check(load_library().arl2_token_query(h, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha_tok), _ptr(beta), _ptr(o),
                                           _stream(stream)), "arl2_token_query")


def arl2_token_commit(h, q, k, v, alpha_tok, beta, o, stream=None) -> None:
    _check(load_library().arl2_token_commit(h, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha_tok), _ptr(beta), _ptr(o),
                                            _stream(stream)), "arl2_token_commit")


def arl2_state_get(h, dst, stream=None) -> int:
    frame = _I64()
    _check(load_library().arl2_state_get(h, _ptr(dst), ctypes.byref(frame), _stream(stream)), "arl2_state_get")
    return frame.value


def arl2_state_set(h, src, frame: int, stream=None) -> None:
    _check(load_library().arl2_state_set(h, _ptr(src), frame, _stream(stream)), "arl2_state_set")


def arl2_last_error(h) -> int:
    return load_library().arl2_last_error(h)


def arl2_state_device_bytes(h) -> int:
    return load_library().arl2_state_device_bytes(h)


def arl2_state_set_wait_limit(h, limit_ns: int) -> None:
    _check(load_library().arl2_state_set_wait_limit(h, limit_ns), "arl2_state_set_wait_limit")


def arl2_state_destroy(h) -> None:
    _check(load_library().arl2_state_destroy(h), "arl2_state_destroy")


def arl2_kv_init(cfg: arl2_config, max_frames: int, stream=None) -> int:
    h = _VP()
    _check(load_library().arl2_kv_init(ctypes.byref(cfg), max_frames, _stream(stream), ctypes.byref(h)),
           "arl2_kv_init")
    return h.value


def arl2_kv_query(h, q, k, v, o, stream=None) -> None:
    _check(load_library().arl2_kv_query(h, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _stream(stream)), "arl2_kv_query")


def arl2_kv_commit(h, q, k, v, o, stream=None) -> None:
    _check(load_library().arl2_kv_commit(h, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _stream(stream)), "arl2_kv_commit")


def arl2_kv_frames(h) -> int:
    return load_library().arl2_kv_frames(h)


def arl2_kv_device_bytes(h) -> int:
    return load_library().arl2_kv_device_bytes(h)


def arl2_kv_last_error(h) -> int:
    return load_library().arl2_kv_last_error(h)


def arl2_kv_query_strided(h, q, k, v, ld, o, stream=None) -> None:
    _check(load_library().arl2_kv_query_strided(h, _ptr(q), _ptr(k), _ptr(v), int(ld), _ptr(o), _stream(stream)),
           "arl2_kv_query_strided")


def arl2_kv_commit_strided(h, q, k, v, ld, o, stream=None) -> None:
    _check(load_library().arl2_kv_commit_strided(h, _ptr(q), _ptr(k), _ptr(v), int(ld), _ptr(o), _stream(stream)),
           "arl2_kv_commit_strided")


def arl2_kv_destroy(h) -> None:
    _check(load_library().arl2_kv_destroy(h), "arl2_kv_destroy")


def _ref(struct):
    return None if struct is None else ctypes.addressof(struct)


def arl2_qk_norm_rope(prep: arl2_qk_prep, dtype, heads, kv_heads, head_dim, tokens, q, k, ld, pos, q_out, k_out,
                      ld_out, stream=None) -> None:
    _check(load_library().arl2_qk_norm_rope(_ref(prep), dtype, heads, kv_heads, head_dim, tokens, _ptr(q), _ptr(k), ld,
                                            _ptr(pos), _ptr(q_out), _ptr(k_out), ld_out, _stream(stream)),
           "arl2_qk_norm_rope")


def arl2_paged_init(cfg: arl2_paged_config, k_pool, v_pool, stream=None) -> int:
    h = _VP()
    _check(load_library().arl2_paged_init(ctypes.byref(cfg), _ptr(k_pool), _ptr(v_pool), _stream(stream),
                                          ctypes.byref(h)), "arl2_paged_init")
    return h.value


def arl2_paged_append(h, batch: arl2_paged_batch, prep, q, k, v, ld, pos, q_out, stream=None) -> None:
    _check(load_library().arl2_paged_append(h, _ref(batch), _ref(prep), _ptr(q), _ptr(k), _ptr(v), ld, _ptr(pos),
                                            _ptr(q_out), _stream(stream)), "arl2_paged_append")


def arl2_paged_attend(h, batch: arl2_paged_batch, q, ld_q, mask_block, o, lse, stream=None) -> None:
    _check(load_library().arl2_paged_attend(h, _ref(batch), _ptr(q), ld_q, mask_block, _ptr(o), _ptr(lse),
                                            _stream(stream)), "arl2_paged_attend")


def arl2_paged_weights(h, batch: arl2_paged_batch, q, ld_q, mask_block, lse, decay, w_in, w_out, w_ld,
                       stream=None) -> None:
    _check(load_library().arl2_paged_weights(h, _ref(batch), _ptr(q), ld_q, mask_block, _ptr(lse), decay, _ptr(w_in),
                                             _ptr(w_out), w_ld, _stream(stream)), "arl2_paged_weights")


def arl2_paged_evict(h, batch: arl2_paged_batch, w_in, w_ld, budget, sink, recent, dst_pages, dst_ld, w_out, kept,
                     kv_len_out, stream=None) -> None:
    _check(load_library().arl2_paged_evict(h, _ref(batch), _ptr(w_in), w_ld, budget, sink, recent, _ptr(dst_pages),
                                           dst_ld, _ptr(w_out), _ptr(kept), _ptr(kv_len_out), _stream(stream)),
           "arl2_paged_evict")


def arl2_paged_last_error(h) -> int:
    return load_library().arl2_paged_last_error(h)


def arl2_paged_device_bytes(h) -> int:
    return load_library().arl2_paged_device_bytes(h)


def arl2_paged_set_wait_limit(h, limit_ns: int) -> None:
    _check(load_library().arl2_paged_set_wait_limit(h, limit_ns), "arl2_paged_set_wait_limit")


def arl2_paged_destroy(h) -> None:
    _check(load_library().arl2_paged_destroy(h), "arl2_paged_destroy")


def arl2_block_init(cfg: arl2_config, w_qkv, w_o, w_gate, phi_q, phi_k, phi_v, stream=None) -> int:
    h = _VP()
    _check(load_library().arl2_block_init(ctypes.byref(cfg), _ptr(w_qkv), _ptr(w_o), _ptr(w_gate), _ptr(phi_q),
                                          _ptr(phi_k), _ptr(phi_v), _stream(stream), ctypes.byref(h)),
           "arl2_block_init")
    return h.value


def arl2_block_query(h, x, y, stream=None) -> None:
    _check(load_library().arl2_block_query(h, _ptr(x), _ptr(y), _stream(stream)), "arl2_block_query")


def arl2_block_commit(h, x, y, stream=None) -> None:
    _check(load_library().arl2_block_commit(h, _ptr(x), _ptr(y), _stream(stream)), "arl2_block_commit")


def arl2_block_layer(h) -> int | None:
    return load_library().arl2_block_layer(h)


def arl2_block_destroy(h) -> None:
    _check(load_library().arl2_block_destroy(h), "arl2_block_destroy")


def arl2_state_write_noalloc(cfg: arl2_config, k, v, phi_k, phi_v, S_prev, alpha, beta, S_next, dev_error,
                             stream=None) -> None:
    """One frame's state write with no handle and no device allocation (its
    work space is the library's static scratch array); ``dev_error`` is a
    device uint32 that a kernel's timed-out wait sets."""
    _check(load_library().arl2_state_write_noalloc(ctypes.byref(cfg), _ptr(k), _ptr(v), _ptr(phi_k), _ptr(phi_v),
                                                   _ptr(S_prev), _ptr(alpha), _ptr(beta), _ptr(S_next),
                                                   _ptr(dev_error), _stream(stream)), "arl2_state_write_noalloc")


def arl2_selftest_wait_timeout(limit_ns: int, stream=None) -> int:
    return load_library().arl2_selftest_wait_timeout(limit_ns, _stream(stream))


def arl2_gemm_bf16(a, b, c, m, n, k, lda=None, ldb=None, ldc=None, stream=None) -> None:
    """C[m, n] = A[m, k] B[k, n] on bf16 device tensors (row-major; leading
    dimensions default to k, n and n)."""
    _check(load_library().arl2_gemm_bf16(_ptr(a), lda or k, _ptr(b), ldb or n, _ptr(c), ldc or n, m, n, k,
                                         _stream(stream)), "arl2_gemm_bf16")


def arl2_attn_partition(batch, heads, q_len, kv_len, pairs, max_segs=1024):
    """The attention kernel's work partition (host only): a list per pair of
    segments (slab, block, j0, j1, n_contrib)."""
    segs = (ctypes.c_int32 * (5 * max_segs))()
    first = (ctypes.c_int32 * 97)()
    n_segs, n_pairs = ctypes.c_int(0), ctypes.c_int(0)
    _check(load_library().arl2_attn_partition(batch, heads, q_len, kv_len, pairs, ctypes.cast(segs, ctypes.c_void_p).value,
                                              max_segs, ctypes.cast(first, ctypes.c_void_p).value,
                                              ctypes.addressof(n_segs), ctypes.addressof(n_pairs)), "arl2_attn_partition")
    out = []
    for c in range(n_pairs.value):
        out.append([tuple(segs[5 * i:5 * i + 5]) for i in range(first[c], first[c + 1])])
    return out


def arl2_selftest_exp2(x, y, stream=None) -> None:
    _check(load_library().arl2_selftest_exp2(_ptr(x), _ptr(y), x.numel(), _stream(stream)), "arl2_selftest_exp2")


def arl2_status_string(status: int) -> str:
    return load_library().arl2_status_string(status).decode()


def arl2_abi_version() -> int:
    return load_library().arl2_abi_version()


def arl2_debug_bounds_enabled() -> bool:
    """Whether the loaded library is the debug build (index checks in its kernels)."""
    return bool(load_library().arl2_debug_bounds_enabled())


# ---------------------------------------------------------------- convenience wrappers
def _torch_dtype(dtype: int):
    import torch
    return torch.float32 if dtype == ARL2_F32 else torch.bfloat16


class HybridLayer:
    """One ARL2 hybrid attention layer over B streams (a handle of the C ABI)."""

    def __init__(self, batch, heads, head_dim, tokens, dtype, phi_q, phi_k, phi_v, *,
                 softmax_scale=0.0, corr_scale=-1.0, flags=0, stream=None):
        self.cfg = make_config(batch, heads, head_dim, tokens, dtype, softmax_scale, corr_scale, flags)
        self.handle = arl2_state_init(self.cfg, phi_q, phi_k, phi_v, stream)

    @property
    def out_shape(self):
        c = self.cfg
        return (c.batch, c.tokens_per_frame, c.heads, c.head_dim)

    def _out(self, like):
        import torch
        return torch.empty(self.out_shape, dtype=_torch_dtype(self.cfg.dtype), device=like.device)

    def query(self, q, k, v, o=None, stream=None):
        o = self._out(q) if o is None else o
        arl2_frame_query(self.handle, q, k, v, o, stream)
        return o

    def commit(self, q, k, v, alpha, beta, o=None, stream=None):
        o = self._out(q) if o is None else o
        arl2_frame_commit(self.handle, q, k, v, alpha, beta, o, stream)
        return o

    def token_query(self, q, k, v, alpha_tok, beta, o=None, stream=None):
        """Token-level access: token t reads the state the earlier tokens of
        this pass left; the handle's state is not written."""
        o = self._out(q) if o is None else o
        arl2_token_query(self.handle, q, k, v, alpha_tok, beta, o, stream)
        return o

    def token_commit(self, q, k, v, alpha_tok, beta, o=None, stream=None):
        """Token-level access on the clean pass: the state after the frame's
        last token becomes the handle's state."""
        o = self._out(q) if o is None else o
        arl2_token_commit(self.handle, q, k, v, alpha_tok, beta, o, stream)
        return o

    def state(self, stream=None):
        import torch
        c = self.cfg
        dst = torch.empty((c.batch, c.heads, c.head_dim, c.head_dim), dtype=torch.float32, device="cuda")
        arl2_state_get(self.handle, dst, stream)
        return dst

    @property
    def frame(self) -> int:
        return arl2_state_get(self.handle, None)

    def set_state(self, S, frame: int, stream=None):
        arl2_state_set(self.handle, S, frame, stream)

    def last_error(self) -> int:
        return arl2_last_error(self.handle)

    def device_bytes(self) -> int:
        return arl2_state_device_bytes(self.handle)

    def close(self):
        if self.handle:
            arl2_state_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class KVLayer:
    """A softmax layer with a growing per-frame KV cache (a handle of the C ABI)."""

    def __init__(self, batch, heads, head_dim, tokens, dtype, max_frames, *, softmax_scale=0.0, stream=None):
        self.cfg = make_config(batch, heads, head_dim, tokens, dtype, softmax_scale, -1.0, 0)
        self.handle = arl2_kv_init(self.cfg, max_frames, stream)

    def _out(self, like):
        import torch
        c = self.cfg
        return torch.empty((c.batch, c.tokens_per_frame, c.heads, c.head_dim), dtype=_torch_dtype(c.dtype),
                           device=like.device)

    def query(self, q, k, v, o=None, stream=None):
        o = self._out(q) if o is None else o
        arl2_kv_query(self.handle, q, k, v, o, stream)
        return o

    def commit(self, q, k, v, o=None, stream=None):
        o = self._out(q) if o is None else o
        arl2_kv_commit(self.handle, q, k, v, o, stream)
        return o

    @property
    def frames(self) -> int:
        return arl2_kv_frames(self.handle)

    def last_error(self) -> int:
        return arl2_kv_last_error(self.handle)

    def device_bytes(self) -> int:
        return arl2_kv_device_bytes(self.handle)

    def close(self):
        if self.handle:
            arl2_kv_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _bad_rows(name, t, h, d, dtype, index):
    return ValueError(f"{name}: expected [tokens, {h}, {d}] of {dtype} on device {index} with contiguous token rows, got "
                      f"{list(t.shape)} of {t.dtype} on {t.device} with strides {list(t.stride())}")


def _not_on_gpu(name, t):
    return ValueError(f"{name}: expected a CUDA tensor, got one on {t.device}")


def _token_rows(d, dtype, index, tensors):
    """The common pitch of [tokens, heads, head_dim] views in elements (0: each
    contiguous), and their tokens, of (name, tensor, heads) triples; raises where
    the library cannot read them."""
    ld = tokens = None
    dense = True
    for name, t, h in tensors:
        if t.dim() != 3 or t.dtype != dtype or t.get_device() != index:
            raise _bad_rows(name, t, h, d, dtype, index)
        n, th, td = t.shape
        s0, s1, s2 = t.stride()
        if th != h or td != d or s2 != 1 or (s1 != d and h > 1):
            raise _bad_rows(name, t, h, d, dtype, index)
        if tokens is None:
            tokens = n
        elif n != tokens:
            raise ValueError(f"{name}: {n} tokens, expected {tokens}")
        if n > 1:
            dense = dense and s0 == h * d
            if ld is None:
                ld = s0
            elif ld != s0:
                ld = -1
    if dense:
        return 0, tokens
    if ld < 0:
        raise ValueError("strided views must have one pitch")
    if ld < max(h for _, _, h in tensors) * d:  # (0, of a view broadcast over tokens, would read as contiguous)
        raise ValueError(f"token rows {ld} elements apart overlap")
    return ld, tokens


def _plain(name, t, dtype, index, shape=None):
    if t.dtype != dtype or t.get_device() != index or not t.is_contiguous() or (shape is not None and t.shape != shape):
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor{'' if shape is None else f' {list(shape)}'} on "
                         f"device {index}, got {list(t.shape)} of {t.dtype} on {t.device}")
    return t


def _stream_of(index, stream):
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """An output that a call on `stream` writes: from that stream's memory, since a block that the current stream gave
    back may still have writes of its own to come."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        raw = _stream_of(None, stream)
        stream = torch.cuda.ExternalStream(raw, device=device) if raw else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


class QKPrep:
    """Norm and rotation of queries and keys: norm weights (None, None: no
    norm) and up to three position axes."""

    def __init__(self, axis_dims, theta=10000.0, halves=False, eps=1e-6, w_q=None, w_k=None):
        axis_dims = list(axis_dims)
        if len(axis_dims) > 3:
            raise ValueError("at most three axes")
        if (w_q is None) != (w_k is None):
            raise ValueError("norm weights come in pairs")
        for name, w in (("w_q", w_q), ("w_k", w_k)):
            if w is not None and (w.dim() != 1 or not w.is_contiguous()):
                raise ValueError(f"{name}: expected contiguous [head_dim]")
        self.w_q, self.w_k, self.n_axes = w_q, w_k, len(axis_dims)
        self.struct = arl2_qk_prep(len(axis_dims), (ctypes.c_int32 * 3)(*axis_dims), int(halves), theta, eps,
                                   _ptr(w_q), _ptr(w_k))

    def _check(self, d, dtype, index, tokens, pos):
        import torch
        if self.w_q is not None:
            _plain("w_q", self.w_q, dtype, index, (d,))
            _plain("w_k", self.w_k, dtype, index, (d,))
        if self.n_axes:
            if pos is None:
                raise ValueError("pos: the prep's axes need positions")
            _plain("pos", pos, torch.int32, index, (tokens, self.n_axes))


def qk_norm_rope(prep: QKPrep, q, k, pos=None, q_out=None, k_out=None, stream=None):
    """Norm and rotate queries [tokens, heads, d] and keys [tokens, kv_heads, d]
    (views of one pitch, or contiguous) in one pass; returns (q_out, k_out).
    Streams as PagedKVLayer's."""
    import torch
    tokens, h, d = q.shape
    hk, dtype, index = k.shape[1], q.dtype, q.get_device()
    if index < 0:
        raise _not_on_gpu("q", q)
    ld, tokens = _token_rows(d, dtype, index, (("q", q, h), ("k", k, hk)))
    prep._check(d, dtype, index, tokens, pos)
    q_out = _empty((tokens, h, d), dtype, q.device, stream) if q_out is None else q_out
    k_out = _empty((tokens, hk, d), dtype, q.device, stream) if k_out is None else k_out
    ld_out, n = _token_rows(d, dtype, index, (("q_out", q_out, h), ("k_out", k_out, hk)))
    if n != tokens:
        raise ValueError("outputs: as many tokens as the inputs")
    args = (prep.struct, _abi_dtype(dtype), h, hk, d, tokens, q, k, ld, pos if prep.n_axes else None, q_out, k_out,
            ld_out, _stream_of(index, stream))
    if torch._C._cuda_getDevice() == index:
        arl2_qk_norm_rope(*args)
    else:
        with torch.cuda.device(index):
            arl2_qk_norm_rope(*args)
    return q_out, k_out


def _abi_dtype(dtype):
    import torch
    if dtype == torch.bfloat16:
        return ARL2_BF16
    if dtype == torch.float32:
        return ARL2_F32
    raise ValueError(f"float32 or bfloat16 tensors, got {dtype}")


class PagedBatch:
    """The streams of one call: q_start int32 [n + 1], kv_len int32 [n], pages
    int32 [n, pages_ld] on the device, and the host's bounds of their values.
    The tensors may be rewritten between calls (and between replays of a graph)."""

    def __init__(self, q_start, kv_len, pages, *, tokens, max_q, max_kv):
        import torch
        n = kv_len.shape[0]
        if pages.dim() != 2 or pages.shape[0] != n:
            raise ValueError("pages: expected [streams, pages]")
        index = kv_len.get_device()
        _plain("kv_len", kv_len, torch.int32, index, (n,))
        _plain("q_start", q_start, torch.int32, index, (n + 1,))
        _plain("pages", pages, torch.int32, index)
        self.q_start, self.kv_len, self.pages = q_start, kv_len, pages
        self.tokens, self.index = tokens, index
        self.struct = arl2_paged_batch(n, tokens, max_q, max_kv, pages.shape[1], _ptr(q_start), _ptr(kv_len),
                                       _ptr(pages))


class PagedKVLayer:
    """A softmax layer on a paged KV cache (a handle of the C ABI).  The pools
    are [n_pages, kv_heads, page_size, head_dim]; the layer keeps them alive.

    Calls run on the current stream, or on ``stream`` (a torch stream or its raw
    number): its work so far must include what the inputs need, and it may read
    and write them until it has passed the call.  Outputs that a call allocates
    belong to that stream: another one waits for it before it reads them, and
    ``record_stream`` tells the allocator where they are used last.  Rows that
    belong to no stream of the batch, and streams that the library leaves out
    (``last_error``), leave an output of attend, weights or append as it was."""

    def __init__(self, heads, kv_heads, head_dim, dtype, k_pool, v_pool, *, softmax_scale=0.0, stream=None):
        import torch
        self.handle = None
        self.dtype, self.device, self.index = _torch_dtype(dtype), k_pool.device, k_pool.get_device()
        if k_pool.dim() != 4 or k_pool.shape[1] != kv_heads or k_pool.shape[3] != head_dim:
            raise ValueError("k_pool: expected [n_pages, kv_heads, page_size, head_dim]")
        if self.index < 0:
            raise _not_on_gpu("k_pool", k_pool)
        _plain("k_pool", k_pool, self.dtype, self.index)
        _plain("v_pool", v_pool, self.dtype, self.index, k_pool.shape)
        self.k_pool, self.v_pool = k_pool, v_pool
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.cfg = arl2_paged_config(heads, kv_heads, head_dim, k_pool.shape[2], k_pool.shape[0], dtype, softmax_scale)
        with torch.cuda.device(self.device):
            self.handle = arl2_paged_init(self.cfg, k_pool, v_pool, _stream_of(self.index, stream))

    def _rows(self, batch, *tensors):
        """The rows' pitch; checks them against the batch, and the batch's device."""
        ld, tokens = _token_rows(self.head_dim, self.dtype, self.index, tensors)
        if tokens != batch.tokens or batch.index != self.index:
            raise ValueError(f"{tokens} token rows on device {self.index}; the batch has {batch.tokens} on {batch.index}")
        return ld

    def append(self, batch, k, v, *, q=None, prep=None, pos=None, q_out=None, stream=None):
        """Store the new tokens' K and V; with a prep, K normed and rotated, and
        q's turned rows are returned (q_out)."""
        if q is None:
            if q_out is not None:
                raise ValueError("q_out without q")
            ld = self._rows(batch, ("k", k, self.kv_heads), ("v", v, self.kv_heads))
        else:
            if prep is None:
                raise ValueError("q without a prep")
            ld = self._rows(batch, ("q", q, self.heads), ("k", k, self.kv_heads), ("v", v, self.kv_heads))
            if q_out is None:
                q_out = _empty((batch.tokens, self.heads, self.head_dim), self.dtype, self.device, stream)
            elif self._rows(batch, ("q_out", q_out, self.heads)):
                raise ValueError("q_out must be contiguous")
        if prep is not None:
            prep._check(self.head_dim, self.dtype, self.index, batch.tokens, pos)
        arl2_paged_append(self.handle, batch.struct, None if prep is None else prep.struct, q, k, v, ld,
                          pos if prep is not None and prep.n_axes else None, q_out, _stream_of(self.index, stream))
        return q_out

    def attend(self, batch, q, *, mask_block=0, o=None, lse=None, stream=None):
        """(O, lse) of the new tokens over their streams' cached keys."""
        import torch
        ld = self._rows(batch, ("q", q, self.heads))
        if o is None:
            o = _empty((batch.tokens, self.heads, self.head_dim), self.dtype, self.device, stream)
        elif self._rows(batch, ("o", o, self.heads)):
            raise ValueError("o must be contiguous")
        if lse is None:
            lse = _empty((batch.tokens, self.heads), torch.float32, self.device, stream)
        else:
            _plain("lse", lse, torch.float32, self.index, (batch.tokens, self.heads))
        arl2_paged_attend(self.handle, batch.struct, q, ld, mask_block, o, lse, _stream_of(self.index, stream))
        return o, lse

    def _weights_shape(self, batch, w):
        import torch
        n = batch.struct.n_seqs
        if w.dim() != 3 or w.shape[0] != n or w.shape[1] != self.kv_heads or batch.index != self.index:
            raise ValueError(f"w: expected [{n}, {self.kv_heads}, keys], got {list(w.shape)}")
        _plain("w", w, torch.float32, self.index)
        return n

    def weights(self, batch, q, lse, w, *, mask_block=0, decay=1.0, w_out=None, stream=None):
        """The cached keys' accumulated attention weights after the new tokens
        (w_out may be w)."""
        import torch
        ld = self._rows(batch, ("q", q, self.heads))
        self._weights_shape(batch, w)
        _plain("lse", lse, torch.float32, self.index, (batch.tokens, self.heads))
        if w_out is None:
            w_out = _empty(w.shape, torch.float32, self.device, stream)
        else:
            _plain("w_out", w_out, torch.float32, self.index, w.shape)
        arl2_paged_weights(self.handle, batch.struct, q, ld, mask_block, lse, decay, w, w_out, w.shape[2],
                           _stream_of(self.index, stream))
        return w_out

    def evict(self, batch, w, dst_pages, *, budget, sink=0, recent=0, stream=None):
        """Cut the streams to at most `budget` keys, moved to dst_pages; returns
        (kv_len, w, kept) of the streams in their new pages."""
        import torch
        n = self._weights_shape(batch, w)
        if dst_pages.dim() != 2 or dst_pages.shape[0] != n:
            raise ValueError("dst_pages: expected [streams, pages]")
        _plain("dst_pages", dst_pages, torch.int32, self.index)
        w_out = _empty(w.shape, torch.float32, self.device, stream)
        kept = _empty((n, self.kv_heads, budget), torch.int32, self.device, stream)
        kv_len = _empty((n,), torch.int32, self.device, stream)
        arl2_paged_evict(self.handle, batch.struct, w, w.shape[2], budget, sink, recent, dst_pages, dst_pages.shape[1],
                         w_out, kept, kv_len, _stream_of(self.index, stream))
        return kv_len, w_out, kept

    def last_error(self) -> int:
        return arl2_paged_last_error(self.handle)

    def device_bytes(self) -> int:
        return arl2_paged_device_bytes(self.handle)

    def close(self):
        if self.handle:
            arl2_paged_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class HybridBlock:
    """A hybrid attention block: X W_qkv -> hybrid layer -> O W_o, with the
    commit's gates from X W_gate (a handle of the C ABI; bf16, head_dim 128)."""

    def __init__(self, batch, heads, tokens, w_qkv, w_o, w_gate, phi_q, phi_k, phi_v, *, softmax_scale=0.0,
                 corr_scale=-1.0, stream=None):
        self.cfg = make_config(batch, heads, 128, tokens, ARL2_BF16, softmax_scale, corr_scale, 0)
        self.handle = arl2_block_init(self.cfg, w_qkv, w_o, w_gate, phi_q, phi_k, phi_v, stream)

    def _out(self, like):
        import torch
        return torch.empty_like(like)

    def query(self, x, y=None, stream=None):
        y = self._out(x) if y is None else y
        arl2_block_query(self.handle, x, y, stream)
        return y

    def commit(self, x, y=None, stream=None):
        y = self._out(x) if y is None else y
        arl2_block_commit(self.handle, x, y, stream)
        return y

    def state(self, stream=None):
        import torch
        c = self.cfg
        dst = torch.empty((c.batch, c.heads, c.head_dim, c.head_dim), dtype=torch.float32, device="cuda")
        arl2_state_get(arl2_block_layer(self.handle), dst, stream)
        return dst

    def last_error(self) -> int:
        return arl2_last_error(arl2_block_layer(self.handle))

    def close(self):
        if self.handle:
            arl2_block_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
