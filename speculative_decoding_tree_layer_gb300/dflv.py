"""ctypes binding of libdflv (include/dflv.h) -- argument marshalling only.

Every function keeps the C name and argument order.  Tensor arguments are
torch CUDA tensors (their ``data_ptr()`` is passed) or plain integers
(device addresses); ``stream`` defaults to torch's current stream.  Each call
returns the library's status code; ``check()`` turns a non-zero code into an
exception.  Every step of the tree-verify path runs in the CUDA library: this
module computes nothing, and there is no CPU fallback -- if the library is
not built, the first call raises.
"""
from __future__ import annotations

import ctypes
import os
import re

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libdflv.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "dflv.h")

DFLV_OK, DFLV_ERR_INVALID_ARG, DFLV_ERR_TOPOLOGY, DFLV_ERR_UNSUPPORTED, DFLV_ERR_CAPACITY, DFLV_ERR_CUDA = range(6)
DFLV_DEV_TOPOLOGY, DFLV_DEV_CAPACITY, DFLV_DEV_PATH, DFLV_DEV_TIMEOUT = 1, 2, 4, 8
DFLV_DEV_PAGE, DFLV_DEV_SAMPLE = 16, 32
DFLV_KV_Q8_0, DFLV_KV_Q4_0, DFLV_KV_F32, DFLV_KV_Q8_0_Q4_0, DFLV_KV_Q4_0_Q8_0, DFLV_KV_TQ3_0 = 0, 1, 2, 3, 4, 5
DFLV_KV_BF16, DFLV_KV_F16 = 6, 7
DFLV_LOGITS_F32, DFLV_LOGITS_BF16, DFLV_LOGITS_F16 = 0, 1, 2
DFLV_FLAG_EARLY_PREFETCH = 1
DFLV_MAX_COMMIT_GDN_LAYERS, DFLV_MAX_COMMIT_ATTN_LAYERS = 128, 64
DFLV_MAX_CONV_LAYERS = 128

_c_i32 = ctypes.c_int32
_vp = ctypes.c_void_p


class dflv_gdn_desc(ctypes.Structure):
    _fields_ = [("B", _c_i32), ("N_max", _c_i32), ("Hk", _c_i32), ("Hv", _c_i32), ("dk", _c_i32), ("dv", _c_i32),
                ("flags", ctypes.c_uint32)]


class dflv_gdn_factors(ctypes.Structure):
    _fields_ = [("u", _vp), ("g", _vp), ("kcopy", _vp)]


class dflv_attn_desc(ctypes.Structure):
    _fields_ = [("B", _c_i32), ("N_max", _c_i32), ("Hq", _c_i32), ("Hkv", _c_i32), ("D", _c_i32),
                ("cap", _c_i32), ("window", _c_i32), ("type", ctypes.c_int), ("scale", ctypes.c_float),
                ("flags", ctypes.c_uint32)]


class dflv_kv_layer(ctypes.Structure):
    _fields_ = [("kq", _vp), ("vq", _vp), ("ks", _vp), ("vs", _vp)]


class dflv_conv_desc(ctypes.Structure):
    _fields_ = [("B", _c_i32), ("N_max", _c_i32), ("C", _c_i32), ("K", _c_i32), ("flags", ctypes.c_uint32)]


class dflv_ddtree_desc(ctypes.Structure):
    _fields_ = [("B", _c_i32), ("D", _c_i32), ("V", _c_i32), ("K", _c_i32), ("budget", _c_i32),
                ("tau", ctypes.c_float), ("flags", ctypes.c_uint32)]


class dflv_pages_desc(ctypes.Structure):
    _fields_ = [("B", _c_i32), ("N_max", _c_i32), ("page", _c_i32), ("n_pages", _c_i32), ("max_pages", _c_i32),
                ("flags", ctypes.c_uint32)]


class dflv_paged_kv_desc(ctypes.Structure):
    _fields_ = [("B", _c_i32), ("N_max", _c_i32), ("Hkv", _c_i32), ("D", _c_i32), ("page", _c_i32),
                ("n_pages", _c_i32), ("type", ctypes.c_int), ("kv_stride", _c_i32), ("flags", ctypes.c_uint32)]


class dflv_prefix_attn_desc(ctypes.Structure):
    _fields_ = [("B", _c_i32), ("N_max", _c_i32), ("Hq", _c_i32), ("Hkv", _c_i32), ("D", _c_i32), ("page", _c_i32),
                ("n_pages", _c_i32), ("max_pages", _c_i32), ("max_prefix_pages", _c_i32), ("type", ctypes.c_int),
                ("scale", ctypes.c_float), ("q_stride", _c_i32), ("flags", ctypes.c_uint32)]


class dflv_sample_desc(ctypes.Structure):
    _fields_ = [("B", _c_i32), ("N_max", _c_i32), ("V", _c_i32), ("type", ctypes.c_int), ("ld", ctypes.c_int64),
                ("flags", ctypes.c_uint32)]


class DflvError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} (status {code})")


_lib = None


def load():
    """Loads libdflv.so; raises if it has not been built (no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libdflv.so is not built ({LIB_PATH} missing); run __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    P = _vp
    S = ctypes.c_size_t
    lib.dflv_tree_gdn_verify.argtypes = [ctypes.POINTER(dflv_gdn_desc)] + [P] * 9 + \
        [ctypes.POINTER(dflv_gdn_factors), P, P, S, P]
    lib.dflv_tree_gdn_verify_pending.argtypes = [ctypes.POINTER(dflv_gdn_desc)] + [P] * 8 + \
        [ctypes.POINTER(dflv_gdn_factors), P, P, P, ctypes.POINTER(dflv_gdn_factors), P, P, S, P]
    lib.dflv_tree_attn_verify.argtypes = [ctypes.POINTER(dflv_attn_desc)] + [P] * 6 + \
        [ctypes.POINTER(dflv_kv_layer), P, P, P, S, P]
    lib.dflv_tree_attn_verify_noalloc.argtypes = [ctypes.POINTER(dflv_attn_desc)] + [P] * 6 + \
        [ctypes.POINTER(dflv_kv_layer), P, P, P]
    lib.dflv_accept_greedy.argtypes = [_c_i32, _c_i32, _c_i32] + [P] * 10
    lib.dflv_commit_rollback.argtypes = [ctypes.POINTER(dflv_gdn_desc), _c_i32, P, ctypes.POINTER(dflv_gdn_factors),
                                         ctypes.POINTER(dflv_attn_desc), _c_i32, ctypes.POINTER(dflv_kv_layer),
                                         P, P, P, P, P]
    lib.dflv_tree_conv_verify.argtypes = [ctypes.POINTER(dflv_conv_desc)] + [P] * 7 + [P]
    lib.dflv_conv_commit.argtypes = [ctypes.POINTER(dflv_conv_desc), _c_i32, P, P, P, P, P, P]
    lib.dflv_ddtree_build.argtypes = [ctypes.POINTER(dflv_ddtree_desc)] + [P] * 10
    lib.dflv_block_tables_grow.argtypes = [ctypes.POINTER(dflv_pages_desc)] + [P] * 9
    lib.dflv_block_tables_release.argtypes = [ctypes.POINTER(dflv_pages_desc)] + [P] * 7
    lib.dflv_paged_kv_append.argtypes = [ctypes.POINTER(dflv_paged_kv_desc), P, P, P, ctypes.POINTER(dflv_kv_layer),
                                         P, P]
    lib.dflv_paged_kv_commit.argtypes = [ctypes.POINTER(dflv_paged_kv_desc), _c_i32, ctypes.POINTER(dflv_kv_layer)] + \
        [P] * 6
    lib.dflv_prefix_attn_verify.argtypes = [ctypes.POINTER(dflv_prefix_attn_desc)] + [P] * 7 + \
        [ctypes.POINTER(dflv_kv_layer), P, P, P, S, P]
    lib.dflv_prefix_attn_workspace_size.argtypes = [ctypes.POINTER(dflv_prefix_attn_desc)]
    lib.dflv_prefix_attn_workspace_size.restype = S
    lib.dflv_sample.argtypes = [ctypes.POINTER(dflv_sample_desc)] + [P] * 11
    lib.dflv_accept_sampled.argtypes = [ctypes.POINTER(dflv_sample_desc)] + [P] * 16
    lib.dflv_gdn_workspace_size.argtypes = [ctypes.POINTER(dflv_gdn_desc)]
    lib.dflv_gdn_workspace_size.restype = S
    lib.dflv_attn_workspace_size.argtypes = [ctypes.POINTER(dflv_attn_desc)]
    lib.dflv_attn_workspace_size.restype = S
    lib.dflv_status_string.argtypes = [ctypes.c_int]
    lib.dflv_status_string.restype = ctypes.c_char_p
    for f in ("dflv_tree_gdn_verify", "dflv_tree_gdn_verify_pending", "dflv_tree_attn_verify",
              "dflv_tree_attn_verify_noalloc", "dflv_accept_greedy",
              "dflv_commit_rollback", "dflv_tree_conv_verify", "dflv_conv_commit", "dflv_ddtree_build",
              "dflv_block_tables_grow", "dflv_block_tables_release", "dflv_paged_kv_append", "dflv_paged_kv_commit",
              "dflv_prefix_attn_verify", "dflv_sample", "dflv_accept_sampled"):
        getattr(lib, f).restype = ctypes.c_int
    _lib = lib
    return lib


def header_symbols():
    """Names of the functions include/dflv.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"^[A-Za-z_][\w \*]*?\b(dflv_\w+)\s*\(", text, flags=re.M)))


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s):
    if s is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def status_string(code: int) -> str:
    return load().dflv_status_string(int(code)).decode()


def check(code: int, where: str = "dflv"):
    if code != DFLV_OK:
        raise DflvError(code, where)
    return code


# ---------------------------------------------------------------- structs from tensors
def gdn_desc(B, N_max, Hk, Hv, dk, dv, flags=0):
    return dflv_gdn_desc(B, N_max, Hk, Hv, dk, dv, flags)


def gdn_factors(u, g, kcopy):
    """The factor buffers' pointers.  The struct holds references to the
    tensors it was made from, so that buffers passed as temporaries stay
    allocated for as long as the struct is in use."""
    f = dflv_gdn_factors(_ptr(u), _ptr(g), _ptr(kcopy))
    f._tensors = (u, g, kcopy)
    return f


def attn_desc(B, N_max, Hq, Hkv, D, cap, window, kv_type, scale, flags=0):
    return dflv_attn_desc(B, N_max, Hq, Hkv, D, cap, window, kv_type, scale, flags)


def kv_layer(kq, vq, ks=None, vs=None):
    """One layer's cache planes; holds references to the tensors, as
    gdn_factors does."""
    c = dflv_kv_layer(_ptr(kq), _ptr(vq), _ptr(ks), _ptr(vs))
    c._tensors = (kq, vq, ks, vs)
    return c


# ---------------------------------------------------------------- the C ABI
def dflv_tree_gdn_verify(desc, parent, n_nodes, q, k, v, beta, log_alpha, state, out, factors,
                         status_dev, workspace=None, ws_bytes=0, stream=None) -> int:
    return load().dflv_tree_gdn_verify(
        ctypes.byref(desc), _ptr(parent), _ptr(n_nodes), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
        _ptr(log_alpha), _ptr(state), _ptr(out), ctypes.byref(factors), _ptr(status_dev),
        _ptr(workspace), ws_bytes, _stream(stream))


def dflv_tree_gdn_verify_pending(desc, parent, n_nodes, q, k, v, beta, log_alpha, state, pending, pending_path,
                                 pending_len, out, factors, status_dev, workspace=None, ws_bytes=0,
                                 stream=None) -> int:
    return load().dflv_tree_gdn_verify_pending(
        ctypes.byref(desc), _ptr(parent), _ptr(n_nodes), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
        _ptr(log_alpha), _ptr(state), ctypes.byref(pending), _ptr(pending_path), _ptr(pending_len), _ptr(out),
        ctypes.byref(factors), _ptr(status_dev), _ptr(workspace), ws_bytes, _stream(stream))


def dflv_tree_attn_verify(desc, parent, n_nodes, n_past, q, k_new, v_new, cache, out, status_dev,
                          workspace=None, ws_bytes=0, stream=None) -> int:
    return load().dflv_tree_attn_verify(
        ctypes.byref(desc), _ptr(parent), _ptr(n_nodes), _ptr(n_past), _ptr(q), _ptr(k_new),
        _ptr(v_new), ctypes.byref(cache), _ptr(out), _ptr(status_dev), _ptr(workspace), ws_bytes,
        _stream(stream))


def dflv_tree_attn_verify_noalloc(desc, parent, n_nodes, n_past, q, k_new, v_new, cache, out, status_dev,
                                  stream=None) -> int:
    return load().dflv_tree_attn_verify_noalloc(
        ctypes.byref(desc), _ptr(parent), _ptr(n_nodes), _ptr(n_past), _ptr(q), _ptr(k_new),
        _ptr(v_new), ctypes.byref(cache), _ptr(out), _ptr(status_dev), _stream(stream))


DFLV_NOALLOC_SCRATCH_BYTES = 16 << 20


def dflv_accept_greedy(B, N_max, vocab, logits, tokens, parent, n_nodes, path, path_len, next_token,
                       best, status_dev, stream=None) -> int:
    return load().dflv_accept_greedy(B, N_max, vocab, _ptr(logits), _ptr(tokens), _ptr(parent),
                                     _ptr(n_nodes), _ptr(path), _ptr(path_len), _ptr(next_token),
                                     _ptr(best), _ptr(status_dev), _stream(stream))


def dflv_commit_rollback(gdn, n_gdn, states, factors, attn, n_attn, caches, path, path_len, n_past,
                         status_dev, stream=None) -> int:
    """``states``: sequence of state tensors (or addresses), ``factors``:
    sequence of dflv_gdn_factors, ``caches``: sequence of dflv_kv_layer."""
    st = (ctypes.c_void_p * max(1, n_gdn))(*[_ptr(s) for s in states][:n_gdn])
    fa = (dflv_gdn_factors * max(1, n_gdn))(*list(factors)[:n_gdn])
    ca = (dflv_kv_layer * max(1, n_attn))(*list(caches)[:n_attn])
    return load().dflv_commit_rollback(
        ctypes.byref(gdn) if gdn is not None else None, n_gdn, ctypes.cast(st, ctypes.c_void_p), fa,
        ctypes.byref(attn) if attn is not None else None, n_attn, ca, _ptr(path), _ptr(path_len),
        _ptr(n_past), _ptr(status_dev), _stream(stream))


def conv_desc(B, N_max, C, K, flags=0):
    return dflv_conv_desc(B, N_max, C, K, flags)


def dflv_tree_conv_verify(desc, parent, n_nodes, x, conv_state, weight, out, status_dev, stream=None) -> int:
    return load().dflv_tree_conv_verify(ctypes.byref(desc), _ptr(parent), _ptr(n_nodes), _ptr(x), _ptr(conv_state),
                                        _ptr(weight), _ptr(out), _ptr(status_dev), _stream(stream))


def dflv_conv_commit(desc, n_layers, states, xs, path, path_len, status_dev, stream=None) -> int:
    """``states``, ``xs``: sequences of tensors (or addresses), one per layer."""
    st = (ctypes.c_void_p * max(1, n_layers))(*[_ptr(s) for s in states][:n_layers])
    xa = (ctypes.c_void_p * max(1, n_layers))(*[_ptr(x) for x in xs][:n_layers])
    return load().dflv_conv_commit(ctypes.byref(desc), n_layers, ctypes.cast(st, ctypes.c_void_p),
                                   ctypes.cast(xa, ctypes.c_void_p), _ptr(path), _ptr(path_len), _ptr(status_dev),
                                   _stream(stream))


def ddtree_desc(B, D, V, K, budget, tau=-1.0, flags=0):
    """tau < 0 (default): no pruning."""
    return dflv_ddtree_desc(B, D, V, K, budget, tau, flags)


def dflv_ddtree_build(desc, draft_logits, root_token, topk_tok, topk_logp, parent, tokens, n_nodes, score,
                      status_dev, stream=None) -> int:
    return load().dflv_ddtree_build(ctypes.byref(desc), _ptr(draft_logits), _ptr(root_token), _ptr(topk_tok),
                                    _ptr(topk_logp), _ptr(parent), _ptr(tokens), _ptr(n_nodes), _ptr(score),
                                    _ptr(status_dev), _stream(stream))


# ---------------------------------------------------------------- paged cache, shared prefix, sampling
class _Refused(Exception):
    pass


_kinds = None


def _types():
    """What the calls below need of torch, which is only imported once one of
    them is made: int32, float32, the 16-bit cache and the logits dtypes by type,
    whether CUDA is up, the current device's and its raw current stream's
    getters."""
    global _kinds
    if _kinds is None:
        import torch as t

        def raw(device):
            return t.cuda.current_stream(device).cuda_stream

        _kinds = (t.int32, t.float32, {DFLV_KV_BF16: (t.bfloat16, t.int16), DFLV_KV_F16: (t.float16, t.int16)},
                  {DFLV_LOGITS_F32: (t.float32, t.float32), DFLV_LOGITS_BF16: (t.bfloat16, t.int16),
                   DFLV_LOGITS_F16: (t.float16, t.int16)}, t.cuda.is_initialized,
                  getattr(t._C, "_cuda_getDevice", t.cuda.current_device),
                  getattr(t._C, "_cuda_getCurrentRawStream", raw))
    return _kinds


def _device():
    """The current device; -2, which no tensor is on, before CUDA is up."""
    kinds = _types()
    return kinds[5]() if kinds[4]() else -2


def _where(stream, dev):
    """The raw stream of a call."""
    if stream is None:
        return _kinds[6](dev) if dev >= 0 else _stream(None)
    return stream if stream.__class__ is int else stream.cuda_stream


def _arg(x, dtype, n, dev):
    """Address of an argument of n elements: an integer or None passes as it
    is (the library checks it); a tensor has to be a contiguous CUDA tensor on
    the current device, of the dtype, with at least n elements."""
    if x is None or x.__class__ is int:
        return x
    if x.dtype is not dtype or x.numel() < n or x.get_device() != dev or not x.is_contiguous():
        raise _Refused
    return x.data_ptr()


def _rows(x, dtypes, B, N, inner, stride, dev):
    """Address of [B][N][inner] of one of two dtypes (16-bit values may come as
    bit patterns) whose rows lie `stride` elements apart (0: inner): contiguous,
    or a view of wider rows with that stride."""
    if x is None or x.__class__ is int:
        return x
    if x.dtype not in dtypes or x.get_device() != dev:
        raise _Refused
    if stride == 0 or stride == inner:
        if x.numel() < B * N * inner or not x.is_contiguous():
            raise _Refused
        return x.data_ptr()
    shape, st = x.shape, x.stride()
    if len(shape) < 3 or not x.numel() or shape[0] < B or shape[1] != N or x[0, 0].numel() != inner or \
            not x[0, 0].is_contiguous() or (N > 1 and st[1] != stride) or (B > 1 and st[0] != N * stride):
        raise _Refused
    return x.data_ptr()


def _planes(c, dtypes, n, dev):
    """A kv_layer made from tensors has to hold the descriptor's pages, n
    elements a plane."""
    for x in getattr(c, "_tensors", ())[:2]:
        if x is not None and x.__class__ is not int and (
                x.dtype not in dtypes or x.numel() < n or x.get_device() != dev or not x.is_contiguous()):
            raise _Refused
    return c


def _refusable(f):
    """A call whose tensors do not fit its descriptor returns
    DFLV_ERR_INVALID_ARG, as the library does for what it can see itself."""
    def call(*args, **kw):
        try:
            return f(*args, **kw)
        except _Refused:
            return DFLV_ERR_INVALID_ARG
    call.__name__, call.__doc__ = f.__name__, f.__doc__
    return call


def pages_desc(B, N_max, page, n_pages, max_pages, flags=0):
    return dflv_pages_desc(B, N_max, page, n_pages, max_pages, flags)


def paged_kv_desc(B, N_max, Hkv, D, page, n_pages, kv_type, kv_stride=0, flags=0):
    return dflv_paged_kv_desc(B, N_max, Hkv, D, page, n_pages, kv_type, kv_stride, flags)


def prefix_attn_desc(B, N_max, Hq, Hkv, D, page, n_pages, max_pages, max_prefix_pages, kv_type, scale, q_stride=0,
                     flags=0):
    return dflv_prefix_attn_desc(B, N_max, Hq, Hkv, D, page, n_pages, max_pages, max_prefix_pages, kv_type, scale,
                                 q_stride, flags)


def sample_desc(B, N_max, V, logits_type=DFLV_LOGITS_F32, ld=0, flags=0):
    return dflv_sample_desc(B, N_max, V, logits_type, ld, flags)


@_refusable
def dflv_block_tables_grow(desc, n_past, n_new, n_held, free_list, n_free, table, slots, status_dev,
                           stream=None) -> int:
    lib, dev, B = _lib or load(), _device(), desc.B
    i32 = _kinds[0]
    return lib.dflv_block_tables_grow(
        ctypes.byref(desc), _arg(n_past, i32, B, dev), _arg(n_new, i32, B, dev), _arg(n_held, i32, B, dev),
        _arg(free_list, i32, desc.n_pages, dev), _arg(n_free, i32, 1, dev), _arg(table, i32, B * desc.max_pages, dev),
        _arg(slots, i32, B * desc.N_max, dev), _arg(status_dev, i32, 1, dev), _where(stream, dev))


@_refusable
def dflv_block_tables_release(desc, keep_len, n_held, free_list, n_free, table, status_dev, stream=None) -> int:
    lib, dev, B = _lib or load(), _device(), desc.B
    i32 = _kinds[0]
    return lib.dflv_block_tables_release(
        ctypes.byref(desc), _arg(keep_len, i32, B, dev), _arg(n_held, i32, B, dev),
        _arg(free_list, i32, desc.n_pages, dev), _arg(n_free, i32, 1, dev), _arg(table, i32, B * desc.max_pages, dev),
        _arg(status_dev, i32, 1, dev), _where(stream, dev))


@_refusable
def dflv_paged_kv_append(desc, slots, k_new, v_new, cache, status_dev, stream=None) -> int:
    lib, dev, B, N, stride = _lib or load(), _device(), desc.B, desc.N_max, desc.kv_stride
    inner, kind = desc.Hkv * desc.D, _kinds[2].get(desc.type, ())
    return lib.dflv_paged_kv_append(
        ctypes.byref(desc), _arg(slots, _kinds[0], B * N, dev), _rows(k_new, kind, B, N, inner, stride, dev),
        _rows(v_new, kind, B, N, inner, stride, dev),
        ctypes.byref(_planes(cache, kind, desc.n_pages * desc.page * inner, dev)),
        _arg(status_dev, _kinds[0], 1, dev), _where(stream, dev))


@_refusable
def dflv_paged_kv_commit(desc, n_layers, caches, slots, path, path_len, n_past, status_dev, stream=None) -> int:
    """``caches``: sequence of dflv_kv_layer, one per layer."""
    lib, dev, B, N = _lib or load(), _device(), desc.B, desc.N_max
    i32, kind, n = _kinds[0], _kinds[2].get(desc.type, ()), desc.n_pages * desc.page * desc.Hkv * desc.D
    if not 0 <= n_layers <= len(caches):
        return DFLV_ERR_INVALID_ARG
    ca = (dflv_kv_layer * max(1, n_layers))(*[_planes(c, kind, n, dev) for c in caches[:n_layers]])
    return lib.dflv_paged_kv_commit(
        ctypes.byref(desc), n_layers, ca, _arg(slots, i32, B * N, dev), _arg(path, i32, B * N, dev),
        _arg(path_len, i32, B, dev), _arg(n_past, i32, B, dev), _arg(status_dev, i32, 1, dev), _where(stream, dev))


@_refusable
def dflv_prefix_attn_verify(desc, prefix_table, prefix_len, table, parent, n_nodes, n_past, q, cache, out,
                            status_dev, workspace, ws_bytes, stream=None) -> int:
    lib, dev, B, N, D = _lib or load(), _device(), desc.B, desc.N_max, desc.D
    i32, inner, kind = _kinds[0], desc.Hq * D, _kinds[2].get(desc.type, ())
    if workspace is not None and workspace.__class__ is not int and (
            workspace.get_device() != dev or not workspace.is_contiguous() or
            workspace.numel() * workspace.element_size() < ws_bytes):
        return DFLV_ERR_INVALID_ARG
    return lib.dflv_prefix_attn_verify(
        ctypes.byref(desc), _arg(prefix_table, i32, desc.max_prefix_pages, dev), _arg(prefix_len, i32, 1, dev),
        _arg(table, i32, B * desc.max_pages, dev), _arg(parent, i32, B * N, dev), _arg(n_nodes, i32, B, dev),
        _arg(n_past, i32, B, dev), _rows(q, kind, B, N, inner, desc.q_stride, dev),
        ctypes.byref(_planes(cache, kind, desc.n_pages * desc.page * desc.Hkv * D, dev)),
        _rows(out, kind, B, N, inner, 0, dev), _arg(status_dev, i32, 1, dev), _ptr(workspace), ws_bytes,
        _where(stream, dev))


def dflv_prefix_attn_workspace_size(desc) -> int:
    return int(load().dflv_prefix_attn_workspace_size(ctypes.byref(desc)))


def _sample_args(desc, logits, temperature, top_k, top_p, min_p, u, dev):
    f32, B, N = _kinds[1], desc.B, desc.N_max
    return (ctypes.byref(desc), _rows(logits, _kinds[3].get(desc.type, ()), B, N, desc.V, desc.ld, dev),
            _arg(temperature, f32, B, dev), _arg(top_k, _kinds[0], B, dev), _arg(top_p, f32, B, dev),
            _arg(min_p, f32, B, dev), _arg(u, f32, B * N, dev))


@_refusable
def dflv_sample(desc, logits, temperature, top_k, top_p, min_p, u, n_nodes, drawn, logp, status_dev,
                stream=None) -> int:
    lib, dev, n = _lib or load(), _device(), desc.B * desc.N_max
    i32 = _kinds[0]
    return lib.dflv_sample(*_sample_args(desc, logits, temperature, top_k, top_p, min_p, u, dev),
                           _arg(n_nodes, i32, desc.B, dev), _arg(drawn, i32, n, dev), _arg(logp, _kinds[1], n, dev),
                           _arg(status_dev, i32, 1, dev), _where(stream, dev))


@_refusable
def dflv_accept_sampled(desc, logits, temperature, top_k, top_p, min_p, u, tokens, parent, n_nodes, path, path_len,
                        next_token, drawn, logp, status_dev, stream=None) -> int:
    lib, dev, B, n = _lib or load(), _device(), desc.B, desc.B * desc.N_max
    i32 = _kinds[0]
    return lib.dflv_accept_sampled(
        *_sample_args(desc, logits, temperature, top_k, top_p, min_p, u, dev), _arg(tokens, i32, n, dev),
        _arg(parent, i32, n, dev), _arg(n_nodes, i32, B, dev), _arg(path, i32, n, dev), _arg(path_len, i32, B, dev),
        _arg(next_token, i32, B, dev), _arg(drawn, i32, n, dev), _arg(logp, _kinds[1], n, dev),
        _arg(status_dev, i32, 1, dev), _where(stream, dev))


def dflv_gdn_workspace_size(desc) -> int:
    return int(load().dflv_gdn_workspace_size(ctypes.byref(desc)))


def dflv_attn_workspace_size(desc) -> int:
    return int(load().dflv_attn_workspace_size(ctypes.byref(desc)))


def dflv_status_string(code: int) -> str:
    return status_string(code)
