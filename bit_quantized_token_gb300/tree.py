"""Binding of the tree-decoding operators (llm_tree_attention, llm_token_probs,
llm_verify_tree, llm_commit_tree in include/llmq.h): argument checks and
marshalling, the work runs in ``libllmq.so``.

Tensors are torch CUDA tensors of the current device (anything with ``shape``,
``stride()``, ``dtype`` and ``data_ptr()``); outputs are given by the caller.
``stream`` is a cudaStream_t as an int, None for the legacy default stream
(torch's default stream); a call on another torch stream passes its
``cuda_stream``. Calls return before the GPU has run them.
"""
from __future__ import annotations

import ctypes as C
import struct

import bit_quantized_token_gb300 as _base
from bit_quantized_token_gb300 import LLM_BF16, LLM_F32, LLM_Q8G32, LlmError

_INVALID, _UNSUPPORTED = -1, -2


class _KvView(C.Structure):
    _fields_ = [("dtype", C.c_int32), ("n_seq", C.c_int32), ("n_layers", C.c_int32), ("n_heads", C.c_int32),
                ("rows", C.c_int32), ("head_dim", C.c_int32), ("k", C.c_void_p), ("v", C.c_void_p),
                ("k_scales", C.c_void_p), ("v_scales", C.c_void_p)] + [
        (p + n, C.c_int64) for p in ("", "scale_") for n in ("seq_stride", "layer_stride", "head_stride", "row_stride")]


class _AttentionArgs(C.Structure):
    _fields_ = [("dtype", C.c_int32), ("n_seq", C.c_int32), ("n_nodes", C.c_int32), ("n_heads", C.c_int32),
                ("q", C.c_void_p), ("out", C.c_void_p), ("q_strides", C.c_int64 * 3), ("out_strides", C.c_int64 * 3),
                ("cache", C.c_void_p), ("tree", C.c_void_p), ("lens", C.c_void_p), ("mask", C.c_void_p),
                ("counts", C.c_void_p), ("scale", C.c_float)]


class _VerifyArgs(C.Structure):
    _fields_ = [("n_seq", C.c_int32), ("n_nodes", C.c_int32), ("vocab", C.c_int32), ("tokens", C.c_void_p),
                ("parents", C.c_void_p), ("counts", C.c_void_p), ("uniforms", C.c_void_p), ("probs", C.c_void_p),
                ("probs_strides", C.c_int64 * 2), ("draft_probs", C.c_void_p), ("draft_strides", C.c_int64 * 2),
                ("targets", C.c_void_p), ("path", C.c_void_p), ("n_path", C.c_void_p), ("next", C.c_void_p)]


# The argument structs as native-layout packers: one call fills a struct, and
# the bytes belong to the calling thread alone.
_ATTENTION = struct.Struct("@4i2P6q5Pf0P").pack
_VERIFY = struct.Struct("@3i5P2qP2q4P").pack

_lib = None
_i32 = _i64 = _f32 = _f16 = _bf16 = _i8 = None  # torch's dtype objects, once a tensor has come in


def _load():
    global _lib, _i32, _i64, _f32, _f16, _bf16, _i8
    if _lib is None:
        lib = _base.lib()
        import torch  # the tensors are torch's
        _i32, _i64, _f32, _f16, _bf16, _i8 = (torch.int32, torch.int64, torch.float32, torch.float16, torch.bfloat16,
                                              torch.int8)
        _lib = lib
    return _lib


def _fail(msg: str, code: int = _INVALID):
    raise LlmError(code, msg)


def _check(rc: int) -> None:
    if rc != 0:
        raise LlmError(rc, _base.lib().llm_last_error(None).decode())


def _name(t) -> str:
    return str(t.dtype).rpartition(".")[2]


def _flat(t, name: str, dtype, shape: tuple) -> int:
    """Address of a contiguous tensor of this type and shape."""
    if t is None:
        _fail(f"{name} is needed")
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _fail(f"{name}: a contiguous {str(dtype).rpartition('.')[2]} tensor of shape {shape} is needed, not {_name(t)} "
              f"{tuple(t.shape)}")
    return t.data_ptr()


class KVView:
    """K and V rows [seq, head, row, head_dim], or [seq, layer, head, row, head_dim].

    bf16 tensors, or int8 codes with fp16 scales [.., head_dim / 32] of each 32
    values. Strides may be anything that keeps a row contiguous and 16-byte
    aligned; k and v (and their scales) share them. The view keeps its tensors.
    """

    def __init__(self, k, v, k_scales=None, v_scales=None):
        _lib or _load()
        q8 = k_scales is not None
        dtype = _i8 if q8 else _bf16
        if len(k.shape) not in (4, 5):
            _fail(f"k has {len(k.shape)} dimensions, not 4 (or 5 with layers)")
        if (k_scales is None) != (v_scales is None):
            _fail("scales are given for both k and v or for neither")
        if k.dtype is not dtype or v.dtype is not dtype:
            _fail(f"k and v are {_name(k)} and {_name(v)}, not {'int8' if q8 else 'bfloat16'}", _UNSUPPORTED)
        if v.shape != k.shape or v.stride() != k.stride():
            _fail("k and v differ in shape or strides")
        s = self._struct = _KvView()
        shape = tuple(k.shape)
        if len(shape) == 4:
            shape = (shape[0], 1) + shape[1:]
        self.shape = shape
        self.dtype = s.dtype = LLM_Q8G32 if q8 else LLM_BF16
        s.n_seq, s.n_layers, s.n_heads, s.rows, s.head_dim = shape
        self._strides(s, "", k)
        if q8:
            want = tuple(k.shape[:-1]) + (shape[-1] // 32,)
            for t in (k_scales, v_scales):
                if t.dtype is not _f16 or tuple(t.shape) != want:
                    _fail(f"scales: float16 of shape {want} are needed, not {_name(t)} {tuple(t.shape)}")
            if k_scales.stride() != v_scales.stride():
                _fail("the scales of k and v differ in strides")
            self._strides(s, "scale_", k_scales)
            s.k_scales, s.v_scales = k_scales.data_ptr(), v_scales.data_ptr()
        s.k, s.v = k.data_ptr(), v.data_ptr()
        self._keep = (k, v, k_scales, v_scales)
        self._at = C.addressof(s)

    @staticmethod
    def _strides(s, prefix, t):
        st = t.stride()
        if st[-1] != 1 and t.shape[-1] > 1:
            _fail("a row's values must be contiguous")
        setattr(s, prefix + "seq_stride", st[0])
        setattr(s, prefix + "layer_stride", st[1] if len(st) == 5 else 0)
        setattr(s, prefix + "head_stride", st[-3])
        setattr(s, prefix + "row_stride", st[-2])


def tree_attention(q, cache: KVView, tree: KVView | None, lens, mask, out, counts=None, scale: float | None = None,
                   stream: int | None = None) -> None:
    """out = attention of q [seq, node, head, head_dim] over the cache's first lens[seq] rows and the tree rows
    whose bits mask [seq, node] (int64) sets; see llm_tree_attention. tree None: the cache alone (mask unused)."""
    L = _lib or _load()
    shape, dt = q.shape, q.dtype
    B, n, H, hd = shape
    if out.shape != shape or out.dtype is not dt:
        _fail("out must have q's shape and type")
    if dt is not _bf16 and dt is not _f32:
        _fail(f"queries of type {_name(q)} (bfloat16 or float32)", _UNSUPPORTED)
    if cache.shape[4] != hd:
        _fail(f"q has head_dim {hd}, the cache {cache.shape[4]}")
    q0, q1, q2, q3 = q.stride()
    o0, o1, o2, o3 = out.stride()
    if q3 != 1 or o3 != 1:
        _fail("a head's values must be contiguous in q and out")
    rc = L.llm_tree_attention(
        _ATTENTION(LLM_F32 if dt is _f32 else LLM_BF16, B, n, H, q.data_ptr(), out.data_ptr(), q0, q1, q2, o0, o1, o2,
                   cache._at, 0 if tree is None else tree._at, _flat(lens, "lens", _i32, (B,)),
                   0 if tree is None else _flat(mask, "mask", _i64, (B, n)),
                   0 if counts is None else _flat(counts, "counts", _i32, (B,)),
                   hd ** -0.5 if scale is None else scale), stream)
    if rc:
        _check(rc)


def tree_status(stream: int | None = None) -> None:
    """Wait for the stream and raise if a tree operator's device-side wait passed its limit; see llm_tree_status."""
    _check(_base.lib().llm_tree_status(stream))


def token_probs(logits, out, temperature: float = 1.0, top_k: int = 0, top_p: float = 1.0,
                stream: int | None = None) -> None:
    """out [rows, vocab] = the distribution that set_sampling's options draw from; see llm_token_probs."""
    L = _lib or _load()
    R, V = logits.shape
    if out.shape != logits.shape or logits.dtype is not _f32 or out.dtype is not _f32:
        _fail("logits and out must be float32 of one shape")
    ls, os_ = logits.stride(), out.stride()
    if V > 1 and (ls[1] != 1 or os_[1] != 1):
        _fail("a row must be contiguous")
    rc = L.llm_token_probs(logits.data_ptr(), ls[0], out.data_ptr(), os_[0], R, V, temperature, top_k, top_p, stream)
    if rc:
        _check(rc)


def verify_tree(tokens, parents, uniforms, probs, path, n_path, next_token, draft_probs=None, targets=None,
                counts=None, stream: int | None = None) -> None:
    """Which drafts are kept (path, n_path) and the token after them (next_token); see llm_verify_tree.
    probs, draft_probs [seq, node, vocab] float32; greedy mode: probs None and targets [seq, node] int32."""
    L = _lib or _load()
    B, n = shape = tokens.shape
    V = p = p0 = p1 = q = q0 = q1 = u = 0
    if probs is not None:
        V = probs.shape[2]
        u = _flat(uniforms, "uniforms", _f32, shape)
        p, p0, p1 = _rows(probs, "probs", (B, n, V))
        if draft_probs is not None:
            q, q0, q1 = _rows(draft_probs, "draft_probs", (B, n, V))
    elif draft_probs is not None:
        _fail("draft_probs need probs")
    rc = L.llm_verify_tree(
        _VERIFY(B, n, V, _flat(tokens, "tokens", _i32, shape), _flat(parents, "parents", _i32, shape),
                0 if counts is None else _flat(counts, "counts", _i32, (B,)), u, p, p0, p1, q, q0, q1,
                0 if targets is None else _flat(targets, "targets", _i32, shape), _flat(path, "path", _i32, shape),
                _flat(n_path, "n_path", _i32, (B,)), _flat(next_token, "next_token", _i32, (B,))), stream)
    if rc:
        _check(rc)


def _rows(t, name: str, shape: tuple):
    """Address and outer strides of a [seq, node, vocab] float32 tensor with contiguous rows."""
    s0, s1, s2 = t.stride()
    if t.dtype is not _f32 or t.shape != shape or (s2 != 1 and shape[2] > 1):
        _fail(f"{name}: float32 of shape {shape} with contiguous rows is needed")
    return t.data_ptr(), s0, s1


def commit_tree(cache: KVView, tree: KVView, lens, path, n_path, new_lens, stream: int | None = None) -> None:
    """Cache rows lens[seq] + k = tree rows path[seq, k], k < n_path[seq], in every layer; see llm_commit_tree."""
    L = _lib or _load()
    B, n = shape = path.shape
    rc = L.llm_commit_tree(cache._at, tree._at, B, n, _flat(lens, "lens", _i32, (B,)),
                           _flat(path, "path", _i32, shape), _flat(n_path, "n_path", _i32, (B,)),
                           _flat(new_lens, "new_lens", _i32, (B,)), stream)
    if rc:
        _check(rc)


def tree_masks(parents) -> list:
    """The mask words (as signed 64-bit ints) of one tree given its nodes' parents (host list; the root's is -1):
    every node sees itself and its ancestors."""
    words = []
    for i, par in enumerate(parents):
        if i and not 0 <= par < i:
            _fail(f"node {i} has parent {par}")
        words.append((words[par] if i else 0) | 1 << i)
    if len(words) > 64:
        _fail("a tree has at most 64 nodes", _UNSUPPORTED)
    return [w - (1 << 64) if w >> 63 else w for w in words]
