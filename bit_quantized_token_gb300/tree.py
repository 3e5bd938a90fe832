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


_lib = None
_names: dict = {}  # dtype object -> its name ("bfloat16", ...)


def _load():
    global _lib
    if _lib is None:
        _lib = _base.lib()
    return _lib


def _fail(msg: str, code: int = _INVALID):
    raise LlmError(code, msg)


def _check(rc: int) -> None:
    if rc != 0:
        raise LlmError(rc, _lib.llm_last_error(None).decode())


def _name(t) -> str:
    d = t.dtype
    n = _names.get(d)
    if n is None:
        n = _names[d] = str(d).rpartition(".")[2]
    return n


def _flat(t, name: str, dtype: str, shape: tuple):
    """Address of a contiguous tensor of this type and shape."""
    if t is None:
        _fail(f"{name} is needed")
    if _name(t) != dtype or t.shape != shape or not t.is_contiguous():
        _fail(f"{name}: a contiguous {dtype} tensor of shape {shape} is needed, not {_name(t)} {tuple(t.shape)}")
    return t.data_ptr()


class KVView:
    """K and V rows [seq, head, row, head_dim], or [seq, layer, head, row, head_dim].

    bf16 tensors, or int8 codes with fp16 scales [.., head_dim / 32] of each 32
    values. Strides may be anything that keeps a row contiguous and 16-byte
    aligned; k and v (and their scales) share them. The view keeps its tensors.
    """

    def __init__(self, k, v, k_scales=None, v_scales=None):
        q8 = k_scales is not None
        dtype = "int8" if q8 else "bfloat16"
        if len(k.shape) not in (4, 5):
            _fail(f"k has {len(k.shape)} dimensions, not 4 (or 5 with layers)")
        if (k_scales is None) != (v_scales is None):
            _fail("scales are given for both k and v or for neither")
        if _name(k) != dtype or _name(v) != dtype:
            _fail(f"k and v are {_name(k)} and {_name(v)}, not {dtype}", _UNSUPPORTED)
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
                if _name(t) != "float16" or tuple(t.shape) != want:
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
    B, n, H, hd = q.shape
    name = _name(q)
    if out.shape != q.shape or _name(out) != name:
        _fail("out must have q's shape and type")
    if name not in ("bfloat16", "float32"):
        _fail(f"queries of type {name} (bfloat16 or float32)", _UNSUPPORTED)
    if cache.shape[4] != hd:
        _fail(f"q has head_dim {hd}, the cache {cache.shape[4]}")
    qs, os_ = q.stride(), out.stride()
    if qs[3] != 1 or os_[3] != 1:
        _fail("a head's values must be contiguous in q and out")
    a = _AttentionArgs(LLM_F32 if name == "float32" else LLM_BF16, B, n, H, q.data_ptr(), out.data_ptr(), qs[:3],
                       os_[:3], cache._at)
    a.lens = _flat(lens, "lens", "int32", (B,))
    if tree is not None:
        a.tree = tree._at
        a.mask = _flat(mask, "mask", "int64", (B, n))
    if counts is not None:
        a.counts = _flat(counts, "counts", "int32", (B,))
    a.scale = hd ** -0.5 if scale is None else scale
    rc = L.llm_tree_attention(C.byref(a), stream)
    if rc:
        _check(rc)


def tree_status(stream: int | None = None) -> None:
    """Wait for the stream and raise if a tree attention's device-side wait passed its limit; see llm_tree_status."""
    L = _lib or _load()
    _check(L.llm_tree_status(stream))


def token_probs(logits, out, temperature: float = 1.0, top_k: int = 0, top_p: float = 1.0,
                stream: int | None = None) -> None:
    """out [rows, vocab] = the distribution that set_sampling's options draw from; see llm_token_probs."""
    L = _lib or _load()
    R, V = logits.shape
    if out.shape != logits.shape or _name(logits) != "float32" or _name(out) != "float32":
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
    B, n = tokens.shape
    a = _VerifyArgs(B, n)
    a.tokens = _flat(tokens, "tokens", "int32", (B, n))
    a.parents = _flat(parents, "parents", "int32", (B, n))
    a.path = _flat(path, "path", "int32", (B, n))
    a.n_path = _flat(n_path, "n_path", "int32", (B,))
    a.next = _flat(next_token, "next_token", "int32", (B,))
    if counts is not None:
        a.counts = _flat(counts, "counts", "int32", (B,))
    if targets is not None:
        a.targets = _flat(targets, "targets", "int32", (B, n))
    if probs is not None:
        a.vocab = probs.shape[-1]
        a.uniforms = _flat(uniforms, "uniforms", "float32", (B, n))
        for t, ptr, strides in ((probs, "probs", "probs_strides"), (draft_probs, "draft_probs", "draft_strides")):
            if t is None:
                continue
            st = t.stride()
            if _name(t) != "float32" or tuple(t.shape) != (B, n, a.vocab) or (a.vocab > 1 and st[2] != 1):
                _fail(f"{ptr}: float32 of shape {(B, n, a.vocab)} with contiguous rows is needed")
            setattr(a, ptr, t.data_ptr())
            setattr(a, strides, st[:2])
    elif draft_probs is not None:
        _fail("draft_probs need probs")
    rc = L.llm_verify_tree(C.byref(a), stream)
    if rc:
        _check(rc)


def commit_tree(cache: KVView, tree: KVView, lens, path, n_path, new_lens, stream: int | None = None) -> None:
    """Cache rows lens[seq] + k = tree rows path[seq, k], k < n_path[seq], in every layer; see llm_commit_tree."""
    L = _lib or _load()
    B, n = path.shape
    rc = L.llm_commit_tree(cache._at, tree._at, B, n, _flat(lens, "lens", "int32", (B,)),
                           _flat(path, "path", "int32", (B, n)), _flat(n_path, "n_path", "int32", (B,)),
                           _flat(new_lens, "new_lens", "int32", (B,)), stream)
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
