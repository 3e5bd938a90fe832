"""Binding of the serving operators (llm_append_kv, llm_read_kv, llm_prefix_attention,
llm_sample_tokens in include/llmq.h): argument checks and marshalling, the work
runs in ``libllmq.so``. Tensors, streams and errors as in ``tree``.
"""
from __future__ import annotations

import struct

from . import tree as _t
from .tree import KVView, _check, _fail, _flat, _name

_APPEND = struct.Struct("@4i4P8q6Pfdi0P").pack
_PREFIX = struct.Struct("@4i2P6q5Pf0PPi0PPPPq").pack
_SAMPLE = struct.Struct("@Pq2i7P").pack
_STRIDES = struct.Struct("@3q").pack
_DTYPES: dict = {}  # torch's dtype objects -> llm_dtype, once a tensor has come in
_UNSUPPORTED = -2


def _load():
    global _DTYPES
    lib = _t._lib or _t._load()
    if not _DTYPES:
        _DTYPES = {_t._f32: _t.LLM_F32, _t._bf16: _t.LLM_BF16}  # all at once: another thread may come in between
    return lib


def _kind(t, name: str) -> int:
    d = _DTYPES.get(t.dtype)
    if d is None:
        _fail(f"{name} of type {_name(t)} (bfloat16 or float32)", _UNSUPPORTED)
    return d


def _heads(t, name: str, dtype, shape):
    """Address and strides of a [token, head, head_dim] tensor."""
    s0, s1, s2 = t.stride()
    if t.dtype is not dtype or t.shape != shape or s2 != 1:
        _fail(f"{name}: {str(dtype).rpartition('.')[2]} of shape {tuple(shape)} with contiguous heads is needed, not "
              f"{_name(t)} {tuple(t.shape)}")
    return t.data_ptr(), s0, s1


def _row(t, name: str, dtype, n: int) -> int:
    """Address of a contiguous tensor of n values of this type."""
    if t is not None and t.dtype is dtype and t.shape == (n,) and (n == 1 or t.stride(0) == 1):
        return t.data_ptr()
    return _flat(t, name, dtype, (n,))  # (says what is wrong)


def _opt(t, name: str, dtype, n: int) -> int:
    return 0 if t is None else _row(t, name, dtype, n)


def append_kv(k, v, cache: KVView, seqs, rows, *, q=None, q_out=None, positions=None, rope_theta: float | None = None,
              rope_neox: bool = False, q_norm=None, k_norm=None, eps: float = 1e-5, stream: int | None = None) -> None:
    """Cache row rows[token] of sequence seqs[token] = k, v [token, kv head, head_dim], k normed (k_norm) and rotated
    by positions (None: rows); q [token, head, head_dim] likewise to q_out (may be q). rope_theta None: no rotation;
    see llm_append_kv."""
    L = _load()
    dt, shape = k.dtype, k.shape
    kind = out_kind = _kind(k, "k")
    T, H, hd = shape
    if cache.shape[2] != H or cache.shape[4] != hd:
        _fail(f"k has {H} heads x {hd}, the cache {cache.shape[2]} x {cache.shape[4]}")
    kp, k0, k1 = _heads(k, "k", dt, shape)
    vp, v0, v1 = _heads(v, "v", dt, shape)
    Hq = qp = q0 = q1 = op = o0 = o1 = 0
    if q is not None:
        of_q = q.shape
        Hq = of_q[1]
        if of_q[0] != T or of_q[2] != hd:
            of_q = (T, Hq, hd)
        qp, q0, q1 = _heads(q, "q", dt, of_q)
        if q_out is None:
            _fail("q needs q_out")
        out_kind = _kind(q_out, "q_out")
        op, o0, o1 = _heads(q_out, "q_out", q_out.dtype, of_q)
    elif q_out is not None:
        _fail("q_out needs q")
    if rope_theta is None:
        rope_theta = 0.0
    elif not rope_theta > 0:
        _fail("rope_theta is not positive (None: no rotation)")
    i32, f32 = _t._i32, _t._f32
    rc = L.llm_append_kv(
        _APPEND(kind, out_kind, T, Hq, qp, kp, vp, op, q0, q1, k0, k1, v0, v1, o0, o1, cache._at,
                _row(seqs, "seqs", i32, T), _row(rows, "rows", i32, T), _opt(positions, "positions", i32, T),
                _opt(q_norm, "q_norm", f32, hd), _opt(k_norm, "k_norm", f32, hd), eps, rope_theta, rope_neox), stream)
    if rc:
        _check(rc)


def read_kv(cache: KVView, seqs, rows, k, v, stream: int | None = None) -> None:
    """k, v [token, head, head_dim] ([layer, token, head, head_dim] of a view with layers) = the values of row
    rows[token] of sequence seqs[token], as bfloat16 or float32; see llm_read_kv."""
    L = _load()
    kind = _kind(k, "k")
    _, layers, H, _, hd = cache.shape
    shape, stride = k.shape, k.stride()
    if v.dtype is not k.dtype or v.shape != shape or v.stride() != stride:
        _fail("k and v differ in shape, strides or type")
    if len(shape) == 3 and layers == 1:
        shape, stride = (1, *shape), (0, *stride)
    if len(shape) != 4 or shape[0] != layers or shape[2] != H or shape[3] != hd or stride[3] != 1:
        _fail(f"k: shape ({layers}, tokens, {H}, {hd}) with contiguous heads is needed, not {tuple(k.shape)}")
    T, i32 = shape[1], _t._i32
    rc = L.llm_read_kv(cache._at, T, _row(seqs, "seqs", i32, T), _row(rows, "rows", i32, T), kind, k.data_ptr(),
                       v.data_ptr(), _STRIDES(*stride[:3]), stream)
    if rc:
        _check(rc)


def prefix_workspace(q) -> int:
    """Bytes of prefix_attention's workspace for queries of q's shape [seq, node, head, head_dim]; see
    llm_prefix_workspace."""
    n = _t._base.lib().llm_prefix_workspace(*q.shape)
    if n < 0:
        _check(n)
    return n


def prefix_attention(q, prefix: KVView, starts, prefix_lens, cache: KVView, tree: KVView | None, lens, mask, out,
                     workspace, counts=None, scale: float | None = None, stream: int | None = None) -> None:
    """tree_attention where sequences starts[g] .. starts[g + 1] - 1 also see the first prefix_lens[g] rows of the
    prefix view's sequence g, which are read once for all of them. workspace: a contiguous CUDA tensor of
    prefix_workspace(q) bytes, one for each of the calls that may overlap. Views narrowed to the batch's longest
    lengths (k[:, :, :rows]) are faster than ones of a cache's whole room; see llm_prefix_attention."""
    L = _load()
    shape, dt = q.shape, q.dtype
    kind = _kind(q, "queries")
    B, n, H, hd = shape
    if out.shape != shape or out.dtype is not dt:
        _fail("out must have q's shape and type")
    if cache.shape[4] != hd:
        _fail(f"q has head_dim {hd}, the cache {cache.shape[4]}")
    q0, q1, q2, q3 = q.stride()
    o0, o1, o2, o3 = out.stride()
    if q3 != 1 or o3 != 1:
        _fail("a head's values must be contiguous in q and out")
    G = prefix_lens.shape[0]
    if not workspace.is_contiguous():
        _fail("the workspace is not contiguous")
    i32 = _t._i32
    rc = L.llm_prefix_attention(
        _PREFIX(kind, B, n, H, q.data_ptr(), out.data_ptr(), q0, q1, q2, o0, o1, o2, cache._at,
                0 if tree is None else tree._at, _row(lens, "lens", i32, B),
                0 if tree is None else _flat(mask, "mask", _t._i64, (B, n)), _opt(counts, "counts", i32, B),
                hd ** -0.5 if scale is None else scale, prefix._at, G, _row(starts, "starts", i32, G + 1),
                _row(prefix_lens, "prefix_lens", i32, G), workspace.data_ptr(), workspace.nbytes), stream)
    if rc:
        _check(rc)


def sample_tokens(logits, uniforms, tokens, temperature=None, top_k=None, top_p=None, min_p=None, probs=None,
                  stream: int | None = None) -> None:
    """tokens [row] int32 = a token of each row of logits [row, vocab], drawn with uniforms [row] under the row's own
    temperature, top_p, min_p (float32 [row]) and top_k (int32 [row]; None: off); probs [row] float32: what it was
    drawn with; see llm_sample_tokens."""
    L = _load()
    R, V = logits.shape
    s0, s1 = logits.stride()
    if logits.dtype is not _t._f32 or (V > 1 and s1 != 1):
        _fail("logits: float32 with contiguous rows is needed")
    f32, i32 = _t._f32, _t._i32
    rc = L.llm_sample_tokens(
        _SAMPLE(logits.data_ptr(), s0, R, V, _row(uniforms, "uniforms", f32, R), _opt(temperature, "temperature", f32, R),
                _opt(top_k, "top_k", i32, R), _opt(top_p, "top_p", f32, R), _opt(min_p, "min_p", f32, R),
                _row(tokens, "tokens", i32, R), _opt(probs, "probs", f32, R)), stream)
    if rc:
        _check(rc)
