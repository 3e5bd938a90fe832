"""Binding of the serving operators (llm_append_kv, llm_read_kv, llm_prefix_attention,
llm_sample_tokens in include/llmq.h): argument checks and marshalling, the work
runs in ``libllmq.so``. Tensors, streams and errors as in ``tree``.
"""
from __future__ import annotations

import struct

from . import tree as _t
from .tree import KVView, _check, _fail, _flat, _name

_APPEND = struct.Struct("@4i4P8q6Pfdi0P").pack
_STRIDES = struct.Struct("@3q").pack
_DTYPES: dict = {}  # torch's dtype objects -> llm_dtype, once a tensor has come in
_UNSUPPORTED = -2


def _load():
    lib = _t._lib or _t._load()
    if not _DTYPES:
        _DTYPES[_t._f32], _DTYPES[_t._bf16] = _t.LLM_F32, _t.LLM_BF16
    return lib


def _kind(t, name: str) -> int:
    d = _DTYPES.get(t.dtype)
    if d is None:
        _fail(f"{name} of type {_name(t)} (bfloat16 or float32)", _UNSUPPORTED)
    return d


def _heads(t, name: str, dtype, shape: tuple):
    """Address and strides of a [token, head, head_dim] tensor."""
    s0, s1, s2 = t.stride()
    if t.dtype is not dtype or t.shape != shape or s2 != 1:
        _fail(f"{name}: {str(dtype).rpartition('.')[2]} of shape {shape} with contiguous heads is needed, not {_name(t)} "
              f"{tuple(t.shape)}")
    return t.data_ptr(), s0, s1


def append_kv(k, v, cache: KVView, seqs, rows, *, q=None, q_out=None, positions=None, rope_theta: float | None = None,
              rope_neox: bool = False, q_norm=None, k_norm=None, eps: float = 1e-5, stream: int | None = None) -> None:
    """Cache row rows[token] of sequence seqs[token] = k, v [token, kv head, head_dim], k normed (k_norm) and rotated
    by positions (None: rows); q [token, head, head_dim] likewise to q_out (may be q). rope_theta None: no rotation;
    see llm_append_kv."""
    L = _load()
    dt = k.dtype
    kind = out_kind = _kind(k, "k")
    T, H, hd = k.shape
    if cache.shape[2] != H or cache.shape[4] != hd:
        _fail(f"k has {H} heads x {hd}, the cache {cache.shape[2]} x {cache.shape[4]}")
    kp, k0, k1 = _heads(k, "k", dt, (T, H, hd))
    vp, v0, v1 = _heads(v, "v", dt, (T, H, hd))
    Hq = qp = q0 = q1 = op = o0 = o1 = 0
    if q is not None:
        Hq = q.shape[1]
        qp, q0, q1 = _heads(q, "q", dt, (T, Hq, hd))
        if q_out is None:
            _fail("q needs q_out")
        out_kind = _kind(q_out, "q_out")
        op, o0, o1 = _heads(q_out, "q_out", q_out.dtype, (T, Hq, hd))
    elif q_out is not None:
        _fail("q_out needs q")
    if rope_theta is not None and not rope_theta > 0:
        _fail("rope_theta is not positive (None: no rotation)")
    rc = L.llm_append_kv(
        _APPEND(kind, out_kind, T, Hq, qp, kp, vp, op, q0, q1, k0, k1, v0, v1, o0, o1, cache._at,
                _flat(seqs, "seqs", _t._i32, (T,)), _flat(rows, "rows", _t._i32, (T,)),
                0 if positions is None else _flat(positions, "positions", _t._i32, (T,)),
                0 if q_norm is None else _flat(q_norm, "q_norm", _t._f32, (hd,)),
                0 if k_norm is None else _flat(k_norm, "k_norm", _t._f32, (hd,)), eps,
                0.0 if rope_theta is None else rope_theta, rope_neox), stream)
    if rc:
        _check(rc)


def read_kv(cache: KVView, seqs, rows, k, v, stream: int | None = None) -> None:
    """k, v [token, head, head_dim] ([layer, token, head, head_dim] of a view with layers) = the values of row
    rows[token] of sequence seqs[token], as bfloat16 or float32; see llm_read_kv."""
    L = _load()
    kind = _kind(k, "k")
    _, layers, H, _, hd = cache.shape
    shape, stride = k.shape, k.stride()
    if v.shape != shape or v.stride() != stride or v.dtype is not k.dtype:
        _fail("k and v differ in shape, strides or type")
    if len(shape) == 3 and layers == 1:
        shape, stride = (1, *shape), (0, *stride)
    if len(shape) != 4 or shape[0] != layers or shape[2] != H or shape[3] != hd or stride[3] != 1:
        _fail(f"k: shape ({layers}, tokens, {H}, {hd}) with contiguous heads is needed, not {tuple(k.shape)}")
    T = shape[1]
    rc = L.llm_read_kv(cache._at, T, _flat(seqs, "seqs", _t._i32, (T,)), _flat(rows, "rows", _t._i32, (T,)), kind,
                       k.data_ptr(), v.data_ptr(), _STRIDES(*stride[:3]), stream)
    if rc:
        _check(rc)
