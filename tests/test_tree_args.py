"""Refusals of the tree-decoding operators: every check that precedes the GPU (no GPU needed)."""
import ctypes as C

import pytest
import torch

import bit_quantized_token_gb300 as bq
from bit_quantized_token_gb300 import tree as bt


@pytest.fixture(scope="module", autouse=True)
def library():
    bq.build()
    return bq.lib()


class Fake:
    """Shape, strides and type of a tensor at an address that is never read."""

    def __init__(self, shape, dtype=torch.bfloat16, stride=None, at=1 << 20):
        self.shape, self.dtype, self._at = torch.Size(shape), dtype, at
        if stride is None:
            stride, n = [], 1
            for s in reversed(shape):
                stride.insert(0, n)
                n *= s
        self._stride = tuple(stride)

    def stride(self):
        return self._stride

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self._at


def view(B=2, H=2, rows=8, hd=64, **kw):
    return bq.KVView(Fake((B, H, rows, hd), **kw), Fake((B, H, rows, hd), **kw))


def attend(B=2, n=3, H=4, hd=64, dtype=torch.bfloat16, cache=None, tree=None, out=None, q=None, **kw):
    q = q or Fake((B, n, H, hd), dtype)
    bq.tree_attention(q, cache or view(B, hd=hd), tree or view(B, rows=n, hd=hd), Fake((B,), torch.int32),
                      Fake((B, n), torch.int64), out or Fake((B, n, H, hd), dtype), **kw)


def verify(B=2, n=3, V=7, **kw):
    i32 = lambda *s: Fake(s, torch.int32)  # noqa: E731
    a = dict(tokens=i32(B, n), parents=i32(B, n), uniforms=Fake((B, n), torch.float32),
             probs=Fake((B, n, V), torch.float32), path=i32(B, n), n_path=i32(B), next_token=i32(B))
    a.update(kw)
    bq.verify_tree(**a)


def probs(R=2, V=9, T=1.0, k=0, p=1.0, logits=None, out=None):
    bq.token_probs(logits or Fake((R, V), torch.float32), out or Fake((R, V), torch.float32, at=1 << 30), T, k, p)


REFUSED = [
    ("n_nodes", lambda: attend(n=65, tree=view(rows=65))),
    ("queries of type float16", lambda: attend(dtype=torch.float16)),
    ("out must have", lambda: attend(out=Fake((2, 3, 4, 64), torch.float32))),
    ("multiple of the cache's heads", lambda: attend(H=3)),
    ("head_dim 96", lambda: attend(hd=96)),
    ("head_dim 64, the cache 128", lambda: attend(cache=view(hd=128))),
    ("fewer sequences", lambda: attend(B=3, cache=view(2), tree=view(3, rows=3))),
    ("do not match", lambda: attend(tree=view(rows=2))),
    ("do not match", lambda: attend(tree=view(H=1, rows=3))),
    ("scale is not finite", lambda: attend(scale=float("nan"))),
    ("multiple of 16 bytes", lambda: attend(cache=view(stride=(1024, 512, 68, 1)))),
    ("values must be contiguous", lambda: attend(cache=view(stride=(1024, 512, 128, 2)))),
    ("not aligned", lambda: attend(cache=view(at=(1 << 20) + 8))),
    ("contiguous int32", lambda: attend(counts=Fake((2,), torch.int64))),
    ("dimensions", lambda: bq.KVView(Fake((2, 8, 64)), Fake((2, 8, 64)))),
    ("not bfloat16", lambda: view(dtype=torch.float16)),
    ("both k and v", lambda: bq.KVView(Fake((1, 1, 4, 64), torch.int8), Fake((1, 1, 4, 64), torch.int8),
                                       Fake((1, 1, 4, 2), torch.float16))),
    ("scales: float16", lambda: bq.KVView(Fake((1, 1, 4, 64), torch.int8), Fake((1, 1, 4, 64), torch.int8),
                                          *[Fake((1, 1, 4, 4), torch.float16)] * 2)),
    ("differ in shape", lambda: bq.KVView(Fake((1, 1, 4, 64)), Fake((1, 1, 5, 64)))),
    ("temperature", lambda: probs(T=0.0)),
    ("temperature", lambda: probs(T=float("inf"))),
    ("temperature", lambda: probs(T=float("nan"))),
    ("temperature", lambda: probs(T=1e-39)),
    ("top_k", lambda: probs(k=65)),
    ("top_k", lambda: probs(k=-1)),
    ("top_p must be", lambda: probs(k=4, p=0.0)),
    ("top_p must be", lambda: probs(k=4, p=1.5)),
    ("needs a top_k", lambda: probs(p=0.9)),
    ("too large", lambda: probs(V=524289, k=1)),
    ("too large", lambda: probs(V=819201)),
    ("rows of probs overlap", lambda: probs(out=Fake((2, 9), torch.float32, stride=(0, 1)))),
    ("float32 of one shape", lambda: probs(logits=Fake((2, 9)))),
    ("n_nodes", lambda: verify(n=65)),
    ("either probs or targets", lambda: verify(targets=Fake((2, 3), torch.int32))),
    ("either probs or targets", lambda: verify(probs=None, uniforms=None)),
    ("draft_probs need probs", lambda: verify(probs=None, draft_probs=Fake((2, 3, 7), torch.float32))),
    ("draft_probs: float32", lambda: verify(draft_probs=Fake((2, 2, 7), torch.float32))),
    ("tokens: a contiguous", lambda: verify(tokens=Fake((2, 3), torch.int64))),
    ("uniforms is needed", lambda: verify(uniforms=None)),
    ("do not match", lambda: bq.commit_tree(view(), view(rows=2), *[Fake((2,), torch.int32), Fake((2, 3), torch.int32),
                                            Fake((2,), torch.int32), Fake((2,), torch.int32)])),
    ("has parent", lambda: bq.tree_masks([-1, 1])),
    ("at most 64", lambda: bq.tree_masks([-1] + [0] * 64)),
]


@pytest.mark.parametrize("i", range(len(REFUSED)), ids=[r[0].replace(" ", "_") + f"-{i}" for i, r in enumerate(REFUSED)])
def test_refused_with_its_reason(i):
    words, call = REFUSED[i]
    with pytest.raises(bq.LlmError, match=words):
        call()


def test_null_arguments(library):
    assert library.llm_tree_attention(None, None) == -1
    assert library.llm_verify_tree(None, None) == -1
    assert library.llm_commit_tree(None, None, 1, 1, None, None, None, None, None) == -1
    assert library.llm_token_probs(None, 4, None, 4, 1, 4, 1.0, 0, 1.0, None) == -1
    assert b"null" in library.llm_last_error(None)


def test_overlapping_outputs_are_refused(library):
    for stride in ((768, 256, 32, 1), (768, 0, 64, 1), (64, 128, 64, 1)):
        with pytest.raises(bq.LlmError, match="rows of out overlap"):
            attend(out=Fake((2, 3, 4, 64), torch.bfloat16, stride=stride))
    four = [Fake((2,), torch.int32), Fake((2, 3), torch.int32), Fake((2,), torch.int32)]
    with pytest.raises(bq.LlmError, match="rows of the cache overlap"):
        bq.commit_tree(view(stride=(0, 512, 64, 1)), view(rows=3), *four, Fake((2,), torch.int32, at=1 << 21))
    # drafts behind the lengths of the cache's own rows, or a head's rows that run into it
    for shift in (0, 5 * 64, -2 * 64):
        with pytest.raises(bq.LlmError, match="lie in the cache"):
            bq.commit_tree(view(rows=8, stride=(2048, 1024, 64, 1)), view(rows=3, stride=(2048, 1024, 64, 1), at=(1 << 20) + 2 * shift),
                           *four, Fake((2,), torch.int32, at=1 << 21))
    for shift in (8 * 64, -3 * 64):  # beside it: refused for no such reason
        with pytest.raises(bq.LlmError, match="current device"):
            bq.commit_tree(view(rows=8, stride=(2048, 1024, 64, 1)), view(rows=3, stride=(2048, 1024, 64, 1), at=(1 << 20) + 2 * shift),
                           *four, Fake((2,), torch.int32, at=1 << 21))
    with pytest.raises(bq.LlmError, match="new_lens overlaps"):
        bq.commit_tree(view(), view(rows=3), *four, Fake((2,), torch.int32, at=(1 << 20) + 4))


def test_tree_masks():
    assert bq.tree_masks([-1, 0, 0, 1, 3]) == [0b1, 0b11, 0b101, 0b1011, 0b11011]
    assert bq.tree_masks([-1] + list(range(63)))[63] == -1


def test_struct_layouts_match_c(tmp_path):
    import os
    import subprocess
    structs = {"llm_kv_view": bt._KvView, "llm_tree_attention_args": bt._AttentionArgs,
               "llm_verify_tree_args": bt._VerifyArgs}
    lines = []
    for name, s in structs.items():
        lines.append(f'printf("%zu ", sizeof({name}));')
        lines += [f'printf("%zu ", offsetof({name}, {f}));' for f, _ in s._fields_]
    src = tmp_path / "l.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "llmq.h"\nint main(void) {' + "".join(lines) +
                   "return 0; }")
    exe = tmp_path / "l"
    subprocess.check_call(["gcc", "-I", os.path.dirname(bq.HEADER), str(src), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    want = []
    for s in structs.values():
        want.append(C.sizeof(s))
        want += [getattr(s, f).offset for f, _ in s._fields_]
    assert got == want
    # the packers lay their bytes out as the structs
    a = bt._AttentionArgs.from_buffer_copy(bt._ATTENTION(*range(1, 18), 18.5))
    assert (a.dtype, a.n_heads, a.q, a.out, list(a.q_strides), list(a.out_strides), a.cache, a.counts, a.scale) == (
        1, 4, 5, 6, [7, 8, 9], [10, 11, 12], 13, 17, 18.5)
    v = bt._VerifyArgs.from_buffer_copy(bt._VERIFY(*range(1, 18)))
    assert (v.vocab, v.tokens, v.probs, list(v.probs_strides), v.draft_probs, list(v.draft_strides), v.next) == (
        3, 4, 8, [9, 10], 11, [12, 13], 17)
