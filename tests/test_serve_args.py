"""Refusals of the serving operators: every check that precedes the GPU (no GPU needed)."""
import pytest
import torch

import bit_quantized_token_gb300 as bq
from test_tree_args import Fake as _Fake
from test_tree_args import view

F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32


class Fake(_Fake):
    @property
    def nbytes(self):
        return self.shape.numel() * self.dtype.itemsize

    def stride(self, i=None):
        return self._stride if i is None else self._stride[i]


@pytest.fixture(scope="module", autouse=True)
def library():
    bq.build()
    return bq.lib()


def append(T=3, H=2, Hq=4, hd=64, dtype=BF16, cache=None, **kw):
    a = dict(k=Fake((T, H, hd), dtype), v=Fake((T, H, hd), dtype), cache=cache or view(H=H, hd=hd),
             seqs=Fake((T,), I32), rows=Fake((T,), I32), q=Fake((T, Hq, hd), dtype), q_out=Fake((T, Hq, hd), dtype))
    a.update(kw)
    bq.append_kv(**a)


def read(T=3, L=1, H=2, hd=64, dtype=BF16, cache=None, **kw):
    a = dict(cache=cache or view(H=H, hd=hd), seqs=Fake((T,), I32), rows=Fake((T,), I32), k=Fake((L, T, H, hd), dtype),
             v=Fake((L, T, H, hd), dtype))
    a.update(kw)
    bq.read_kv(**a)


REFUSED = [
    ("k of type float16", lambda: append(dtype=torch.float16)),
    ("v: bfloat16", lambda: append(v=Fake((3, 2, 64), F32))),
    ("v: bfloat16 of shape", lambda: append(v=Fake((3, 1, 64)))),
    ("q: bfloat16", lambda: append(q=Fake((3, 4, 64), F32))),
    ("q_out of type", lambda: append(q_out=Fake((3, 4, 64), torch.int8))),
    ("q_out: bfloat16 of shape", lambda: append(q_out=Fake((3, 2, 64)))),
    ("q needs q_out", lambda: append(q_out=None)),
    ("q_out needs q", lambda: append(q=None)),
    ("contiguous heads", lambda: append(k=Fake((3, 2, 64), stride=(256, 128, 2)))),
    ("the cache 1 x 64", lambda: append(cache=view(H=1))),
    ("the cache 2 x 128", lambda: append(cache=view(hd=128))),
    ("head_dim 96", lambda: append(hd=96)),
    ("contiguous int32", lambda: append(seqs=Fake((3,), torch.int64))),
    ("contiguous int32", lambda: append(rows=Fake((2,), I32))),
    ("contiguous int32", lambda: append(positions=Fake((3,), torch.int64))),
    ("q_norm: a contiguous float32", lambda: append(q_norm=Fake((64,), BF16))),
    ("k_norm: a contiguous float32", lambda: append(k_norm=Fake((32,), F32))),
    ("rope_theta", lambda: append(rope_theta=-1.0)),
    ("rope_theta", lambda: append(rope_theta=0.0)),
    ("rope_theta", lambda: append(rope_theta=float("inf"))),
    ("rope_theta", lambda: append(rope_theta=float("nan"))),
    ("rope_neox", lambda: append(rope_theta=1e4, rope_neox=2)),
    ("norm_eps", lambda: append(q_norm=Fake((64,), F32), eps=0.0)),
    ("several layers", lambda: append(cache=bq.KVView(*[Fake((2, 3, 2, 8, 64))] * 2))),
    ("stride of k", lambda: append(k=Fake((3, 2, 64), stride=(130, 64, 1)))),
    ("rows of q_out overlap", lambda: append(q_out=Fake((3, 4, 64), stride=(64, 64, 1), at=1 << 30))),
    ("rows of the cache overlap", lambda: append(cache=view(stride=(0, 512, 64, 1)))),
    ("q_out is q with another", lambda: append(q_out=Fake((3, 4, 64), F32))),
    ("not aligned", lambda: append(cache=view(at=(1 << 20) + 8))),
    ("n_tokens", lambda: append(T=0)),
    ("differ in shape", lambda: read(v=Fake((1, 2, 2, 64)))),
    ("differ in shape, strides or type", lambda: read(v=Fake((1, 3, 2, 64), F32))),
    ("k of type float16", lambda: read(dtype=torch.float16)),
    ("shape (1, tokens, 2, 64)", lambda: read(L=2)),
    ("shape (1, tokens, 2, 64)", lambda: read(k=Fake((1, 3, 2, 32)), v=Fake((1, 3, 2, 32)))),
    ("contiguous int32", lambda: read(rows=Fake((4,), I32))),
    ("rows of the outputs overlap", lambda: read(k=Fake((1, 3, 2, 64), stride=(384, 64, 64, 1)),
                                                 v=Fake((1, 3, 2, 64), stride=(384, 64, 64, 1)))),
    ("n_tokens", lambda: read(T=0)),
]


@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_refused(i):
    text, call = REFUSED[i]
    with pytest.raises(bq.LlmError) as e:
        call()
    assert text in str(e.value), str(e.value)


def attend(B=4, n=2, H=4, hd=64, G=2, dtype=BF16, cache=None, tree=None, prefix=None, size=None, **kw):
    q = Fake((B, n, H, hd), dtype)
    a = dict(q=q, prefix=prefix or view(G, hd=hd), starts=Fake((G + 1,), I32), prefix_lens=Fake((G,), I32),
             cache=cache or view(B, hd=hd), tree=tree or view(B, rows=n, hd=hd), lens=Fake((B,), I32),
             mask=Fake((B, n), torch.int64), out=Fake((B, n, H, hd), dtype), workspace=Fake((1 << 20,), torch.uint8))
    a.update(kw)
    bq.prefix_attention(**a)


REFUSED_PREFIX = [
    ("n_nodes", lambda: attend(n=65, tree=view(4, rows=65))),
    ("queries of type float16", lambda: attend(dtype=torch.float16)),
    ("out must have", lambda: attend(out=Fake((4, 2, 4, 64), F32))),
    ("multiple of the cache's heads", lambda: attend(H=3)),
    ("head_dim 64, the cache 128", lambda: attend(cache=view(4, hd=128))),
    ("fewer sequences", lambda: attend(cache=view(3))),
    ("scale is not finite", lambda: attend(scale=float("inf"))),
    ("contiguous int32", lambda: attend(starts=Fake((2,), I32))),
    ("contiguous int32", lambda: attend(prefix_lens=Fake((2,), torch.int64))),
    ("contiguous int64", lambda: attend(mask=Fake((4, 2), I32))),
    ("not aligned", lambda: attend(cache=view(4, at=(1 << 20) + 8))),
]


@pytest.mark.parametrize("i", range(len(REFUSED_PREFIX)))
def test_prefix_refused(i):
    text, call = REFUSED_PREFIX[i]
    with pytest.raises(bq.LlmError) as e:
        call()
    assert text in str(e.value), str(e.value)


def test_prefix_workspace_sizes():
    assert bq.prefix_workspace(Fake((4, 2, 6, 64))) == 4 * 2 * 6 * (8 * (64 * 4 + 8) + 4)
    for shape in ((0, 2, 6, 64), (4, 65, 6, 64), (4, 2, 6, 96), (4, 2, 0, 128), (1 << 17, 2, 6, 64)):
        with pytest.raises(bq.LlmError):
            bq.prefix_workspace(Fake(shape))


def sample(R=3, V=100, **kw):
    f = lambda *s: Fake(s, F32)  # noqa: E731
    a = dict(logits=f(R, V), uniforms=f(R), tokens=Fake((R,), I32), temperature=f(R), top_k=Fake((R,), I32), top_p=f(R),
             min_p=f(R), probs=f(R))
    a.update(kw)
    bq.sample_tokens(**a)


REFUSED_SAMPLE = [
    ("logits: float32", lambda: sample(logits=Fake((3, 100), BF16))),
    ("logits: float32", lambda: sample(logits=Fake((3, 100), F32, stride=(200, 2)))),
    ("uniforms is needed", lambda: sample(uniforms=None)),
    ("tokens: a contiguous int32", lambda: sample(tokens=Fake((3,), torch.int64))),
    ("temperature: a contiguous float32", lambda: sample(temperature=Fake((2,), F32))),
    ("top_k: a contiguous int32", lambda: sample(top_k=Fake((3,), F32))),
    ("top_p: a contiguous float32", lambda: sample(top_p=Fake((3, 1), F32))),
    ("min_p: a contiguous float32", lambda: sample(min_p=Fake((3,), BF16))),
    ("probs: a contiguous float32", lambda: sample(probs=Fake((3,), I32))),
    ("n_rows or vocab", lambda: sample(R=0)),
    ("n_rows or vocab", lambda: sample(V=0)),
    ("too large", lambda: sample(V=524289)),
    ("not aligned", lambda: sample(logits=Fake((3, 100), F32, at=(1 << 20) + 2))),
]


@pytest.mark.parametrize("i", range(len(REFUSED_SAMPLE)))
def test_sample_refused(i):
    text, call = REFUSED_SAMPLE[i]
    with pytest.raises(bq.LlmError) as e:
        call()
    assert text in str(e.value), str(e.value)
