"""Bounded waits of the tree operators, made to run out (GPU).

One barrier of each CTA expects an arrival more than it gets, with a limit of 1 ms: the kernel gives up, lets its own
copies and products finish, frees what it holds and returns, and the status says so. Nothing faults, traps or hangs.
"""
import numpy as np
import pytest
import torch

import bit_quantized_token_gb300 as bq
import synth
from test_gpu_tree import Problem, gen
from test_gpu_tree_model import config

pytestmark = pytest.mark.gpu
TIMEOUT = -6


@pytest.fixture(autouse=True)
def library():
    bq.build()
    torch.cuda.set_device(0)
    yield
    bq.debug_expire_waits(False)


def times_out(call):
    bq.debug_expire_waits(True)
    try:
        with pytest.raises(bq.LlmError, match="wait") as e:
            call()
    finally:
        bq.debug_expire_waits(False)
    assert e.value.code == TIMEOUT


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("kv", ["bf16", "q8"])
@pytest.mark.parametrize("q", ["bf16", "f32"])
@pytest.mark.parametrize("n,lens", [(1, (40,)), (6, (3000, 200)), (64, (700, 1500, 0)),
                                    (64, (300, 900) * 10)], ids=["1", "2x6", "3x64", "20x64"])
def test_attention(n, lens, q, kv, hd):
    p = Problem(B=len(lens), n=n, Hkv=2, gq=2, hd=hd, cap=max(lens) + 1, lens=lens, q=q, kv=kv)
    p.counts = torch.tensor([n] + [max(1, n - 3)] * (len(lens) - 1), dtype=torch.int32, device="cuda")
    times_out(p.call)
    for b in range(len(lens)):
        assert (p.out[b, int(p.counts[b]):] == 7.0).all(), "rows past the count were written"
    p.out.fill_(7.0)
    p.call()  # the status was taken back: the next calls are as ever
    p.check()


@pytest.mark.parametrize("R,V", [(1, 5), (3, 32000), (40, 151936), (2, 300001)])
def test_token_probs(R, V):
    x = 3 * torch.randn(R, V, device="cuda", generator=gen(V))
    out = torch.full((R, V + 4), 7.0, device="cuda")

    def call():
        bq.token_probs(x, out[:, :V])
        bq.tree_status()

    times_out(call)
    assert (out[:, V:] == 7.0).all()
    call()
    ref = torch.softmax(x.double(), -1)
    assert ((out[:, :V] - ref).abs() <= 1e-4 * ref).all()


@pytest.mark.parametrize("flags", [0, bq.LLM_KV_Q8])
def test_decode_tree(flags):
    cfg = config("tiny")
    w = synth.make_weights(cfg)
    with bq.Model(cfg, w, max_seq=400, flags=flags) as m:
        m.prefill(0, [5, 9, 2] * 50)
        times_out(lambda: m.decode_tree(0, [8, 3, 2], [-1, 0, 0]))
        assert m.kv_len(0) == 150
        with pytest.raises(bq.LlmError) as e:  # the model refuses further work
            m.decode_tree(0, [8], [-1])
        assert e.value.code == TIMEOUT
    with bq.Model(cfg, w, max_seq=400, flags=flags) as m:
        m.prefill(0, [5, 9, 2] * 50)
        am = np.zeros(1, np.int32)
        path, nxt = m.decode_tree(0, [8], [-1])
        m.kv_reset(0)
        m.prefill(0, [5, 9, 2] * 50 + [8], argmax=am)
        assert path.tolist() == [0] and nxt == int(am[0])
