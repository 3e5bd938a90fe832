"""Bounded waits of the attention behind shared prefixes, made to run out (GPU).

As for the tree operators: a barrier of each CTA expects more arrivals than it gets, with a limit of 1 ms, in either
part of the call. The kernels give up in order, the status says so, and the next calls are as ever.
"""
import pytest
import torch

import bit_quantized_token_gb300 as bq
from test_gpu_prefix import Problem
from test_gpu_tree_waits import times_out

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def library():
    bq.build()
    torch.cuda.set_device(0)
    yield
    bq.debug_expire_waits(False)


# one row tile and several of a group, few rows (the tree attention's kernel), several groups, one of them empty
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("kv,q,starts,n,plens", [
    ("bf16", "bf16", (0, 70), 1, (900,)), ("bf16", "bf16", (0, 200, 200, 330), 1, (4100, 5, 63)),
    ("bf16", "bf16", (0, 3), 1, (2000,)), ("bf16", "f32", (0, 40, 90), 3, (700, 300)),
    ("q8", "bf16", (0, 40, 90), 3, (700, 0))], ids=["70", "330", "3", "f32", "q8"])
def test_attention(kv, q, starts, n, plens, hd):
    p = Problem(starts=starts, n=n, hd=hd, gq=4, P=max(plens), plens=plens, lens=(17, 40, 0), q=q, kv=kv, counts=(n, 1))

    def call():
        p.call()
        bq.tree_status()

    times_out(call)
    for b, c in enumerate(p.counts):
        assert (p.out[b, c:] == 7.0).all(), "rows past the count were written"
    p.out.fill_(7.0)
    call()
    p.check()
