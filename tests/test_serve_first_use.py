"""First use of the serving operators by two threads at once (no GPU needed)."""
import threading

import torch

import bit_quantized_token_gb300 as bq
from bit_quantized_token_gb300 import serve, tree
from test_serve_args import Fake


class Slow:
    """The tree binding's names; while one of the types is looked up another thread comes in, once."""

    def __init__(self, other):
        self._other, self._done = other, False

    def __getattr__(self, name):
        if name == "_bf16" and not self._done:
            self._done = True
            t = threading.Thread(target=self._other)
            t.start()
            t.join()
        return getattr(tree, name)


def test_two_threads(monkeypatch):
    """The second thread finds every type or none, and fills them in itself."""
    bq.build()
    kinds = []

    def other():
        try:
            serve._load()
            kinds.append([serve._kind(Fake((1,), d), "k") for d in (torch.bfloat16, torch.float32)])
        except bq.LlmError as e:
            kinds.append(e)

    tree._load()
    monkeypatch.setattr(serve, "_DTYPES", {})
    monkeypatch.setattr(serve, "_t", Slow(other))
    serve._load()
    want = [bq.LLM_BF16, bq.LLM_F32]
    assert kinds == [want]
    assert [serve._kind(Fake((1,), d), "k") for d in (torch.bfloat16, torch.float32)] == want
