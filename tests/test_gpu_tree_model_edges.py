"""llm_decode_tree as a caller meets it: what it leaves behind on an error, what has run when it returns (GPU)."""
import numpy as np
import pytest
import torch

import bit_quantized_token_gb300 as bq
import synth
from test_gpu_tree_model import config, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    bq.build()


@pytest.mark.parametrize("temperature", [0.0, 0.9])
def test_an_error_leaves_rows_length_and_next_token(temperature):
    """A node whose embedding is NaN fails the call; the sequences then go on as in a model that never saw it."""
    cfg = config("tiny")
    w = synth.make_weights(cfg)
    bad = 77
    w["embed"]["data"] = w["embed"]["data"].copy()
    w["embed"]["data"].reshape(cfg["vocab"], -1)[bad] = np.nan
    prompts = [[5, 9, 2], [1, 3]]
    ends = []
    for fail in (False, True):
        with bq.Model(cfg, w, max_seq=48, max_batch=2) as m:
            for s, p in enumerate(prompts):
                m.prefill(s, p)
            m.decode_step_batch([4, 6])  # leaves each sequence's next token on the device
            before = [m.kv_len(s) for s in range(2)]
            if fail:
                m.set_sampling(temperature, top_k=4)
                with pytest.raises(bq.LlmError, match="NaN"):
                    m.decode_tree(1, [8, 3, bad, 2], [-1, 0, 1, 0], uniforms=[0.5] * 4)
                m.set_sampling(0.0)
                assert [m.kv_len(s) for s in range(2)] == before
            got = []
            for _ in range(3):
                am = np.zeros(2, np.int32)
                m.decode_step_batch(None, argmax=am)
                got.append(am.tolist())
            ends.append((got, [np.stack(rows(m, 1, l, 0, m.kv_len(1), "bf16")) for l in range(cfg["n_layers"])]))
    assert ends[0][0] == ends[1][0]
    for a, b in zip(ends[0][1], ends[1][1]):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("flags", [0, bq.LLM_KV_Q8])
def test_batched_steps_continue_from_the_next_token(flags):
    """After a tree the device-side token is the one that follows the kept nodes."""
    cfg = config("tiny")
    w = synth.make_weights(cfg)
    with bq.Model(cfg, w, max_seq=48, max_batch=2, flags=flags) as m:
        m.prefill(0, [5, 9, 2])
        m.prefill(1, [1, 3])
        try:
            m.decode_step_batch([4, 6])
        except bq.LlmError as e:
            pytest.skip(str(e))
        path, nxt = m.decode_tree(1, [8, 3, 2], [-1, 0, 0])
        a, b = np.zeros(2, np.int32), np.zeros(2, np.int32)
        m.decode_step_batch(None, argmax=a)
    with bq.Model(cfg, w, max_seq=48, max_batch=2, flags=flags) as m:
        m.prefill(0, [5, 9, 2])
        m.prefill(1, [1, 3])
        m.decode_step_batch([4, 6])
        _, again = m.decode_tree(1, [8, 3, 2], [-1, 0, 0])
        assert again == nxt
        am = np.zeros(2, np.int32)
        m.decode_step(1, nxt, argmax=am)
        b[1] = am[0]
    assert a[1] == b[1]


def test_all_work_has_run_when_the_call_returns():
    """The call is synchronous: nothing is left on the model's stream, the commit and the next token among it. Large
    kernels on another stream delay every launch, so that what the call would leave behind is still there."""
    cfg = config("tiny")
    stream = torch.cuda.Stream()
    tokens, parents = np.array([8, 3, 2], np.int32), np.array([-1, 0, 0], np.int32)
    out = [np.zeros(k, np.int32) for k in (3, 1, 1)]
    at = [x.ctypes.data for x in out]
    with bq.Model(cfg, synth.make_weights(cfg), max_seq=400, stream=stream.cuda_stream) as m:
        m.prefill(0, [5, 9, 2])
        call, busy = bq.lib().llm_decode_tree, 0
        x = torch.zeros(1 << 28, device="cuda")
        other = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            for _ in range(400):
                x.add_(1.0)
        for _ in range(4):
            rc = call(m.h, 0, tokens.ctypes.data, parents.ctypes.data, 3, None, None, *at, None)
            busy += not stream.query()
            assert rc == 0
        assert not other.query(), "the other stream had nothing left to do"
        other.synchronize()
    assert busy == 0


@pytest.mark.parametrize("side", [False, True], ids=["default-stream", "side-stream"])
def test_draft_probabilities_in_the_making(side):
    """draft_probs written by work that the caller's stream has yet to run, at the call."""
    cfg = config("tiny")
    V = cfg["vocab"]
    with bq.Model(cfg, synth.make_weights(cfg), max_seq=48) as m:
        m.set_sampling(2.0, top_k=50, top_p=1.0)

        def step(x, q, stream=None):
            m.kv_reset(0)
            m.prefill(0, [5, 9, 2])
            if stream is not None:  # q is on its way
                torch.cuda._sleep(200_000_000)  # about 0.1 s
                q.copy_(sure)
                assert not stream.query()
            logits = np.empty((2, V), np.float32)
            path, nxt = m.decode_tree(0, [3, x], [-1, 0], draft_probs=q, uniforms=[0.5, 0.97], logits=logits)
            return path.tolist(), nxt, logits[0]

        x = int(step(1, torch.zeros(2, V, device="cuda"))[2].argmax())
        sure = torch.zeros(2, V, device="cuda")
        sure[0, x] = 1.0
        zeros = torch.zeros(2, V, device="cuda")
        torch.cuda.synchronize()
        assert step(x, zeros)[0] == [0, 1]  # a draft that had no probability is kept: what reading early gives
        want = step(x, sure)
        assert want[0] == [0]
        stream = torch.cuda.Stream() if side else torch.cuda.default_stream()
        for _ in range(3):
            q = torch.zeros(2, V, device="cuda")
            torch.cuda.synchronize()
            with torch.cuda.stream(stream):
                got = step(x, q, stream)
            assert got[:2] == want[:2]


def test_rows_of_another_size_or_type_are_refused():
    cfg = config("tiny")
    V = cfg["vocab"]
    with bq.Model(cfg, synth.make_weights(cfg), max_seq=48) as m:
        m.prefill(0, [5, 9, 2])
        m.set_sampling(0.7, top_k=5)
        tree, u = ([8, 3, 2], [-1, 0, 0]), [0.5] * 3
        zeros = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
        for q in (zeros(2, V), zeros(3, V - 1), zeros(3, V, dtype=torch.float64), zeros(3, V, dtype=torch.bfloat16),
                  zeros(3, 2 * V)[:, :V], zeros(2 * V)):
            with pytest.raises(bq.LlmError, match="draft_probs: contiguous float32"):
                m.decode_tree(0, *tree, draft_probs=q, uniforms=u)
        for out in (np.zeros((2, V), np.float32), np.zeros((3, V)), np.zeros((V, 3), np.float32).T,
                    zeros(2, V)):
            with pytest.raises(bq.LlmError, match="logits: contiguous float32"):
                m.decode_tree(0, *tree, uniforms=u, logits=out)
        assert m.kv_len(0) == 3
        m.decode_tree(0, *tree, uniforms=u, draft_probs=zeros(32, V),  # room for more nodes
                      logits=np.zeros((32, V), np.float32))


def test_sampling_over_too_large_a_vocabulary_is_refused():
    cfg = dict(config("tiny"), vocab=524_320, dim=128, ffn_dim=128, n_layers=1, n_heads=2, n_kv_heads=2)
    with bq.Model(cfg, synth.make_weights(cfg), max_seq=32) as m:
        m.prefill(0, [5, 9, 2])
        m.set_sampling(0.7, top_k=5)
        with pytest.raises(bq.LlmError, match="UNSUPPORTED.*524288") as e:
            m.decode_tree(0, [8, 3], [-1, 0], uniforms=[0.5, 0.5])
        assert e.value.code == -2
        m.set_sampling(0.0)
        assert m.kv_len(0) == 3
        path, _ = m.decode_tree(0, [8], [-1])  # the model is as before
        assert path.tolist() == [0] and m.kv_len(0) == 4


@pytest.mark.parametrize("temperature", [1e-3, 1e-30, 5e-39, 1e-40, 1.5e-45])
def test_sampling_at_the_smallest_temperatures_is_greedy(temperature):
    """set_sampling takes any temperature above 0: down to the smallest fp32 number the largest logit has it all."""
    cfg = config("tiny")
    with bq.Model(cfg, synth.make_weights(cfg), max_seq=48) as m:
        m.prefill(0, [5, 9, 2])
        logits = np.empty((3, cfg["vocab"]), np.float32)
        _, first = m.decode_tree(0, [8], [-1], logits=logits[:1])
        m.kv_reset(0)
        m.prefill(0, [5, 9, 2])
        m.set_sampling(temperature, top_k=20, top_p=1.0)
        tokens = [8, (first + 1) % cfg["vocab"], first]
        path, nxt = m.decode_tree(0, tokens, [-1, 0, 0], uniforms=[0.99, 0.0, 0.99], logits=logits)
        gap = np.sort(logits, -1)
        # the others' mass: at most 19 e^-10 < 1e-3 of the largest's, which passes 0.99 and, first or not, is drawn
        assert (gap[:, -1] - gap[:, -2] > 10 * temperature).all()
        assert path.tolist() == [0, 2] and nxt == int(logits[2].argmax())
