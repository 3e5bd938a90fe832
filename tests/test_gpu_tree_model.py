"""llm_decode_tree: a drafted tree through the model's own pipeline, against the oracle (GPU).

Bars as in the batched pipeline's tests: logits at 5e-3 of max|logit|; greedy tokens identical to the oracle's;
appended K/V rows against token-by-token decoding at 1e-2 of a row's largest value (bf16 neighbours travel).
Sampled verification is decided from the call's own logits, in 64 bits.
"""
import numpy as np
import pytest
import torch

import bit_quantized_token_gb300 as bq
import oracle
import synth
from test_gpu_tree import probs_reference, verify_reference

pytestmark = pytest.mark.gpu
LOGIT_REL = 5e-3


@pytest.fixture(scope="module", autouse=True)
def _built():
    bq.build()
    oracle.build()


def config(name):
    cfg = dict(synth.workload(0 if name == "tiny" else 2))
    if name == "qwen":  # two layers and a small vocabulary of the 128-dim, q/k-normed, tied shape
        cfg.update(n_layers=2, vocab=4099)
    return cfg


def tree_around(rng, right, vocab, n, chain):
    """n nodes: node 0 is right[0]; the right tokens up to depth `chain` lie on one path, the others are random."""
    tokens, parents, on, depth = [right[0]], [-1], [0], [0]
    while len(tokens) < n:
        i = len(tokens)
        left = n - i
        if len(on) <= chain and (rng.random() < 0.4 or left <= chain + 1 - len(on)):
            parents.append(on[-1])
            tokens.append(right[len(on)])
            depth.append(len(on))
            on.append(i)
        else:
            par = int(rng.integers(0, i))
            t = int(rng.integers(0, vocab))
            if par in on and t == right[on.index(par) + 1]:
                t = (t + 1) % vocab
            parents.append(par)
            tokens.append(t)
            depth.append(depth[par] + 1)
    return tokens, parents, on


@pytest.mark.parametrize("name,flags", [("tiny", 0), ("tiny", bq.LLM_NO_PDL), ("qwen", 0), ("tiny", bq.LLM_KV_Q8),
                                        ("qwen", bq.LLM_KV_Q8)])
def test_greedy_trees_decode_like_the_oracle(name, flags):
    cfg = config(name)
    w = synth.make_weights(cfg)
    om = oracle.OracleModel(cfg, w)
    kv = "q8" if flags & bq.LLM_KV_Q8 else "bf16"
    prompt = [int(t) for t in synth.make_prompt(cfg)]
    rng = np.random.default_rng(3)
    cap = 96
    cache = om.new_cache(cap, kv) if kv == "q8" else om.new_cache(cap)
    for t in prompt:
        ref = om.step(cache, t)
    right = [oracle.argmax_f32(ref)]
    refs = []
    for _ in range(30):
        refs.append(om.step(cache, right[-1]))
        right.append(oracle.argmax_f32(refs[-1]))
    with bq.Model(cfg, w, max_seq=cap, max_batch=2, flags=flags) as m:
        seq, at = 1, 0
        m.prefill(seq, prompt)
        for n, chain in ((1, 0), (2, 1), (7, 3), (32, 5), (13, 0), (9, 8)):
            tokens, parents, on = tree_around(rng, right[at:], cfg["vocab"], n, chain)
            logits = np.empty((n, cfg["vocab"]), np.float32)
            path, nxt = m.decode_tree(seq, tokens, parents, logits=logits)
            assert path.tolist() == on, (n, chain)
            assert nxt == right[at + len(on)]
            for d, node in enumerate(on):
                r = refs[at + d]
                err = np.abs(logits[node] - r).max() / np.abs(r).max()
                assert err <= LOGIT_REL, (n, node, err)
            at += len(on)
            assert m.kv_len(seq) == len(prompt) + at and m.kv_len(0) == 0
        rest = m.decode_greedy(seq, right[at], 4).tolist()  # the plain steps continue from there
        assert rest == right[at + 1:at + 5]
        # the appended rows against token-by-token decoding
        m.prefill(0, prompt)
        m.decode_greedy(0, right[0], at)
        for l in range(cfg["n_layers"]):
            for a, b in zip(rows(m, 0, l, len(prompt), at, kv), rows(m, seq, l, len(prompt), at, kv)):
                tol = 1e-2 if kv == "bf16" else 2.0 / 127 + 1e-2  # a code may fall to its neighbour
                assert (np.abs(a - b) <= tol * np.abs(a).max(-1, keepdims=True)).all(), l


def rows(m, seq, l, pos0, n, kv):
    if kv == "bf16":
        return [(x.astype(np.uint32) << 16).view(np.float32) for x in m.kv_read(seq, l, pos0, n)]
    k, ks, v, vs = m.kv_read_q8(seq, l, pos0, n)
    return [c.astype(np.float32) * np.repeat(s.view(np.float16).astype(np.float32), 32, -1) for c, s in ((k, ks), (v, vs))]


def test_every_branch_sees_its_own_ancestors():
    """Logits of nodes off the kept path: each equals the oracle's after the tokens of its own branch."""
    cfg = config("tiny")
    w = synth.make_weights(cfg)
    om = oracle.OracleModel(cfg, w)
    prompt = [int(t) for t in synth.make_prompt(cfg)]
    rng = np.random.default_rng(5)
    n = 12
    tokens = [int(t) for t in rng.integers(0, cfg["vocab"], n)]
    parents = [-1] + [int(rng.integers(0, i)) for i in range(1, n)]
    with bq.Model(cfg, w, max_seq=64) as m:
        m.prefill_batched(0, prompt)
        logits = torch.empty(n, cfg["vocab"], device="cuda")
        m.decode_tree(0, tokens, parents, logits=logits)
        logits = logits.cpu().numpy()
    for i in range(n):
        branch, j = [], i
        while j >= 0:
            branch.insert(0, tokens[j])
            j = parents[j]
        cache = om.new_cache(64)
        for t in prompt + branch:
            ref = om.step(cache, t)
        err = np.abs(logits[i] - ref).max() / np.abs(ref).max()
        assert err <= LOGIT_REL, (i, err)


@pytest.mark.parametrize("soft", [False, True])
def test_sampled_trees_follow_the_verification_of_their_logits(soft):
    cfg = config("tiny")
    w = synth.make_weights(cfg)
    rng = np.random.default_rng(7)
    V, n = cfg["vocab"], 10
    T, k, p = 1.1, 30, 0.9
    kept = 0
    with bq.Model(cfg, w, max_seq=400) as m:
        m.prefill(0, synth.make_prompt(cfg))
        m.set_sampling(T, top_k=k, top_p=p, seed=1)
        tok = 3
        for step in range(20):
            parents = [-1] + [int(rng.integers(max(0, i - 3), i)) for i in range(1, n)]
            tokens = [tok] + [int(t) for t in rng.integers(0, V, n - 1)]
            u = rng.random(n).astype(np.float32)
            q = None
            if step:  # drafts from the last step's distributions, so that some are kept
                best = np.argsort(-last)[:8]
                for i in range(1, n):
                    tokens[i] = int(best[rng.integers(0, 8)])
            if soft:
                q = np.full((n, V), 0.02 / V, np.float32)
                for i in range(1, n):
                    q[parents[i], tokens[i]] += 0.1
            logits = np.empty((n, V), np.float32)
            before = m.kv_len(0)
            path, nxt = m.decode_tree(0, tokens, parents, draft_probs=None if q is None else torch.tensor(q).cuda(),
                                      uniforms=u, logits=logits)
            probs = np.stack([probs_reference(logits[i], T, k, p) for i in range(n)])
            want, t = verify_reference(tokens, parents, u, probs, q, n)
            assert path.tolist() == want and nxt == t, step
            assert m.kv_len(0) == before + len(want)
            kept += len(want) - 1
            last, tok = probs[want[-1]], nxt
        m.set_sampling(0.0)
        m.decode_tree(0, [tok], [-1])
    assert kept > 0


def test_refusals_leave_the_model_usable():
    cfg = config("tiny")
    w = synth.make_weights(cfg)
    prompt = synth.make_prompt(cfg)
    with bq.Model(cfg, w, max_seq=32) as m:
        m.prefill(0, prompt)
        at = m.kv_len(0)
        V = cfg["vocab"]
        for words, call in [("1 to 32 nodes", lambda: m.decode_tree(0, [1] * 33, [-1] + [0] * 32)),
                            ("exceed max_seq", lambda: m.decode_tree(0, [1] * 17, [-1] + [0] * 16)),
                            ("lower node", lambda: m.decode_tree(0, [1, 2], [-1, 1])),
                            ("lower node", lambda: m.decode_tree(0, [1, 2], [-1, -1])),
                            ("out of range", lambda: m.decode_tree(0, [1, V], [-1, 0])),
                            ("seq out of range", lambda: m.decode_tree(1, [1], [-1])),
                            ("one length", lambda: m.decode_tree(0, [1, 2], [-1])),
                            ("draft_probs are for sampled",
                             lambda: m.decode_tree(0, [1], [-1], draft_probs=torch.zeros(1, V).cuda()))]:
            with pytest.raises(bq.LlmError, match=words):
                call()
        m.set_sampling(0.7, top_k=5)
        for words, kw in [("needs uniforms", {}), (r"\[0, 1\)", dict(uniforms=[1.0])),
                          (r"\[0, 1\)", dict(uniforms=[float("nan")])),
                          ("device memory", dict(uniforms=[0.5], draft_probs=np.zeros((1, V), np.float32)))]:
            with pytest.raises(bq.LlmError, match=words):
                m.decode_tree(0, [1], [-1], **kw)
        m.set_sampling(0.0)
        assert m.kv_len(0) == at
        _, tok = m.decode_tree(0, [5], [-1])
        am = np.zeros(1, np.int32)
        m.kv_reset(0)
        m.prefill(0, list(prompt) + [5], argmax=am)
        assert tok == int(am[0])


def test_nan_leaves_the_sequence_as_it_was():
    cfg = config("tiny")
    w = synth.make_weights(cfg)
    w["final_norm"]["data"] = w["final_norm"]["data"].copy()
    w["final_norm"]["data"].reshape(-1)[0] = np.nan
    with bq.Model(cfg, w, max_seq=32) as m:
        rng = np.random.default_rng(0)
        kv = rng.integers(0, 1 << 14, (4, cfg["n_kv_heads"], cfg["head_dim"])).astype(np.uint16)
        m.kv_write(0, 0, 0, kv, kv)
        with pytest.raises(bq.LlmError, match="NaN"):
            m.decode_tree(0, [1, 2], [-1, 0])
        assert m.kv_len(0) == 4
