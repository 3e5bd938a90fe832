"""Verification of fixed choices whose tokens are a row's whole support (GPU).

Rows in fp32 (or bf16, widened) need not sum to 1, so every child of a node can be rejected although no other token has
mass: the rejection that leaves nothing does not count, and the next token is one of the target's. The reference decides
in exact fractions.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

import bit_quantized_token_gb300 as bq
from test_gpu_tree import gen

pytestmark = pytest.mark.gpu
BELOW_1 = 1 - 2.0 ** -24  # the largest fp32 number below 1


@pytest.fixture(scope="module", autouse=True)
def library():
    bq.build()
    torch.cuda.set_device(0)


def reference(tokens, parents, u, p):
    """One sequence: (path, next). p: a {token: probability} for every node."""
    cur, path = 0, [0]
    r, m = {t: Fraction(x) for t, x in p[0].items()}, Fraction(1)
    for i in range(1, len(tokens)):
        if parents[i] != cur:
            continue
        x = r.get(tokens[i], Fraction(0))
        if Fraction(u[i]) * m < x:
            cur, r, m = i, {t: Fraction(y) for t, y in p[i].items()}, Fraction(1)
            path.append(i)
        elif sum(r.values()) > x:
            m -= x
            r[tokens[i]] = Fraction(0)
    total, run = sum(r.values()), Fraction(0)
    for t in sorted(r):
        run += r[t]
        if run > Fraction(u[0]) * total:
            return path, t
    raise AssertionError("a row without mass")


def verify(tokens, parents, u, probs):
    t = [torch.tensor(x, dtype=d, device="cuda") for x, d in ((tokens, torch.int32), (parents, torch.int32),
                                                            (u, torch.float32))]
    B, n = t[0].shape
    path = torch.empty(B, n, dtype=torch.int32, device="cuda")
    n_path, nxt = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
    bq.verify_tree(*t, probs, path, n_path, nxt)
    return path.tolist(), n_path.tolist(), nxt.tolist()


def test_two_tokens_that_sum_to_less_than_one():
    p = torch.zeros(1, 3, 32, device="cuda")
    p[:, :, 2], p[:, :, 5] = 0.9998816, 0.000118301316
    u = [[0.25, 0.99999994, 0.9996895]]
    path, n_path, nxt = verify([[0, 2, 5]], [[-1, 0, 0]], u, p)
    assert (path, n_path, nxt) == ([[0, -1, -1]], [1], [5])


@pytest.mark.parametrize("V", [7, 300, 32000, 70001])
@pytest.mark.parametrize("rounded", ["fp32", "bf16"])
def test_children_cover_the_support(rounded, V):
    """Rows of one to four tokens, all of them children of the root in any order, with doubles (the same token twice,
    the second with children of its own) and tokens without probability among them; uniforms that reject what they can."""
    B, n = 300, 9
    rng = np.random.default_rng(V)
    probs = torch.zeros(B, n, V)
    tokens, parents, u = np.zeros((B, n), int), np.zeros((B, n), int), np.zeros((B, n), np.float32)
    rows = []
    for b in range(B):
        rows.append([])
        for i in range(n):
            k = int(rng.integers(1, 5))
            ids = rng.choice(V, k, replace=False)
            x = np.exp(4 * rng.standard_normal(k)).astype(np.float32)
            x = torch.tensor(x / x.sum(dtype=np.float32))
            x = (x.bfloat16().float() if rounded == "bf16" else x)
            x = torch.where(x < 1, x, torch.tensor(1 - 2.0 ** -9))  # (a row of one token is rejected too)
            probs[b, i, torch.tensor(ids)] = x
            rows[b].append(dict(zip(ids.tolist(), x.tolist())))
        parents[b] = [-1] + [0] * 6 + [int(rng.integers(1, 7)) for _ in range(2)]
        for i in range(1, n):
            of = list(rows[b][parents[b, i]])
            tokens[b, i] = rng.choice(of) if rng.random() < 0.8 else rng.integers(0, V)
        order = rng.permutation(list(rows[b][0]))
        at = rng.permutation(np.arange(1, 7))[:len(order)]
        tokens[b, at] = order
        u[b] = np.where(rng.random(n) < 0.9, BELOW_1, rng.random(n).astype(np.float32) * np.float32(BELOW_1))
    path, n_path, nxt = verify(tokens, parents, u, probs.cuda())
    nothing_left = 0
    for b in range(B):
        want, t = reference(tokens[b].tolist(), parents[b].tolist(), u[b].tolist(), rows[b])
        assert path[b] == want + [-1] * (n - len(want)) and n_path[b] == len(want) and nxt[b] == t, b
        kids = {int(tokens[b, i]) for i in range(1, n) if parents[b, i] == want[-1]}
        nothing_left += set(rows[b][want[-1]]) <= kids
    assert nothing_left > 30


@pytest.mark.parametrize("k", [1, 2, 3, 5])
def test_drafts_of_the_samplers_own_top_k(k):
    """token_probs' rows with all of their tokens drafted: what comes out always has a probability."""
    B, V = 4000, 1000
    logits = 3 * torch.randn(B, V, device="cuda", generator=gen(k))
    probs = torch.empty_like(logits)
    bq.token_probs(logits, probs, 0.8, k, 1.0)
    tokens = torch.zeros(B, k + 1, dtype=torch.int64, device="cuda")
    tokens[:, 1:] = probs.topk(k, -1).indices
    u = torch.full((B, k + 1), BELOW_1, device="cuda")
    u[:, 2:] -= torch.randint(0, 4096, (B, k - 1), device="cuda", generator=gen(1)) * 2.0 ** -24 if k > 1 else 0
    parents = [[-1] + [0] * k] * B
    path, n_path, nxt = verify(tokens.tolist(), parents, u.tolist(), probs[:, None].expand(B, k + 1, V))
    for b in range(B):
        if n_path[b] == 1:
            assert float(probs[b, nxt[b]]) > 0, b
        else:
            assert float(probs[b, int(tokens[b, path[b][1]])]) > 0, b
