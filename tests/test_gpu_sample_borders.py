"""sample_tokens where a border falls between two buckets of its histogram, or on odd values (GPU)."""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import bit_quantized_token_gb300 as bq
from test_gpu_sample_rows import choose

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    bq.build()
    torch.cuda.set_device(0)


def draw(x, u, **options):
    R = x.shape[0]
    tokens, probs = torch.full((R,), -7, dtype=torch.int32, device="cuda"), torch.full((R,), -7.0, device="cuda")
    full = {k: torch.full((R,), v, device="cuda", dtype=torch.int32 if k == "top_k" else torch.float32) for k, v in options.items()}
    bq.sample_tokens(x, torch.full((R,), u, device="cuda"), tokens, probs=probs, **full)
    return tokens.cpu().numpy(), probs.cpu().numpy()


def rows_around_a_half(R, step):
    """A token at 0, `near` ones in the bucket from -0.0650 to -0.0433 and `far` ones below them in one bucket, and two
    that fill up, so that half of the row's mass is that of the first two kinds plus `step` times -R/2 .. R/2. (R rows;
    how many tokens of the first kinds)"""
    getcontext().prec = 40
    near, n_far = np.linspace(-0.045, -0.063, 2000).astype(np.float32), 3000
    far = np.linspace(-0.305, -0.320, n_far).astype(np.float32)
    exp = lambda v: Decimal(float(v)).exp()  # noqa: E731
    front = 1 + sum(map(exp, near))
    cum = np.cumsum(np.exp(far.astype(np.float64)))
    n_far = int(np.searchsorted(cum, float(front)))  # leaves less than a weight of theirs
    far = far[:n_far]
    left = front - sum(map(exp, far))
    first = np.float32(float(left.ln()) - 2.0 ** -20)    # leaves about 2^-20 of its weight
    left -= exp(first)
    x = np.empty((R, 1 + len(near) + n_far + 2), np.float32)
    x[:, 0], x[:, 1:2001], x[:, 2001:-2], x[:, -2] = 0, near, far, first
    x[:, -1] = [float((left + 2 * Decimal(step) * (r - R // 2)).ln()) for r in range(R)]
    return x, 2001


def test_borders_between_buckets():
    """Half of the mass lies within 2^-36 of the whole, in steps of 2^-44 of the largest weight times 800, around the end
    of a bucket: its tokens add up to a little less than the bucket, since every weight is rounded, and a border between
    the two is at the bucket's last token or the one behind it, never at some other of the gathered ones."""
    x, n = rows_around_a_half(2048, 800 * 2.0 ** -44)
    order = np.argsort(-x[0], kind="stable")
    xs = torch.from_numpy(x).cuda()
    tokens, _ = draw(xs, 0.5)
    assert set(tokens.tolist()) <= {int(order[n - 1]), int(order[n])}
    for u in (0.25, 0.999):
        kept = {choose(x[0], 1.0, k, 1.0, 0.0, np.float32(u))[0] for k in (n - 1, n, n + 1)}
        assert set(draw(xs, u, top_p=0.5)[0].tolist()) <= kept
        assert set(draw(xs, u, top_p=0.5, min_p=0.5)[0].tolist()) <= kept
        assert set(draw(xs, u, top_p=0.5, top_k=x.shape[1] - 1)[0].tolist()) <= kept


@pytest.mark.parametrize("V,at", [(3000, 2999), (3000, 5), (9001, 5), (40000, 20001)])
def test_an_infinite_logit_at_an_infinite_temperature(V, at):
    """All tokens but those of -inf are alike; an infinite logit counts as the largest finite one."""
    x = torch.zeros(8, V, device="cuda")
    x[:, at] = math.inf
    x[:, 7] = -math.inf
    for u in (0.0, 0.5, 0.99):
        token, prob = choose(x[0].cpu().numpy(), math.inf, 0, 1.0, 0.0, np.float32(u))
        tokens, probs = draw(x, u, temperature=math.inf)
        assert set(tokens.tolist()) == {token}
        assert (abs(probs - prob) <= prob * 2.0 ** -20).all()


@pytest.mark.parametrize("gap", [1, 512, 4096])
def test_the_largest_finite_and_an_infinite_logit_are_a_tie(gap):
    """The lower id is the greedy choice, whether or not one thread has the two."""
    x = torch.zeros(2, 9000, device="cuda")
    x[0, 100], x[0, 100 + gap] = torch.finfo(torch.float32).max, math.inf
    x[1, 100], x[1, 100 + gap] = math.inf, torch.finfo(torch.float32).max
    tokens, probs = draw(x, 0.5, temperature=0.0)
    assert tokens.tolist() == [100, 100] and probs.tolist() == [1.0, 1.0]


@pytest.mark.parametrize("below", [2.8, 3.1, 4.0, 5.5])
def test_equal_logits_in_the_tail(below):
    """One token and 4000 equal ones below 1/16 of it, draws at their borders. The equal ones have the same error: the
    place is rounded by 2^-25 of a bucket of 2^28.5 steps, the polynomial and their product by 16 steps each, the rest
    comes to 2, so 45 steps of 2^-34 of the bucket's largest weight, 2^-28.5. The draw is off by 2^-28 of the mass at
    most."""
    n, R = 4000, 4000
    x = torch.full((1, 1 + n), -below, device="cuda")
    x[0, 0] = 0.0
    w = math.exp(float(x[0, 1]))
    total = 1 + n * w
    u = ((1 + w * np.arange(R)) / total).astype(np.float32)
    tokens = torch.empty(R, dtype=torch.int32, device="cuda")
    bq.sample_tokens(x.expand(R, -1), torch.from_numpy(u).cuda(), tokens)
    lo, hi = (np.floor((u.astype(np.float64) * total - 1 + s * 2.0 ** -28 * total) / w) + 1 for s in (-1, 1))
    got = tokens.cpu().numpy()
    assert ((got >= np.maximum(lo, 0)) & (got <= np.minimum(hi, n))).all()
