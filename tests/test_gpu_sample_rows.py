"""sample_tokens against a plain sampler in 64 bits (GPU).

Tokens are equal. Where a border lies within 2^-34 of the row's mass of the other side (sums are promised to 2^-36),
the neighbouring choice is right too. The probability of the token is within 2^-20: a term of 2^-30 (fixed point), exp2f,
three roundings and a sum of 2^-36.
"""
import math

import numpy as np
import pytest
import torch

import bit_quantized_token_gb300 as bq
import oracle.sampling
import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    bq.build()
    torch.cuda.set_device(0)


def choose(x, T, k, p, m, u, shift=(0.0, 0.0)):
    """(token, probability): the definition in 64 bits, the targets of top_p and of the draw shifted by parts of the mass."""
    x = np.where(np.isnan(x), -np.inf, np.minimum(x.astype(np.float64), np.finfo(np.float32).max))
    if not (x > -np.inf).any():
        return -1, 0.0
    if not T > 0:
        return int(x.argmax()), 1.0
    ids = np.argsort(-x, kind="stable")
    ids = ids[:int((x > -np.inf).sum())]
    w = np.exp((x[ids] - x[ids[0]]) / np.float64(T))
    w = w[w > 2.0 ** -64] if T < 1e30 else w
    whole = w.sum()
    if k > 0:
        w = w[:k]
    cum = np.cumsum(w)
    if p < 1:
        w = w[:max(1, int(np.searchsorted(cum, np.float64(max(p, 0.0)) * cum[-1] + shift[0] * whole)) + 1)]
    if m > 0:
        w = w[:int((w >= min(np.float64(m), 1.0)).sum())]
    cum = np.cumsum(w)
    u = min(np.float64(u), 1 - 2.0 ** -24) if u >= 0 else 0.0
    j = min(int(np.searchsorted(cum, u * cum[-1] + shift[1] * whole, side="right")), len(w) - 1)
    return int(ids[j]), w[j] / cum[-1]


def check(x, T, k, p, m, u, stream=None):
    R = x.shape[0]
    f = lambda v, t: torch.from_numpy(np.ascontiguousarray(np.broadcast_to(np.asarray(v, t), (R,)))).cuda()  # noqa: E731
    T, p, m, u = (np.broadcast_to(np.asarray(v, np.float32), (R,)) for v in (T, p, m, u))
    k = np.broadcast_to(np.asarray(k, np.int32), (R,))
    tokens = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    probs = torch.full((R,), -7.0, device="cuda")
    bq.sample_tokens(x, f(u, np.float32), tokens, f(T, np.float32), f(k, np.int32), f(p, np.float32), f(m, np.float32),
                     probs=probs, stream=stream)
    torch.cuda.synchronize()
    tokens, probs, xs, near = tokens.cpu().numpy(), probs.cpu().numpy(), x.cpu().numpy(), 0
    e = 2.0 ** -34
    for r in range(R):
        a = (xs[r], T[r], int(k[r]), p[r], m[r], u[r])
        want, prob = choose(*a)
        if tokens[r] != want:
            other = {choose(*a, shift=(i * e, j * e))[0] for i in (-1, 0, 1) for j in (-1, 0, 1)}
            assert tokens[r] in other, (r, a[1:], int(tokens[r]), want)
            near += 1
        else:
            assert abs(probs[r] - prob) <= prob * 2.0 ** -20, (r, a[1:], probs[r], prob)
    assert near <= max(1, R // 100)
    return tokens


def logits(R, V, sd, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return sd * torch.randn(R, V, device="cuda", generator=g)


def options(R, rng, V):
    return dict(T=rng.choice([0.0, 0.3, 0.7, 1.0, 1.0, 1.5, 2.5, 7.0], R), k=rng.choice([0, 0, 1, 2, 40, 300, max(1, V - 1), V], R),
                p=rng.choice([1.0, 1.0, 0.999, 0.95, 0.5, 0.01], R), m=rng.choice([0.0, 0.0, 0.001, 0.05, 0.3, 1.0], R),
                u=rng.random(R).astype(np.float32))


@pytest.mark.parametrize("V", [1, 2, 5, 31, 511, 513, 4097, 32000, 50257, 151936, 163841, 300001, 524288])
def test_every_option(V):
    rng = np.random.default_rng(V)
    R = 64 if V < 100000 else 24
    for sd in (2.5, 0.7):
        check(logits(R, V, sd, V), **options(R, rng, V))


@pytest.mark.parametrize("T", [1e-38, 1e-6, 0.05, 2.0, 20.0, 1e4, 1e30, math.inf])
def test_temperatures(T):
    rng = np.random.default_rng(7)
    R, V = 32, 9001
    check(logits(R, V, 3.0, 5), T=T, k=rng.choice([0, 50], R), p=rng.choice([1.0, 0.9], R), m=rng.choice([0.0, 0.1], R),
          u=rng.random(R))


@pytest.mark.parametrize("V", [3000, 40000, 151936])
def test_crowds(V):
    """Rows whose borders lie among thousands of equal or close logits: the long way."""
    rng = np.random.default_rng(V)
    R = 24
    o = options(R, rng, V)
    same = torch.zeros(R, V, device="cuda")
    check(same, **o)
    check(same - 17.25, T=1.0, k=0, p=0.5, m=0.0, u=np.linspace(0, 1, R, endpoint=False))
    two = same.clone()
    two[:, 1::3] = 1.5
    two[:, 2::3] = -200.0
    check(two, **o)
    check(logits(R, V, 2.0, 1).to(torch.bfloat16).float().round(), **o)  # whole numbers
    check(logits(R, V, 1e-4, 1), **o)  # all within one bucket
    check(logits(R, V, 2.5, 1).to(torch.bfloat16).float(), **o)
    mixed = logits(R, V, 0.002, 3)
    mixed[:, V // 2] = 5.0
    mixed[:, :100] = -math.inf
    check(mixed, **o)


@pytest.mark.parametrize("V,sd", [(151936, 2.5), (151936, 0.75), (151936, 0.1), (300001, 2.0), (524288, 1.0), (65536, 0.3)])
def test_flat_rows(V, sd):
    """High temperatures and narrow logits: thousands of tokens in the buckets around a border, or finer buckets."""
    R = 12
    rng = np.random.default_rng(V)
    for k, m in ((0, 0.0), (V // 3, 0.0), (V // 2, 0.001)):
        check(logits(R, V, sd, k + 11), T=rng.choice([1.0, 1.4, 1.79], R), k=k, p=rng.choice([0.9, 0.5, 0.97], R), m=m,
              u=rng.random(R).astype(np.float32))


@pytest.mark.parametrize("at", [100.0, -3e3, 2e4])
def test_logits_far_from_zero(at):
    """Bucket numbers are large where the logits are, or where the buckets are fine: their borders must not be missed."""
    R, V = 24, 26105
    for sd in (0.01, 0.3, 2.5):
        rng = np.random.default_rng(int(abs(at)))
        for x in (logits(R, V, sd, 3), logits(R, V, sd, 4).to(torch.bfloat16).float()):
            check(x + at, T=rng.choice([0.7, 1.0, 1.79, 4.0], R), k=rng.choice([0, 0, 900, V // 2], R),
                  p=rng.choice([1.0, 0.95, 0.5], R), m=rng.choice([0.0, 0.0, 0.01], R), u=rng.random(R).astype(np.float32))


def test_odd_values():
    R, V = 9, 7001
    x = logits(R, V, 2.0, 2)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, 77] = math.inf
    x[3, [5, 900]] = math.inf
    x[4, ::2] = math.nan
    x[5, 1:] = -math.inf
    x[6] = -1e9
    x[6, 33] = -1e9 + 1000
    x[7] = 3e38
    x[7, ::2] = -3e38
    x[8] = 0.0
    x[8, ::2] = -0.0
    for T, k, p, m in ((1.0, 0, 1.0, 0.0), (0.7, 40, 0.9, 0.05), (0.0, 0, 1.0, 0.0), (1e20, 0, 0.7, 0.0)):
        t = check(x, T=T, k=k, p=p, m=m, u=np.linspace(0.01, 0.99, R))
        assert (t[:2] == -1).all() and t[2] == 77 and t[3] in (5, 900) and t[5] == 0


def test_options_out_of_range():
    x = logits(8, 5000, 2.0, 3)
    x[:, 100] = 30.0
    check(x, T=[-1.0, math.nan, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0], k=[0, 0, -5, 10 ** 9, 0, 0, 0, 0],
          p=[1.0, 1.0, 2.0, 0.0, -1.0, math.nan, 1.0, 1.0], m=[0.0, 0.0, -1.0, 0.0, 0.0, 0.0, 2.0, math.nan],
          u=[0.5, 0.5, 0.999, 0.5, 0.5, 1.0, -1.0, math.nan])


def test_defaults_rows_of_their_own_and_strides():
    """Options left out; a row's token does not depend on its batch; rows at a stride."""
    x = logits(40, 32003, 2.5, 9)
    u = torch.rand(40, device="cuda")
    tokens = torch.empty(40, dtype=torch.int32, device="cuda")
    bq.sample_tokens(x, u, tokens)
    want = [choose(x[r].cpu().numpy(), 1.0, 0, 1.0, 0.0, float(u[r]))[0] for r in range(40)]
    assert tokens.tolist() == want
    alone = torch.empty(1, dtype=torch.int32, device="cuda")
    for r in (0, 17, 39):
        bq.sample_tokens(x[r:r + 1], u[r:r + 1], alone)
        assert int(alone) == want[r]
    bq.sample_tokens(x[::2], u[:20].contiguous(), tokens[:20])
    assert tokens[:20].tolist() == [choose(x[2 * r].cpu().numpy(), 1.0, 0, 1.0, 0.0, float(u[r]))[0] for r in range(20)]


def test_the_tokens_follow_the_distribution():
    """Uniforms on a grid: the share of every token is its probability to within a grid step."""
    x = logits(1, 50, 1.0, 4).expand(4096, -1)
    u = ((torch.arange(4096) + 0.5) / 4096).float().cuda()
    tokens = torch.empty(4096, dtype=torch.int32, device="cuda")
    bq.sample_tokens(x, u, tokens, top_k=torch.full((4096,), 20, dtype=torch.int32, device="cuda"))
    share = torch.bincount(tokens.long(), minlength=50).double() / 4096
    v, i = x[0].double().topk(20)
    want = torch.zeros(50, dtype=torch.float64, device="cuda").scatter_(0, i, torch.softmax(v, 0))
    assert ((share - want).abs() <= 1 / 4096 + 1e-9).all()


def test_captured_and_on_two_streams():
    xs = [logits(8, 32000, 2.5, s) for s in (1, 2)]
    us = [torch.rand(8, device="cuda") for _ in xs]
    out = [torch.empty(8, dtype=torch.int32, device="cuda") for _ in xs]
    side = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(4):
        for x, u, o, s in zip(xs, us, out, side):
            bq.sample_tokens(x, u, o, stream=s.cuda_stream)
    torch.cuda.synchronize()
    want = [[choose(x[r].cpu().numpy(), 1.0, 0, 1.0, 0.0, float(u[r]))[0] for r in range(8)] for x, u in zip(xs, us)]
    assert [o.tolist() for o in out] == want
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side[0]):
        bq.sample_tokens(xs[0], us[0], out[0], stream=torch.cuda.current_stream().cuda_stream)
    us[0].copy_(torch.rand(8))
    graph.replay()
    torch.cuda.synchronize()
    assert out[0].tolist() == [choose(xs[0][r].cpu().numpy(), 1.0, 0, 1.0, 0.0, float(us[0][r]))[0] for r in range(8)]


def test_a_batched_decode_step_draws_as_set_sampling_does():
    """The batch's logits and the uniforms of set_sampling's generator give its choice (the sampler's oracle from the same
    logits; a batch-1 prefill's own token); the tokens go back into the next step on the device."""
    cfg = synth.workload(0)
    V, n, seed = cfg["vocab"], 3, 11
    prompts = [np.arange(3 + i, dtype=np.int32) + i for i in range(n)]
    opt = dict(temperature=torch.full((n,), 0.9, device="cuda"), top_k=torch.full((n,), 30, dtype=torch.int32, device="cuda"),
               top_p=torch.full((n,), 0.9, device="cuda"))
    with bq.Model(cfg, synth.make_weights(cfg), max_seq=32, max_batch=n) as m:
        m.set_sampling(0.9, top_k=30, top_p=0.9, seed=seed)
        x, first = torch.empty(n, V, device="cuda"), []
        for i, prompt in enumerate(prompts):
            tok = np.zeros(1, np.int32)
            m.prefill(i, prompt, x[i], tok)
            first.append(int(tok[0]))
        m.set_sampling(0.0)
        tokens = torch.empty(n, dtype=torch.int32, device="cuda")
        for step in range(7):
            u = [oracle.sampling.uniform(seed, i, len(prompts[i]) - 1 + step) for i in range(n)]
            m.sync()
            bq.sample_tokens(x, torch.tensor(u, dtype=torch.float32, device="cuda"), tokens, **opt)
            torch.cuda.synchronize()
            want = [oracle.sampling.sample(x[i].cpu().numpy(), float(np.float32(0.9)), 30, float(np.float32(0.9)), u[i])[0]
                    for i in range(n)]
            assert tokens.tolist() == want, step
            if step == 0:
                assert want == first
            m.decode_step_batch(tokens, x)
