"""Edges of tree attention's and the token probabilities' domains (GPU): scores of any size, terms far below the largest,
the bits that fp32 queries carry."""
import math

import pytest
import torch

import bit_quantized_token_gb300 as bq
from test_gpu_tree import Problem, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    bq.build()
    torch.cuda.set_device(0)


def seen_rows(p, b, i):
    """K and V rows that node i of sequence b sees, [head, row, dim]."""
    L, js = int(p.lens[b]), [j for j in range(p.n) if int(p.mask[b, i]) >> j & 1]
    return [torch.cat([a[b, :, :L], t[b, :, js]], 1) for a, t in ((p.k, p.tk), (p.v, p.tv))]


@pytest.mark.parametrize("exponent,scale", [(20, None), (31, -0.3), (34, None), (60, 4.0), (100, None)])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("q", ["f32", "bf16"])
@pytest.mark.parametrize("kv", ["bf16", "q8"])
@pytest.mark.parametrize("n", [5, 24, 64])
def test_attention_scores_of_any_size(n, kv, q, hd, exponent, scale):
    """A query is 2^exponent in one dim, the keys there are whole numbers from -7 to 7: scores are exact, two of them
    apart by 2^exponent at least, so a row's output is the mean of the V rows of its largest score. Exact sums of V
    (bf16 products with 1, or code times scale 1 / 64) over at most N rows, cut off by up to 2^-23 a step; 1 / l and its
    product 2^-23; one rounding of the output."""
    p = Problem(B=3, n=n, Hkv=2, gq=2, hd=hd, cap=701, lens=(700, 129, 5), q=q, kv=kv, seed=exponent)
    g = gen(n)
    dims = torch.randint(0, hd, p.q.shape[:3], device="cuda", generator=g)
    sign = torch.randint(0, 2, p.q.shape[:3], device="cuda", generator=g) * 2 - 1
    p.q.zero_().scatter_(3, dims[..., None], (sign * 2.0 ** exponent)[..., None].to(p.q.dtype))
    for t in (p.k, p.tk):
        t.copy_(torch.randint(-7, 8, t.shape, device="cuda", generator=g))
    if kv == "q8":
        for t in (p.ks, p.tks):
            t.fill_(1.0)
        for t in (p.vs, p.tvs):
            t.fill_(1 / 64)
    p.scale = scale
    p.call()
    for b in range(3):
        for i in range(0, n, max(1, n // 12)):
            K, V = seen_rows(p, b, i)
            for h in range(4):
                s = K[h // 2].double() @ p.q[b, i, h].double() * (1.0 if scale is None else scale)
                v = V[h // 2][s == s.max()].double() * (1.0 if kv == "bf16" else 1 / 64)
                o, A = v.mean(0), v.abs().mean(0)
                tol = o.abs() * (2.0 ** -8 if q == "bf16" else 2.0 ** -24) + A * (v.shape[0] + 4) * 2.0 ** -23
                err = (p.out[b, i, h].double() - o).abs()
                assert (err <= tol).all(), (b, i, h, float((err / tol).max()))


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("q", ["f32", "bf16"])
@pytest.mark.parametrize("kv", ["bf16", "q8"])
@pytest.mark.parametrize("n", [3, 64])
def test_attention_large_random_scores(n, kv, q, hd):
    """Scores around 2^40, rounded as fp32 sums are: an output is a mean of visible V rows, whichever the weights."""
    p = Problem(B=2, n=n, Hkv=2, gq=2, hd=hd, cap=401, lens=(400, 77), q=q, kv=kv, seed=3)
    p.q *= 2.0 ** 40
    p.call()
    for b in range(2):
        for i in range(n):
            V = seen_rows(p, b, i)[1].double()
            if kv == "q8":
                js = [j for j in range(n) if int(p.mask[b, i]) >> j & 1]
                sc = torch.cat([p.vs[b, :, :int(p.lens[b])], p.tvs[b][:, js]], 1).double()
                V = V * sc.repeat_interleave(32, -1)
            lo, hi = V.amin(1).repeat_interleave(2, 0), V.amax(1).repeat_interleave(2, 0)
            room = 2.0 ** -6 * V.abs().amax()
            o = p.out[b, i].double()
            assert ((o >= lo - room) & (o <= hi + room)).all(), (b, i)


@pytest.mark.parametrize("V", [32768, 151936, 1000])
@pytest.mark.parametrize("T", [1.0, 0.02, 30.0])
def test_token_probs_keep_terms_far_below_the_largest(T, V):
    """Eighths of a row (what a CTA takes) at levels of their own, in powers of two of the probability: the second half
    of one lies up to 2^59 above its first, all of it up to 2^200 below the largest. Terms above 2^-126 keep fp32's
    precision (tolerance as for all rows: the argument's roundings, exp2f, the sum, the normalising)."""
    half = V // 16
    levels = torch.full((6, 16), -300.0, dtype=torch.float64)
    levels[:, 0:2] = 0.0                       # the largest eighth
    levels[0, 2:4] = torch.tensor([-140.0, -81.0])
    levels[1, 2:4] = torch.tensor([-170.0, -111.0])
    levels[2, 2:4] = torch.tensor([-100.0, -41.0])
    levels[3, 0:2] = torch.tensor([-59.0, 0.0])  # the largest, as a sum of terms around 2^59
    levels[3, 2:4] = torch.tensor([-160.0, -101.0])
    levels[4, 0:2] = torch.tensor([-59.0, 0.0])
    levels[4, 2:4] = torch.tensor([-110.0, -52.0])
    levels[4, 4:6] = torch.tensor([-30.0, -80.0])
    levels[5, 2:] = -20.0
    x = levels.repeat_interleave(half, 1)
    x = torch.cat([x, torch.full((6, V - x.shape[1]), -300.0, dtype=torch.float64)], 1)
    x = ((x + 0.2 * torch.rand(6, V, dtype=torch.float64, generator=torch.Generator().manual_seed(V))) * math.log(2) * T).float()
    out = torch.empty(6, V, device="cuda")
    bq.token_probs(x.cuda(), out, T, 0, 1.0)
    for r in range(6):
        got, ref = out[r].double().cpu(), torch.softmax(x[r].double() / T, 0)
        tol = ref * ((3 * 300 * math.log(2) * 2.0 ** -24 + 2.0 ** -22) * 2 + 210 * 2.0 ** -24) + 2.0 ** -140
        err = (got - ref).abs()
        assert (err <= tol).all(), (r, float((err / tol).max()))


def bf16_parts(x, n):
    """x in n bf16 parts: their sum."""
    total = torch.zeros_like(x)
    for _ in range(n):
        total = total + (x - total).bfloat16().float()
    return total


@pytest.mark.parametrize("kv", ["bf16", "q8"])
@pytest.mark.parametrize("what", ["queries", "probabilities"])
def test_fp32_queries_and_probabilities_carry_24_bits(what, kv):
    """Two keys, 64 in a dim of their own; values 1 in a dim of their own, so that the outputs are the probabilities
    p = r / (1 + r) and 1 / (1 + r), r = 2^y, y = c (s1 - s0). Scores are exact (64 times a query's value), as is their
    difference (both lie in one binade). y: the roundings of c and of the product, so r is off by |y| ln 2 2^-23, exp2
    2^-22 and three parts 2^-23; then the sum, its reciprocal and two products 4 2^-24. Queries far enough apart show
    their own third part (8 units of y to a unit of q), those close together that of the probabilities: with two parts
    of either, which the same formulas give on the host, a good part of the outputs is off by more."""
    B, n, H, hd = 4, 16, 8, 64
    a = 1 + torch.rand(2, B, n, H, generator=torch.Generator().manual_seed(3))
    if what == "probabilities":
        a[1] = a[0] + (a[1] - a[0]) / 16  # r from 0.5 to 2
    q = torch.zeros(B, n, H, hd)
    q[..., 0], q[..., 1] = a[0], a[1]
    rows = torch.zeros(2, B, 1, 2, hd)
    rows[0, :, :, 0, 0] = rows[0, :, :, 1, 1] = 64
    rows[1, :, :, 0, 5] = rows[1, :, :, 1, 40] = 1
    scales = None if kv == "bf16" else torch.ones(B, 1, 2, hd // 32, dtype=torch.float16, device="cuda")
    k, v = (x.cuda().to(torch.bfloat16 if kv == "bf16" else torch.int8) for x in rows)
    out = torch.empty(B, n, H, hd, device="cuda")
    lens = torch.full((B,), 2, dtype=torch.int32, device="cuda")
    bq.tree_attention(q.cuda(), bq.KVView(k, v, scales, scales), None, lens, None, out, scale=1 / 8)
    bq.tree_status()

    def probabilities(a, parts):
        y = 8 * (a[1].double() - a[0].double()) / math.log(2)
        w = torch.exp2(torch.stack([torch.zeros_like(y), y]))
        if parts:
            w = bf16_parts(w.float(), parts).double()
        return w / w.sum(0), y

    ref, y = probabilities(a, 0)
    tol = ref[0] * ref[1] * (y.abs() * math.log(2) * 2.0 ** -23 + 2.0 ** -22 + 2.0 ** -23) + 4 * 2.0 ** -24 * ref
    got = torch.stack([out[..., 5], out[..., 40]]).double().cpu()
    assert ((got - ref).abs() <= tol).all(), float(((got - ref).abs() / tol).max())
    less = probabilities(bf16_parts(a, 2), 0)[0] if what == "queries" else probabilities(a, 2)[0]
    assert ((less - ref).abs() > tol).double().mean() > 0.25
