"""The tree-decoding operators against plain implementations in 64 bits (GPU).

Tolerances come from the operations' roundings, not from runs. Attention, per
output element, with A = sum_j p_j |v_j| (the largest any error in p can weigh):
  score: a product chain of hd fp32 adds, each off by at most 2^-23 of the sum of
    magnitudes (the tensor cores may truncate), the scaling and the subtraction
    of the maximum 2^-24 each: ds = (hd + 8) 2^-23 max_j sum_d |q k| scale;
  p: exp2f 2^-22, fp32 parts 2^-24 (fp32 queries) or two bf16 parts (2^-8)^2; bf16 queries of more than 64 rows
    (nodes x heads of a kv head) over bf16 rows: one part, 2^-8 of each p in o and again in l;
  sums over N keys: N 2^-23 for each of o and l (rescaling included), joined over
    splits: 64 more.
  output: one rounding, 2^-8 |o| (bf16) or 2^-24 |o| (fp32).
  underflow: a reference is at most the row's maximum, and a p below 2^-126 of its reference is 0: N 2^-126 max |v|.
The relative errors of o and l add: tol = round |o| + A (2 ds + 2^-21 + part + 2 (N + 64) 2^-23).
int8 rows: the products of a group's scale add 2 2^-24 to each score term (inside the 8 above), and a value, code
  times scale, is rounded to two bf16 parts for bf16 queries, (2^-8)^2 of it (three for fp32 hold it exactly).
"""
import math

import numpy as np
import pytest
import torch

import bit_quantized_token_gb300 as bq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    bq.build()
    torch.cuda.set_device(0)


def gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def make_rows(B, H, R, hd, kv, g):
    x = torch.randn(B, H, R, hd, device="cuda", generator=g)
    if kv == "bf16":
        return x.to(torch.bfloat16), None
    x = x.view(B, H, R, hd // 32, 32)
    s = (x.abs().amax(-1, keepdim=True) / 127).to(torch.float16)
    return (x / s.float()).round().clamp(-127, 127).to(torch.int8).view(B, H, R, hd), s.squeeze(-1)


def values(rows, scales):
    if scales is None:
        return rows.double()
    sh = rows.shape
    return (rows.view(*sh[:-1], sh[-1] // 32, 32).double() * scales.double()[..., None]).view(sh)


def random_parents(n, rng, spread=5):
    return [-1] + [int(rng.integers(max(0, i - spread), i)) for i in range(1, n)]


class Problem:
    def __init__(self, B=2, n=5, Hkv=2, gq=2, hd=64, cap=64, lens=(40, 17), q="f32", kv="bf16", seed=0):
        g, rng = gen(seed), np.random.default_rng(seed)
        self.kv, self.gq, self.hd, self.n, self.B = kv, gq, hd, n, B
        self.k, self.ks = make_rows(B, Hkv, cap, hd, kv, g)
        self.v, self.vs = make_rows(B, Hkv, cap, hd, kv, g)
        self.tk, self.tks = make_rows(B, Hkv, n, hd, kv, g)
        self.tv, self.tvs = make_rows(B, Hkv, n, hd, kv, g)
        self.q = torch.randn(B, n, Hkv * gq, hd, device="cuda", generator=g).to(
            torch.float32 if q == "f32" else torch.bfloat16)
        self.lens = torch.tensor([lens[b % len(lens)] for b in range(B)], dtype=torch.int32, device="cuda")
        self.parents = [random_parents(n, rng) for _ in range(B)]
        self.mask = torch.tensor([bq.tree_masks(p) for p in self.parents], device="cuda")
        self.out = torch.full_like(self.q, 7.0)
        self.counts = None
        self.scale = None
        self.with_tree = True

    def cache(self):
        return bq.KVView(self.k, self.v, self.ks, self.vs)

    def tree(self):
        return bq.KVView(self.tk, self.tv, self.tks, self.tvs) if self.with_tree else None

    def call(self, **kw):
        bq.tree_attention(self.q, self.cache(), self.tree(), self.lens, self.mask, self.out, counts=self.counts,
                          scale=self.scale, **kw)
        bq.tree_status()
        return self.out

    def check(self, out=None):
        out = self.out if out is None else out
        scale = self.hd ** -0.5 if self.scale is None else self.scale
        worst = 0.0
        k, v, tk, tv = (values(a, b) for a, b in
                        ((self.k, self.ks), (self.v, self.vs), (self.tk, self.tks), (self.tv, self.tvs)))
        for b in range(self.B):
            L = min(max(int(self.lens[b]), 0), self.k.shape[2])
            cnt = self.n if self.counts is None else int(self.counts[b])
            if cnt < self.n:
                assert (out[b, cnt:] == 7.0).all(), "rows past the count were written"
            for i in range(cnt):
                word = int(self.mask[b, i]) & ((1 << cnt) - 1) if self.with_tree else 0
                js = [j for j in range(cnt) if word >> j & 1]
                for h in range(self.q.shape[2]):
                    g = h // self.gq
                    K, V = torch.cat([k[b, g, :L], tk[b, g, js]]), torch.cat([v[b, g, :L], tv[b, g, js]])
                    got = out[b, i, h].double()
                    if K.shape[0] == 0:
                        assert (got == 0).all(), "a row that sees nothing must be 0"
                        continue
                    x = self.q[b, i, h].double()
                    s = K @ x * scale
                    w = torch.softmax(s, 0)
                    o, A = w @ V, w @ V.abs()
                    ds = (self.hd + 8) * 2.0 ** -23 * float((K.abs() @ x.abs()).max()) * abs(scale)
                    bf = self.q.dtype == torch.bfloat16
                    rnd, part = (2.0 ** -8, 2.0 ** -16) if bf else (2.0 ** -24, 2.0 ** -23)
                    if bf and self.kv == "bf16" and self.n * self.gq > 64:
                        part = 2 * 2.0 ** -8
                    if bf and self.kv == "q8":
                        part += 2.0 ** -16
                    tol = rnd * o.abs() + A * (2 * ds + 2.0 ** -21 + part + 2 * (K.shape[0] + 64) * 2.0 ** -23)
                    tol = tol + K.shape[0] * 2.0 ** -126 * V.abs().max()
                    err = (got - o).abs()
                    assert (err <= tol).all(), (b, i, h, float((err / tol).max()))
                    worst = max(worst, float((err / tol).max()))
        return worst


SHAPES = [  # n, Hkv, gq, hd, lens
    (1, 2, 1, 64, (1,)), (1, 1, 8, 64, (0, 1)), (1, 8, 2, 128, (63, 64, 65)), (3, 2, 5, 64, (127, 128, 129, 0)),
    (7, 1, 2, 128, (33,)), (8, 2, 2, 128, (200, 5)), (9, 3, 7, 64, (300,)), (16, 1, 1, 128, (1000,)),
    (17, 2, 2, 64, (511,)), (33, 1, 3, 128, (130, 64)), (64, 1, 8, 64, (700, 0)), (64, 2, 2, 128, (257,)),
    (63, 1, 1, 64, (1,)), (5, 1, 16, 128, (90,)),
]


@pytest.mark.parametrize("kv", ["bf16", "q8"])
@pytest.mark.parametrize("q", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_attention(shape, q, kv):
    n, Hkv, gq, hd, lens = shape
    p = Problem(B=len(lens), n=n, Hkv=Hkv, gq=gq, hd=hd, cap=max(lens) + 3, lens=lens, q=q, kv=kv, seed=n)
    p.call()
    p.check()


@pytest.mark.parametrize("q", ["f32", "bf16"])
def test_attention_long_cache_is_split(q):
    p = Problem(B=1, n=2, Hkv=1, gq=2, hd=128, cap=5000, lens=(4999,), q=q)
    p.call()
    p.check()


@pytest.mark.parametrize("kv", ["bf16", "q8"])
def test_attention_counts_and_arbitrary_masks(kv):
    p = Problem(B=4, n=20, Hkv=2, gq=3, lens=(0, 9, 64, 0), kv=kv, q="bf16")
    p.counts = torch.tensor([20, 0, 7, 1], dtype=torch.int32, device="cuda")
    g = np.random.default_rng(1)
    p.mask = torch.tensor(g.integers(-(1 << 63), 1 << 62, (4, 20)), device="cuda")
    p.mask[0, 3] = 0  # with an empty cache: a row that sees nothing
    p.mask[3, 0] = 0
    p.call()
    p.check()


@pytest.mark.parametrize("n", [3, 64])
@pytest.mark.parametrize("q", ["f32", "bf16"])
def test_attention_without_tree(q, n):
    p = Problem(B=3, n=n, Hkv=2, gq=2, hd=128, cap=70, lens=(0, 70, 31), q=q)
    p.with_tree = False
    p.mask = None
    p.call()
    p.check()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("q", ["f32", "bf16"])
@pytest.mark.parametrize("kv", ["bf16", "q8"])
@pytest.mark.parametrize("n", [1, 20])
def test_attention_many_tiles_to_a_cta(n, kv, q, hd):
    """More (sequence, kv head) pairs than SMs, so that each is one CTA's, over ragged caches of up to 17 tiles."""
    lens = (2100, 1300, 129, 1919, 640, 1, 1664, 0)
    p = Problem(B=40, n=n, Hkv=4, gq=1, hd=hd, cap=2101, lens=lens, q=q, kv=kv)
    for b in range(40):
        if kv == "bf16":
            p.v[b, :, int(p.lens[b]):] = float("nan")
        else:
            p.vs[b, :, int(p.lens[b]):] = float("nan")
    p.call()
    keep, p.B = p.out, 8
    p.check()
    p.out, p.lens = keep[32:], p.lens[32:]
    for name in ("q", "k", "v", "ks", "vs", "tk", "tv", "tks", "tvs", "mask"):
        t = getattr(p, name)
        setattr(p, name, None if t is None else t[32:])
    p.check()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("kv", ["bf16", "q8"])
@pytest.mark.parametrize("n", [1, 20, 64])
def test_attention_repeats_bit_for_bit(n, kv, hd):
    """The order of every sum is fixed, so calls in a row agree; long rows, where tiles take turns in a ring."""
    p = Problem(B=40, n=n, Hkv=4, gq=2, hd=hd, cap=2101, lens=(2100, 1919, 1300, 1664), q="bf16", kv=kv)
    first = p.call().clone()
    for _ in range(20):
        p.out.fill_(float("nan"))
        assert torch.equal(p.call(), first)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("q", ["f32", "bf16"])
@pytest.mark.parametrize("kv", ["bf16", "q8"])
@pytest.mark.parametrize("n", [5, 24, 64])
def test_attention_renews_its_references_in_any_tile(n, kv, q, hd):
    """Every third node's scores spread over hundreds, so that tiles along a CTA's way renew the references of the
    block's other rows too, whose sums so far are scaled."""
    p = Problem(B=40, n=n, Hkv=4, gq=2, hd=hd, cap=1301, lens=(1300, 700, 1151, 260), q=q, kv=kv)
    p.q[:, ::3] *= 60
    p.call()
    p.B = 4
    p.check()


@pytest.mark.parametrize("kv", ["bf16", "q8"])
def test_attention_fp32_sums_do_not_drift(kv):
    """fp32 queries over rows of one CTA each: the outputs are not low on the whole. An MMA step cuts off up to
    2^-23 of its sum, half of that on average; of the steps between two roundings at most 16 add to sums of full
    size, so the mean is off by less than 16 2^-24 (sums of 250 steps would be off by several times that)."""
    L = 4000
    p = Problem(B=20, n=2, Hkv=8, gq=2, hd=64, cap=L + 1, lens=(L,) * 20, q="f32", kv=kv)
    p.call()
    k, v, tk, tv = (values(a, b) for a, b in ((p.k, p.ks), (p.v, p.vs), (p.tk, p.tks), (p.tv, p.tvs)))
    off = size = 0.0
    for b in (0, 19):
        for i in range(2):
            seen = [j for j in range(2) if int(p.mask[b, i]) >> j & 1]
            for h in range(0, 16, 3):
                K = torch.cat([k[b, h // 2, :L], tk[b, h // 2][seen]]).double()
                V = torch.cat([v[b, h // 2, :L], tv[b, h // 2][seen]]).double()
                o = torch.softmax(K @ p.q[b, i, h].double() * 64 ** -0.5, 0) @ V
                off += float(((p.out[b, i, h].double() - o) * o).sum())
                size += float((o * o).sum())
    assert abs(off / size) < 16 * 2.0 ** -24, off / size


def test_attention_scores_far_apart_and_scale():
    for scale in (0.0, -0.3, 4.0):
        p = Problem(B=1, n=4, cap=200, lens=(200,), q="f32")
        p.q *= 3
        p.scale = scale
        p.call()
        p.check()


@pytest.mark.parametrize("n", [6, 64])
@pytest.mark.parametrize("q", ["f32", "bf16"])
@pytest.mark.parametrize("kv", ["bf16", "q8"])
def test_attention_unseen_rows_do_not_matter(kv, q, n):
    """NaN and infinities behind the lengths, in tree rows nobody sees, and in rows only some nodes see."""
    p = Problem(B=2, n=n, Hkv=2, gq=4, hd=64, cap=90, lens=(50, 0), q=q, kv=kv)
    p.mask &= ~(1 << 2)  # nobody sees node 2
    p.mask[:, 2] = 0b11
    p.mask &= ~(1 << 4)
    p.mask[:, 4] = (1 << 4) | 1  # only node 4 sees node 4
    bad = [float("nan"), float("inf"), float("-inf")]
    for b in range(2):
        L = int(p.lens[b])
        for j, x in enumerate(bad):
            if kv == "bf16":
                p.k[b, :, L + j] = x
                p.v[b, :, L + j] = x
                p.tk[b, :, 2, j::3] = x
                p.tv[b, :, 2, j::3] = x
                p.tv[b, :, 4, 5 + j] = x
            else:
                for s in (p.ks, p.vs):
                    s[b, :, L + j] = x
                for s in (p.tks, p.tvs):
                    s[b, :, 2] = bad[j]
                p.tvs[b, :, 4, 1] = float("nan")
    p.call()
    bad4 = p.out[:, 4].clone()
    if kv == "bf16":
        assert bad4[..., 5].isnan().all() and (bad4[..., 6] == math.inf).all() and (bad4[..., 7] == -math.inf).all()
        rest = torch.cat([bad4[..., :5], bad4[..., 8:]], -1)
        assert rest.isfinite().all()
    else:
        assert bad4[..., 32:].isnan().all() and bad4[..., :32].isfinite().all()
    for i in range(n):  # node 4 is checked above; the others must not notice
        if i == 4:
            continue
        assert p.out[:, i].isfinite().all(), i
    p.mask[:, 4] = 0b1
    fixed = p.out.clone()
    p.call()
    fixed[:, 4] = p.out[:, 4]
    p.check(fixed)


def test_attention_strided_tensors():
    B, n, Hkv, gq, hd = 2, 6, 2, 3, 64
    p = Problem(B=B, n=n, Hkv=Hkv, gq=gq, hd=hd, cap=80, lens=(61, 80), q="bf16")
    big = torch.full((80, B, 3, Hkv + 1, hd + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    for i, name in ((0, "k"), (1, "v")):
        w = big.clone()[:, :, i, :Hkv, :hd].permute(1, 2, 0, 3)
        w.copy_(getattr(p, name))
        setattr(p, name, w)
    qb = torch.zeros(n, B, Hkv * gq + 2, hd + 8, dtype=torch.bfloat16, device="cuda")
    q = qb[:, :, 1:-1, :hd].permute(1, 0, 2, 3)
    q.copy_(p.q)
    p.q = q
    ob = torch.full((Hkv * gq, n, B, hd + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    p.out = ob[..., :hd].permute(2, 1, 0, 3)
    p.call()
    p.check()
    assert (ob[..., hd:] == 7.0).all()


@pytest.mark.parametrize("kv", ["bf16", "q8"])
def test_attention_shared_rows(kv):
    """One prefix for every sequence, one kv head for all: strides of 0."""
    p = Problem(B=3, n=4, Hkv=2, gq=2, cap=150, lens=(150, 3, 77), kv=kv)
    for name in ("k", "v", "ks", "vs"):
        t = getattr(p, name)
        if t is not None:
            setattr(p, name, t[:1, :1].expand(3, 2, *t.shape[2:]))
    for name in ("tk", "tv", "tks", "tvs"):
        t = getattr(p, name)
        if t is not None:
            setattr(p, name, t[:, :1].expand(3, 2, *t.shape[2:]))
    p.call()
    p.check()


def test_attention_offsets_beyond_32_bits():
    """The second sequence lies more than 2^32 elements behind the first."""
    stride = (1 << 32) + 512
    n, hd, L = 3, 64, 40
    big = [torch.empty(stride + 2 * (L + 8) * hd, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    p = Problem(B=2, n=n, Hkv=2, gq=1, hd=hd, cap=L + 8, lens=(L, L - 7))
    for i, name in ((0, "k"), (1, "v")):
        w = big[i].as_strided((2, 2, L + 8, hd), (stride, (L + 8) * hd, hd, 1))
        w.copy_(getattr(p, name))
        setattr(p, name, w)
    p.call()
    p.check()


def test_attention_lengths_out_of_range_are_clamped():
    p = Problem(B=2, n=2, cap=30, lens=(1000, -5))
    p.call()
    p.check()


def test_streams_and_graphs():
    """A captured call follows its inputs; two graphs and an eager call may run at once."""
    probs = [Problem(B=2, n=4, cap=600, lens=(500, 77), seed=s, q="bf16") for s in range(3)]
    views = [(p.cache(), p.tree()) for p in probs]

    def run(i, st):
        p = probs[i]
        bq.tree_attention(p.q, *views[i], p.lens, p.mask, p.out, stream=st.cuda_stream)

    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        gph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gph, stream=streams[i]):
            run(i, streams[i])
        graphs.append(gph)
    for rep in range(3):
        for p in probs:
            p.lens -= 31
            p.out.fill_(7.0)
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        run(2, streams[2])
        torch.cuda.synchronize()
        for p in probs:
            p.check()


def test_host_memory_is_refused():
    p = Problem()
    p.lens = p.lens.cpu()
    with pytest.raises(bq.LlmError, match="lens is not memory of the current device"):
        p.call()
    q = torch.empty(3, 5)
    with pytest.raises(bq.LlmError, match="not memory"):
        bq.token_probs(q, torch.empty(3, 5, device="cuda"))


# ---- token probabilities -------------------------------------------------------
def probs_reference(row, T, k, p):
    """The sampler's distribution of one row in 64 bits."""
    x = np.where(np.isnan(row), -np.inf, np.minimum(row.astype(np.float64), np.finfo(np.float32).max))
    out = np.zeros(len(x))
    if not np.isfinite(x.max()):
        return out
    w = np.exp((x - x.max()) / T)
    if k == 0:
        return w / w.sum()
    order = np.lexsort((np.arange(len(x)), -x))[:k]
    w = w[order] / w[order].sum()
    keep = np.cumsum(w) - w < p
    keep[0] = True
    out[order[keep]] = w[keep] / w[keep].sum()
    return out


def check_probs(got, ref, T, spread):
    """fp32: the argument (l - m) c has three roundings of 2^-24 relative, so e is off by 3 |arg| 2^-24 and exp2f's
    2^-22; the sum of V terms by at most 2^-24 a level (block sums: under 200 adds in a row) on top of the terms' own;
    normalising and storing 3 2^-24."""
    arg = spread / T
    tol = ref * ((3 * arg * 2.0 ** -24 + 2.0 ** -22) * 2 + 210 * 2.0 ** -24) + 2.0 ** -140
    err = np.abs(got - ref)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("R,V", [(1, 1), (3, 2), (2, 7), (1, 63), (5, 65), (2, 2049), (3, 4099), (1, 32000),
                                 (2, 32003), (40, 1000), (1, 151936), (2, 300001)])
@pytest.mark.parametrize("opt", [(1.0, 0, 1.0), (0.7, 0, 1.0), (0.8, 40, 0.95), (1.3, 64, 1.0), (0.5, 1, 0.5),
                                 (1.0, 7, 1e-6)], ids=str)
def test_token_probs(R, V, opt):
    T, k, p = opt
    x = 3 * torch.randn(R, V, device="cuda", generator=gen(V))
    out = torch.full((R, V + 3), 7.0, device="cuda")[:, :V]
    bq.token_probs(x, out, T, k, p)
    xs, got = x.cpu().numpy(), out.cpu().numpy()
    for r in range(R):
        spread = float(xs[r].max() - xs[r].min())
        check_probs(got[r], probs_reference(xs[r], T, k, p), T, spread)
    inplace = x.clone()
    bq.token_probs(inplace, inplace, T, k, p)
    assert torch.equal(inplace, out)


@pytest.mark.parametrize("V", [5, 700, 33333])
@pytest.mark.parametrize("k", [1, 3, 64])
def test_token_probs_ties_go_to_the_lower_id(V, k):
    x = torch.randint(-2, 3, (4, V), generator=gen(1), device="cuda").float()
    x[1] = 0.0
    x[2] = -0.0
    x[2, ::2] = 0.0
    out = torch.empty_like(x)
    bq.token_probs(x, out, 1.0, k, 1.0)
    got = out.cpu().numpy()
    for r in range(4):
        ref = probs_reference(x[r].cpu().numpy(), 1.0, k, 1.0)
        assert ((got[r] > 0) == (ref > 0)).all()
        check_probs(got[r], ref, 1.0, 4)


def test_token_probs_crowded_group():
    """All large logits in one thread's elements: the candidate list at its longest."""
    x = torch.randn(2, 40000, device="cuda", generator=gen(2))
    x[:, 8::512] += 30
    x[1, :2048] += 40
    out = torch.empty_like(x)
    bq.token_probs(x, out, 1.0, 64, 0.99)
    for r in range(2):
        row = x[r].cpu().numpy()
        check_probs(out[r].cpu().numpy(), probs_reference(row, 1.0, 64, 0.99), 1.0, float(row.max() - row.min()))


@pytest.mark.parametrize("k", [0, 5])
def test_token_probs_special_values(k):
    nan, inf = float("nan"), float("inf")
    x = torch.randn(6, 5000, device="cuda", generator=gen(3))
    x[0] = -inf
    x[1] = nan
    x[2, 7] = nan
    x[2, 9:4000] = -inf
    x[3, [3, 4444]] = inf
    x[4] = torch.finfo(torch.float32).min
    x[5] = -inf
    x[5, [0, 4999]] = 1.0
    out = torch.full_like(x, 7.0)
    bq.token_probs(x, out, 0.9, k, 1.0)
    got = out.cpu().numpy()
    for r in range(6):
        ref = probs_reference(x[r].cpu().numpy(), 0.9, k, 1.0)
        if r == 4 and k == 0:
            assert np.allclose(got[r], 1 / 5000, rtol=210 * 2.0 ** -24, atol=0)
        else:
            check_probs(got[r], ref, 0.9, 10.0)


@pytest.mark.parametrize("V", [9, 700, 33333, 151936])
@pytest.mark.parametrize("T", [1.0, 0.05, 20.0])
def test_token_probs_large_logits_come_late(V, T):
    """Rows whose largest logits are far from the ones before them, in either direction."""
    h = V // 2
    x = 2 * T * torch.randn(7, V, device="cuda", generator=gen(7))
    x[0, -1] += 1000 * T
    x[1, h:] += 300 * T
    x[2, :h] = -math.inf
    x[2, h:] -= 40 * T
    x[3, :h] = -math.inf
    x[3, h:] = 6 * (x[3, h:] - 15 * T)
    x[4, :-2] = torch.finfo(torch.float32).min
    x[5, :h] = -1e30
    x[5, V - 1] = 3e38
    x[6, :h] += 500 * T
    out = torch.empty_like(x)
    bq.token_probs(x, out, T, 0, 1.0)
    xs, got = x.cpu().numpy(), out.cpu().numpy()
    for r in range(7):  # terms further than 110 down are below the tolerance's floor
        check_probs(got[r], probs_reference(xs[r], T, 0, 1.0), T, 110.0 * T)


# ---- verification ------------------------------------------------------------------
def verify_reference(tokens, parents, u, p, q, cnt):
    """One sequence in 64 bits: (path, next)."""
    p = np.maximum(np.nan_to_num(p.astype(np.float64), nan=0.0), 0.0)
    q = None if q is None else np.maximum(np.nan_to_num(q.astype(np.float64), nan=0.0), 0.0)
    V = p.shape[1]
    if cnt == 0:
        return [], -1
    cur, path, r, m = 0, [0], p[0], 1.0
    for i in range(1, cnt):
        if parents[i] != cur:
            continue
        x = int(tokens[i])
        ok = 0 <= x < V
        qx = (1.0 if q is None else q[cur, x]) if ok else 0.0
        if ok and float(u[i]) * qx * m < r[x]:
            cur, r, m = i, p[i], 1.0
            path.append(i)
        elif q is None:
            if ok:
                m -= r[x]
                r = r.copy()
                r[x] = 0.0
        else:
            rest = np.maximum(r / m - q[cur], 0.0)
            if rest.sum() > 0:
                r, m = rest, rest.sum()
    c = np.cumsum(r)
    over = np.nonzero((c > float(u[0]) * c[-1]) & (r > 0))[0]
    return path, int(over[0]) if len(over) else V - 1


def verify_problem(B, n, V, soft, seed, chain=False, sharp=3.0, near=0.5):
    g, rng = gen(seed), np.random.default_rng(seed)
    x = sharp * torch.randn(B, n, V, device="cuda", generator=g)
    p = torch.softmax(x, -1)
    q = torch.softmax(x + near * torch.randn(B, n, V, device="cuda", generator=g), -1)
    parents = np.array([list(range(-1, n - 1)) if chain else random_parents(n, rng, 4) for _ in range(B)])
    tok = np.zeros((B, n), np.int64)
    qc = q.cpu().numpy().astype(np.float64)
    for b in range(B):
        for i in range(1, n):
            w = qc[b, parents[b, i]]
            tok[b, i] = rng.choice(V, p=w / w.sum()) if soft or rng.random() < 0.3 else int(w.argmax())
    d = dict(tokens=torch.tensor(tok, dtype=torch.int32, device="cuda"),
             parents=torch.tensor(parents, dtype=torch.int32, device="cuda"),
             uniforms=torch.rand(B, n, device="cuda", generator=g), probs=p,
             path=torch.full((B, n), 9, dtype=torch.int32, device="cuda"),
             n_path=torch.full((B,), 9, dtype=torch.int32, device="cuda"),
             next_token=torch.full((B,), 9, dtype=torch.int32, device="cuda"))
    if soft:
        d["draft_probs"] = q
    return d


def check_verify(d):
    bq.verify_tree(**d)
    B, n = d["tokens"].shape
    q = d.get("draft_probs")
    cnt = d.get("counts")
    kept = 0
    for b in range(B):
        c = n if cnt is None else min(max(int(cnt[b]), 0), n)
        path, nxt = verify_reference(d["tokens"][b].cpu().numpy(), d["parents"][b].cpu().numpy(),
                                     d["uniforms"][b].cpu().numpy(), d["probs"][b].cpu().numpy(),
                                     None if q is None else q[b].cpu().numpy(), c)
        got = d["path"][b].tolist()
        assert got == path + [-1] * (n - len(path)), (b, got, path)
        assert int(d["n_path"][b]) == len(path)
        assert int(d["next_token"][b]) == nxt, b
        kept += len(path)
    return kept


@pytest.mark.parametrize("soft", [False, True])
@pytest.mark.parametrize("B,n,V", [(1, 1, 1), (2, 1, 50), (3, 2, 2), (4, 5, 33), (2, 64, 300), (5, 16, 1031),
                                   (1, 5, 32000), (3, 9, 4097), (2, 6, 151936), (1, 3, 70001)])
def test_verify(B, n, V, soft):
    check_verify(verify_problem(B, n, V, soft, seed=V + n))


@pytest.mark.parametrize("soft", [False, True])
def test_verify_many_small_trees(soft):
    d = verify_problem(300, 12, 11, soft, seed=5, sharp=1.0, near=1.0)
    assert check_verify(d) > 300  # some walks go beyond the root
    d = verify_problem(100, 6, 40, soft, seed=6, chain=True, near=0.2)
    assert check_verify(d) > 100


def test_verify_counts_parents_and_tokens_out_of_range():
    for soft in (False, True):
        d = verify_problem(6, 8, 90, soft, seed=7, sharp=1.0)
        d["counts"] = torch.tensor([8, 0, 3, 1, 100, -4], dtype=torch.int32, device="cuda")
        d["parents"][0, 3] = 5   # not a lower node
        d["parents"][0, 4] = -1
        d["parents"][4, 2] = 2
        d["tokens"][4, 1] = 90
        d["tokens"][2, 1] = -3
        d["parents"][4, 1] = 0
        check_verify(d)


def test_verify_edge_distributions():
    """Rows without mass, NaN and negative entries, a draft equal to the target, siblings with the same token."""
    V, n = 17, 4
    for soft in (False, True):
        d = verify_problem(8, n, V, soft, seed=11)
        d["parents"][:] = torch.tensor([-1, 0, 0, 0], dtype=torch.int32)
        d["uniforms"].clamp_(min=0.01)
        p = d["probs"]
        p[0] = 0.0
        p[1, 0, 3] = float("nan")
        p[2, 0, 4] = -0.5
        d["tokens"][3, 1:] = 6
        p[4, 0] = 0.0
        p[4, 0, 16] = 1.0   # everything on the last token
        d["uniforms"][5, 0] = 0.0
        d["uniforms"][6, 0] = 1.0 - 2.0 ** -24
        if soft:
            d["draft_probs"][7] = p[7]
            d["draft_probs"][4, 0] = p[4, 0]
            d["tokens"][4, 1:] = 2   # p(x) = q(x) = 0: rejected, and nothing is left of p - q
        check_verify(d)


def test_verify_greedy():
    g, rng = gen(1), np.random.default_rng(1)
    B, n = 40, 15
    d = verify_problem(B, n, 5, False, seed=3)
    d["targets"] = torch.randint(0, 5, (B, n), generator=g, device="cuda", dtype=torch.int32)
    d["tokens"] = torch.randint(0, 5, (B, n), generator=g, device="cuda", dtype=torch.int32)
    d["counts"] = torch.tensor(rng.integers(0, n + 1, B), dtype=torch.int32, device="cuda")
    d["probs"] = d["uniforms"] = None
    bq.verify_tree(**d)
    for b in range(B):
        tok, par, tgt = (d[k][b].tolist() for k in ("tokens", "parents", "targets"))
        cur, path = 0, [0]
        for i in range(1, int(d["counts"][b])):
            if par[i] == cur and tok[i] == tgt[cur]:
                cur = i
                path.append(i)
        if int(d["counts"][b]) == 0:
            path, nxt = [], -1
        else:
            nxt = tgt[cur]
        assert d["path"][b].tolist() == path + [-1] * (n - len(path))
        assert int(d["n_path"][b]) == len(path) and int(d["next_token"][b]) == nxt


@pytest.mark.parametrize("soft", [False, True])
def test_verified_tokens_follow_the_target(soft):
    """The first token that comes out (the first kept draft's, else next) has the target's distribution: counts of
    200,000 trials within 6 standard deviations of a binomial."""
    B, V = 200_000, 6
    g = gen(21)
    p = torch.tensor([0.05, 0.4, 0.1, 0.25, 0.15, 0.05], device="cuda")
    q = torch.tensor([0.3, 0.1, 0.2, 0.2, 0.1, 0.1], device="cuda")
    tok = torch.zeros(B, 3, dtype=torch.int32, device="cuda")
    if soft:
        tok[:, 1:] = torch.multinomial(q, 2 * B, replacement=True, generator=g).view(B, 2)
    else:
        tok[:, 1:] = torch.tensor([1, 3], dtype=torch.int32)
    par = torch.tensor([-1, 0, 0], dtype=torch.int32, device="cuda").repeat(B, 1)
    out = [torch.empty(B, 3, dtype=torch.int32, device="cuda")] + [torch.empty(B, dtype=torch.int32, device="cuda")
                                                                  for _ in range(2)]
    bq.verify_tree(tok, par, torch.rand(B, 3, device="cuda", generator=g), p.expand(B, 3, V), *out,
                   draft_probs=q.expand(B, 3, V) if soft else None)
    path, n_path, nxt = out
    second = path[:, 1].clamp_min(0).long()
    first = torch.where(n_path > 1, tok.gather(1, second[:, None])[:, 0], nxt)
    freq = torch.bincount(first, minlength=V).double()
    dev = (freq - B * p.double()).abs() / (B * p.double() * (1 - p.double())).sqrt()
    assert float(dev.max()) < 6, dev


# ---- commit ------------------------------------------------------------------------
@pytest.mark.parametrize("kv", ["bf16", "q8"])
@pytest.mark.parametrize("B,L,H,n,hd,cap", [(1, 1, 1, 1, 64, 1), (3, 2, 2, 7, 128, 20), (2, 5, 3, 64, 64, 100),
                                            (4, 1, 8, 5, 128, 9)])
def test_commit(B, L, H, n, hd, cap, kv):
    g, rng = gen(n), np.random.default_rng(n)
    cache = [make_rows(B * L, H, cap, hd, kv, g) for _ in range(2)]
    tree = [make_rows(B * L, H, n, hd, kv, g) for _ in range(2)]
    shape = lambda t: None if t is None else t.view(B, L, *t.shape[1:])  # noqa: E731
    cache, tree = ([tuple(shape(x) for x in t) for t in s] for s in (cache, tree))
    want = [tuple(None if x is None else x.clone() for x in t) for t in cache]
    lens = [int(rng.integers(0, cap)) for _ in range(B)]
    path = np.full((B, n), -1, np.int32)
    n_path = np.zeros(B, np.int32)
    for b in range(B):
        m = int(rng.integers(1, n + 1))
        path[b, :m] = np.sort(rng.permutation(n)[:m])
        n_path[b] = m
    if B > 2:
        n_path[1] = 0
        path[2, 0] = n + 3  # out of range: its cache row stays
    end = []
    for b in range(B):
        m = min(n_path[b], cap - lens[b])
        for j in range(m):
            if 0 <= path[b, j] < n:
                for t in range(2):
                    for w, x in zip(want[t], tree[t]):
                        if w is not None:
                            w[b, :, :, lens[b] + j] = x[b, :, :, path[b, j]]
        end.append(lens[b] + m)
    dev = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (lens, path, n_path)]
    views = [bq.KVView(s[0][0], s[1][0], s[0][1], s[1][1]) for s in (cache, tree)]
    new = torch.empty(B, dtype=torch.int32, device="cuda")
    bq.commit_tree(*views, *dev, new)
    assert new.tolist() == end
    for t in range(2):
        for got, w in zip(cache[t], want[t]):
            assert w is None or torch.equal(got, w)
    bq.commit_tree(*views, *dev, dev[0])  # the lengths advance in place, the same rows are written
    assert dev[0].tolist() == end


def test_commit_strided_single_layer():
    B, H, n, hd, cap = 2, 3, 4, 64, 16
    g = gen(0)
    big = torch.randn(cap, H, B, 2, hd + 8, device="cuda", generator=g).to(torch.bfloat16)
    before = big.clone()
    k, v = (big[..., i, :hd].permute(2, 1, 0, 3) for i in range(2))
    tk, tv = (torch.randn(B, H, n, hd, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    bq.commit_tree(bq.KVView(k, v), bq.KVView(tk, tv), i32([3, 14]), i32([[0, 2, 3, -1], [0, 1, 2, 3]]), i32([3, 4]),
                   i32([0, 0]))
    want = before.clone()
    for i, t in ((0, tk), (1, tv)):
        for j, node in enumerate([0, 2, 3]):
            want[3 + j, :, 0, i, :hd] = t[0, :, node]
        for j in range(2):
            want[14 + j, :, 1, i, :hd] = t[1, :, j]
    assert torch.equal(big, want)


# ---- together ------------------------------------------------------------------------
@pytest.mark.parametrize("kv", ["bf16", "q8"])
def test_a_decoding_step_of_all_four(kv):
    """Attention over cache and tree, probabilities of its (synthetic) logits, verification, commit; then the kept
    nodes' attention over the grown cache alone equals their attention in the tree."""
    B, n, Hkv, gq, hd, cap, V = 3, 9, 2, 2, 64, 80, 777
    p = Problem(B=B, n=n, Hkv=Hkv, gq=gq, hd=hd, cap=cap, lens=(40, 0, 70), q="f32", kv=kv, seed=4)
    g = gen(9)
    head = torch.randn(Hkv * gq * hd, V, device="cuda", generator=g) * 0.3
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    path, n_path, nxt, new = i32(B, n), i32(B), i32(B), i32(B)
    tokens = torch.zeros(B, n, dtype=torch.int32, device="cuda")
    par = torch.tensor(p.parents, dtype=torch.int32, device="cuda")
    probs, u = torch.empty(B * n, V, device="cuda"), torch.rand(B, n, device="cuda", generator=g) * 0.2
    p.call()
    p.check()
    logits = p.out.view(B * n, -1) @ head
    bq.token_probs(logits, probs, 0.8, 20, 0.9)
    best = probs.view(B, n, V).argmax(-1)
    for i in range(1, n):
        tokens[:, i] = best.gather(1, par[:, i:i + 1].long())[:, 0]
    bq.verify_tree(tokens, par, u, probs.view(B, n, V), path, n_path, nxt)
    bq.commit_tree(p.cache(), p.tree(), p.lens, path, n_path, new)
    assert int(n_path.max()) > 1
    for b in range(B):
        want, t = verify_reference(tokens[b].cpu().numpy(), par[b].cpu().numpy(), u[b].cpu().numpy(),
                                   probs.view(B, n, V)[b].cpu().numpy(), None, n)
        assert path[b, :int(n_path[b])].tolist() == want and int(nxt[b]) == t
    assert torch.equal(new, p.lens + n_path)
    last = path.gather(1, (n_path - 1)[:, None].long())[:, 0].long()
    q1 = p.q[torch.arange(B, device="cuda"), last][:, None].contiguous()
    one = Problem(B=B, n=1, Hkv=Hkv, gq=gq, hd=hd, cap=cap, kv=kv)
    one.k, one.v, one.ks, one.vs, one.q, one.lens, one.with_tree, one.mask = p.k, p.v, p.ks, p.vs, q1, new, False, None
    one.out = torch.full_like(q1, 7.0)
    one.call()
    one.check()


def test_a_captured_step_replays_like_the_eager_one():
    """Attention, probabilities (with and without top-k), verification and commit in a graph each on two streams,
    replayed at once with new inputs, leave the bits that eager calls leave."""
    B, n, Hkv, gq, hd, cap, V = 3, 9, 2, 2, 64, 400, 3001
    par = torch.tensor(random_parents(n, np.random.default_rng(4)), dtype=torch.int32, device="cuda").expand(B, n).contiguous()

    class Step:
        def __init__(self, k):
            self.k = k
            self.p = Problem(B=B, n=n, Hkv=Hkv, gq=gq, hd=hd, cap=cap, lens=(40, 0, 350), q="bf16", seed=k)
            self.views = self.p.cache(), self.p.tree()
            self.logits = torch.empty(B * n, V, device="cuda")
            self.probs = torch.empty_like(self.logits)
            self.tokens = torch.empty(B, n, dtype=torch.int32, device="cuda")
            self.u = torch.empty(B, n, device="cuda")
            self.path, self.outs = self.tokens.clone(), [torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2)]

        def renew(self, seed):
            g = gen(seed)
            self.logits.normal_(generator=g).mul_(2)
            self.tokens.random_(0, V, generator=g)
            best = self.logits.view(B, n, V).argmax(-1).int()
            self.u.uniform_(generator=g).mul_(0.3)
            self.tokens[:, 1:] = torch.where(self.u[:, 1:] < 0.2, best.gather(1, par[:, 1:].long()), self.tokens[:, 1:])
            self.p.lens.copy_(torch.tensor([40, 0, 350], dtype=torch.int32))
            self.p.k.normal_(generator=g)
            self.p.v.normal_(generator=g)
            self.p.out.fill_(7.0)

        def run(self, st):
            p = self.p
            bq.tree_attention(p.q, *self.views, p.lens, p.mask, p.out, stream=st)
            bq.token_probs(self.logits, self.probs, 0.8, self.k, 1.0, stream=st)
            bq.verify_tree(self.tokens, par, self.u, self.probs.view(B, n, V), self.path, *self.outs, stream=st)
            bq.commit_tree(*self.views, p.lens, self.path, self.outs[0], p.lens, stream=st)

        def state(self):
            p = self.p
            return [t.clone() for t in (p.out, self.probs, self.path, *self.outs, p.lens, p.k, p.v)]

    steps, streams, graphs = [Step(0), Step(20)], [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for s, st in zip(steps, streams):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=st):
            s.run(st.cuda_stream)
    for rep in range(3):
        want = []
        for s in steps:
            s.renew(rep)
            s.run(None)
            want.append(s.state())
        for s in steps:
            s.renew(rep)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            for a, b in zip(s.state(), w):
                assert torch.equal(a, b)
            assert (s.p.lens > torch.tensor([40, 0, 350], dtype=torch.int32, device="cuda")).all()
    bq.tree_status()
