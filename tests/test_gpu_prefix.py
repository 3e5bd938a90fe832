"""prefix_attention against a plain implementation in 64 bits (GPU).

Tolerances are those of the tree attention's tests (its docstring derives them), over all the keys that a node sees:
per output element, with A = sum_j p_j |v_j|,
  tol = round |o| + A (2 ds + 2^-21 + part + 2 (N + 64) 2^-23) + N 2^-126 max |v|,  ds = (hd + 8) 2^-23 max_j sum_d |q k| scale,
part = 2^-23 for fp32 queries (three bf16 parts), 2^-16 for bf16 ones and 2 2^-8 where the batch has more than 64 query
rows of a kv head over bf16 rows (one part), 2^-16 more for int8 values. One part: every p of the prefix is rounded to
bf16 once, half a step of 2^-8 p at most, so sum p v is off by 2^-8 A; where the sum of p is taken of the rounded ones it
is off by 2^-8 of itself, 2^-8 A again. The kernel is chosen on the host, which knows the batch's rows and not how they
fall into groups, so it is the batch's number that counts: a small group beside large ones has one part too. Joining the two parts: their two weights are within 2^-21
(exp2, products, a quotient), so 2^-20 A more.
"""
import math

import numpy as np
import pytest
import torch

import bit_quantized_token_gb300 as bq

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def library():
    bq.build()
    torch.cuda.set_device(0)


def make_rows(shape, kv, g):
    x = torch.randn(shape, device="cuda", generator=g)
    if kv == "bf16":
        return x.to(torch.bfloat16), None
    z = x.view(*shape[:-1], shape[-1] // 32, 32)
    s = (z.abs().amax(-1, keepdim=True) / 127).half()
    return (z / s.float()).round().clamp(-127, 127).to(torch.int8).view(shape), s.squeeze(-1)


def values(rows, scales):
    return rows.double() if scales is None else rows.double() * scales.double().repeat_interleave(32, -1)


class Problem:
    """B sequences of n nodes in groups from `starts`; own lengths, prefix lengths and counts as given (repeated)."""

    def __init__(self, starts=(0, 3), n=1, Hkv=2, gq=2, hd=64, P=300, own=40, lens=(17, 40, 0), plens=(300,), q="bf16",
                 kv="bf16", tree=True, counts=None, B=None, seed=0, scale=None):
        g, rng = torch.Generator("cuda"), np.random.default_rng(seed)
        g.manual_seed(seed)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.B = B = starts[-1] if B is None else B
        self.G = len(starts) - 1
        self.n, self.gq, self.hd, self.kv, self.scale = n, gq, hd, kv, scale
        self.starts, self.plens = starts, [plens[i % len(plens)] for i in range(self.G)]
        self.lens = [lens[i % len(lens)] for i in range(B)]
        self.counts = None if counts is None else [counts[i % len(counts)] for i in range(B)]
        self.rows = {}
        for name, seqs, R in (("prefix", self.G, P), ("cache", B, own), ("tree", B, n)):
            ks, vs = make_rows((seqs, Hkv, R, hd), kv, g), make_rows((seqs, Hkv, R, hd), kv, g)
            self.rows[name] = [ks[0], vs[0], ks[1], vs[1]]
        self.q = torch.randn(B, n, Hkv * gq, hd, device="cuda", generator=g).to(TYPES[q])
        self.words = [[int(rng.integers(0, 1 << n)) | (1 << i) for i in range(n)] for _ in range(B)]
        if n > 2:
            self.words[0][1] = 0  # a node that sees none of the tree
        self.tree = tree
        self.t = dict(starts=i32(starts), plens=i32(self.plens), lens=i32(self.lens),
                      counts=None if counts is None else i32(self.counts), mask=torch.tensor(self.words, device="cuda"))
        self.out = torch.full_like(self.q, 7.0)
        self.workspace = torch.full((bq.prefix_workspace(self.q),), 255, dtype=torch.uint8, device="cuda")  # NaNs

    def view(self, name):
        return bq.KVView(*self.rows[name])

    def call(self, **kw):
        t = self.t
        bq.prefix_attention(self.q, self.view("prefix"), t["starts"], t["plens"], self.view("cache"),
                            self.view("tree") if self.tree else None, t["lens"], t["mask"], self.out, self.workspace,
                            counts=t["counts"], scale=self.scale, **kw)
        return self.out

    def check(self):
        bq.tree_status()
        bf, hd, gq, n = self.q.dtype == torch.bfloat16, self.hd, self.gq, self.n
        scale = hd ** -0.5 if self.scale is None else self.scale
        Hkv = self.q.shape[2] // gq
        wide = {name: [values(r[i], r[2 + i]) for i in (0, 1)] for name, r in self.rows.items()}
        for b in range(self.B):
            cnt = n if self.counts is None else min(max(self.counts[b], 0), n)
            assert (self.out[b, cnt:] == 7).all(), "rows past the count were written"
            g = next((g for g in range(self.G) if self.starts[g] <= b < self.starts[g + 1]), None)
            P = 0 if g is None else min(max(self.plens[g], 0), self.rows["prefix"][0].shape[2])
            L = min(max(self.lens[b], 0), self.rows["cache"][0].shape[2])
            for i in range(cnt):
                js = [j for j in range(cnt) if self.tree and self.words[b][i] >> j & 1]
                K, V = (torch.cat([wide["prefix"][m][g or 0, :, :P], wide["cache"][m][b, :, :L], wide["tree"][m][b][:, js]], 1)
                        for m in (0, 1))
                got = self.out[b, i].double().view(Hkv, gq, hd)
                if K.shape[1] == 0:
                    assert (got == 0).all(), "a row that sees nothing must be 0"
                    continue
                x = self.q[b, i].double().view(Hkv, gq, hd)
                w = torch.softmax(x @ K.transpose(1, 2) * scale, -1)
                o, A = w @ V, w @ V.abs()
                ds = (hd + 8) * 2.0 ** -23 * (x.abs() @ K.abs().transpose(1, 2)).amax(-1, keepdim=True) * abs(scale)
                rnd, part = (2.0 ** -8, 2.0 ** -16) if bf else (2.0 ** -24, 2.0 ** -23)
                if bf and self.kv == "bf16" and self.B * n * gq > 64:
                    part = 2 * 2.0 ** -8
                if bf and self.kv == "q8":
                    part += 2.0 ** -16
                tol = rnd * o.abs() + A * (2 * ds + 2.0 ** -21 + 2.0 ** -20 + part + 2 * (K.shape[1] + 64) * 2.0 ** -23)
                tol = tol + K.shape[1] * 2.0 ** -126 * V.abs().max()
                err = (got - o).abs()
                assert (err <= tol).all(), (b, i, float((err / tol).max()))


CASES = [
    dict(),
    dict(starts=(0, 1), P=1, plens=(1,), lens=(0,), tree=False, q="f32", gq=1, Hkv=1),
    dict(starts=(0, 2), P=257, plens=(257,), lens=(3, 40), Hkv=4, gq=8, q="f32"),
    dict(starts=(0, 2, 7, 7, 9), n=3, P=200, plens=(200, 129, 5, 0), gq=3, hd=128),
    dict(starts=(0, 2, 7, 9), n=2, P=200, plens=(1000, 128, -4), q="f32", hd=128, gq=5, Hkv=1),
    dict(starts=(0, 5), n=4, P=300, plens=(290,), kv="q8", counts=(4, 0, 1, 9, -2)),
    dict(starts=(0, 3, 8), n=2, P=140, plens=(140, 77), kv="q8", hd=128, gq=4, q="f32"),
    dict(starts=(2, 4, 6), B=9, n=1, P=130, plens=(100, 130), gq=2),  # sequences of no group
    dict(starts=(0, 40), n=1, P=700, plens=(650,), gq=4, Hkv=2, lens=(0, 1, 39)),  # 160 rows a kv head
    dict(starts=(0, 33, 50), n=2, P=515, plens=(515, 384), gq=7, Hkv=1, hd=128),
    dict(starts=(0, 100, 130, 131), n=1, P=1100, plens=(1100, 1024, 999), gq=8, Hkv=2),
    dict(starts=(0, 65, 130), n=1, P=700, plens=(650, 0), gq=4, Hkv=2, lens=(0, 1, 39)),  # 520 rows of 64 dims
    dict(starts=(0, 129), n=1, P=1290, plens=(1283,), gq=2, Hkv=2, hd=128, tree=False),
    dict(starts=(0, 20), n=7, P=256, plens=(256,), gq=2, kv="q8", hd=64),
    dict(starts=(0, 3), P=300, scale=-0.3, q="f32"),
    dict(starts=(0, 40), P=300, scale=0.0, gq=4),
    dict(starts=(0, 70), P=300, scale=4.0, gq=2, hd=128),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_against_the_formula(i):
    p = Problem(**CASES[i], seed=i)
    p.call()
    p.check()


@pytest.mark.parametrize("starts,gq", [((0, 3), 2), ((0, 90), 4), ((0, 130), 4)])
@pytest.mark.parametrize("kv", ["bf16", "q8"])
def test_rows_that_nobody_sees(starts, gq, kv):
    """Infinities and NaN behind the prefix's, the cache's and the tree's ends have no influence."""
    p = Problem(starts=starts, gq=gq, n=2, kv=kv, P=200, plens=(131,), own=300, lens=(0, 129, 290))
    for b in range(p.B):
        for w in range(2):
            p.words[b][w] = 1 << w
    p.t["mask"] = torch.tensor(p.words, device="cuda")
    p.call()
    p.check()
    clean = p.out.clone()
    bad = 2 if kv == "q8" else 0
    for name, seq_lens in (("prefix", [131]), ("cache", p.lens)):
        for s, L in enumerate(seq_lens):
            for m in (bad, bad + 1):
                p.rows[name][m][s, :, L:] = math.nan
                p.rows[name][m][s, :, L + 1::2] = math.inf
    p.call()
    bq.tree_status()
    assert torch.equal(p.out, clean)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("q", ["bf16", "f32"])
@pytest.mark.parametrize("starts,gq,n", [((0, 3), 2, 4), ((0, 3), 4, 4), ((0, 90), 2, 3), ((0, 130), 2, 3)])
def test_infinities_and_nan_of_the_tree(starts, gq, n, q, hd):
    """Where they are seen they are the result, elsewhere they have no influence."""
    p = Problem(starts=starts, gq=gq, n=n, hd=hd, q=q, P=150, plens=(140,))
    p.words = [[1 << i for i in range(n)] for _ in range(p.B)]
    p.t["mask"] = torch.tensor(p.words, device="cuda")
    clean = p.call().clone()
    v = p.rows["tree"][1]
    v[1, :, 1, 5::7] = math.inf
    v[1, :, 1, 6::7] = -math.inf
    v[1, :, 2, 9] = math.nan
    p.rows["tree"][0][2, :, 0] = math.nan  # every score of node 0's own row
    out = p.call()
    bq.tree_status()
    want = clean.clone()
    want[1, 1, :, 5::7] = math.inf
    want[1, 1, :, 6::7] = -math.inf
    want[1, 2, :, 9] = math.nan
    want[2, 0] = math.nan
    assert torch.equal(out.isnan(), want.isnan())
    assert torch.equal(out[~want.isnan()], want[~want.isnan()])


@pytest.mark.parametrize("starts,gq", [((0, 3), 2), ((0, 3), 16), ((0, 90), 4), ((0, 130), 4)])
@pytest.mark.parametrize("kv", ["bf16", "q8"])
def test_a_nan_query_is_its_rows_result(starts, gq, kv):
    for lens, tree in (((17,), True), ((0,), False)):
        p = Problem(starts=starts, gq=gq, kv=kv, lens=lens, tree=tree)
        clean = p.call().clone()
        p.q[1, 0, 0] = math.nan
        out = p.call()
        bq.tree_status()
        assert out[1, 0, 0].isnan().all()
        out[1, 0, 0] = clean[1, 0, 0]
        assert torch.equal(out, clean)


@pytest.mark.parametrize("kv,hd,own", [("bf16", 64, 16000), ("bf16", 128, 380), ("q8", 128, 9000)])
def test_long_fp32_sums_do_not_come_out_low(kv, hd, own):
    """Positive values, so that what is cut off adds up: a step's three products lose less than 2^-23 of its sum each,
    always downwards; all other additions round, either way. The mean error is below 4 2^-23."""
    p = Problem(starts=(0, 1), B=1, gq=4, hd=hd, q="f32", kv=kv, P=16, plens=(1,), own=own, lens=(own,), tree=False)
    p.q *= 0.05
    for name in ("prefix", "cache"):
        p.rows[name][1].abs_()
    p.call()
    bq.tree_status()
    K, V = (torch.cat([values(p.rows["prefix"][i], p.rows["prefix"][2 + i])[0][:, :1],
                       values(p.rows["cache"][i], p.rows["cache"][2 + i])[0]], 1) for i in (0, 1))
    want = (torch.softmax(p.q[0, 0].double().view(2, 4, hd) @ K.transpose(1, 2) * hd ** -0.5, -1) @ V).view(8, hd)
    assert abs(float(((p.out[0, 0].double() - want) / want).mean())) < 2.0 ** -21


@pytest.mark.parametrize("B,gq,hd,kv", [(100, 4, 64, "bf16"), (256, 1, 128, "bf16"), (70, 2, 128, "q8"), (300, 2, 64, "bf16")])
def test_many_sequences_of_rising_lengths(B, gq, hd, kv):
    lens = [b * 300 // B for b in range(B)]
    p = Problem(starts=(0, B - 3), B=B, gq=gq, hd=hd, kv=kv, P=130, plens=(129,), own=300, lens=lens, Hkv=1)
    p.call()
    p.check()
    assert torch.equal(p.out, p.call())


@pytest.mark.parametrize("starts,gq", [((0, 3), 2), ((0, 90), 4), ((0, 130), 4)])
def test_scores_of_any_size(starts, gq):
    """Scores far apart, in the prefix or in the own rows: one key takes it all."""
    for where in ("prefix", "cache"):
        p = Problem(starts=starts, gq=gq, P=400, plens=(400,), own=40, lens=(40,), tree=False, hd=64)
        p.q[:] = 1.0
        for name in ("prefix", "cache"):
            p.rows[name][0][:] = -2.0 ** 20
        p.rows[where][0][:, :, 37] = 2.0 ** 20
        p.call()
        bq.tree_status()
        want = p.rows[where][1][:, :, 37]  # [group or seq, Hkv, hd]
        want = want.expand(p.B, -1, -1).repeat_interleave(gq, 1)[:, None]
        assert torch.equal(p.out, want)


def test_strides_shared_heads_and_streams():
    """Queries and outputs of another order, a prefix that all heads share (a stride of 0), two calls at once on two
    streams with a workspace each."""
    ps = []
    for seed in (1, 2):
        p = Problem(starts=(0, 4, 50), n=2, gq=2, Hkv=2, P=333, plens=(333, 200), seed=seed)
        p.q = p.q.permute(2, 1, 0, 3).contiguous().permute(2, 1, 0, 3)
        p.out = torch.full((2, *p.q.shape), 7.0, device="cuda", dtype=p.q.dtype)[1]
        for m in (0, 1):
            p.rows["prefix"][m] = p.rows["prefix"][m][:, :1].expand(-1, 2, -1, -1)
        ps.append(p)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(5):
        for p, s in zip(ps, streams):
            p.call(stream=s.cuda_stream)
    torch.cuda.synchronize()
    for p in ps:
        p.check()


def test_captured_and_repeated():
    """A captured call reads lengths and groups when it is replayed, and gives the same bits every time."""
    p = Problem(starts=(0, 30, 60), n=1, gq=4, P=600, plens=(600, 311), lens=(40, 3, 0))
    p.call()
    p.check()
    first = p.out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        p.call(stream=torch.cuda.current_stream().cuda_stream)
    for _ in range(3):
        p.out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.out, first)
    p.starts, p.plens, p.lens = (0, 10, 59), [17, 600], [p.lens[(b + 1) % 3] for b in range(p.B)]
    for name, v in (("starts", p.starts), ("plens", p.plens), ("lens", p.lens)):
        p.t[name].copy_(torch.tensor(v, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("starts,gq,hd", [((0, 64), 2, 128), ((0, 64), 2, 64), ((0, 30, 90, 154, 300), 1, 128), ((0, 257), 4, 64)])
def test_many_calls_in_a_row(starts, gq, hd):
    """The same bits from every one of 300 calls behind one another, row tiles without rows among them, and no wait that
    runs out."""
    p = Problem(starts=starts, gq=gq, hd=hd, Hkv=8, P=2100, plens=(2100, 130, 1999), own=20, lens=(7, 20), tree=False)
    p.call()
    p.check()
    first = p.out.clone()
    outs = [torch.empty_like(p.out) for _ in range(3)]
    for i in range(300):
        p.out = outs[i % 3]
        p.call()
        if i % 3 == 2:
            assert all(torch.equal(o, first) for o in outs), i
    bq.tree_status()


def test_a_step_of_a_served_batch():
    """Append, then attend with the appended row as the last own row, on one stream without waits between them."""
    g = torch.Generator("cuda")
    g.manual_seed(3)
    for kv in ("bf16", "q8"):
        p = Problem(starts=(0, 12), n=1, gq=2, Hkv=2, hd=128, P=300, plens=(300,), own=20, lens=(19, 7, 0), tree=False, kv=kv)
        k, v = (torch.randn(12, 2, 128, device="cuda", generator=g) for _ in range(2))
        raw = p.q.float().view(12, 4, 128)
        seqs = torch.arange(12, dtype=torch.int32, device="cuda")
        rows = p.t["lens"].clone()
        p.t["lens"] += 1
        p.lens = [x + 1 for x in p.lens]
        torch.cuda.synchronize()
        bq.append_kv(k, v, p.view("cache"), seqs, rows, q=raw, q_out=p.q.view(12, 4, 128), positions=rows + 300,
                     rope_theta=10000.0, rope_neox=True)
        p.call()
        p.check()  # over the cache's rows as they are now
        back = [torch.empty(12, 2, 128, device="cuda") for _ in range(2)]
        bq.read_kv(p.view("cache"), seqs, rows, *back)
        assert ((back[1] - v).abs() <= v.abs().amax() * (2.0 ** -8 if kv == "bf16" else 0.5 / 127 + 2.0 ** -11)).all()
