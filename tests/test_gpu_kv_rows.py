"""append_kv and read_kv against the formulas in 64 bits (GPU).

Tolerances from the roundings, with u = 2^-24: the norm's sum of hd squares is within hd u, its square root halves
that; the reciprocal root 4 u and two products 2 u, so a normed value is within (hd / 2 + 8) u. cos and sin: a quarter half-turn
in fp32, sincospi within 2 steps, the turn's table 2^-50 a position: 2^-22 + 2 pi |pos| 2^-50. A rotated value is two
products and a sum: tol = (|a| + |b|) ((hd / 2 + 8) u + 2^-22 + 2 pi |pos| 2^-50 + 3 u), and half a step of the output.
Int8: a code is within half a scale of the value that it stands for (the scale's own rounding leaves 127.07 at most, so
nothing is clamped), the scale within half a step of fp16 (2^-11, or 2^-25 below its normal range).
"""
import math

import numpy as np
import pytest
import torch

import bit_quantized_token_gb300 as bq
import synth

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def library():
    bq.build()
    torch.cuda.set_device(0)


def gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def make_cache(B, H, R, hd, kv, g, L=None):
    shape = (B, H, R, hd) if L is None else (B, L, H, R, hd)
    if kv == "bf16":
        return [torch.randn(shape, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2)] + [None, None]
    codes = [torch.randint(-127, 128, shape, device="cuda", generator=g).to(torch.int8) for _ in range(2)]
    return codes + [(torch.rand(*shape[:-1], hd // 32, device="cuda", generator=g) * 0.02).half() for _ in range(2)]


def quantised(x):
    """Codes and scales of fp32 values, decided in fp32."""
    z = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    s = (z.abs().amax(-1, keepdim=True) / 127).half()
    r = z / torch.where(s == 0, 1, s.float())
    c = torch.where(s == 0, 0, ((r.abs().double() + 0.5).floor().clamp_max(127) * r.sign()))
    return c.to(torch.int8).reshape(x.shape), s.squeeze(-1)


def reference(x, w, pos, theta, neox):
    """(value, |a| + |b|) of the normed and rotated heads in 64 bits."""
    x, hd = x.double(), x.shape[-1]
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.double()
    if theta is None:
        return x, x.abs()
    i = torch.arange(hd // 2, device="cuda")
    a = pos.double()[:, None, None] * theta ** (-2.0 * i.double() / hd)
    ia, ib = (i, i + hd // 2) if neox else (2 * i, 2 * i + 1)
    out, size = torch.empty_like(x), torch.empty_like(x)
    out[..., ia] = x[..., ia] * a.cos() - x[..., ib] * a.sin()
    out[..., ib] = x[..., ia] * a.sin() + x[..., ib] * a.cos()
    size[..., ia] = size[..., ib] = x[..., ia].abs() + x[..., ib].abs()
    return out, size


def tolerance(size, out, pos, hd, dtype):
    far = 2 * math.pi * pos.double().abs()[:, None, None] * 2.0 ** -50
    return size * ((hd / 2 + 8) * 2.0 ** -24 + 2.0 ** -22 + far + 3 * 2.0 ** -24) + out.abs() * torch.finfo(dtype).eps / 2


CASES = [
    # T, Hq, Hkv, hd, in, out, cache, norm, theta, neox, positions up to
    (1, 32, 4, 64, "f32", "f32", "bf16", False, 10000.0, False, 4),
    (1, 1, 1, 128, "bf16", "bf16", "q8", True, 1e6, True, 1 << 31),
    (5, 7, 1, 64, "bf16", "f32", "q8", True, 10000.0, False, 1 << 20),
    (33, 16, 8, 128, "f32", "bf16", "q8", True, 1e6, True, 40000),
    (33, 6, 3, 64, "f32", "f32", "bf16", True, 500000.0, True, 1 << 24),
    (257, 5, 5, 128, "bf16", "bf16", "bf16", False, None, True, 9),
    (1000, 16, 8, 128, "bf16", "bf16", "bf16", True, 10000.0, True, 1 << 30),
    (4099, 8, 2, 64, "f32", "f32", "q8", False, 10000.0, True, 131072),
]
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("T,Hq,Hkv,hd,xt,ot,kv,norm,theta,neox,far", CASES)
def test_append(T, Hq, Hkv, hd, xt, ot, kv, norm, theta, neox, far):
    g, rng = gen(T + hd), np.random.default_rng(T)
    B, R = 3, (T + 2) // 3 + 5
    qkv = torch.randn(T, Hq + 2 * Hkv, hd, device="cuda", generator=g).to(TYPES[xt])
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    qw, kw = (1 + 0.3 * torch.randn(hd, device="cuda", generator=g) if norm else None for _ in range(2))
    cache = make_cache(B, Hkv, R, hd, kv, g)
    before = [None if x is None else x.clone() for x in cache]
    at = torch.from_numpy(rng.permutation(B * R)[:T])
    seqs, rows = (at // R).to(torch.int32).cuda(), (at % R).to(torch.int32).cuda()
    gone = torch.zeros(T, dtype=torch.bool, device="cuda")
    if T > 4:  # padding of four kinds
        for i, (s, r) in enumerate([(-1, 0), (B, 0), (0, -1), (1, R)]):
            seqs[i], rows[i], gone[i] = s, r, True
    pos = torch.from_numpy(rng.integers(0, far, T)).to(torch.int32).cuda()
    if T > 6:
        pos[5] = -3
    out = torch.empty(T, Hq, hd, device="cuda", dtype=TYPES[ot])
    bq.append_kv(k, v, bq.KVView(*cache), seqs, rows, q=q, q_out=out, positions=pos, rope_theta=theta, rope_neox=neox,
                 q_norm=qw, k_norm=kw, eps=EPS)
    want, size = reference(q, qw, pos, theta, neox)
    assert ((out.double() - want).abs() <= tolerance(size, want, pos, hd, out.dtype)).all()
    kept = ~gone
    s, r = seqs[kept].long(), rows[kept].long()
    want, size = reference(k[kept], kw, pos[kept], theta, neox)
    near = tolerance(size, want, pos[kept], hd, torch.float32)
    if kv == "bf16":
        assert ((cache[0][s, :, r].double() - want).abs() <= near + want.abs() * 2.0 ** -8).all()
        assert torch.equal(cache[1][s, :, r], v[kept].to(torch.bfloat16))
    else:
        codes, scales = cache[0][s, :, r].double(), cache[2][s, :, r].double()
        group = lambda x: x.reshape(*x.shape[:-1], hd // 32, 32)  # noqa: E731
        amax, slack = group(want).abs().amax(-1), group(near).amax(-1)
        assert ((scales - amax / 127).abs() <= (amax + slack) / 127 * 2.0 ** -11 + slack / 127 + 2.0 ** -25).all()
        wide = scales.repeat_interleave(32, -1)
        assert ((codes * wide - want).abs() <= wide / 2 + near).all()
        vc, vs = quantised(v[kept].float())
        assert torch.equal(cache[1][s, :, r], vc) and torch.equal(cache[3][s, :, r], vs)
    untouched = torch.ones(B, R, dtype=torch.bool, device="cuda")
    untouched[s, r] = False
    for x, old in zip(cache, before):
        if x is not None:
            assert torch.equal(x.transpose(1, 2)[untouched], old.transpose(1, 2)[untouched])


def test_in_place_views_and_another_stream():
    """q_out = q; a cache with its own order and gaps; default positions; not on the default stream."""
    g, T, hd = gen(5), 40, 64
    qkv = torch.randn(T, 8, hd, device="cuda", generator=g)
    keep = qkv.clone()
    store = torch.zeros(2, 50, 2, 3, hd, device="cuda", dtype=torch.bfloat16)  # [k or v][row][head][seq][dim]
    k, v = store[0].permute(2, 1, 0, 3), store[1].permute(2, 1, 0, 3)
    seqs = (torch.arange(T, device="cuda") % 3).to(torch.int32)
    rows = torch.arange(T, device="cuda").to(torch.int32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bq.append_kv(qkv[:, 4:6], qkv[:, 6:], bq.KVView(k, v), seqs, rows, q=qkv[:, :4], q_out=qkv[:, :4],
                     rope_theta=10000.0, stream=side.cuda_stream)
    side.synchronize()
    for got, x in ((qkv[:, :4].double(), keep[:, :4]), (k[seqs.long(), :, rows.long()].double(), keep[:, 4:6])):
        want, size = reference(x, None, rows, 10000.0, False)
        tol = tolerance(size, want, rows, hd, torch.float32) + (want.abs() * 2.0 ** -8 if x.shape[1] == 2 else 0)
        assert ((got - want).abs() <= tol).all()
    assert torch.equal(v[seqs.long(), :, rows.long()], keep[:, 6:].to(torch.bfloat16))
    assert (store != 0).any(-1).sum() == 2 * 2 * T  # nothing else was written


def test_int8_extremes():
    """Zeros, the smallest and the largest values, infinities and NaN of an int8 row."""
    x = torch.zeros(1, 1, 128, device="cuda")
    x[0, 0, 0:32] = 0.0
    x[0, 0, 32:64] = torch.linspace(-1e9, 1e9, 32, device="cuda")  # past 65504 * 127
    x[0, 0, 64] = math.inf
    x[0, 0, 65] = -math.inf
    x[0, 0, 96] = math.nan
    x[0, 0, 97] = 1.0
    cache = make_cache(1, 1, 2, 128, "q8", gen(1))
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    bq.append_kv(x, x, bq.KVView(*cache), zero, zero)
    back = [torch.empty(1, 1, 128, device="cuda") for _ in range(2)]
    bq.read_kv(bq.KVView(*cache), zero, zero, *back)
    for b in back:
        b = b[0, 0]
        assert (b[0:32] == 0).all()
        assert b[32] == -65504 * 127 and b[63] == 65504 * 127
        assert b[64] == 65504 * 127 and b[65] == -65504 * 127 and (b[66:96] == 0).all()
        assert b[96:].isnan().all()


@pytest.mark.parametrize("T,L,H,hd,kv,xt", [(1, 1, 1, 64, "bf16", "bf16"), (7, 3, 5, 128, "q8", "f32"),
                                            (131, 2, 4, 64, "q8", "bf16"), (515, 4, 8, 128, "bf16", "f32")])
def test_read(T, L, H, hd, kv, xt):
    g, rng = gen(T), np.random.default_rng(T)
    B, R = 3, 200
    cache = make_cache(B, H, R, hd, kv, g, L)
    seqs, rows = (torch.from_numpy(rng.integers(0, n, T)).to(torch.int32).cuda() for n in (B, R))  # some twice
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    if T > 5:
        for i, (s, r) in enumerate([(-1, 0), (B, 1), (0, -5), (1, R), (2 ** 30, 2 ** 30)]):
            seqs[i], rows[i], bad[i] = s, r, True
    room = torch.full((2, L, T + 2, H, hd), 7.0, device="cuda", dtype=TYPES[xt])
    bq.read_kv(bq.KVView(*cache), seqs, rows, room[0, :, :T], room[1, :, :T])
    for i in (0, 1):
        x = cache[i].double()
        if kv == "q8":
            x = x * cache[2 + i].double().repeat_interleave(32, -1)
        want = x[seqs.clamp(0, B - 1).long(), :, :, rows.clamp(0, R - 1).long()].transpose(0, 1)
        want = torch.where(bad[:, None, None], 0, want).to(TYPES[xt])  # (a code times a scale is exact in fp32)
        assert torch.equal(room[i, :, :T], want)
        assert (room[i, :, T:] == 7).all()


def test_same_bits_as_a_models_cache():
    """Rows quantised as they are written are the ones that a model's own int8 cache holds."""
    cfg = synth.workload(0)
    H, hd, n = cfg["n_kv_heads"], cfg["head_dim"], 9
    x = torch.randn(2, n, H, hd, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    bits = x.view(torch.int16).numpy().view(np.uint16)
    with bq.Model(cfg, synth.make_weights(cfg), max_seq=16, flags=bq.LLM_KV_Q8) as m:
        m.kv_write(0, 1, 0, bits[0].copy(), bits[1].copy())
        k, ks, v, vs = m.kv_read_q8(0, 1, 0, n)
    cache = make_cache(1, H, 16, hd, "q8", gen(2))
    rows = torch.arange(n, dtype=torch.int32, device="cuda")
    bq.append_kv(x[0].cuda(), x[1].cuda(), bq.KVView(*cache), torch.zeros_like(rows), rows)
    for got, codes, scales in ((cache[0::2], k, ks), (cache[1::2], v, vs)):
        assert np.array_equal(got[0][0, :, :n].transpose(0, 1).cpu().numpy(), codes)
        assert np.array_equal(got[1][0, :, :n].transpose(0, 1).contiguous().cpu().numpy().view(np.uint16), scales)
