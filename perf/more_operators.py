"""Cases of the serving operators: queries, keys and values of new tokens into
the K/V cache (append_kv), cached rows back out of it (read_kv), attention of a
batch whose sequences share long prefixes (prefix_attention), and the next token
of every row of logits under its own options (sample_tokens).

A decoding step of a served batch runs them in this order: the layer's q, k and
v heads are normed, rotated and appended, every sequence attends to the prefix
that it shares and to its own rows, and the logits become tokens from given
uniform numbers. Cached rows are read back where a prefix is handed on.
"""
import math

import torch

own = False

EPS = 1e-5


def listed():
    return [
        # one token of the 22-layer Llama shape: fp32 activations, pairs (2i, 2i + 1), no norms
        dict(name="append-1-f32", op="append", T=1, Hq=32, Hkv=4, hd=64, x="f32", kv="bf16", norm=False, neox=False,
             B=1, far=300),
        # one token of each sequence of the 32-sequence serving batch, int8 cache, the rows read back
        dict(name="append-32-q8", op="append", T=32, Hq=16, Hkv=8, hd=128, x="f32", kv="q8", norm=True, neox=True,
             B=32, far=4096),
        # prompt tokens of several sequences at once, far positions
        dict(name="append-8192-norm", op="append", T=8192, Hq=16, Hkv=8, hd=128, x="bf16", kv="bf16", norm=True,
             neox=True, B=5, far=131072),
        # the rows of a short prefix, all layers
        dict(name="read-37-f32", op="read", T=37, L=22, Hkv=4, hd=64, cap=64, B=2, kv="bf16", x="f32"),
        # a long int8 prefix of 28 layers on its way to another cache
        dict(name="read-4099-q8", op="read", T=4099, L=28, Hkv=8, hd=128, cap=4099, B=1, kv="q8", x="bf16"),
        # two sequences behind one short system prompt, fp32 activations
        dict(name="prefix-2-257-f32", op="prefix", B=2, n=1, G=1, Hq=32, Hkv=4, hd=64, P=257, lo=3, hi=40, q="f32",
             kv="bf16"),
        # the 32-sequence serving batch behind a common prompt
        dict(name="prefix-32-2048", op="prefix", B=32, n=1, G=1, Hq=16, Hkv=8, hd=128, P=2048, lo=64, hi=512, q="bf16",
             kv="bf16"),
        # drafts of three nodes behind four prompts of different lengths, int8 rows
        dict(name="prefix-24x3-1531-q8", op="prefix", B=24, n=3, G=4, Hq=16, Hkv=8, hd=128, P=1531, lo=5, hi=700,
             q="bf16", kv="q8"),
        # many samples of one long document
        dict(name="prefix-256-16384", op="prefix", B=256, n=1, G=1, Hq=32, Hkv=4, hd=64, P=16384, lo=16, hi=300,
             q="bf16", kv="bf16"),
        # the next token of one chat, the sampler's usual options
        dict(name="sample-1-32000", op="sample", R=1, V=32000, sd=2.5, mix="chat"),
        # the serving batch, every request with options of its own
        dict(name="sample-32-151936", op="sample", R=32, V=151936, sd=2.5, mix="mixed"),
        # many samples, thresholds over the whole vocabulary
        dict(name="sample-256-151936", op="sample", R=256, V=151936, sd=2.5, mix="nucleus"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "prefix", "prefix", "prefix", "sample", "sample"])
    hd, Hkv, gq = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "append":
        while True:
            T = _log(rng, 1, 16384)
            if T * (Hkv * gq + 2 * Hkv) * hd <= 8192 * 32 * 128:
                break
        return dict(op=op, T=T, Hq=Hkv * gq, Hkv=Hkv, hd=hd, x=rng.choice(["bf16", "f32"]),
                    kv=rng.choice(["bf16", "q8"]), norm=rng.random() < 0.5, neox=rng.random() < 0.7,
                    B=_log(rng, 1, min(32, T)), far=_log(rng, 64, 1 << 20))
    if op == "read":
        while True:
            T, L = _log(rng, 1, 8192), _log(rng, 1, 28)
            if T * L * Hkv * hd <= 4099 * 28 * 8 * 128:
                break
        B = _log(rng, 1, 8)
        return dict(op=op, T=T, L=L, Hkv=Hkv, hd=hd, cap=_log(rng, (T + B - 1) // B, T), B=B,
                    kv=rng.choice(["bf16", "q8"]), x=rng.choice(["bf16", "f32"]))
    if op == "prefix":
        while True:
            B, n, P, hi = _log(rng, 1, 256), rng.choice([1, 1, 1, 2, 4, 7]), _log(rng, 1, 32768), _log(rng, 1, 2048)
            M = B * n * Hkv * gq
            if M * hd * (P + hi) <= 256 * 32 * 64 * 16684 and B * Hkv * hd * hi <= 1 << 26 and M * (P + hi) <= 1 << 27:
                break
        q = rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, B=B, n=n, G=_log(rng, 1, min(8, B)), Hq=Hkv * gq, Hkv=Hkv, hd=hd, P=P, lo=_log(rng, 1, hi),
                    hi=hi, q=q, kv=rng.choice(["bf16", "bf16", "q8"]))
    V = _log(rng, 2000, 160000)
    return dict(op=op, R=_log(rng, 1, 256 * 151936 // V if V > 151936 else 256), V=V, sd=round(rng.uniform(1.0, 4.0), 2),
                mix=rng.choice(["chat", "mixed", "nucleus", "plain"]))


def _lens(c):  # own rows of each sequence
    B = c["B"]
    return [c["lo"] + (c["hi"] - c["lo"]) * b // max(1, B - 1) if B > 1 else c["hi"] for b in range(B)]


def _groups(c):  # first sequence of each group (and the end), rows of its prefix
    B, G = c["B"], c["G"]
    starts = [min(b, B) for b in (round(B * (g / G) ** 1.3) for g in range(G))] + [B]
    return starts, [c["P"] - (c["P"] * g) // (2 * G) for g in range(G)]


def work(case):
    c = case
    if c["op"] == "append":
        size = 2 if c["x"] == "bf16" else 4
        row = 2 * c["hd"] if c["kv"] == "bf16" else c["hd"] + c["hd"] // 16
        n = c["T"] * (2 * c["Hq"] + 2 * c["Hkv"]) * c["hd"] * size + 2 * c["T"] * c["Hkv"] * row
        if c["kv"] == "q8":  # the rows read back
            n += 2 * c["T"] * c["Hkv"] * (row + 2 * c["hd"])
        return {"bytes": n, "flops": 10 * c["T"] * (c["Hq"] + 2 * c["Hkv"]) * c["hd"]}
    if c["op"] == "read":
        row = 2 * c["hd"] if c["kv"] == "bf16" else c["hd"] + c["hd"] // 16
        out = c["hd"] * (2 if c["x"] == "bf16" else 4)
        n = 2 * c["T"] * c["L"] * c["Hkv"]
        return {"bytes": n * (row + out) + 8 * c["T"], "flops": n * c["hd"]}
    if c["op"] == "prefix":
        starts, plens = _groups(c)
        row = c["hd"] * 2 if c["kv"] == "bf16" else c["hd"] + c["hd"] // 16
        keys = sum(_lens(c)) + c["B"] * c["n"]
        shared = sum(p for g, p in enumerate(plens) if starts[g + 1] > starts[g])
        pairs = sum((starts[g + 1] - starts[g]) * p for g, p in enumerate(plens)) + sum(_lens(c)) + c["B"] * (c["n"] + 1) // 2
        io = 2 * c["B"] * c["n"] * c["Hq"] * c["hd"] * (2 if c["q"] == "bf16" else 4)
        return {"bytes": 2 * c["Hkv"] * (keys + shared) * row + io, "flops": 4 * c["Hq"] * c["hd"] * c["n"] * pairs}
    return {"bytes": 4 * c["R"] * c["V"] + 28 * c["R"], "flops": 6 * c["R"] * c["V"]}


# ---- inputs ------------------------------------------------------------------
def _rows(shape, kv, g):
    """Cached rows as they are stored: bf16, or int8 codes with a half scale for every 32 values."""
    x = torch.randn(shape, device="cuda", generator=g)
    if kv == "bf16":
        return x.to(torch.bfloat16), None
    return _quantised(x)


def _quantised(x):
    shape = x.shape
    x = x.reshape(*shape[:-1], shape[-1] // 32, 32)
    s = (x.abs().amax(-1, keepdim=True) / 127).to(torch.float16)
    r = x / torch.where(s == 0, 1, s.float())
    codes = (r.abs() + 0.5).floor().clamp_max(127) * r.sign()  # halves away from zero
    return codes.to(torch.int8).view(shape), s.squeeze(-1)


def _options(c, g):
    R = c["R"]
    pick = lambda *v: torch.tensor(v, device="cuda")[torch.randint(len(v), (R,), device="cuda", generator=g)]  # noqa: E731
    if c["mix"] == "chat":
        T, k, p, m = pick(0.8), pick(40), pick(0.95), pick(0.0)
    elif c["mix"] == "nucleus":
        T, k, p, m = pick(0.7, 1.0), pick(0), pick(0.9, 0.95), pick(0.0, 0.02)
    elif c["mix"] == "plain":
        T, k, p, m = pick(1.0, 1.3), pick(0), pick(1.0), pick(0.0)
    else:  # every request its own, some greedy
        T, k, p, m = pick(0.0, 0.6, 0.8, 1.0, 1.5), pick(0, 1, 20, 50, 400), pick(0.5, 0.9, 0.95, 1.0), pick(0.0, 0.05, 0.1)
    return T.float(), k.to(torch.int32), p.float(), m.float()


def prepare(case, seed):
    c, g, h = case, torch.Generator("cuda"), torch.Generator()
    g.manual_seed(seed)
    h.manual_seed(seed)
    s = dict(case=c)
    kind = lambda k: torch.bfloat16 if k == "bf16" else torch.float32  # noqa: E731
    randn = lambda *shape: torch.randn(shape, device="cuda", generator=g)  # noqa: E731
    if c["op"] == "append":
        T, Hq, Hkv, hd, B = c["T"], c["Hq"], c["Hkv"], c["hd"], c["B"]
        qkv = randn(T, Hq + 2 * Hkv, hd).to(kind(c["x"]))  # one projection's output
        s["q"], s["k"], s["v"] = qkv.split([Hq, Hkv, Hkv], 1)
        s["q_out"] = torch.empty(T, Hq, hd, device="cuda", dtype=kind(c["x"]))
        each = (T + B - 1) // B
        cap = each + 8
        t = torch.arange(T)
        first = torch.randint(0, 8, (B,), generator=h)
        s["seqs"] = (t // each).to(torch.int32).cuda()
        s["rows"] = (first[t // each] + t % each).to(torch.int32).cuda()
        s["positions"] = (torch.randint(0, c["far"], (B,), generator=h)[t // each] + t % each).to(torch.int32).cuda()
        ks, vs = _rows((B, Hkv, cap, hd), c["kv"], g), _rows((B, Hkv, cap, hd), c["kv"], g)
        s["cache"] = (ks[0], vs[0], ks[1], vs[1])
        s["q_norm"], s["k_norm"] = (1 + 0.1 * randn(hd) if c["norm"] else None for _ in range(2))
        s["back"] = tuple(torch.empty(T, Hkv, hd, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    elif c["op"] == "read":
        T, L, Hkv, hd, B = c["T"], c["L"], c["Hkv"], c["hd"], c["B"]
        ks, vs = _rows((B, L, Hkv, c["cap"], hd), c["kv"], g), _rows((B, L, Hkv, c["cap"], hd), c["kv"], g)
        s["cache"] = (ks[0], vs[0], ks[1], vs[1])
        at = torch.randperm(B * c["cap"], generator=h)[:T].sort().values
        s["seqs"], s["rows"] = (at // c["cap"]).to(torch.int32).cuda(), (at % c["cap"]).to(torch.int32).cuda()
        s["back"] = tuple(torch.empty(L, T, Hkv, hd, device="cuda", dtype=kind(c["x"])) for _ in range(2))
    elif c["op"] == "prefix":
        B, n, Hq, Hkv, hd = c["B"], c["n"], c["Hq"], c["Hkv"], c["hd"]
        starts, plens = _groups(c)
        s["starts"] = torch.tensor(starts, dtype=torch.int32).cuda()
        s["prefix_lens"] = torch.tensor(plens, dtype=torch.int32).cuda()
        lens = torch.tensor(_lens(c), dtype=torch.int32)
        s["lens"] = lens[torch.randperm(B, generator=h)].cuda()
        for name, seqs, rows in (("prefix", c["G"], c["P"]), ("cache", B, c["hi"]), ("tree", B, n)):
            ks, vs = _rows((seqs, Hkv, rows, hd), c["kv"], g), _rows((seqs, Hkv, rows, hd), c["kv"], g)
            s[name] = (ks[0], vs[0], ks[1], vs[1])
        s["q"] = randn(B, n, Hq, hd).to(kind(c["q"]))
        # every new token sees itself and those before it: a chain
        s["mask"] = torch.tensor([(2 << j) - 1 for j in range(n)], device="cuda").repeat(B, 1)
        s["out"] = torch.empty_like(s["q"])
    else:
        s["logits"] = c["sd"] * randn(c["R"], c["V"])
        s["temperature"], s["top_k"], s["top_p"], s["min_p"] = _options(c, g)
        s["u"] = torch.rand(c["R"], device="cuda", generator=g)
        s["tokens"] = torch.empty(c["R"], dtype=torch.int32, device="cuda")
        s["probs"] = torch.empty(c["R"], device="cuda")
    if own:
        import bit_quantized_token_gb300 as bq

        for name in ("prefix", "cache", "tree"):
            if name in s:
                s[name + "_view"] = bq.KVView(*s[name])
        if c["op"] == "prefix":
            size = bq.prefix_workspace(s["q"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


# ---- one pass ----------------------------------------------------------------
def run(s):
    c, op = s["case"], s["case"]["op"]
    if own:
        import bit_quantized_token_gb300 as bq

        if op == "append":
            bq.append_kv(s["k"], s["v"], s["cache_view"], s["seqs"], s["rows"], q=s["q"], q_out=s["q_out"],
                         positions=s["positions"], rope_theta=10000.0, rope_neox=c["neox"], q_norm=s["q_norm"],
                         k_norm=s["k_norm"], eps=EPS)
            if c["kv"] == "bf16":
                return s["q_out"], s["cache"][0], s["cache"][1]
            bq.read_kv(s["cache_view"], s["seqs"], s["rows"], *s["back"])
            return s["q_out"], *s["back"]
        if op == "read":
            bq.read_kv(s["cache_view"], s["seqs"], s["rows"], *s["back"])
            return s["back"]
        if op == "prefix":
            bq.prefix_attention(s["q"], s["prefix_view"], s["starts"], s["prefix_lens"], s["cache_view"],
                                s["tree_view"], s["lens"], s["mask"], s["out"], s["workspace"])
            return s["out"]
        bq.sample_tokens(s["logits"], s["u"], s["tokens"], s["temperature"], s["top_k"], s["top_p"], s["min_p"],
                         probs=s["probs"])
        return s["tokens"], s["probs"]
    return {"append": _append, "read": _read, "prefix": _prefix, "sample": _sample}[op](s)


def _values(rows, scales):
    if scales is None:
        return rows.float()
    shape = rows.shape
    return (rows.view(*shape[:-1], shape[-1] // 32, 32).float() * scales.float()[..., None]).view(shape)


def _rotated(x, weight, positions, neox):
    """x [token, head, dim] in 32 bits: normed with its weight (or not), then rotated; the angles in 64 bits."""
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    half = x.shape[-1] // 2
    freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    angle = positions.double()[:, None, None] * freq
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    a, b = (x[..., :half], x[..., half:]) if neox else (x[..., 0::2], x[..., 1::2])
    a, b = a * cos - b * sin, a * sin + b * cos
    return torch.cat([a, b], -1) if neox else torch.stack([a, b], -1).flatten(-2)


def _append(s):
    c, at = s["case"], s["positions"]
    q = _rotated(s["q"].float(), s["q_norm"], at, c["neox"]).to(s["q"].dtype)
    k = _rotated(s["k"].float(), s["k_norm"], at, c["neox"])
    seqs, rows = s["seqs"].long(), s["rows"].long()
    if c["kv"] == "bf16":
        for x, cached in ((k, s["cache"][0]), (s["v"], s["cache"][1])):
            cached[seqs, :, rows] = x.to(torch.bfloat16)
        return q, s["cache"][0], s["cache"][1]
    back = []
    for x, cached, scales in ((k, s["cache"][0], s["cache"][2]), (s["v"].float(), s["cache"][1], s["cache"][3])):
        cached[seqs, :, rows], scales[seqs, :, rows] = _quantised(x)
        back.append(_values(cached[seqs, :, rows], scales[seqs, :, rows]).to(torch.bfloat16))
    return q, *back


def _read(s):
    seqs, rows, out = s["seqs"].long(), s["rows"].long(), []
    for i, back in enumerate(s["back"]):
        x, scales = s["cache"][i], s["cache"][2 + i]
        x = _values(x[seqs, :, :, rows], None if scales is None else scales[seqs, :, :, rows])
        out.append(x.transpose(0, 1).to(back.dtype, memory_format=torch.contiguous_format))
    return tuple(out)


def _prefix(s):
    q, c = s["q"], s["case"]
    B, n, Hq, hd = q.shape
    Hkv, G, P, hi = c["Hkv"], c["G"], c["P"], c["hi"]
    gq = Hq // Hkv
    starts, _ = _groups(c)
    most = max(starts[g + 1] - starts[g] for g in range(G))
    group = (torch.arange(B, device="cuda")[:, None] >= s["starts"][1:]).sum(-1).clamp_max(G - 1)
    place = torch.arange(B, device="cuda") - s["starts"][group]
    member = (s["starts"][:-1, None] + torch.arange(most, device="cuda")).clamp_max(B - 1)  # [G, most], the rest repeated
    x = q.float().view(B, n, Hkv, gq, hd).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * gq, hd) / math.sqrt(hd)
    pk, pv = (_values(s["prefix"][i], s["prefix"][2 + i]) for i in (0, 1))
    k, v = (torch.cat([_values(s["cache"][i], s["cache"][2 + i]), _values(s["tree"][i], s["tree"][2 + i])], 2)
            for i in (0, 1))
    xg = x[member].transpose(1, 2).reshape(G, Hkv, most * n * gq, hd)
    zp = (xg @ pk.transpose(-1, -2)).view(G, Hkv, most, n * gq, P)
    seen = torch.arange(P, device="cuda") < s["prefix_lens"][:, None]
    zp = torch.where(seen[:, None, None, None], zp, -math.inf).transpose(1, 2)[group, place]  # [B, Hkv, n gq, P]
    in_cache = torch.arange(hi, device="cuda") < s["lens"][:, None]
    in_tree = (s["mask"][:, :, None] >> torch.arange(n, device="cuda")) & 1
    sees = torch.cat([in_cache[:, None].expand(B, n, hi), in_tree.bool()], -1)
    zo = (x @ k.transpose(-1, -2)).view(B, Hkv, n, gq, hi + n)
    zo = torch.where(sees[:, None, :, None], zo, -math.inf).view(B, Hkv, n * gq, hi + n)
    top = torch.maximum(zp.amax(-1, keepdim=True), zo.amax(-1, keepdim=True)).clamp_min(-3e38)
    ep, eo = torch.exp(zp - top), torch.exp(zo - top)
    eg = ep[member].transpose(1, 2).reshape(G, Hkv, most * n * gq, P)
    op = (eg @ pv).view(G, Hkv, most, n * gq, hd).transpose(1, 2)[group, place]
    o = (op + eo @ v) / (ep.sum(-1, keepdim=True) + eo.sum(-1, keepdim=True))
    return o.view(B, Hkv, n, gq, hd).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, hd).to(q.dtype)


def _sample(s):
    x = s["logits"]
    R, V = x.shape
    order = x.sort(dim=-1, descending=True, stable=True)
    z = order.values.double()
    at = torch.arange(V, device="cuda")
    greedy = s["temperature"][:, None] == 0
    w = torch.exp((z - z[:, :1]) / torch.where(greedy, 1, s["temperature"].double()[:, None]))
    k = torch.where(s["top_k"] == 0, V, s["top_k"])[:, None]
    w = torch.where((at < k) & (~greedy | (at == 0)), w, 0)
    cum = w.cumsum(-1)
    p = s["top_p"].double()[:, None]
    w = torch.where(((cum - w < p * cum[:, -1:]) | (p >= 1)) & (w >= s["min_p"].double()[:, None]), w, 0)
    cum = w.cumsum(-1)
    pick = (cum <= s["u"].double()[:, None] * cum[:, -1:]).sum(-1, keepdim=True)
    pick = torch.minimum(pick, (w > 0).sum(-1, keepdim=True) - 1)
    return order.indices.gather(-1, pick)[:, 0].to(torch.int32), (w.gather(-1, pick) / cum[:, -1:])[:, 0].float()


# ---- the same in 64 bits, from the definitions ---------------------------------
def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "append":
        T, hd = c["T"], c["hd"]
        pair = torch.arange(hd // 2, device="cuda")
        i, j = (pair, pair + hd // 2) if c["neox"] else (2 * pair, 2 * pair + 1)
        theta = s["positions"].double()[:, None] * torch.pow(torch.tensor(10000.0, dtype=torch.float64, device="cuda"),
                                                             -2.0 * pair.double() / hd)
        turn = torch.polar(torch.ones_like(theta), theta)[:, None]

        def heads(x, weight):
            x = x.double()
            if weight is not None:
                x = x * torch.rsqrt(x.square().sum(-1, keepdim=True) / hd + EPS) * weight.double()
            z = torch.complex(x[..., i], x[..., j]) * turn
            out = torch.empty_like(x)
            out[..., i], out[..., j] = z.real, z.imag
            return out

        q, k, v = heads(s["q"], s["q_norm"]), heads(s["k"], s["k_norm"]), s["v"].double()
        if c["kv"] == "bf16":
            out = [s["cache"][0].double(), s["cache"][1].double()]
            for b in range(c["B"]):
                mine = s["seqs"] == b
                for m, x in enumerate((k, v)):
                    out[m][b].transpose(0, 1)[s["rows"][mine].long()] = x[mine]
            return q, *out

        def stood_for(x):
            x = x.view(T, c["Hkv"], hd // 32, 32)
            scale = (x.abs().amax(-1, keepdim=True) / 127).to(torch.float16).double()
            code = torch.copysign((x.abs() / scale.clamp_min(1e-30) + 0.5).floor().clamp(max=127), x)
            return (code * scale).reshape(T, c["Hkv"], hd)

        return q, stood_for(k), stood_for(v)
    if c["op"] == "read":
        out = []
        for m in (0, 1):
            x = s["cache"][m].double()
            if c["kv"] == "q8":
                x = x * s["cache"][2 + m].double().repeat_interleave(32, -1)
            flat = x.permute(1, 0, 3, 2, 4).reshape(c["L"], c["B"] * c["cap"], c["Hkv"], c["hd"])
            out.append(flat[:, s["seqs"].long() * c["cap"] + s["rows"].long()])
        return tuple(out)
    if c["op"] == "prefix":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        gq, (starts, plens) = c["Hq"] // c["Hkv"], _groups(c)
        wide = {}
        for name in ("prefix", "cache", "tree"):
            for m in (0, 1):
                x = s[name][m].double()
                if c["kv"] == "q8":
                    x = x * s[name][2 + m].double().repeat_interleave(32, -1)
                wide[name, m] = x
        lens = s["lens"].tolist()
        for g in range(c["G"]):
            for b in range(starts[g], starts[g + 1]):
                k, v = (torch.cat([wide["prefix", m][g, :, :plens[g]], wide["cache", m][b, :, :lens[b]],
                                   wide["tree", m][b]], 1) for m in (0, 1))
                vis = torch.ones(c["n"], k.shape[1], dtype=torch.bool, device="cuda")
                vis[:, k.shape[1] - c["n"]:] = torch.ones(c["n"], c["n"], device="cuda").tril().bool()
                z = torch.einsum("nhgd,hkd->nhgk", s["q"][b].double().view(c["n"], c["Hkv"], gq, c["hd"]), k)
                z = (z / math.sqrt(c["hd"])).masked_fill(~vis[:, None, None], -math.inf)
                w = torch.exp(z - torch.logsumexp(z, -1, keepdim=True))
                out[b] = torch.einsum("nhgk,hkd->nhgd", w, v).reshape(c["n"], c["Hq"], c["hd"])
        return out
    import numpy as np

    x = s["logits"].cpu().numpy().astype(np.float64)
    T, k, p, m, u = (s[name].cpu().numpy().astype(np.float64) for name in ("temperature", "top_k", "top_p", "min_p", "u"))
    tokens, probs = np.empty(c["R"], np.int32), np.empty(c["R"])
    for r in range(c["R"]):
        if T[r] == 0:
            tokens[r], probs[r] = int(x[r].argmax()), 1.0
            continue
        ids = np.argsort(-x[r], kind="stable")
        if k[r]:
            ids = ids[:int(k[r])]
        w = np.exp((x[r][ids] - x[r].max()) / T[r])
        if p[r] < 1:
            w = w[:int(np.searchsorted(np.cumsum(w), p[r] * math.fsum(w))) + 1]
        w = w[:int((w >= m[r]).sum())]
        cum = np.cumsum(w)
        n = min(int(np.searchsorted(cum, u[r] * cum[-1], side="right")), len(w) - 1)
        tokens[r], probs[r] = ids[n], w[n] / cum[-1]
    return torch.from_numpy(tokens).cuda(), torch.from_numpy(probs).cuda()
