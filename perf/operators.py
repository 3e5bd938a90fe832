"""Cases of the tree-decoding operators: attention of drafted tokens over the K/V
cache, token probabilities under the sampling options, verification of the
drafts against them, and the commit of the accepted rows into the cache.

A decoding step with drafts runs all four: the target model scores a tree of
drafted tokens in one pass (tree_attention per layer), its logits become
probabilities (token_probs), given uniforms decide which drafts are kept
(verify_tree), and the kept nodes' keys and values move from the tree's buffer
into the cache (commit_tree).
"""
import math

import torch

own = False

HEADS = {"gqa8-64": (32, 4, 64), "gqa2-128": (16, 8, 128), "gqa2-64": (4, 2, 64)}


def listed():
    return [
        # one token against a short cache: the step of a chat turn's first answer tokens
        dict(name="attend-1x1-256", op="attend", B=1, n=1, Hq=32, Hkv=4, hd=64, lo=256, hi=256, q="bf16", kv="bf16"),
        # a drafted tree of one sequence at the long-context workload's cache, fp32 activations as in the model's own step
        dict(name="attend-1x16-4097-f32", op="attend", B=1, n=16, Hq=32, Hkv=4, hd=64, lo=4097, hi=4097, q="f32",
             kv="bf16"),
        # the 32-sequence serving batch, a small tree for each sequence
        dict(name="attend-32x8-2048", op="attend", B=32, n=8, Hq=16, Hkv=8, hd=128, lo=512, hi=2048, q="bf16",
             kv="bf16"),
        # int8 cache, odd node count and lengths
        dict(name="attend-8x13-4099-q8", op="attend", B=8, n=13, Hq=16, Hkv=8, hd=128, lo=301, hi=4099, q="bf16",
             kv="q8"),
        # the widest trees over long ragged caches
        dict(name="attend-16x64-8192", op="attend", B=16, n=64, Hq=32, Hkv=4, hd=64, lo=1024, hi=8192, q="bf16",
             kv="bf16"),
        # one row of logits of a 32000-token vocabulary, the sampler's usual options
        dict(name="probs-1x32000-k40", op="probs", R=1, V=32000, T=0.8, k=40, p=0.95),
        # every node of the serving batch's trees, plain softmax over the largest vocabulary
        dict(name="probs-256x151936", op="probs", R=256, V=151936, T=1.0, k=0, p=1.0),
        # one sequence, four drafts in a chain with their own probabilities
        dict(name="verify-1x5-chain", op="verify", B=1, n=5, V=32000, tree=False),
        # the serving batch, chains of seven drafts
        dict(name="verify-32x8-chain", op="verify", B=32, n=8, V=151936, tree=False),
        # the serving batch, trees of top candidates (no draft probabilities)
        dict(name="verify-32x16-tree", op="verify", B=32, n=16, V=151936, tree=True),
        # three accepted nodes of one sequence into the cache of 22 layers
        dict(name="commit-1x5", op="commit", B=1, L=22, n=5, kept=3, Hkv=4, hd=64, cap=2048),
        # the serving batch, 28 layers
        dict(name="commit-32x16", op="commit", B=32, L=28, n=16, kept=9, Hkv=8, hd=128, cap=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "probs", "verify", "verify", "commit"])
    if op == "attend":
        while True:
            hd, Hkv, gq = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8])
            B, n, hi = _log(rng, 1, 32), _log(rng, 1, 64), _log(rng, 1, 16384)
            if B * n * Hkv * gq * hd * hi <= 16 * 64 * 32 * 64 * 4608:
                break
        return dict(op=op, B=B, n=n, Hq=Hkv * gq, Hkv=Hkv, hd=hd, lo=_log(rng, 1, hi), hi=hi,
                    q=rng.choice(["bf16", "f32"]), kv=rng.choice(["bf16", "bf16", "q8"]))
    if op == "probs":
        V = _log(rng, 2000, 160000)
        return dict(op=op, R=_log(rng, 1, 256 * 151936 // V if V > 151936 else 256), V=V,
                    T=round(rng.uniform(0.3, 1.5), 3), **rng.choice([dict(k=0, p=1.0), dict(k=rng.randint(1, 64), p=1.0),
                                                                   dict(k=rng.randint(2, 64), p=round(rng.uniform(0.3, 0.99), 3))]))
    if op == "verify":
        return dict(op=op, B=_log(rng, 1, 32), n=_log(rng, 2, 16), V=_log(rng, 2000, 160000),
                    tree=rng.random() < 0.5)
    n = _log(rng, 1, 64)
    B, L, Hkv, hd = _log(rng, 1, 32), _log(rng, 1, 28), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    return dict(op=op, B=B, L=L, n=n, kept=_log(rng, 1, n), Hkv=Hkv, hd=hd, cap=n + _log(rng, 1, 64))


def _lens(c):
    B = c["B"]
    return [c["lo"] + (c["hi"] - c["lo"]) * b // max(1, B - 1) if B > 1 else c["hi"] for b in range(B)]


def work(case):
    c = case
    if c["op"] == "attend":
        keys = sum(_lens(c)) + c["B"] * c["n"]
        row = c["hd"] * 2 if c["kv"] == "bf16" else c["hd"] + c["hd"] // 16
        io = 2 * c["B"] * c["n"] * c["Hq"] * c["hd"] * (2 if c["q"] == "bf16" else 4)
        # every node sees the whole cache; the tree's own columns count half
        return {"bytes": 2 * c["Hkv"] * keys * row + io + 12 * c["B"] * c["n"],
                "flops": 4 * c["Hq"] * c["hd"] * c["n"] * (sum(_lens(c)) + c["B"] * c["n"] // 2)}
    if c["op"] == "probs":
        return {"bytes": 8 * c["R"] * c["V"], "flops": 5 * c["R"] * c["V"]}
    if c["op"] == "verify":  # the row that the last token is drawn from: its probabilities, for chains the drafts' too
        rows = 1 if c["tree"] else 2
        return {"bytes": c["B"] * (4 * rows * c["V"] + 28 * c["n"]), "flops": 2 * rows * c["B"] * c["V"]}
    return {"bytes": 8 * c["B"] * c["L"] * c["kept"] * c["Hkv"] * c["hd"] + 4 * c["B"] * (c["n"] + 3),
            "flops": 0}


# ---- inputs ------------------------------------------------------------------
def _tree(g, B, n, chain):
    """parents [B, n] (node 0 is the root) and, bit by bit, which nodes every node sees."""
    par = torch.zeros(B, n, dtype=torch.int64)
    for i in range(1, n):
        par[:, i] = i - 1 if chain else torch.randint(max(0, i - 6), i, (B,), generator=g)
    sees = torch.zeros(B, n, n, dtype=torch.bool)
    rows = torch.arange(B)
    for i in range(n):
        if i:
            sees[:, i] = sees[rows, par[:, i]]
        sees[:, i, i] = True
    par[:, 0] = -1
    weight = torch.tensor([1 << i if i < 63 else -(1 << 63) for i in range(n)], dtype=torch.int64)
    return par.to(torch.int32).cuda(), (sees * weight).sum(-1).cuda()


def _rows(shape, kv, g):
    """Cached rows as they are stored: bf16, or int8 codes with a half scale for every 32 values."""
    x = torch.randn(shape, device="cuda", generator=g)
    if kv == "bf16":
        return x.to(torch.bfloat16), None
    x = x.view(*shape[:-1], shape[-1] // 32, 32)
    s = (x.abs().amax(-1, keepdim=True) / 127).to(torch.float16)
    codes = (x / s.float()).round().clamp(-127, 127).to(torch.int8)
    return codes.view(shape), s.squeeze(-1)


def prepare(case, seed):
    c, g, h = case, torch.Generator("cuda"), torch.Generator()
    g.manual_seed(seed)
    h.manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "attend":
        B, n, Hq, Hkv, hd = c["B"], c["n"], c["Hq"], c["Hkv"], c["hd"]
        cap = c["hi"] + n
        s["parents"], s["mask"] = _tree(h, B, n, False)
        lens = torch.tensor(_lens(c), dtype=torch.int32)
        s["lens"] = lens[torch.randperm(B, generator=h)].cuda()
        for name, rows in (("cache", cap), ("tree", n)):
            k, ks = _rows((B, Hkv, rows, hd), c["kv"], g)
            v, vs = _rows((B, Hkv, rows, hd), c["kv"], g)
            s[name] = (k, v, ks, vs)
        s["q"] = torch.randn(B, n, Hq, hd, device="cuda", generator=g).to(
            torch.bfloat16 if c["q"] == "bf16" else torch.float32)
        s["out"] = torch.empty_like(s["q"])
    elif c["op"] == "probs":
        s["logits"] = 2.5 * torch.randn(c["R"], c["V"], device="cuda", generator=g)
        s["out"] = torch.empty_like(s["logits"])
    elif c["op"] == "verify":
        B, n, V = c["B"], c["n"], c["V"]
        s["parents"], s["mask"] = _tree(h, B, n, not c["tree"])
        p = torch.randn(B, n, V, device="cuda", generator=g).mul_(3.0)
        q = None
        if not c["tree"]:  # the draft model's logits: the target's with an error
            q = torch.softmax(p + 0.7 * torch.randn(B, n, V, device="cuda", generator=g), -1)
        s["probs"] = torch.softmax(p, -1)
        tokens = torch.zeros(B, n, dtype=torch.int64, device="cuda")
        if c["tree"]:  # every node's children are its most likely tokens, best first
            best = p.topk(min(V, n), -1).indices
            for i in range(1, n):
                rank = (s["parents"][:, 1:i] == s["parents"][:, i:i + 1]).sum(-1)
                tokens[:, i] = best[torch.arange(B, device="cuda"), s["parents"][:, i].long(), rank]
        else:
            tokens[:, 1:] = torch.multinomial(q.view(B * n, V), 1, generator=g).view(B, n)[:, :-1]
        s["tokens"] = tokens.to(torch.int32)
        s["draft"] = q
        s["u"] = torch.rand(B, n, device="cuda", generator=g)
        s["path"] = torch.empty(B, n, dtype=torch.int32, device="cuda")
        s["n_path"], s["next"] = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
    else:
        B, L, n, kept, Hkv, hd = c["B"], c["L"], c["n"], c["kept"], c["Hkv"], c["hd"]
        for name, rows in (("cache", c["cap"]), ("tree", n)):
            s[name] = tuple(torch.randn(B, L, Hkv, rows, hd, device="cuda", generator=g).to(torch.bfloat16)
                            for _ in range(2)) + (None, None)
        s["lens"] = torch.randint(0, c["cap"] - n + 1, (B,), generator=h).to(torch.int32).cuda()
        path = torch.full((B, n), -1, dtype=torch.int32)
        for b in range(B):
            path[b, :kept] = torch.cat([torch.zeros(1, dtype=torch.int64),
                                        torch.randperm(n - 1, generator=h)[:kept - 1].sort().values + 1])
        s["path"] = path.cuda()
        s["n_path"] = torch.full((B,), kept, dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.empty(B, dtype=torch.int32, device="cuda")
    if own:
        import bit_quantized_token_gb300 as bq

        for name in ("cache", "tree"):
            if name in s:
                s[name + "_view"] = bq.KVView(*s[name])
    return s


# ---- one pass ----------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        import bit_quantized_token_gb300 as bq

        c = s["case"]
        if op == "attend":
            bq.tree_attention(s["q"], s["cache_view"], s["tree_view"], s["lens"], s["mask"], s["out"])
            return s["out"]
        if op == "probs":
            bq.token_probs(s["logits"], s["out"], c["T"], c["k"], c["p"])
            return s["out"]
        if op == "verify":
            bq.verify_tree(s["tokens"], s["parents"], s["u"], s["probs"], s["path"], s["n_path"], s["next"],
                           draft_probs=s["draft"])
            return s["path"], s["n_path"], s["next"]
        bq.commit_tree(s["cache_view"], s["tree_view"], s["lens"], s["path"], s["n_path"], s["new_lens"])
        return s["cache"][0], s["cache"][1], s["new_lens"]
    return {"attend": _attend, "probs": _probs, "verify": _verify, "commit": _commit}[op](s)


def _values(rows, scales):
    if scales is None:
        return rows.float()
    shape = rows.shape
    return (rows.view(*shape[:-1], shape[-1] // 32, 32).float() * scales.float()[..., None]).view(shape)


def _attend(s):
    q, c = s["q"], s["case"]
    B, n, Hq, hd = q.shape
    Hkv, hi = c["Hkv"], c["hi"]
    k, v = (torch.cat([_values(s["cache"][i][:, :, :hi], None if s["cache"][2 + i] is None else s["cache"][2 + i][:, :, :hi]),
                       _values(s["tree"][i], s["tree"][2 + i])], 2) for i in (0, 1))
    in_cache = torch.arange(hi, device="cuda") < s["lens"][:, None]
    in_tree = (s["mask"][:, :, None] >> torch.arange(n, device="cuda")) & 1
    sees = torch.cat([in_cache[:, None].expand(B, n, hi), in_tree.bool()], -1)[:, None, None]
    x = q.float().view(B, n, Hkv, Hq // Hkv, hd).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, hd)
    score = (x @ k.transpose(-1, -2) / math.sqrt(hd)).view(B, Hkv, Hq // Hkv, n, hi + n)
    score = torch.where(sees, score, -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(-3e38)
    e = torch.exp(score - top)
    o = e.view(B, Hkv, -1, hi + n) @ v
    o = o / e.sum(-1).view(B, Hkv, -1, 1).clamp_min(1e-38)
    o = o.view(B, Hkv, Hq // Hkv, n, hd).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, hd)
    return o.to(q.dtype)


def _probs(s):
    x, c = s["logits"], s["case"]
    R, V = x.shape
    e = torch.exp((x - x.amax(-1, keepdim=True)) / c["T"])
    if c["k"] == 0:
        return e / e.sum(-1, keepdim=True)
    k = min(c["k"], V)
    least = x.topk(k, -1).values[:, -1:]
    above, same = x > least, x == least
    keep = above | (same & (same.cumsum(-1) <= k - above.sum(-1, keepdim=True)))
    ids = torch.where(keep, torch.arange(V, device="cuda"), V).topk(k, -1, largest=False, sorted=True).values
    order = x.gather(-1, ids).sort(dim=-1, descending=True, stable=True).indices
    ids = ids.gather(-1, order)
    w = e.gather(-1, ids).double()
    w = w / w.sum(-1, keepdim=True)
    w = torch.where(w.cumsum(-1) - w < c["p"], w, 0)
    return torch.zeros_like(x).scatter_(-1, ids, (w / w.sum(-1, keepdim=True)).float())


def _verify(s):
    tok, par, p, u = s["tokens"].long(), s["parents"].long(), s["probs"], s["u"].double()
    B, n, V = p.shape
    up, at = par.clamp_min(0), torch.arange(n, device="cuda")
    rows = torch.arange(B, device="cuda")[:, None]
    px = p[rows, up, tok].double()
    if s["draft"] is not None:  # a chain: every draft against its own probability
        taken = u * s["draft"][rows, up, tok].double() < px
        taken = taken.index_fill(1, at[:1], True)
        on_path = taken.long().cumprod(-1).bool()
    else:  # best candidates: each against what its earlier siblings left
        earlier = (par[:, :, None] == par[:, None, :]) & (at[:, None] > at)
        left = 1 - (earlier * px[:, None, :]).sum(-1)
        taken = (u * left < px).index_fill(1, at[:1], True)
        first = taken & ~(earlier & taken[:, None, :]).any(-1)
        sees = ((s["mask"][:, :, None] >> at) & 1).bool()
        on_path = (first[:, None, :] | ~sees).all(-1)
    last = torch.where(on_path, at, -1).amax(-1)
    r = p[rows[:, 0], last].double()
    child = par == last[:, None]
    if s["draft"] is not None:
        rest = (r - s["draft"][rows[:, 0], last].double()).clamp_min(0)
        r = torch.where(child.any(-1, keepdim=True) & (rest.sum(-1, keepdim=True) > 0), rest, r)
    else:
        hit = torch.zeros(B, V + 1, device="cuda").scatter_(1, torch.where(child, tok, V), 1.0)[:, :V]
        r = torch.where(hit > 0, 0, r)
    cum = r.cumsum(-1)
    nxt = (cum <= u[:, :1] * cum[:, -1:]).sum(-1).clamp_max(V - 1)
    length = on_path.sum(-1)
    order = torch.where(on_path, at, n).sort(-1).values
    path = torch.where(at < length[:, None], order, -1)
    return path.to(torch.int32), length.to(torch.int32), nxt.to(torch.int32)


def _commit(s):
    B, n = s["path"].shape
    steps = torch.arange(n, device="cuda")
    to = s["lens"].long()[:, None] + steps
    valid = steps < s["n_path"][:, None]
    b = torch.arange(B, device="cuda")[:, None]
    for cache, tree in zip(s["cache"][:2], s["tree"][:2]):
        at = to.clamp_max(cache.shape[3] - 1)
        kept = tree[b, :, :, s["path"].long().clamp_min(0)]
        cache[b, :, :, at] = torch.where(valid[:, :, None, None, None], kept, cache[b, :, :, at])
    s["new_lens"].copy_(s["lens"] + s["n_path"])
    return s["cache"][0], s["cache"][1], s["new_lens"]


# ---- the same in 64 bits, from the definitions ---------------------------------
def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "attend":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        gq = c["Hq"] // c["Hkv"]
        for b in range(c["B"]):
            n_old = int(s["lens"][b])
            vis = torch.ones(c["n"], n_old + c["n"], dtype=torch.bool, device="cuda")
            for j in range(c["n"]):
                vis[:, n_old + j] = (s["mask"][b] >> j) & 1 == 1
            for head in range(c["Hkv"]):
                kv = []
                for i in (0, 1):
                    parts = []
                    for name, m in (("cache", n_old), ("tree", c["n"])):
                        x = s[name][i][b, head, :m].double()
                        if s[name][2 + i] is not None:
                            x = x * s[name][2 + i][b, head, :m].double().repeat_interleave(32, -1)
                        parts.append(x)
                    kv.append(torch.cat(parts))
                for j in range(gq):
                    z = s["q"][b, :, head * gq + j].double() @ kv[0].T / math.sqrt(c["hd"])
                    z = z.masked_fill(~vis, -math.inf)
                    w = torch.exp(z - torch.logsumexp(z, -1, keepdim=True))
                    out[b, :, head * gq + j] = w @ kv[1]
        return out
    if c["op"] == "probs":
        out = torch.empty(s["logits"].shape, dtype=torch.float64, device="cuda")
        for r in range(c["R"]):
            w = torch.exp((s["logits"][r].double() - s["logits"][r].double().max()) / c["T"])
            if c["k"] == 0:
                out[r] = w / w.sum()
                continue
            w, ids = w.sort(dim=-1, descending=True, stable=True)
            w, ids = w[:c["k"]] / w[:c["k"]].sum(), ids[:c["k"]]
            cum, keep = 0.0, 0
            for x in w.tolist():
                if cum >= c["p"]:
                    break
                cum, keep = cum + x, keep + 1
            out[r] = 0
            out[r, ids[:keep]] = w[:keep] / w[:keep].sum()
        return out
    if c["op"] == "verify":
        B, n, V = c["B"], c["n"], c["V"]
        par, tok, u = s["parents"].tolist(), s["tokens"].tolist(), s["u"].double().tolist()
        path = torch.full((B, n), -1, dtype=torch.int32)
        count, nxt = torch.zeros(B, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
        for b in range(B):
            cur, seen, r, mass = 0, [0], s["probs"][b, 0].double(), 1.0
            for i in range(1, n):
                if par[b][i] != cur:
                    continue
                x = tok[b][i]
                qx = 1.0 if s["draft"] is None else s["draft"][b, cur, x].item()
                if u[b][i] * qx < r[x].item() / mass:
                    cur, r, mass = i, s["probs"][b, i].double(), 1.0
                    seen.append(i)
                elif s["draft"] is None:
                    mass, r = mass - r[x].item(), r.clone()
                    r[x] = 0
                else:
                    rest = (r / mass - s["draft"][b, cur].double()).clamp_min(0)
                    if rest.sum() > 0:
                        r, mass = rest, rest.sum().item()
            path[b, :len(seen)] = torch.tensor(seen, dtype=torch.int32)
            count[b] = len(seen)
            cum = r.cumsum(0)
            nxt[b] = int(torch.searchsorted(cum, (u[b][0] * cum[-1]).reshape(1), right=True)[0].clamp_max(V - 1))
        return path.cuda(), count.cuda(), nxt.cuda()
    for b in range(c["B"]):
        at = int(s["lens"][b])
        for j, node in enumerate(s["path"][b, :c["kept"]].tolist()):
            for i in (0, 1):
                s["cache"][i][b, :, :, at + j] = s["tree"][i][b, :, :, node]
    return s["cache"][0].double(), s["cache"][1].double(), s["lens"] + s["n_path"]
