"""Cases of the operators around the paged 8-bit cache: norm and rotation of
queries and keys, attention over a sliding window with sinks, attention of a
tree of drafted tokens, and log probabilities of tokens with entropy and top
alternatives.

With `own` false, run() computes each operator in its plain form (elementary
torch operations in fp32, angles in fp64); with `own` true it makes the
library's calls. exact() is the definition in 64 bits."""
import math
import random

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
TREE = 64   # new tokens of a sequence that can branch


def listed():
    return [
        # one decoded token: latency counts
        dict(name="rotate 1 token", op="rotate", T=1, heads=32, kv=8, dim=128, rot=128, pairs="halves", norm=True,
             far=131072, dt="bf16"),
        # a step of a speculating batch, odd sizes: neighbours turn together, half of each head, no norm
        dict(name="rotate odd batch", op="rotate", T=777, heads=12, kv=3, dim=64, rot=32, pairs="neighbours", norm=False,
             far=8192, dt="f16"),
        # a prefill batch behind a fused projection: memory counts
        dict(name="rotate prefill", op="rotate", T=8192, heads=32, kv=8, dim=128, rot=128, pairs="halves", norm=True,
             far=131072, dt="bf16"),
        # one chat of a window model: a single token sees a few hundred of its thousands
        dict(name="window short", op="window", S=1, new=1, ctx=5003, heads=8, group=4, dim=128, page=16, window=500,
             sinks=4, dt="f16"),
        # a serving batch of ragged contexts, some slots idle
        dict(name="window batch", op="window", S=48, new=1, ctx=32768, heads=8, group=4, dim=128, page=32, window=4096,
             sinks=4, dt="bf16"),
        # chunks of prompts behind earlier context
        dict(name="window prompts", op="window", S=4, new=2048, ctx=8000, heads=8, group=4, dim=128, page=32, window=1024,
             sinks=16, dt="bf16"),
        # one chat, a small tree of drafts: latency counts
        dict(name="tree small", op="tree", S=1, new=11, ctx=1200, heads=8, group=4, dim=128, page=16, dt="f16"),
        # a serving batch that verifies drafts
        dict(name="tree batch", op="tree", S=16, new=26, ctx=8192, heads=8, group=4, dim=128, page=32, dt="bf16"),
        # one long document, the widest tree: the context has to be split over the chip
        dict(name="tree long", op="tree", S=1, new=64, ctx=131071, heads=8, group=8, dim=128, page=64, dt="bf16"),
        # the sampled token of one chat, with its alternatives
        dict(name="logprobs 1 row", op="logprobs", M=1, V=131071, top=20, dt="f32"),
        # a batch of drafted tokens to verify, an odd vocabulary, some of it masked by a grammar
        dict(name="logprobs batch", op="logprobs", M=200, V=50001, top=5, dt="f16"),
        # a scored prompt
        dict(name="logprobs prompt", op="logprobs", M=2048, V=128000, top=20, dt="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "window", "window", "tree", "tree", "logprobs"])
    dt = rng.choice(["f16", "bf16"])
    if op == "rotate":
        dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 3, 4, 8])
        return dict(op=op, T=min(_log(rng, 1, 8192), 2 ** 25 // ((heads + kv) * dim)), heads=heads, kv=kv, dim=dim,
                    rot=rng.choice([dim, dim, 16 * rng.randint(1, dim // 16)]), pairs=rng.choice(["halves", "neighbours"]),
                    norm=rng.random() < 0.6, far=_log(rng, 64, 2 ** 20), dt=dt)
    if op == "logprobs":
        M = _log(rng, 1, 2048)
        return dict(op=op, M=M, V=_log(rng, 100, min(262144, 2 ** 27 // M)), top=rng.choice([0, 1, 5, 20, rng.randint(2, 64)]),
                    dt=rng.choice(["f16", "bf16", "f32"]))
    dim, page, heads = rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 64]), rng.choice([1, 2, 4, 8, 8])
    group = rng.choice([1, 2, 3, 4, 8, 16])
    if op == "tree":
        S, new = _log(rng, 1, 32), rng.choice([_log(rng, 2, TREE), _log(rng, 2, TREE), rng.randint(TREE + 1, 200)])
        ctx = new + _log(rng, 1, min(131072, 2 ** 20 // (S * heads), 2 ** 35 // (S * heads * group * dim * new)))
        return dict(op=op, S=S, new=new, ctx=ctx, heads=heads, group=group, dim=dim, page=page, dt=dt)
    window, sinks = _log(rng, 1, 8192), rng.choice([0, 4, _log(rng, 1, 256)])
    if rng.random() < 0.6:  # decoding, now and then a few speculated tokens
        S, new = _log(rng, 1, 64), rng.choice([1, 1, 1, rng.randint(2, 8)])
        ctx = new + _log(rng, 1, min(131072, 2 ** 22 // (S * heads)))
    else:
        S, new = _log(rng, 1, 8), _log(rng, 9, 2048)
        ctx = new + _log(rng, 1, 6000)
        group = max(1, min(group, 2 ** 28 // (S * new * min(ctx, window + new))))
        heads = max(1, min(heads, 32 // group, 2 ** 28 // (S * new * group * min(ctx, window + new))))
    return dict(op=op, S=S, new=new, ctx=ctx, heads=heads, group=group, dim=dim, page=page, window=window, sinks=sinks, dt=dt)


# ------------------------------------------------------------------- inputs


def _lengths(r, S, hi, lo):
    """S ragged lengths in [lo, hi]; the first one is hi. They are the case's, so that every seed has the same shapes."""
    return [hi] + [r.randint(lo, hi) for _ in range(S - 1)]


def _plan(case):
    """New tokens and lengths of every sequence, and for a tree each new token's parent."""
    S, new, ctx = case["S"], case["new"], case["ctx"]
    r = random.Random(S * 1000003 + ctx)
    n = _lengths(r, S, new, max(1, new // 2))
    before = _lengths(r, S, ctx - new, (ctx - new) // 8)
    lens = [a + b for a, b in zip(before, n)]
    if S > 8:
        lens[1::16] = [0] * len(lens[1::16])  # idle slots: no key is seen
    parents = []
    if case["op"] == "tree":
        for m in n:
            b = max(0, m - TREE)
            # a chain, then drafts: most continue one of the last few, some branch off earlier, a few start anew
            parents.append([i - 1 if i <= b else -1 if r.random() < 0.05 else
                            r.randint(max(b, i - 4), i - 1) if r.random() < 0.7 else r.randint(b, i - 1) for i in range(m)])
            parents[-1][b:b + 1] = [-1]
    return n, lens, parents


def _paths(parents):
    """For each new token the earlier ones that it sees among them, and itself."""
    b, sees = max(0, len(parents) - TREE), []
    for i, p in enumerate(parents):
        sees.append([*(sees[p] if i > b and p >= b else range(b) if i >= b else range(i)), i])
    return sees


def _pool(g, P, heads, page, dim):
    """A cache as earlier appends left it: codes of normal values, scales that differ by page and head."""
    def codes(shape):
        c = torch.empty(shape, device="cuda", dtype=torch.float16)
        return c.normal_(0, 40, generator=g).clamp_(-127, 127).round_().to(torch.int8)
    k, v = codes((P, heads, page, dim)), codes((P, heads, dim, page))
    scale = [0.025 * torch.exp(0.3 * torch.randn(P, heads, generator=g, device="cuda")) for _ in range(2)]
    return {"k": k, "v": v, "k_scales": scale[0], "v_scales": scale[1]}


def _tables(g, held, W, P):
    """Rows of page numbers in shuffled order, -1 past each sequence's pages."""
    order = torch.randperm(P, generator=g, device="cuda").int()
    at = torch.cumsum(held, 0) - held
    j = torch.arange(W, device="cuda")
    have = j[None] < held[:, None]
    return torch.where(have, order[(at[:, None] + j[None]).clamp(max=P - 1)], -1).int().contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    st, dt = {"case": case}, DT[case["dt"]]
    if case["op"] == "rotate":
        T, H, K, D, rot = case["T"], case["heads"], case["kv"], case["dim"], case["rot"]
        # one fused projection's output: queries and keys are slices of its rows, a few channels loud
        qkv = (rand(T, H + 2 * K, D) * torch.exp(0.5 * rand(D))).to(dt)
        st["q"], st["k"] = qkv[:, :H], qkv[:, H:H + K]
        st["pos"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
        st["freq"] = (10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)).float()
        st["wq"], st["wk"] = [(1 + 0.2 * rand(D)).to(dt) if case["norm"] else None for _ in range(2)]
        return st
    if case["op"] == "logprobs":
        M, V = case["M"], case["V"]
        x = torch.empty(M, V, device="cuda", dtype=dt)
        for a in range(0, M, 256):  # a few likely tokens over many unlikely ones
            y = rand(min(256, M - a), V)
            x[a:a + 256] = (2 * y + 0.5 * y.clamp(min=2) ** 2).to(dt)
        at = torch.arange(M, device="cuda")
        # some rows are restricted to a part of the vocabulary, one allows nothing
        cut = torch.randint(0, V, (M,), generator=g, device="cuda")
        for i, c in list(enumerate(cut.tolist()))[3::8]:
            x[i, c // 2:] = -math.inf
        if M > 100:
            x[100] = -math.inf
        st["x"] = x
        st["tokens"] = torch.where(at % 2 == 0, x.argmax(1), cut).int()
        return st
    S, B, H, D = case["S"], case["page"], case["heads"], case["dim"]
    n, lens, parents = _plan(case)
    st["n"], st["lens_host"], st["T"] = n, lens, sum(n)
    W = -(-case["ctx"] // B) + 1
    ints = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
    st["lens"], st["cu"] = ints(lens), ints([0] + n).cumsum(0).int()
    held = (st["lens"] + B - 1) // B
    P = -(-int(held.sum()) * 9 // 8) + 8
    cache = _pool(g, P, H, B, D)
    st.update(cache=cache, table=_tables(g, held, W, P))
    # one projection's output: q is a slice of its rows
    st["q"] = (1.5 * rand(st["T"], H * (case["group"] + 1), D)).to(dt)[:, : H * case["group"]]
    if parents:
        st["parents_host"], st["parent"] = parents, ints([p for row in parents for p in row])
    if own:
        from group_wise_affine_amd import qmm
        st["handle"] = qmm.Kv8Cache.of(cache["k"], cache["v"], cache["k_scales"], cache["v_scales"])
    return st


# -------------------------------------------------------------- plain forms


def _plain_rotate(st):
    rot, halves = st["case"]["rot"], st["case"]["pairs"] == "halves"
    angle = st["pos"].double()[:, None] * st["freq"].double()[None]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out = []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(2, keepdim=True) + 1e-6) * w.float()
        a, b = (y[..., :rot // 2], y[..., rot // 2:rot]) if halves else (y[..., 0:rot:2], y[..., 1:rot:2])
        u, v = a * cos - b * sin, b * cos + a * sin
        turned = torch.cat([u, v], 2) if halves else torch.stack([u, v], 3).flatten(2)
        out.append(torch.cat([turned, y[..., rot:]], 2).to(x.dtype))
    return {"q": out[0], "k": out[1]}


def _places(st):
    """Sequence and index of every new token."""
    cu = st["cu"].long()
    t = torch.arange(st["T"], device="cuda")
    s = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return s, t - cu[:-1][s]


def _plain_attend(st):
    """Pages that no query of a sequence sees are left out; the rest is dense."""
    case, c = st["case"], st["cache"]
    B, G, D, H, S = case["page"], case["group"], case["dim"], case["heads"], case["S"]
    most_n, most = max(st["n"]), max(max(st["lens_host"]), 1)
    lens = st["lens"].long()[:, None]
    n = (st["cu"][1:] - st["cu"][:-1]).long()[:, None]
    # the table's columns that are looked at, [S, columns]
    if case["op"] == "window":
        reach = min(-(-most // B), (case["window"] + most_n - 1) // B + 2)
        lo = (lens - n - case["window"] + 1).clamp(min=0) // B
        near = lo + torch.arange(reach, device="cuda")[None]
        first = torch.arange(min(-(-case["sinks"] // B), -(-most // B)), device="cuda")[None].expand(S, -1)
        cols = torch.cat([first, torch.where(near < first.shape[1], -1, near)], 1)
    else:
        cols = torch.arange(-(-most // B), device="cuda")[None].expand(S, -1)
    W = cols.shape[1]
    there = (cols >= 0) & (cols < st["table"].shape[1])
    rows = st["table"].gather(1, torch.where(there, cols, 0)).clamp(min=0).long()
    k = (c["k"][rows].float() * c["k_scales"][rows][..., None, None]).transpose(1, 2).reshape(S, H, W * B, D)
    v = (c["v"][rows].float() * c["v_scales"][rows][..., None, None]).permute(0, 2, 1, 4, 3).reshape(S, H, W * B, D)
    s, i = _places(st)
    q = torch.zeros(S, most_n, H * G, D, device="cuda")
    q[s, i] = st["q"].float()
    q = q.reshape(S, most_n, H, G, D).permute(0, 2, 1, 3, 4).reshape(S, H, most_n * G, D)
    x = torch.matmul(q, k.transpose(2, 3).contiguous()) * (D ** -0.5)
    pos = torch.where(there[:, :, None], cols[:, :, None] * B + torch.arange(B, device="cuda"), -1).reshape(S, 1, W * B)
    at = (lens - n + torch.arange(most_n, device="cuda")[None])[:, :, None]   # [S, new, 1]
    seen = (pos >= 0) & (pos <= at)
    if case["op"] == "window":
        seen &= (pos > at - case["window"]) | (pos < case["sinks"])
    else:
        # which new tokens each one sees: itself, its parent, theirs, and what precedes the tree
        j = torch.arange(most_n, device="cuda")
        b = (n - TREE).clamp(min=0)
        up = torch.full((S, most_n), -1, device="cuda")
        up[s, i] = st["parent"].long()
        up = torch.where((up >= b) & (up < j[None]), up, -1)
        line = ((up[:, :, None] == j) | (j[:, None] == j)).float()
        for _ in range(6):   # paths of twice the length
            line = (torch.matmul(line, line) > 0).float()
        line = (line > 0) | ((j < b[:, :, None]) & (j <= j[:, None]))
        new = pos - (lens - n)[:, :, None]   # index among the new tokens
        of = line.gather(2, new.clamp(0, most_n - 1).expand(-1, most_n, -1))
        seen = (pos >= 0) & (pos < lens[:, :, None]) & (at >= 0) & ((new < 0) | of)
    x = x.reshape(S, H, most_n, G, W * B).masked_fill_(~seen[:, None, :, None], -math.inf)
    m = x.amax(4, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x.sub_(m))
    z = p.sum(4, keepdim=True)
    o = torch.matmul(p.reshape(S, H, most_n * G, W * B), v).reshape(S, H, most_n, G, D)
    o = o / torch.where(z > 0, z, 1.0)
    lse = (m + torch.log(z))[..., 0]
    pick = lambda y: y.permute(0, 2, 1, 3, *range(4, y.dim()))[s, i].flatten(1, 2)  # noqa: E731
    return {"out": pick(o).to(st["q"].dtype), "lse": pick(lse)}


def _plain_logprobs(st):
    x, tokens, top = st["x"].float(), st["tokens"].long(), st["case"]["top"]
    m = x.amax(1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(x - m)
    z = e.sum(1, keepdim=True)
    lse = m + torch.log(z)
    # (where nothing is allowed every log probability is -inf and the entropy 0)
    lse = torch.where(lse == -math.inf, 0.0, lse)
    lp = x - lse
    h = -(e * torch.where(e > 0, lp, 0.0)).sum(1) / torch.where(z > 0, z, 1.0)[:, 0]
    out = {"logprob": lp.gather(1, tokens[:, None])[:, 0], "entropy": h}
    if top:
        # ordered like the values, and among equal ones by index
        b, V = (x + 0.0).view(torch.int32), x.shape[1]
        key = torch.where(b < 0, b ^ 0x7FFFFFFF, b).long() * 2 ** 32 + (V - 1 - torch.arange(V, device="cuda"))
        ids = V - 1 - (key.topk(top, dim=1).values & 0xFFFFFFFF)
        out.update(ids=ids.int(), top=lp.gather(1, ids))
    return out


PLAIN = {"rotate": _plain_rotate, "window": _plain_attend, "tree": _plain_attend, "logprobs": _plain_logprobs}


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return PLAIN[op](st)
    from group_wise_affine_amd import qmm
    if op == "rotate":
        q, k = qmm.qk_norm_rope(st["q"], st["k"], st["pos"], st["freq"], st["wq"], st["wk"], eps=1e-6,
                                interleaved=case["pairs"] == "neighbours")
        return {"q": q, "k": k}
    if op == "logprobs":
        lp, h, ids, top = qmm.logprobs(st["x"], st["tokens"], top=case["top"])
        return {"logprob": lp, "entropy": h, **({"ids": ids, "top": top} if case["top"] else {})}
    args = st["handle"], st["q"], st["table"], st["lens"], st["cu"]
    if op == "window":
        out, lse = qmm.kv8_attention_window(*args, case["window"], case["sinks"], return_lse=True)
    else:
        out, lse = qmm.kv8_attention_tree(*args, st["parent"], return_lse=True)
    return {"out": out, "lse": lse}


# --------------------------------------------------------------- the yardstick


def work(case):
    if case["op"] == "rotate":
        T, heads, D, rot = case["T"], case["heads"] + case["kv"], case["dim"], case["rot"]
        # the norm: a square and a sum, two products; the turn: two products and a sum per element
        return {"bytes": 4 * T * heads * D + 4 * T + 2 * rot + (4 * D if case["norm"] else 0),
                "flops": T * heads * ((4 * D if case["norm"] else 0) + 3 * rot)}
    if case["op"] == "logprobs":
        M, V = case["M"], case["V"]
        return {"bytes": M * (V * (4 if case["dt"] == "f32" else 2) + 12 + 8 * case["top"]), "flops": 5 * M * V}
    B, H, D, G = case["page"], case["heads"], case["dim"], case["group"]
    n, lens, parents = _plan(case)
    keys = pairs = 0
    for s, (m, L) in enumerate(zip(n, lens)):
        if not L:
            continue
        if case["op"] == "tree":
            keys += L
            pairs += m * (L - m) + sum(map(len, _paths(parents[s])))
            continue
        w, sinks = case["window"], case["sinks"]
        lo = max(0, L - m - w + 1)
        keys += L - lo + min(lo, sinks)
        for p in range(L - m, L):
            a = max(0, p - w + 1)
            pairs += p + 1 - a + min(a, sinks)
    return {"bytes": 2 * keys * H * D + 8 * H * (keys // B) + 4 * (keys // B) + 4 * sum(n) * H * G * (D + 1),
            "flops": 4 * pairs * H * G * D}


def exact(case, seed):
    """The definition in 64 bits."""
    st = prepare(case, seed)
    if case["op"] == "rotate":
        rot, D = case["rot"], case["dim"]
        a = torch.arange(rot // 2, device="cuda")
        # element i of a pair and the one it turns with
        i, j = (a, a + rot // 2) if case["pairs"] == "halves" else (2 * a, 2 * a + 1)
        turn = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"),
                           torch.outer(st["pos"].double(), st["freq"].double()))[:, None]
        res = {}
        for name, w in (("q", st["wq"]), ("k", st["wk"])):
            x = st[name].double()
            if w is not None:
                x = x / ((x * x).sum(2, keepdim=True) / D + 1e-6).sqrt() * w.double()
            z = torch.complex(x[..., i], x[..., j]) * turn
            x = x.clone()
            x[..., i], x[..., j] = z.real, z.imag
            res[name] = x
        return res
    if case["op"] == "logprobs":
        M, V, top = case["M"], case["V"], case["top"]
        res = {"logprob": torch.empty(M, dtype=torch.float64, device="cuda"),
               "entropy": torch.empty(M, dtype=torch.float64, device="cuda")}
        if top:
            res.update(ids=None, top=torch.empty(M, min(top, V), dtype=torch.float64, device="cuda"))
        for r in range(0, M, 64):
            x = st["x"][r:r + 64].double()
            lp = torch.log_softmax(x, 1)
            lp[(x == -math.inf).all(1)] = -math.inf
            res["logprob"][r:r + 64] = lp.gather(1, st["tokens"][r:r + 64].long()[:, None])[:, 0]
            res["entropy"][r:r + 64] = -torch.special.xlogy(lp.exp(), lp.exp()).sum(1)
            if top:
                res["top"][r:r + 64] = lp.sort(dim=1, descending=True).values[:, :top]
        return res
    B, H, D, G = case["page"], case["heads"], case["dim"], case["group"]
    c, (n, lens, parents) = st["cache"], _plan(case)
    table = st["table"].cpu()
    out = torch.zeros(st["T"], H * G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((st["T"], H * G), -math.inf, dtype=torch.float64, device="cuda")
    t0 = 0
    for s in range(case["S"]):
        L, m = lens[s], n[s]
        if L:
            at = torch.arange(L, device="cuda")
            mine = torch.arange(L - m, L, device="cuda")[:, None]
            if case["op"] == "window":
                hidden = (at > mine) | ((at <= mine - case["window"]) & (at >= case["sinks"]))
                keep = ~hidden.all(0)
            else:
                hidden = at.expand(m, -1) >= L - m
                for i, path in enumerate(_paths(parents[s])):
                    hidden[i, [L - m + j for j in path]] = False
                keep = torch.ones(L, dtype=torch.bool, device="cuda")
            hidden = hidden[:, keep]
            row = table[s, : -(-L // B)].cuda().long()
            for h in range(H):
                k = (c["k"][row, h].double() * c["k_scales"][row, h].double()[:, None, None]).reshape(-1, D)[:L][keep]
                v = (c["v"][row, h].double() * c["v_scales"][row, h].double()[:, None, None]).transpose(1, 2).reshape(-1, D)[:L][keep]
                kt = k.t().contiguous()
                for g in range(G):
                    x = (st["q"][t0:t0 + m, h * G + g].double() @ kt) / math.sqrt(D)
                    x[hidden] = -math.inf
                    lse[t0:t0 + m, h * G + g] = torch.logsumexp(x, 1)
                    out[t0:t0 + m, h * G + g] = torch.softmax(x, 1) @ v
        t0 += m
    return {"out": out, "lse": lse}
