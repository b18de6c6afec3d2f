"""What the drafted-decoding and scoring operators are measured on.

Each case is one call a user's program makes: attention of a drafted token tree over a key/value
cache, log probabilities of given tokens (with entropy and top alternatives) from logits, their
gradient, and the acceptance of a drafted tree.  ``run`` makes that call through the framework
(``own``) or computes the same thing from elementary torch operations; ``exact`` is the definition
in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the smallest serving call: one new token of one sequence over a GPT-2 cache
        dict(name="tree_single", op="tree", B=1, N=1, nh=12, hs=64, cap=1024, lo=700, hi=700, dtype="bf16"),
        # a small draft per sequence, GPT-2 heads and context, requests of every age
        dict(name="tree_gpt2", op="tree", B=8, N=16, nh=12, hs=64, cap=1024, lo=0, hi=1000, dtype="bf16"),
        # the widest draft (two or three absent nodes in some sequences), a longer context
        dict(name="tree_wide", op="tree", B=32, N=64, nh=16, hs=64, cap=4096, lo=100, hi=4096, dtype="bf16"),
        # the largest: 25 heads, a full serving batch, long contexts of odd lengths
        dict(name="tree_long", op="tree", B=48, N=23, nh=25, hs=64, cap=8192, lo=1501, hi=8185, dtype="bf16"),
        # fp32 storage, an odd draft
        dict(name="tree_f32", op="tree", B=8, N=9, nh=12, hs=64, cap=1024, lo=17, hi=1013, dtype="f32"),
        # scoring a training-sized batch without the padding columns of the vocabulary
        dict(name="score_batch", op="score", rows=12288, V=50257, ld=50304, k=20, T=1.0, dtype="bf16", banned=0),
        # the logits of one decoding step: a few fp32 rows, the alternatives shown to a reader
        dict(name="score_step", op="score", rows=8, V=50304, ld=50304, k=5, T=0.8, dtype="f32", banned=47),
        # an odd vocabulary, rows that start at every alignment, some tokens forbidden
        dict(name="score_odd", op="score", rows=1001, V=32003, ld=32003, k=64, T=1.3, dtype="f32", banned=300),
        # a training step that weighs each token's log probability and the entropy
        dict(name="grad_batch", op="grad", rows=12288, V=50304, ld=50304, T=1.0, dtype="bf16"),
        # the same in fp32 with an odd vocabulary
        dict(name="grad_odd", op="grad", rows=519, V=50257, ld=50257, T=0.7, dtype="f32"),
        # after a verification step of GPT-2: few sequences
        dict(name="accept_gpt2", op="accept", B=8, N=16, L=12, nh=12, hs=64, cap=1024, lo=0, hi=1000, dtype="bf16"),
        # many sequences with wide trees
        dict(name="accept_wide", op="accept", B=64, N=64, L=24, nh=16, hs=64, cap=128, lo=3, hi=101, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = {}
    for c in listed():
        w = work(c)
        top[c["op"]] = max(top.get(c["op"], 0), w["bytes"])
    while True:
        op = rng.choice(["tree", "tree", "tree", "score", "score", "grad", "accept"])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if op == "tree":
            cap = _log_int(rng, 64, 8192)
            hi = rng.randint(0, cap)
            c = dict(op=op, B=_log_int(rng, 1, 64), N=rng.choice([1, rng.randint(1, 16), rng.randint(1, 64)]),
                     nh=rng.choice([1, 4, 12, 16, 25]), hs=64 if dtype == "bf16" else rng.choice([32, 64, 128]),
                     cap=cap, lo=rng.randint(0, hi), hi=hi, dtype=dtype)
        elif op in ("score", "grad"):
            V = _log_int(rng, 65, 131072)
            c = dict(op=op, rows=_log_int(rng, 1, 12288), V=V, ld=V + rng.choice([0, 0, 1, 47]),
                     T=rng.choice([1.0, round(rng.uniform(0.3, 2.0), 3)]), dtype=dtype)
            if op == "score":
                c["k"] = rng.choice([0, 1, rng.randint(2, 64)])
                c["banned"] = rng.choice([0, min(V // 16, V - 64)])
        else:
            cap = _log_int(rng, 64, 1024)
            N = rng.randint(1, 64)
            hi = rng.randint(0, cap - 8)
            c = dict(op=op, B=_log_int(rng, 1, 64), N=N, L=rng.choice([1, 4, 12, 24]), nh=rng.choice([4, 12, 16, 25]),
                     hs=64 if dtype == "bf16" else 32, cap=cap, lo=rng.randint(0, hi), hi=hi, dtype=dtype)
            es = 2 if dtype == "bf16" else 4
            if c["L"] * c["B"] * cap * 2 * c["nh"] * c["hs"] * es > 1 << 29:
                continue
        if work(c)["bytes"] <= top[op]:
            return c


# Lengths are the same evenly spread values for every seed, in an order that the seed gives.
def _length_list(c):
    if c["B"] == 1:
        return [c["hi"]]
    return [c["lo"] + (c["hi"] - c["lo"]) * i // (c["B"] - 1) for i in range(c["B"])]


# Nodes present in sequence b: a batch pads its trees to the widest one.
def _present(c, b):
    return max(1, c["N"] - b % 4)


# Tokens accepted, the same counts for every seed in an order that the seed gives.
def _accept_list(c):
    return [1 + i % _chain(c) for i in range(c["B"])]


# A tree starts with a chain of this many nodes (the draft's first guesses).
def _chain(c):
    return min(6, max(1, c["N"] - 3))


def work(c):
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "tree":
        C, keys = c["nh"] * c["hs"], sum(_length_list(c))
        nodes = c["B"] * c["N"]
        return {"bytes": keys * 2 * C * es + nodes * 4 * C * es + nodes * 4 + c["B"] * 4,
                "flops": 4 * C * c["N"] * keys + 2 * C * nodes * (c["N"] + 1)}
    if c["op"] == "score":
        n = c["rows"] * c["V"]
        return {"bytes": n * es + c["rows"] * (8 + 12 + 12 * c["k"]), "flops": 6 * n}
    if c["op"] == "grad":
        n = c["rows"] * c["V"]
        return {"bytes": 2 * n * es + c["rows"] * 24, "flops": 7 * n}
    C = c["nh"] * c["hs"]
    return {"bytes": sum(_accept_list(c)) * c["L"] * 2 * C * es * 2 + c["B"] * c["N"] * 24 + c["B"] * 20,
            "flops": c["B"] * c["N"]}


# ---------------------------------------------------------------- inputs
def _trees(c, g):
    """Parents int32 [B, N] on the CPU: a chain, then nodes on earlier ones at random; -2 where absent."""
    B, N, D = c["B"], c["N"], _chain(c)
    u = torch.rand((B, N), generator=g)
    p = (u * torch.arange(N)).floor().to(torch.int32)
    p = torch.minimum(p, torch.arange(N, dtype=torch.int32) - 1)
    p[:, :D] = torch.arange(D, dtype=torch.int32) - 1
    for b in range(B):
        p[b, _present(c, b):] = -2
    return p


def prepare(case, seed):
    c = case
    cpu = torch.Generator().manual_seed(seed)
    gpu = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] in ("tree", "accept"):
        B, N, C, cap = c["B"], c["N"], c["nh"] * c["hs"], c["cap"]
        order = torch.randperm(B, generator=cpu)
        s["lengths"] = torch.tensor(_length_list(c), dtype=torch.int32)[order].cuda()
        parents = _trees(c, cpu)
        s["parents"] = parents.cuda()
    if c["op"] == "tree":
        s["qkv"] = torch.randn((B, N, 3, C), generator=gpu, device="cuda").to(dt)
        s["cache"] = _normal((B, cap, 2, C), gpu, dt)
    elif c["op"] == "accept":
        tokens = torch.stack([torch.randperm(50257, generator=cpu)[:N] for _ in range(B)])
        chosen = torch.randint(0, 50257, (B, N), generator=cpu)
        n_acc = torch.tensor(_accept_list(c))[torch.randperm(B, generator=cpu)]
        for b in range(B):                       # the model confirms the chain up to its n-th node
            n = min(int(n_acc[b]), _present(c, b))
            chosen[b, :n - 1] = tokens[b, 1:n]
            chosen[b, n - 1:] = 50257 + torch.arange(N - n + 1)
        s["tokens"], s["chosen"] = tokens.cuda(), chosen.cuda()
        s["qkv"] = _normal((c["L"], B, N, 3, C), gpu, dt)
        s["cache"] = _normal((c["L"], B, cap, 2, C), gpu, dt)
    else:
        rows, V, ld = c["rows"], c["V"], c["ld"]
        z = _normal((rows, ld), gpu, dt, 3.0)
        ids = torch.randperm(V, generator=cpu)
        banned = c.get("banned", 0)              # forbidden tokens
        z[:, ids[:banned].cuda()] = float("-inf")
        s["logits"] = z[:, :V]
        tokens = ids[torch.randint(banned, V, (rows,), generator=cpu)]
        tokens[::17] = -1                        # prompt positions, not scored
        s["tokens"] = tokens.cuda()
        if c["op"] == "grad":
            s["lse"], s["entropy"] = _lse_entropy(s["logits"], c["T"])
            s["dlogp"] = torch.randn(rows, generator=gpu, device="cuda")
            s["dentropy"] = 0.01 * torch.randn(rows, generator=gpu, device="cuda")
    if own and c["op"] == "accept":
        from decoder_only_transformer_causal_b200 import GPTConfig
        s["cfg"] = GPTConfig(n_layer=c["L"], n_head=c["nh"], n_embd=C, block_size=cap, vocab_size=50304,
                             dtype=c["dtype"])
    return s


def _normal(shape, gen, dt, scale=1.0):
    """Normal values in dt, made a slab at a time."""
    out = torch.empty(shape, dtype=dt, device="cuda")
    flat = out.view(-1)
    step = 1 << 27
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        part.copy_(torch.randn(part.numel(), generator=gen, device="cuda").mul_(scale))
    return out


def _lse_entropy(logits, T):
    """The forward's saved row values, in 64 bits rounded once."""
    lse = torch.empty(logits.shape[0], device="cuda")
    ent = torch.empty_like(lse)
    for i in range(0, logits.shape[0], 1024):
        z = logits[i:i + 1024].double() / T
        l = torch.logsumexp(z, 1)
        p = (z - l[:, None]).exp_()
        lse[i:i + 1024] = l.float()
        ent[i:i + 1024] = (l - torch.where(p > 0, p * z, 0.0).sum(1)).float()
    return lse, ent


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"tree": _own_tree, "score": _own_score, "grad": _own_grad, "accept": _own_accept}[op](state)
    return {"tree": _plain_tree, "score": _plain_score, "grad": _plain_grad, "accept": _plain_accept}[op](state)


def _own_tree(s):
    from decoder_only_transformer_causal_b200 import native
    return native.tree_attention(s["qkv"], s["cache"], s["lengths"], s["parents"], s["case"]["nh"])


def _own_score(s):
    from decoder_only_transformer_causal_b200 import native
    c = s["case"]
    r = native.token_logprobs(s["logits"], s["tokens"], k=c["k"], temperature=c["T"])
    return [r.logp, r.entropy, r.lse] + ([r.top_ids, r.top_logp] if c["k"] else [])


def _own_grad(s):
    from decoder_only_transformer_causal_b200 import native
    return native.token_logprobs_backward(s["logits"], s["tokens"], s["lse"], s["entropy"], dlogp=s["dlogp"],
                                          dentropy=s["dentropy"], temperature=s["case"]["T"])


def _own_accept(s):
    from decoder_only_transformer_causal_b200 import native
    r = native.tree_accept(s["cfg"], s["parents"], s["tokens"], s["chosen"], s["lengths"], s["qkv"], s["cache"])
    return [r.path, r.n_accepted, r.next_token, r.lengths, s["cache"]]


# ---------------------------------------------------------------- plain forms
def _ancestors(parents):
    """bool [B, N, N]: does node i see node j (itself and its ancestors); False rows for absent nodes."""
    B, N = parents.shape
    see = torch.zeros((B, N, N), dtype=torch.bool, device=parents.device)
    rows = torch.arange(B, device=parents.device)
    for i in range(N):
        p = parents[:, i].long()
        see[:, i] = see[rows, p.clamp(min=0)] & (p >= 0)[:, None]
        see[:, i, i] = p >= -1
    return see


def _plain_tree(s):
    c = s["case"]
    B, N, nh, hs, cap = c["B"], c["N"], c["nh"], c["hs"], c["cap"]
    see = _ancestors(s["parents"])
    here = s["parents"] >= -1
    y = torch.empty((B, N, nh * hs), dtype=s["qkv"].dtype, device="cuda")
    t = torch.arange(cap, device="cuda")
    for b in range(B):
        q, kn, vn = (s["qkv"][b, :, j].float().view(N, nh, hs).transpose(0, 1) for j in range(3))
        kc, vc = (s["cache"][b, :, j].float().view(cap, nh, hs).transpose(0, 1) for j in range(2))
        live = t < s["lengths"][b]
        vc = torch.where(live[None, :, None], vc, 0.0)
        mask = torch.cat([live[None, :] & here[b][:, None], see[b]], 1)
        sc = torch.cat([q @ kc.transpose(1, 2), q @ kn.transpose(1, 2)], 2) / math.sqrt(hs)
        sc = sc.masked_fill(~mask, float("-inf"))
        m = sc.amax(2, keepdim=True).clamp(min=-3e38)
        p = torch.exp(sc - m)
        l = p.sum(2, keepdim=True).clamp(min=1e-38)
        o = (p[..., :cap] @ vc + p[..., cap:] @ vn) / l
        y[b] = o.transpose(0, 1).reshape(N, nh * hs).to(y.dtype)
    return y


def _order_keys(z):
    """int64 keys that order values of z, ties to the lower column."""
    bits = (z.float() + 0.0).view(torch.int32).long()
    order = torch.where(bits >= 0, bits, -(bits & 0x7fffffff))
    return (order << 32) - torch.arange(z.shape[1], device=z.device)


def _plain_score(s):
    c = s["case"]
    rows, k = c["rows"], c["k"]
    outs = [[], [], [], [], []]
    step = max(1, (1 << 27) // c["V"])
    for i in range(0, rows, step):
        z0 = s["logits"][i:i + step]
        z = z0.float() / c["T"]
        m = z.amax(1, keepdim=True)
        e = torch.exp(z - m)
        tot = e.sum(1, keepdim=True)
        lse = m + torch.log(tot)
        logp_all = z - lse
        p = e / tot
        ent = -torch.where(p > 0, p * logp_all, 0.0).sum(1)
        t = s["tokens"][i:i + step]
        lp = logp_all.gather(1, t.clamp(min=0)[:, None])[:, 0]
        outs[0].append(torch.where(t >= 0, lp, 0.0))
        outs[1].append(ent)
        outs[2].append(lse[:, 0])
        if k:
            key = torch.topk(_order_keys(z0), k, 1).values
            ids = (-key) & 0xffffffff
            outs[3].append(ids)
            outs[4].append(logp_all.gather(1, ids))
    return [torch.cat(o) for o in outs[:5 if k else 3]]


def _plain_grad(s):
    c = s["case"]
    z0 = s["logits"]
    out = torch.empty(z0.shape, dtype=z0.dtype, device="cuda")
    step = max(1, (1 << 27) // c["V"])
    for i in range(0, c["rows"], step):
        sl = slice(i, i + step)
        t, g, h = s["tokens"][sl], s["dlogp"][sl], s["dentropy"][sl]
        lp = z0[sl].float() / c["T"] - s["lse"][sl, None]
        p = torch.exp(lp)
        g = torch.where(t >= 0, g, 0.0)
        d = -p * (g[:, None] + h[:, None] * (lp + s["entropy"][sl, None]))
        d.scatter_add_(1, t.clamp(min=0)[:, None], g[:, None])
        out[sl] = (d / c["T"]).to(out.dtype)
    return out


def _plain_accept(s):
    c = s["case"]
    B, N, L, cap = c["B"], c["N"], c["L"], c["cap"]
    parents, tokens, chosen = s["parents"].long(), s["tokens"], s["chosen"]
    dev = parents.device
    rows = torch.arange(B, device=dev)
    ok = torch.zeros((B, N), dtype=torch.bool, device=dev)
    depth = torch.zeros((B, N), dtype=torch.long, device=dev)
    for i in range(N):
        p = parents[:, i]
        pc = p.clamp(min=0)
        ok[:, i] = (p == -1) | ((p >= 0) & ok[rows, pc] & (tokens[:, i] == chosen[rows, pc]))
        depth[:, i] = torch.where(p >= 0, depth[rows, pc] + 1, 1)
    rank = torch.where(ok, depth, 0) * N + (N - 1 - torch.arange(N, device=dev))
    leaf = N - 1 - rank.amax(1) % N
    full = torch.where(ok[rows, leaf], depth[rows, leaf], 0)
    room = cap - s["lengths"].long()
    n = torch.minimum(full, room)
    path = torch.full((B, N), -1, dtype=torch.long, device=dev)
    cur = leaf
    for j in range(N):                           # from the deepest node up to the root
        at = full - 1 - j
        keep = (at >= 0) & (at < n)
        path[rows, at.clamp(min=0)] = torch.where(keep, cur, path[rows, at.clamp(min=0)])
        cur = torch.where(at > 0, parents[rows, cur], cur)
    last = path[rows, (n - 1).clamp(min=0)]
    nxt = torch.where(n > 0, chosen[rows, last.clamp(min=0)], -1)
    for j in range(N):
        dst = (s["lengths"].long() + j).clamp(max=cap - 1)
        new = s["qkv"][:, rows, path[:, j].clamp(min=0), 1:]
        s["cache"][:, rows, dst] = torch.where((j < n)[:, None, None], new, s["cache"][:, rows, dst])
    return [path.int(), n.int(), nxt, (s["lengths"] + n).int(), s["cache"]]


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "score": _exact_score, "grad": _exact_grad, "accept": _exact_accept}[case["op"]](s)


def _exact_tree(s):
    c = s["case"]
    N, nh, hs = c["N"], c["nh"], c["hs"]
    lens, parents = s["lengths"].tolist(), s["parents"].tolist()
    y = torch.zeros((c["B"], N, nh, hs), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        kv = torch.cat([s["cache"][b, :n], s["qkv"][b, :, 1:]]).double().view(n + N, 2, nh, hs)
        allowed = torch.zeros((N, n + N), dtype=torch.bool)
        for i, p in enumerate(parents[b]):
            if p == -2:
                continue
            allowed[i, :n] = True
            j = i
            while j >= 0:
                allowed[i, n + j] = True
                j = parents[b][j]
        present = [i for i, p in enumerate(parents[b]) if p != -2]
        q = s["qkv"][b, present, 0].double().view(len(present), nh, hs)
        z = torch.einsum("ihd,jhd->hij", q, kv[:, 0]) * hs ** -0.5
        z.masked_fill_(~allowed[present].cuda(), -math.inf)
        y[b, present] = torch.einsum("hij,jhd->ihd", torch.softmax(z, -1), kv[:, 1])
    return y.view(c["B"], N, nh * hs)


def _exact_score(s):
    c = s["case"]
    rows, k = c["rows"], c["k"]
    logp = torch.zeros(rows, dtype=torch.float64, device="cuda")
    ent, lse = torch.empty_like(logp), torch.empty_like(logp)
    top_lp = torch.empty((rows, k), dtype=torch.float64, device="cuda")
    for i in range(0, rows, 512):
        sl = slice(i, i + 512)
        z = s["logits"][sl].double()
        lp = torch.log_softmax(z / c["T"], 1)
        ent[sl] = torch.special.entr(lp.exp()).sum(1)
        lse[sl] = torch.logsumexp(z / c["T"], 1)
        t = s["tokens"][sl]
        logp[sl] = torch.where(t < 0, 0.0, torch.take_along_dim(lp, t.clamp(min=0)[:, None], 1)[:, 0])
        if k:
            top_lp[sl] = torch.topk(z, k, 1).values / c["T"] - lse[sl, None]
    return [logp, ent, lse] + ([None, top_lp] if k else [])


def _exact_grad(s):
    c = s["case"]
    out = torch.empty((c["rows"], c["V"]), dtype=torch.float64, device="cuda")
    for i in range(0, c["rows"], 512):
        sl = slice(i, i + 512)
        lp = torch.log_softmax(s["logits"][sl].double() / c["T"], 1)
        p = lp.exp()
        t = s["tokens"][sl]
        g = s["dlogp"][sl].double() * (t >= 0)
        ent = -(p * lp).sum(1)
        d = -g[:, None] * p - s["dentropy"][sl].double()[:, None] * p * (lp + ent[:, None])
        d[torch.arange(len(t), device="cuda"), t.clamp(min=0)] += g
        out[sl] = d / c["T"]
    return out


def _exact_accept(s):
    c = s["case"]
    parents, tokens, chosen = s["parents"].tolist(), s["tokens"].tolist(), s["chosen"].tolist()
    lens = s["lengths"].tolist()
    paths, counts, nxt, new_len = [], [], [], []
    cache = s["cache"]
    for b in range(c["B"]):
        best = []
        walks = {}
        for i, p in enumerate(parents[b]):
            if p == -1:
                walks[i] = [i]
            elif p in walks and tokens[b][i] == chosen[b][p]:
                walks[i] = walks[p] + [i]
            if i in walks and len(walks[i]) > len(best):
                best = walks[i]
        best = best[:c["cap"] - lens[b]]
        for j, node in enumerate(best):
            cache[:, b, lens[b] + j] = s["qkv"][:, b, node, 1:]
        paths.append(best + [-1] * (c["N"] - len(best)))
        counts.append(len(best))
        nxt.append(chosen[b][best[-1]] if best else -1)
        new_len.append(lens[b] + len(best))
    return [torch.tensor(v, dtype=torch.float64, device="cuda") for v in (paths, counts, nxt, new_len)] + [cache]
