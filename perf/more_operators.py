"""Trees of drafts, rotary positions and constrained target tokens: their operators, measured case by case.

attend    attention of the rows of drafted trees over the paged cache: a row sees its request's
          tokens and its own ancestors
rotary    rotary positions of a step's queries and keys, and the keys and values laid into the pages
target    a step's tokens from its logits: penalties for repeated tokens, biases, grammar masks
history   the repeated tokens' record: rows cleared, prompts and answers entered
tree      a tree's bookkeeping: chains merged into a tree, its depths and ancestors, the accepted
          path, and that path's keys and values moved together

Row j of request r lies at row offsets[r] + lead * r + j of the packed tensors, n_r = offsets[r+1]
- offsets[r] + lead rows in all, at positions len[r] + j of the cache.  Its node's parent is another
node of the request, or -1; a word of 64 bits per row says which nodes the row sees.  The cache is k
[layers, n_pages, Hkv, page/16, D/8, 16, 8] and v [layers, n_pages, Hkv, page/16, D, 16]; table
[rows, width] holds page ids (-1: none), len [rows] the tokens kept (-1: a vacant row).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"


def listed():
    return [
        # small trees of four requests with short contexts: the latency of a small verification step
        dict(name="attend: 4 small trees", op="attend", R=4, K=15, H=32, Hkv=8, D=128, dtype="bf16", page=16, own_len=700,
             groups=0, shared=0, vacant=0),
        # a full verification step of trees of up to 32 nodes behind one long system prompt
        dict(name="attend: 256 trees, shared 8192", op="attend", R=256, K=31, H=64, Hkv=8, D=128, dtype="bf16", page=64,
             own_len=1024, groups=1, shared=8192, vacant=6),
        # two requests with very long contexts and the largest trees
        dict(name="attend: 2 of 131072 tokens, fp16", op="attend", R=2, K=63, H=32, Hkv=4, D=64, dtype="fp16", page=128,
             own_len=131072, groups=0, shared=0, vacant=0),
        # a full verification step of trees, whole heads in two halves
        dict(name="rotary: verify", op="rotary", R=256, K=7, lead=1, H=64, Hkv=8, D=128, dtype="bf16", page=64, own_len=512,
             vacant=6, dim=128, first=0, interleaved=False, base=10000.0, scaling="none", factor=1.0),
        # whole prompts of a few requests, half of each head turned, neighbouring dims paired, stretched for long contexts
        dict(name="rotary: prompts, fp16", op="rotary", R=8, K=4099, lead=0, H=32, Hkv=8, D=128, dtype="fp16", page=128,
             own_len=300, vacant=0, dim=64, first=64, interleaved=True, base=500000.0, scaling="ramp", factor=16.0),
        # single tokens of four requests, everything on: the latency of a small constrained step
        dict(name="target: 4 single tokens", op="target", R=4, K=0, V=129280, dtype="bf16", seen=700, biased=50, masks=4,
             allow=0.3, processed=False),
        # a full verification step of trees, with penalties, biases and grammar masks of some of the rows
        dict(name="target: verify", op="target", R=256, K=7, V=129280, dtype="bf16", seen=2000, biased=100, masks=64, allow=0.3,
             processed=False),
        # the processed logits themselves, for a sampler: an odd vocabulary, full precision, penalties alone
        dict(name="target: processed logits, fp32", op="target", R=96, K=5, V=32771, dtype="fp32", seen=500, biased=0, masks=0,
             allow=1.0, processed=True),
        # a few requests admitted, with the rows of those before them cleared
        dict(name="history: 4 admitted", op="history", R=4, V=129280, prompt=1000, answer=8),
        # a large engine's rows rebuilt, long prompts and answers
        dict(name="history: 128 rebuilt", op="history", R=128, V=129280, prompt=16000, answer=2000),
        # a small step of four chains a request over a few layers
        dict(name="tree: 16 requests", op="tree", R=16, S=4, K=7, V=129280, layers=2, Hkv=8, D=128, dtype="bf16", page=16,
             own_len=200, vacant=0),
        # a full step over many layers
        dict(name="tree: 256 requests, 16 layers", op="tree", R=256, S=4, K=7, V=129280, layers=16, Hkv=8, D=128, dtype="bf16",
             page=64, own_len=60, vacant=6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "rotary", "target", "target", "history", "tree"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    D, dtype, page = rng.choice([64, 128, 128, 256]), rng.choice(["bf16", "fp16"]), rng.choice([16, 32, 64, 128])
    if op == "attend":
        R = _log(rng, 1, 200)
        c = dict(op=op, R=R, K=rng.choice([1, 4, 7, 15, 24, 31] + [63] * (R < 64)), H=Hkv * rng.choice([1, 2, 3, 5, 8]), Hkv=Hkv,
                 D=D, dtype=dtype, page=page, own_len=_log(rng, 1, 131072 // R), groups=0, shared=0,
                 vacant=rng.choice([0, R // 9]))
        if rng.random() < 0.5:
            c.update(groups=rng.randint(1, min(R, 3)), shared=page * _log(rng, 1, 4096 // page))
        return c
    if op == "rotary":
        prompts = rng.random() < 0.4
        R = _log(rng, 1, 6) if prompts else _log(rng, 1, 256)
        dim = 16 * rng.randint(1, D // 16)
        return dict(op=op, R=R, K=_log(rng, 2, 4000) if prompts else rng.choice([0, 3, 7, 15]), lead=0 if prompts else 1,
                    H=Hkv * rng.choice([1, 2, 3, 4]), Hkv=Hkv, D=D, dtype=dtype, page=page,
                    own_len=_log(rng, 1, 40000 // R if not prompts else 500), vacant=rng.choice([0, R // 9]), dim=dim,
                    first=8 * rng.randint(0, (D - dim) // 8), interleaved=rng.random() < 0.5,
                    base=rng.choice([10000.0, 500000.0, 1e6]), scaling=rng.choice(["none", "linear", "bands", "ramp"]),
                    factor=rng.choice([2.0, 4.0, 16.0]))
    if op == "target":
        dtype, processed = rng.choice(["bf16", "fp16", "fp32"]), rng.random() < 0.4
        return dict(op=op, R=_log(rng, 1, 200 // (2 if processed else 1) // (2 if dtype == "fp32" else 1)), K=rng.choice([0, 3, 7]),
                    V=_log(rng, 1000, 129280), dtype=dtype, seen=_log(rng, 1, 2000), biased=rng.choice([0, 1, 30, 200]),
                    masks=rng.choice([0, 1, 16]), allow=rng.choice([0.001, 0.3, 0.99]), processed=processed)
    if op == "history":
        R = _log(rng, 1, 96)
        return dict(op=op, R=R, V=_log(rng, 1000, 129280), prompt=_log(rng, 1, 12000), answer=_log(rng, 1, 2000))
    K = rng.randint(1, 15)
    R = _log(rng, 1, 200)
    return dict(op=op, R=R, S=rng.randint(1, 63 // K if K > 7 else 8), K=K, V=_log(rng, 1000, 129280), layers=rng.randint(1, 8),
                Hkv=Hkv, D=D, dtype=dtype, page=page, own_len=_log(rng, 1, 300), vacant=rng.choice([0, R // 9]))


# ---- the sizes of a case, the same whatever the seed -----------------------------------------------------------------------


def _requests(c):
    """[(tokens of its own before the step or -1, rows of the step)] of the case's requests, in no particular order."""
    R, K, lead = c["R"], c["K"], c.get("lead", 1)
    got = []
    for i in range(R):
        drafts = ((i * 7 + 3) % R) * (K + 1) // R if lead else 1 + ((i * 7 + 3) % R) * K // R
        n_own = -1 if i < c.get("vacant", 0) else max(0, round(c.get("own_len", 0) * (i + 1) / R) - (0 if lead else 1))
        got.append((n_own, min(drafts, K) + lead))
    return got


def work(c):
    op, R = c["op"], c["R"]
    size = 4 if c.get("dtype") == "fp32" else 2
    if op == "attend":
        H, Hkv, D, sh = c["H"], c["Hkv"], c["D"], c["shared"]
        keys = pairs = rows = 0
        for n_own, n in _requests(c):
            if n_own >= 0:
                keys += n_own + n
                pairs += n * (sh + n_own) + n * math.log2(n + 1)  # about as many ancestors
            rows += n
        keys += sh * c["groups"]
        return {"bytes": 2 * keys * Hkv * D * 2 + rows * H * (2 * D * 2 + 4) + 8 * rows, "flops": 4.0 * pairs * H * D}
    if op == "rotary":
        rows, live = sum(n for _, n in _requests(c)), sum(n for n_own, n in _requests(c) if n_own >= 0)
        return {"bytes": (rows * c["H"] + live * 2 * c["Hkv"]) * c["D"] * 2 * 2, "flops": 3.0 * rows * (c["H"] + c["Hkv"]) * c["dim"]}
    if op == "target":
        rows = sum(n for _, n in _requests(c))
        return {"bytes": rows * (c["V"] * size * (2 if c["processed"] else 1) + 4) + min(rows, c["masks"]) * c["V"] / 8
                + R * c["V"] / 4 + R * c["biased"] * 8, "flops": 0}
    if op == "history":
        return {"bytes": R * (c["V"] * 4 + c["V"] / 4 + 4.0 * (c["prompt"] + c["answer"])), "flops": 0}
    moved = (R - c["vacant"]) * (c["K"] / 2) * (1 - 1 / c["S"])  # nodes of the accepted paths off the first chain
    return {"bytes": 2.0 * moved * c["layers"] * c["Hkv"] * c["D"] * 2 * 2 + R * c["S"] * (c["K"] * 24.0 + 4), "flops": 0}


# ---- inputs -----------------------------------------------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _uniform(g, shape):
    return torch.rand(shape, generator=g, device=DEV, dtype=torch.float64)


def _tokens(g, shape, V):
    """Token ids as text has them: the lower, the more frequent."""
    return (_uniform(g, shape) ** 4 * V).int().clamp(max=V - 1)


def _kv(g, c, layers, n_pages):
    """The whole cache filled: what lies in free pages and behind a sequence's end is some old token's."""
    pb, D, t = c["page"] // 16, c["D"], DTYPES[c["dtype"]]
    k = torch.empty((layers, n_pages, c["Hkv"], pb, D // 8, 16, 8), dtype=t, device=DEV)
    v = torch.empty((layers, n_pages, c["Hkv"], pb, D, 16), dtype=t, device=DEV)
    for x in (k, v):
        x.normal_(generator=g)
    return k, v


def _handle(s, layers, n_pages, c, width):
    """The framework's handle of the cache, which a user's program keeps as long as the buffers."""
    from confidence_scheduled_verification_amd import binding as B
    return B.PagedCache(layers, n_pages, c["page"], c["Hkv"], c["D"], B.DSPARK_F16 if c["dtype"] == "fp16" else B.DSPARK_BF16,
                        s["table"].shape[0], width, k=s["k"], v=s["v"], table=s["table"], len=s["len"], ref=s["ref"])


def _place(order, pages_of, rows, width, n_pages):
    """A table whose rows hold `pages_of[r]` pages each, dealt from `order`, and the counts."""
    table = torch.full((rows, width), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(pages_of):
        table[r, :n] = order[at:at + n]
        at += n
    ref = torch.zeros(n_pages, dtype=torch.int32)
    ref[order[:at].long()] = 1
    return table, ref


def _cache(s, c, g, cpu, reqs, layers):
    """Pages for the requests (a shared prefix among them) and the cache over them."""
    page, R, sh, n_groups = c["page"], c["R"], c.get("shared", 0), c.get("groups", 0)
    sp = sh // page if n_groups else 0
    pages_of = [0 if n < 0 else -(-(n + m) // page) for n, m in reqs]
    width = sp + max(pages_of) + 2
    n_pages = sum(pages_of) + sp * n_groups + 3
    order = torch.randperm(n_pages, generator=cpu).to(torch.int32)
    own_table, ref = _place(order[sp * n_groups:], pages_of, R, width, n_pages)
    table = own_table
    if n_groups:
        bound = [i * R // n_groups for i in range(n_groups + 1)]
        shared = order[:sp * n_groups].reshape(n_groups, sp)
        table = torch.full((R, width), -1, dtype=torch.int32)
        for i in range(n_groups):
            table[bound[i]:bound[i + 1], :sp] = shared[i]
            ref[shared[i].long()] += bound[i + 1] - bound[i]
        table[:, sp:] = own_table[:, :width - sp]
        s.update(group_off=_i32(bound), shared_table=shared.contiguous().to(DEV), shared_pages=_i32([sp] * n_groups), sp=sp,
                 n_groups=n_groups, width_g=max(b - a for a, b in zip(bound, bound[1:])))
    s.update(own_pages=max(1, max(pages_of)), table=table.to(DEV), ref=ref.to(DEV),
             len=_i32([n if n < 0 else n + sp * page for n, _ in reqs]))
    s["k"], s["v"] = _kv(g, c, layers, n_pages)
    if own:
        s["cache"] = _handle(s, layers, n_pages, c, width)


def _some_tree(s, cpu, rows):
    """Parents of the packed rows: each node hangs on one of the four before it, the first on the cache."""
    _, j, ok, _, _ = _rows_of(s, rows)
    back = 1 + (torch.rand(rows, generator=cpu, dtype=torch.float64) * 4).int().to(DEV)
    return torch.where(ok & (j > 0), (j - back).clamp(min=0), -1).int()


def _pack(bits):
    """Truth values [..., V] as words of 32, rows of whole 16 bytes."""
    V = bits.shape[-1]
    words = (V + 127) // 128 * 4
    full = torch.zeros(bits.shape[:-1] + (words * 32,), dtype=torch.bool, device=bits.device)
    full[..., :V] = bits
    weight = (torch.ones((), dtype=torch.int64, device=bits.device) << torch.arange(32, device=bits.device)).int()
    return (full.unflatten(-1, (words, 32)).int() * weight).sum(-1, dtype=torch.int32)


def _unpack(words, V):
    at = torch.arange(V, device=words.device)
    return (words[..., at // 32] >> (at % 32).int()) & 1 != 0


def prepare(case, seed):
    c, g = case, _gen(seed)
    cpu = torch.Generator().manual_seed(int(seed) + 1)
    s = {"op": c["op"], "case": c}
    return {"attend": _prepare_attend, "rotary": _prepare_rotary, "target": _prepare_target, "history": _prepare_history,
            "tree": _prepare_tree}[c["op"]](s, c, g, cpu)


def _step(s, c, cpu):
    """The step's requests in a random order, and their offsets."""
    reqs = _requests(c)
    reqs = [reqs[i] for i in torch.randperm(len(reqs), generator=cpu).tolist()]
    lead = c.get("lead", 1)
    off = [0]
    for _, n in reqs:
        off.append(off[-1] + n - lead)
    s.update(lead=lead, max_new=c["K"] + lead, offsets=_i32(off), rows=off[-1] + lead * c["R"] + 2)  # two rows of nobody
    return reqs


def _prepare_attend(s, c, g, cpu):
    reqs = _step(s, c, cpu)
    _cache(s, c, g, cpu, reqs, 1)
    rows, H, D, t = s["rows"], c["H"], c["D"], DTYPES[c["dtype"]]
    s["anc"] = _plan(s, _some_tree(s, cpu, rows))[1]
    s["q"] = _normal(g, (rows, H, D), t)
    s["out"] = torch.zeros((rows, H, D), dtype=t, device=DEV)
    s["lse"] = torch.zeros((rows, H), dtype=torch.float32, device=DEV)
    s["scale"] = 1.0 / math.sqrt(D)
    if own:
        from confidence_scheduled_verification_amd import binding as B
        s["ws"] = B.cache_workspace(s["cache"], c["R"], H, s["max_new"], c["groups"])
    return s


def _prepare_rotary(s, c, g, cpu):
    reqs = _step(s, c, cpu)
    _cache(s, c, g, cpu, reqs, 1)
    rows, H, Hkv, D, t = s["rows"], c["H"], c["Hkv"], c["D"], DTYPES[c["dtype"]]
    s["depth"] = _plan(s, _some_tree(s, cpu, rows))[0] if c["lead"] else None
    qkv = _normal(g, (rows, (H + 2 * Hkv) * D), t)  # as one projection gives them
    s["q"] = qkv[:, :H * D].unflatten(1, (H, D))
    s["k_new"] = qkv[:, H * D:(H + Hkv) * D].unflatten(1, (Hkv, D))
    s["v_new"] = qkv[:, (H + Hkv) * D:].unflatten(1, (Hkv, D))
    s["q_out"] = torch.zeros((rows, H, D), dtype=t, device=DEV)
    s["attention"] = 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == "ramp" else 1.0
    if own:
        from confidence_scheduled_verification_amd import binding as B
        s["rotary"] = B.Rotary(c["dim"], c["base"], first=c["first"], interleaved=c["interleaved"], attention=s["attention"],
                               scaling=c["scaling"], factor=c["factor"], **SCALED.get(c["scaling"], {}))
    return s


# contexts stretched: frequencies between `low` and `high` turns over the original length are blended
SCALED = {"bands": dict(original=8192, low=1.0, high=4.0), "ramp": dict(original=4096, low=1.0, high=32.0)}


def _prepare_target(s, c, g, cpu):
    _step(s, c, cpu)
    R, V, rows = c["R"], c["V"], s["rows"]
    s["logits"] = (torch.randn((rows, V), generator=g, device=DEV, dtype=torch.float32) * 3.0).to(DTYPES[c["dtype"]])
    s["anc"] = _plan(s, _some_tree(s, cpu, rows))[1]
    s["node_tokens"] = _tokens(g, (max(1, rows),), V)
    prompt, answer = _tokens(g, (R, c["seen"]), V), _tokens(g, (R, 1 + c["seen"] // 4), V)
    count = torch.zeros((R, V), dtype=torch.int32, device=DEV)
    count.scatter_add_(1, answer.long(), torch.ones_like(answer))
    told = torch.zeros((R, V), dtype=torch.bool, device=DEV)
    told.scatter_(1, prompt.long(), True)
    s["count"], s["seen"] = count, torch.stack((_pack(told), _pack(count > 0)), 1)
    s["repetition"], s["presence"], s["frequency"] = (
        (lo + (hi - lo) * _uniform(g, (R,))).float() for lo, hi in ((0.9, 1.5), (-0.2, 1.0), (0.0, 0.5)))
    if c["biased"]:
        n = min(c["biased"], V)
        at = torch.sort(torch.rand((R, V), generator=g, device=DEV).topk(n, 1).indices, 1).values
        s["bias_off"] = _i32([n * r for r in range(R + 1)])
        s["bias_tok"], s["bias_val"] = at.int().reshape(-1), (torch.randn((R * n,), generator=g, device=DEV) * 2.0)
    if c["masks"]:
        n = c["masks"]
        allowed = _uniform(g, (n, V)) < c["allow"]
        s["allowed"] = _pack(allowed)
        pick = torch.randint(-1, n, (rows,), generator=cpu)  # -1: a row that no grammar binds
        s["allowed_row"] = _i32(pick)
    s["target"] = torch.full((rows,), -7, dtype=torch.int32, device=DEV)
    s["adjusted"] = torch.zeros_like(s["logits"]) if c["processed"] else None
    if own:
        from confidence_scheduled_verification_amd import binding as B
        s["history"] = B.History(R, V, seen=s["seen"], count=s["count"])
        s["ws"] = B.target_workspace(rows, V)
    return s


def _prepare_history(s, c, g, cpu):
    R, V = c["R"], c["V"]
    s["prompt"], s["answer"] = _tokens(g, (R, c["prompt"]), V), _tokens(g, (R, c["answer"]), V)
    s["prompt"][:, c["prompt"] - c["prompt"] // 8:][::2] = -1  # shorter prompts, padded
    s["rows"] = _i32(torch.randperm(R, generator=cpu))
    old = _tokens(g, (R, 3000), V)  # what the rows held for the requests before
    s["count"] = torch.zeros((R, V), dtype=torch.int32, device=DEV)
    s["count"].scatter_add_(1, old.long(), torch.ones_like(old))
    s["seen"] = torch.stack((_pack(s["count"] > 2), _pack(s["count"] > 0)), 1)
    if own:
        from confidence_scheduled_verification_amd import binding as B
        s["history"] = B.History(R, V, seen=s["seen"], count=s["count"])
    return s


def _prepare_tree(s, c, g, cpu):
    R, S, K, V = c["R"], c["S"], c["K"], c["V"]
    n = S * K
    s.update(lead=1, max_new=n + 1, rows=R * (n + 1))
    reqs = [(-1 if i < c["vacant"] else round(c["own_len"] * (i + 1) / R), n + 1) for i in torch.randperm(R, generator=cpu).tolist()]
    _cache(s, c, g, cpu, reqs, c["layers"])
    # chains that go with the first one for a while; the first one is the longest
    tokens = _tokens(g, (R, S, K), V)
    common = (_uniform(g, (R, S, 1)) * (K + 1)).int()
    tokens = torch.where(torch.arange(K, device=DEV) < common, tokens[:, :1], tokens)
    length = (_uniform(g, (R, S)) * (K + 1)).int()
    length[:, 0] = K
    s["tokens"], s["prefix_len"] = tokens.reshape(R * S, K).contiguous(), length.reshape(-1).contiguous()
    s["counts"], s["offsets"] = _i32([0] * R), _i32([0] * (R + 1))
    s["node_tokens"], s["parent"] = _i32([-1] * (R * n)), _i32([-1] * (R * (n + 1)))
    s["depth"], s["anc"] = _i32([0] * (R * (n + 1))), torch.zeros(R * (n + 1), dtype=torch.int64, device=DEV)
    s["accept_len"], s["next_prev0"] = _i32([0] * R), _i32([0] * R)
    s["path"], s["out_tokens"] = _i32([[0] * K] * R), _i32([[0] * (K + 1)] * R)
    # the target goes along one chain for some of its tokens
    t = {k: v.clone() if torch.is_tensor(v) else v for k, v in s.items() if k not in ("k", "v", "cache")}
    t["offsets"], t["parent"], t["node_tokens"], node = _merge(t)
    s["target"] = _tokens(g, (R * (n + 1),), V)
    which = (_uniform(g, (R,)) * S).long()
    upto = (_uniform(g, (R,)) * (1 + torch.gather(length, 1, which[:, None])[:, 0])).long()
    ri = torch.arange(R, device=DEV)
    along, chain = node[ri, which], tokens[ri, which]  # the nodes of that chain, and its tokens
    before = torch.cat((torch.zeros_like(along[:, :1]), along[:, :-1]), 1)
    take = torch.arange(K, device=DEV) < upto[:, None]
    row = t["offsets"][:-1, None] + ri[:, None] + before
    s["target"][row[take].long()] = chain[take].int()
    return s


# ---- the plain forms --------------------------------------------------------------------------------------------------------


def _rows_of(s, rows=None):
    """Request and place of each packed row, whether it belongs to one, and each request's start and count."""
    off, lead = s["offsets"].long(), s["lead"]
    R = off.shape[0] - 1
    start = off[:-1] + lead * torch.arange(R, device=DEV)
    count = off[1:] - off[:-1] + lead
    t = torch.arange(s["rows"] if rows is None else rows, device=DEV)
    r = (torch.searchsorted(start, t, right=True) - 1).clamp(0, R - 1)
    j = t - start[r]
    return r, j, j < count[r], start, count


def _padded(s, x, fill):
    """Packed rows as [R, max_new, ...], with `fill` where a request has fewer."""
    _, _, _, start, count = _rows_of(s)
    j = torch.arange(s["max_new"], device=DEV)
    at = (start[:, None] + j).clamp(max=s["rows"] - 1)
    there = (j < count[:, None]).reshape(at.shape + (1,) * (x.dim() - 1))
    return torch.where(there, x[at], torch.full((), fill, dtype=x.dtype, device=DEV))


def _plan(s, parent):
    """Depth and ancestors (bit j: node j, the row's own among them) of the packed rows; 0 for rows of nobody."""
    n = s["max_new"]
    p = _padded(s, parent, -1).long()
    up = (p[:, :, None] == torch.arange(n, device=DEV)).float() + torch.eye(n, device=DEV)
    up = (up @ up).clamp(max=1.0)  # closed over 2, 4, ... 64 steps
    up = (up @ up).clamp(max=1.0)
    up = (up @ up).clamp(max=1.0)
    up = (up @ up).clamp(max=1.0)
    up = (up @ up).clamp(max=1.0)
    up = (up @ up) > 0
    word = (up * (torch.ones((), dtype=torch.int64, device=DEV) << torch.arange(n, device=DEV))).sum(2)
    r, j, ok, _, _ = _rows_of(s)
    j = j.clamp(0, n - 1)
    return (up.sum(2, dtype=torch.int32)[r, j] - 1).clamp(min=0) * ok, word[r, j] * ok


def _gathered(s, ids):
    """K and V of pages ids [A, W] as [A, Hkv, W * page, D] in float32."""
    A = ids.shape[0]
    Hkv, D = s["k"].shape[2], s["v"].shape[4]
    ids = ids.clamp(min=0)
    k = s["k"][0][ids].permute(0, 2, 1, 3, 5, 4, 6).reshape(A, Hkv, -1, D).float()
    v = s["v"][0][ids].permute(0, 2, 1, 3, 5, 4).reshape(A, Hkv, -1, D).float()
    return k, v


def _attend(s):
    R, n = s["len"].shape[0], s["max_new"]
    H, D = s["q"].shape[1:]
    Hkv, page = s["k"].shape[2], s["case"]["page"]
    G = H // Hkv
    row_r, row_j, row_ok, _, _ = _rows_of(s)
    q = _padded(s, s["q"], 0).float().reshape(R, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, n * G, D) * s["scale"]
    ln = s["len"].long()
    sp = s.get("sp", 0)
    k, v = _gathered(s, s["table"][:, sp:sp + s["own_pages"]].long())
    x = q @ k.transpose(2, 3)
    past = sp * page + torch.arange(x.shape[3], device=DEV) - ln[:, None]  # below 0: the request's tokens, else its nodes
    node = past.clamp(0, 63)[:, None, :]
    bit = (_padded(s, s["anc"], 0)[:, :, None] >> node) & 1
    sees = ((past < 0)[:, None] | (past < n)[:, None] & (bit != 0)) & (ln >= 0)[:, None, None]
    x = x.reshape(R, Hkv, n, G, -1).masked_fill(~sees[:, None, :, None], -math.inf).reshape(x.shape)
    m = x.amax(3, keepdim=True)
    if sp:
        first, last = s["group_off"][:-1].long(), s["group_off"][1:].long()
        of = torch.searchsorted(last, torch.arange(R, device=DEV), right=True)
        within = torch.arange(R, device=DEV) - first[of]
        pick = (first[:, None] + torch.arange(s["width_g"], device=DEV)).clamp(max=R - 1)
        kg, vg = _gathered(s, s["shared_table"].long())
        qg = q[pick].permute(0, 2, 1, 3, 4).reshape(s["n_groups"], Hkv, -1, D)
        y = qg @ kg.transpose(2, 3)
        my = y.amax(3, keepdim=True)
        e = torch.exp(y - my)
        del y
        oy, ly, my = (p.reshape(s["n_groups"], Hkv, s["width_g"], n * G, -1)[of, :, within]
                      for p in (e @ vg, e.sum(3, keepdim=True), my))
        del e
        my = my.masked_fill((ln < 0)[:, None, None, None], -math.inf)
        top = torch.maximum(m, my)
    else:
        top = m
    safe = top.masked_fill(top == -math.inf, 0.0)
    e = torch.exp(x - safe)
    o, l = e @ v, e.sum(3, keepdim=True)
    if sp:
        w = torch.exp(my - safe)
        o, l = o + w * oy, l + w * ly
    o = torch.where(l > 0, o / l, torch.zeros((), device=DEV))
    lse = (safe + torch.log(l)).reshape(R, Hkv, n, G).permute(0, 2, 1, 3).reshape(R, n, H)
    o = o.reshape(R, Hkv, n, G, D).permute(0, 2, 1, 3, 4).reshape(R, n, H, D)
    jj = row_j.clamp(0, n - 1)
    s["out"].copy_(torch.where(row_ok[:, None, None], o[row_r, jj].to(s["out"].dtype), s["out"]))
    s["lse"].copy_(torch.where(row_ok[:, None], lse[row_r, jj], s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


def _frequencies(c):
    """Radians a token of each pair of dims, in 64 bits."""
    dim, base, factor = c["dim"], c["base"], c["factor"]
    i = torch.arange(dim // 2, dtype=torch.float64, device=DEV)
    f = torch.exp(-2.0 * i / dim * math.log(base))
    how = SCALED.get(c["scaling"])
    if c["scaling"] == "linear":
        return f / factor
    if c["scaling"] == "bands":
        turns = how["original"] * f / (2.0 * math.pi)
        keep = ((turns - how["low"]) / (how["high"] - how["low"])).clamp(0.0, 1.0)
        return f * (keep + (1.0 - keep) / factor)
    if c["scaling"] == "ramp":
        a, b = (dim * math.log(how["original"] / (x * 2.0 * math.pi)) / (2.0 * math.log(base)) for x in (how["high"], how["low"]))
        a, b = max(math.floor(a), 0), min(math.ceil(b), dim - 1)
        lost = ((i - a) / max(b - a, 0.001)).clamp(0.0, 1.0)
        return f * (1.0 - lost + lost / factor)
    return f


def _turned(s, x, pos):
    """Rows [n, heads, D] turned to their positions [n], in float32, rounded once."""
    c = s["case"]
    first, dim, half = c["first"], c["dim"], c["dim"] // 2
    angle = pos.double()[:, None] * _frequencies(c)  # far positions lose their angle in 32 bits
    co, si = (f(angle).float()[:, None] * s["attention"] for f in (torch.cos, torch.sin))
    x = x.float()
    part = x[:, :, first:first + dim]
    a, b = (part[:, :, 0::2], part[:, :, 1::2]) if c["interleaved"] else (part[:, :, :half], part[:, :, half:])
    a, b = a * co - b * si, a * si + b * co
    part = torch.stack((a, b), 3).flatten(2) if c["interleaved"] else torch.cat((a, b), 2)
    return torch.cat((x[:, :, :first], part, x[:, :, first + dim:]), 2).to(s["k"].dtype)


def _rotary(s):
    row_r, row_j, ok, _, _ = _rows_of(s)
    ln = s["len"].long()
    page = s["case"]["page"]
    t = (ok & (ln[row_r] >= 0)).nonzero()[:, 0]
    r = row_r[t]
    turn = ln[r] + (row_j if s["depth"] is None else s["depth"].long())[t]
    p = ln[r] + row_j[t]
    ids = s["table"][r, p // page].long()
    blk, slot = p % page // 16, p % 16
    D = s["v"].shape[4]
    s["q_out"][t] = _turned(s, s["q"][t], turn)
    s["k"][0][ids, :, blk, :, slot] = _turned(s, s["k_new"][t], turn).unflatten(2, (D // 8, 8))
    s["v"][0][ids, :, blk, :, slot] = s["v_new"][t]
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _target(s):
    c = s["case"]
    R, V, rows, n = c["R"], c["V"], s["rows"], s["max_new"]
    r, j, ok, start, _ = _rows_of(s)
    x = s["logits"].double()  # in 64 bits: which of two near values is larger decides
    # the drafts that a row's node has behind it, counted as if they had been answered
    nodes = torch.arange(n, device=DEV)
    on = ((s["anc"][:, None] >> nodes) & 1 != 0) & (nodes >= s["lead"]) & ok[:, None]
    at = (s["offsets"][r].long()[:, None] + nodes - s["lead"]).clamp(0, s["node_tokens"].shape[0] - 1)
    times = torch.zeros((rows, V), dtype=torch.int32, device=DEV)
    times.scatter_add_(1, s["node_tokens"][at].long(), on.int())
    times += s["count"][r]
    seen = _unpack(s["seen"][:, 0], V)[r] | (times > 0)
    rep = s["repetition"].double()[r][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"].double()[r][:, None] * times
    x = x - s["presence"].double()[r][:, None] * (times > 0)
    if c["biased"]:
        bias = torch.zeros((R, V), dtype=torch.float64, device=DEV)
        bias.scatter_(1, s["bias_tok"].long().reshape(R, -1), s["bias_val"].double().reshape(R, -1))
        x = x + bias[r]
    if c["masks"]:
        pick = s["allowed_row"].long()
        free = _unpack(s["allowed"], V)[pick.clamp(min=0)] | (pick < 0)[:, None]
        x = x.masked_fill(~free, -math.inf)
    top = x.amax(1, keepdim=True)
    best = torch.where(x == top, torch.arange(V, device=DEV), V).amin(1)
    s["target"].copy_(torch.where(ok, best.int(), s["target"]))
    if s["adjusted"] is None:
        return {"target": s["target"]}
    s["adjusted"].copy_(torch.where(ok[:, None], x.to(s["adjusted"].dtype), s["adjusted"]))
    return {"target": s["target"], "adjusted": s["adjusted"]}


def _history(s):
    R, V = s["case"]["R"], s["case"]["V"]
    rows = s["rows"].long()
    prompt, answer = s["prompt"].long(), s["answer"].long()
    told = torch.zeros((R, V), dtype=torch.int32, device=DEV)
    told.scatter_add_(1, prompt.clamp(min=0), (prompt >= 0).int())
    count = torch.zeros((R, V), dtype=torch.int32, device=DEV)
    count.scatter_add_(1, answer, torch.ones_like(answer, dtype=torch.int32))
    s["count"][rows] = count
    s["seen"][rows] = torch.stack((_pack(told > 0), _pack(count > 0)), 1)
    return {"seen": s["seen"], "count": s["count"]}


def _merge(s):
    """The chains [R, S, K] of the first prefix_len tokens each as one tree a request, equal beginnings taken
    once: offsets, parents and tokens of the nodes, and which node each chain's token is."""
    c = s["case"]
    R, S, K = c["R"], c["S"], c["K"]
    tok, ln = s["tokens"].reshape(R, S, K), s["prefix_len"].reshape(R, S)
    valid = torch.arange(K, device=DEV) < ln[:, :, None]
    same = (tok[:, :, None] == tok[:, None]) & valid[:, :, None] & valid[:, None]
    same = same.int().cumprod(3) != 0  # [r, s, s', i]: s and s' begin with the same i + 1 tokens
    first = same.int().argmax(2)       # the lowest of them
    new = valid & (first == torch.arange(S, device=DEV)[:, None])
    number = new.reshape(R, -1).cumsum(1).reshape(R, S, K)
    node = torch.gather(number, 1, first)
    parent = torch.cat((torch.zeros_like(node[:, :, :1]), node[:, :, :-1]), 2)
    counts = new.sum((1, 2), dtype=torch.int32)
    offsets = torch.cat((torch.zeros_like(counts[:1]), counts.cumsum(0, dtype=torch.int32)))
    r = torch.arange(R, device=DEV)[:, None, None].expand_as(new)
    at = offsets[r].long() + number - 1
    s["counts"].copy_(counts)
    s["node_tokens"][at[new]] = tok[new]
    s["parent"][offsets[:-1].long() + r[:, 0, 0]] = -1
    s["parent"][(at + r + 1)[new]] = parent[new].int()
    return offsets, s["parent"], s["node_tokens"], node


def _tree(s):
    c = s["case"]
    R, n, K, page = c["R"], s["max_new"], c["K"], c["page"]
    s["offsets"].copy_(_merge(s)[0])
    depth, anc = _plan(s, s["parent"])
    s["depth"].copy_(depth)
    s["anc"].copy_(anc)
    # a node is accepted if its token and those of all before it are the target's choice there
    parent = _padded(s, s["parent"], -1).long()
    target = _padded(s, s["target"], -1)
    _, _, _, start, count = _rows_of(s)
    nodes = torch.arange(n, device=DEV)
    at = (s["offsets"][:-1].long()[:, None] + nodes - 1).clamp(0, s["node_tokens"].shape[0] - 1)
    token = s["node_tokens"][at]
    there = nodes < count[:, None]
    hit = there & ((nodes == 0) | (torch.gather(target, 1, parent.clamp(min=0)) == token))
    on = ((_padded(s, s["anc"], 0)[:, :, None] >> nodes) & 1) != 0
    good = there & (~on | hit[:, None]).all(2)
    deep = torch.where(good, _padded(s, s["depth"], 0), -1)
    last = deep.argmax(1)
    accept = deep.amax(1)
    ri = torch.arange(R, device=DEV)
    way = on[ri, last] & (nodes > 0)
    order = torch.where(way, nodes, n).sort(1).values[:, :K]
    step = torch.arange(K, device=DEV)
    path = torch.where(step < accept[:, None], order, -1)
    bonus = target[ri, last]
    drafts = torch.gather(token, 1, path.clamp(min=0))
    out = torch.cat((torch.where(path >= 0, drafts, -1), torch.full((R, 1), -1, dtype=torch.int32, device=DEV)), 1)
    out[ri, accept.long()] = bonus
    s["accept_len"].copy_(accept)
    s["path"].copy_(path)
    s["next_prev0"].copy_(bonus)
    s["out_tokens"].copy_(out)
    # the path's keys and values behind the first row's
    ln = s["len"].long()
    r, i = ((path >= 0) & (ln >= 0)[:, None]).nonzero(as_tuple=True)
    a, b = ln[r] + path[r, i], ln[r] + 1 + i
    pa, pb = s["table"][r, a // page].long(), s["table"][r, b // page].long()
    s["k"][:, pb, :, b % page // 16, :, b % 16] = s["k"][:, pa, :, a % page // 16, :, a % 16]
    s["v"][:, pb, :, b % page // 16, :, b % 16] = s["v"][:, pa, :, a % page // 16, :, a % 16]
    return _tree_outputs(s)


def _tree_outputs(s):
    return {k: s[k] for k in ("counts", "offsets", "node_tokens", "parent", "depth", "anc", "accept_len", "path", "next_prev0",
                              "out_tokens", "k", "v")}


def run(s):
    if own:
        return _own(s)
    return {"attend": _attend, "rotary": _rotary, "target": _target, "history": _history, "tree": _tree}[s["op"]](s)


def _own(s):
    from confidence_scheduled_verification_amd import binding as B
    op = s["op"]
    if op == "attend":
        shared = (s["group_off"], s["shared_table"], s["shared_pages"]) if "sp" in s else None
        B.dspark_cache_attend_tree(s["cache"], 0, s["q"], s["offsets"], s["lead"], s["max_new"], s["anc"], s["scale"], s["out"],
                                   lse=s["lse"], shared=shared, ws=s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "rotary":
        B.dspark_cache_append_rotary(s["cache"], 0, s["rotary"], s["q"], s["q_out"], s["k_new"], s["v_new"], s["offsets"],
                                     s["lead"], s["max_new"], depth=s["depth"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    if op == "target":
        bias = (s["bias_off"], s["bias_tok"], s["bias_val"]) if "bias_off" in s else None
        B.dspark_target_tokens(s["logits"], s["offsets"], s["lead"], s["max_new"], s["target"], history=s["history"],
                               penalties=(s["repetition"], s["presence"], s["frequency"]), node_tokens=s["node_tokens"],
                               anc=s["anc"], bias=bias, allowed=s.get("allowed"), allowed_row=s.get("allowed_row"),
                               adjusted=s["adjusted"], ws=s["ws"])
        return {"target": s["target"]} if s["adjusted"] is None else {"target": s["target"], "adjusted": s["adjusted"]}
    if op == "history":
        B.dspark_history_clear(s["history"], s["rows"])
        B.dspark_history_add(s["history"], s["prompt"], answered=False, rows=s["rows"])
        B.dspark_history_add(s["history"], s["answer"], answered=True, rows=s["rows"])
        return {"seen": s["seen"], "count": s["count"]}
    B.dspark_tree_merge(s["tokens"], s["prefix_len"], s["case"]["S"], s["counts"], s["offsets"], s["node_tokens"], s["parent"])
    B.dspark_tree_plan(s["parent"], s["offsets"], s["lead"], s["max_new"], s["depth"], s["anc"])
    B.dspark_accept_tree(s["node_tokens"], s["offsets"], s["parent"], s["target"], s["accept_len"], s["path"], s["next_prev0"],
                         s["out_tokens"])
    B.dspark_cache_keep_path(s["cache"], s["path"], s["accept_len"], s["lead"])
    return _tree_outputs(s)


# ---- the definitions, in 64 bits --------------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    f = {"attend": _exact_attend, "rotary": _exact_rotary, "target": _exact_target, "history": _exact_history,
         "tree": _exact_tree}[s["op"]]
    return f(s, case)


def _token(c, p):
    """Where position p of a row lies: page in the row, block and slot in the page."""
    return p // c["page"], p % c["page"] // 16, p % 16


def _exact_attend(s, c):
    out, lse = s["out"].double(), s["lse"].double()
    off, ln, table, anc = s["offsets"].tolist(), s["len"].tolist(), s["table"].long(), s["anc"].tolist()
    H, Hkv, D, page = c["H"], c["Hkv"], c["D"], c["page"]
    for r in range(c["R"]):
        a, b = off[r] + r, off[r + 1] + r + 1
        if ln[r] < 0:
            out[a:b], lse[a:b] = 0.0, -math.inf
            continue
        T = ln[r] + b - a
        ids = table[r, :-(-T // page)]
        hidden = torch.tensor([[not anc[t] >> j & 1 for j in range(b - a)] for t in range(a, b)], device=DEV)
        for h in range(Hkv):  # K [T, D] and V [D, T] of one head
            K = s["k"][0, ids, h].double().movedim(3, 2).flatten(3).flatten(0, 2)[:T]
            V = s["v"][0, ids, h].double().movedim(2, 0).flatten(1)[:, :T]
            hs = slice(h * (H // Hkv), (h + 1) * (H // Hkv))
            z = torch.tensordot(s["q"][a:b, hs].double(), K, dims=([2], [1])) * (1.0 / math.sqrt(D))
            z[:, :, ln[r]:] = z[:, :, ln[r]:].masked_fill(hidden[:, None], -math.inf)
            ls = torch.logsumexp(z, 2)
            lse[a:b, hs] = ls
            out[a:b, hs] = torch.tensordot(torch.exp(z - ls[:, :, None]), V, dims=([2], [1]))
    return {"out": out, "lse": lse}


def _exact_frequency(c, i):
    f = c["base"] ** (-2.0 * i / c["dim"])
    if c["scaling"] == "linear":
        return f / c["factor"]
    if c["scaling"] == "bands":
        wave, how = 2.0 * math.pi / f, SCALED["bands"]
        if wave > how["original"] / how["low"]:
            return f / c["factor"]
        if wave < how["original"] / how["high"]:
            return f
        t = (how["original"] / wave - how["low"]) / (how["high"] - how["low"])
        return (1.0 - t) * f / c["factor"] + t * f
    if c["scaling"] == "ramp":
        how = SCALED["ramp"]
        lo, hi = (c["dim"] * math.log(how["original"] / (2.0 * math.pi * x)) / (2.0 * math.log(c["base"]))
                  for x in (how["high"], how["low"]))
        lo, hi = max(0, math.floor(lo)), min(c["dim"] - 1, math.ceil(hi))
        t = min(1.0, max(0.0, (i - lo) / max(0.001, hi - lo)))
        return t * f / c["factor"] + (1.0 - t) * f
    return f


def _exact_rotary(s, c):
    off, ln, table = s["offsets"].tolist(), s["len"].tolist(), s["table"].tolist()
    depth = None if s["depth"] is None else s["depth"].tolist()
    f = torch.tensor([_exact_frequency(c, i) for i in range(c["dim"] // 2)], dtype=torch.float64, device=DEV)
    at, turn, where = [], [], []
    for r in range(c["R"]):
        a, b = off[r] + c["lead"] * r, off[r + 1] + c["lead"] * (r + 1)
        for t in range(a, b if ln[r] >= 0 else a):
            i, blk, slot = _token(c, ln[r] + t - a)
            at.append(t)
            turn.append(ln[r] + (t - a if depth is None else depth[t]))
            where.append((table[r][i], blk, slot))
    q, k, v = s["q_out"].double(), s["k"].double(), s["v"].double()
    if not at:
        return {"q": q, "k": k, "v": v}
    at = torch.tensor(at, device=DEV)
    page, blk, slot = torch.tensor(where, device=DEV).T
    turn = torch.exp(1j * torch.tensor(turn, dtype=torch.float64, device=DEV)[:, None, None] * f) * s["attention"]
    lo, dim = c["first"], c["dim"]

    def turned(x):
        x = x[at].double()
        pairs = slice(lo, lo + dim, 2), slice(lo + 1, lo + dim, 2)
        if not c["interleaved"]:
            pairs = slice(lo, lo + dim // 2), slice(lo + dim // 2, lo + dim)
        z = torch.complex(x[:, :, pairs[0]].contiguous(), x[:, :, pairs[1]].contiguous()) * turn
        x[:, :, pairs[0]], x[:, :, pairs[1]] = z.real, z.imag
        return x

    q[at] = turned(s["q"])
    kn, vn = turned(s["k_new"]), s["v_new"][at].double()
    for d in range(c["D"]):
        k[0, page, :, blk, d // 8, slot, d % 8] = kn[:, :, d]
        v[0, page, :, blk, d, slot] = vn[:, :, d]
    return {"q": q, "k": k, "v": v}


def _bits(words, V):
    w = words.long().cpu() & 0xFFFFFFFF
    return torch.stack([(w >> i) & 1 for i in range(32)], -1).flatten(-2)[..., :V].bool().to(DEV)


def _exact_target(s, c):
    V, off = c["V"], s["offsets"].tolist()
    target, adjusted = s["target"].clone(), None if s["adjusted"] is None else s["adjusted"].double()
    prompt = _bits(s["seen"][:, 0], V)
    allowed = _bits(s["allowed"], V) if c["masks"] else None
    pick = s["allowed_row"].tolist() if c["masks"] else None
    node, anc = s["node_tokens"].tolist(), s["anc"].tolist()
    rep, pres, freq = (s[k].double().tolist() for k in ("repetition", "presence", "frequency"))
    n = min(c["biased"], V)
    for r in range(c["R"]):
        a, b = off[r] + r, off[r + 1] + r + 1
        for t in range(a, b):
            x = s["logits"][t].double()
            times = s["count"][r].double()
            for j in range(1, b - a):
                if anc[t] >> j & 1:
                    times[node[off[r] + j - 1]] += 1
            told = prompt[r] | (times > 0)
            x[told] = torch.where(x > 0, x / rep[r], x * rep[r])[told]
            x -= freq[r] * times
            x[times > 0] -= pres[r]
            if n:
                x[s["bias_tok"][n * r:n * r + n].long()] += s["bias_val"][n * r:n * r + n].double()
            if c["masks"] and pick[t] >= 0:
                x[~allowed[pick[t]]] = -math.inf
            target[t] = (x == x.max()).nonzero()[0, 0]
            if adjusted is not None:
                adjusted[t] = x
    return {"target": target} if adjusted is None else {"target": target, "adjusted": adjusted}


def _exact_history(s, c):
    V, seen, count = c["V"], s["seen"].clone(), torch.zeros_like(s["count"])
    bit = torch.tensor([1 << i if i < 31 else -(1 << 31) for i in range(32)], dtype=torch.int32, device=DEV)

    def words(ids):
        full = torch.zeros(seen.shape[2] * 32, dtype=torch.int32, device=DEV)
        full[ids] = 1
        return (full.view(-1, 32) * bit).sum(1, dtype=torch.int32)

    for i, r in enumerate(s["rows"].tolist()):
        p, a = s["prompt"][i], s["answer"][i]
        n = torch.bincount(a.long(), minlength=V)
        count[r] = n
        seen[r, 0], seen[r, 1] = words(p[p >= 0].long()), words(n.nonzero()[:, 0])
    return {"seen": seen, "count": count}


def _exact_tree(s, c):
    R, S, K = c["R"], c["S"], c["K"]
    tokens, ln = s["tokens"].reshape(R, S, K).tolist(), s["prefix_len"].reshape(R, S).tolist()
    target, kept, table = s["target"].tolist(), s["len"].tolist(), s["table"].tolist()
    got = {k: s[k].tolist() for k in ("counts", "offsets", "node_tokens", "parent", "depth", "anc", "accept_len", "path", "next_prev0",
                                      "out_tokens")}
    moves = []
    for r in range(R):
        names, parent, toks = {(): 0}, [-1], []
        for chain, n in zip(tokens[r], ln[r]):
            for i in range(n):
                if tuple(chain[:i + 1]) not in names:
                    names[tuple(chain[:i + 1])] = len(parent)
                    parent.append(names[tuple(chain[:i])])
                    toks.append(chain[i])
        o = got["offsets"][r]
        row = o + r
        got["counts"][r], got["offsets"][r + 1] = len(toks), o + len(toks)
        got["node_tokens"][o:o + len(toks)] = toks
        got["parent"][row:row + len(parent)] = parent
        for j, p in enumerate(parent):
            got["depth"][row + j] = got["depth"][row + p] + 1 if p >= 0 else 0
            word = (got["anc"][row + p] if p >= 0 else 0) | 1 << j
            got["anc"][row + j] = word - (1 << 64) if word >> 63 == 1 else word
        way, prefix = [], ()
        while len(way) < K:
            prefix += (target[row + (way[-1] if way else 0)],)
            if prefix not in names:
                break
            way.append(names[prefix])
        bonus = target[row + (way[-1] if way else 0)]
        got["accept_len"][r], got["next_prev0"][r] = len(way), bonus
        got["path"][r] = way + [-1] * (K - len(way))
        got["out_tokens"][r] = [toks[j - 1] for j in way] + [bonus] + [-1] * (K - len(way))
        if kept[r] >= 0:
            moves += [(r, kept[r] + j, kept[r] + 1 + i) for i, j in enumerate(way)]
    got = {k: torch.tensor(v, dtype=s[k].dtype, device=DEV) for k, v in got.items()}
    k, v = s["k"].clone(), s["v"].clone()
    for r, a, b in moves:  # in this order a token is read before another takes its place
        (ia, ba, sa), (ib, bb, sb) = _token(c, a), _token(c, b)
        k[:, table[r][ib], :, bb, :, sb] = k[:, table[r][ia], :, ba, :, sa]
        v[:, table[r][ib], :, bb, :, sb] = v[:, table[r][ia], :, ba, :, sa]
    return {**got, "k": k, "v": v}
