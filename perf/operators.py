"""Cases of the drafted-tree operators: attention of a tree of drafted tokens
over the shared caches (lora_attn_tree), per-head norms of queries and keys
with the rotation and the cache rows (lora_qk_norm_rope), and the low-rank
products of tokens grouped by agent in ragged segments (lora_grouped_delta).

`run` computes one pass in plain torch operations (fp32, angles in fp64), or,
with `own` true, through the library's entry points.  `exact` computes the same
outputs from the definitions in fp64.
"""
import math

import torch

own = False

DEV = "cuda"
STD = 1.28          # 0.02 * sqrt(4096): the standard deviation of X W in the seeded workloads
B_STD = 0.02        # up- and down-projections
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _tree(name, **kw):
    c = dict(name=name, op="tree", dtype="bf16", seqs=1, agents=3, heads=32, kv=8, d=128, r=16,
             ctx=8192, nodes=16, per_agent=False, keys=True, ragged=False, base=500000.0)
    c.update(kw)
    return c


def _norm(name, **kw):
    c = dict(name=name, op="norm", dtype="bf16", seqs=1, agents=3, heads=32, kv=8, d=128,
             ctx=1024, tokens=16, tree=True, per_agent=False, weights=True, ragged=False,
             base=500000.0)
    c.update(kw)
    return c


def _grouped(name, **kw):
    c = dict(name=name, op="grouped", dtype="bf16", agents=3, tokens=48, hidden=4096, out=4096,
             r=16, segs=3, shared=False, skip=False)
    c.update(kw)
    return c


def listed():
    return [
        # the tiny fp32 layer: an exact-arithmetic check path, one short tree per agent
        _tree("tree_fp32_tiny", dtype="fp32", agents=2, heads=4, kv=2, d=64, r=8, ctx=256,
              nodes=8, base=10000.0),
        # one request's verification step: 16 drafted nodes, three agents on one trajectory
        _tree("tree_8k"),
        # a batch of requests of odd lengths, every agent with a tree of its own, rank 64
        _tree("tree_odd_batch", seqs=3, agents=4, r=64, ctx=3001, nodes=13, per_agent=True,
              ragged=True),
        # keys shared outright (LoRA on queries and values only), a full 64-node tree
        _tree("tree_qv_16k", agents=3, ctx=16384, nodes=64, keys=False),
        # a serving batch of long contexts: 5 agents, rank 32, 32 nodes each
        _tree("tree_32k_batch", seqs=4, agents=5, r=32, ctx=32768, nodes=32, per_agent=True),
        # the rows of one verification step: latency only
        _norm("norm_tree"),
        # a prompt chunk of an odd length for a batch, no tree
        _norm("norm_chunk", seqs=2, agents=3, tokens=1021, tree=False, ragged=True, ctx=2000),
        # a long prompt chunk, four agents
        _norm("norm_long", agents=4, tokens=4096, tree=False, ctx=4096),
        # one verification step's tokens, three agents of 16 tokens
        _grouped("grouped_step"),
        # fp32 layer, a few ragged segments
        _grouped("grouped_fp32", dtype="fp32", agents=2, tokens=37, hidden=256, out=256, r=8,
                 segs=4),
        # a mixed batch of odd segments, one agent without tokens, some tokens without adapter
        _grouped("grouped_odd", agents=5, tokens=1501, out=1024, r=32, segs=9, skip=True),
        # a large prompt batch, rank 64
        _grouped("grouped_large", agents=4, tokens=16384, r=64, segs=4),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "norm", "grouped"])
    dtype = "fp32" if rng.random() < 0.15 else "bf16"
    d = 64 if rng.random() < 0.2 else 128
    if op == "tree":
        kv = rng.choice([1, 2, 4, 8])
        c = _tree("", dtype=dtype, kv=kv, heads=kv * rng.choice([1, 2, 3, 4, 4, 7, 8]), d=d,
                  r=rng.choice([8, 16, 16, 32, 64]), agents=rng.randint(1, 5),
                  nodes=_logint(rng, 1, 64), per_agent=rng.random() < 0.5,
                  keys=rng.random() < 0.75, ragged=rng.random() < 0.5,
                  base=rng.choice([10000.0, 500000.0]))
        plain = dtype == "bf16" and d == 128 and c["r"] > 8
        c["ctx"] = _logint(rng, 1, 32768 if plain else 4096)
        # at most the largest listed case's keys x agents x KV heads, in blocks of 128 query rows
        blocks = -(-c["nodes"] * c["heads"] // (kv * 128))
        cap = 5242880 if plain else 262144
        c["ctx"] = min(c["ctx"], cap // (c["agents"] * kv * blocks))
        c["seqs"] = _logint(rng, 1, max(1, min(16, cap // (c["ctx"] * c["agents"] * kv * blocks))))
    elif op == "norm":
        kv = rng.choice([1, 2, 4, 8])
        c = _norm("", dtype=dtype, kv=kv, heads=kv * rng.choice([1, 2, 3, 4, 7]), d=d,
                  agents=rng.randint(1, 4), tree=rng.random() < 0.5,
                  weights=rng.random() < 0.8, ragged=rng.random() < 0.5,
                  ctx=_logint(rng, 1, 32768), base=rng.choice([10000.0, 500000.0]))
        c["tokens"] = _logint(rng, 1, 64 if c["tree"] else 4096)
        c["per_agent"] = c["tree"] and rng.random() < 0.5
        c["seqs"] = _logint(rng, 1, max(1, min(8, 4096 // c["tokens"])))
    else:
        c = _grouped("", dtype=dtype, agents=rng.randint(1, 8), tokens=_logint(rng, 1, 16384),
                     hidden=8 * _logint(rng, 8, 512), out=8 * _logint(rng, 8, 512),
                     r=rng.choice([8, 16, 32, 64]), segs=rng.randint(1, 16),
                     shared=rng.random() < 0.3, skip=rng.random() < 0.3)
        if dtype == "fp32":
            c["tokens"] = min(c["tokens"], 2048)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std, dt):
    return torch.randn(shape, generator=g, device=DEV).mul_(std).to(dt)


def _parents(g, shape, n):
    """Random trees: node j hangs below the context (about one in five) or an earlier node."""
    j = torch.arange(n, device=DEV)
    u = torch.rand((*shape, n), generator=g, device=DEV)
    p = (torch.rand((*shape, n), generator=g, device=DEV) * j).floor()
    return torch.where((u < 0.2) | (j == 0), -torch.ones_like(p), p).to(torch.int32)


def _lengths(g, c, n, lo, hi):
    if not c["ragged"]:
        return torch.full((n,), hi, dtype=torch.int32, device=DEV)
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV, dtype=torch.int32)


def prepare(case, seed):
    c, g = case, _gen(seed)
    dt = DTYPES[c["dtype"]]
    st = {"case": c}
    if c["op"] == "grouped":
        T, H, N, r = c["tokens"], c["hidden"], c["out"], c["r"]
        a_std = B_STD if dt == torch.bfloat16 else 1 / math.sqrt(H)
        st["x"] = _normal(g, (T, H), 1.0, dt)
        st["y"] = _normal(g, (T, N), STD, dt)
        st["A"] = _normal(g, (H, r) if c["shared"] else (c["agents"], H, r), a_std, dt)
        st["B"] = _normal(g, (c["agents"], r, N), a_std, dt)
        st["out"] = torch.zeros_like(st["y"])
        cuts = torch.randint(0, T + 1, (c["segs"] - 1,), generator=g, device=DEV).sort().values
        if c["segs"] == c["agents"] and not c["skip"]:   # equal shares
            cuts = torch.arange(1, c["segs"], device=DEV) * T // c["segs"]
        st["seg_start"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)]).to(torch.int32)
        ag = torch.arange(c["segs"], device=DEV) % c["agents"]
        if c["skip"]:                                    # every third segment has no adapter
            ag = torch.where(torch.arange(c["segs"], device=DEV) % 3 == 2, -1, ag)
        st["seg_agent"] = ag.to(torch.int32)
        st["scale"] = 2.0
        if own:
            from rank_attention_b200 import lora_attn as la
            st["args"] = la.make_grouped_args(st["x"], st["A"], st["B"], st["y"], st["out"],
                                              st["seg_start"], st["seg_agent"],
                                              lora_scale=st["scale"])
        return st
    S, A, kv, d = c["seqs"], c["agents"], c["kv"], c["d"]
    n = c["nodes"] if c["op"] == "tree" else c["tokens"]
    trees = A if c["per_agent"] else 1
    L = c["ctx"] + trees * n
    cap = (L + 15) // 16 * 16                            # rows allocated: a few stale ones behind
    st["max_kv_len"] = L
    st["k_base"] = _normal(g, (S, kv, cap, d), STD, dt)
    st["v_base"] = _normal(g, (S, kv, cap, d), STD, dt)
    st["kv_len"] = _lengths(g, c, S, c["ctx"] // 2, c["ctx"])
    if c["op"] == "tree" or c["tree"]:
        st["parent"] = _parents(g, (S, trees), n)
        st["tree_len"] = _lengths(g, c, S * trees, 1, n).view(S, trees)
    else:
        st["parent"] = None
        st["tree_len"] = _lengths(g, c, S, 1, n).view(S, 1)
    if c["op"] == "tree":
        st["lr"] = _normal(g, (S, cap, 2 * c["r"]), STD, dt)
        b = B_STD if dt == torch.bfloat16 else 1 / math.sqrt(c["r"])
        st["B_k"] = _normal(g, (A, c["r"], kv * d), b, dt) if c["keys"] else None
        st["B_v"] = _normal(g, (A, c["r"], kv * d), b, dt)
        st["q"] = _normal(g, (S, A, n, c["heads"], d), STD, dt)
        st["out"] = torch.zeros_like(st["q"])
        st["scale"] = 2.0
        if own:
            from rank_attention_b200 import lora_attn as la
            st["args"] = la.make_args(st["k_base"], st["v_base"], st["lr"], st["B_k"], st["B_v"],
                                      st["q"], st["out"], lora_scale=st["scale"],
                                      rope_base=c["base"], kv_len=st["kv_len"],
                                      max_kv_len=st["max_kv_len"])
            st["tree"] = la.make_tree_args(st["parent"], st["tree_len"])
    else:
        st["q"] = _normal(g, (S, A, n, c["heads"], d), STD, dt)
        st["k"] = _normal(g, (S, trees, n, kv, d), STD, dt)
        st["v"] = _normal(g, (S, trees, n, kv, d), STD, dt)
        w = c["weights"]
        st["w_q"] = (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(dt) if w else None
        st["w_k"] = (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(dt) if w else None
        st["out"] = torch.zeros_like(st["q"])
        if own:
            from rank_attention_b200 import lora_attn as la
            st["args"] = la.make_qk_args(st["q"], st["k"], st["v"], st["w_q"], st["w_k"],
                                         st["out"], st["k_base"], st["v_base"], st["kv_len"],
                                         eps=EPS, rope_base=c["base"],
                                         max_kv_len=st["max_kv_len"])
            st["tree"] = la.make_tree_args(st["parent"], st["tree_len"])
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    if own:
        return _run_own(state)
    return {"tree": _tree_plain, "norm": _norm_plain, "grouped": _grouped_plain}[state["case"]["op"]](state)


def _run_own(state):
    from rank_attention_b200 import lora_attn as la
    op = state["case"]["op"]
    if op == "tree":
        la.lora_attn_tree(state["args"], state["tree"])
        return {"out": state["out"]}
    if op == "norm":
        la.lora_qk_norm_rope(state["args"], state["tree"])
        return {"q": state["out"], "k": state["k_base"], "v": state["v_base"]}
    la.lora_grouped_delta(state["args"])
    return {"out": state["out"]}


def _ancestors(parent):
    """[.., n, n] truth values: node j sees node i (its ancestors and itself)."""
    n = parent.shape[-1]
    i = torch.arange(n, device=parent.device)
    step = (parent[..., :, None] == i) | (i[:, None] == i)
    return torch.linalg.matrix_power(step.double(), max(n - 1, 1)) > 0


def _angles(pos, d, base):
    i = torch.arange(d // 2, device=pos.device, dtype=torch.float64)
    a = pos.double()[..., None] * torch.pow(torch.tensor(base, dtype=torch.float64, device=pos.device), -2 * i / d)
    return torch.cos(a).float(), torch.sin(a).float()


def _rotate(x, cos, sin):
    h = x.shape[-1] // 2
    x1, x2 = x[..., :h], x[..., h:]
    return torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], dim=-1)


def _tree_plain(st):
    c = st["case"]
    S, A, n, kv, d, r = c["seqs"], c["agents"], c["nodes"], c["kv"], c["d"], c["r"]
    g = c["heads"] // kv
    L, trees = st["max_kv_len"], st["parent"].shape[1]
    sees = _ancestors(st["parent"])                                   # [S, trees, n, n]
    depth = sees.sum(-1) - 1
    C = st["kv_len"].long()
    row = torch.arange(L, device=DEV)
    node = row - C[:, None]                                           # [S, L], < 0 in the context
    t = torch.arange(trees, device=DEV)
    j = (node[:, None] - t[:, None] * n)                              # [S, trees, L]
    drafted = (j >= 0) & (j < n)
    jc = j.clamp(0, n - 1)
    pos = torch.where(drafted, C[:, None, None] + depth.gather(2, jc), row)   # [S, trees, L]
    vis = (node[:, None] < 0)[:, :, None] | (
        drafted[:, :, None] & sees.gather(3, jc[:, :, None].expand(S, trees, n, L)))  # [S, trees, n, L]
    vis = vis.expand(S, A, n, L)
    lr = st["lr"][:, :L].float()
    K = st["k_base"][:, :, :L].float()[:, None]                       # [S, 1, kv, L, d]
    if c["keys"]:
        cos, sin = _angles(pos, d, c["base"])                         # [S, trees, L, d/2]
        B = st["B_k"].float().view(A, r, kv, d).permute(0, 2, 1, 3)   # [A, kv, r, d]
        delta = st["scale"] * (lr[:, None, None, :, :r] @ B)          # [S, A, kv, L, d]
        K = K + _rotate(delta, cos[:, :, None], sin[:, :, None])
        del delta
    q = st["q"].float().view(S, A, n, kv, g, d).permute(0, 1, 3, 2, 4, 5).reshape(S, A, kv, n * g, d)
    s = (q @ K.transpose(-1, -2)) * (1 / math.sqrt(d))                # [S, A, kv, n g, L]
    del K
    s = s.view(S, A, kv, n, g, L).masked_fill_(~vis[:, :, None, :, None], -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True)).exp_()
    p = s.div_(s.sum(-1, keepdim=True)).view(S, A, kv, n * g, L)
    o = p @ st["v_base"][:, :, :L].float()[:, None]
    low = p @ lr[:, None, None, :, r:]                                # [S, A, kv, n g, r]
    o = o + st["scale"] * (low @ st["B_v"].float().view(A, r, kv, d).permute(0, 2, 1, 3))
    o = o.view(S, A, kv, n, g, d).permute(0, 1, 3, 2, 4, 5).reshape(S, A, n, kv * g, d)
    live = torch.arange(n, device=DEV) < st["tree_len"].expand(S, A)[..., None]
    st["out"].copy_(torch.where(live[..., None, None], o.to(st["out"].dtype), st["out"]))
    return {"out": st["out"]}


def _norm_plain(st):
    c = st["case"]
    S, A, n, d = c["seqs"], c["agents"], c["tokens"], c["d"]
    trees = st["k"].shape[1]
    C = st["kv_len"].long()
    j = torch.arange(n, device=DEV)
    depth = j.expand(S, trees, n) if st["parent"] is None else _ancestors(st["parent"]).sum(-1) - 1
    cos, sin = _angles(C[:, None, None] + depth, d, c["base"])        # [S, trees, n, d/2]

    def normed(x, w):
        x = x.float()
        if w is None:
            return x
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()

    dt = st["q"].dtype
    live = j < st["tree_len"][..., None]                              # [S, trees, n]
    q = _rotate(normed(st["q"], st["w_q"]), cos[..., None, :], sin[..., None, :]).to(dt)
    st["out"].copy_(torch.where(live.expand(S, A, n)[..., None, None], q, st["out"]))
    k = _rotate(normed(st["k"], st["w_k"]), cos[..., None, :], sin[..., None, :]).to(dt)
    row = (C[:, None, None] + torch.arange(trees, device=DEV)[:, None] * n + j).view(S, trees * n)
    s = torch.arange(S, device=DEV)[:, None]
    lv = live.reshape(S, trees * n, 1, 1)
    for cache, new in ((st["k_base"], k), (st["v_base"], st["v"])):
        rows = cache.transpose(1, 2)                                  # [S, L, kv, d]
        rows[s, row] = torch.where(lv, new.reshape(S, trees * n, c["kv"], d), rows[s, row])
    return {"q": st["out"], "k": st["k_base"], "v": st["v_base"]}


def _grouped_plain(st):
    c = st["case"]
    T, r, A = c["tokens"], c["r"], c["agents"]
    seg = torch.bucketize(torch.arange(T, device=DEV, dtype=torch.int32), st["seg_start"][1:-1], right=True)
    agent = st["seg_agent"][seg]                                      # [T], -1: no adapter
    mine = agent[:, None] == torch.arange(A, device=DEV)              # [T, A]
    x = st["x"].float()
    if c["shared"]:
        low = (x @ st["A"].float())[:, None].expand(T, A, r)
    else:
        low = (x @ st["A"].float().permute(1, 0, 2).reshape(-1, A * r)).view(T, A, r)
    low = torch.where(mine[..., None], low, torch.zeros_like(low)).reshape(T, A * r)
    y = st["y"].float() + st["scale"] * (low @ st["B"].float().reshape(A * r, -1))
    st["out"].copy_(y.to(st["out"].dtype))
    return {"out": st["out"]}


# ---------------------------------------------------------------- work
def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "grouped":
        T, H, N, r, A = c["tokens"], c["hidden"], c["out"], c["r"], c["agents"]
        w = (1 if c["shared"] else A) * H * r + A * r * N
        return {"bytes": es * (T * H + 2 * T * N + w), "flops": 2.0 * T * r * (H + N)}
    S, A, kv, d, hq = c["seqs"], c["agents"], c["kv"], c["d"], c["heads"]
    trees = A if c["per_agent"] else 1
    ctx = c["ctx"] * (0.75 if c["ragged"] else 1.0)
    if c["op"] == "norm":
        n = c["tokens"] * (0.5 if c["ragged"] else 1.0)
        rows = S * n * (A * hq + trees * kv)
        return {"bytes": es * d * 2 * (rows + S * n * trees * kv), "flops": 10.0 * d * rows}
    r, n = c["r"], c["nodes"] * (0.5 if c["ragged"] else 1.0)
    keys = S * (ctx + trees * n)
    q = S * A * n * hq * d
    b = es * (keys * (2 * kv * d + (2 if c["keys"] else 1) * r) + 2 * q
              + (2 if c["keys"] else 1) * A * r * kv * d)
    pairs = S * A * hq * n * (ctx + n / 2)
    f = pairs * (4 * d + 2 * r)
    if c["keys"]:
        f += S * A * kv * (ctx + n) * (2 * r * d + 3 * d)
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------- the definitions in fp64
def _tree_rows(parent, n):
    """Per node of one tree: the list of visible nodes (ancestors, itself last)."""
    chains = []
    for j in range(n):
        chains.append((chains[parent[j]] if parent[j] >= 0 else []) + [j])
    return chains


def _turn(x, pos, base):
    """Rows of x turned as complex numbers x1 + i x2 by exp(i pos theta)."""
    d = x.shape[-1]
    th = base ** (-2 * torch.arange(d // 2, device=x.device, dtype=torch.float64) / d)
    z = torch.complex(x[..., : d // 2].contiguous(), x[..., d // 2:].contiguous())
    z = z * torch.polar(torch.ones_like(pos[..., None] * th), pos[..., None] * th)
    return torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] == "grouped":
        out = st["out"].double()
        cut, ag = st["seg_start"].tolist(), st["seg_agent"].tolist()
        for lo, hi, a in zip(cut[:-1], cut[1:], ag):
            out[lo:hi] = st["y"][lo:hi].double()
            if a >= 0 and hi > lo:
                Aa = st["A"].double() if c["shared"] else st["A"][a].double()
                out[lo:hi] += st["scale"] * ((st["x"][lo:hi].double() @ Aa) @ st["B"][a].double())
        return {"out": out}
    S, A, kv, d = c["seqs"], c["agents"], c["kv"], c["d"]
    g = c["heads"] // kv
    lens, tl = st["kv_len"].tolist(), st["tree_len"].tolist()
    par = None if st["parent"] is None else st["parent"].tolist()
    out = st["out"].double()
    if c["op"] == "norm":
        kc, n = st["k_base"].double(), c["tokens"]

        def normed(x, w):
            return x if w is None else x / (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * w.double()

        for s in range(S):
            for t in range(st["k"].shape[1]):
                m = tl[s][t]
                dep = range(n) if par is None else [len(x) - 1 for x in _tree_rows(par[s][t], n)]
                pos = lens[s] + torch.tensor(list(dep)[:m], device=DEV, dtype=torch.float64)
                k = _turn(normed(st["k"][s, t, :m].double(), st["w_k"]).transpose(0, 1), pos, c["base"])
                kc[s, :, lens[s] + t * n: lens[s] + t * n + m] = k
                for a in (range(A) if not c["per_agent"] else [t]):
                    q = _turn(normed(st["q"][s, a, :m].double(), st["w_q"]).transpose(0, 1), pos, c["base"])
                    out[s, a, :m] = q.transpose(0, 1)
        return {"q": out, "k": kc, "v": None}
    n, r = c["nodes"], c["r"]
    for s in range(S):
        for a in range(A):
            t = a if c["per_agent"] else 0
            C, m = lens[s], tl[s][t]
            chains = _tree_rows(par[s][t], n)[:m]
            rows = torch.cat([torch.arange(C), C + t * n + torch.arange(m)]).to(DEV)
            pos = torch.cat([torch.arange(C), C + torch.tensor([len(x) - 1 for x in chains])]).to(DEV).double()
            see = torch.zeros(m, C + m, dtype=torch.bool)
            see[:, :C] = True
            for j, x in enumerate(chains):
                see[j, [C + i for i in x]] = True
            see = see.to(DEV).repeat_interleave(g, 0)
            lr = st["lr"][s, rows].double()
            for h in range(kv):
                K, V = st["k_base"][s, h, rows].double(), st["v_base"][s, h, rows].double()
                if c["keys"]:
                    K = K + st["scale"] * _turn(lr[:, :r] @ st["B_k"][a, :, h * d:(h + 1) * d].double(), pos, c["base"])
                V = V + st["scale"] * (lr[:, r:] @ st["B_v"][a, :, h * d:(h + 1) * d].double())
                q = st["q"][s, a, :m, h * g:(h + 1) * g].double().reshape(m * g, d)
                z = (q @ K.T / math.sqrt(d)).masked_fill(~see, -math.inf)
                out[s, a, :m, h * g:(h + 1) * g] = (torch.softmax(z, -1) @ V).view(m, g, d)
    return {"out": out}
