"""Workloads of the operators that bring prompts and trees of drafts into the
serving step: attention over packed prompts, attention of a tree of drafted
tokens over the paged cache, greedy verification of such a tree, block tables
with slot maps from the requests' lengths, and writing keys and values to the
slots.

Each case is one call (two for the tables).  With ``own`` false it is computed
by elementary torch operations in 32 bits; with ``own`` true it is the
library's call.
"""

import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_ES = {"bf16": 2, "fp16": 2, "fp32": 4}
_DEV = "cuda"


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one chat's first question: latency is what counts
        {"name": "prompt, one question", "op": "prompt", "batch": 1, "len_min": 201,
         "len_max": 201, "kv_heads": 8, "group": 4, "dim": 128, "dtype": "bf16", "window": 0},
        # the prompts that one step of a serving batch admits, of every length
        {"name": "prompt, packed batch", "op": "prompt", "batch": 24, "len_min": 1,
         "len_max": 4000, "kv_heads": 8, "group": 4, "dim": 128, "dtype": "bf16", "window": 0},
        # a document
        {"name": "prompt, long", "op": "prompt", "batch": 1, "len_min": 16001, "len_max": 16001,
         "kv_heads": 8, "group": 4, "dim": 128, "dtype": "bf16", "window": 0},
        # a sliding window, many query heads a KV head
        {"name": "prompt, window", "op": "prompt", "batch": 3, "len_min": 5000,
         "len_max": 12001, "kv_heads": 4, "group": 7, "dim": 64, "dtype": "fp16", "window": 2048},
        # one chat whose drafter proposes a small tree
        {"name": "tree attention, one request", "op": "tree", "batch": 1, "kv_min": 900,
         "kv_max": 900, "k_min": 24, "k_max": 24, "kv_heads": 8, "group": 4, "dim": 128,
         "page": 16, "layers": 4, "dtype": "bf16", "window": 0},
        # a batch with trees of up to 64 nodes (the verification workloads' lengths)
        {"name": "tree attention, batch", "op": "tree", "batch": 32, "kv_min": 2001,
         "kv_max": 8190, "k_min": 8, "k_max": 63, "kv_heads": 8, "group": 4, "dim": 128,
         "page": 16, "layers": 2, "dtype": "bf16", "window": 0},
        # the same chat's decision
        {"name": "verify tree, 8 requests", "op": "verify", "batch": 8, "k_min": 5, "k_max": 24,
         "vocab": 32000},
        # a large batch's decisions
        {"name": "verify tree, 4096 requests", "op": "verify", "batch": 4096, "k_min": 0,
         "k_max": 63, "vocab": 151936},
        # a step of a few chats: each grows by a token or a few
        {"name": "tables, 8 requests", "op": "tables", "batch": 8, "kv_min": 1, "kv_max": 2000,
         "new_max": 16, "prompts": 0, "ended": 0, "cols": 128, "page": 16, "spare": 64},
        # a large server's step: a third ended, some bring prompts, the rest grow
        {"name": "tables, 1024 requests", "op": "tables", "batch": 1024, "kv_min": 1,
         "kv_max": 30000, "new_max": 16, "prompts": 100, "ended": 300, "cols": 2048, "page": 16,
         "spare": 20000},
        # the keys and values of one question, one layer
        {"name": "write, 201 rows", "op": "write", "rows": 201, "kv_heads": 8, "dim": 128,
         "q_heads": 32, "page": 16, "layers": 4, "dtype": "bf16", "padded": 7},
        # those of the prompts of a step, one layer
        {"name": "write, 32768 rows", "op": "write", "rows": 32768, "kv_heads": 8, "dim": 128,
         "q_heads": 32, "page": 16, "layers": 2, "dtype": "bf16", "padded": 100},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "tree", "tree", "verify", "tables", "write"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp16", "fp16", "fp32"])
    dim = rng.choice([64, 128, 128, 128, 256, 80])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16])
    group = rng.choice([1, 2, 4, 4, 7, 8])
    if op == "prompt":
        # operations at most the longest listed case's; 32 bits, which run on other units, a
        # sixty-fourth, heads that no listed case has a third
        cap = 2.0e12 / (64 if dtype == "fp32" else 3 if dim in (80, 256) else 1)
        batch = _log(rng, 1, 32)
        most = int(math.sqrt(cap / (2.0 * dim * kv_heads * group * batch)))
        most = max(1, min(32768, most, (1 << 28) // (kv_heads * group * dim * batch)))
        len_max = _log(rng, 1, most)
        return {"op": op, "batch": batch, "len_min": max(0, int(len_max * rng.random()) - 3),
                "len_max": len_max, "kv_heads": kv_heads, "group": group, "dim": dim,
                "dtype": dtype, "window": rng.choice([0, 0, 0, _log(rng, 1, 4096)])}
    if op == "tree":
        k_max = rng.choice([0, 3, 7, 15, 31, 63])
        batch = _log(rng, 1, 64)
        cap = (1 << 29) if dtype != "fp32" and dim != 80 else 1 << 26
        per_key = 2 * kv_heads * dim * _ES[dtype]
        most = min(131072, cap // (per_key * batch), (1 << 30) // (batch * kv_heads * group *
                                                                   (k_max + 1)))
        kv_max = _log(rng, 1, max(2, most))
        return {"op": op, "batch": batch, "kv_min": max(0, int(kv_max * rng.random()) - 3),
                "kv_max": kv_max, "k_min": rng.randint(0, k_max), "k_max": k_max,
                "kv_heads": kv_heads, "group": group, "dim": dim,
                "page": rng.choice([1, 7, 16, 16, 32, 64, 128]), "layers": rng.choice([1, 2]),
                "dtype": dtype, "window": rng.choice([0, 0, 0, _log(rng, 1, 4096)])}
    if op == "verify":
        k_max = rng.choice([1, 3, 7, 15, 24, 31, 63])
        return {"op": op, "batch": _log(rng, 1, 4096), "k_min": rng.randint(0, k_max),
                "k_max": k_max, "vocab": _log(rng, 1000, 151936)}
    if op == "tables":
        batch = _log(rng, 1, 1024)
        page = rng.choice([1, 7, 16, 16, 32, 64])
        kv_max = _log(rng, 1, min(30000, 2000 * page))
        ended = rng.randint(0, batch // 2)
        return {"op": op, "batch": batch, "kv_min": rng.randint(0, kv_max), "kv_max": kv_max,
                "new_max": rng.choice([1, 16, 64]), "prompts": rng.randint(0, (batch - ended) // 4),
                "ended": ended, "cols": -(-(kv_max + 2000) // page) + rng.randint(0, 40),
                "page": page, "spare": _log(rng, 1, 20000)}
    return {"op": op, "rows": _log(rng, 1, max(2, 32768 * 2048 // (kv_heads * dim * _ES[dtype]))
                                   if kv_heads * dim * _ES[dtype] > 2048 else 32768),
            "kv_heads": kv_heads, "dim": dim, "q_heads": kv_heads * group,
            "page": rng.choice([1, 7, 16, 16, 32, 64]), "layers": rng.choice([1, 2]),
            "dtype": dtype, "padded": rng.choice([0, 0, 1, 50])}


# -------------------------------------------------------------------- inputs
def _spread(n, lo, hi, seed, salt):
    """n lengths between lo and hi, spread over their logarithm (always the same ones; zero
    among them where lo is 0), in the seed's order."""
    rng = random.Random(salt)
    a = [int(round(math.exp(rng.uniform(math.log(max(1, lo)), math.log(max(1, hi))))))
         for _ in range(n)]
    if n:
        a[rng.randrange(n)] = hi
    if lo == 0 and n > 2:
        a[rng.randrange(n)] = 0
    random.Random(seed * 7919 + salt).shuffle(a)
    return a


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=_DEV)


def _randn(shape, dtype, g):
    return torch.randn(shape, dtype=dtype, device=_DEV, generator=g)


def _nodes(case, seed):
    """Draft counts in the seed's order."""
    rng = random.Random(7)
    k = [rng.randint(case["k_min"], case["k_max"]) for _ in range(case["batch"])]
    random.Random(seed * 104729 + 7).shuffle(k)
    return k


def _tree(k, seed):
    """Parents of every request's nodes: node 0 is the last emitted token, a draft hangs from
    one of the last few nodes before it, more often from an early one."""
    rng = random.Random(seed * 31 + 5)
    parent = []
    for n in k:
        parent.append(-1)
        for j in range(1, n + 1):
            lo = max(0, (j - 4) // 3)
            parent.append(lo + int((j - lo) * rng.random() ** 2))
    return parent


def _prompt_inputs(st, case, seed, g):
    n = _spread(case["batch"], case["len_min"], case["len_max"], seed, 13)
    Hk, D = case["kv_heads"], case["dim"]
    Hq, T = Hk * case["group"], sum(n)
    at = [0]
    for x in n:
        at.append(at[-1] + x)
    # one projection's rows: queries of twice the keys' spread, then keys, then values
    qkv = _randn((T, (Hq + 2 * Hk) * D), _DT[case["dtype"]], g)
    qkv[:, :Hq * D] *= 2
    st.update(n=n, at=at, qkv=qkv, offsets=_i32(at))


def _tree_inputs(st, case, seed, g):
    n = _spread(case["batch"], case["kv_min"], case["kv_max"], seed, 13)
    k = _nodes(case, seed)
    parent = _tree(k, seed)
    dt, S, D, Hk = _DT[case["dtype"]], case["page"], case["dim"], case["kv_heads"]
    need = [-(-x // S) for x in n]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(n), max(1, max(need) + 1)), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = torch.tensor(order[at:at + c], dtype=torch.int32)
        at += c
    rows = sum(k) + len(k)
    st.update(n=n, k=k, parent_list=parent, layer=case["layers"] - 1, table=table.to(_DEV),
              kv_len=_i32(n), k_per_req=_i32(k), parent=_i32(parent),
              cache=_randn((pool, case["layers"], 2, S, Hk * D), dt, g),
              q=_randn((rows, Hk * case["group"], D), dt, g) * 2,
              spec=_randn((len(n), max(k) + 1, case["layers"], 2, Hk * D), dt, g))


def _verify_inputs(st, case, seed):
    k, V = _nodes(case, seed), case["vocab"]
    parent = _tree(k, seed)
    rng = random.Random(seed * 17 + 3)
    argmax, drafts, t = [], [], 0
    for n in k:
        tokens = [rng.randrange(V) for _ in range(n + 1)]
        drafts += tokens[1:]
        best = [rng.randrange(V) for _ in range(n + 1)]
        # a good drafter: most nodes have the target's choice among their children
        for j in range(n, 0, -1):
            if rng.random() < 0.6:
                best[parent[t + j]] = tokens[j]
        argmax += best
        t += n + 1
    st.update(k=k, parent_list=parent, argmax=_i32(argmax), parent=_i32(parent),
              drafts=_i32(drafts), k_per_req=_i32(k))


def _requests(case, seed):
    """(cached length, pages' worth of tokens held, new tokens) of every request of a step,
    always the same ones in the seed's order."""
    rng = random.Random(11)
    n = _spread(case["batch"], case["kv_min"], case["kv_max"], 0, 13)
    kind = ["ended"] * case["ended"] + ["prompt"] * case["prompts"]
    kind += ["grows"] * (len(n) - len(kind))
    rng.shuffle(kind)
    got = []
    for x, what in zip(n, kind):
        new = 0 if what == "ended" else rng.randint(1, 2000) if what == "prompt" else \
            rng.randint(1, case["new_max"])
        got.append((x if what == "grows" else 0, 0 if what == "prompt" else x, new))
    random.Random(seed * 271 + 1).shuffle(got)
    return got


def _tables_inputs(st, case, seed):
    S, cols = case["page"], case["cols"]
    start, filled, count = zip(*_requests(case, seed))
    held = [-(-x // S) for x in filled]
    pages = sum(held) + case["spare"]
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int()
    table = torch.full((len(held), cols), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(held):
        table[b, :c] = order[at:at + c]
        at += c
    free = torch.full((pages,), -1, dtype=torch.int32)
    free[:case["spare"]] = order[at:]
    st.update(table=table.to(_DEV), held=_i32(held), start=_i32(start), count=_i32(count),
              want=_i32([x + c for x, c in zip(start, count)]), rows=sum(count) + 5,
              free=free.to(_DEV), free_count=_i32([case["spare"]]))
    st.update(out_table=torch.empty_like(st["table"]), out_held=torch.empty_like(st["held"]),
              out_free=torch.empty_like(st["free"]), out_count=torch.empty_like(st["free_count"]))


def _write_inputs(st, case, seed, g):
    R, Hk, D, S = case["rows"], case["kv_heads"], case["dim"], case["page"]
    dt = _DT[case["dtype"]]
    pool = -(-R // S) + 5
    # a few prompts of consecutive positions on scattered pages, as the slot map gives them
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(seed))
    p = torch.arange(R)
    slots = order[p // S] * S + p % S
    slots = torch.cat([slots, torch.full((case["padded"],), -1)])
    width = (case["q_heads"] + 2 * Hk) * D
    st.update(slots=slots.to(_DEV), layer=case["layers"] - 1,
              qkv=_randn((R + case["padded"], width), dt, g),
              cache=torch.zeros((pool, case["layers"], 2, S, Hk * D), dtype=dt, device=_DEV))


def prepare(case, seed):
    g = torch.Generator(device=_DEV).manual_seed(seed)
    st = {"case": case}
    op = case["op"]
    if op == "prompt":
        _prompt_inputs(st, case, seed, g)
    elif op == "tree":
        _tree_inputs(st, case, seed, g)
    elif op == "verify":
        _verify_inputs(st, case, seed)
    elif op == "tables":
        _tables_inputs(st, case, seed)
    else:
        _write_inputs(st, case, seed, g)
    return st


# --------------------------------------------------------------- plain forms
def _split(st):
    """q, k and v of the projection's rows."""
    c = st["case"]
    Hk, D = c["kv_heads"], c["dim"]
    Hq = Hk * c["group"] if "group" in c else c["q_heads"]
    q = st["qkv"][:, :Hq * D].unflatten(1, (Hq, D))
    k = st["qkv"][:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    return q, k, st["qkv"][:, (Hq + Hk) * D:].unflatten(1, (Hk, D))


def _softmax_product(s, see, v):
    """Weighted sum of v [n, h, d] by the softmax of s [h, g, i, n], and its lse."""
    s = torch.where(see, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    tot = p.sum(-1, keepdim=True)
    return torch.einsum("hgin,nhd->ihgd", p, v) / tot.permute(2, 0, 1, 3), \
        (m + torch.log(tot))[..., 0].permute(2, 0, 1)


def _prompt(st):
    c = st["case"]
    q, k, v = _split(st)
    T, Hq, D = q.shape
    W = c["window"]
    out = torch.empty((T, Hq, D), dtype=q.dtype, device=_DEV)
    lse = torch.empty((T, Hq), device=_DEV)
    for a, n in zip(st["at"], st["n"]):
        i0 = 0
        while i0 < n:
            # as many rows as keep the scores at a gigabyte
            i1 = min(n, i0 + max(1, (1 << 28) // (Hq * n)))
            lo = max(0, i0 - W + 1) if W else 0
            x = q[a + i0:a + i1].float().unflatten(1, (c["kv_heads"], c["group"]))
            s = torch.einsum("ihgd,nhd->hgin", x, k[a + lo:a + i1].float()) / math.sqrt(D)
            i = torch.arange(i0, i1, device=_DEV)[:, None]
            p = torch.arange(lo, i1, device=_DEV)
            see = (p <= i) & (p > i - W) if W else p <= i
            o, z = _softmax_product(s, see, v[a + lo:a + i1].float())
            out[a + i0:a + i1] = o.flatten(1, 2).to(out.dtype)
            lse[a + i0:a + i1] = z.flatten(1)
            i0 = i1
    return out, lse


def _paths(parent):
    """Of one request's nodes: which it sees of them (itself and its ancestors), and depths."""
    see = [[False] * len(parent) for _ in parent]
    for j, x in enumerate(parent):
        if j:
            see[j] = list(see[x])
        see[j][j] = True
    return see, [sum(x) - 1 for x in see]


def _tree_attention(st):
    c = st["case"]
    S, Hk, D, W = c["page"], c["kv_heads"], c["dim"], c["window"]
    out, lse = torch.empty_like(st["q"]), torch.empty(st["q"].shape[:2], device=_DEV)
    t = 0
    for b, (n, k) in enumerate(zip(st["n"], st["k"])):
        pages = st["table"][b, :-(-n // S)].long()
        kv = st["cache"][pages, st["layer"]].transpose(0, 1).reshape(2, -1, Hk, D)[:, :n]
        kv = torch.cat([kv, st["spec"][b, :k + 1, st["layer"]].transpose(0, 1)
                        .reshape(2, k + 1, Hk, D)], 1).float()
        path, depth = _paths(st["parent_list"][t:t + k + 1])
        at = n + torch.tensor(depth, device=_DEV)
        p = torch.cat([torch.arange(n, device=_DEV), at])
        see = torch.cat([torch.ones((k + 1, n), dtype=torch.bool, device=_DEV),
                         torch.tensor(path, device=_DEV)], 1)
        if W:
            see &= p > at[:, None] - W
        x = st["q"][t:t + k + 1].float().unflatten(1, (Hk, c["group"]))
        s = torch.einsum("ihgd,nhd->hgin", x, kv[0]) / math.sqrt(D)
        o, z = _softmax_product(s, see, kv[1])
        out[t:t + k + 1] = o.flatten(1, 2).to(out.dtype)
        lse[t:t + k + 1] = z.flatten(1)
        t += k + 1
    return out, lse


def _verify(st):
    """All requests together, a level of the trees at a time."""
    k = st["k_per_req"].long()
    B, most = k.numel(), int(st["case"]["k_max"]) + 1
    t0 = torch.cumsum(k + 1, 0) - (k + 1)
    j = torch.arange(most, device=_DEV)
    live = j <= k[:, None]
    row = torch.where(live, t0[:, None] + j, 0)
    parent = torch.where(live, st["parent"][row], -1).long()
    draft = torch.where(live & (j > 0), row - torch.arange(B, device=_DEV)[:, None] - 1, 0)
    token = st["drafts"][draft].long() if st["drafts"].numel() else torch.zeros_like(draft)
    argmax = st["argmax"][row].long()
    path = torch.full((B, most), -1, device=_DEV)
    tokens = torch.full((B, most), -1, device=_DEV)
    path[:, 0] = 0
    accept = torch.zeros_like(k)
    cur = torch.zeros_like(k)
    going = torch.ones_like(k, dtype=torch.bool)
    for step in range(most):
        best = argmax.gather(1, cur[:, None])[:, 0]
        tokens[:, step] = torch.where(going, best, tokens[:, step])
        hit = (parent == cur[:, None]) & (token == best[:, None]) & live & (j > 0)
        found = hit.any(1) & going
        nxt = torch.where(hit, j, most).amin(1)
        if step + 1 < most:
            path[:, step + 1] = torch.where(found, nxt, -1)
        accept += found
        cur = torch.where(found, nxt, cur)
        going = found
    return accept.int(), tokens[live].int(), path[live].int()


def _tables(st):
    c = st["case"]
    S, B, R = c["page"], c["batch"], st["rows"]
    held, n = st["held"].long(), st["free_count"].long()[0]
    need = -(-st["want"].long() // S)
    col = torch.arange(c["cols"], device=_DEV)
    table, free = st["table"].clone(), st["free"].clone()
    gone = (col >= need[:, None]) & (col < held[:, None])
    stack = torch.cat([free[:n], table[gone]])
    table[gone] = -1
    avail = stack.numel()
    want = (need - held).clamp_min(0)
    upto = torch.cumsum(want, 0)
    take = torch.where(upto <= avail, want, 0)
    new = (col >= held[:, None]) & (col < (held + take)[:, None])
    nth = (upto - want)[:, None] + col - held[:, None]
    table[new] = stack[avail - 1 - nth[new]]
    left = avail - take.sum()
    free[left:n] = -1
    free[:left] = stack[:left]
    held = torch.where(upto <= avail, need, torch.minimum(need, held))
    # the new tokens' slots
    count, start = st["count"].long(), st["start"].long()
    at = torch.cat([count.new_zeros(1), torch.cumsum(count, 0)])
    req = torch.repeat_interleave(torch.arange(B, device=_DEV), count)
    pos = start[req] + torch.arange(req.numel(), device=_DEV) - at[req]
    page = table[req, pos // S].long()
    out = torch.full((3, R), -1, device=_DEV)
    out[:, :req.numel()] = torch.stack([torch.where(page < 0, -1, page * S + pos % S), req, pos])
    return table, held.int(), free, left.int()[None], out[0], out[1].int(), out[2].int(), at.int()


def _write(st):
    c = st["case"]
    _, k, v = _split(st)
    live = st["slots"] >= 0
    s = st["slots"][live]
    page, at = s // c["page"], s % c["page"]
    st["cache"][page, st["layer"], 0, at] = k[live].flatten(1)
    st["cache"][page, st["layer"], 1, at] = v[live].flatten(1)
    return st["cache"]


# ----------------------------------------------------------------------- run
def run(state):
    st, op = state, state["case"]["op"]
    if not own:
        return {"prompt": _prompt, "tree": _tree_attention, "verify": _verify,
                "tables": _tables, "write": _write}[op](st)
    import speculative_decoding_verification_13_gb300 as sv
    c = st["case"]
    if op == "prompt":
        q, k, v = _split(st)
        return sv.prompt_attention(q, k, v, st["offsets"], window=c["window"])
    if op == "tree":
        return sv.tree_attention(st["q"], st["cache"], st["layer"], st["kv_len"], st["table"],
                                 st["k_per_req"], st["parent"], st["spec"], window=c["window"])
    if op == "verify":
        return sv.verify_tree_greedy(st["argmax"], st["drafts"], st["parent"], st["k_per_req"],
                                     c["vocab"])
    if op == "tables":
        t = sv.kv_reserve(st["table"], st["held"], st["want"], st["free"], st["free_count"],
                          c["page"], out_table=st["out_table"], out_held=st["out_held"],
                          out_free=st["out_free"], out_count=st["out_count"])
        s = sv.kv_slots(st["out_table"], st["start"], st["count"], st["rows"], c["page"])
        return tuple(t) + tuple(s)
    _, k, v = _split(st)
    return sv.kv_write(st["cache"], st["layer"], k, v, st["slots"])


# ---------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "prompt":
        n = _spread(case["batch"], case["len_min"], case["len_max"], 0, 13)
        W, Hk, D = case["window"], case["kv_heads"], case["dim"]
        Hq = Hk * case["group"]
        pairs = sum(x * (x + 1) // 2 if not W or x <= W else W * (W + 1) // 2 + (x - W) * W
                    for x in n)
        rows = sum(n)
        return {"bytes": rows * (2 * Hq + 2 * Hk) * D * _ES[case["dtype"]] + rows * Hq * 4 +
                4 * len(n) + 4, "flops": 4 * pairs * Hq * D}
    if op == "tree":
        n, k = _spread(case["batch"], case["kv_min"], case["kv_max"], 0, 13), _nodes(case, 0)
        parent, W = _tree(k, 0), case["window"]
        es, D, Hk = _ES[case["dtype"]], case["dim"], case["kv_heads"]
        Hq = Hk * case["group"]
        t = rows = keys = pairs = 0
        for x, y in zip(n, k):
            depth = _paths(parent[t:t + y + 1])[1]
            t += y + 1
            rows += y + 1
            keys += min(x, max(0, W - 1)) + y + 1 if W else x + y + 1
            # of depth d it sees d + 1 on its path, as far as the window goes, and the cache
            pairs += sum(min(x + d + 1, W) if W else x + d + 1 for d in depth)
        q = rows * Hq * D * es
        return {"bytes": 2 * keys * Hk * D * es + 2 * q + rows * Hq * 4 + 4 * rows +
                4 * (keys // case["page"] + 3 * len(n)), "flops": 4 * pairs * Hq * D}
    if op == "verify":
        rows = sum(_nodes(case, 0)) + case["batch"]
        return {"bytes": 4 * (5 * rows + case["batch"]), "flops": 0}
    if op == "tables":
        # tables and lists are read once and written once, a slot's page is read again
        _, filled, count = zip(*_requests(case, 0))
        pages = case["spare"] + sum(-(-x // case["page"]) for x in filled)
        return {"bytes": 8 * case["batch"] * case["cols"] + 8 * pages + 24 * case["batch"] +
                20 * sum(count), "flops": 0}
    entry = case["kv_heads"] * case["dim"] * _ES[case["dtype"]]
    return {"bytes": 4 * case["rows"] * entry + 8 * (case["rows"] + case["padded"]), "flops": 0}


# --------------------------------------------------------------------- exact
def exact(case, seed):
    op = case["op"]
    if op == "prompt":
        return _exact_prompt(case, seed)
    if op == "tree":
        return _exact_tree(prepare(case, seed))
    if op == "verify":
        return _exact_verify(prepare(case, seed))
    if op == "write":
        return _exact_write(prepare(case, seed))
    return None   # whole numbers, which the plain form has as they are


def _exact_prompt(case, seed):
    if work(case)["flops"] > 8e12:
        return None
    st = prepare(case, seed)
    q, k, v = _split(st)
    T, Hq, D = q.shape
    G, W = case["group"], case["window"] or T + 1
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=_DEV)
    lse = torch.zeros((T, Hq), dtype=torch.float64, device=_DEV)
    for b, n in enumerate(st["n"]):
        a = st["at"][b]
        for h in range(Hq):
            K, V = k[a:a + n, h // G].double(), v[a:a + n, h // G].double()
            for i in range(0, n, 1024):
                j = min(n, i + 1024)
                first = max(0, i + 1 - W)
                z = q[a + i:a + j, h].double() @ K[first:j].T * D ** -0.5
                # distance of query and key: 0 is the token itself
                gap = torch.arange(i, j, device=_DEV)[:, None] - torch.arange(first, j,
                                                                              device=_DEV)
                z.masked_fill_((gap < 0) | (gap >= W), -math.inf)
                total = torch.logsumexp(z, 1)
                out[a + i:a + j, h] = torch.exp(z - total[:, None]) @ V[first:j]
                lse[a + i:a + j, h] = total
    return out, lse


def _exact_tree(st):
    c, S, D, G = st["case"], st["case"]["page"], st["case"]["dim"], st["case"]["group"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=_DEV)
    lse = torch.zeros(out.shape[:2], dtype=torch.float64, device=_DEV)
    t = 0
    for b, (n, k) in enumerate(zip(st["n"], st["k"])):
        where = torch.arange(n, device=_DEV)
        kv = st["cache"][st["table"][b].long()[where // S], st["layer"], :, where % S]
        kv = torch.cat([kv, st["spec"][b, :k + 1, st["layer"]]]).double()
        for j in range(k + 1):
            path, x = [], j
            while x > 0:
                path.append(x)
                x = st["parent_list"][t + x]
            path = [0] + path[::-1]
            at = n + len(path) - 1
            lo = max(0, at - c["window"] + 1) if c["window"] else 0
            keys = list(range(lo, n)) + [n + y for i, y in enumerate(path) if n + i >= lo]
            seen = kv[torch.tensor(keys, device=_DEV)]
            for h in range(c["kv_heads"]):
                K, V = seen[:, 0, h * D:(h + 1) * D], seen[:, 1, h * D:(h + 1) * D]
                z = st["q"][t + j, h * G:(h + 1) * G].double() @ K.T * D ** -0.5
                total = torch.logsumexp(z, 1)
                out[t + j, h * G:(h + 1) * G] = torch.exp(z - total[:, None]) @ V
                lse[t + j, h * G:(h + 1) * G] = total
        t += k + 1
    return out, lse


def _exact_verify(st):
    argmax, drafts = st["argmax"].tolist(), st["drafts"].tolist()
    accept, tokens, paths, t = [], [], [], 0
    for b, k in enumerate(st["k"]):
        path = [0]
        while True:
            best = argmax[t + path[-1]]
            nxt = [j for j in range(1, k + 1) if st["parent_list"][t + j] == path[-1] and
                   drafts[t - b + j - 1] == best]
            if not nxt:
                break
            path.append(nxt[0])
        rest = [-1] * (k + 1 - len(path))
        accept.append(len(path) - 1)
        tokens += [argmax[t + j] for j in path] + rest
        paths += path + rest
        t += k + 1
    return tuple(torch.tensor(x, dtype=torch.int32) for x in (accept, tokens, paths))


def _exact_write(st):
    c, E = st["case"], st["case"]["kv_heads"] * st["case"]["dim"]
    S = c["page"]
    cache = st["cache"].double()
    # the row that each slot of the pool gets, or none
    row = {s: r for r, s in enumerate(st["slots"].tolist()) if s >= 0}
    taken = torch.tensor([row.get(s, -1) for s in range(cache.shape[0] * S)], device=_DEV)
    entries = cache.movedim(3, 1).flatten(0, 1)   # slot, layer, key or value, elements
    both = st["qkv"][:, -2 * E:].double().unflatten(1, (2, E))
    entries[:, st["layer"]] = torch.where((taken >= 0)[:, None, None], both[taken],
                                          entries[:, st["layer"]])
    return entries.unflatten(0, (-1, S)).movedim(1, 3)
