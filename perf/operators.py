"""Workloads of the serving operators next to verification: attention over the
paged KV cache, accumulated attention weights, cache eviction by them, and
log probabilities of given tokens with their gradient.

Each case is one call.  With ``own`` false the call is computed by elementary
torch operations in 32 bits; with ``own`` true it is the library's call.
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
        # one chat being answered, one new token a pass: latency is what counts
        {"name": "attention, one request", "op": "attention", "batch": 1, "kv_min": 900,
         "kv_max": 900, "k_min": 0, "k_max": 0, "kv_heads": 8, "group": 4, "dim": 128, "page": 16,
         "layers": 4, "dtype": "bf16", "window": 0, "spec": True},
        # a serving batch without drafts, prompts of every length
        {"name": "attention, new tokens", "op": "attention", "batch": 64, "kv_min": 1,
         "kv_max": 16000, "k_min": 0, "k_max": 0, "kv_heads": 8, "group": 4, "dim": 128,
         "page": 16, "layers": 2, "dtype": "bf16", "window": 0, "spec": True},
        # the target's pass over up to 15 drafts a request (the verification workloads' lengths)
        {"name": "attention, 15 drafts", "op": "attention", "batch": 32, "kv_min": 2001,
         "kv_max": 8190, "k_min": 1, "k_max": 15, "kv_heads": 8, "group": 4, "dim": 128,
         "page": 16, "layers": 2, "dtype": "bf16", "window": 0, "spec": True},
        # a few requests over book-length contexts, one KV head per query head
        {"name": "attention, long contexts", "op": "attention", "batch": 3, "kv_min": 100001,
         "kv_max": 131071, "k_min": 7, "k_max": 7, "kv_heads": 16, "group": 1, "dim": 64,
         "page": 64, "layers": 1, "dtype": "fp16", "window": 0, "spec": True},
        # the weights of one layer of a decoding batch, added to the running scores
        {"name": "weights, new tokens", "op": "weights", "batch": 24, "kv_min": 500,
         "kv_max": 9001, "k_min": 0, "k_max": 0, "kv_heads": 8, "group": 4, "dim": 128,
         "page": 16, "layers": 2, "dtype": "bf16", "window": 0, "spec": True},
        # the same behind a verification pass, rejected drafts left out
        {"name": "weights, 15 drafts", "op": "weights", "batch": 32, "kv_min": 2001,
         "kv_max": 8190, "k_min": 1, "k_max": 15, "kv_heads": 8, "group": 4, "dim": 128,
         "page": 16, "layers": 2, "dtype": "bf16", "window": 0, "spec": True},
        # one chat over its budget, a model of few layers
        {"name": "evict, one request", "op": "evict", "batch": 1, "kv_min": 1041, "kv_max": 1041,
         "entry": 1024, "page": 16, "layers": 4, "dtype": "bf16", "budget": 512, "sinks": 4,
         "recent": 128},
        # a batch whose caches all passed a budget, every layer moved
        {"name": "evict, batch", "op": "evict", "batch": 4, "kv_min": 3001, "kv_max": 9003,
         "entry": 1024, "page": 16, "layers": 36, "dtype": "bf16", "budget": 2000, "sinks": 4,
         "recent": 256},
        # the tokens of one small step, with five alternatives each
        {"name": "logprobs, 8 rows", "op": "logprobs", "rows": 8, "vocab": 32000, "pad": 0,
         "dtype": "fp32", "n_top": 5, "temperature": False},
        # the rows of a verified batch (256 requests, 15 drafts), twenty alternatives each
        {"name": "logprobs, 4096 rows", "op": "logprobs", "rows": 4096, "vocab": 151936, "pad": 0,
         "dtype": "bf16", "n_top": 20, "temperature": True},
        # a short training sequence for a drafter, odd vocabulary in packed rows
        {"name": "logprobs gradient, 61 rows", "op": "grad", "rows": 61, "vocab": 50257, "pad": 0,
         "dtype": "fp32", "entropy": True, "temperature": False},
        # a training batch for a drafter at the verification workloads' vocabulary
        {"name": "logprobs gradient, 2048 rows", "op": "grad", "rows": 2048, "vocab": 151936,
         "pad": 0, "dtype": "bf16", "entropy": True, "temperature": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "weights", "evict", "logprobs", "grad"])
    if op in ("attention", "weights"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp16", "fp16", "fp32"])
        dim = rng.choice([64, 128, 128, 128, 256, 80])
        kv_heads = rng.choice([1, 2, 4, 8, 8, 16])
        group = rng.choice([1, 2, 4, 4, 7, 8])
        k_max = rng.choice([0, 0, 3, 7, 15, 32])
        batch = _log(rng, 1, 64)
        # bytes and score elements at most a large listed case's; wide types and odd
        # head sizes, which no listed case has, a tenth of it
        cap = 1 << 30 if dtype != "fp32" and dim != 80 else 1 << 27
        per_key = 2 * kv_heads * dim * _ES[dtype]
        most = min(131072, cap // (per_key * batch), (1 << 31) // (batch * kv_heads * group *
                                                                    (k_max + 1)))
        kv_max = _log(rng, 1, max(2, most))
        return {"op": op, "batch": batch, "kv_min": max(0, int(kv_max * rng.random()) - 3),
                "kv_max": kv_max, "k_min": rng.randint(0, k_max), "k_max": k_max,
                "kv_heads": kv_heads, "group": group, "dim": dim,
                "page": rng.choice([1, 7, 16, 16, 32, 64, 128]), "layers": rng.choice([1, 2]),
                "dtype": dtype, "window": rng.choice([0, 0, 0, _log(rng, 1, 4096)]),
                "spec": rng.random() < 0.75}
    if op == "evict":
        kv_max = _log(rng, 32, 40000)
        batch = _log(rng, 1, 32)
        entry = rng.choice([64, 512, 1024, 2048])
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        batch = min(batch, max(1, (1 << 30) // (kv_max * 2 * entry * _ES[dtype])))
        most = max(1, (1 << 30) // (batch * kv_max * 2 * entry * _ES[dtype]))
        budget = _log(rng, 8, kv_max)
        sinks = rng.randint(0, min(8, budget // 3))
        return {"op": op, "batch": batch, "kv_min": rng.randint(1, kv_max), "kv_max": kv_max,
                "entry": entry, "page": rng.choice([1, 7, 16, 16, 32, 64]),
                "layers": rng.randint(1, min(36, most)), "dtype": dtype, "budget": budget,
                "sinks": sinks, "recent": rng.randint(0, budget - sinks)}
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    vocab = _log(rng, 1000, 151936)
    most = (4096 if op == "logprobs" else 2048) * 151936 * 2 // (vocab * _ES[dtype])
    case = {"op": op, "rows": _log(rng, 1, min(4096, most)), "vocab": vocab,
            "pad": rng.choice([0, 0, 1, 8, 24]), "dtype": dtype,
            "temperature": rng.random() < 0.5}
    if op == "logprobs":
        case["n_top"] = rng.choice([0, 1, 5, 20, 32])
    else:
        case["entropy"] = rng.random() < 0.5
    return case


# -------------------------------------------------------------------- inputs
def _lengths(case, seed):
    """The case's cache lengths (always the same ones) in the seed's order."""
    rng = random.Random(13)
    lo, hi = max(1, case["kv_min"]), max(1, case["kv_max"])
    n = [int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))) for _ in
         range(case["batch"])]
    n[rng.randrange(len(n))] = case["kv_max"]
    if case["kv_min"] == 0 and len(n) > 2:
        n[rng.randrange(len(n))] = 0
    random.Random(seed * 7919 + 13).shuffle(n)
    return n


def _drafts(case, seed):
    """The case's draft counts in the seed's order, and accept lengths."""
    rng = random.Random(7)
    k = [rng.randint(case["k_min"], case["k_max"]) for _ in range(case["batch"])]
    rng = random.Random(seed * 104729 + 7)
    rng.shuffle(k)
    accept = [rng.randint(0, x) for x in k]
    return k, accept


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=_DEV)


def _pages(lengths, page, spare, g, seed):
    """A block table over a shuffled pool; unused columns hold -1."""
    need = [-(-n // page) for n in lengths]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).tolist()
    cols = max(1, max(need) + 1)
    table = torch.full((len(need), cols), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = torch.tensor(order[at:at + c], dtype=torch.int32)
        at += c
    return table.to(_DEV), pool


def _randn(shape, dtype, g):
    return torch.randn(shape, dtype=dtype, device=_DEV, generator=g)


def prepare(case, seed):
    g = torch.Generator(device=_DEV).manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if op in ("attention", "weights"):
        dt = _DT[case["dtype"]]
        n = _lengths(case, seed)
        k, accept = _drafts(case, seed)
        D, Hk, Hq = case["dim"], case["kv_heads"], case["kv_heads"] * case["group"]
        E = Hk * D
        table, pool = _pages(n, case["page"], 3, g, seed)
        cache = _randn((pool, case["layers"], 2, case["page"], E), dt, g)
        rows = sum(k) + len(k)
        # queries of twice the keys' spread: attention that has clear peaks
        st.update(n=n, k=k, accept=accept, layer=case["layers"] - 1, cache=cache, table=table,
                  kv_len=_i32(n), k_per_req=_i32(k), accept_len=_i32(accept),
                  q=_randn((rows, Hq, D), dt, g) * 2,
                  spec=_randn((len(n), max(k) + 1, case["layers"], 2, E), dt, g)
                  if case["spec"] else None)
        if op == "weights":
            # what the attention call of this layer left behind
            st["lse"] = _attention(st)[1]
            cols = max(n) + max(k) + 1
            st["score"] = torch.rand((len(n), cols), device=_DEV, generator=g) * 4
            for b, x in enumerate(n):
                st["score"][b, x:] = 0
            st["out_score"] = st["score"].clone()
    elif op == "evict":
        n = _lengths(case, seed)
        dt = _DT[case["dtype"]]
        table, pool = _pages(n, case["page"], 3, g, seed)
        kept = [min(x, case["budget"]) for x in n]
        out_table, out_pool = _pages(kept, case["page"], 1, g, seed + 1)
        shape = (case["layers"], 2, case["page"], case["entry"])
        # attention weights summed over a long answer: a few positions hold most of it
        score = torch.exp(2 * _randn((len(n), max(n) + 5), torch.float32, g))
        for b, x in enumerate(n):
            score[b, x:] = 0
        st.update(n=n, kv_len=_i32(n), table=table, out_table=out_table, score=score,
                  cache=_randn((pool,) + shape, dt, g),
                  out_cache=torch.zeros((out_pool,) + shape, dtype=dt, device=_DEV),
                  out_score=torch.zeros_like(score), out_len=_i32([0] * len(n)))
    else:
        R, V = case["rows"], case["vocab"]
        x = _randn((R, V + case["pad"]), torch.float32, g)
        x *= 2.5
        st["logits"] = x.to(_DT[case["dtype"]])[:, :V]
        del x
        st["tokens"] = torch.randint(0, V, (R,), dtype=torch.int32, device=_DEV, generator=g)
        st["T"] = (0.5 + torch.rand(R, device=_DEV, generator=g)) if case["temperature"] else None
        if op == "grad":
            # what the forward call left behind, and the loss's gradients
            _, ent, m, ls = _row_stats(st["logits"], st["tokens"], st["T"])
            st.update(max=m, logsum=ls, entropy=ent,
                      g_lp=_randn((R,), torch.float32, g),
                      g_ent=_randn((R,), torch.float32, g) * 0.1 if case["entropy"] else None)
    return st


# --------------------------------------------------------------- plain forms
def _span(case, n, k, j):
    """The positions that query j of a request sees: [lo, hi)."""
    at = n + j if case["spec"] else n - 1 - k + j
    return max(0, at - case["window"] + 1) if case["window"] else 0, max(0, at + 1)


def _request(st, b, t):
    """Keys and values of request b as [keys, kv_heads, dim] in 32 bits, and its queries."""
    c = st["case"]
    n, k, S, Hk, D = st["n"][b], st["k"][b], c["page"], c["kv_heads"], c["dim"]
    pages = st["table"][b, :-(-n // S)].long()
    kv = st["cache"][pages, st["layer"]]
    kv = kv.transpose(0, 1).reshape(2, -1, Hk, D)[:, :n]
    if st["spec"] is not None:
        kv = torch.cat([kv, st["spec"][b, :k + 1, st["layer"]].transpose(0, 1)
                        .reshape(2, k + 1, Hk, D)], 1)
    q = st["q"][t:t + k + 1].float().reshape(k + 1, Hk, c["group"], D)
    lo, hi = zip(*[_span(c, n, k, j) for j in range(k + 1)])
    p = torch.arange(kv.shape[1], device=_DEV)
    lo, hi = (torch.tensor(x, device=_DEV)[:, None] for x in (lo, hi))
    return q, kv[0].float(), kv[1].float(), (p >= lo) & (p < hi)


def _attention(st):
    c = st["case"]
    out, lse = torch.empty_like(st["q"]), torch.empty(st["q"].shape[:2], device=_DEV)
    t = 0
    for b, k in enumerate(st["k"]):
        q, K, V, see = _request(st, b, t)
        s = torch.einsum("jhgd,nhd->hjgn", q, K) / math.sqrt(c["dim"])
        s = torch.where(see[None, :, None], s, -math.inf)
        m = s.amax(-1, keepdim=True) if s.shape[-1] else s.new_full(s.shape[:-1] + (1,), -math.inf)
        m = torch.where(m == -math.inf, 0, m)
        p = torch.exp(s - m)
        del s
        tot = p.sum(-1, keepdim=True)
        o = torch.einsum("hjgn,nhd->hjgd", p, V) / torch.where(tot == 0, 1, tot)
        out[t:t + k + 1] = o.permute(1, 0, 2, 3).reshape(k + 1, -1, c["dim"]).to(out.dtype)
        lse[t:t + k + 1] = (m + torch.log(tot))[..., 0].permute(1, 0, 2).reshape(k + 1, -1)
        t += k + 1
    return out, lse


def _weights(st):
    c, out, t = st["case"], st["out_score"], 0
    for b, (n, k) in enumerate(zip(st["n"], st["k"])):
        q, K, _, see = _request(st, b, t)
        take = st["accept"][b] + 1
        lse = st["lse"][t:t + k + 1].reshape(k + 1, c["kv_heads"], c["group"])
        s = torch.einsum("jhgd,nhd->hjgn", q, K) / math.sqrt(c["dim"])
        s = torch.where(see[None, :, None], s, -math.inf)
        lse = torch.where(lse == -math.inf, 0, lse).permute(1, 0, 2)[..., None]
        w = torch.exp(s - lse)[:, :take].sum((0, 1, 2))
        end = n + take if c["spec"] else n
        out[b, :end] = st["score"][b, :end] + w[:end]
        t += k + 1
    return out


def _evict(st):
    c = st["case"]
    m, sinks, recent, S = c["budget"], c["sinks"], c["recent"], c["page"]
    kept = torch.full((len(st["n"]), m), -1, dtype=torch.int32, device=_DEV)
    for b, n in enumerate(st["n"]):
        sc = st["score"][b]
        if n <= m:
            keep = torch.arange(n, device=_DEV)
        else:
            order = torch.sort(sc[sinks:n - recent], descending=True, stable=True)[1] + sinks
            all_ = torch.arange(n, device=_DEV)
            keep = torch.cat([all_[:sinks], order[:m - sinks - recent].sort()[0],
                              all_[n - recent:]])
        i = torch.arange(keep.numel(), device=_DEV)
        kept[b, :keep.numel()] = keep.int()
        src, dst = st["table"][b].long(), st["out_table"][b].long()
        st["out_cache"][dst[i // S], :, :, i % S] = st["cache"][src[keep // S], :, :, keep % S]
        st["out_score"][b, :keep.numel()] = sc[keep]
        st["out_score"][b, keep.numel():n] = 0
        st["out_len"][b] = keep.numel()
    return kept


def _row_stats(x, tokens, T):
    """Log probability of the rows' tokens, entropy, maximum and log-sum, 512 rows at a time."""
    parts = []
    for r in range(0, x.shape[0], 512):
        z = x[r:r + 512].float()
        m = z.amax(1)
        y = z - m[:, None]
        if T is not None:
            y = y / T[r:r + 512, None]
        e = torch.exp(y)
        tot = e.sum(1)
        ls = torch.log(tot)
        mean = (e * y).sum(1) / tot
        lp = y.gather(1, tokens[r:r + 512, None].long())[:, 0] - ls
        parts.append((lp, ls - mean, m, ls))
    return [torch.cat(p) for p in zip(*parts)]


def _logprobs(st):
    x, c = st["logits"], st["case"]
    lp, ent, m, ls = _row_stats(x, st["tokens"], st["T"])
    if not c["n_top"]:
        return lp, ent, m, ls
    tok, top = [], []
    index = torch.arange(c["vocab"], device=_DEV)
    for r in range(0, x.shape[0], 512):
        z = x[r:r + 512].float()
        bits = z.view(torch.int32).long()
        key = torch.where(bits < 0, -(bits & 0x7fffffff), bits)  # ordered like z, -0 equal to 0
        i = torch.topk(key * (1 << 32) - index, c["n_top"], dim=1)[1]  # ties: lowest index
        y = z.gather(1, i) - m[r:r + 512, None]
        if st["T"] is not None:
            y = y / st["T"][r:r + 512, None]
        tok.append(i.int())
        top.append(y - ls[r:r + 512, None])
    return lp, ent, m, ls, torch.cat(tok), torch.cat(top)


def _grad(st):
    x, T = st["logits"], st["T"]
    out = torch.empty(x.shape, dtype=x.dtype, device=_DEV)
    for r in range(0, x.shape[0], 512):
        s = slice(r, r + 512)
        y = x[s].float() - st["max"][s, None]
        if T is not None:
            y = y / T[s, None]
        lp = y - st["logsum"][s, None]
        p = torch.exp(lp)
        d = -st["g_lp"][s, None] * p
        if st["g_ent"] is not None:
            d -= st["g_ent"][s, None] * p * (lp + st["entropy"][s, None])
        i = st["tokens"][s, None].long()
        d.scatter_add_(1, i, st["g_lp"][s, None])
        if T is not None:
            d /= T[s, None]
        out[s] = d.to(out.dtype)
    return out


# ----------------------------------------------------------------------- run
def run(state):
    st, op = state, state["case"]["op"]
    if not own:
        if op == "attention":
            return _attention(st)
        if op == "weights":
            return _weights(st)
        if op == "evict":
            kept = _evict(st)
            return kept, st["out_len"], st["out_score"], st["out_cache"]
        return _logprobs(st) if op == "logprobs" else _grad(st)
    import speculative_decoding_verification_13_gb300 as sv
    c = st["case"]
    if op == "attention":
        return sv.attention(st["q"], st["cache"], st["layer"], st["kv_len"], st["table"],
                            st["k_per_req"], st["spec"], window=c["window"])
    if op == "weights":
        return sv.attention_weights(st["q"], st["cache"], st["layer"], st["kv_len"], st["table"],
                                    st["k_per_req"], st["lse"], st["score"], st["spec"],
                                    st["accept_len"], window=c["window"],
                                    out_score=st["out_score"])
    if op == "evict":
        n, kept = sv.kv_evict(st["cache"], st["score"], st["kv_len"], st["table"], c["budget"],
                              c["sinks"], c["recent"], out_cache=st["out_cache"],
                              out_table=st["out_table"], out_score=st["out_score"],
                              out_len=st["out_len"], with_kept=True)
        return kept, n, st["out_score"], st["out_cache"]
    if op == "logprobs":
        r = sv.logprobs(st["logits"], st["tokens"], st["T"], c["n_top"])
        lp = (r.logprob, r.entropy, r.max, r.logsum)
        return lp + (r.top_tokens, r.top_logprobs) if c["n_top"] else lp
    return sv.logprobs_grad(st["logits"], st["tokens"], st["max"], st["logsum"], st["entropy"],
                            st["g_lp"], st["g_ent"], st["T"])


# ---------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op in ("attention", "weights"):
        # lengths and drafts in one seed's order
        n, (k, accept) = _lengths(case, 0), _drafts(case, 0)
        es, D, Hk = _ES[case["dtype"]], case["dim"], case["kv_heads"]
        Hq = Hk * case["group"]
        rows, keys, pairs = 0, 0, 0
        for b in range(len(n)):
            take = k[b] + 1 if op == "attention" else accept[b] + 1
            spans = [_span(case, n[b], k[b], j) for j in range(take)]
            rows += take
            keys += max(h for _, h in spans) - min(lo for lo, _ in spans)
            pairs += sum(h - lo for lo, h in spans)
        q = rows * Hq * D * es
        tables = 4 * (keys // case["page"] + 3 * len(n))
        if op == "attention":
            return {"bytes": 2 * keys * Hk * D * es + 2 * q + rows * Hq * 4 + tables,
                    "flops": 4 * pairs * Hq * D}
        return {"bytes": keys * Hk * D * es + q + rows * Hq * 4 + 8 * keys + tables,
                "flops": 2 * pairs * Hq * D}
    if op == "evict":
        n = _lengths(case, 0)
        kept = sum(min(x, case["budget"]) for x in n)
        moved = kept * case["layers"] * 2 * case["entry"] * _ES[case["dtype"]]
        return {"bytes": 2 * moved + 8 * sum(n) + 4 * len(n) * case["budget"], "flops": 0}
    size = case["rows"] * case["vocab"]
    if op == "logprobs":
        return {"bytes": size * _ES[case["dtype"]] + case["rows"] * (24 + 8 * case["n_top"]),
                "flops": 6 * size}
    return {"bytes": 2 * size * _ES[case["dtype"]] + case["rows"] * 28, "flops": 8 * size}


# --------------------------------------------------------------------- exact
def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op in ("attention", "weights"):
        return _exact_attention(st)
    if op == "evict":
        return _exact_evict(st)
    rows = []
    x, T = st["logits"], st["T"]
    for r in range(0, x.shape[0], 128):
        z = x[r:r + 128].double()
        if T is not None:
            z = z / T[r:r + 128, None].double()
        lp = torch.log_softmax(z, 1)
        p = torch.exp(lp)
        H = -(p * lp).sum(1)
        tok = st["tokens"][r:r + 128].long()
        at = torch.arange(len(tok), device=_DEV)
        if op == "grad":
            one = torch.zeros_like(p)
            one[at, tok] = 1
            d = st["g_lp"][r:r + 128, None].double() * (one - p)
            if st["g_ent"] is not None:
                d = d - st["g_ent"][r:r + 128, None].double() * p * (lp + H[:, None])
            rows.append(d if T is None else d / T[r:r + 128, None].double())
            continue
        top = z.amax(1)
        got = [lp[at, tok], H, x[r:r + 128].double().amax(1), torch.logsumexp(z, 1) - top]
        if case["n_top"]:
            got.append(lp.sort(1, descending=True)[0][:, :case["n_top"]].clone())
        rows.append(got)
    if op == "grad":
        return torch.cat(rows)
    got = [torch.cat(p) for p in zip(*rows)]
    return tuple(got[:4]) + ((None, got[4]) if case["n_top"] else ())


def _exact_attention(st):
    c, S, D, G = st["case"], st["case"]["page"], st["case"]["dim"], st["case"]["group"]
    pairs = sum(n * (k + 1) for n, k in zip(st["n"], st["k"])) * c["kv_heads"] * G
    if pairs * D > 1 << 40:
        return None
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=_DEV)
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device=_DEV)
    score = st["score"].double() if "score" in st else None
    t = 0
    for b, (n, k) in enumerate(zip(st["n"], st["k"])):
        where = torch.arange(n, device=_DEV)
        kv = st["cache"][st["table"][b].long()[where // S], st["layer"], :, where % S]
        if st["spec"] is not None:
            kv = torch.cat([kv, st["spec"][b, :k + 1, st["layer"]]])
        for h in range(c["kv_heads"]):
            K, V = kv[:, 0, h * D:(h + 1) * D].double(), kv[:, 1, h * D:(h + 1) * D].double()
            for j in range(k + 1):
                lo, hi = _span(c, n, k, j)
                if hi <= lo:
                    continue
                z = st["q"][t + j, h * G:(h + 1) * G].double() @ K[lo:hi].T * D ** -0.5
                total = torch.logsumexp(z, 1)
                p = torch.exp(z - total[:, None])
                out[t + j, h * G:(h + 1) * G] = p @ V[lo:hi]
                lse[t + j, h * G:(h + 1) * G] = total
                if score is not None and j <= st["accept"][b]:
                    score[b, lo:hi] += p.sum(0)
        t += k + 1
    return (out, lse) if score is None else score


def _exact_evict(st):
    c = st["case"]
    kept = torch.full((len(st["n"]), c["budget"]), -1, dtype=torch.int32)
    score = torch.zeros(st["score"].shape, dtype=torch.float64)
    for b, n in enumerate(st["n"]):
        s = st["score"][b].tolist()
        keep = set(range(n)) if n <= c["budget"] else \
            set(range(c["sinks"])) | set(range(n - c["recent"], n))
        for p in sorted(range(n), key=lambda p: (-s[p], p)):
            if len(keep) >= min(n, c["budget"]):
                break
            keep.add(p)
        keep = sorted(keep)
        kept[b, :len(keep)] = torch.tensor(keep, dtype=torch.int32)
        score[b, :len(keep)] = torch.tensor([s[p] for p in keep], dtype=torch.float64)
    return kept, None, score, None
