"""The paged-cache operators, in plain torch and as calls of the library, with the cases they
are measured on.

Three operators work on one paged key-value cache of grouped query heads (pool
[pages][2][Hkv][64][d], bf16 or fp16, per-sequence page tables):

  append  new tokens' keys and values go behind each sequence's last token; pages are taken
          from the sequence's stack of free pages when its tail page is full
  attn    one new token per sequence attends over the pages of its table: scores capped by a
          tanh, a bias that grows with distance, prefix / document / window masks, and each
          page's attention weight added to its running score
  evict   of each sequence's pages keep the first `sink`, the last `recent` and those of the
          rest with the largest scores, `budget` in all; the others go to the free stack

`run` computes them in elementary torch operations where `own` is false, and calls the
library where it is true. Everything is synthetic and seeded.
"""
import numpy as np
import torch

own = False

PAGE = 64
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------ cases
def _attn(name, B, H, Hkv, d, tokens, dtype="bf16", ragged=False, gap=1, cap=0.0, slopes=False,
          window=0, prefix=0, docs=False, score=False, plan=1):
    c = {"op": "attn", "B": B, "H": H, "Hkv": Hkv, "d": d, "tokens": tokens, "dtype": dtype,
         "ragged": ragged, "gap": gap, "cap": cap, "slopes": slopes, "window": window,
         "prefix": prefix, "docs": docs, "score": score, "plan": plan}
    return dict(c, name=name) if name else c


def _evict(name, B, entries, budget, sink, recent, ragged=False, plan=1):
    c = {"op": "evict", "B": B, "entries": entries, "budget": budget, "sink": sink,
         "recent": recent, "ragged": ragged, "plan": plan}
    return dict(c, name=name) if name else c


def _append(name, B, Hkv, d, new, held, dtype="bf16", plan=1):
    c = {"op": "append", "B": B, "Hkv": Hkv, "d": d, "new": new, "held": held, "dtype": dtype,
         "plan": plan}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a chat's first tokens: one page, where only latency counts
        _attn("attn_first_page", 1, 8, 1, 128, 17),
        # one sequence of the smallest workload (16,384 tokens, 8 heads of 128), capped scores,
        # its pages' weights kept for eviction
        _attn("attn_16k_cap_score", 1, 8, 1, 128, 16384, cap=50.0, score=True),
        # a serving batch of a grouped-query model in fp16: a sliding window behind a prompt prefix
        _attn("attn_gqa_window_fp16", 16, 32, 8, 128, 8009, dtype="fp16", ragged=True, cap=30.0,
              window=2048, prefix=100),
        # a large ragged batch: packed documents, distance bias, page weights
        _attn("attn_gqa_ragged_bias", 64, 64, 8, 128, 4096, ragged=True, slopes=True, docs=True,
              score=True),
        # eight 131,072-token sequences, 64 heads of 512 on one key head, some 205 of 2,048 pages kept
        _attn("attn_b8_128k_kept", 8, 64, 1, 512, 13117, gap=10, cap=50.0, score=True),
        # one 1M-token sequence with some 1,350 of its 16,385 pages kept, distance bias
        _attn("attn_1m_kept_bias", 1, 64, 1, 512, 86417, gap=12, slopes=True, score=True),
        # the same sequence whole: the largest read
        _attn("attn_1m_dense_score", 1, 64, 1, 512, 1048577, score=True),
        # small caches trimmed while they decode
        _evict("evict_b8_65", 8, 65, 64, 1, 16),
        # a ragged batch trimmed to 512 pages each
        _evict("evict_b64_ragged", 64, 4096, 512, 4, 64, ragged=True),
        # a 1M-token prompt trimmed once to the pages that its decoding keeps
        _evict("evict_1m", 1, 16385, 1351, 1, 129),
        # one decoded token per sequence
        _append("append_decode_b64", 64, 8, 128, 0, 1000),
        # ragged prompts written at once, fp16
        _append("append_prompts_fp16", 16, 8, 128, 4096, 777, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    plan = rng.randrange(1 << 20)
    op = rng.choice(["attn", "attn", "attn", "evict", "append"])
    if op == "evict":
        sink, recent = rng.randrange(0, 9), _log(rng, 1, 130)
        budget = sink + recent + _log(rng, 1, 1500)
        return _evict(None, _log(rng, 1, 64), min(16385, budget + _log(rng, 1, 15000)), budget, sink,
                      recent, rng.random() < 0.5, plan)
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "append":
        B, Hkv, d = _log(rng, 1, 64), rng.choice([1, 2, 4, 8]), rng.choice([128, 256, 512])
        most = max(2, (1 << 26) // (B * Hkv * d))       # tokens of one sequence
        return _append(None, B, Hkv, d, rng.choice([0, _log(rng, 2, min(most, 8192))]),
                       _log(rng, 1, min(most, 2000)), dtype, plan)
    Hkv = rng.choice([1, 1, 2, 4, 8])
    group = rng.choice([1, 3, 4, 7, 8, 12, 16, 20, 32, 64]) if Hkv == 1 else rng.choice([1, 3, 4, 7, 8, 16])
    d = rng.choice([128, 128, 256, 384, 512])
    B = _log(rng, 1, 64)
    most = max(2, (1 << 28) // (B * Hkv * d))           # about 1 GB of keys and values
    return _attn(None, B, Hkv * group, Hkv, d, _log(rng, 1, min(most, 1 << 18)), dtype,
                 rng.random() < 0.6, rng.choice([1, 1, 4, 12]), rng.choice([0.0, 0.0, 20.0, 50.0]),
                 rng.random() < 0.4, rng.choice([0, 0, _log(rng, 1, 8192)]),
                 rng.choice([0, 0, _log(rng, 1, 500)]), rng.random() < 0.3, rng.random() < 0.5, plan)


def _lengths(rs, B, most, ragged):
    """Lengths of 1 .. most, the first one the longest; all of them the longest if not ragged."""
    n = np.full(B, most, np.int64)
    return np.where(np.arange(B) > 0, rs.randint(1, most + 1, B), n) if ragged else n


def _attn_plan(c):
    """Host arrays of the case's page tables, the same for every seed: entries, tail length, the
    position (in pages of the context) of each entry, prefix and document bounds, and which
    tokens the new one sees."""
    rs = np.random.RandomState(c["plan"])
    tokens = _lengths(rs, c["B"], c["tokens"], c["ragged"])
    n = (tokens + PAGE - 1) // PAGE
    tail = tokens - (n - 1) * PAGE
    E = int(n.max())
    j = np.arange(E)[None, :]
    recent = np.minimum(n, 1 + n // 8)[:, None]          # the newest entries are consecutive
    step = 1 + rs.randint(0, 2 * c["gap"] - 1, (c["B"], E))
    step[(j >= n[:, None] - recent) | (j == 0)] = 1
    pos = np.cumsum(step, 1) - 1
    last = pos[np.arange(c["B"]), n - 1] * PAGE + tail - 1   # the new token's own position
    prefix = np.minimum(c["prefix"] + rs.randint(0, 40, c["B"]) * (c["prefix"] > 0), last + 1)
    docs = rs.randint(0, last + 1) if c["docs"] else np.zeros(c["B"], np.int64)
    low = np.maximum(docs, last - c["window"] + 1) if c["window"] else docs
    at = pos[:, :, None] * PAGE + np.arange(PAGE)
    held = np.arange(PAGE)[None, None, :] < np.where(j < n[:, None] - 1, PAGE, np.where(j == n[:, None] - 1, tail[:, None], 0))[:, :, None]
    sees = held & ((at < prefix[:, None, None]) | (at >= low[:, None, None]))
    return dict(n=n, tail=tail, pos=pos, last=last, prefix=prefix, docs=docs, low=low, sees=sees)


def _evict_plan(c):
    rs = np.random.RandomState(c["plan"])
    return _lengths(rs, c["B"], c["entries"], c["ragged"])


def _append_plan(c):
    """(tokens held, new tokens) of each sequence."""
    rs = np.random.RandomState(c["plan"])
    held = rs.randint(0, c["held"] + 1, c["B"])
    new = rs.randint(0, c["new"] + 1, c["B"]) if c["new"] else np.ones(c["B"], np.int64)
    if c["new"]:
        new[0] = c["new"]
    return held, new


# ------------------------------------------------------------------------------ inputs
def _dev(a, dtype):
    return torch.as_tensor(np.ascontiguousarray(a)).to(dtype).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s, **k: torch.randn(*s, generator=g, device="cuda", **k)  # noqa: E731
    c, i32 = case, dict(dtype=torch.int32, device="cuda")
    s = {"case": dict(c)}
    if c["op"] == "attn":
        p = _attn_plan(c)
        B, E, d, t = c["B"], p["pos"].shape[1], c["d"], TYPES[c["dtype"]]
        pages = int(p["n"].sum()) + 3
        # scattered pages; entries behind a sequence's last hold whatever was there
        perm = torch.randperm(pages, generator=g, device="cuda").int()
        live = torch.arange(E, device="cuda")[None] < _dev(p["n"], torch.int32)[:, None]
        table = torch.full((B, E), -1, **i32)
        table[live] = perm[: int(p["n"].sum())]
        s.update(pool=randn(pages, 2, c["Hkv"], PAGE, d, dtype=t), block_table=table,
                 block_pos=_dev(p["pos"], torch.int32), n_entries=_dev(p["n"], torch.int32),
                 tail_len=_dev(p["tail"], torch.int32), q=randn(B, c["H"], d, dtype=t),
                 out=torch.empty(B, c["H"], d, dtype=t, device="cuda"), scale=d ** -0.5)
        s["score"] = randn(B, E).abs() if c["score"] else None
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, c["H"] + 1, device="cuda") / c["H"]) if c["slopes"] else None
        s["prefix_len"] = _dev(p["prefix"], torch.int32) if c["prefix"] else None
        s["doc_start"] = _dev(p["docs"], torch.int32) if c["docs"] else None
    elif c["op"] == "evict":
        n = _evict_plan(c)
        B, E = c["B"], int(n.max())
        # weights of pages that were attended to spread over decades; some pages never were
        score = torch.exp(2.0 * randn(B, E)) * (torch.rand(B, E, generator=g, device="cuda") > 0.1)
        s.update(block_table=torch.randint(0, 1 << 22, (B, E), generator=g, **i32),
                 block_pos=torch.cumsum(torch.randint(1, 9, (B, E), generator=g, **i32), 1, dtype=torch.int32),
                 score=score, n_entries=_dev(n, torch.int32), tail_len=torch.full((B,), PAGE, **i32),
                 free_list=torch.zeros((B, E + 8), **i32), free_cnt=torch.randint(0, 8, (B,), generator=g, **i32))
        s["dst"] = dict(block_table=torch.zeros((B, E), **i32), block_pos=torch.zeros((B, E), **i32),
                        score=torch.zeros((B, E), device="cuda"), n_entries=torch.zeros(B, **i32),
                        tail_len=s["tail_len"], free_list=s["free_list"], free_cnt=torch.zeros(B, **i32))
        s["pool"] = torch.zeros(1, 2, 1, PAGE, 128, dtype=torch.bfloat16, device="cuda")
    else:
        held, new = _append_plan(c)
        B, t = c["B"], TYPES[c["dtype"]]
        n = (held + PAGE - 1) // PAGE
        tail = np.where(n > 0, held - (n - 1) * PAGE, 0)
        more = (held + new + PAGE - 1) // PAGE - n
        E, F = int((n + more).max()), int(more.max()) + 2
        pages = B * (E + F)
        perm = torch.randperm(pages, generator=g, device="cuda").int().view(B, E + F)
        total = int(new.sum())
        s.update(pool=randn(pages, 2, c["Hkv"], PAGE, c["d"], dtype=t), block_table=perm[:, :E].contiguous(),
                 block_pos=torch.arange(E, **i32).repeat(B, 1), score=randn(B, E).abs(),
                 n_entries=_dev(n, torch.int32), tail_len=_dev(tail, torch.int32),
                 free_list=perm[:, E:].contiguous(), free_cnt=torch.full((B,), F, **i32),
                 k=randn(total, c["Hkv"], c["d"], dtype=t), v=randn(total, c["Hkv"], c["d"], dtype=t),
                 tok_off=_dev(np.concatenate([[0], np.cumsum(new)]), torch.int32) if c["new"] else None)
        # the counts go to tensors of their own, so that the call can be made again; tables are shared
        s["dst"] = dict(block_table=s["block_table"], block_pos=s["block_pos"], score=s["score"],
                        n_entries=torch.zeros(B, **i32), tail_len=torch.zeros(B, **i32),
                        free_list=s["free_list"], free_cnt=torch.zeros(B, **i32))
    if own:
        # the handle that a serving loop keeps beside its cache
        import lookahead_sparse_kv_lsa_b200 as lsa
        tables = ("block_table", "block_pos", "score", "n_entries", "tail_len", "free_list", "free_cnt")
        s["cache"] = lsa.LsaPagedCache(s["pool"], lsa.LsaPagedTables(**{k: s.get(k) for k in tables}),
                                       H=c.get("H", c.get("Hkv", 1)), scale=s.get("scale", 1.0), cap=c.get("cap", 0.0),
                                       window=c.get("window", 0), decay=DECAY, slopes=s.get("slopes"),
                                       prefix_len=s.get("prefix_len"), doc_start=s.get("doc_start"))
        if "dst" in s:
            s["dst_tables"] = lsa.LsaPagedTables(**s["dst"])
    return s


DECAY = 0.97      # of a page's score per decoded token


# ------------------------------------------------------------------------------ the operators
def run(state):
    s, c = state, state["case"]
    if c["op"] == "attn":
        if own:
            s["cache"].attend(s["q"], s["out"])
        else:
            _plain_attn(s, c)
        return {"out": s["out"], "score": s["score"]} if c["score"] else {"out": s["out"]}
    if c["op"] == "evict":
        if own:
            s["cache"].evict(c["budget"], c["sink"], c["recent"], dst=s["dst_tables"])
        else:
            _plain_evict(s, c)
        return {k: v for k, v in s["dst"].items() if k != "tail_len"}
    if own:
        s["cache"].append(s["k"], s["v"], s["tok_off"], dst=s["dst_tables"])
    else:
        _plain_append(s, c)
    return dict(s["dst"], pool=s["pool"])


def _plain_attn(s, c):
    B, E = s["block_table"].shape
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    live = torch.arange(E, device="cuda")[None] < s["n_entries"][:, None]
    at = s["block_pos"].long()[:, :, None] * PAGE + torch.arange(PAGE, device="cuda")      # [B,E,64]
    last = (s["n_entries"].long() - 1).clamp(min=0)
    now = s["block_pos"].long().gather(1, last[:, None]) * PAGE + s["tail_len"].long()[:, None] - 1
    in_tail = torch.arange(E, device="cuda")[None] == last[:, None]
    sees = live[:, :, None] & (~in_tail[:, :, None] | (torch.arange(PAGE, device="cuda") < s["tail_len"][:, None, None]))
    low = s["doc_start"].long()[:, None] if c["docs"] else torch.zeros_like(now)
    low = torch.maximum(low, now - c["window"] + 1) if c["window"] else low
    pre = s["prefix_len"].long()[:, None] if c["prefix"] else torch.zeros_like(now)
    sees &= (at < pre[:, :, None]) | (at >= low[:, :, None])
    sees = sees.reshape(B, 1, 1, E * PAGE)
    kv = s["pool"][torch.where(live, s["block_table"], 0).long()]                          # [B,E,2,Hkv,64,d]
    k, v = (kv[:, :, x].transpose(1, 2).float().reshape(B, Hkv, E * PAGE, d) for x in (0, 1))
    q = s["q"].float().reshape(B, Hkv, H // Hkv, d)
    z = (q @ k.transpose(2, 3)) * s["scale"]                                               # [B,Hkv,G,T]
    z = c["cap"] * torch.tanh(z / c["cap"]) if c["cap"] else z
    if c["slopes"]:      # far positions: the bias and the difference to the largest in 64 bits
        far = (now[:, :, None] - at).double().reshape(B, 1, 1, E * PAGE)
        z = z.double() - s["slopes"].double().reshape(1, Hkv, H // Hkv, 1) * far
    z = z.masked_fill(~sees, float("-inf"))
    top = z.amax(3, keepdim=True)
    w = torch.exp((z - torch.where(top == float("-inf"), 0, top)).float())
    w = w / w.sum(3, keepdim=True).clamp(min=1e-38)
    o = w @ torch.where(sees.reshape(B, 1, E * PAGE, 1), v, 0)
    s["out"].copy_(o.reshape(B, H, d))
    if c["score"]:
        mass = w.sum((1, 2)).reshape(B, E, PAGE).sum(2)
        s["score"].copy_(torch.where(live, s["score"] * DECAY + mass, s["score"]))


def _plain_evict(s, c):
    E = s["score"].shape[1]
    j = torch.arange(E, device="cuda")[None]
    n = s["n_entries"].long()[:, None]
    over = n > c["budget"]
    live = j < n
    bound = live & ((j < c["sink"]) | (j >= n - c["recent"]))
    rank_by = torch.where(live & ~bound, s["score"], float("-inf"))
    order = torch.sort(rank_by, dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, j.expand_as(order))
    keep = live & (~over | bound | (rank < c["budget"] - c["sink"] - c["recent"]))
    to = torch.cumsum(keep, 1) - 1
    d = s["dst"]
    b, i = keep.nonzero(as_tuple=True)
    for name in ("block_table", "block_pos", "score"):
        d[name][b, to[b, i]] = s[name][b, i]
    d["n_entries"].copy_(keep.sum(1))
    gone = live & ~keep
    b, i = gone.nonzero(as_tuple=True)
    d["free_list"][b, s["free_cnt"].long()[b] + (torch.cumsum(gone, 1) - 1)[b, i]] = s["block_table"][b, i]
    d["free_cnt"].copy_(s["free_cnt"] + gone.sum(1))


def _plain_append(s, c):
    n, tail, have = (s[x].long() for x in ("n_entries", "tail_len", "free_cnt"))
    B = n.shape[0]
    off = s["tok_off"].long() if c["new"] else torch.arange(B + 1, device="cuda")
    new = off[1:] - off[:-1]
    held = torch.where(n > 0, (n - 1) * PAGE + tail, 0)
    total = held + new
    n_out = (total + PAGE - 1) // PAGE
    # pages taken from the top of each stack, in order
    E, F = s["block_table"].shape[1], s["free_list"].shape[1]
    j = torch.arange(E, device="cuda")[None]
    opened = (j >= n[:, None]) & (j < n_out[:, None])
    top = (have[:, None] - 1 - (j - n[:, None])).clamp(0, F - 1)
    table = torch.where(opened, s["free_list"].gather(1, top), s["block_table"])
    before = torch.where(n > 0, s["block_pos"].long().gather(1, (n - 1).clamp(min=0)[:, None])[:, 0], -1)
    d = s["dst"]
    d["block_table"].copy_(table)
    d["block_pos"].copy_(torch.where(opened, before[:, None] + 1 + j - n[:, None], s["block_pos"]))
    d["score"].copy_(torch.where(opened, 0, s["score"]))
    d["n_entries"].copy_(n_out)
    d["tail_len"].copy_(torch.where(n_out > 0, total - (n_out - 1) * PAGE, 0))
    d["free_cnt"].copy_(have - (n_out - n))
    i = torch.arange(s["k"].shape[0], device="cuda")
    b = torch.bucketize(i, off[1:], right=True)
    at = held[b] + i - off[b]
    page = table[b, at // PAGE].long()
    s["pool"][page, 0, :, at % PAGE] = s["k"]
    s["pool"][page, 1, :, at % PAGE] = s["v"]


# ------------------------------------------------------------------------------ what they cost
def work(case):
    c = case
    if c["op"] == "attn":
        p = _attn_plan(c)
        seen = int(p["sees"].sum())
        pages = int(p["sees"].any(2).sum())
        size = 2 * (2 * seen * c["Hkv"] * c["d"] + 2 * c["B"] * c["H"] * c["d"])
        return {"bytes": size + pages * 8 + c["B"] * 8 + (8 * int(p["n"].sum()) if c["score"] else 0),
                "flops": 4.0 * c["H"] * c["d"] * seen}
    if c["op"] == "evict":
        n = _evict_plan(c)
        kept = int(np.minimum(n, c["budget"]).sum())
        return {"bytes": 12 * int(n.sum()) + 12 * kept + 4 * int(n.sum() - kept) + 16 * c["B"], "flops": 0}
    held, new = _append_plan(c)
    return {"bytes": 2 * 2 * 2 * int(new.sum()) * c["Hkv"] * c["d"] + 24 * c["B"], "flops": 0}


def exact(case, seed):
    """Attention from its definition, one sequence and key head at a time, in 64 bits. The other two
    operators compute no numbers: they move and compare what they are given."""
    if case["op"] != "attn":
        return None
    c, s = case, prepare(case, seed)
    B, G = c["B"], c["H"] // c["Hkv"]
    out = torch.zeros(B, c["H"], c["d"], dtype=torch.float64, device="cuda")
    score = s["score"].double() * DECAY if c["score"] else None
    p = _attn_plan(c)
    for b in range(B):
        n = int(p["n"][b])
        if c["score"]:
            score[b, n:] = s["score"][b, n:].double()
        seen = torch.from_numpy(p["sees"][b, :n].reshape(-1)).cuda().nonzero()[:, 0]
        if seen.numel() == 0:
            continue
        at = torch.from_numpy((p["pos"][b, :n, None] * PAGE + np.arange(PAGE)).reshape(-1)).cuda()[seen]
        for h in range(c["Hkv"]):
            rows = s["pool"][s["block_table"][b, :n].long(), :, h]                # [n,2,64,d]
            key = rows[:, 0].reshape(-1, c["d"])[seen].double()
            val = rows[:, 1].reshape(-1, c["d"])[seen].double()
            heads = slice(h * G, (h + 1) * G)
            z = key @ s["q"][b, heads].double().T * float(s["scale"])             # [tokens, G]
            if c["cap"]:
                z = c["cap"] * torch.tanh(z / c["cap"])
            if c["slopes"]:
                z = z + s["slopes"][heads].double() * (at - int(p["last"][b])).double()[:, None]
            w = torch.softmax(z, 0)
            out[b, heads] = w.T @ val
            if c["score"]:
                score[b].index_add_(0, seen // PAGE, w.sum(1))
    return {"out": out, "score": score} if c["score"] else {"out": out}
