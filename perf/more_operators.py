"""Measured cases of several continuations of one prompt: beam search, parallel samples and
requests behind one system prompt, over the paged key-value cache.

A decoding step of such a batch needs, beside what `perf/operators.py` measures, four
operators, each here with its plain form in elementary torch operations:

  select  the best continuations of every request over its beams and the vocabulary,
          from the LM head's logits: log-softmax, running scores, sorted candidates,
          and the beams that go on
  fork    page tables after a step's selection: which page each beam now shares, takes
          over, copies or gives back, with the number of holders of every page, and
          how long the prefix is that a request's beams still share
  copy    pages copied inside a cache (BF16 or 8 bits with scales), one or several layers
          at once
  attend  attention of new tokens whose requests share a prefix: its keys and values are
          read once for all of them, then each request's own ones

Head layouts are those of the benchmark's decoder layer (48 and 8 heads of 128, or 24 and
4 of 256) and generic ones; the vocabulary of 151936 is its LM head's.
"""
import math
import random

import torch

own = False

MOST_KV_BYTES = 6.5e8  # keys and values that the largest attend case reads
MOST_LOGITS = 128 * 151936


def listed():
    return [
        # a single user with four beams: latency alone
        {"name": "select-one", "op": "select", "requests": 1, "beams": 4, "vocab": 151936, "dtype": "bf16",
         "allowed": 0.0, "eos": True},
        # constrained output (a grammar allows a tenth of the tokens), fp32 logits, odd sizes
        {"name": "select-grammar", "op": "select", "requests": 7, "beams": 5, "vocab": 50257, "dtype": "fp32",
         "allowed": 0.1, "eos": True},
        # a server's beam search: sixteen requests with eight beams each
        {"name": "select-batch", "op": "select", "requests": 16, "beams": 8, "vocab": 151936, "dtype": "bf16",
         "allowed": 0.0, "eos": True},
        # page tables of a single user's four beams
        {"name": "fork-one", "op": "fork", "requests": 1, "beams": 4, "kv": 700, "prompt": 500, "page": 16,
         "blocks": 64},
        # a server's step: 128 requests with eight beams, some of them finished
        {"name": "fork-busy", "op": "fork", "requests": 128, "beams": 8, "kv": 3000, "prompt": 2500, "page": 16,
         "blocks": 256},
        # the last, partly filled pages of 32 beams after a selection, in eight layers at once
        {"name": "copy-beams", "op": "copy", "pairs": 32, "used": 0.6, "rows": True, "layers": 8, "kv_heads": 8,
         "dim": 128, "page": 32, "cache": "bf16"},
        # whole pages moved to other places of a pool
        {"name": "copy-move", "op": "copy", "pairs": 2500, "used": 1.0, "rows": False, "layers": 1, "kv_heads": 8,
         "dim": 128, "page": 64, "cache": "bf16"},
        # four beams of a single user after a short prompt: latency alone
        {"name": "attend-beams", "op": "attend", "groups": 1, "members": 4, "prefix": 1500, "kv": 40, "new": 1,
         "heads": 48, "kv_heads": 8, "dim": 128, "page": 16, "cache": "bf16", "tree": False},
        # a server's conversations behind one system prompt
        {"name": "attend-system", "op": "attend", "groups": 1, "members": 64, "prefix": 4000, "kv": 225, "new": 1,
         "heads": 48, "kv_heads": 8, "dim": 128, "page": 32, "cache": "bf16", "tree": False},
        # eight beams of each of eight requests, 8-bit cache
        {"name": "attend-beams-q8", "op": "attend", "groups": 8, "members": 8, "prefix": 6000, "kv": 130, "new": 1,
         "heads": 48, "kv_heads": 8, "dim": 128, "page": 64, "cache": "q8", "tree": False},
        # trees of four drafted tokens for the parallel samples of four prompts, wide heads
        {"name": "attend-draft", "op": "attend", "groups": 4, "members": 5, "prefix": 10000, "kv": 333, "new": 4,
         "heads": 24, "kv_heads": 4, "dim": 256, "page": 64, "cache": "bf16", "tree": True},
        # sixteen samples over a whole book
        {"name": "attend-book", "op": "attend", "groups": 1, "members": 16, "prefix": 100000, "kv": 700, "new": 1,
         "heads": 48, "kv_heads": 8, "dim": 128, "page": 64, "cache": "bf16", "tree": False},
    ]


def _log_int(rng, lo, hi):
    hi = max(lo, hi)
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["select", "select", "fork", "copy", "attend", "attend", "attend", "attend"])
    page = rng.choice([16, 32, 48, 64, 128])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    cache = rng.choice(["bf16", "bf16", "q8"])
    if op == "select":
        vocab = _log_int(rng, 1000, 200000)
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        beams = rng.choice([1, 2, 3, 4, 5, 8, 16, 32])
        most = MOST_LOGITS // vocab // beams // (2 if dtype == "fp32" else 1)
        return {"op": op, "requests": _log_int(rng, 1, min(256, most)), "beams": beams, "vocab": vocab, "dtype": dtype,
                "allowed": rng.choice([0.0, 0.0, rng.uniform(0.05, 0.9)]), "eos": rng.random() < 0.7}
    if op == "fork":
        beams = rng.choice([2, 3, 4, 5, 8, 16])
        kv = _log_int(rng, 32, 4000)
        prompt = rng.randint(16, kv)
        return {"op": op, "requests": _log_int(rng, 1, 1024 // beams), "beams": beams, "kv": kv, "prompt": prompt,
                "page": page, "blocks": min(256, -(-(kv + 8) // page) + rng.randrange(40))}
    if op == "copy":
        layers = 1 if cache == "q8" else rng.choice([1, 1, 3, 8, 16])
        size = layers * kv_heads * page * dim * 4
        return {"op": op, "pairs": _log_int(rng, 1, min(4000, int(3e8 / size))), "used": rng.uniform(0.3, 1.0),
                "rows": rng.random() < 0.5, "layers": layers, "kv_heads": kv_heads, "dim": dim, "page": page,
                "cache": cache}
    group = rng.choice([1, 2, 4, 6, 6, 8, 12])
    new = rng.choice([1, 1, 1, 2, 4])
    groups = rng.choice([1, 1, 2, 3, 8])
    members = _log_int(rng, 2, max(2, 64 // groups // new))
    size = 4 * kv_heads * dim
    kv = _log_int(rng, new + 1, min(1000, int(MOST_KV_BYTES / 3 / size / groups / members)))
    most = min(int(MOST_KV_BYTES / 2 / size / groups), int(1.2e11 / (4 * kv_heads * group * dim * new * groups * members)),
               int(1.2e10 / (2 * size * groups * members)))
    return {"op": op, "groups": groups, "members": members, "prefix": _log_int(rng, 64, min(100000, most)), "kv": kv,
            "new": new, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "page": page, "cache": cache,
            "tree": new > 1 and rng.random() < 0.5}


# ---------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _dev(v, dtype=torch.int32):
    return torch.tensor(v, device="cuda", dtype=dtype)


def _cache(case, pages, g):
    """Keys and values of every page: [pages, kv_heads, page, dim], BF16, or 8-bit whole
    numbers with a scale per row ([..., 0] of k, [..., 1] of v)."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    if case["cache"] == "bf16":
        return {"k": torch.randn(shape, device="cuda", generator=g, dtype=torch.bfloat16),
                "v": torch.randn(shape, device="cuda", generator=g, dtype=torch.bfloat16), "scales": None}
    return {"k": torch.randint(-127, 128, shape, device="cuda", generator=g, dtype=torch.int8),
            "v": torch.randint(-127, 128, shape, device="cuda", generator=g, dtype=torch.int8),
            "scales": torch.rand(shape[:3] + (2,), device="cuda", generator=g) * 0.01 + 0.01}


def _prepare_select(case, seed):
    g, rng = _generator(seed), random.Random(seed)
    n, b, v = case["requests"], case["beams"], case["vocab"]
    logits = torch.randn(n * b, v, device="cuda", generator=g) * 2.5
    eos = rng.randrange(v) if case["eos"] else -1
    if case["eos"]:  # near the top now and then: some beams end
        logits[:, eos] += 12.0 * (torch.rand(n * b, device="cuda", generator=g) < 0.4)
    allowed = None
    if case["allowed"]:
        words = -(-v // 32)
        bits = torch.rand(n * b, words, 32, device="cuda", generator=g) < case["allowed"]
        allowed = (bits.long() << torch.arange(32, device="cuda")).sum(-1)
        allowed = torch.where(allowed >= 2 ** 31, allowed - 2 ** 32, allowed).to(torch.int32)
    scores = -torch.rand(n, b, device="cuda", generator=g).cumsum(1) * 2 - 10
    return {"case": case, "logits": logits.to(torch.bfloat16) if case["dtype"] == "bf16" else logits, "eos": eos,
            "allowed": allowed, "scores": scores}


def _prepare_fork(case, seed):
    """Tables as earlier steps left them: a request's beams share the prompt's pages and
    what followed up to some step; behind that each has its own.  Parents are random beams
    of the same request; a twentieth of the requests has finished (no parents)."""
    rng, g = random.Random(seed), _generator(seed)
    n, b, page, blocks = case["requests"], case["beams"], case["page"], case["blocks"]
    rows = n * b
    total = [rng.randint(case["prompt"], min(case["kv"], blocks * page)) for _ in range(n)]
    held = [-(-t // page) for t in total]
    shared = [rng.randint(min(case["prompt"], t) // page, t // page) for t in total]
    fresh = sum(s + b * (h - s) for s, h in zip(shared, held))
    pages = rows * (blocks + 2) + 7
    ids = torch.randperm(pages, device="cuda", generator=g, dtype=torch.int32)
    col = torch.arange(blocks, device="cuda")[None, None]
    s, h = _dev(shared, torch.int64)[:, None, None], _dev(held, torch.int64)[:, None, None]
    beam = torch.arange(b, device="cuda")[None, :, None]
    start = [0]
    for x, y in zip(shared, held):
        start.append(start[-1] + x + b * (y - x))
    at = _dev(start[:-1], torch.int64)[:, None, None] + torch.where(col < s, col, s + beam * (h - s) + col - s)
    tables = torch.where(col < h, ids[at.clamp(max=pages - 1)], -1).reshape(rows, blocks).contiguous()
    shares = torch.zeros(pages, device="cuda", dtype=torch.int32)
    shares[tables.view(n, b, blocks)[:, 0][torch.arange(blocks, device="cuda")[None] < s[:, 0]].long()] = b - 1
    free = pages - fresh
    head = rng.randrange(1 << 20)
    ring = torch.full((pages,), -1, device="cuda", dtype=torch.int32)
    ring[(head + torch.arange(free, device="cuda")) % pages] = ids[fresh:]
    lens, parents = [], []
    for r in range(n):
        done = n > 1 and rng.random() < 0.05
        keep = max(1, total[r] - rng.choice([0, 0, 0, 1, 5]))  # drafted tokens that were not accepted
        for _ in range(b):
            parents.append(-1 if done else r * b + rng.randrange(b))
            lens.append(keep)
    return {"case": case, "tables": tables, "owned": _dev([x for x in held for _ in range(b)]), "ring": ring,
            "ring_state": _dev([head, head + free], torch.int64), "shares": shares, "parents": _dev(parents),
            "lens": _dev(lens), "groups": torch.arange(n + 1, device="cuda", dtype=torch.int32) * b}


def _prepare_copy(case, seed):
    rng, g = random.Random(seed), _generator(seed)
    n = case["pairs"]
    pages = 2 * n + 5
    layers = [_cache(case, pages, g) for _ in range(case["layers"])]
    ids = torch.randperm(pages, device="cuda", generator=g, dtype=torch.int32)
    use = torch.rand(n, device="cuda", generator=g) < case["used"]
    use[rng.randrange(n)] = True
    none = torch.full((n,), -1, device="cuda", dtype=torch.int32)
    rows = None
    if case["rows"]:  # tokens that the pages hold so far
        rows = torch.randint(1, case["page"] + 1, (n,), device="cuda", generator=g, dtype=torch.int32)
    dst = torch.where(use, ids[n:2 * n], none)
    token = torch.arange(case["page"], device="cuda")
    slots = (ids[n:2 * n, None].long() * case["page"] + token).reshape(-1).contiguous()
    return {"case": case, "layers": layers, "src": torch.where(use, ids[:n], none), "dst": dst, "rows": rows,
            "slots": slots}


def _attend_lengths(case):
    """Prefix of each group, own cached tokens (new ones included) and new tokens of each
    request: they depend on the case alone, so that its work does."""
    page, members = case["page"], case["members"]
    prefix = [max(page, int(case["prefix"] * (1.0 - 0.3 * (0.618033988749895 * g % 1.0))) // page * page)
              for g in range(case["groups"])]
    kv, new = [], []
    for b in range(case["groups"] * members):
        new.append(case["new"] - (case["new"] // 2 if b % 3 == 2 else 0))
        kv.append(max(new[-1], int(case["kv"] * (0.5 + 0.618033988749895 * (b + 1) % 1.0))))
    return prefix, kv, new


def _prepare_attend(case, seed):
    rng, g = random.Random(seed), _generator(seed)
    prefix, own_kv, new = _attend_lengths(case)
    page, members = case["page"], case["members"]
    n = len(own_kv)
    ahead = [p // page for p in prefix]
    behind = [-(-t // page) for t in own_kv]
    width = max(ahead[b // members] + behind[b] for b in range(n))
    pages = sum(ahead) + sum(behind) + 3
    cache = _cache(case, pages, g)
    ids = torch.randperm(pages, device="cuda", generator=g, dtype=torch.int32)
    tables = torch.full((n, width), -1, device="cuda", dtype=torch.int32)
    at = sum(ahead)
    for b in range(n):
        grp = b // members
        first = sum(ahead[:grp])
        tables[b, :ahead[grp]] = ids[first:first + ahead[grp]]
        tables[b, ahead[grp]:ahead[grp] + behind[b]] = ids[at:at + behind[b]]
        at += behind[b]
    # what lies behind a request's last token is stale memory
    last = _dev([ahead[b // members] + behind[b] - 1 for b in range(n)], torch.int64)
    last = tables[torch.arange(n, device="cuda"), last].long()
    left = _dev([t - (c - 1) * page for t, c in zip(own_kv, behind)], torch.int64)
    stale = (torch.arange(page, device="cuda")[None] >= left[:, None])[:, None, :, None]
    for name in ("k", "v") if case["cache"] == "bf16" else ("scales",):
        cache[name][last] = torch.where(stale, torch.full_like(cache[name][last], float("nan")), cache[name][last])
    tree = None
    if case["tree"]:  # bit j of a token's mask: it attends to new token j of its request
        masks = []
        for m in new:
            one = []
            for i in range(m):
                one.append((one[rng.randrange(i)] if i else 0) | 1 << i)
            masks += one
        tree = _dev(masks)
    shared = [prefix[b // members] for b in range(n)]
    q = torch.randn(sum(new), case["heads"] * case["dim"], device="cuda", generator=g).to(torch.bfloat16)
    return {"case": case, "q": q, "tables": tables, "lens": _dev([s + t - m for s, t, m in zip(shared, own_kv, new)]),
            "cu_new": _dev([sum(new[:b]) for b in range(n + 1)]), "tree": tree, "prefix_lens": _dev(shared),
            "prefix_cu": _dev([g * members for g in range(case["groups"] + 1)]), "cache_k": cache["k"],
            "cache_v": cache["v"], "scales": cache["scales"]}


def prepare(case, seed):
    return {"select": _prepare_select, "fork": _prepare_fork, "copy": _prepare_copy,
            "attend": _prepare_attend}[case["op"]](case, seed)


# ---------------------------------------------------------------- plain forms
def _allowed(s):
    v = s["case"]["vocab"]
    bit = (s["allowed"][..., None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
    return bit.reshape(s["allowed"].shape[0], -1)[:, :v] != 0


def _plain_select(s):
    """In 64 bits: candidates of different beams may lie closer than 32 bits tell."""
    case = s["case"]
    n, b, v = case["requests"], case["beams"], case["vocab"]
    take = 2 * b
    x = s["logits"].double()
    x = torch.where(torch.isnan(x), -math.inf, x)
    if s["allowed"] is not None:
        x = torch.where(_allowed(s), x, -math.inf)
    top = x.amax(-1, keepdim=True)
    safe = torch.where(torch.isinf(top), 0.0, top)
    total = torch.exp(x - safe).sum(-1, keepdim=True)
    score = s["scores"].double().reshape(n * b, 1) + ((x - safe) - torch.log(total))
    score = torch.where(torch.isnan(score), -math.inf, score).view(n, b * v)
    kept = torch.topk(score, take, -1).values[:, -1:]  # equal scores go by their place
    above, level = score > kept, score == kept
    chosen = above | (level & (torch.cumsum(level, 1) <= take - above.sum(1, keepdim=True)))
    at = torch.where(chosen, torch.cumsum(chosen, 1) - 1, take)
    place = torch.arange(b * v, device="cuda").expand(n, -1)
    cand = torch.zeros(n, take + 1, device="cuda", dtype=torch.int64).scatter_(1, at, place)[:, :take]
    order = torch.sort(torch.gather(score, 1, cand), dim=1, descending=True, stable=True).indices
    cand = torch.gather(cand, 1, order)
    best = torch.gather(score, 1, cand)
    real = best > -math.inf
    token = torch.where(real, cand % v, -1)
    parent = torch.where(real, torch.arange(n, device="cuda")[:, None] * b + cand // v, -1)
    goes_on = real & (token != s["eos"])
    order = torch.sort((~goes_on).to(torch.int8), dim=-1, stable=True).indices[:, :b]
    on = torch.gather(goes_on, 1, order)

    def next_of(t, none):
        return torch.where(on, torch.gather(t, 1, order), none)

    return {"cand_tokens": token.to(torch.int32), "cand_parents": parent.to(torch.int32), "cand_scores": best.float(),
            "tokens": next_of(token, -1).to(torch.int32).reshape(-1),
            "parents": next_of(parent, -1).to(torch.int32).reshape(-1), "scores": next_of(best, -math.inf).float()}


def _plain_fork(s):
    page = s["case"]["page"]
    tables, owned, ring, shares = s["tables"], s["owned"].long(), s["ring"], s["shares"]
    rows, blocks = tables.shape
    count = shares.numel()
    parent = s["parents"].long()
    real = (parent >= 0) & (parent < rows)
    source = torch.where(real, parent, 0)
    keep = torch.where(real, torch.minimum(s["lens"].long().clamp(min=0), owned[source] * page), 0)
    need = (keep + page - 1) // page
    part = keep % page != 0
    col = torch.arange(blocks, device="cuda")[None]
    held = (col < owned[:, None]) & (tables >= 0) & (tables < count)
    old = torch.where(held, tables, count).long()  # page `count` stands for none
    new = torch.where(col < need[:, None], old[source], count)
    last = part[:, None] & (col == need[:, None] - 1)
    full = torch.where(last, count, new)
    holders = torch.zeros(count + 1, device="cuda", dtype=torch.int64)
    holders[:count] = shares.long() + 1
    holders.index_add_(0, old.reshape(-1), torch.full((rows * blocks,), -1, device="cuda"))
    holders.index_add_(0, full.reshape(-1), torch.ones(rows * blocks, device="cuda", dtype=torch.int64))
    # a partly filled page goes to the first child that wants it if no one else holds it
    i = torch.arange(rows, device="cuda")
    wanted = torch.where(part, new[i, (need - 1).clamp(min=0)], count)
    first = torch.full((count + 1,), rows, device="cuda", dtype=torch.int64)
    first.scatter_reduce_(0, wanted, i, "amin")
    first = torch.where(holders == 0, first, rows)
    takes = (wanted < count) & (first[wanted] == i)
    copies = (wanted < count) & ~takes
    # the other children copy it to pages from the ring, in row order
    head, tail = s["ring_state"][0], s["ring_state"][1]
    rank = torch.cumsum(copies.long(), 0) - 1
    given = copies & (rank < tail - head)
    fresh = ring[(head + rank) % ring.numel()]
    fresh = torch.where(given, fresh, -1)
    # pages that no one holds any more go back, by entry and then by row
    by_entry = old.t().reshape(-1)
    is_freed = torch.zeros(count + 1, device="cuda", dtype=torch.bool)
    is_freed[by_entry] = True
    is_freed &= (holders == 0) & (first == rows)
    is_freed[count] = False
    where = torch.full((count + 1,), rows * blocks, device="cuda", dtype=torch.int64)
    where.scatter_reduce_(0, by_entry, torch.arange(rows * blocks, device="cuda"), "amin")
    freed = is_freed[by_entry] & (where[by_entry] == torch.arange(rows * blocks, device="cuda"))
    at = torch.cumsum(freed.long(), 0) - 1
    wide = torch.cat([ring, ring[:1]])
    wide[torch.where(freed, (tail + at) % ring.numel(), ring.numel())] = by_entry.to(torch.int32)
    ring.copy_(wide[:-1])
    # holders - 1 of every page that is held; 0 of free ones
    after = holders[:count] + (first[:count] < rows).long() - 1
    shares.copy_(after.clamp(min=0))
    entry = torch.where(last & copies[:, None], fresh[:, None].long(), torch.where(new < count, new, -1))
    tables.copy_(torch.where(col < need[:, None], entry, tables.long()))
    s["owned"].copy_(need)
    s["ring_state"].add_(torch.stack([given.sum(), freed.sum()]))
    lens = keep.to(torch.int32)
    # the leading full pages that all live rows of a group have in common
    cu = s["groups"].long()
    group = torch.searchsorted(cu, i, right=True) - 1
    whole = torch.where(col < (keep // page)[:, None], tables, -1)
    live = keep > 0
    lead = torch.full((cu.numel() - 1,), rows, device="cuda", dtype=torch.int64)
    lead.scatter_reduce_(0, group, torch.where(live, i, rows), "amin")
    same = (whole == whole[lead[group].clamp(max=rows - 1)]) & (whole >= 0)
    run_ = torch.cumprod(same.long(), 1).sum(1)
    shortest = torch.full((cu.numel() - 1,), blocks, device="cuda", dtype=torch.int64)
    shortest.scatter_reduce_(0, group, torch.where(live, run_, blocks), "amin")
    alive = torch.zeros(cu.numel() - 1, device="cuda", dtype=torch.int64).index_add_(0, group, live.long())
    prefix = torch.where(live & (alive[group] > 1), shortest[group] * page, 0).to(torch.int32)
    none = torch.full_like(fresh, -1)
    return {"tables": tables, "owned": s["owned"], "ring": ring, "ring_state": s["ring_state"], "shares": shares,
            "lens": lens, "src": torch.where(given, wanted.to(torch.int32), none), "dst": fresh,
            "rows": torch.where(given, keep % page, 0).to(torch.int32), "prefix": prefix}


def _plain_read(layer, slots, page):
    out = {}
    for i, name in enumerate(("k", "v")):
        rows = layer[name][slots // page, :, slots % page].float()
        if layer["scales"] is not None:
            rows = rows * layer["scales"][slots // page, :, slots % page, i][..., None]
        out[name] = rows.to(torch.bfloat16)
    return out


def _plain_copy(s):
    page = s["case"]["page"]
    here = (s["src"] >= 0) & (s["dst"] >= 0)
    # a pair that is none repeats the first real one
    one = here.to(torch.int8).argmax()
    src = torch.where(here, s["src"], s["src"][one]).long()
    dst = torch.where(here, s["dst"], s["dst"][one]).long()
    mask = None
    if s["rows"] is not None:
        rows = torch.where(here, s["rows"], s["rows"][one])
        mask = (torch.arange(page, device="cuda")[None] < rows[:, None])[:, None, :, None]
    for layer in s["layers"]:
        for t in (layer["k"], layer["v"], layer["scales"]):
            if t is not None:
                x = t[src]
                t[dst] = x if mask is None else torch.where(mask, x, t[dst])
    return _copied(s)


def _copied(s, cache=None):
    """Every layer's cache; of an 8-bit one the rows of the pages that were written to, as
    the values that they stand for."""
    page = s["case"]["page"]
    if s["case"]["cache"] == "bf16":
        return [{"k": layer["k"], "v": layer["v"]} for layer in s["layers"]]
    if cache is None:
        return [_plain_read(layer, s["slots"], page) for layer in s["layers"]]
    return [dict(zip(("k", "v"), c.read(s["slots"]))) for c in cache]


def _plain_attend(s):
    case = s["case"]
    d, hk, group, most = case["dim"], case["kv_heads"], case["heads"] // case["kv_heads"], case["new"]
    tables, lens, cu = s["tables"], s["lens"].long(), s["cu_new"].long()
    n, blocks = tables.shape
    new = cu[1:] - cu[:-1]
    q = s["q"].view(-1, hk, group, d)
    length = blocks * case["page"]
    key = torch.arange(length, device=q.device)
    step = torch.arange(most, device=q.device)
    out = torch.zeros(q.shape[0], hk, group, d, device=q.device)
    lse = torch.zeros(q.shape[0], hk, group, device=q.device)
    for b0 in range(0, n, 8):  # eight requests at a time
        b = slice(b0, min(n, b0 + 8))
        at = tables[b].clamp(min=0).long()
        m = at.shape[0]
        inside = key[None] < (lens[b] + new[b])[:, None]
        rows = {}
        for i, name in enumerate(("k", "v")):
            x = s["cache_" + name][at].float()
            if s["scales"] is not None:
                x = x * s["scales"][at][..., i, None]
            x = x.permute(0, 2, 1, 3, 4).reshape(m, hk, length, d)
            rows[name] = torch.where(inside[:, None, :, None], x, torch.zeros_like(x))
        token = cu[:-1][b, None] + step
        mine = step[None] < new[b, None]
        token = torch.where(mine, token, cu[:-1][b, None])
        asked = q[token].float().permute(0, 2, 1, 3, 4).reshape(m, hk, most * group, d)
        score = asked @ rows["k"].transpose(2, 3) / math.sqrt(d)
        own_at = lens[b, None] + step
        if s["tree"] is None:
            seen = key[None, None] <= own_at[..., None]
        else:
            bit = (key[None] - lens[b, None]).clamp(0, 31)
            drawn = (s["tree"][token].long()[..., None] >> bit[:, None]) & 1
            seen = (key[None] < lens[b, None])[:, None] | ((drawn > 0) & ((key[None] - lens[b, None]) < 32)[:, None])
        seen = (seen & inside[:, None])[:, None, :, None].expand(m, hk, most, group, length)
        score = torch.where(seen.reshape(m, hk, most * group, length), score, -math.inf)
        top = score.amax(-1, keepdim=True)
        weight = torch.exp(score - top)
        total = weight.sum(-1, keepdim=True)
        y = (weight @ rows["v"] / total).view(m, hk, most, group, d).transpose(1, 2)
        z = (top + torch.log(total)).view(m, hk, most, group).transpose(1, 2)
        out[token[mine]] = y[mine]
        lse[token[mine]] = z[mine]
    return {"out": out.to(torch.bfloat16).reshape(-1, case["heads"] * d), "lse": lse.reshape(-1, case["heads"])}


# ---------------------------------------------------------------- this framework's calls
def _kept(s):
    """The handles that a program makes once for its caches, tables and buffers."""
    from lossless_bit_weight_encode_gb300 import Beams, KVCache, KVCopies, KVPages, KVPrefix, KVStep

    case, op = s["case"], s["case"]["op"]
    if op == "select":
        return {"beams": Beams(case["requests"], case["beams"], eos=s["eos"] if case["eos"] else None)}
    if op == "fork":
        return {"pages": KVPages(s["tables"], s["owned"], s["ring"], s["ring_state"], case["page"],
                                 shares=s["shares"]),
                "copies": KVCopies.empty(s["parents"].numel()), "lens_out": torch.empty_like(s["lens"]),
                "prefix": KVPrefix(s["groups"], torch.zeros_like(s["lens"]), max_requests=case["beams"])}
    if op == "copy":
        return {"caches": [KVCache(x["k"], x["v"], x["scales"]) for x in s["layers"]],
                "copies": KVCopies(s["src"], s["dst"], s["rows"])}
    prefix = KVPrefix(s["prefix_cu"], s["prefix_lens"], max_requests=case["members"])
    return {"cache": KVCache(s["cache_k"], s["cache_v"], s["scales"]), "out": torch.empty_like(s["q"]),
            "step": KVStep(s["tables"], s["lens"], s["cu_new"], max_new=case["new"], tree=s["tree"], prefix=prefix),
            "lse": torch.empty(s["q"].shape[0], case["heads"], device="cuda")}


def _own(s):
    kept = s.get("kept")
    if kept is None:
        kept = s["kept"] = _kept(s)
    op = s["case"]["op"]
    if op == "select":
        beams = kept["beams"]
        beams.select(s["logits"], allowed=s["allowed"], scores=s["scores"])
        return {"cand_tokens": beams.cand_tokens, "cand_parents": beams.cand_parents, "cand_scores": beams.cand_scores,
                "tokens": beams.tokens, "parents": beams.parents, "scores": beams.scores}
    if op == "fork":
        copies, prefix = kept["copies"], kept["prefix"]
        kept["pages"].fork(s["parents"], s["lens"], copies, prefix=prefix, lens_out=kept["lens_out"])
        return {"tables": s["tables"], "owned": s["owned"], "ring": s["ring"], "ring_state": s["ring_state"],
                "shares": s["shares"], "lens": kept["lens_out"], "src": copies.src, "dst": copies.dst,
                "rows": copies.rows, "prefix": prefix.lens}
    if op == "copy":
        caches = kept["caches"]
        caches[0].copy(kept["copies"], others=caches[1:])
        return _copied(s, caches)
    kept["cache"].attend(s["q"], kept["step"], out=kept["out"], lse=kept["lse"])
    return {"out": kept["out"], "lse": kept["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"select": _plain_select, "fork": _plain_fork, "copy": _plain_copy,
            "attend": _plain_attend}[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "select":
        rows, v = case["requests"] * case["beams"], case["vocab"]
        mask = 4 * -(-v // 32) if case["allowed"] else 0
        return {"bytes": rows * (v * (2 if case["dtype"] == "bf16" else 4) + mask + 4) + rows * 3 * 12,
                "flops": 4 * rows * v}
    if case["op"] == "fork":
        # lengths, parents and pages held in and out, copies and prefix lengths; the tables'
        # entries in and out
        rows = case["requests"] * case["beams"]
        return {"bytes": rows * 36 + 32 + 8 * rows * -(-case["prompt"] // case["page"]), "flops": 0}
    d, hk, page = case["dim"], case["kv_heads"], case["page"]
    row = hk * (2 * d if case["cache"] == "bf16" else d + 4)  # bytes of a token's keys, and of its values
    if case["op"] == "copy":
        tokens = case["pairs"] * case["used"] * (0.5 if case["rows"] else 1.0) * page
        data = case["layers"] * tokens * 2 * 2 * row + case["pairs"] * (12 if case["rows"] else 8)
        if case["cache"] == "q8":  # the pages are read back
            data += case["layers"] * case["pairs"] * page * (8 + 2 * row + 4 * hk * d)
        return {"bytes": data, "flops": 0}
    prefix, kv, new = _attend_lengths(case)
    h, tokens = case["heads"], sum(new)
    pairs = sum((prefix[b // case["members"]] + kv[b]) * new[b] for b in range(len(kv)))
    return {"bytes": (sum(prefix) + sum(kv)) * 2 * row + tokens * h * (4 * d + 4), "flops": 4 * h * d * pairs}


# ---------------------------------------------------------------- from the definition, in 64 bits
def _exact_select(case, s):
    b, v = case["beams"], case["vocab"]
    if case["requests"] * b * v > 3e7:
        return None
    x = s["logits"].double()
    if s["allowed"] is not None:
        word = torch.arange(v, device="cuda")
        x = x.masked_fill(((s["allowed"][:, word // 32] >> (word % 32).to(torch.int32)) & 1) == 0, -math.inf)
    x = torch.log_softmax(x, -1).view(-1, b, v) + s["scores"].double()[..., None]
    best = x.flatten(1).sort(descending=True).values[:, :2 * b].float()
    if case["eos"]:
        x[..., s["eos"]] = -math.inf
    on = x.flatten(1).sort(descending=True).values[:, :b].float()
    return {"cand_tokens": None, "cand_parents": None, "cand_scores": best.double(), "tokens": None, "parents": None,
            "scores": on.double()}


def _exact_copy(case, s):
    pairs = [(a, b, m) for a, b, m in zip(s["src"].tolist(), s["dst"].tolist(), [case["page"]] * case["pairs"]
                                          if s["rows"] is None else s["rows"].tolist()) if a >= 0 and b >= 0]
    got = []
    for layer in s["layers"]:
        values = {}
        for i, name in enumerate(("k", "v")):
            x = layer[name].double()
            if layer["scales"] is not None:
                x = x * layer["scales"][..., i, None].double()
            for a, b, m in pairs:
                x[b, :, :m] = x[a, :, :m]
            if layer["scales"] is not None:
                x = x.transpose(1, 2).reshape(-1, case["kv_heads"], case["dim"])[s["slots"]]
            values[name] = x
        got.append(values)
    return got


def _exact_attend(case, s):
    d, hk, page = case["dim"], case["kv_heads"], case["page"]
    cu, lens = s["cu_new"].tolist(), s["lens"].tolist()
    out = torch.zeros(cu[-1], case["heads"], d, device="cuda", dtype=torch.float64)
    lse = torch.zeros(cu[-1], case["heads"], device="cuda", dtype=torch.float64)
    q = s["q"].view(cu[-1], hk, -1, d).double()
    for b, past in enumerate(lens):
        m = cu[b + 1] - cu[b]
        ids = s["tables"][b, :-(-(past + m) // page)].long()
        kv = []
        for i, name in enumerate(("cache_k", "cache_v")):
            x = s[name][ids].double()
            if s["scales"] is not None:
                x = x * s["scales"][ids][..., i, None].double()
            kv.append(x.transpose(1, 2).reshape(-1, hk, d)[:past + m])
        for i in range(m):
            keys = list(range(past, past + i + 1))
            if s["tree"] is not None:
                mask = int(s["tree"][cu[b] + i]) & 0xFFFFFFFF
                keys = [past + j for j in range(m) if mask >> j & 1]
            keys = torch.cat([torch.arange(past, device="cuda"), _dev(keys, torch.int64)])
            score = torch.einsum("hgd,khd->hgk", q[cu[b] + i], kv[0][keys]) / d ** 0.5
            out[cu[b] + i] = torch.einsum("hgk,khd->hgd", torch.softmax(score, -1), kv[1][keys]).reshape(-1, d)
            lse[cu[b] + i] = torch.logsumexp(score, -1).reshape(-1)
    return {"out": out.reshape(cu[-1], -1), "lse": lse}


def exact(case, seed):
    if case["op"] == "fork":
        return None  # whole numbers throughout
    s = prepare(case, seed)
    return {"select": _exact_select, "copy": _exact_copy, "attend": _exact_attend}[case["op"]](case, s)
