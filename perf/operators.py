"""Measured cases of the attention side of a decoder layer over a paged key-value cache.

The W12 matrices of a layer give q, k and v and take the attention's output; what
lies between them is four operators, each with its plain form in elementary torch
operations:

  plan    page tables, positions and cache slots of a step's tokens, from the
          requests' lengths and a ring of free pages
  store   per-head RMS norm of q and k, position rotation, and the write of k and
          v into the cache (BF16, or 8 bits with a scale per token and head)
  read    cached rows back as BF16, by slot
  attend  attention of the new tokens (one, or a block or tree of drafted ones)
          over the cached ones

Head layouts are those of the benchmark's decoder layer (q 6144 and k, v 1024
columns: 48 and 8 heads of 128, or 24 and 4 heads of 256) and generic ones.
"""
import math
import random

import torch

own = False

EPS = 1e-6
ROPE_ROWS = 32768
BF16_MAX_BYTES = 2.2e9  # keys and values of the largest attend case


def listed():
    return [
        # one request adds one token: a chat with a single user, latency alone
        {"name": "plan-one", "op": "plan", "requests": 1, "kv": 500, "new": 1, "page": 16, "blocks": 64, "trim": False},
        # a busy server's step: every request brings up to 32 drafted or prompt
        # tokens, finished ones give their pages back
        {"name": "plan-busy", "op": "plan", "requests": 1024, "kv": 3000, "new": 32, "page": 16, "blocks": 512,
         "trim": True},
        # one token of one request through a layer: latency alone
        {"name": "store-one", "op": "store", "tokens": 1, "heads": 48, "kv_heads": 8, "dim": 128, "page": 16,
         "cache": "bf16", "norm": True, "rot": 128, "interleaved": False},
        # drafted tokens of a dozen requests into an 8-bit cache, half of each head rotated
        {"name": "store-verify-q8", "op": "store", "tokens": 97, "heads": 48, "kv_heads": 8, "dim": 128, "page": 64,
         "cache": "q8", "norm": True, "rot": 64, "interleaved": False},
        # a chunk of long prompts
        {"name": "store-prompt", "op": "store", "tokens": 8192, "heads": 24, "kv_heads": 4, "dim": 256, "page": 32,
         "cache": "bf16", "norm": True, "rot": 256, "interleaved": True},
        # a short shared prefix, taken out of an 8-bit cache
        {"name": "read-q8", "op": "read", "tokens": 1000, "kv_heads": 8, "dim": 128, "page": 16, "cache": "q8"},
        # a long conversation moved to another cache
        {"name": "read-long", "op": "read", "tokens": 30000, "kv_heads": 4, "dim": 256, "page": 64, "cache": "bf16"},
        # one request's next token after a short conversation: latency alone
        {"name": "attend-one", "op": "attend", "requests": 1, "kv": 777, "new": 1, "heads": 48, "kv_heads": 8,
         "dim": 128, "page": 16, "cache": "bf16", "window": 0, "tree": False},
        # a full batch on a layer with a sliding window and small heads
        {"name": "attend-window", "op": "attend", "requests": 128, "kv": 6000, "new": 1, "heads": 64, "kv_heads": 8,
         "dim": 64, "page": 16, "cache": "bf16", "window": 1024, "tree": False},
        # trees of up to 16 drafted tokens verified at once, 8-bit cache
        {"name": "attend-tree-q8", "op": "attend", "requests": 8, "kv": 16000, "new": 16, "heads": 48, "kv_heads": 8,
         "dim": 128, "page": 64, "cache": "q8", "window": 0, "tree": True},
        # two users with whole books in their prompts
        {"name": "attend-long", "op": "attend", "requests": 2, "kv": 100001, "new": 1, "heads": 24, "kv_heads": 4,
         "dim": 256, "page": 128, "cache": "bf16", "window": 0, "tree": False},
        # a server's batch of ordinary conversations
        {"name": "attend-batch", "op": "attend", "requests": 64, "kv": 8000, "new": 1, "heads": 48, "kv_heads": 8,
         "dim": 128, "page": 32, "cache": "bf16", "window": 0, "tree": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "store", "store", "read", "attend", "attend", "attend", "attend"])
    page = rng.choice([16, 32, 48, 64, 128])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    cache = rng.choice(["bf16", "bf16", "q8"])
    if op == "plan":
        requests = _log_int(rng, 1, 1024)
        kv = _log_int(rng, 16, 8000)
        new = rng.choice([1, 1, 4, 7, 16, 32])
        blocks = -(-(kv + new) // page) + 3 + rng.randrange(64)
        return {"op": op, "requests": requests, "kv": kv, "new": new, "page": page, "blocks": blocks,
                "trim": rng.random() < 0.5}
    if op == "store":
        group = rng.choice([1, 3, 4, 6, 8])
        tokens = _log_int(rng, 1, max(1, 50_000_000 // (kv_heads * (group + 2) * dim)) if kv_heads * group * dim > 6144
                          else 8192)
        interleaved = rng.random() < 0.4
        return {"op": op, "tokens": tokens, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "page": page,
                "cache": cache, "norm": rng.random() < 0.7, "rot": rng.choice([dim, dim, dim // 2, 0]),
                "interleaved": interleaved}
    if op == "read":
        return {"op": op, "tokens": _log_int(rng, 1, 30000), "kv_heads": min(kv_heads, 1024 // dim), "dim": dim,
                "page": page, "cache": cache}
    group = rng.choice([1, 2, 4, 6, 6, 8, 12])
    requests = _log_int(rng, 1, 128)
    new = rng.choice([1, 1, 1, 2, 5, 8, 16])
    size = 4 * kv_heads * dim
    most = min(120000, int(BF16_MAX_BYTES / size / requests / 1.5),
               int(6e12 / (4 * kv_heads * group * dim) / new / requests / 500))
    kv = _log_int(rng, 16, max(17, most))
    window = rng.choice([0, 0, 0, _log_int(rng, 16, 4096)])
    return {"op": op, "requests": requests, "kv": kv, "new": new, "heads": kv_heads * group, "kv_heads": kv_heads,
            "dim": dim, "page": page, "cache": cache, "window": window, "tree": new > 1 and rng.random() < 0.5}


# ---------------------------------------------------------------- inputs
def _attend_lengths(case):
    """Cached lengths (new tokens included) and new tokens of each request: they
    depend on the case alone, so that its work does; the seed only orders them."""
    n, kv = case["requests"], case["kv"]
    new = [case["new"] - (case["new"] // 2 if b % 3 == 2 else 0) for b in range(n)]
    if n == 1:
        return [max(kv, new[0])], new
    total = [max(int(kv * (0.5 + (0.618033988749895 * (b + 1)) % 1.0)), new[b]) for b in range(n)]
    return total, new


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g).to(torch.bfloat16)


def _cache(case, pages, g):
    """Keys and values of every page: [pages, kv_heads, page, dim], BF16, or
    8-bit whole numbers with a scale per row ([..., 0] of k, [..., 1] of v)."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    if case["cache"] == "bf16":
        return {"k": torch.randn(shape, device="cuda", generator=g, dtype=torch.bfloat16),
                "v": torch.randn(shape, device="cuda", generator=g, dtype=torch.bfloat16), "scales": None}
    return {"k": torch.randint(-127, 128, shape, device="cuda", generator=g, dtype=torch.int8),
            "v": torch.randint(-127, 128, shape, device="cuda", generator=g, dtype=torch.int8),
            "scales": torch.rand(shape[:3] + (2,), device="cuda", generator=g) * 0.01 + 0.01}


def _rope_table(rot):
    if not rot:
        return None
    freq = 1e6 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = torch.arange(ROPE_ROWS, device="cuda", dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _slots(count, pages, page, g):
    """Distinct slots in random pages; now and then a token that has none (-1)."""
    slots = torch.randperm(pages * page, device="cuda", generator=g)[:count]
    pad = torch.rand(count, device="cuda", generator=g) < 0.02
    if count > 4:
        slots = torch.where(pad, torch.full_like(slots, -1), slots)
    return slots


def _prepare_plan(case, seed):
    rng = random.Random(seed)
    g = _generator(seed)
    n, page, blocks = case["requests"], case["page"], case["blocks"]
    lens = [rng.randint(0, min(case["kv"], blocks * page - case["new"])) for _ in range(n)]
    new = [case["new"] if case["new"] == 1 else rng.randint(0, case["new"]) for _ in range(n)]
    owned = []
    for b in range(n):
        if case["trim"] and rng.random() < 0.05:  # a finished request
            lens[b], new[b] = 0, 0
            owned.append(rng.randint(0, blocks))
        else:  # pages kept from drafted tokens that were not accepted, now and then
            owned.append(min(blocks, -(-lens[b] // page) + (rng.random() < 0.2)))
    pages = n * (blocks + -(-case["new"] // page) + 1)
    ids = torch.randperm(pages, device="cuda", generator=g, dtype=torch.int32)
    held = torch.tensor(owned, device="cuda", dtype=torch.int32)
    col = torch.arange(blocks, device="cuda", dtype=torch.int32)
    start = torch.cumsum(held, 0, dtype=torch.int32) - held
    at = (start[:, None] + col[None]).clamp(max=pages - 1)
    tables = torch.where(col[None] < held[:, None], ids[at.long()], torch.full_like(at, -1))
    free = pages - sum(owned)
    head = rng.randrange(1 << 20)
    ring = torch.full((pages,), -1, device="cuda", dtype=torch.int32)
    ring[(head + torch.arange(free, device="cuda")) % pages] = ids[pages - free:]
    dev = lambda v, t: torch.tensor(v, device="cuda", dtype=t)  # noqa: E731
    return {"case": case, "lens": dev(lens, torch.int32), "new": dev(new, torch.int32), "owned": held,
            "tables": tables.contiguous(), "ring": ring, "ring_state": dev([head, head + free], torch.int64)}


def _prepare_store(case, seed):
    g = _generator(seed)
    t, h, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    pages = -(-t // case["page"]) + 3
    weight = lambda: (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(torch.bfloat16)  # noqa: E731
    return {"case": case, "q": _randn(g, t, h * d), "k": 3 * _randn(g, t, hk * d), "v": _randn(g, t, hk * d),
            "q_norm": weight() if case["norm"] else None, "k_norm": weight() if case["norm"] else None,
            "rope": _rope_table(case["rot"]),
            "positions": torch.randint(0, ROPE_ROWS, (t,), device="cuda", generator=g, dtype=torch.int32),
            "slots": _slots(t, pages, case["page"], g), **_cached(_cache(case, pages, g))}


def _prepare_read(case, seed):
    g = _generator(seed)
    pages = -(-case["tokens"] // case["page"]) + 3
    return {"case": case, "slots": _slots(case["tokens"], pages, case["page"], g), **_cached(_cache(case, pages, g))}


def _cached(cache):
    return {"cache_k": cache["k"], "cache_v": cache["v"], "scales": cache["scales"]}


def _prepare_attend(case, seed):
    rng = random.Random(seed)
    g = _generator(seed)
    total, new = _attend_lengths(case)
    order = list(range(case["requests"]))
    rng.shuffle(order)
    total, new = [total[b] for b in order], [new[b] for b in order]
    page = case["page"]
    need = [-(-n // page) for n in total]
    pages = sum(need) + 3
    cache = _cache(case, pages, g)
    ids = torch.randperm(pages, device="cuda", generator=g, dtype=torch.int32)
    held = torch.tensor(need, device="cuda", dtype=torch.int32)
    start = torch.cumsum(held, 0, dtype=torch.int32) - held
    col = torch.arange(max(need), device="cuda", dtype=torch.int32)
    at = (start[:, None] + col[None]).clamp(max=pages - 1)
    tables = torch.where(col[None] < held[:, None], ids[at.long()], torch.full_like(at, -1)).contiguous()
    # what lies behind a request's last token is stale memory
    last = ids[(start + held - 1).long()].long()
    left = torch.tensor([n - (c - 1) * page for n, c in zip(total, need)], device="cuda")
    stale = (torch.arange(page, device="cuda")[None] >= left[:, None])[:, None, :, None]
    for name in ("k", "v") if case["cache"] == "bf16" else ("scales",):
        cache[name][last] = torch.where(stale, torch.full_like(cache[name][last], float("nan")), cache[name][last])
    tokens = sum(new)
    tree = None
    if case["tree"]:  # bit j of a token's mask: it attends to new token j of its request
        masks = []
        for n in new:
            m = []
            for i in range(n):
                m.append((m[rng.randrange(max(0, i - 4), i)] if i else 0) | 1 << i)
            masks += m
        tree = torch.tensor(masks, device="cuda", dtype=torch.int64).to(torch.int32)
    dev = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
    return {"case": case, "q": _randn(g, tokens, case["heads"] * case["dim"]), "tables": tables,
            "lens": dev([a - b for a, b in zip(total, new)]), "cu_new": dev([sum(new[:b]) for b in range(len(new) + 1)]),
            "tree": tree, **_cached(cache)}


def prepare(case, seed):
    return {"plan": _prepare_plan, "store": _prepare_store, "read": _prepare_read,
            "attend": _prepare_attend}[case["op"]](case, seed)


# ---------------------------------------------------------------- plain forms
def _plain_plan(s):
    case, page = s["case"], s["case"]["page"]
    tables, ring = s["tables"], s["ring"]
    n, blocks = tables.shape
    tokens = n * case["new"]
    lens, new, owned = s["lens"].long(), s["new"].long(), s["owned"].long()
    need = (lens + new + page - 1) // page
    grow = (need - owned).clamp(min=0)
    drop = (owned - need).clamp(min=0) if case["trim"] else torch.zeros_like(owned)
    head, tail = s["ring_state"][0], s["ring_state"][1]
    given = torch.cumsum(grow, 0) - grow
    dropped = torch.cumsum(drop, 0) - drop
    col = torch.arange(blocks, device=tables.device)[None]
    taken = ring[(head + given[:, None] + col - owned[:, None]) % ring.numel()]
    is_new = (col >= owned[:, None]) & (col < need[:, None])
    is_old = (col >= need[:, None]) & (col < (need + drop)[:, None])
    to = torch.where(is_old, (tail + dropped[:, None] + col - need[:, None]) % ring.numel(), ring.numel())
    wide = torch.cat([ring, ring[:1]])
    wide[to.reshape(-1)] = tables.reshape(-1)
    ring.copy_(wide[:-1])
    tables.copy_(torch.where(is_new, taken, tables))
    cu = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)])
    t = torch.arange(tokens, device=tables.device)
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=n - 1)
    real = t < cu[-1]
    at = lens[b] + t - cu[b]
    slots = tables[b, (at // page).clamp(max=blocks - 1)].long() * page + at % page
    return {"tables": tables, "owned": torch.maximum(owned, need).sub(drop).to(torch.int32) if not case["trim"]
            else need.to(torch.int32), "ring": ring, "ring_state": s["ring_state"] + torch.stack([grow.sum(), drop.sum()]),
            "cu_new": cu.to(torch.int32), "positions": torch.where(real, at, 0).to(torch.int32),
            "slots": torch.where(real, slots, -1)}


def _plain_head(x, weight, rope, positions, interleaved):
    """RMS norm over a head and rotation of its first columns, in 32 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    if rope is None:
        return x
    rot = rope.shape[1]
    row = rope[positions.long()][:, None]
    cos, sin = row[..., :rot // 2], row[..., rot // 2:]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_read(s):
    pages, hk, page, d = s["cache_k"].shape
    slots = s["slots"]
    at = slots.clamp(min=0)
    out = {}
    for i, name in enumerate(("k", "v")):
        rows = s["cache_" + name][at // page, :, at % page].float()
        if s["scales"] is not None:
            rows = rows * s["scales"][at // page, :, at % page, i][..., None]
        out[name] = torch.where((slots >= 0)[:, None, None], rows, torch.zeros_like(rows)).to(torch.bfloat16)
    return out


def _plain_store(s):
    case = s["case"]
    t, d, page = case["tokens"], case["dim"], case["page"]
    q = _plain_head(s["q"].view(t, -1, d), s["q_norm"], s["rope"], s["positions"], case["interleaved"])
    k = _plain_head(s["k"].view(t, -1, d), s["k_norm"], s["rope"], s["positions"], case["interleaved"])
    rows = {"k": k, "v": s["v"].view(t, -1, d).float()}
    slots = s["slots"]
    here = slots >= 0
    at = torch.where(here, slots, slots.max().clamp(min=0))  # a token without a slot repeats a stored one
    src = torch.arange(t, device=slots.device)
    src = torch.where(here, src, slots.argmax())
    for i, name in enumerate(("k", "v")):
        x = rows[name][src]
        if s["scales"] is None:
            x = torch.where(here.any(), x, s["cache_" + name][at // page, :, at % page].float())
            s["cache_" + name][at // page, :, at % page] = x.to(torch.bfloat16)
        else:
            scale = x.abs().amax(-1) / 127.0
            x = torch.where(scale[..., None] > 0, x / scale[..., None], torch.zeros_like(x)).round().clamp(-127, 127)
            s["cache_" + name][at // page, :, at % page] = x.to(torch.int8)
            s["scales"][at // page, :, at % page, i] = scale
    q = q.to(torch.bfloat16)
    if s["scales"] is None:
        return {"q": q, "k": s["cache_k"], "v": s["cache_v"]}
    return {"q": q, **_plain_read(s), "scales": s["scales"]}


def _plain_attend(s):
    case = s["case"]
    d, hk, group, most = case["dim"], case["kv_heads"], case["heads"] // case["kv_heads"], case["new"]
    tables, lens, cu = s["tables"], s["lens"].long(), s["cu_new"].long()
    n, blocks = tables.shape
    new = cu[1:] - cu[:-1]
    q = s["q"].view(-1, hk, group, d)
    at = tables.clamp(min=0).long()
    length = blocks * case["page"]
    rows = {}
    key = torch.arange(length, device=q.device)
    inside = key[None] < (lens + new)[:, None]
    for i, name in enumerate(("k", "v")):
        x = s["cache_" + name][at].float()
        if s["scales"] is not None:
            x = x * s["scales"][at][..., i, None]
        x = x.permute(0, 2, 1, 3, 4).reshape(n, hk, length, d)
        rows[name] = torch.where(inside[:, None, :, None], x, torch.zeros_like(x))
    step = torch.arange(most, device=q.device)
    token = (cu[:-1, None] + step).clamp(max=q.shape[0] - 1)
    asked = q[token].float().permute(0, 2, 1, 3, 4).reshape(n, hk, most * group, d)
    score = asked @ rows["k"].transpose(2, 3) / math.sqrt(d)
    own_at = lens[:, None] + step
    if s["tree"] is None:
        seen = key[None, None] <= own_at[..., None]
    else:
        bit = (key[None] - lens[:, None]).clamp(0, 31)
        drawn = (s["tree"][token].long()[..., None] >> bit[:, None]) & 1
        seen = (key[None] < lens[:, None])[:, None] | ((drawn > 0) & ((key[None] - lens[:, None]) < 32)[:, None])
    seen = seen & inside[:, None]
    if case["window"]:
        seen = seen & (key[None, None] > own_at[..., None] - case["window"])
    seen = seen[:, None, :, None].expand(n, hk, most, group, length).reshape(n, hk, most * group, length)
    score = torch.where(seen, score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    weight = torch.exp(score - top)
    total = weight.sum(-1, keepdim=True)
    out = weight @ rows["v"] / torch.where(total > 0, total, torch.ones_like(total))
    lse = top + torch.log(total)
    t = torch.arange(q.shape[0], device=q.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[b]
    out = out.view(n, hk, most, group, d)[b, :, i].to(torch.bfloat16)
    return {"out": out.reshape(-1, case["heads"] * d),
            "lse": lse.view(n, hk, most, group)[b, :, i].reshape(-1, case["heads"])}


# ---------------------------------------------------------------- this framework's calls
def _kept(s):
    """The handles that a program makes once for its cache, tables and buffers."""
    from lossless_bit_weight_encode_gb300 import KVCache, KVPages, KVStep

    case, kept = s["case"], {}
    if "cache_k" in s:
        kept["cache"] = KVCache(s["cache_k"], s["cache_v"], s["scales"])
    if case["op"] == "plan":
        kept["pages"] = KVPages(s["tables"], s["owned"], s["ring"], s["ring_state"], case["page"])
        kept["step"] = kept["pages"].step(case["requests"] * case["new"], max_new=case["new"])
        kept["owned_out"] = torch.empty_like(s["owned"])
        kept["ring_state_out"] = torch.empty_like(s["ring_state"])
    if case["op"] == "store":
        kept["step"] = KVStep(positions=s["positions"], slots=s["slots"])
        kept["q_out"] = torch.empty_like(s["q"])
    if case["op"] == "attend":
        kept["step"] = KVStep(s["tables"], s["lens"], s["cu_new"], max_new=case["new"], tree=s["tree"])
        kept["out"] = torch.empty_like(s["q"])
        kept["lse"] = torch.empty(s["q"].shape[0], case["heads"], device="cuda")
    return kept


def _own(s):
    case = s["case"]
    kept = s.get("kept")
    if kept is None:
        kept = s["kept"] = _kept(s)
    if case["op"] == "plan":
        step = kept["step"]
        kept["pages"].plan(s["lens"], s["new"], step, trim=case["trim"], owned_out=kept["owned_out"],
                           ring_state_out=kept["ring_state_out"])
        return {"tables": s["tables"], "owned": kept["owned_out"], "ring": s["ring"],
                "ring_state": kept["ring_state_out"], "cu_new": step.cu_new, "positions": step.positions,
                "slots": step.slots}
    cache = kept["cache"]
    if case["op"] == "store":
        q = cache.store(s["q"], s["k"], s["v"], kept["step"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS,
                        rope=s["rope"], interleaved=case["interleaved"], out=kept["q_out"])
        if s["scales"] is None:
            return {"q": q, "k": s["cache_k"], "v": s["cache_v"]}
        k, v = cache.read(s["slots"])
        return {"q": q, "k": k, "v": v, "scales": s["scales"]}
    if case["op"] == "read":
        k, v = cache.read(s["slots"])
        return {"k": k, "v": v}
    cache.attend(s["q"], kept["step"], window=case["window"], out=kept["out"], lse=kept["lse"])
    return {"out": kept["out"], "lse": kept["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"plan": _plain_plan, "store": _plain_store, "read": _plain_read,
            "attend": _plain_attend}[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "plan":
        # lengths, counts and pages held in and out; a position and a slot for
        # each token; a page from the ring into the table for each page of new
        # tokens
        n, tokens = case["requests"], case["requests"] * case["new"]
        return {"bytes": n * 20 + 4 + 32 + tokens * 12 + 8 * n * case["new"] / case["page"], "flops": 0}
    d, hk, t = case["dim"], case["kv_heads"], case.get("tokens", 0)
    held = hk * (2 * d if case["cache"] == "bf16" else d + 4)  # bytes of a token's keys, and of its values
    if case["op"] == "read":
        return {"bytes": t * (8 + 2 * held + 4 * hk * d), "flops": 0 if case["cache"] == "bf16" else 2 * t * hk * d}
    if case["op"] == "store":
        h = case["heads"]
        data = t * (4 * h * d + 4 * hk * d + 2 * held + 12 + 4 * case["rot"])
        if case["cache"] == "q8":  # the stored rows are read back
            data += t * (8 + 2 * held + 4 * hk * d)
        return {"bytes": data, "flops": t * (h + hk) * (4 * d * case["norm"] + 3 * case["rot"]) + 4 * t * hk * d}
    total, new = _attend_lengths(case)
    h, tokens = case["heads"], sum(new)
    window = case["window"]
    seen = sum(min(n, window + m - 1) if window else n for n, m in zip(total, new))  # keys read
    pairs = sum(m * (min(n, window) if window else n) for n, m in zip(total, new))
    return {"bytes": seen * 2 * held + tokens * h * (4 * d + 4), "flops": 4 * h * d * pairs}


# ---------------------------------------------------------------- from the definition, in 64 bits
def _exact_rows(x, weight, rope, positions, interleaved):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
    if rope is None:
        return x
    half = rope.shape[1] // 2
    turn = rope.double()[positions.long()]
    turn = torch.complex(turn[:, :half], turn[:, half:])[:, None]
    first = torch.arange(half, device=x.device) * (2 if interleaved else 1)
    second = first + (1 if interleaved else half)
    z = torch.complex(x[..., first], x[..., second]) * turn
    x = x.clone()
    x[..., first], x[..., second] = z.real, z.imag
    return x


def _exact_held(s, name):
    x = s["cache_" + name].double()
    if s["scales"] is not None:
        x = x * s["scales"][..., 0 if name == "k" else 1].double()[..., None]
    return x


def _exact_store(s):
    case = s["case"]
    t, d, page = case["tokens"], case["dim"], case["page"]
    q = _exact_rows(s["q"].view(t, -1, d), s["q_norm"], s["rope"], s["positions"], case["interleaved"])
    k = _exact_rows(s["k"].view(t, -1, d), s["k_norm"], s["rope"], s["positions"], case["interleaved"])
    keep = torch.nonzero(s["slots"] >= 0)[:, 0]
    slot = s["slots"][keep]
    got = {"q": q}
    scales = None if s["scales"] is None else s["scales"].double()
    for name, x in (("k", k), ("v", s["v"].view(t, -1, d).double())):
        if scales is None:
            held = s["cache_" + name].double()
            held[slot // page, :, slot % page] = x[keep]
            got[name] = held
            continue
        scale = x.abs().max(-1).values / 127
        x = torch.round(x / scale.clamp(min=1e-300)[..., None]) * scale[..., None]
        scales[slot // page, :, slot % page, 0 if name == "k" else 1] = scale[keep]
        got[name] = torch.zeros_like(x).index_copy(0, keep, x[keep])
    if scales is not None:
        got["scales"] = scales
    return got


def _exact_attend(s):
    case = s["case"]
    d, hk, page = case["dim"], case["kv_heads"], case["page"]
    cu, lens = s["cu_new"].tolist(), s["lens"].tolist()
    out = torch.zeros(cu[-1], case["heads"], d, device="cuda", dtype=torch.float64)
    lse = torch.zeros(cu[-1], case["heads"], device="cuda", dtype=torch.float64)
    q = s["q"].view(cu[-1], hk, -1, d).double()
    for b, past in enumerate(lens):
        m = cu[b + 1] - cu[b]
        pages = s["tables"][b, :-(-(past + m) // page)].long()
        one = {**s, "cache_k": s["cache_k"][pages], "cache_v": s["cache_v"][pages],
               "scales": None if s["scales"] is None else s["scales"][pages]}
        k, v = (_exact_held(one, x).transpose(1, 2).reshape(-1, hk, d)[:past + m] for x in ("k", "v"))
        for i in range(m):
            t = cu[b] + i
            first = max(0, past + i - case["window"] + 1) if case["window"] else 0
            if s["tree"] is None:
                keys = torch.arange(first, past + i + 1, device="cuda")
            else:
                mask = int(s["tree"][t]) & 0xFFFFFFFF
                keys = torch.cat([torch.arange(min(first, past), past, device="cuda"),
                                  torch.tensor([past + j for j in range(m) if mask >> j & 1 and past + j >= first],
                                               device="cuda", dtype=torch.int64)])
            score = torch.einsum("hgd,khd->hgk", q[t], k[keys]) / d ** 0.5
            out[t] = torch.einsum("hgk,khd->hgd", torch.softmax(score, -1), v[keys]).reshape(-1, d)
            lse[t] = torch.logsumexp(score, -1).reshape(-1)
    return {"out": out.reshape(cu[-1], -1), "lse": lse}


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers throughout
    s = prepare(case, seed)
    if case["op"] == "store":
        return _exact_store(s)
    if case["op"] == "attend":
        return _exact_attend(s)
    at, page = s["slots"].clamp(min=0), case["page"]
    return {name: _exact_held(s, name)[at // page, :, at % page] * (s["slots"] >= 0)[:, None, None]
            for name in ("k", "v")}
