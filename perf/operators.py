"""Cases of the verification step over a paged cache: pages, cache writes, attention, tree acceptance.

A verification step of speculative decoding takes R requests with a context in
a paged key/value cache and, for each, a segment of new elements (an anchor and
its drafted tokens, as a chain or as a tree).  The operators of that step:

  pages    dspark_page_map (pages and slots for the new elements out of a ring of
           free pages), then dspark_page_trim (the pages of rejected drafts back);
  store    dspark_kv_store (keys and values of the new elements into their slots);
  attend   dspark_tree_attention (each element over its context and its ancestors);
  tree     dspark_tree_pack (parents to ancestor masks and positions), then
           dspark_verify_tree (the accepted path under the target's logits);
  commit   dspark_kv_commit (the accepted path's keys and values moved to the front).

The caches hold, for pages of P tokens, Hk heads of D values and c = 16 / itemsize:
keys as [pages, Hk, D / c, P, c] and values as [pages, Hk, D, P].

With `own` false run() computes the same in plain torch operations.
"""
import numpy as np
import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0


# ---- sizes: a case fixes every length, a seed only the values ----

def _spread(n, lo, hi, step):
    """n whole numbers over [lo, hi], the ends among them where n > 1 (a fixed sequence)."""
    f = np.mod(np.arange(n) * step + 0.5, 1.0)
    x = lo + np.floor(f * (hi - lo + 1)).astype(np.int64)
    if n > 1:
        x[0], x[-1] = hi, lo
    return x


def _contexts(case):
    return _spread(case["R"], case["ctx_lo"], case["ctx_hi"], 0.6180339887498949)


def _counts(case):
    return _spread(case["R"], case["n_lo"], case["n_hi"], 0.7548776662466927)


def _starts(n):
    return np.concatenate([[0], np.cumsum(n)])


def _up(a, b):
    return -(-a // b)


def listed():
    return [
        # One step of a full batch of chains: an anchor and up to five drafts per request, the latency of the bookkeeping.
        {"name": "pages-step", "op": "pages", "R": 256, "ctx_lo": 1, "ctx_hi": 8191, "n_lo": 1, "n_hi": 6, "P": 16},
        # New prompts of a serving batch admitted at once, long ones among them.
        {"name": "pages-prompts", "op": "pages", "R": 64, "ctx_lo": 0, "ctx_hi": 100, "n_lo": 257, "n_hi": 16384, "P": 32},
        # Keys and values of one step of 256 chains.
        {"name": "store-step", "op": "store", "R": 256, "ctx_lo": 1, "ctx_hi": 1023, "n_lo": 1, "n_hi": 6, "P": 16,
         "Hk": 8, "D": 128, "type": "bf16", "cache": "bf16"},
        # A batch of prompts written to an 8-bit cache.
        {"name": "store-prompts-e4m3", "op": "store", "R": 12, "ctx_lo": 0, "ctx_hi": 40, "n_lo": 100, "n_hi": 4000, "P": 64,
         "Hk": 8, "D": 128, "type": "bf16", "cache": "e4m3"},
        # One request, one token, a short context: the latency of a single step.
        {"name": "attend-one", "op": "attend", "R": 1, "ctx_lo": 200, "ctx_hi": 200, "n_lo": 1, "n_hi": 1, "P": 16,
         "Hq": 16, "Hk": 2, "D": 64, "type": "bf16", "cache": "bf16", "tree": False, "lse": False},
        # A serving batch of chains (anchor + up to five drafts) over ragged contexts.
        {"name": "attend-chains", "op": "attend", "R": 64, "ctx_lo": 37, "ctx_hi": 8100, "n_lo": 1, "n_hi": 6, "P": 16,
         "Hq": 32, "Hk": 8, "D": 128, "type": "bf16", "cache": "bf16", "tree": False, "lse": False},
        # Wide trees, where the products weigh as much as the cache.
        {"name": "attend-trees-fp16", "op": "attend", "R": 24, "ctx_lo": 1000, "ctx_hi": 6000, "n_lo": 33, "n_hi": 64, "P": 32,
         "Hq": 64, "Hk": 8, "D": 128, "type": "fp16", "cache": "fp16", "tree": True, "lse": True},
        # A few requests with very long contexts and an 8-bit cache, small trees.
        {"name": "attend-long-e4m3", "op": "attend", "R": 6, "ctx_lo": 30000, "ctx_hi": 131000, "n_lo": 5, "n_hi": 16, "P": 64,
         "Hq": 32, "Hk": 8, "D": 128, "type": "bf16", "cache": "e4m3", "tree": True, "lse": False},
        # A few small trees over a small vocabulary: latency.
        {"name": "tree-small", "op": "tree", "R": 4, "n_lo": 2, "n_hi": 9, "V": 4096},
        # A batch of trees at a full vocabulary.
        {"name": "tree-batch", "op": "tree", "R": 32, "n_lo": 16, "n_hi": 64, "V": 129280},
        # The accepted paths of one layer.
        {"name": "commit-layer", "op": "commit", "R": 32, "ctx_lo": 10, "ctx_hi": 1000, "n_lo": 24, "n_hi": 48, "P": 16,
         "Hk": 8, "D": 128, "cache": "bf16", "layers": 1},
        # The accepted paths of all layers in one call, 8-bit cache.
        {"name": "commit-layers-e4m3", "op": "commit", "R": 64, "ctx_lo": 1, "ctx_hi": 500, "n_lo": 24, "n_hi": 64, "P": 32,
         "Hk": 8, "D": 128, "cache": "e4m3", "layers": 32},
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))

    op = rng.choice(["pages", "store", "attend", "attend", "attend", "tree", "commit"])
    P = rng.choice([16, 32, 64, 128])
    if op == "pages":
        R = log(1, 1000)
        hi = max(1, min(log(1, 16384), 500000 // R))
        return {"op": op, "R": R, "ctx_lo": 0, "ctx_hi": log(1, 9000), "n_lo": max(1, hi // rng.randint(1, 9)), "n_hi": hi, "P": P}
    if op == "store":
        R = log(1, 300)
        hi = max(1, min(log(1, 4000), 20000 // R))
        t = rng.choice(["bf16", "fp16"])
        return {"op": op, "R": R, "ctx_lo": 0, "ctx_hi": log(1, 1000), "n_lo": max(1, hi // rng.randint(1, 9)), "n_hi": hi, "P": P,
                "Hk": rng.choice([1, 2, 4, 8]), "D": rng.choice([64, 96, 128, 192, 256]), "type": t, "cache": rng.choice([t, t, "e4m3"])}
    if op == "attend":
        tree = rng.random() < 0.5
        # chains: a draft block, or now and then a piece of a prompt
        n = log(1, 64) if tree else log(1, 17) if rng.random() < 0.8 else log(17, 700)
        R = max(1, min(log(1, 256), 1500 // n))
        Hk, g = rng.choice([(8, 4), (8, 8), (4, 7), (2, 8), (1, 16), (16, 1), (8, 5)])
        D = rng.choice([64, 96, 128, 128, 192, 256])
        t = rng.choice(["bf16", "bf16", "fp16"])
        hi = max(16, min(log(16, 131000), int(2.4e8 / (R * Hk * D)) - n, int(2.5e10 / (R * n * Hk * g * D)) - n))
        return {"op": op, "R": R, "ctx_lo": rng.choice([0, 1, hi // 4, hi // 2, hi]), "ctx_hi": hi, "n_lo": max(1, n // rng.randint(1, 4)), "n_hi": n,
                "P": P, "Hq": Hk * g, "Hk": Hk, "D": D, "type": t, "cache": rng.choice([t, t, "e4m3"]), "tree": tree, "lse": rng.random() < 0.3}
    if op == "tree":
        V = rng.choice([4096, 32003, 50257, 129280, 151936])
        n = log(2, 64)
        R = max(1, min(log(1, 256), 150000000 // (V * n)))
        return {"op": op, "R": R, "n_lo": max(1, n // rng.randint(1, 4)), "n_hi": n, "V": V}
    R = log(1, 64)
    return {"op": op, "R": R, "ctx_lo": 0, "ctx_hi": log(1, 500), "n_lo": 24, "n_hi": rng.randint(24, 64), "P": P, "Hk": rng.choice([1, 2, 8]),
            "D": rng.choice([64, 128, 256]), "cache": rng.choice(["bf16", "fp16", "e4m3"]), "layers": rng.randint(1, 10)}


def work(case):
    n = _counts(case)
    N, R = int(n.sum()), case["R"]
    if case["op"] == "pages":
        ctx = _contexts(case)
        new, keep, P = ctx + n, ctx + np.minimum(n, 1), case["P"]
        took = int((_up(new, P) - _up(ctx, P)).sum())
        back = int((_up(new, P) - _up(keep, P)).sum())
        # lengths and starts in, lengths and slots out; a page id read and written for each page that moves
        return {"bytes": 4 * (2 * R + R + 1) + 4 * R + 8 * N + 8 * (took + back), "flops": N}
    if case["op"] == "tree":
        W = _up(case["n_hi"], 32)
        return {"bytes": 4 * N * case["V"] + 4 * N * (2 + W + 2) + 4 * R * (3 + case["n_hi"]), "flops": N * case["V"]}
    size = {"bf16": 2, "fp16": 2, "e4m3": 1}[case["cache"]]
    row = case["Hk"] * case["D"]
    if case["op"] == "store":
        return {"bytes": 2 * N * row * (2 + size) + 8 * N, "flops": 2 * N * row}
    if case["op"] == "commit":
        moved = int((_depths(case) * (1 + 1)).sum()) * row * size * 2 * case["layers"]
        return {"bytes": moved + 4 * R * (3 + case["n_hi"]), "flops": 0}
    ctx = _contexts(case)
    if case["tree"]:
        seen = sum(int(c) * int(k) + _tree_pairs(int(k)) for c, k in zip(ctx, n))
    else:
        seen = sum(int(c) * int(k) + int(k) * (int(k) + 1) // 2 for c, k in zip(ctx, n))
    b = 2 * int((ctx + n).sum()) * row * size + 4 * N * case["Hq"] * case["D"] + (4 * N * case["Hq"] if case["lse"] else 0)
    return {"bytes": b, "flops": 4 * seen * case["Hq"] * case["D"]}


# ---- trees: node 0 is the anchor, the first level wide, then by a fixed rule ----

def _parents(n):
    """Parents of n nodes in order of their depth: up to seven children of the anchor, then about two for each."""
    p = np.full(n, -1, np.int64)
    for i in range(1, n):
        p[i] = 0 if i <= 7 else (i - 8) // 2 + 1
    return p


def _ancestors(p):
    a = np.zeros((len(p), len(p)), bool)
    for i in range(len(p)):
        if p[i] >= 0:
            a[i] = a[p[i]]
        a[i, i] = True
    return a


def _tree_pairs(n):
    return int(_ancestors(_parents(n)).sum())


def _words(a, words):
    """Rows of truth values as 32-bit words, the lowest bit first."""
    pad = np.zeros((a.shape[0], words * 32), bool)
    pad[:, :a.shape[1]] = a
    return np.packbits(pad, axis=1, bitorder="little").view(np.int32)


def _depths(case):
    """Accepted drafts of each request of a commit case: two to four levels below the anchor."""
    n = _counts(case)
    return np.array([min(2 + r % 3, 3 if k >= 40 else 2) for r, k in enumerate(n)])


# ---- inputs ----

def _dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)


def _randn(gen, shape, dtype, std=1.0):
    x = torch.empty(shape, dtype=torch.float16 if dtype == torch.float8_e4m3fn else dtype, device=DEV)
    x.normal_(0.0, std, generator=gen)
    return x.to(dtype)


def _caches(gen, case, pages, std_k=1.0):
    t = TYPES[case["cache"]]
    c = 16 // torch.empty((), dtype=t).element_size()
    lead = (case["layers"],) if "layers" in case else ()
    Hk, D, P = case["Hk"], case["D"], case["P"]
    return _randn(gen, lead + (pages, Hk, D // c, P, c), t, std_k), _randn(gen, lead + (pages, Hk, D, P), t)


def _table(gen, lens, P, pages):
    """Pages in a random order, rows padded with -1."""
    need = _up(lens, P)
    width = max(1, int(need.max()))
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    start = _dev(_starts(need)[:-1])[:, None]
    col = torch.arange(width, device=DEV, dtype=torch.int32)[None, :]
    at = (start + col).clamp_(max=pages - 1).long()
    return torch.where(col < _dev(need)[:, None], order[at], torch.full_like(at, -1, dtype=torch.int32)), order


def _slots(table, first, n, P):
    r = np.repeat(np.arange(len(n)), n)
    pos = np.repeat(first, n) + np.arange(n.sum()) - np.repeat(_starts(n)[:-1], n)
    r, pos = _dev(r, torch.int64), _dev(pos, torch.int64)
    return table[r, pos // P].long() * P + pos % P


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed) * 2 + 1)
    rng = np.random.default_rng([int(seed), case["R"]])
    n, R = _counts(case), case["R"]
    N, op = int(n.sum()), case["op"]
    s = {"case": dict(case), "op": op, "cu": _dev(_starts(n)), "N": N}
    if op == "tree":
        V = case["V"]
        par = [_parents(int(k)) for k in n]
        flat = np.concatenate(par)
        tok = rng.integers(0, V, N).astype(np.int32)
        first = np.repeat(_starts(n)[:-1], n)
        logits = torch.empty((N, V), dtype=torch.float32, device=DEV).normal_(0.0, 2.0, generator=gen)
        # the target agrees with one child of most inner nodes
        hit = np.nonzero((flat >= 0) & (rng.random(N) < 0.45))[0]
        logits[_dev(first[hit] + flat[hit], torch.int64), _dev(tok[hit], torch.int64)] = 20.0
        s.update(logits=logits, tokens=_dev(tok), parents=_dev(flat), pos0=_dev(rng.integers(0, 9000, R)), nodes=case["n_hi"],
                 words=_up(case["n_hi"], 32))
        return s
    P = case["P"]
    ctx = _contexts(case)
    total = ctx + n
    if op == "pages":
        pages = int(_up(total, P).sum()) + 64
        held = int(_up(ctx, P).sum())
        table, order = _table(gen, ctx, P, pages)
        width = int(_up(total, P).max())
        full = torch.full((R, width), -1, dtype=torch.int32, device=DEV)
        w = min(width, table.shape[1])
        full[:, :w] = table[:, :w]
        # a ring of free pages: those that no request holds, from a place in the middle on
        head = pages // 3
        ring = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
        at = (torch.arange(pages - held, device=DEV) + head) % pages
        ring[at] = order[held:]
        s.update(cur=_dev(ctx), table=full, ring=ring, pool=_dev([head, pages - held, 0, 0]), keep=_dev(ctx + np.minimum(n, 1)), width=width)
        return s
    pages = int(_up(total, P).sum()) + 3
    table, _ = _table(gen, total, P, pages)
    s.update(table=table, ctx=_dev(ctx))
    if op == "commit":
        k, v = _caches(gen, case, pages)
        depth = _depths(case)
        path = np.full((R, case["n_hi"]), -1, np.int64)
        for r in range(R):
            # a path whose nodes all lie behind the positions that they move to, so that a pass can be made again
            node = {2: 8 + int(rng.integers(0, 2)), 3: 22 + int(rng.integers(0, 2))}[int(depth[r])]
            p = _parents(int(n[r]))
            walk = [node]
            while p[walk[-1]] >= 0:
                walk.append(int(p[walk[-1]]))
            walk = walk[::-1]
            walk[1] = 7 if walk[1] < 2 else walk[1]
            path[r, :len(walk)] = walk
            depth[r] = len(walk) - 1
        s.update(k=k, v=v, path=_dev(path), accepted=_dev(depth))
        return s
    scaled = case["cache"] == "e4m3"
    s["ks"] = (0.5 + torch.rand(case["Hk"], generator=gen, device=DEV)) * 0.05 if scaled else None
    s["vs"] = (0.5 + torch.rand(case["Hk"], generator=gen, device=DEV)) * 0.05 if scaled else None
    if op == "store":
        k, v = _caches(gen, case, pages)
        t = TYPES[case["type"]]
        s.update(k=k, v=v, slots=_slots(table, ctx, n, P), new_k=_randn(gen, (N, case["Hk"], case["D"]), t, 2.0),
                 new_v=_randn(gen, (N, case["Hk"], case["D"]), t))
        return s
    # 8-bit keys stand for values of about the size that 16-bit ones have
    k, v = _caches(gen, case, pages, 20.0 if scaled else 1.0)
    s.update(k=k, v=v, q=_randn(gen, (N, case["Hq"], case["D"]), TYPES[case["type"]], 1.5), nmax=case["n_hi"], mask=None)
    if case["tree"]:
        W = _up(case["n_hi"], 32)
        s["mask"] = _dev(np.concatenate([_words(_ancestors(_parents(int(c))), W) for c in n]))
    return s


# ---- the plain forms ----

def _keys(k, pages):
    """Keys of the pages `pages` [R, M] as fp32 [R, Hk, M * P, D]."""
    x = k.view(torch.uint8)[pages].view(k.dtype) if k.element_size() == 1 else k[pages]
    R, M, Hk, C, P, c = x.shape
    return x.permute(0, 2, 1, 4, 3, 5).reshape(R, Hk, M * P, C * c).float()


def _values(v, pages):
    x = v.view(torch.uint8)[pages].view(v.dtype) if v.element_size() == 1 else v[pages]
    R, M, Hk, D, P = x.shape
    return x.permute(0, 2, 1, 4, 3).reshape(R, Hk, M * P, D).float()


def _places(cu, N):
    """The request and the place in its segment of each element."""
    e = torch.arange(N, device=cu.device)
    r = (e[:, None] >= cu[None, 1:]).sum(1)
    return r, e - cu[r]


def _plain_attend(s):
    c = s["case"]
    q, cu, ctx, nmax = s["q"], s["cu"].long(), s["ctx"].long(), s["nmax"]
    N, Hq, D = q.shape
    Hk = c["Hk"]
    g = Hq // Hk
    R = ctx.numel()
    pages = s["table"].long().clamp(min=0)
    k, v = _keys(s["k"], pages), _values(s["v"], pages)
    if s["ks"] is not None:
        k, v = k * s["ks"][None, :, None, None], v * s["vs"][None, :, None, None]
    L = k.shape[2]
    n = cu[1:] - cu[:-1]
    i = torch.arange(nmax, device=q.device)
    at = (cu[:-1, None] + i).clamp(max=N - 1)
    x = q[at].float().reshape(R, nmax, Hk, g, D).permute(0, 2, 1, 3, 4).reshape(R, Hk, nmax * g, D)
    j = torch.arange(L, device=q.device)[None, :] - ctx[:, None]                  # place among the new elements
    if s["mask"] is not None:
        words = s["mask"][at].long()                                               # [R, nmax, W]
        jc = j.clamp(0, words.shape[2] * 32 - 1)
        bits = words.gather(2, (jc // 32)[:, None, :].expand(R, nmax, L)) >> (jc % 32)[:, None, :]
        own_ = (bits & 1).bool()
    else:
        own_ = j[:, None, :] <= i[None, :, None]
    seen = (j < 0)[:, None, :] | (own_ & (j >= 0)[:, None, :] & (j < n[:, None])[:, None, :])
    score = torch.matmul(x, k.transpose(2, 3).contiguous()) * (D ** -0.5)
    score = score.reshape(R, Hk, nmax, g, L)
    score = torch.where(seen[:, None, :, None, :], score, torch.full_like(score, -torch.inf))
    top = score.amax(-1, keepdim=True)
    safe = torch.where(top == -torch.inf, torch.zeros_like(top), top)
    p = torch.exp(score - safe)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(R, Hk, nmax * g, L), v).reshape(R, Hk, nmax, g, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    r, place = _places(cu, N)
    out = o[r, :, place].reshape(N, Hq, D).to(q.dtype)
    if not c["lse"]:
        return out
    return out, (safe + torch.log(total))[r, :, place, :, 0].reshape(N, Hq)


def _plain_pages(s):
    P, cur, cu, ring, table = s["case"]["P"], s["cur"].long(), s["cu"].long(), s["ring"], s["table"]
    pages, N, W = ring.numel(), s["N"], s["width"]
    head, count = s["pool"][0].long(), s["pool"][1].long()
    n = cu[1:] - cu[:-1]
    has, want = (cur + P - 1) // P, (cur + n + P - 1) // P
    fits = want <= W
    need = torch.where(fits, want - has, torch.zeros_like(has))
    before = need.cumsum(0) - need
    ok = fits & ((need == 0) | (before + need <= count))
    took = torch.where(ok, need, torch.zeros_like(need)).sum()
    new_len = torch.where(ok, cur + n, cur)
    col = torch.arange(W, device=cur.device)[None, :]
    fresh = ring[(head + before[:, None] + (col - has[:, None]).clamp(min=0)) % pages]
    table.copy_(torch.where((col >= has[:, None]) & (col < want[:, None]) & ok[:, None], fresh, table))
    r, place = _places(cu, N)
    pos = cur[r] + place
    slots = torch.where(ok[r], table[r, (pos // P).clamp(max=W - 1)].long() * P + pos % P, torch.full_like(pos, -1))
    failed = (~ok).sum()
    mapped = torch.stack([(head + took) % pages, count - took, failed, torch.zeros_like(failed)]).int()
    # the pages behind what is kept, to the ring's end
    keep = torch.minimum(s["keep"].long().clamp(min=0), new_len)
    has, want = (new_len + P - 1) // P, (keep + P - 1) // P
    give = has - want
    before = give.cumsum(0) - give
    gone = (col >= want[:, None]) & (col < has[:, None])
    to = (mapped[0] + mapped[1] + before[:, None] + col - want[:, None]) % pages
    ring = torch.cat([ring, ring.new_zeros(1)])
    ring[torch.where(gone, to, torch.full_like(to, pages))] = table
    s["ring"].copy_(ring[:pages])
    back = give.sum()
    trimmed = torch.stack([mapped[0].long(), mapped[1].long() + back, torch.zeros_like(back), torch.zeros_like(back)]).int()
    return table, slots, new_len.int(), mapped, trimmed, s["ring"]


def _to_cache(x, t, scale):
    if t != torch.float8_e4m3fn:
        return x.to(t)
    return (x.float() / scale[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(t)


def _plain_store(s):
    k, v, slots, P = s["k"], s["v"], s["slots"], s["case"]["P"]
    new_k, new_v = _to_cache(s["new_k"], k.dtype, s["ks"]), _to_cache(s["new_v"], v.dtype, s["vs"])
    N, Hk, D = new_k.shape
    raw = torch.uint8 if k.element_size() == 1 else torch.int16
    page, at = slots // P, slots % P
    k.view(raw)[page, :, :, at] = new_k.view(raw).reshape(N, Hk, k.shape[2], k.shape[4])
    v.view(raw)[page, :, :, at] = new_v.view(raw)
    return k, v


def _first_top(x):
    """The lowest index of each row's largest value."""
    i = torch.arange(x.shape[1], device=x.device, dtype=torch.int32)[None, :]
    return torch.where(x == x.amax(1, keepdim=True), i, torch.full_like(i, x.shape[1])).amin(1)


def _plain_tree(s):
    cu, par, tok, n, W, N = s["cu"].long(), s["parents"].long(), s["tokens"], s["nodes"], s["words"], s["N"]
    dev = cu.device
    R = cu.numel() - 1
    i = torch.arange(n, device=dev)
    live = i[None, :] < (cu[1:] - cu[:-1])[:, None]
    at = (cu[:-1, None] + i).clamp(max=N - 1)
    p = torch.where(live, par[at], torch.full_like(at, -1))                       # [R, n]
    link = (p[:, :, None] == i[None, None, :]).double()                            # child, parent
    up = torch.linalg.matrix_power(link + torch.eye(n, device=dev, dtype=torch.float64), n) > 0
    bits = torch.zeros((R, n, W * 32), dtype=torch.int64, device=dev)
    bits[:, :, :n] = up
    words = (bits.reshape(R, n, W, 32) << torch.arange(32, device=dev)).sum(-1)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).int()
    r, place = _places(cu, N)
    mask = words[r, place]
    pos = (s["pos0"].long()[:, None] + up.sum(2) - 1)[r, place].int()
    top = _first_top(s["logits"])
    t, x = top[at], tok[at]
    # a child is taken where its token is its parent's top and no earlier sibling's is
    match = live & (p >= 0) & (x == torch.gather(t, 1, p.clamp(min=0)))
    same = (p[:, :, None] == p[:, None, :]) & match[:, None, :] & (i[None, None, :] < i[None, :, None])
    taken = match & ~same.any(2)
    taken[:, 0] = True
    on = ((taken[:, None, :] | ~up).all(2)) & live & up[:, :, 0]
    accepted = on.sum(1) - 1
    path = torch.where(on, i[None, :], torch.full_like(at, n)).sort(1).values
    path = torch.where(path == n, torch.full_like(path, -1), path)
    last = torch.where(on, i[None, :], torch.zeros_like(at)).amax(1)
    return mask, pos, top, accepted.int(), path.int(), torch.gather(t, 1, last[:, None])[:, 0]


def _plain_commit(s):
    k, v, path, P = s["k"], s["v"], s["path"].long(), s["case"]["P"]
    raw = torch.uint8 if k.element_size() == 1 else torch.int16
    k8, v8 = k.view(raw), v.view(raw)
    ctx, acc = s["ctx"].long(), s["accepted"].long()
    r = torch.arange(path.shape[0], device=path.device)[:, None]
    i = torch.arange(path.shape[1], device=path.device)[None, :]
    move = (i >= 1) & (i <= acc[:, None])
    src = ctx[:, None] + torch.where(move, path, torch.zeros_like(path))
    dst = ctx[:, None] + torch.where(move, i.expand_as(path), torch.zeros_like(path))
    table = s["table"].long()
    sp, so, dp, do = table[r, src // P], src % P, table[r, dst // P], dst % P
    k8[:, dp, :, :, do] = k8[:, sp, :, :, so]
    v8[:, dp, :, :, do] = v8[:, sp, :, :, so]
    return k, v, (ctx + 1 + acc).int()


def run(s):
    op = s["op"]
    if own:
        import draft_head_step_amd as D
        if op == "pages":
            P = s["case"]["P"]
            slots, new_len, mapped = D.dspark_page_map(s["cur"], s["cu"], s["table"], s["ring"], s["pool"], P, s["N"])
            trimmed = D.dspark_page_trim(new_len, s["keep"], s["table"], s["ring"], mapped, P)
            return s["table"], slots, new_len, mapped, trimmed, s["ring"]
        if op == "store":
            D.dspark_kv_store(s["new_k"], s["new_v"], s["slots"], s["k"], s["v"], k_scale=s["ks"], v_scale=s["vs"])
            return s["k"], s["v"]
        if op == "attend":
            got = D.dspark_tree_attention(s["q"], s["k"], s["v"], s["table"], s["ctx"], s["cu"], tree_mask=s["mask"],
                                          k_scale=s["ks"], v_scale=s["vs"], want_lse=s["case"]["lse"])
            return got if s["case"]["lse"] else got[0]
        if op == "tree":
            mask, pos = D.dspark_tree_pack(s["parents"], s["cu"], s["words"], s["pos0"])
            accepted, path, nxt, top = D.dspark_verify_tree(s["logits"], s["cu"], s["tokens"], s["parents"], s["nodes"])
            return mask, pos, top, accepted, path, nxt
        return s["k"], s["v"], D.dspark_kv_commit(s["k"], s["v"], s["table"], s["ctx"], s["path"], s["accepted"])
    return {"pages": _plain_pages, "store": _plain_store, "attend": _plain_attend, "tree": _plain_tree, "commit": _plain_commit}[op](s)


# ---- from the definitions, in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    return {"pages": _exact_pages, "store": _exact_store, "attend": _exact_attend, "tree": _exact_tree, "commit": _exact_commit}[case["op"]](case, s)


def _np(x):
    return x.cpu().numpy()


def _exact_pages(case, s):
    P, cur, cu, table, ring = case["P"], _np(s["cur"]), _np(s["cu"]), _np(s["table"]).copy(), _np(s["ring"]).copy()
    head, count = int(s["pool"][0]), int(s["pool"][1])
    at, first, pages = head, count, len(ring)
    slots, new_len, failed = np.full(s["N"], -1, np.int64), cur.copy(), 0
    for r in range(case["R"]):
        n = int(cu[r + 1] - cu[r])
        has, want = _up(int(cur[r]), P), _up(int(cur[r]) + n, P)
        if want > table.shape[1] or want - has > count:
            failed += 1
            continue
        for i in range(has, want):
            table[r, i] = ring[at % pages]
            at, count = at + 1, count - 1
        new_len[r] = cur[r] + n
        pos = cur[r] + np.arange(n)
        slots[cu[r]:cu[r + 1]] = table[r, pos // P].astype(np.int64) * P + pos % P
    mapped = np.array([at % pages, count, failed, 0], np.int32)
    end, keep = at + count, _np(s["keep"])
    for r in range(case["R"]):
        for i in range(_up(int(min(keep[r], new_len[r])), P), _up(int(new_len[r]), P)):
            ring[end % pages] = table[r, i]
            end, count = end + 1, count + 1
    assert first >= mapped[1]
    return table, slots, new_len, mapped, np.array([at % pages, count, 0, 0], np.int32), ring


def _exact_store(case, s):
    P, slots = case["P"], s["slots"]
    k, v = s["k"].double(), s["v"].double()
    new = []
    for x, scale in ((s["new_k"], s["ks"]), (s["new_v"], s["vs"])):
        x = x.double()
        if scale is not None:
            # the quotient in 32 bits is part of the definition of what is stored
            x = (x / scale.double()[None, :, None]).float().double()
            a = x.abs().clamp(max=E4M3_MAX)
            unit = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
            x = torch.sign(x) * torch.round(a / unit) * unit
        new.append(x)
    Hk, D, c = case["Hk"], case["D"], k.shape[4]
    for h in range(Hk):
        for d in range(D):
            k[slots // P, h, d // c, slots % P, d % c] = new[0][:, h, d]
            v[slots // P, h, d, slots % P] = new[1][:, h, d]
    return k, v


def _exact_attend(case, s):
    cu, ctx, table, P = _np(s["cu"]), _np(s["ctx"]), s["table"].long(), case["P"]
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    out = torch.zeros((s["N"], Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((s["N"], Hq), dtype=torch.float64, device=DEV)
    for r in range(case["R"]):
        lo, hi, c = int(cu[r]), int(cu[r + 1]), int(ctx[r])
        n, t = hi - lo, torch.arange(c + hi - lo, device=DEV)
        page, at = table[r, t // P], t % P
        ok = torch.ones((n, c + n), dtype=torch.bool, device=DEV)
        rows = _ancestors(_parents(n)) if case["tree"] else np.tril(np.ones((n, n), bool))
        ok[:, c:] = torch.from_numpy(rows).to(DEV)
        for h in range(Hk):
            ks, vs = (float(s["ks"][h]), float(s["vs"][h])) if s["ks"] is not None else (1.0, 1.0)
            # whole pages of this head, then their tokens: [t, D]
            used = table[r, :_up(c + n, P)]
            kh = s["k"].view(torch.uint8)[used, h].view(s["k"].dtype) if case["cache"] == "e4m3" else s["k"][used, h]
            vh = s["v"].view(torch.uint8)[used, h].view(s["v"].dtype) if case["cache"] == "e4m3" else s["v"][used, h]
            kh = kh.transpose(1, 2).reshape(-1, D)[:c + n].double() * ks
            vh = vh.transpose(1, 2).reshape(-1, D)[:c + n].double() * vs
            for y in range(Hq // Hk):
                w = h * (Hq // Hk) + y
                z = (s["q"][lo:hi, w].double() @ kh.T) / D ** 0.5
                z = z.masked_fill(~ok, -torch.inf)
                lse[lo:hi, w] = torch.logsumexp(z, 1)
                out[lo:hi, w] = torch.exp(z - lse[lo:hi, w][:, None]) @ vh
    return (out, lse) if case["lse"] else out


def _exact_tree(case, s):
    cu, par, tok, N = _np(s["cu"]), _np(s["parents"]), _np(s["tokens"]), s["N"]
    top = np.concatenate([np.argmax(_np(x), axis=1) for x in s["logits"].split(256)]).astype(np.int32)
    mask, pos = np.zeros((N, s["words"]), np.int32), np.zeros(N, np.int32)
    path, accepted, nxt = np.full((case["R"], s["nodes"]), -1, np.int32), np.zeros(case["R"], np.int32), np.zeros(case["R"], np.int32)
    pos0 = _np(s["pos0"])
    for r in range(case["R"]):
        lo, hi = int(cu[r]), int(cu[r + 1])
        a = _ancestors(par[lo:hi])
        mask[lo:hi] = _words(a, s["words"])
        pos[lo:hi] = pos0[r] + a.sum(1) - 1
        node, walk = 0, [0]
        while True:
            kids = [i for i in range(1, hi - lo) if par[lo + i] == node and tok[lo + i] == top[lo + node]]
            if not kids:
                break
            node = kids[0]
            walk.append(node)
        path[r, :len(walk)] = walk
        accepted[r], nxt[r] = len(walk) - 1, top[lo + node]
    return mask, pos, top, accepted, path, nxt


def _exact_commit(case, s):
    P, table, ctx, path, acc = case["P"], _np(s["table"]), _np(s["ctx"]), _np(s["path"]), _np(s["accepted"])
    k, v = s["k"].double(), s["v"].double()
    for r in range(case["R"]):
        for i in range(1, int(acc[r]) + 1):
            src, dst = int(ctx[r] + path[r, i]), int(ctx[r]) + i
            sp, dp = int(table[r, src // P]), int(table[r, dst // P])
            k[:, dp, :, :, dst % P] = k[:, sp, :, :, src % P]
            v[:, dp, :, :, dst % P] = v[:, sp, :, :, src % P]
    return k, v, (ctx + 1 + acc).astype(np.int32)
