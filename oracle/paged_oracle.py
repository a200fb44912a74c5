"""CPU oracle of the verification over a paged cache: the definitions of
include/dspark.h in numpy, in 64 bits, request by request.  Test infrastructure
only; shares no code with the library.

Caches are arrays in the library's storage order, k [pages, Hk, D / c, P, c] and
v [pages, Hk, D, P], of any dtype that converts to float64 (or raw integers
where values only move).
"""
from __future__ import annotations

import numpy as np


def _up(a, b):
    return -(-int(a) // int(b))


def page_map(cur, cu, table, ring, pool, P, max_tokens, slots):
    """Returns (table, slots, new_len, pool) after the call; `slots` is what the
    output held before."""
    cur, cu = np.asarray(cur, np.int64), np.asarray(cu, np.int64)
    table, slots = table.copy(), slots.copy()
    R, width = table.shape
    n_pages = len(ring)
    head, count = int(pool[0]), int(pool[1])
    asked = taken = refused = 0
    new_len = cur.copy()
    for r in range(R):
        n = int(cu[r + 1] - cu[r])
        fits = cur[r] >= 0 and n >= 0 and _up(cur[r] + n, P) <= width and cur[r] + n < 2 ** 31
        has = _up(cur[r], P) if fits else 0
        need = _up(cur[r] + n, P) - has if fits else 0
        served = fits and (need == 0 or asked + need <= count)
        if served:
            for i in range(need):
                table[r, has + i] = ring[(head + asked + i) % n_pages]
            new_len[r] = cur[r] + n
            taken = max(taken, asked + need if need else 0)
        else:
            refused += 1
        asked += need
        for j in range(max(n, 0)):
            e = cu[r] + j
            if not 0 <= e < min(cu[R], max_tokens):
                continue
            pos = int(cur[r]) + j
            page = int(table[r, pos // P]) if served else -1
            slots[e] = page * P + pos % P if 0 <= page < n_pages else -1
    return (table, slots, new_len.astype(np.int32),
            np.array([(head + taken) % n_pages, count - taken, refused, 0], np.int32))


def page_trim(cur, keep, table, ring, pool, P):
    """Returns (ring, pool) after the call."""
    R, width = table.shape
    n_pages = len(ring)
    ring = ring.copy()
    head, count = int(pool[0]), int(pool[1])
    back, refused = [], 0
    for r in range(R):
        c = int(cur[r])
        if c < 0 or _up(c, P) > width:
            refused += 1
            continue
        k = min(max(int(keep[r]), 0), c)
        back += [table[r, i] for i in range(_up(k, P), _up(c, P))]
    if count + len(back) > n_pages:
        return ring, np.array([head, count, R, 0], np.int32)
    for i, page in enumerate(back):
        ring[(head + count + i) % n_pages] = page
    return ring, np.array([head, count + len(back), refused, 0], np.int32)


def kv_store(k, v, slots, k_cache, v_cache, P, count=None):
    """Rows k, v [N, Hk, D] (already of the cache's type) into copies of the caches."""
    k_cache, v_cache = k_cache.copy(), v_cache.copy()
    N, Hk, D = k.shape
    c = k_cache.shape[-1]
    n_pages = k_cache.shape[0]
    for e in range(N if count is None else min(N, count)):
        s = int(slots[e])
        if not 0 <= s < n_pages * P:
            continue
        page, o = s // P, s % P
        k_cache[page, :, :, o, :] = k[e].reshape(Hk, D // c, c)
        v_cache[page, :, :, o] = v[e]
    return k_cache, v_cache


def kv_commit(k_cache, v_cache, table, ctx, path, accepted, P, mapped=None):
    """[layers, pages, ...] caches.  Returns copies after the move, and new_len."""
    k_cache, v_cache = k_cache.copy(), v_cache.copy()
    R, width = table.shape
    n_pages = k_cache.shape[1]
    new_len = np.full(R, -1, np.int32) if mapped is None else np.array(ctx, np.int32)
    for r in range(R):
        c, a = int(ctx[r]), int(accepted[r])
        room = width * P if mapped is None else min(width * P, int(mapped[r]))
        if c < 0 or a < -1 or a >= path.shape[1] or c + 1 + a > room:
            continue
        p = [int(x) for x in path[r, :a + 1]]
        if a >= 0 and (p[0] != 0 or any(y <= x for x, y in zip(p, p[1:])) or c + p[-1] >= room):
            continue
        moves = [(c + p[i], c + i) for i in range(1, a + 1)]
        if any(not 0 <= table[r, t // P] < n_pages for m in moves for t in m):
            continue
        new_len[r] = c + 1 + a
        for src, dst in moves:
            k_cache[:, table[r, dst // P], :, :, dst % P] = k_cache[:, table[r, src // P], :, :, src % P]
            v_cache[:, table[r, dst // P], :, :, dst % P] = v_cache[:, table[r, src // P], :, :, src % P]
    return k_cache, v_cache, new_len


def ancestors(parents):
    """(mask [n, n] of truth values, depth [n]): the node itself and its ancestors;
    an empty row and depth -1 where a link on the way is bad."""
    n = len(parents)
    mask, depth = np.zeros((n, n), bool), np.full(n, -1)
    for i in range(n):
        p = int(parents[i])
        if p == -1:
            depth[i] = 0
        elif 0 <= p < i and depth[p] >= 0:
            mask[i] = mask[p]
            depth[i] = depth[p] + 1
        else:
            continue
        mask[i, i] = True
    return mask, depth


def tree_pack(parents, cu, pos0, words):
    """Returns (mask words [N, words] uint32, positions [N], requests [N])."""
    N = int(cu[-1])
    mask, pos, req = np.zeros((N, words), np.uint32), np.full(N, -1, np.int32), np.zeros(N, np.int32)
    for r in range(len(cu) - 1):
        lo, hi = int(cu[r]), int(cu[r + 1])
        req[lo:hi] = r
        n = min(hi - lo, 32 * words)
        m, depth = ancestors(parents[lo:lo + n])
        for i in range(n):
            for j in np.nonzero(m[i])[0]:
                mask[lo + i, j // 32] |= np.uint32(1 << (j % 32))
            if depth[i] >= 0:
                pos[lo + i] = (0 if pos0 is None else pos0[r]) + depth[i]
    return mask, pos, req


def verify_tree(logits, cu, tokens, parents, max_nodes, ctx=None, mapped=None):
    top = np.argmax(logits, axis=1).astype(np.int32)
    R = len(cu) - 1
    path = np.full((R, max_nodes), -1, np.int32)
    accepted, nxt = np.full(R, -1, np.int32), np.full(R, -1, np.int32)
    for r in range(R):
        lo, n = int(cu[r]), min(int(cu[r + 1] - cu[r]), max_nodes)
        if n <= 0 or (mapped is not None and int(ctx[r]) + int(cu[r + 1] - cu[r]) > mapped[r]):
            continue
        walk = [0]
        while True:
            at = walk[-1]
            kids = [i for i in range(at + 1, n) if parents[lo + i] == at and tokens[lo + i] == top[lo + at]]
            if not kids:
                break
            walk.append(kids[0])
        path[r, :len(walk)] = walk
        accepted[r], nxt[r] = len(walk) - 1, top[lo + walk[-1]]
    return accepted, path, nxt, top


def tree_attention(q, k_cache, v_cache, table, ctx, cu, P, scale, mask=None, k_scale=None, v_scale=None,
                   mapped=None):
    """Returns (out [N, Hq, D], lse [N, Hq], weight [N, Hq, D], size [N, Hq], top [N, Hq]) in
    64 bits: weight = sum_t p_t |v_t|, size = the largest scale * sum_d |q_d k_td| that a
    row sees and top the largest |score|, for error bounds.  Rows of a request whose
    lengths or pages are bad are NaN."""
    N, Hq, D = q.shape
    n_pages, Hk, C, _, c = k_cache.shape
    g = Hq // Hk
    out, lse = np.zeros((N, Hq, D)), np.full((N, Hq), -np.inf)
    weight, size, high = np.zeros((N, Hq, D)), np.zeros((N, Hq)), np.zeros((N, Hq))
    width = table.shape[1]
    for r in range(len(cu) - 1):
        lo, n, cx = int(cu[r]), int(cu[r + 1] - cu[r]), int(ctx[r])
        if n <= 0:
            continue
        total = cx + n
        need = _up(total, P) if cx >= 0 else 0
        held = mapped is None or total <= mapped[r]
        if cx < 0 or not held or need > width or any(not 0 <= p < n_pages for p in table[r, :need]):
            out[lo:lo + n], lse[lo:lo + n] = np.nan, np.nan
            continue
        pages = table[r, :need]
        k = k_cache[pages].astype(np.float64).transpose(1, 0, 3, 2, 4).reshape(Hk, need * P, D)[:, :total]
        v = v_cache[pages].astype(np.float64).transpose(1, 0, 3, 2).reshape(Hk, need * P, D)[:, :total]
        for i in range(n):
            e = lo + i
            if e >= N:
                break
            seen = np.ones(total, bool)
            for j in range(n):
                seen[cx + j] = (j <= i) if mask is None else (
                    j // 32 < mask.shape[1] and bool((int(mask[e, j // 32]) >> (j % 32)) & 1))
            if not seen.any():
                continue
            for y in range(Hq):
                h = y // g
                ks = 1.0 if k_scale is None else float(k_scale[h])
                vs = 1.0 if v_scale is None else float(v_scale[h])
                kk, vv = k[h][seen] * ks, v[h][seen] * vs
                x = q[e, y].astype(np.float64)
                s = scale * (kk @ x)
                m = s.max()
                p = np.exp(s - m)
                out[e, y] = (p @ vv) / p.sum()
                weight[e, y] = (p @ np.abs(vv)) / p.sum()
                lse[e, y] = m + np.log(p.sum())
                size[e, y] = abs(scale) * (np.abs(kk) @ np.abs(x)).max()
                high[e, y] = np.abs(s).max()
    return out, lse, weight, size, high
