"""Steps in which the pool runs short: block_table rows still name pages that were given
back, and others hold those by then.  What a request that dspark_page_map turned down
does afterwards must touch no one else's pages."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.dirname(__file__))
import draft_head_step_amd as D  # noqa: E402
import paged_helpers as H  # noqa: E402
from oracle import paged_oracle as O  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _raw(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16).cpu().numpy()


def attention_bound(ref, T):
    """Error bound of bf16 rows against the oracle's (out, lse, W, A, M): the result's own
    rounding u, the probabilities' u on W, and e and (T + 16) f of the fp32 scores and sums."""
    u, f = H.half_step(torch.bfloat16), 2.0 ** -24
    out, _, W, A, M = ref
    e = 2 * ((out.shape[2] + 4) * f * A + 4 * f * (2 * M + 2))[..., None]
    return u * np.abs(out) * (1 + e) + W * (u + e + 2 * (T + 16) * f) + 2.0 ** -126


# Two requests of 15 and 14 tokens with one free page, 2, which both rows name behind the
# page that their request holds: the first is given it, the second is turned down.
P = 16
CUR, N = np.array([15, 14], np.int32), [3, 5]
TABLE = np.array([[0, 2, -1], [1, 2, -1]], np.int32)
RING = np.array([2, -1, -1], np.int32)
POOL = np.array([0, 1, 0, 0], np.int32)


def mapped():
    table = dev(TABLE)
    cu = dev(H.starts(N))
    slots, new, pool = D.dspark_page_map(dev(CUR), cu, table, dev(RING), dev(POOL), P, 8)
    assert new.tolist() == [18, 14] and pool.tolist()[2] == 1 and slots.tolist()[3:] == [-1] * 5
    return table, cu, slots, new


@pytest.mark.parametrize("accepted", [0, 1, 2, -1])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_commit_leaves_the_pages_of_others(cache, accepted):
    print(f"case short pool commit {cache} accepted={accepted}", flush=True)
    rng = np.random.default_rng(1)
    k, v = H.caches(rng, 3, 2, 64, P, cache, DEV)
    table, _, _, new = mapped()
    path = np.array([[0, 2, -1, -1], [0, 2, 4, -1]], np.int32)
    path[1, accepted + 1:] = -1
    acc = np.array([1, accepted], np.int32)
    want = O.kv_commit(_raw(k)[None], _raw(v)[None], table.cpu().numpy(), CUR, path, acc, P, new.cpu().numpy())
    assert want[2].tolist() == [17, 14]
    kept = D.dspark_kv_commit(k, v, table, dev(CUR), dev(path), dev(acc), mapped_len=new)
    torch.cuda.synchronize()
    assert kept.tolist() == [17, 14]
    assert np.array_equal(_raw(k), want[0][0]) and np.array_equal(_raw(v), want[1][0])
    # and a trim to it gives nothing back that the request does not hold
    ring = dev(RING)
    pool = D.dspark_page_trim(new, kept, table, ring, dev(np.array([1, 0, 0, 0], np.int32)), P)
    assert pool.tolist() == [1, 0, 0, 0] and ring.tolist() == RING.tolist()


def test_commit_with_mapped_lengths_keeps_the_context_of_refused_paths():
    print("case short pool refused paths", flush=True)
    rng = np.random.default_rng(2)
    R, nodes = 10, 6
    cur = rng.integers(0, 40, R).astype(np.int32)
    n = rng.integers(1, 7, R)
    total = cur + n
    table = H.tables(rng, total, P, 60, 4)
    k, v = H.caches(rng, 60, 2, 64, P, "fp16", DEV)
    path = np.stack([np.sort(rng.permutation(nodes)) for _ in range(R)]).astype(np.int32)
    acc = rng.integers(-1, nodes, R).astype(np.int32)
    mapped_len = np.where(rng.random(R) < 0.3, cur, total).astype(np.int32)
    path[0], acc[0] = [0, -5, -3, 1, 2, 3], 2
    path[1], acc[1] = [0, 2, 2, 3, 4, 5], 2
    acc[2] = nodes
    table[3, :], acc[3], path[3], mapped_len[3] = 60, 2, [0, 2, 3, 4, 5, 6], total[3]
    cur[4], mapped_len[4] = -7, -7
    path[5], acc[5], mapped_len[5] = [0, n[5], -1, -1, -1, -1], 1, total[5]      # the source is the first place behind
    path[6, :2], acc[6], mapped_len[6] = [0, max(1, n[6] - 1)], min(1, n[6] - 1), total[6]
    want = O.kv_commit(_raw(k)[None], _raw(v)[None], table, cur, path, acc, P, mapped_len)
    assert want[2].tolist()[:6] == cur.tolist()[:6] and want[2][6] == cur[6] + 1 + acc[6]
    kept = D.dspark_kv_commit(k, v, dev(table), dev(cur), dev(path), dev(acc), mapped_len=dev(mapped_len))
    torch.cuda.synchronize()
    assert np.array_equal(kept.cpu().numpy(), want[2])
    assert np.array_equal(_raw(k), want[0][0]) and np.array_equal(_raw(v), want[1][0])
    with pytest.raises(ValueError):
        D.dspark_kv_commit(k, v, dev(table), dev(cur), dev(path), dev(acc), mapped_len=dev(mapped_len[1:]))
    with pytest.raises(TypeError):
        D.dspark_kv_commit(k, v, dev(table), dev(cur), dev(path), dev(acc), mapped_len=dev(mapped_len.astype(np.int64)))
    with pytest.raises(D.DsparkError):
        m = dev(mapped_len)
        D.dspark_kv_commit(k, v, dev(table), dev(cur), dev(path), dev(acc), mapped_len=m, new_len=m)


@pytest.mark.parametrize("ring", [False, True])
@pytest.mark.parametrize("tree", [False, True])
def test_attention_reads_no_pages_of_others(tree, ring):
    # the rows of the request that was turned down are NaN, the others' are computed
    print(f"case short pool attention tree={tree} ring={ring}", flush=True)
    rng = np.random.default_rng(3)
    g = 16 if ring else 1
    k, v = H.caches(rng, 3, 2, 64, P, "bf16", DEV)
    table, cu, _, new = mapped()
    q = torch.from_numpy(rng.normal(0, 1, (8, 2 * g, 64)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    mask = dev(np.array([[1], [3], [5], [1], [3], [7], [9], [17]], np.int32)) if tree else None
    out, lse = D.dspark_tree_attention(q, k, v, table, dev(CUR), cu, tree_mask=mask, mapped_len=new, want_lse=True)
    torch.cuda.synchronize()
    assert torch.isnan(out[3:]).all() and torch.isnan(lse[3:]).all()
    ref = O.tree_attention(H.np64(q), H.np64(k), H.np64(v), table.cpu().numpy(), CUR, H.starts(N), P, 0.125,
                           None if mask is None else mask.cpu().numpy().view(np.uint32), mapped=new.cpu().numpy())
    assert np.isnan(ref[0][3:]).all() and np.isfinite(ref[0][:3]).all()
    assert (np.abs(H.np64(out) - ref[0]) <= attention_bound(ref, 18))[:3].all()
    # a length that the elements fill exactly is held
    full = dev((CUR + np.array(N)).astype(np.int32))
    a = D.dspark_tree_attention(q, k, v, table, dev(CUR), cu, tree_mask=mask, mapped_len=full)[0]
    b = D.dspark_tree_attention(q, k, v, table, dev(CUR), cu, tree_mask=mask)[0]
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.isfinite(a).all()
    with pytest.raises(ValueError):
        D.dspark_tree_attention(q, k, v, table, dev(CUR), cu, mapped_len=full[:1])
    with pytest.raises(TypeError):
        D.dspark_tree_attention(q, k, v, table, dev(CUR), cu, mapped_len=full.float())


def test_attention_of_many_requests_with_some_turned_down():
    # cut tiles, several requests a workgroup, refused ones between served ones
    print("case short pool attention many", flush=True)
    rng = np.random.default_rng(4)
    R = 30
    cur = rng.integers(0, 900, R).astype(np.int32)
    n = rng.integers(0, 9, R)
    cu = H.starts(n)
    pages = int(sum(-(-int(x) // P) for x in cur + n)) + 2
    k, v = H.caches(rng, pages, 2, 128, P, "bf16", DEV)
    table = H.tables(rng, cur + n, P, pages)
    held = np.where(rng.random(R) < 0.4, cur, cur + n).astype(np.int32)
    q = torch.from_numpy(rng.normal(0, 1, (int(cu[-1]), 8, 128)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    a, la = D.dspark_tree_attention(q, k, v, dev(table), dev(cur), dev(cu), mapped_len=dev(held), want_lse=True)
    ref = O.tree_attention(H.np64(q), H.np64(k), H.np64(v), table, cur, cu, P, 128 ** -0.5, mapped=held)
    torch.cuda.synchronize()
    down = np.isnan(ref[0][:, 0, 0])
    assert 5 < down.sum() < len(down) - 5
    got = H.np64(a)
    assert np.isnan(got[down]).all() and np.isnan(la.cpu().numpy()[down]).all()
    assert (np.abs(got - ref[0]) <= attention_bound(ref, 910))[~down].all()


def test_acceptance_takes_nothing_of_a_request_that_was_turned_down():
    print("case short pool acceptance", flush=True)
    rng = np.random.default_rng(5)
    R, V, nodes = 40, 97, 8
    cur = rng.integers(0, 100, R).astype(np.int32)
    n = rng.integers(0, 9, R)
    cu = H.starts(n)
    N_ = int(cu[-1])
    held = np.where(rng.random(R) < 0.4, cur, cur + n).astype(np.int32)
    par = np.concatenate([H.random_parents(rng, int(x)) for x in n]).astype(np.int32)
    tok = rng.integers(0, V, N_).astype(np.int32)
    logits = rng.normal(0, 1, (N_, V)).astype(np.float32)
    for r in range(R):
        for i in range(1, n[r]):
            logits[cu[r] + par[cu[r] + i], tok[cu[r] + i]] = 9.0
    want = O.verify_tree(logits, cu, tok, par, nodes, cur, held)
    down = np.nonzero((n > 0) & (cur + n > held))[0]
    assert len(down) > 5 and (want[0][down] == -1).all() and (want[0] > 0).sum() > 5
    bad = logits.copy()
    for r in down:                       # as the logits of NaN rows would be
        bad[cu[r]:cu[r + 1]] = np.nan
    acc, path, nxt, top = D.dspark_verify_tree(dev(bad), dev(cu), dev(tok), dev(par), nodes, ctx_len=dev(cur), mapped_len=dev(held))
    torch.cuda.synchronize()
    assert np.array_equal(acc.cpu().numpy(), want[0]) and np.array_equal(path.cpu().numpy(), want[1])
    assert np.array_equal(nxt.cpu().numpy(), want[2])
    live = np.ones(N_, bool)
    for r in down:
        live[cu[r]:cu[r + 1]] = False
    assert np.array_equal(top.cpu().numpy()[live], want[3][live])
    with pytest.raises(ValueError):
        D.dspark_verify_tree(dev(logits), dev(cu), dev(tok), dev(par), nodes, mapped_len=dev(held))
    with pytest.raises(ValueError):
        D.dspark_verify_tree(dev(logits), dev(cu), dev(tok), dev(par), nodes, ctx_len=dev(cur[1:]), mapped_len=dev(held))


@pytest.mark.parametrize("pages", [5, 8, 11])
def test_steps_over_a_short_pool(pages):
    # Whole steps with fewer pages than the batch would like, requests that end and begin
    # again, and rows of the table that name pages of others: every request's cache holds what
    # it accepted, every length is right, and no page is held twice or lost.
    print(f"case short pool steps pages={pages}", flush=True)
    rng = np.random.default_rng(pages)
    R, Hk, Dh, V, width, nodes = 7, 1, 64, 50, 6, 12
    kc = torch.full((pages, Hk, Dh // 8, P, 8), -1.0, dtype=torch.bfloat16, device=DEV)
    vc = torch.full((pages, Hk, Dh, P), -1.0, dtype=torch.bfloat16, device=DEV)
    table = dev(rng.integers(0, pages, (R, width)).astype(np.int32))        # stale ids from the start
    ring, pool = dev(rng.permutation(pages).astype(np.int32)), dev(np.array([0, pages, 0, 0], np.int32))
    lens = dev(np.zeros(R, np.int32))
    held = [[] for _ in range(R)]            # the element numbers that each request's cache should hold
    serial = turned_down = moved = 0
    for step in range(25):
        n = rng.integers(0, 20, R) if step == 0 else rng.integers(0, nodes + 1, R)
        n = np.where([len(h) + x > width * P for h, x in zip(held, n)], 1, n)
        cu = H.starts(n)
        N_ = int(cu[-1])
        par = np.concatenate([H.random_parents(rng, int(x)) for x in n] + [np.zeros(0)]).astype(np.int32)
        tok = rng.integers(0, V, N_).astype(np.int32)
        ids = serial + np.arange(N_)
        serial += N_
        rows = np.zeros((N_, Hk, Dh), np.float32)
        rows[..., 0::2], rows[..., 1::2] = (ids // 128)[:, None, None], (ids % 128)[:, None, None]    # exact in bf16
        kv = torch.from_numpy(rows).to(torch.bfloat16).to(DEV)
        logits = rng.normal(0, 1, (N_, V)).astype(np.float32)
        for r in range(R):
            for i in range(1, n[r]):
                if rng.random() < 0.7:
                    logits[cu[r] + par[cu[r] + i], tok[cu[r] + i]] = 9.0
        dcu, dpar, dtok = dev(cu), dev(par), dev(tok)
        slots, new, pool1 = D.dspark_page_map(lens, dcu, table, ring, pool, P, N_)
        mask, _ = D.dspark_tree_pack(dpar, dcu, 1, lens)
        D.dspark_kv_store(kv, kv, slots, kc, vc, count=dcu[R:])
        out, _ = D.dspark_tree_attention(kv, kc, vc, table, lens, dcu, tree_mask=mask, mapped_len=new)
        z = dev(logits) + out[:, 0, :1].float() * 0.0        # NaN where the rows are
        acc, path, nxt, _ = D.dspark_verify_tree(z, dcu, dtok, dpar, 20, ctx_len=lens, mapped_len=new)
        kept = D.dspark_kv_commit(kc, vc, table, lens, path, acc, mapped_len=new)
        end = rng.random(R) < 0.08
        keep = torch.where(dev(end), torch.zeros_like(kept), kept)
        pool = D.dspark_page_trim(new, keep, table, ring, pool1, P)
        torch.cuda.synchronize()
        a, p, was, now = (x.cpu().numpy() for x in (acc, path, lens, new))
        assert int(pool[2]) == 0
        for r in range(R):
            down = n[r] > 0 and now[r] == was[r]
            turned_down += int(down)
            rows_ = out[int(cu[r]):int(cu[r + 1])]
            assert torch.isnan(rows_).all() if down else torch.isfinite(rows_).all()
            assert (a[r] == -1) == (down or n[r] == 0) and (int(nxt[r]) == -1) == (a[r] == -1)
            held[r] += [int(ids[cu[r] + p[r, i]]) for i in range(a[r] + 1)]
            moved += int(a[r] >= 0 and (p[r, :a[r] + 1] != np.arange(a[r] + 1)).any())
            assert int(kept[r]) == len(held[r])
            if end[r]:
                held[r] = []
        lens = keep
        t, k, v = table.cpu().numpy(), H.np64(kc), H.np64(vc)
        used = []
        for r in range(R):
            pos = np.arange(len(held[r]))
            page, o = t[r, pos // P], pos % P
            for lo, hi in ((k[page, 0, 0, o, 0], k[page, 0, 0, o, 1]), (v[page, 0, 0, o], v[page, 0, 1, o]),
                           (k[page, 0, 7, o, 6], k[page, 0, 7, o, 7]), (v[page, 0, 62, o], v[page, 0, 63, o])):
                assert (lo * 128 + hi).astype(int).tolist() == held[r], (step, r)
            used += t[r, :-(-len(held[r]) // P)].tolist()
        head, count, _, _ = pool.tolist()
        free = [int(ring[(head + i) % pages]) for i in range(count)]
        assert sorted(used + free) == list(range(pages)), step
    print(f"  turned down {turned_down}, moved {moved}", flush=True)
    assert turned_down >= 5 and moved >= 10


def test_a_step_over_a_short_pool_replays_in_a_graph():
    # the whole step with its commit; what it changes in place is put back between the replays
    print("case short pool graph", flush=True)
    rng = np.random.default_rng(8)
    R, pages, Hk, Dh, V, nodes = 6, 30, 2, 64, 40, 9
    cur = rng.integers(0, 60, R).astype(np.int32)
    n = rng.integers(3, nodes + 1, R)
    cu = H.starts(n)
    N_ = int(cu[-1])
    need = -(-cur // P)
    table = np.resize(rng.permutation(pages), (R, 5)).astype(np.int32)      # every row full of ids
    order = rng.permutation(pages).astype(np.int32)
    at = 0
    for r in range(R):
        table[r, :need[r]] = order[at:at + need[r]]
        at += need[r]
    ring = np.full(pages, -1, np.int32)
    ring[:2] = order[at:at + 2]                                            # two pages for all of them
    par = np.concatenate([H.random_parents(rng, int(x)) for x in n]).astype(np.int32)
    tok = rng.integers(0, V, N_).astype(np.int32)
    logits = rng.normal(0, 1, (N_, V)).astype(np.float32)
    for r in range(R):
        for i in range(1, n[r]):
            logits[cu[r] + par[cu[r] + i], tok[cu[r] + i]] = 9.0
    kc, vc = H.caches(rng, pages, Hk, Dh, P, "bf16", DEV)
    start = dict(table=dev(table), ring=dev(ring), kc=kc, vc=vc)
    s = {k: t.clone() for k, t in start.items()}
    c, u, p, t, z = dev(cur), dev(cu), dev(par), dev(tok), dev(logits)
    pool = dev(np.array([0, 2, 0, 0], np.int32))
    x = torch.from_numpy(rng.normal(0, 1, (N_, Hk, Dh)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    o = dict(slots=torch.zeros(N_, dtype=torch.int64, device=DEV), new=torch.zeros(R, **i32), a=torch.zeros(4, **i32),
             b=torch.zeros(4, **i32), mask=torch.zeros(N_, 1, **i32), out=torch.zeros_like(x), acc=torch.zeros(R, **i32),
             path=torch.zeros(R, nodes, **i32), nxt=torch.zeros(R, **i32), top=torch.zeros(N_, **i32), kept=torch.zeros(R, **i32),
             ws=torch.zeros(D.dspark_tree_attention_workspace(R, N_, Hk, Hk, Dh), dtype=torch.uint8, device=DEV))

    def step():
        D.dspark_page_map(c, u, s["table"], s["ring"], pool, P, slots=o["slots"], new_len=o["new"], pool_out=o["a"])
        D.dspark_tree_pack(p, u, 1, c, mask=o["mask"])
        D.dspark_kv_store(x, x, o["slots"], s["kc"], s["vc"], count=u[R:])
        D.dspark_tree_attention(x, s["kc"], s["vc"], s["table"], c, u, tree_mask=o["mask"], mapped_len=o["new"], out=o["out"],
                                workspace=o["ws"])
        D.dspark_verify_tree(z, u, t, p, nodes, ctx_len=c, mapped_len=o["new"], target_argmax=o["top"], accepted=o["acc"],
                             path=o["path"], next_token=o["nxt"])
        D.dspark_kv_commit(s["kc"], s["vc"], s["table"], c, o["path"], o["acc"], mapped_len=o["new"], new_len=o["kept"])
        D.dspark_page_trim(o["new"], o["kept"], s["table"], s["ring"], o["a"], P, pool_out=o["b"])

    step()
    torch.cuda.synchronize()
    down = (o["new"].cpu().numpy() == cur)
    assert 0 < down.sum() < R and (o["kept"].cpu().numpy()[down] == cur[down]).all() and (o["acc"].cpu().numpy()[~down] > 0).all()
    want = {k: v.clone() for k, v in {**s, **o}.items() if k != "ws"}
    for k, v in start.items():
        s[k].copy_(v)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(3):
        for k, v in start.items():
            s[k].copy_(v)
        for v in o.values():
            v.view(torch.uint8).fill_(0xA5 + rep)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, v in want.items():
            got = s[k] if k in s else o[k]
            assert torch.equal(got.view(torch.uint8), v.view(torch.uint8)), (rep, k)
