"""GPU page bookkeeping, cache writes, path commit and tree acceptance against the
oracle.  All of it is exact: integers, copies, and one rounding to e4m3 that is
defined bit by bit (an fp32 quotient, clamped, to nearest even)."""
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


def _up(a, b):
    return -(-int(a) // int(b))


# ---- pages ----

def make_pool(rng, cur, P, width, spare):
    R = len(cur)
    held = [_up(max(int(c), 0), P) for c in cur]
    pages = sum(held) + spare
    table = H.tables(rng, [h * P for h in held], P, pages, width)
    used = set(int(table[r, i]) for r in range(R) for i in range(held[r]))
    free = rng.permutation([p for p in range(pages) if p not in used])
    head = int(rng.integers(0, pages))
    ring = np.full(pages, -1, np.int32)
    for i, p in enumerate(free):
        ring[(head + i) % pages] = p
    return table, ring, np.array([head, len(free), 77, 88], np.int32)


def run_map(cur, cu, table, ring, pool, P, room):
    t, slots = dev(table), torch.full((room,), -9, dtype=torch.int64, device=DEV)
    s, new, out = D.dspark_page_map(dev(cur), dev(cu), t, dev(ring), dev(pool), P, slots=slots)
    torch.cuda.synchronize()
    return t.cpu().numpy(), s.cpu().numpy(), new.cpu().numpy(), out.cpu().numpy()


def check_map(cur, n, P, width, spare, seed, room=None):
    rng = np.random.default_rng(seed)
    cur, cu = np.asarray(cur, np.int32), H.starts(n)
    table, ring, pool = make_pool(rng, cur, P, width, spare)
    room = max(1, int(cu[-1])) + 3 if room is None else room
    got = run_map(cur, cu, table, ring, pool, P, room)
    want = O.page_map(cur, cu, table, ring, pool, P, room, np.full(room, -9, np.int64))
    for name, g, w in zip(("table", "slots", "new_len", "pool"), got, want):
        assert np.array_equal(g, w), name
    return got, (cur, cu, table, ring, pool)


@pytest.mark.parametrize("P", [16, 64, 1024])
@pytest.mark.parametrize("R,top,most", [(1, 1, 1), (1, 0, 5000), (5, 100, 40), (257, 70, 7), (1000, 3000, 6), (64, 9, 900)])
def test_page_map(R, top, most, P):
    print(f"case page_map R={R} top={top} most={most} P={P}", flush=True)
    rng = np.random.default_rng(R + P)
    cur = rng.integers(0, top + 1, R)
    n = rng.integers(0, most + 1, R)
    check_map(cur, n, P, _up(top + most, P) + 1, 5 + sum(_up(x, P) + 1 for x in n), R * 7 + P)


@pytest.mark.parametrize("spare", [0, 1, 5, 40, 41, 60])
def test_page_map_of_a_short_pool(spare):
    # a request that finds too few pages is turned down, and every later one that needs a page
    print(f"case page_map short pool {spare}", flush=True)
    rng = np.random.default_rng(3)
    got, _ = check_map(rng.integers(0, 64, 50), rng.integers(0, 40, 50), 16, 8, spare, spare)
    assert (got[3][2] > 0) == (got[3][1] < 20) or spare > 50


def test_page_map_refuses_bad_requests():
    # negative lengths, more pages than a row has, segments past the room for slots
    print("case page_map bad requests", flush=True)
    cur = np.array([5, -1, 10, 60, 0, 2 ** 31 - 1], np.int32)
    n = [3, 4, 100, 5, 0, 2]
    rng = np.random.default_rng(1)
    cu = H.starts(n)
    table, ring, pool = make_pool(rng, np.array([5, 0, 10, 60, 0, 0]), 16, 4, 9)
    got = run_map(cur, cu, table, ring, pool, 16, 60)
    want = O.page_map(cur, cu, table, ring, pool, 16, 60, np.full(60, -9, np.int64))
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    assert got[3][2] == 4
    # page ids outside the pool give slots of -1
    table[0, 0] = len(ring)
    table[3, 3] = -5
    got = run_map(cur, cu, table, ring, pool, 16, 200)
    assert (got[1][:3] == -1).all() and (got[1][cu[3]:cu[3] + 4] == -1).all()


def test_page_map_at_the_largest_request_count():
    print("case page_map largest R", flush=True)
    R = 16384
    rng = np.random.default_rng(8)
    check_map(rng.integers(0, 40, R), rng.integers(0, 4, R), 16, 4, 9000, 9)
    with pytest.raises(D.DsparkError) as e:
        D.dspark_page_map(dev(np.zeros(R + 1, np.int32)), dev(np.zeros(R + 2, np.int32)), dev(np.zeros((R + 1, 2), np.int32)),
                          dev(np.zeros(4, np.int32)), dev(np.zeros(4, np.int32)), 16, 8)
    assert e.value.status == 3


def test_pages_of_many_requests_replay_in_a_graph():
    # lengths that take more LDS than a kernel has without asking
    print("case pages of 9000 requests in a graph", flush=True)
    R, P, width = 9000, 16, 4
    rng = np.random.default_rng(10)
    cur, n = rng.integers(0, 40, R), rng.integers(0, 5, R)
    cu = np.concatenate([[0], np.cumsum(n)])
    N = int(cu[-1])
    table, ring, pool = make_pool(rng, cur, P, width, 9000)
    c, u, k = (dev(x.astype(np.int32)) for x in (cur, cu, cur // 2))
    out = dict(table=dev(table), ring=dev(ring), slots=torch.zeros(N, dtype=torch.int64, device=DEV),
               new=torch.zeros(R, dtype=torch.int32, device=DEV), a=dev(pool), b=dev(pool))
    first = dev(pool)

    def step(o):
        D.dspark_page_map(c, u, o["table"], o["ring"], first, P, slots=o["slots"], new_len=o["new"], pool_out=o["a"])
        D.dspark_page_trim(o["new"], k, o["table"], o["ring"], o["a"], P, pool_out=o["b"])

    want = {x: t.clone() for x, t in out.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out)
    step(want)
    for _ in range(3):
        out["slots"].zero_()
        out["new"].zero_()
        out["table"].copy_(dev(table))
        out["ring"].copy_(dev(ring))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x in out:
            assert torch.equal(out[x], want[x]), x


def check_trim(cur, keep, table, ring, pool, P):
    r = dev(ring)
    out = D.dspark_page_trim(dev(cur), dev(keep), dev(table), r, dev(pool), P)
    torch.cuda.synchronize()
    want = O.page_trim(cur, keep, table, ring, pool, P)
    assert np.array_equal(r.cpu().numpy(), want[0]) and np.array_equal(out.cpu().numpy(), want[1])
    return want


@pytest.mark.parametrize("R,top,P", [(1, 0, 16), (1, 90000, 16), (9, 100, 16), (300, 2000, 64), (16384, 50, 16)])
def test_page_trim(R, top, P):
    print(f"case page_trim R={R} top={top} P={P}", flush=True)
    rng = np.random.default_rng(R + top)
    cur = rng.integers(0, top + 1, R).astype(np.int32)
    keep = rng.integers(-3, top + 5, R).astype(np.int32)
    table, ring, pool = make_pool(rng, cur, P, _up(top, P) + 1, 11)
    check_trim(cur, keep, table, ring, pool, P)


def test_page_trim_refusals():
    print("case page_trim refusals", flush=True)
    rng = np.random.default_rng(2)
    cur = np.array([40, -1, 200, 16], np.int32)
    table, ring, pool = make_pool(rng, np.array([40, 0, 60, 16]), 16, 4, 3)
    check_trim(cur, np.zeros(4, np.int32), table, ring, pool, 16)
    full = pool.copy()
    full[1] = len(ring) - 1       # the pages would not fit: given back twice
    want = check_trim(cur, np.zeros(4, np.int32), table, ring, full, 16)
    assert want[1][2] == 4


def test_pages_come_and_go_over_many_steps():
    # map, trim, map ... : no page is ever held twice, none is lost
    print("case pages over steps", flush=True)
    rng = np.random.default_rng(12)
    R, P, width = 40, 16, 12
    cur = np.zeros(R, np.int32)
    pages = 300
    table = torch.full((R, width), -1, dtype=torch.int32, device=DEV)
    ring = torch.arange(pages, dtype=torch.int32, device=DEV)
    pool = dev(np.array([0, pages, 0, 0], np.int32))
    lens = dev(cur)
    for step in range(12):
        n = rng.integers(0, 60, R)
        slots, new, pool = D.dspark_page_map(lens, dev(H.starts(n)), table, ring, pool, P, max_tokens=R * 60)
        keep = torch.minimum(new, dev(rng.integers(0, 150, R).astype(np.int32)))
        pool2 = D.dspark_page_trim(new, keep, table, ring, pool, P)
        torch.cuda.synchronize()
        lens, pool = keep.contiguous(), pool2
        k, t, r, (head, count, _, _) = (x.cpu().numpy() for x in (lens, table, ring, pool))
        held = [int(t[i, j]) for i in range(R) for j in range(_up(k[i], P))]
        free = [int(r[(head + i) % pages]) for i in range(count)]
        assert sorted(held + free) == list(range(pages)), step


# ---- cache writes ----

def _raw(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16).cpu().numpy()


def e4m3(x, scale):
    """The stored form by the definition: fp32 quotient, clamp, nearest even."""
    q = (x.astype(np.float32) / scale.astype(np.float32)[None, :, None]).astype(np.float32)
    c = torch.from_numpy(np.where(q > 448, np.float32(448), np.where(q < -448, np.float32(-448), q)))
    return c.to(torch.float8_e4m3fn).view(torch.uint8).numpy()


@pytest.mark.parametrize("cache", ["same", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("N,Hk,Dh,P", [(1, 1, 64, 16), (5, 3, 96, 16), (16, 2, 128, 32), (37, 8, 128, 64),
                                       (100, 1, 192, 1024), (300, 2, 256, 16)])
@pytest.mark.parametrize("order", ["run", "mixed"])
def test_kv_store(N, Hk, Dh, P, dtype, cache, order):
    print(f"case kv_store N={N} Hk={Hk} D={Dh} P={P} {dtype} {cache} {order}", flush=True)
    rng = np.random.default_rng(N + Dh)
    pages = _up(N + 9, P) + 3
    kc, vc = H.caches(rng, pages, Hk, Dh, P, dtype if cache == "same" else "e4m3", DEV)
    # a row stride of its own, as in a fused projection
    wide = torch.from_numpy(rng.normal(0, 3, (N, 2 * Hk + 1, Dh)).astype(np.float32)).to(H.TYPES[dtype])
    wide[0, 0, :6] = torch.tensor([0.0, -0.0, float("nan"), float("inf"), -float("inf"), 60000.0])
    k, v = wide[:, :Hk], wide[:, Hk:2 * Hk]
    slots = np.arange(N) + 7 if order == "run" else rng.permutation(pages * P)[:N]
    slots = slots.astype(np.int64)
    if N > 4:
        slots[[1, 3]] = [-1, pages * P]       # skipped
    ks = vs = None
    if cache == "e4m3":
        ks, vs = ((0.5 + rng.random(Hk)).astype(np.float32) / 30 for _ in range(2))
        rk = e4m3(H.np64(k).astype(np.float32), ks)
        rv = e4m3(H.np64(v).astype(np.float32), vs)
    else:
        rk, rv = _raw(k.contiguous()), _raw(v.contiguous())
    for count in (None, max(0, N - 3), N + 5):
        a, b = kc.clone(), vc.clone()
        w = wide.to(DEV)
        D.dspark_kv_store(w[:, :Hk], w[:, Hk:2 * Hk], dev(slots), a, b,
                          count=None if count is None else dev(np.array([count], np.int32)), k_scale=dev(ks), v_scale=dev(vs))
        torch.cuda.synchronize()
        want = O.kv_store(rk, rv, slots, _raw(kc), _raw(vc), P, count)
        got = _raw(a), _raw(b)
        for g, w_ in zip(got, want):
            if cache == "e4m3":   # any NaN pattern
                assert np.array_equal(g[(w_ & 127) != 127], w_[(w_ & 127) != 127])
                assert ((g[(w_ & 127) == 127] & 127) == 127).all()
            else:
                assert np.array_equal(g, w_)


def test_kv_store_rounds_every_value_to_the_nearest():
    # every finite bf16 value once, at scale 1 and at an odd scale
    print("case kv_store all bf16", flush=True)
    bits = np.arange(65536, dtype=np.uint16)
    x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).reshape(512, 1, 128)
    for s in (1.0, 0.0371):
        kc = torch.zeros((32, 1, 8, 16, 16), dtype=torch.float8_e4m3fn, device=DEV)
        vc = torch.zeros((32, 1, 128, 16), dtype=torch.float8_e4m3fn, device=DEV)
        sc = dev(np.array([s], np.float32))
        D.dspark_kv_store(x.to(DEV), x.to(DEV), torch.arange(512, device=DEV), kc, vc, k_scale=sc, v_scale=sc)
        torch.cuda.synchronize()
        want = e4m3(x.float().numpy(), np.array([s], np.float32))[:, 0]
        k = _raw(kc).transpose(0, 3, 1, 2, 4).reshape(512, 128)
        v = _raw(vc).transpose(0, 3, 1, 2).reshape(512, 128)
        nan = (want & 127) == 127
        for g in (k, v):
            assert np.array_equal(g[~nan], want[~nan]) and ((g[nan] & 127) == 127).all()


@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("fp16", "e4m3")])
@pytest.mark.parametrize("N,Hk,Dh,P", [(8201, 8, 64, 16), (5500, 12, 96, 64), (66000, 1, 128, 32), (4127, 16, 256, 16), (2100, 32, 192, 128)])
def test_kv_store_of_many_elements(N, Hk, Dh, P, dtype, cache):
    test_kv_store(N, Hk, Dh, P, dtype, cache, "run" if Dh % 64 else "mixed")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_kv_store_divides_by_any_scale(dtype):
    # every value of the type by scales with exact ties, near ties, and none that a
    # reciprocal could stand for; the quotient is fp32, rounded twice
    print(f"case kv_store scales {dtype}", flush=True)
    rng = np.random.default_rng(5)
    scales = [1.0, 0.5, 2.0 ** -6, 3.0, 1 / 3, 0.1, 7.0, 1e-3, 448.0, 1e-30, 1e30, 1e-38, 3e38, 1e-40, 1e-45, 1.0000001, 0.99999994]
    scales = np.array(scales + list(np.exp(rng.uniform(-20, 20, 15))), np.float32)
    H = len(scales)
    bits = torch.from_numpy(np.arange(65536, dtype=np.uint16).view(np.int16))
    x = bits.view(torch.bfloat16 if dtype == "bf16" else torch.float16).reshape(512, 1, 128)
    rows = x.expand(512, H, 128).contiguous().to(DEV)
    kc = torch.zeros((32, H, 8, 16, 16), dtype=torch.float8_e4m3fn, device=DEV)
    vc = torch.zeros((32, H, 128, 16), dtype=torch.float8_e4m3fn, device=DEV)
    D.dspark_kv_store(rows, rows, torch.arange(512, device=DEV), kc, vc, k_scale=dev(scales), v_scale=dev(scales))
    torch.cuda.synchronize()
    k = _raw(kc).transpose(0, 3, 1, 2, 4).reshape(512, H, 128)
    v = _raw(vc).transpose(0, 3, 1, 2).reshape(512, H, 128)
    for i in range(H):
        want = e4m3(x.float().numpy(), scales[i:i + 1])[:, 0]
        nan = (want & 127) == 127
        for g in (k[:, i], v[:, i]):
            assert np.array_equal(g[~nan], want[~nan]), scales[i]
            assert ((g[nan] & 127) == 127).all(), scales[i]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("layers", [None, 3])
@pytest.mark.parametrize("Hk,Dh,P", [(1, 64, 16), (3, 96, 32), (8, 128, 16)])
def test_kv_commit(Hk, Dh, P, layers, cache):
    print(f"case kv_commit Hk={Hk} D={Dh} P={P} layers={layers} {cache}", flush=True)
    rng = np.random.default_rng(Hk + P)
    n = np.array([1, 9, 40, 64, 30, 7, 5, 5, 12, 3])
    ctx = np.array([0, 13, 31, 100, 16, 3, 2, 9, 8, 7], np.int32)
    R = len(n)
    total = ctx + n
    pages = sum(_up(t, P) for t in total) + 1
    table = H.tables(rng, total, P, pages)
    nodes = 64
    path = np.full((R, nodes), -1, np.int32)
    acc = np.zeros(R, np.int32)
    # every kind of path: none, the chain itself, sparse, overlapping sources and targets
    picks = [[0], [0, 2, 3, 4, 8], list(range(40)), [0] + list(range(2, 64, 2)), [0, 1, 2, 5, 6, 29],
             [0, 3, 2], [1, 2], [0, 4], [0, 5, 11], None]
    for r, p in enumerate(picks):
        if p is None:
            acc[r] = -1
            continue
        path[r, :len(p)] = p
        acc[r] = len(p) - 1
    acc[7] = nodes            # beyond the path's columns
    L = layers or 1
    kc = [H.caches(rng, pages, Hk, Dh, P, cache, DEV) for _ in range(L)]
    k, v = torch.stack([x[0] for x in kc]), torch.stack([x[1] for x in kc])
    table[8, _up(8 + 11, P) - 1] = pages      # a bad page on request 8's path
    want = O.kv_commit(_raw(k), _raw(v), table, ctx, path, acc, P)
    if layers is None:
        k, v = k[0], v[0]
    new = D.dspark_kv_commit(k, v, dev(table), dev(ctx), dev(path), dev(acc))
    torch.cuda.synchronize()
    assert np.array_equal(new.cpu().numpy(), want[2])
    assert [r for r in range(R) if want[2][r] < 0] == [5, 6, 7, 8]
    shape = lambda t: t.reshape(want[0].shape if t.ndim in (5, 6) and t.shape[-1] in (8, 16) and t.ndim - (layers is not None) == 5 else want[1].shape)  # noqa: E731
    assert np.array_equal(shape(_raw(k)), want[0]) and np.array_equal(shape(_raw(v)), want[1])


def test_kv_commit_of_strided_layers():
    print("case kv_commit strided layers", flush=True)
    rng = np.random.default_rng(4)
    kc, vc = H.caches(rng, 4, 2, 64, 16, "fp16", DEV)
    big_k = torch.stack([kc + i for i in range(5)])
    big_v = torch.stack([vc + i for i in range(5)])
    ref = [big_k.clone(), big_v.clone()]
    table = np.array([[2, 0, 3]], np.int32)
    path, acc, ctx = np.array([[0, 3, 9, 17]], np.int32), np.array([3], np.int32), np.array([14], np.int32)
    D.dspark_kv_commit(big_k[::2], big_v[::2], dev(table), dev(ctx), dev(path), dev(acc))
    torch.cuda.synchronize()
    want = O.kv_commit(_raw(ref[0])[::2], _raw(ref[1])[::2], table, ctx, path, acc, 16)
    assert np.array_equal(_raw(big_k)[::2], want[0]) and np.array_equal(_raw(big_v)[::2], want[1])
    assert np.array_equal(_raw(big_k)[1::2], _raw(ref[0])[1::2])


# ---- trees ----

@pytest.mark.parametrize("words", [1, 2, 3, 32])
def test_tree_pack(words):
    print(f"case tree_pack words={words}", flush=True)
    rng = np.random.default_rng(words)
    top = min(32 * words, 400)
    n = np.array([1, 2, 0, top, 31, 32, 33, 7, min(64, top), 0, top + 9, 5])
    cu = H.starts(n)
    par = np.concatenate([H.random_parents(rng, int(x), roots=bool(r % 2)) for r, x in enumerate(n)]).astype(np.int32)
    if len(par) > 300:
        par[cu[3]:cu[4]] = np.arange(-1, n[3] - 1)        # a chain
    par[cu[7] + 3] = 3                                     # its own parent
    par[cu[7] + 5] = 3                                     # a child of it
    par[cu[8] + 1] = -2
    par[cu[11] + 2] = 2 ** 31 - 1
    pos0 = rng.integers(0, 5000, len(n)).astype(np.int32)
    N = int(cu[-1])
    for p0 in (pos0, None):
        want = O.tree_pack(par, cu, p0, words)
        mask = torch.full((N + 4, words), 0x55555555, dtype=torch.int32, device=DEV)
        pos = torch.full((N + 4,), -7, dtype=torch.int32, device=DEV)
        req = torch.full((N + 4,), -7, dtype=torch.int32, device=DEV)
        full = dev(np.concatenate([par, np.zeros(4, np.int32)]))
        D.dspark_tree_pack(full, dev(cu), words, dev(p0), mask=mask, flat_pos=pos, flat_req=req)
        torch.cuda.synchronize()
        assert np.array_equal(mask.cpu().numpy()[:N].view(np.uint32), want[0])
        assert np.array_equal(pos.cpu().numpy()[:N], want[1]) and np.array_equal(req.cpu().numpy()[:N], want[2])
        assert (mask[N:] == 0x55555555).all() and (pos[N:] == -7).all() and (req[N:] == -7).all()


def test_tree_pack_of_a_chain_is_the_causal_mask():
    print("case tree_pack chain", flush=True)
    n = [6, 1, 40]
    cu = H.starts(n)
    par = np.concatenate([np.arange(-1, x - 1) for x in n]).astype(np.int32)
    mask, pos = D.dspark_tree_pack(dev(par), dev(cu), 2)
    m = mask.cpu().numpy().view(np.uint32)
    for r, x in enumerate(n):
        for i in range(x):
            assert int(m[cu[r] + i, 0]) | int(m[cu[r] + i, 1]) << 32 == (1 << (i + 1)) - 1


@pytest.mark.parametrize("V", [1, 7, 4096, 5001])
@pytest.mark.parametrize("agree", [0.0, 0.6, 1.0])
def test_verify_tree(V, agree):
    print(f"case verify_tree V={V} agree={agree}", flush=True)
    rng = np.random.default_rng(V + int(10 * agree))
    n = np.array([1, 5, 0, 64, 65, 130, 20, 33, 2])
    cu = H.starts(n)
    N = int(cu[-1])
    par = np.concatenate([H.random_parents(rng, int(x)) for x in n]).astype(np.int32)
    par[cu[6] + 4] = 9            # a bad parent: never followed
    tok = rng.integers(0, V, N).astype(np.int32)
    logits = rng.normal(0, 1, (N + 3, V)).astype(np.float32)
    for r in range(len(n)):
        for i in range(1, n[r]):
            if par[cu[r] + i] >= 0 and rng.random() < agree:
                logits[cu[r] + par[cu[r] + i], tok[cu[r] + i]] = 9.0
    for nodes in (130, 40, 1):
        want = O.verify_tree(logits[:N], cu, tok, par, nodes)
        room = lambda a: dev(np.concatenate([a, np.zeros(3, np.int32)]))  # noqa: E731
        top = torch.full((N + 3,), -9, dtype=torch.int32, device=DEV)
        acc, path, nxt, top = D.dspark_verify_tree(dev(logits), dev(cu), room(tok), room(par), nodes, target_argmax=top)
        torch.cuda.synchronize()
        assert np.array_equal(acc.cpu().numpy(), want[0]) and np.array_equal(path.cpu().numpy(), want[1])
        assert np.array_equal(nxt.cpu().numpy(), want[2]) and np.array_equal(top.cpu().numpy()[:N], want[3])
        assert (top[N:] == -9).all()


def test_verify_tree_of_chains_equals_verify_greedy():
    print("case verify_tree chains", flush=True)
    from draft_head_step_amd.inputs import make_verify_workload
    wl = make_verify_workload(50, 5, 4099, seed=3, match_rate=0.8)
    ft, _, _, cu = D.dspark_verify_pack(dev(wl["anchors"]), dev(wl["tokens"]), dev(wl["lengths"]))
    c = cu.cpu().numpy()
    N = int(c[-1])
    logits = dev(np.concatenate([wl["target"][r, :c[r + 1] - c[r]] for r in range(50)]))
    acc, nxt, top = D.dspark_verify_greedy(logits, cu, dev(wl["tokens"]))
    par = dev(np.concatenate([np.arange(-1, x - 1) for x in np.diff(c)]).astype(np.int32))
    acc2, path, nxt2, top2 = D.dspark_verify_tree(logits, cu, ft[:N].contiguous(), par, 6)
    torch.cuda.synchronize()
    assert torch.equal(acc, acc2) and torch.equal(nxt, nxt2) and torch.equal(top[:N], top2)
    for r in range(50):
        assert path[r].tolist() == list(range(int(acc[r]) + 1)) + [-1] * (5 - int(acc[r]))


def test_lengths_beyond_an_int32_are_refused():
    print("case lengths at 2^31", flush=True)
    top, P, width = 2 ** 31 - 1, 1024, (1 << 21) + 4
    table = torch.zeros((2, width), dtype=torch.int32, device=DEV)
    cur = dev(np.array([top - 2, 5], np.int32))
    cu = dev(np.array([0, 4, 6], np.int32))
    ring = dev(np.arange(8, dtype=np.int32))
    pool = dev(np.array([0, 8, 0, 0], np.int32))
    slots, new, after = D.dspark_page_map(cur, cu, table, ring, pool, P, 6)
    assert new.tolist() == [top - 2, 7] and after.tolist() == [0, 8, 1, 0]
    assert slots.tolist() == [-1] * 4 + [5, 6]
    kc = torch.zeros((8, 1, 8, P, 8), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros((8, 1, 64, P), dtype=torch.bfloat16, device=DEV)
    path = dev(np.array([[0, 2, 3, -1], [0, 1, -1, -1]], np.int32))
    new = D.dspark_kv_commit(kc, vc, table, cur, path, dev(np.array([2, 1], np.int32)))
    assert new.tolist() == [-1, 7]


@pytest.mark.parametrize("path", [[0, -5, -3, 4], [0, -2 ** 30, -2 ** 30 + 1, -2 ** 30 + 2], [0, -2 ** 31, -1, 3],
                                  [-1, 0, 1, 2], [0, 2, 2, 3], [0, 1, 3, 2 ** 31 - 1]])
def test_kv_commit_refuses_paths_out_of_the_segment(path):
    # entries before the segment or past the table: nothing is moved, the other request is served
    print(f"case kv_commit path {path}", flush=True)
    rng = np.random.default_rng(6)
    k, v = H.caches(rng, 8, 2, 64, 16, "bf16", DEV)
    table = np.array([[3, 1, 6], [0, 7, 2]], np.int32)
    ctx, acc = np.array([20, 21], np.int32), np.array([3, 3], np.int32)
    both = np.array([path, [0, 2, 5, 9]], np.int64).astype(np.int32)
    want = O.kv_commit(_raw(k)[None], _raw(v)[None], table, ctx, both, acc, 16)
    assert want[2].tolist() == [-1, 25]
    new = D.dspark_kv_commit(k, v, dev(table), dev(ctx), dev(both), dev(acc))
    torch.cuda.synchronize()
    assert np.array_equal(new.cpu().numpy(), want[2])
    assert np.array_equal(_raw(k), want[0][0]) and np.array_equal(_raw(v), want[1][0])
