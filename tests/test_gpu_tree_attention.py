"""GPU attention of drafted elements over a paged cache against the 64-bit oracle.

Tolerance, derived from the kernel's documented arithmetic (u = half a step of
the element type, f = 2^-24, W = sum_t p_t |v_t|, A = the largest scale *
sum_d |q_d k_td| of a row, M = the largest |score|, T positions, D channels):
  * a score is a sum of D exact products in fp32, scaled once by a rounded
    factor: |ds| <= (D + 4) f A; forming x - m and the hardware 2^x add
    4 f (M + 1) + 4 f relative to p;
  * so every p is off by e = 2 ((D + 4) f A + 4 f (2 M + 2)) at most (the
    factor 2: the maximum it is taken against, and the sum, carry the same);
  * p is rounded to the element type: u relative, below fp16's normal range
    2^-25 absolute against a sum of at least 1;
  * sums over T positions in fp32: (T + 8) f relative to W, the same for the
    sum of p, and a few rescales;
  * the result is rounded once: u |out|.
  |out - ref| <= u |ref| (1 + e) + W (u + e + 2 (T + 16) f) + tiny
  |lse - ref| <= e + (T + 16) f + 4 f |ref|
"""
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
F = 2.0 ** -24


def make(seed, n, ctx, Hq, Hk, Dh, P, dtype="bf16", cache=None, tree=False, q_std=1.0, extra_rows=0,
         width=None, words=None):
    rng = np.random.default_rng(seed)
    cache = cache or dtype
    n, ctx = np.asarray(n), np.asarray(ctx)
    R, cu = len(n), H.starts(n)
    N = int(cu[-1]) + extra_rows
    total = ctx + n
    pages = int(sum(-(-int(t) // P) for t in total)) + 2
    kc, vc = H.caches(rng, pages, Hk, Dh, P, cache, DEV, 40.0 if cache == "e4m3" else 1.0)
    c = dict(cu=cu, ctx=ctx.astype(np.int32), P=P, N=N, R=R, kc=kc, vc=vc,
             table=H.tables(rng, total, P, pages, width), mask=None, ks=None, vs=None,
             scale=float(Dh ** -0.5),
             q=torch.from_numpy(rng.normal(0, q_std, (N, Hq, Dh)).astype(np.float32)).to(H.TYPES[dtype]).to(DEV))
    if cache == "e4m3":
        c["ks"] = (0.5 + rng.random(Hk)).astype(np.float32) / 40
        c["vs"] = (0.5 + rng.random(Hk)).astype(np.float32) / 40
    if tree:
        par = np.concatenate([H.random_parents(rng, int(x), roots=True) for x in n] + [np.full(extra_rows, -1)])
        W = words or max(1, -(-int(n.max()) // 32))
        m = np.zeros((N, W), np.uint32)
        m[:int(cu[-1])] = O.tree_pack(par, cu, None, W)[0]
        m[int(cu[-1]):] = rng.integers(0, 2 ** 32, (extra_rows, W))
        c["mask"] = m
    return c


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def call(c, **kw):
    mask = None if c["mask"] is None else dev(c["mask"].view(np.int32))
    return D.dspark_tree_attention(c["q"], c["kc"], c["vc"], dev(c["table"]), dev(c["ctx"]), dev(c["cu"]),
                                   c["scale"], tree_mask=mask, k_scale=dev(c["ks"]), v_scale=dev(c["vs"]), **kw)


def oracle(c):
    return O.tree_attention(H.np64(c["q"]), H.np64(c["kc"]), H.np64(c["vc"]), c["table"], c["ctx"], c["cu"],
                            c["P"], c["scale"], c["mask"], c["ks"], c["vs"])


def check(c, out, lse, rows=None):
    ref, rlse, W, A, M = oracle(c)
    Dh = ref.shape[2]
    u = H.half_step(out.dtype)
    T = int((c["ctx"].astype(np.int64) + np.diff(c["cu"])).max())
    A, M = np.where(np.isnan(ref[..., 0]), 0, A), np.where(np.isnan(ref[..., 0]), 0, M)
    e = 2 * ((Dh + 4) * F * A + 4 * F * (2 * M + 2))
    v = np.abs(H.np64(c["vc"]))
    vmax = float(v[np.isfinite(v)].max()) * (1.0 if c["vs"] is None else float(c["vs"].max()))
    tiny = 2.0 ** -25 * (1 + T * vmax) if out.dtype == torch.float16 else 2.0 ** -126
    tol = u * np.abs(ref) * (1 + e[..., None]) + W * (u + e[..., None] + 2 * (T + 16) * F) + tiny
    got = H.np64(out)
    sel = np.arange(int(c["cu"][-1])) if rows is None else np.asarray(rows)
    err = np.abs(got - ref)[sel]
    assert np.isfinite(got[sel]).all()
    worst = float((err / tol[sel]).max()) if len(sel) else 0.0
    print(f"  worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0
    if lse is not None:
        gl = lse.cpu().numpy().astype(np.float64)[sel]
        rl = rlse[sel]
        empty = np.isneginf(rl)
        assert np.array_equal(empty, np.isneginf(gl))
        assert np.array_equal(got[sel][empty], np.zeros_like(got[sel][empty]))
        lt = e[sel] + (T + 16) * F + 4 * F * np.where(empty, 0, np.abs(rl))
        assert (np.abs(gl - rl)[~empty] <= lt[~empty]).all()


CASES = [
    # n per request, ctx per request, Hq, Hk, D, P
    ([1], [0], 1, 1, 64, 16),                       # one token, nothing before it
    ([1], [1], 4, 4, 64, 16),
    ([1], [15], 16, 2, 128, 16),
    ([1], [16], 16, 2, 128, 16),
    ([3], [0], 8, 1, 96, 16),                       # a prompt of three
    ([6, 1, 4], [31, 32, 33], 32, 8, 128, 16),      # around a tile's end
    ([2, 5], [63, 64], 8, 2, 192, 32),
    ([7, 3], [127, 130], 14, 2, 64, 64),            # seven heads a group
    ([5, 5], [1000, 17], 4, 1, 256, 128),
    ([17, 1, 33], [100, 999, 5], 10, 2, 128, 16),   # several row tiles
    ([1, 2], [2500, 3], 16, 16, 64, 1024),          # one large page
    ([130], [40], 8, 2, 128, 16),                   # a piece of a prompt
    ([1, 300], [70, 0], 4, 2, 64, 32),
]


@pytest.mark.parametrize("cache", ["same", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_oracle(case, tree, dtype, cache):
    n, ctx, Hq, Hk, Dh, P = CASES[case]
    print(f"case attention {CASES[case]} tree={tree} {dtype} cache={cache}", flush=True)
    c = make(case, n, ctx, Hq, Hk, Dh, P, dtype, dtype if cache == "same" else "e4m3", tree)
    out, lse = call(c, want_lse=True)
    torch.cuda.synchronize()
    check(c, out, lse)


def test_many_requests_of_every_length():
    print("case attention 70 requests", flush=True)
    rng = np.random.default_rng(5)
    n = rng.integers(0, 9, 70)
    n[3] = n[69] = 0
    ctx = rng.integers(0, 300, 70)
    c = make(50, n, ctx, 8, 2, 64, 16, tree=True)
    out, lse = call(c, want_lse=True)
    torch.cuda.synchronize()
    check(c, out, lse)


@pytest.mark.parametrize("tree", [False, True])
def test_long_context_split_and_joined(tree):
    print(f"case attention long tree={tree}", flush=True)
    c = make(60, [6, 2], [9001, 4000], 8, 2, 128, 16, tree=tree, q_std=2.0)
    out, lse = call(c, want_lse=True)
    torch.cuda.synchronize()
    check(c, out, lse)


@pytest.mark.parametrize("Dh", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("n,ctx", [([1], [9000]), ([6], [1100]), ([50], [5000]), ([3, 64], [4000, 20])])
def test_few_tiles_in_many_parts(n, ctx, Dh):
    # one or two requests over all workgroups: tiles of up to dozens of parts
    print(f"case attention many parts n={n} ctx={ctx} D={Dh}", flush=True)
    c = make(320 + Dh, n, ctx, 4, 1, Dh, 16, "bf16", "e4m3" if Dh == 96 else "bf16", tree=len(n) == 1)
    out, lse = call(c, want_lse=True)
    torch.cuda.synchronize()
    check(c, out, lse)
    again, _ = call(c)
    torch.cuda.synchronize()
    assert torch.equal(out, again)


@pytest.mark.parametrize("Dh", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("P", [16, 32, 64, 256])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3")])
def test_many_rows_over_a_cut_context(Dh, P, dtype, cache):
    # tiles of all waves and of some, cut between workgroups, in every head size and page kind
    print(f"case attention many rows D={Dh} P={P} {dtype} {cache}", flush=True)
    c = make(300 + Dh + P, [70, 3, 33], [1500, 2100, 640], 8, 2, Dh, P, dtype, cache, tree=P != 32)
    out, lse = call(c, want_lse=True)
    torch.cuda.synchronize()
    check(c, out, lse)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [[5, 2, 4], [40, 30, 50]])
def test_long_masks(n, cache):
    # mask rows of more than two words, for few rows and for many, around an odd start
    print(f"case attention long masks n={n} {cache}", flush=True)
    c = make(310, n, [45, 700, 131], 4, 2, 128, 16, "bf16", cache, tree=True, words=6)
    out, lse = call(c, want_lse=True)
    torch.cuda.synchronize()
    check(c, out, lse)
    c = make(311, [150, 97], [77, 3], 2, 1, 64, 64, "bf16", cache, tree=True)
    out, lse = call(c, want_lse=True)
    torch.cuda.synchronize()
    check(c, out, lse)


def test_hundreds_of_requests():
    # more requests than threads scan their lengths
    print("case attention 700 requests", flush=True)
    rng = np.random.default_rng(9)
    c = make(312, rng.integers(0, 4, 700), rng.integers(0, 60, 700), 2, 1, 64, 16)
    out, lse = call(c, want_lse=True)
    torch.cuda.synchronize()
    check(c, out, lse)
    c = make(313, rng.integers(0, 3, 600), rng.integers(0, 600, 600), 2, 2, 64, 32)
    out, lse = call(c, want_lse=True)
    torch.cuda.synchronize()
    check(c, out, lse)


@pytest.mark.parametrize("scale", [0.0, -0.11])
def test_scales_without_a_usual_sign(scale):
    print(f"case attention scale {scale}", flush=True)
    for tree in (False, True):
        c = make(314, [5, 40], [70, 600], 8, 2, 64, 16, tree=tree)
        c["scale"] = scale
        out, lse = call(c, want_lse=True)
        torch.cuda.synchronize()
        check(c, out, lse)


@pytest.mark.parametrize("n", [[1, 5, 3], [40, 9, 30]])
def test_output_over_the_queries(n):
    # the same rows as q: cut tiles and uncut ones, few rows and many
    print(f"case attention in place n={n}", flush=True)
    for ctx in ([3, 90, 20], [3000, 700, 1500]):
        c = make(316, n, ctx, 8, 2, 128, 16)
        want, _ = call(c)
        c["q"] = c["q"].clone()
        got, _ = call(c, out=c["q"])
        torch.cuda.synchronize()
        assert got.data_ptr() == c["q"].data_ptr()
        assert torch.equal(got, want)


def test_binding_refuses_what_does_not_fit():
    print("case attention refusals", flush=True)
    c = make(315, [3, 2], [20, 5], 4, 2, 64, 16)
    f = make(315, [3, 2], [20, 5], 4, 2, 64, 16, cache="e4m3")

    def bad(error, base=c, **kw):
        d = dict(base)
        d.update(kw)
        with pytest.raises(error):
            call(d)

    bad(ValueError, table=c["table"][:1])
    bad(TypeError, table=c["table"].astype(np.int64))
    bad(ValueError, ctx=c["ctx"][:1])
    bad(ValueError, cu=c["cu"][:2])
    bad(TypeError, q=c["q"].float())
    bad(ValueError, q=c["q"].transpose(0, 1))
    bad(ValueError, q=c["q"][:, :, :32])
    bad(TypeError, vc=c["vc"].half())
    bad(ValueError, vc=c["vc"][:-1])
    bad(ValueError, kc=c["kc"].transpose(2, 3))
    bad(ValueError, mask=np.zeros((3, 1), np.uint32))
    bad(D.DsparkError, q=c["q"][:, :3].contiguous())             # heads no multiple of the caches'
    bad(D.DsparkError, q=c["q"].half())                          # another type than the cache's
    bad(D.DsparkError, base=f, ks=None, vs=None)                 # no scales
    bad(D.DsparkError, ks=np.ones(2, np.float32), vs=np.ones(2, np.float32))
    bad(ValueError, base=f, vs=None)
    bad(D.DsparkError, scale=float("nan"))
    bad(D.DsparkError, q=c["q"][:1].expand(5, 4, 64))            # rows that lie on each other
    with pytest.raises(D.DsparkError):
        call(c, workspace=torch.empty(512, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        call(c, workspace=torch.empty(1 << 26, dtype=torch.uint8))
    with pytest.raises(ValueError):
        call(c, out=torch.empty((5, 4, 32), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(TypeError):
        call(c, lse=torch.empty((5, 4), dtype=torch.float16, device=DEV))


def test_rows_that_see_nothing():
    # mask rows of zeros: without a context nothing is seen, with one the context alone
    print("case attention empty rows", flush=True)
    c = make(61, [5, 4], [0, 20], 4, 2, 64, 16, tree=True)
    c["mask"][1] = 0
    c["mask"][3] = 0
    c["mask"][6] = 0
    out, lse = call(c, want_lse=True)
    torch.cuda.synchronize()
    assert np.isneginf(lse.cpu().numpy()[[1, 3]]).all() and not out[1].any() and not out[3].any()
    check(c, out, lse)


def test_mask_bits_beyond_the_segment_are_not_set():
    print("case attention mask bits beyond", flush=True)
    c = make(62, [3, 40], [10, 50], 4, 2, 64, 16, tree=True, words=3)
    c["mask"][:3] |= np.uint32(0xfffffff8)
    c["mask"][:, 2] = 0xffffffff
    out, lse = call(c, want_lse=True)
    short = dict(c)
    torch.cuda.synchronize()
    check(c, out, lse)
    # one word only: nodes from 32 on are seen by no one
    short["mask"] = np.ascontiguousarray(c["mask"][:, :1])
    out, lse = call(short, want_lse=True)
    torch.cuda.synchronize()
    check(short, out, lse)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("cache", ["bf16", "fp16", "e4m3"])
def test_unseen_places_do_not_matter(cache, bad):
    # Keys and values behind the last element, and those of nodes that a row does not
    # see, hold NaN or infinities.
    if cache == "e4m3" and not np.isnan(bad):
        pytest.skip("e4m3 has no infinities")
    print(f"case attention unseen {cache} {bad}", flush=True)
    c = make(63, [6, 40], [45, 131], 8, 2, 128, 32, "fp16" if cache == "fp16" else "bf16", cache, tree=True)
    clean = call(c)[0].clone()
    total = c["ctx"] + np.diff(c["cu"])
    P = c["P"]
    kf, vf = c["kc"].float(), c["vc"].float()
    held = set()
    for r in range(c["R"]):
        pages = c["table"][r, :-(-int(total[r]) // P)]
        held |= set(int(p) for p in pages)
        tail = int(total[r]) % P
        if tail:
            kf[int(pages[-1]), :, :, tail:] = bad
            vf[int(pages[-1]), :, :, tail:] = bad
    for p in set(range(kf.shape[0])) - held:
        kf[p] = bad
        vf[p] = bad
    c["kc"], c["vc"] = kf.to(c["kc"].dtype), vf.to(c["vc"].dtype)
    out, lse = call(c, want_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(out, clean), "what lies behind the last element reached a row"
    check(c, out, lse)
    # node 2 of the first request: only rows that see it may change
    pos = int(c["ctx"][0]) + 2
    page, o = int(c["table"][0, pos // P]), pos % P
    kf, vf = c["kc"].float(), c["vc"].float()
    kf[page, :, :, o] = bad
    vf[page, :, :, o] = bad
    kept = (c["kc"], c["vc"])
    c["kc"], c["vc"] = kf.to(kept[0].dtype), vf.to(kept[1].dtype)
    out = call(c)[0]
    torch.cuda.synchronize()
    rows = [e for e in range(int(c["cu"][-1])) if e >= 6 or not (int(c["mask"][e, 0]) >> 2) & 1]
    assert 2 not in rows and len(rows) > 30
    c["kc"], c["vc"] = kept
    check(c, out, None, rows)
    assert not torch.isfinite(out[2]).all()


def test_masked_infinities_of_many_nodes():
    # every value of nodes 1, 4 and 9 infinite, half of them negative: rows that see none
    # of them, one, or several
    print("case attention infinities in a tree", flush=True)
    c = make(64, [20], [33], 4, 2, 64, 16, tree=True)
    P = c["P"]
    vf = c["vc"].float()
    bits = [1, 4, 9]
    for b in bits:
        pos = 33 + b
        vf[int(c["table"][0, pos // P]), :, :, pos % P] = float("inf") if b != 4 else -float("inf")
    clean = c["vc"]
    c["vc"] = vf.to(clean.dtype)
    out = H.np64(call(c)[0])
    torch.cuda.synchronize()
    got = dict(c)
    got["vc"] = clean
    sees = np.array([[bool((int(c["mask"][e, 0]) >> b) & 1) for b in bits] for e in range(20)])
    for e in range(20):
        up, down = sees[e, 0] or sees[e, 2], sees[e, 1]
        if up and down:
            assert np.isnan(out[e]).all()
        elif up:
            assert (out[e] == np.inf).all()
        elif down:
            assert (out[e] == -np.inf).all()
    rows = [e for e in range(20) if not sees[e].any()]
    assert rows
    check(got, call(c)[0], None, rows)


def test_scores_far_below_and_above():
    # large scores: sums of one, differences that leave every other p at zero
    print("case attention large scores", flush=True)
    c = make(65, [4, 4], [200, 3], 8, 2, 128, 16, q_std=60.0)
    out, lse = call(c, want_lse=True)
    torch.cuda.synchronize()
    check(c, out, lse)


def test_strides_of_queries_and_outputs():
    print("case attention strides", flush=True)
    c = make(66, [5, 9], [50, 7], 8, 2, 64, 16)
    wide = torch.zeros((c["N"], 16, 64), dtype=torch.bfloat16, device=DEV)
    wide[:, 4:12] = c["q"]
    ref = call(c)[0]
    c["q"] = wide[:, 4:12]
    outw = torch.full((c["N"], 12, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    call(c, out=outw[:, 2:10])
    torch.cuda.synchronize()
    assert torch.equal(outw[:, 2:10], ref)
    assert (outw[:, :2] == 7).all() and (outw[:, 10:] == 7).all()


def test_rows_behind_the_last_sequence_stay():
    print("case attention rows behind", flush=True)
    for tree in (False, True):
        c = make(67, [5, 2], [50, 7], 8, 2, 64, 16, tree=tree, extra_rows=9)
        out = torch.full((c["N"], 8, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((c["N"], 8), 7.0, device=DEV)
        call(c, out=out, lse=lse)
        torch.cuda.synchronize()
        assert (out[7:] == 7).all() and (lse[7:] == 7).all()
        check(c, out, lse)


def test_bad_requests_give_nan_and_leave_the_others():
    print("case attention bad requests", flush=True)
    n, ctx = [3, 2, 4, 1, 2, 5], [40, 33, 70, 5, 20, 64]
    c = make(68, n, ctx, 8, 2, 128, 16, width=6)
    c["table"][1, 1] = c["kc"].shape[0]      # past the last page
    c["table"][2, 4] = -1
    c["ctx"] = c["ctx"].copy()
    c["ctx"][3] = -1
    c["ctx"][4] = 6 * 16                     # more positions than the table has
    out, lse = call(c, want_lse=True)
    torch.cuda.synchronize()
    good = []
    for r in range(6):
        s = slice(int(c["cu"][r]), int(c["cu"][r + 1]))
        if r in (1, 2, 3, 4):
            assert torch.isnan(out[s]).all() and torch.isnan(lse[s]).all(), r
        else:
            good += range(s.start, s.stop)
    check(c, out, lse, good)


def test_results_repeat_and_do_not_depend_on_the_workspace():
    print("case attention repeat", flush=True)
    c = make(69, [6, 33, 1], [5000, 800, 3], 16, 2, 128, 16, tree=True)
    ws = torch.empty(D.dspark_tree_attention_workspace(3, c["N"], 16, 2, 128), dtype=torch.uint8, device=DEV)
    ref = None
    for fill in (0, 255, 165):
        ws.fill_(fill)
        out, lse = call(c, want_lse=True, workspace=ws)
        torch.cuda.synchronize()
        if ref is None:
            ref = (out, lse)
        assert torch.equal(out.view(torch.int16), ref[0].view(torch.int16))
        assert torch.equal(lse.view(torch.int32), ref[1].view(torch.int32))


def test_no_scratch_for_long_tables_and_far_pages():
    # pages beyond 2^31 elements of the cache: 64-bit offsets
    print("case attention far pages", flush=True)
    Hk, Dh, P = 8, 128, 64
    pages = (1 << 31) // (Hk * Dh * P) + 40
    kc = torch.zeros((pages, Hk, Dh // 8, P, 8), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros((pages, Hk, Dh, P), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    kc[-9:].normal_(generator=g)
    vc[-9:].normal_(generator=g)
    table = np.arange(pages - 9, pages, dtype=np.int32)[None, ::-1].copy()
    q = torch.randn((3, 8, Dh), device=DEV, generator=g).to(torch.bfloat16)
    small = dict(cu=np.array([0, 3], np.int32), ctx=np.array([500], np.int32), P=P, N=3, R=1, kc=kc, vc=vc,
                 table=table, mask=None, ks=None, vs=None, scale=Dh ** -0.5, q=q)
    out, lse = call(small, want_lse=True)
    torch.cuda.synchronize()
    near = dict(small, kc=kc[-9:].contiguous(), vc=vc[-9:].contiguous(),
                table=np.arange(9, dtype=np.int32)[None, ::-1].copy())
    check(near, out, lse)


def test_seeded_sweep():
    rng = np.random.default_rng(2024)
    for it in range(40):
        R = int(rng.integers(1, 12))
        tree = bool(rng.integers(0, 2))
        Hk = int(rng.choice([1, 2, 3]))
        g = int(rng.choice([1, 2, 4, 5, 8, 16]))
        Dh = int(rng.choice([64, 96, 128, 192, 256]))
        P = int(rng.choice([16, 32, 64, 256]))
        dtype = str(rng.choice(["bf16", "fp16"]))
        cache = str(rng.choice([dtype, dtype, "e4m3"]))
        n = rng.integers(0 if R > 1 else 1, int(rng.choice([2, 8, 40])) + 1, R)
        n[0] = max(n[0], 1)
        ctx = rng.integers(0, int(rng.choice([4, 70, 700])), R)
        print(f"case attention sweep {it}: n={n.tolist()} ctx={ctx.tolist()} Hk={Hk} g={g} D={Dh} P={P} {dtype} {cache} tree={tree}", flush=True)
        c = make(1000 + it, n, ctx, Hk * g, Hk, Dh, P, dtype, cache, tree, extra_rows=int(rng.integers(0, 3)))
        out, lse = call(c, want_lse=True)
        torch.cuda.synchronize()
        check(c, out, lse)


def test_outputs_on_parts_of_the_queries_are_refused():
    print("case attention outputs on queries", flush=True)
    c = make(70, [3, 2], [20, 5], 4, 2, 64, 16)
    wide = torch.zeros((7, 12, 64), dtype=torch.bfloat16, device=DEV)
    c["q"] = wide[:5, :4]
    c["q"].copy_(make(70, [3, 2], [20, 5], 4, 2, 64, 16)["q"])
    want = call(dict(c, q=c["q"].contiguous()))[0]
    for out in (wide[1:6, :4], wide[:5, 1:5], wide[2:7, :4]):
        with pytest.raises(D.DsparkError) as e:
            call(c, out=out)
        assert e.value.status == 1
    got = call(c, out=wide[:5, 4:8])[0]              # beside them
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    call(c, out=c["q"])                              # on them
    torch.cuda.synchronize()
    assert torch.equal(c["q"], want)


@pytest.mark.parametrize("width", [40, 5000, 70000])
@pytest.mark.parametrize("n,ctx,tree", [([1], [200], False), ([6, 0, 2], [200, 31, 500], False), ([40, 9], [90, 300], True)])
def test_tables_much_wider_than_the_requests(n, ctx, tree, width):
    # what a server's table looks like; ids behind a request's last page are no one's
    print(f"case attention width {width} n={n} ctx={ctx}", flush=True)
    c = make(71, n, ctx, 8, 2, 128, 16, tree=tree, width=width)
    out, lse = call(c, want_lse=True)
    torch.cuda.synchronize()
    check(c, out, lse)
