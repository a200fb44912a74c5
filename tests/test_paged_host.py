"""Verification over a paged cache without a GPU: the index arithmetic that guards
every address (compiled for the host), the refusals of the C entry points and of
the binding, and pins of the oracle."""
import ctypes
import os
import shutil
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import draft_head_step_amd as D  # noqa: E402
from oracle import paged_oracle as O  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
no_gpu = pytest.mark.skipif(os.path.exists("/dev/kfd"),
                            reason="placeholder-pointer checks run only where no GPU is visible")
OK, EINVAL, EWORKSPACE, EUNSUPPORTED = 0, 1, 2, 3
P = 0x10000

SHIM = r"""
#include "paged.h"
using namespace dspark;
extern "C" {
int t_shift(int p) { return page_shift(p); }
int t_page_ok(int p, int n) { return page_ok(p, n); }
int t_slot_ok(int64_t s, int sh, int n) { return slot_ok(s, sh, n); }
void t_need(int c, int a, int b, int sh, int mp, int64_t* o) { PageNeed p = page_need(c, a, b, sh, mp); o[0] = p.has; o[1] = p.want; o[2] = p.fits; }
void t_give(int c, int k, int sh, int mp, int64_t* o) { PageNeed p = page_give(c, k, sh, mp); o[0] = p.has; o[1] = p.want; o[2] = p.fits; }
int t_head(int h, int n) { return ring_head(h, n); }
int t_count(int c, int n) { return ring_count(c, n); }
int t_ring(int h, int64_t i, int n) { return ring_at(h, i, n); }
int64_t t_k(int64_t p, int h, int d, int o, int Hk, int D, int sh, int c) { return k_offset(p, h, d, o, Hk, D, sh, c); }
int64_t t_v(int64_t p, int h, int d, int o, int Hk, int D, int sh) { return v_offset(p, h, d, o, Hk, D, sh); }
int t_parent(int p, int i) { return parent_ok(p, i); }
int t_path(const int* p, int i) { return path_step_ok(p, i); }
}
"""
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("paged")
    (d / "shim.cpp").write_text(SHIM)
    so = str(d / "shim.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-static-libubsan",
                    "-shared", "-fPIC", "-I", os.path.join(ROOT, "draft_head_step_amd", "csrc"),
                    str(d / "shim.cpp"), "-o", so], check=True)
    L = ctypes.CDLL(so)
    i64, i32 = ctypes.c_int64, ctypes.c_int
    L.t_slot_ok.argtypes = [i64, i32, i32]
    L.t_ring.argtypes = [i32, i64, i32]
    L.t_k.argtypes = [i64] + [i32] * 7
    L.t_k.restype = i64
    L.t_v.argtypes = [i64] + [i32] * 6
    L.t_v.restype = i64
    return L


def test_page_sizes(shim):
    assert [p for p in range(-5, 5000) if shim.t_shift(p) >= 0] == [16, 32, 64, 128, 256, 512, 1024]
    assert all(shim.t_shift(1 << s) == s for s in range(4, 11))
    assert shim.t_shift(BIG) == shim.t_shift(-BIG - 1) == -1


def test_bad_pages_and_slots_are_seen(shim):
    for n in (1, 7, BIG):
        for p in (-BIG - 1, -1, 0, 1, 6, 7, BIG - 1, BIG):
            assert bool(shim.t_page_ok(p, n)) == (0 <= p < n)
        for sh in (4, 10):
            top = n << sh
            for s in (-2 ** 63, -1, 0, 15, top - 1, top, 2 ** 63 - 1):
                assert bool(shim.t_slot_ok(s, sh, n)) == (0 <= s < top)


def _three(f, *a):
    o = (ctypes.c_int64 * 3)()
    f(*a, o)
    return list(o)


@pytest.mark.parametrize("shift", [4, 7])
def test_page_needs(shim, shift):
    size = 1 << shift
    edges = [-BIG - 1, -1, 0, 1, size - 1, size, size + 1, 1000, BIG - 1, BIG]
    for cur in edges:
        for a, b in ((0, 0), (3, 2), (-1, 5), (0, 1), (5, 5 + size), (0, BIG), (7, -4)):
            for mp in (1, 3, BIG):
                has, want, fits = _three(shim.t_need, cur, a, b, shift, mp)
                n = b - a
                ok = cur >= 0 and n >= 0 and a >= 0 and -(-(cur + n) // size) <= mp and cur + n <= BIG
                assert bool(fits) == ok
                if ok:
                    assert (has, want) == (-(-cur // size), -(-(cur + n) // size))
        for keep in edges:
            for mp in (1, 3, BIG):
                has, want, fits = _three(shim.t_give, cur, keep, shift, mp)
                ok = cur >= 0 and -(-cur // size) <= mp
                assert bool(fits) == ok
                assert (has, want) == ((-(-cur // size), -(-min(max(keep, 0), cur) // size)) if ok else (0, 0))


def test_ring_places(shim):
    for n in (1, 5, BIG):
        for h in (-BIG - 1, -6, -1, 0, 4, 5, BIG):
            assert shim.t_head(h, n) == h % n
            assert shim.t_count(h, n) == min(max(h, 0), n)
        for h in (0, n // 2, n - 1):
            for i in (0, 1, n - 1, n, 2 * n):
                assert shim.t_ring(h, i, n) == (h + i) % n


def test_cache_offsets_are_a_permutation_and_64_bit(shim):
    for Hk, Dh, sh, c in ((3, 64, 4, 8), (2, 96, 5, 16)):
        size = 1 << sh
        k = np.arange(2 * Hk * Dh * size).reshape(2, Hk, Dh // c, size, c)
        v = np.arange(2 * Hk * Dh * size).reshape(2, Hk, Dh, size)
        for p in range(2):
            for h in range(Hk):
                for d in range(Dh):
                    for o in range(size):
                        assert shim.t_k(p, h, d, o, Hk, Dh, sh, c) == k[p, h, d // c, o, d % c]
                        assert shim.t_v(p, h, d, o, Hk, Dh, sh) == v[p, h, d, o]
    p = BIG - 1
    assert shim.t_v(p, 7, 127, 63, 8, 128, 6) == ((p * 8 + 7) * 128 + 127) * 64 + 63
    assert shim.t_k(p, 7, 127, 63, 8, 128, 6, 8) == (((p * 8 + 7) * 16 + 15) * 64 + 63) * 8 + 7


def test_links_and_paths(shim):
    for i in (0, 1, 5):
        for p in (-BIG - 1, -2, -1, 0, i - 1, i, i + 1, BIG):
            assert bool(shim.t_parent(p, i)) == (-1 <= p < i)
    for path, good in (([0, 1, 4], [1, 1, 1]), ([1, 2, 2], [0, 1, 0]), ([0, -3, BIG], [1, 0, 1])):
        a = (ctypes.c_int * 3)(*path)
        assert [shim.t_path(a, i) for i in range(3)] == good


def test_every_entry_of_a_path_is_safe_by_itself(shim):
    # Each entry is judged by a thread of its own, whatever the others find: one that passes is
    # a node of the segment, at or behind its own place.
    low = -2 ** 30
    for path, good in (([0, -5, -3], [1, 0, 0]), ([0, low, low + 1], [1, 0, 0]), ([0, -BIG - 1, -BIG], [1, 0, 0]),
                       ([0, 0, 1], [1, 0, 0]), ([0, 1, 2], [1, 1, 1]), ([0, 7, BIG], [1, 1, 1])):
        a = (ctypes.c_int * 3)(*path)
        assert [shim.t_path(a, i) for i in range(3)] == good, path
    rng = np.random.default_rng(0)
    for _ in range(300):
        path = rng.integers(-4, 7, 5)
        a = (ctypes.c_int * 5)(*path.tolist())
        for i in range(5):
            if shim.t_path(a, i):
                assert path[i] >= i and (i == 0 or path[i] > path[i - 1])


# ---- refusals of the C entry points ----

@no_gpu
@pytest.mark.parametrize("kw,want", [
    *[(dict([(n, None)]), EINVAL) for n in ("cur", "cu", "table", "ring", "pool", "out", "slots", "new")],
    (dict(R=0), EINVAL), (dict(N=0), EINVAL), (dict(mp=0), EINVAL), (dict(np_=-1), EINVAL),
    (dict(ps=8), EINVAL), (dict(ps=48), EINVAL), (dict(ps=2048), EINVAL), (dict(out=P), EINVAL),
    (dict(new=2 * P), EINVAL), (dict(new=2 * P + 12), EINVAL), (dict(out=P + 8), EINVAL), (dict(R=16385), EUNSUPPORTED),
])
def test_page_map_rejects(kw, want):
    a = dict(cur=2 * P, cu=P, R=4, N=8, ps=16, mp=4, np_=9, table=P, ring=P, pool=P, out=3 * P, slots=P, new=P)
    a.update(kw)
    assert D.lib().dspark_page_map(a["cur"], a["cu"], a["R"], a["N"], a["ps"], a["mp"], a["np_"], a["table"],
                                   a["ring"], a["pool"], a["out"], a["slots"], a["new"], None) == want
    assert D.lib().dspark_last_error() != b""


@no_gpu
@pytest.mark.parametrize("kw,want", [
    *[(dict([(n, None)]), EINVAL) for n in ("cur", "keep", "table", "ring", "pool", "out")],
    (dict(R=-1), EINVAL), (dict(ps=15), EINVAL), (dict(mp=0), EINVAL), (dict(np_=0), EINVAL), (dict(out=P), EINVAL),
    (dict(R=20000), EUNSUPPORTED),
])
def test_page_trim_rejects(kw, want):
    a = dict(cur=P, keep=P, R=4, ps=16, mp=4, np_=9, table=P, ring=P, pool=P, out=3 * P)
    a.update(kw)
    assert D.lib().dspark_page_trim(a["cur"], a["keep"], a["R"], a["ps"], a["mp"], a["np_"], a["table"], a["ring"],
                                    a["pool"], a["out"], None) == want


@no_gpu
@pytest.mark.parametrize("kw,want", [
    *[(dict([(n, None)]), EINVAL) for n in ("k", "v", "slots", "kc", "vc")],
    (dict(N=0), EINVAL), (dict(Hk=0), EINVAL), (dict(D=0), EINVAL), (dict(ps=17), EINVAL), (dict(np_=0), EINVAL),
    (dict(dt=2), EINVAL), (dict(dt=7), EINVAL), (dict(ct=1), EINVAL), (dict(ct=2), EINVAL), (dict(ct=2, sk=P), EINVAL),
    (dict(sk=P, sv=P), EINVAL), (dict(ks=508), EINVAL), (dict(ks=504), EINVAL), (dict(vs=513), EINVAL),
    (dict(k=P + 8), EINVAL), (dict(vc=P + 4), EINVAL), (dict(D=80, ks=640, vs=640), EUNSUPPORTED),
    (dict(D=512, ks=1 << 20, vs=1 << 20), EUNSUPPORTED), (dict(Hk=65536, ks=1 << 24, vs=1 << 24), EUNSUPPORTED),
])
def test_kv_store_rejects(kw, want):
    a = dict(k=P, v=P, ks=512, vs=512, dt=0, slots=P, count=None, N=4, Hk=4, D=128, ps=16, np_=9, ct=0, sk=None, sv=None,
             kc=P, vc=P)
    a.update(kw)
    assert D.lib().dspark_kv_store(a["k"], a["v"], a["ks"], a["vs"], a["dt"], a["slots"], a["count"], a["N"], a["Hk"],
                                   a["D"], a["ps"], a["np_"], a["ct"], a["sk"], a["sv"], a["kc"], a["vc"], None) == want


@no_gpu
@pytest.mark.parametrize("kw,want", [
    *[(dict([(n, None)]), EINVAL) for n in ("kc", "vc", "table", "ctx", "path", "acc", "new")],
    *[(dict([(n, 0)]), EINVAL) for n in ("L", "R", "nodes", "Hk", "D", "mp", "np_")],
    (dict(ct=3), EINVAL), (dict(ct=-1), EINVAL), (dict(ps=20), EINVAL), (dict(kl=4), EINVAL), (dict(vl=12), EINVAL),
    (dict(ct=2, kl=8), EINVAL), (dict(kc=P + 8), EINVAL), (dict(D=72), EUNSUPPORTED), (dict(L=70000), EUNSUPPORTED),
    (dict(R=70000), EUNSUPPORTED), (dict(new=P), EINVAL), (dict(ctx=2 * P, new=P + 4), EINVAL),
    (dict(acc=2 * P, new=P - 4), EINVAL),
])
def test_kv_commit_rejects(kw, want):
    a = dict(kc=P, vc=P, kl=0, vl=0, L=1, ct=0, table=P, ctx=P, path=P, acc=P, R=2, nodes=8, Hk=2, D=64, ps=16, mp=4, np_=9,
             new=P)
    a.update(kw)
    assert D.lib().dspark_kv_commit(a["kc"], a["vc"], a["kl"], a["vl"], a["L"], a["ct"], a["table"], a["ctx"], a["path"],
                                    a["acc"], a["R"], a["nodes"], a["Hk"], a["D"], a["ps"], a["mp"], a["np_"], a["new"],
                                    None) == want


@no_gpu
@pytest.mark.parametrize("kw,want", [
    *[(dict([(n, None)]), EINVAL) for n in ("q", "kc", "vc", "table", "ctx", "cu", "out")],
    *[(dict([(n, 0)]), EINVAL) for n in ("R", "N", "Hq", "Hk", "D", "mp", "np_")],
    (dict(Hq=9), EINVAL), (dict(ps=12), EINVAL), (dict(dt=2), EINVAL), (dict(ct=1), EINVAL), (dict(ct=2), EINVAL),
    (dict(sk=P), EINVAL), (dict(words=1), EINVAL), (dict(mask=P, words=0), EINVAL), (dict(mask=P, words=-1), EINVAL),
    (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(scale=3e38), EINVAL), (dict(q=P + 2), EINVAL), (dict(qs=516), EINVAL),
    (dict(qs=504), EINVAL), (dict(os=504), EINVAL), (dict(out=P + 8), EINVAL), (dict(D=48, qs=512), EUNSUPPORTED),
    (dict(mask=P, words=33), EUNSUPPORTED), (dict(R=(1 << 20) + 1), EUNSUPPORTED), (dict(N=1 << 29), EUNSUPPORTED),
    (dict(ws=None), EWORKSPACE), (dict(wb=16), EWORKSPACE), (dict(ws=P + 128), EINVAL),
])
def test_tree_attention_rejects(kw, want):
    a = dict(q=P, qs=512, dt=0, kc=P, vc=P, ct=0, sk=None, sv=None, table=P, ctx=P, cu=P, mask=None, words=0, R=2, N=4, Hq=8,
             Hk=2, D=64, ps=16, mp=4, np_=9, scale=0.125, out=P, os=512, lse=None, ws=P, wb=1 << 40)
    a.update(kw)
    assert D.lib().dspark_tree_attention(a["q"], a["qs"], a["dt"], a["kc"], a["vc"], a["ct"], a["sk"], a["sv"], a["table"],
                                         a["ctx"], a["cu"], a["mask"], a["words"], a["R"], a["N"], a["Hq"], a["Hk"], a["D"],
                                         a["ps"], a["mp"], a["np_"], a["scale"], a["out"], a["os"], a["lse"], a["ws"], a["wb"],
                                         None) == want
    assert D.lib().dspark_last_error() != b""


def test_tree_attention_workspace_sizes():
    f = D.dspark_tree_attention_workspace
    assert f(0, 4, 8, 2, 64) == f(2, 0, 8, 2, 64) == f(2, 4, 9, 2, 64) == f(2, 4, 8, 2, 80) == f(2, 1 << 29, 8, 2, 64) == 0
    assert f(2, 4, 8, 2, 64) > 0


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(par=None), EINVAL), (dict(cu=None), EINVAL), (dict(mask=None), EINVAL), (dict(R=0), EINVAL), (dict(N=0), EINVAL),
    (dict(words=0), EINVAL), (dict(words=33), EUNSUPPORTED),
])
def test_tree_pack_rejects(kw, want):
    a = dict(par=P, cu=P, R=2, N=8, words=1, mask=P)
    a.update(kw)
    assert D.lib().dspark_tree_pack(a["par"], a["cu"], None, a["R"], a["N"], a["words"], a["mask"], None, None, None) == want


@no_gpu
@pytest.mark.parametrize("kw,want", [
    *[(dict([(n, None)]), EINVAL) for n in ("z", "cu", "tok", "par", "top", "acc", "path", "nxt")],
    *[(dict([(n, 0)]), EINVAL) for n in ("R", "N", "nodes", "V")],
])
def test_verify_tree_rejects(kw, want):
    a = dict(z=P, cu=P, tok=P, par=P, R=2, N=8, nodes=4, V=100, top=P, acc=P, path=P, nxt=P)
    a.update(kw)
    assert D.lib().dspark_verify_tree(a["z"], a["cu"], a["tok"], a["par"], a["R"], a["N"], a["nodes"], a["V"], a["top"],
                                      a["acc"], a["path"], a["nxt"], None) == want


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(kc=None), EINVAL), (dict(acc=None), EINVAL), (dict(R=0), EINVAL), (dict(D=72), EUNSUPPORTED), (dict(ps=20), EINVAL),
    (dict(mapped=4 * P, new=4 * P), EINVAL), (dict(mapped=4 * P, new=4 * P - 4), EINVAL), (dict(new=P), EINVAL),
])
def test_kv_commit_ex_rejects(kw, want):
    a = dict(kc=P, vc=P, kl=0, vl=0, L=1, ct=0, table=P, ctx=P, mapped=2 * P, path=P, acc=P, R=2, nodes=8, Hk=2, D=64, ps=16,
             mp=4, np_=9, new=3 * P)
    a.update(kw)
    assert D.lib().dspark_kv_commit_ex(a["kc"], a["vc"], a["kl"], a["vl"], a["L"], a["ct"], a["table"], a["ctx"], a["mapped"],
                                       a["path"], a["acc"], a["R"], a["nodes"], a["Hk"], a["D"], a["ps"], a["mp"], a["np_"],
                                       a["new"], None) == want
    assert D.lib().dspark_last_error() != b""


@no_gpu
@pytest.mark.parametrize("kl,vl,layers,want", [
    # a layer is 9 * 2 * 64 * 16 = 18432 elements; new_len on ctx_len is the next refusal either way
    (0, 18432, 2, b"overlap"), (18432, 0, 2, b"overlap"), (18424, 18432, 3, b"overlap"), (-18424, 18432, 3, b"overlap"),
    (8, 8, 2, b"overlap"), (18432, 18432, 3, b"new_len"), (-18432, 18440, 3, b"new_len"), (0, 0, 1, b"new_len"),
])
def test_kv_commit_refuses_layers_on_each_other(kl, vl, layers, want):
    assert D.lib().dspark_kv_commit(P, P, kl, vl, layers, 0, P, P, P, P, 2, 8, 2, 64, 16, 4, 9, P, None) == EINVAL
    assert want in D.lib().dspark_last_error()


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(q=None), EINVAL), (dict(out=None), EINVAL), (dict(R=0), EINVAL), (dict(Hq=9), EINVAL), (dict(D=48, qs=512), EUNSUPPORTED),
    (dict(scale=float("nan")), EINVAL), (dict(ws=None), EWORKSPACE),
])
def test_tree_attention_ex_rejects(kw, want):
    a = dict(q=P, qs=512, out=2 * P, R=2, N=4, Hq=8, Hk=2, D=64, scale=0.125, ws=P)
    a.update(kw)
    assert D.lib().dspark_tree_attention_ex(a["q"], a["qs"], 0, P, P, 0, None, None, P, P, 3 * P, P, None, 0, a["R"], a["N"],
                                            a["Hq"], a["Hk"], a["D"], 16, 4, 9, a["scale"], a["out"], 512, None, a["ws"],
                                            1 << 40, None) == want
    assert D.lib().dspark_last_error() != b""


@no_gpu
@pytest.mark.parametrize("q,qs,out,os_,n,meet", [
    # rows of 512 elements, offsets in elements; EWORKSPACE is the next refusal
    (0, 512, 0, 512, 4, False), (0, 1040, 0, 1040, 4, False), (0, 512, 0, 1040, 1, False),       # q itself
    (0, 512, 0, 1040, 4, True), (0, 1040, 0, 512, 2, True),                                       # with another stride
    (0, 512, 512, 512, 4, True), (512, 512, 0, 512, 4, True), (0, 512, 8, 512, 1, True), (8, 512, 0, 512, 1, True),
    (0, 512, 2048, 512, 4, False), (2048, 512, 0, 512, 4, False), (0, 512, 2040, 512, 4, True), (0, 512, 512, 512, 1, False),
    (0, 1040, 512, 1040, 4, False), (512, 1040, 0, 1040, 4, False),                               # side by side in wider rows
    (0, 1536, 512, 1536, 4, False), (0, 1536, 1024, 1536, 4, False), (0, 1040, 504, 1040, 4, True), (0, 1040, 536, 1040, 4, True),
    (0, 1040, 536, 1040, 1, False), (536, 1040, 0, 1040, 4, True), (504, 1040, 0, 1040, 4, True),
    (0, 1040, 4 * 1040 - 8, 1040, 4, False), (0, 1040, 3 * 1040 + 504, 1040, 4, True), (0, 1040, 3 * 1040 + 512, 1040, 4, False),
    (0, 1040, 3 * 1040, 1040, 4, True), (0, 1040, -3 * 1040, 1040, 4, True), (0, 1040, -4 * 1040 + 536, 1040, 4, True),
    (0, 1040, -4 * 1040 + 512, 1040, 4, False), (0, 512, 4096, 1040, 4, False),
])
def test_tree_attention_refuses_outputs_on_parts_of_the_queries(q, qs, out, os_, n, meet):
    base = 16 * P
    st = D.lib().dspark_tree_attention(base + 2 * q, qs, 0, P, P, 0, None, None, P, P, P, None, 0, 2, n, 8, 2, 64, 16, 4, 9, 0.125,
                                       base + 2 * out, os_, None, None, 0, None)
    assert st == (EINVAL if meet else EWORKSPACE)
    # the definition: byte by byte over the rows
    if not (q == out and (qs == os_ or n == 1)) and qs == os_:
        a = set(x for i in range(n) for x in range(q + i * qs, q + i * qs + 512, 8))
        b = set(x for i in range(n) for x in range(out + i * os_, out + i * os_ + 512, 8))
        assert meet == bool(a & b)


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(z=None), EINVAL), (dict(R=0), EINVAL), (dict(V=0), EINVAL), (dict(ctx=None), EINVAL), (dict(mapped=None), EINVAL),
])
def test_verify_tree_ex_rejects(kw, want):
    a = dict(z=P, ctx=P, mapped=P, R=2, V=100)
    a.update(kw)
    assert D.lib().dspark_verify_tree_ex(a["z"], P, P, P, a["ctx"], a["mapped"], a["R"], 8, 4, a["V"], P, P, P, P, None) == want
    assert D.lib().dspark_last_error() != b""


# ---- refusals of the binding: nothing that is not on a device is taken ----

def test_binding_refuses_host_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    t = torch.zeros((4, 2), dtype=torch.int32)
    kc, vc = torch.zeros((3, 2, 8, 16, 8), dtype=torch.bfloat16), torch.zeros((3, 2, 64, 16), dtype=torch.bfloat16)
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    cu = torch.zeros(5, dtype=torch.int32)
    for f in (lambda: D.dspark_page_map(i, cu, t, i, i, 16, 4), lambda: D.dspark_page_trim(i, i, t, i, i, 16),
              lambda: D.dspark_kv_store(x, x, torch.zeros(4, dtype=torch.int64), kc, vc),
              lambda: D.dspark_kv_commit(kc, vc, t, i, t, i), lambda: D.dspark_tree_attention(x, kc, vc, t, i, cu),
              lambda: D.dspark_tree_pack(i, cu, 1), lambda: D.dspark_verify_tree(torch.zeros((4, 9)), cu, i, i, 4)):
        with pytest.raises(ValueError, match="device"):
            f()


def test_every_name_of_the_package_can_be_had_without_pytorch():
    code = ("import sys\n"
            "sys.modules['torch'] = None\n"
            "from draft_head_step_amd import *\n"
            "import draft_head_step_amd as D\n"
            "assert all(hasattr(D, n) for n in D.__all__)\n"
            "assert dspark_page_map.__name__ == 'dspark_page_map'\n"
            "try:\n"
            "    dspark_page_map()\n"
            "except ImportError:\n"
            "    print('raised')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "raised", r.stderr


# ---- pins of the oracle ----

def test_oracle_attention_equals_a_softmax():
    rng = np.random.default_rng(0)
    P_, Hk, Hq, Dh = 16, 2, 4, 64
    n, ctx = [3, 2], np.array([20, 0])
    cu = np.array([0, 3, 5])
    kc, vc = rng.normal(size=(6, Hk, Dh // 8, P_, 8)), rng.normal(size=(6, Hk, Dh, P_))
    table = np.array([[4, 1], [3, 0]])
    q = rng.normal(size=(5, Hq, Dh))
    out, lse, W, A, M = O.tree_attention(q, kc, vc, table, ctx, cu, P_, 0.3)
    # element 1 of request 0, head 3: positions 0 .. 21
    k = np.array([[kc[table[0, t // 16], 1, d // 8, t % 16, d % 8] for d in range(Dh)] for t in range(22)])
    v = np.array([[vc[table[0, t // 16], 1, d, t % 16] for d in range(Dh)] for t in range(22)])
    s = 0.3 * (k @ q[1, 3])
    p = np.exp(s) / np.exp(s).sum()
    assert np.allclose(out[1, 3], p @ v, rtol=1e-12) and np.isclose(lse[1, 3], np.log(np.exp(s).sum()))
    assert np.allclose(W[1, 3], p @ np.abs(v)) and np.isclose(M[1, 3], np.abs(s).max())
    # the first element of a request without context sees itself alone
    assert np.allclose(out[3, 0], vc[3, 0, :, 0])
    # a chain's mask gives what no mask gives
    mask = np.array([[1], [3], [7], [1], [3]], np.uint32)
    assert np.allclose(O.tree_attention(q, kc, vc, table, ctx, cu, P_, 0.3, mask)[0], out)


def test_oracle_pages_by_hand():
    table = np.full((2, 3), -1, np.int32)
    table[0, 0] = 5
    ring = np.array([7, 8, -1, -1, -1, -1, 2, 3, 4], np.int32)
    t, s, new, pool = O.page_map(np.array([14, 0]), np.array([0, 4, 7]), table, ring, np.array([6, 5, 0, 0]), 16, 7,
                                 np.full(7, -9))
    assert s.tolist() == [5 * 16 + 14, 5 * 16 + 15, 2 * 16, 2 * 16 + 1, 48, 49, 50]
    assert new.tolist() == [18, 3] and pool.tolist() == [8, 3, 0, 0] and t.tolist() == [[5, 2, -1], [3, -1, -1]]
    r, pool = O.page_trim(new, np.array([16, 0]), t, ring, pool, 16)
    assert pool.tolist() == [8, 5, 0, 0] and r[[2, 3]].tolist() == [2, 3]


def test_oracle_trees_by_hand():
    par = np.array([-1, 0, 0, 1, 5, 1], np.int32)
    m, d = O.ancestors(par)
    assert d.tolist() == [0, 1, 1, 2, -1, 2] and m[3].tolist() == [True, True, False, True, False, False] and not m[4].any()
    logits = np.zeros((6, 9), np.float32)
    logits[0, 4] = logits[1, 7] = logits[5, 2] = 1
    acc, path, nxt, top = O.verify_tree(logits, np.array([0, 6]), np.array([0, 4, 4, 1, 7, 7]), par, 4)
    assert acc.tolist() == [1] and path.tolist() == [[0, 1, -1, -1]] and nxt.tolist() == [7]
    acc, path, nxt, top = O.verify_tree(logits, np.array([0, 6]), np.array([0, 4, 4, 1, 7, 7]), par, 6)
    assert acc.tolist() == [2] and path[0, :3].tolist() == [0, 1, 5] and nxt.tolist() == [2]


def test_oracle_of_a_short_pool():
    # 15 and 14 tokens, one free page that both rows still name: the second request is turned
    # down, and its path must not move into the page that the first was given
    table = np.array([[0, 2, -1], [1, 2, -1]], np.int32)
    cur, cu = np.array([15, 14]), np.array([0, 3, 8])
    t, s, new, pool = O.page_map(cur, cu, table, np.array([2, -1, -1]), np.array([0, 1, 0, 0]), 16, 8, np.full(8, -9))
    assert new.tolist() == [18, 14] and pool.tolist() == [1, 0, 1, 0] and s.tolist() == [15, 32, 33, -1, -1, -1, -1, -1]
    k, v = np.arange(3 * 16.0).reshape(1, 3, 1, 1, 16, 1), np.arange(3 * 16.0).reshape(1, 3, 1, 1, 16)
    path, acc = np.array([[0, 2, -1], [0, 2, 4]]), np.array([1, 2])
    _, v2, kept = O.kv_commit(k, v, t, cur, path, acc, 16)
    assert kept.tolist() == [17, 17] and v2[0, 2, 0, 0, 0] != v[0, 2, 0, 0, 1]
    _, v2, kept = O.kv_commit(k, v, t, cur, path, acc, 16, new)
    assert kept.tolist() == [17, 14] and v2[0, 2, 0, 0, 0] == v[0, 2, 0, 0, 1]
    assert (v2 != v).sum() == 1
