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
