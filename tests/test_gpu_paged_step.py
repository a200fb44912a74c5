"""The paged-cache operators together, as a target engine runs them: pages, cache
writes, attention, acceptance, commit, trim, over several steps; the same in a
replayed HIP graph, on another stream, and with two calls at once."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.dirname(__file__))
import draft_head_step_amd as D  # noqa: E402
import paged_helpers as H  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HQ, HK, DH, P, V = 8, 2, 64, 16, 211


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


class Toy:
    """A one-layer target: token embeddings to q, k, v (positions added), attention,
    logits.  Everything is a fixed table, so a token's row depends only on what it
    attends to."""

    def __init__(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.eq = torch.randn((V, HQ, DH), generator=g, device=DEV)
        self.ek = torch.randn((V, HK, DH), generator=g, device=DEV)
        self.ev = torch.randn((V, HK, DH), generator=g, device=DEV)
        self.pos = torch.randn((4096, DH), generator=g, device=DEV) * 0.3
        self.head = torch.randn((HQ * DH, V), generator=g, device=DEV)

    def qkv(self, tok, pos):
        p = self.pos[pos.long()][:, None]
        t = tok.long()
        return ((self.eq[t] + p).to(torch.bfloat16), (self.ek[t] + p).to(torch.bfloat16), self.ev[t].to(torch.bfloat16))

    def logits(self, x):
        return x.float().reshape(x.shape[0], -1) @ self.head


def dense_logits(toy, seq):
    """Logits after each token of `seq` by plain causal attention in fp64."""
    tok = dev(np.asarray(seq, np.int32))
    pos = torch.arange(len(seq), device=DEV)
    q, k, v = (x.double() for x in toy.qkv(tok, pos))
    out = torch.zeros((len(seq), HQ, DH), dtype=torch.float64, device=DEV)
    for y in range(HQ):
        h = y // (HQ // HK)
        s = (q[:, y] @ k[:, h].T.contiguous()) * DH ** -0.5
        s = s.masked_fill(~torch.ones_like(s, dtype=torch.bool).tril(), -torch.inf)
        out[:, y] = torch.softmax(s, 1) @ v[:, h]
    return out.reshape(len(seq), -1) @ toy.head.double()


def test_decoding_with_trees_equals_decoding_one_by_one():
    # Greedy decoding through drafted trees gives the sequence that plain greedy decoding
    # gives: every emitted token is the dense model's, up to ties within the tolerance.
    print("case paged step decode", flush=True)
    toy, rng = Toy(1), np.random.default_rng(1)
    R, pages, width = 5, 120, 14
    seqs = [list(rng.integers(0, V, int(x))) for x in (1, 7, 16, 33, 50)]
    kc = torch.full((pages, HK, DH // 8, P, 8), float("nan"), dtype=torch.bfloat16, device=DEV)
    vc = torch.full((pages, HK, DH, P), float("nan"), dtype=torch.bfloat16, device=DEV)
    table = torch.full((R, width), -1, dtype=torch.int32, device=DEV)
    ring = dev(rng.permutation(pages).astype(np.int32))
    pool = dev(np.array([0, pages, 0, 0], np.int32))
    ctx = dev(np.zeros(R, np.int32))
    drafted = accepted_total = 0
    # A logit sums 512 outputs times unit normals; an output is off by at most 2 * 2^-9 W (its own
    # rounding and that of the probabilities), W = sum p |v| < 1.5: a standard deviation below
    # sqrt(512) * 2^-8 * 1.5 = 0.13.  Five of them on the difference of two logits.
    margin = 1.0
    for step in range(7):
        # the anchor is the last token of each sequence; the first step brings whole prompts
        n, par, tok = [], [], []
        for r in range(R):
            if step == 0:
                t = np.array(seqs[r], np.int32)
                p = np.arange(-1, len(t) - 1)
            else:
                k = int(rng.integers(1, 12))
                p = H.random_parents(rng, k)
                t = rng.integers(0, V, k).astype(np.int32)
                t[0] = seqs[r][-1]
                # plant the dense model's own continuation along a random path
                full = list(seqs[r])
                at = 0
                while rng.random() < 0.8:
                    kids = [i for i in range(at + 1, k) if p[i] == at]
                    if not kids:
                        break
                    c = int(rng.choice(kids))
                    t[c] = int(dense_logits(toy, full)[-1].argmax())
                    full.append(int(t[c]))
                    at = c
            n.append(len(t))
            par.append(p)
            tok.append(t)
        drafted += sum(n) - R
        cu = H.starts(n)
        N = int(cu[-1])
        dcu, dpar, dtok = dev(cu), dev(np.concatenate(par).astype(np.int32)), dev(np.concatenate(tok).astype(np.int32))
        words = -(-max(n) // 32)
        mask, pos = D.dspark_tree_pack(dpar, dcu, words, ctx)
        slots, new_len, pool2 = D.dspark_page_map(ctx, dcu, table, ring, pool, P, N)
        q, k, v = toy.qkv(dtok, pos)
        D.dspark_kv_store(k, v, slots, kc, vc, count=dcu[R:])
        out, _ = D.dspark_tree_attention(q, kc, vc, table, ctx, dcu, tree_mask=mask)
        logits = toy.logits(out)
        if step == 0:
            # prompts: the last logits give the first token; every token is kept
            last = logits[dcu[1:].long() - 1].argmax(1).int()
            lens = new_len
            pool = pool2
            nxt = last
        else:
            acc, path, nxt, top = D.dspark_verify_tree(logits, dcu, dtok, dpar, max(n))
            lens = D.dspark_kv_commit(kc, vc, table, ctx, path, acc)
            pool = D.dspark_page_trim(new_len, lens, table, ring, pool2, P)
            a, pa = acc.cpu().numpy(), path.cpu().numpy()
            accepted_total += int(a.sum())
            for r in range(R):
                seqs[r] += [int(tok[r][pa[r, i]]) for i in range(1, a[r] + 1)]
        torch.cuda.synchronize()
        assert pool.cpu().numpy()[2] == 0
        for r in range(R):
            d = dense_logits(toy, seqs[r])[-1]
            x = int(nxt[r])
            assert float(d.max() - d[x]) <= margin, f"step {step} request {r}"
            seqs[r].append(x)
        ctx = lens
        assert ctx.cpu().numpy().tolist() == [len(s) - 1 for s in seqs]
        held = sum(-(-(len(s) - 1) // P) for s in seqs)
        assert int(pool[1]) == pages - held
    assert accepted_total >= 20, (accepted_total, drafted)


def _step_state(seed, R=6, n=7, ctx_top=300):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, ctx_top, R).astype(np.int32)
    ns = np.full(R, n)
    cu = H.starts(ns)
    N = int(cu[-1])
    pages = int(sum(-(-int(c + n) // P) for c in ctx)) + 4
    held = H.tables(rng, ctx, P, pages, -(-int(ctx_top + n) // P) + 1)
    used = set(int(held[r, i]) for r in range(R) for i in range(-(-int(ctx[r]) // P)))
    ring = np.full(pages, -1, np.int32)
    free = [p for p in range(pages) if p not in used]
    ring[:len(free)] = free
    kc, vc = H.caches(rng, pages, HK, DH, P, "bf16", DEV)
    g = torch.Generator(device=DEV).manual_seed(seed)
    f = lambda *s: torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    return dict(ctx=dev(ctx), cu=dev(cu), table=dev(held), ring=dev(ring), pool=dev(np.array([0, len(free), 0, 0], np.int32)),
                kc=kc, vc=vc, q=f(N, HQ, DH), k=f(N, HK, DH), v=f(N, HK, DH), logits=torch.randn((N, V), generator=g, device=DEV),
                tok=dev(rng.integers(0, V, N).astype(np.int32)),
                par=dev(np.concatenate([H.random_parents(rng, n) for _ in range(R)]).astype(np.int32)), N=N, R=R, n=n)


def _step(s, o, stream=None):
    D.dspark_tree_pack(s["par"], s["cu"], 1, s["ctx"], mask=o["mask"], flat_pos=o["pos"], stream=stream)
    D.dspark_page_map(s["ctx"], s["cu"], s["table"], s["ring"], s["pool"], P, slots=o["slots"], new_len=o["new"],
                      pool_out=o["pool1"], stream=stream)
    D.dspark_kv_store(s["k"], s["v"], o["slots"], s["kc"], s["vc"], count=s["cu"][s["R"]:], stream=stream)
    D.dspark_tree_attention(s["q"], s["kc"], s["vc"], s["table"], s["ctx"], s["cu"], tree_mask=o["mask"], out=o["out"],
                            lse=o["lse"], workspace=o["ws"], stream=stream)
    D.dspark_verify_tree(s["logits"], s["cu"], s["tok"], s["par"], s["n"], target_argmax=o["top"], accepted=o["acc"],
                         path=o["path"], next_token=o["nxt"], stream=stream)
    D.dspark_page_trim(o["new"], s["ctx"], s["table"], s["ring"], o["pool1"], P, pool_out=o["pool2"], stream=stream)


def _outs(s):
    N, R, i32 = s["N"], s["R"], torch.int32
    e = lambda *sh, t=i32: torch.empty(sh, dtype=t, device=DEV)  # noqa: E731
    return dict(mask=e(N, 1), pos=e(N), slots=e(N, t=torch.int64), new=e(R), pool1=e(4), pool2=e(4),
                out=e(N, HQ, DH, t=torch.bfloat16), lse=e(N, HQ, t=torch.float32), top=e(N), acc=e(R), path=e(R, s["n"]), nxt=e(R),
                ws=e(D.dspark_tree_attention_workspace(R, N, HQ, HK, DH), t=torch.uint8))


def _same(a, b):
    for k in a:
        if k != "ws":
            assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k


def test_step_replays_in_a_graph():
    print("case paged step graph", flush=True)
    s = _step_state(3)
    ref, o = _outs(s), _outs(s)
    _step(s, ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(s, o)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    _same(o, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(s, o)
    for rep in range(3):
        for t in o.values():
            t.view(torch.uint8).fill_(0xA5 + rep)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        _same(o, ref)
    # new values in the same buffers: the replay follows them
    new = _step_state(4)
    for k in s:
        if torch.is_tensor(s[k]) and s[k].shape == new[k].shape and k not in ("kc", "vc", "table", "ring", "pool", "ctx"):
            s[k].copy_(new[k])
    graph.replay()
    again = _outs(s)
    torch.cuda.synchronize()
    got = {k: t.clone() for k, t in o.items()}
    _step(s, again)
    torch.cuda.synchronize()
    _same(got, again)


def test_two_graphs_share_a_workspace():
    # graphs replayed one after the other on one stream may share one workspace
    print("case paged two graphs", flush=True)
    a, b = _step_state(5), _step_state(6, R=9, n=3, ctx_top=3000)
    oa, ob = _outs(a), _outs(b)
    ws = torch.empty(max(oa["ws"].numel(), ob["ws"].numel()), dtype=torch.uint8, device=DEV)
    oa["ws"] = ob["ws"] = ws
    ra, rb = _outs(a), _outs(b)
    _step(a, ra)
    _step(b, rb)
    torch.cuda.synchronize()
    graphs = []
    for s, o in ((a, oa), (b, ob)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _step(s, o)
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
        ws.fill_(0xff)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        _same(oa, ra)
        _same(ob, rb)


def test_two_calls_at_once_on_two_streams():
    print("case paged two streams", flush=True)
    a, b = _step_state(7, R=20, ctx_top=2000), _step_state(8, R=20, ctx_top=2000)
    ra, rb = _outs(a), _outs(b)
    _step(a, ra)
    _step(b, rb)
    torch.cuda.synchronize()
    oa, ob = _outs(a), _outs(b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        _step(a, oa, stream=s1)
        _step(b, ob, stream=s2)
    torch.cuda.synchronize()
    _same(oa, ra)
    _same(ob, rb)


def test_allocations_of_a_call_belong_to_its_stream():
    # outputs that the binding allocates are safe on the given stream
    print("case paged stream allocations", flush=True)
    s = _step_state(9)
    ref = D.dspark_tree_attention(s["q"], s["kc"], s["vc"], s["table"], s["ctx"] * 0, s["cu"])[0]
    side = torch.cuda.Stream()
    zero = s["ctx"] * 0
    torch.cuda.synchronize()
    out = D.dspark_tree_attention(s["q"], s["kc"], s["vc"], s["table"], zero, s["cu"], stream=side)[0]
    side.synchronize()
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16))


class _Spy:
    """The library, with the arguments of every call kept."""

    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        f = getattr(self.lib, name)

        def call(*args):
            self.calls.append((name, args))
            return f(*args)
        return call


def _stream_of(address):
    """The stream that the allocator's block at an address belongs to."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= address < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("no block at that address")


def test_memory_of_a_call_is_the_streams_own(monkeypatch):
    # A workspace is released when the call returns: only a block of the call's own stream is
    # safe from other streams' work then.  Outputs that the binding makes are such blocks too.
    print("case paged stream ownership", flush=True)
    s = _step_state(11)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    spy = _Spy(D.lib())
    monkeypatch.setattr(D, "_LIB", spy)
    for stream in (side, None):
        want = side.cuda_stream if stream is side else torch.cuda.current_stream().cuda_stream
        spy.calls.clear()
        made = []
        slots, new, pool = D.dspark_page_map(s["ctx"], s["cu"], s["table"], s["ring"], s["pool"], P, s["N"], stream=stream)
        made += [slots, new, pool]
        made += D.dspark_tree_pack(s["par"], s["cu"], 1, s["ctx"], want_req=True, stream=stream)
        made += D.dspark_tree_attention(s["q"], s["kc"], s["vc"], s["table"], s["ctx"], s["cu"], tree_mask=made[3], mapped_len=new,
                                        want_lse=True, stream=stream)
        acc, path, nxt, top = D.dspark_verify_tree(s["logits"], s["cu"], s["tok"], s["par"], s["n"], ctx_len=s["ctx"], mapped_len=new,
                                                   stream=stream)
        made += [acc, path, nxt, top]
        kc, vc = s["kc"].clone(), s["vc"].clone()
        torch.cuda.synchronize()
        kept = D.dspark_kv_commit(kc, vc, s["table"], s["ctx"], path, acc, mapped_len=new, stream=stream)
        made += [kept, D.dspark_page_trim(new, s["ctx"], s["table"], s["ring"].clone(), pool, P, stream=stream)]
        torch.cuda.synchronize()
        assert [_stream_of(t.data_ptr()) for t in made] == [want] * 14
        (ws,) = [a[-3] for n, a in spy.calls if n == "dspark_tree_attention_ex"]
        assert _stream_of(ws) == want
        assert all(a[-1] == want for n, a in spy.calls if n != "dspark_tree_attention_workspace")
