"""Verification over a paged key/value cache: binding of the page, cache, tree and
attention entry points of include/dspark.h (same names as the C ABI).

Like the rest of the binding it only marshals arguments: dtypes, devices and
shapes are checked here, outputs and workspaces are allocated with PyTorch on
the calling stream, and every step runs in the library's HIP kernels.  A call
runs on its tensors' device, whichever device is current.
"""
from __future__ import annotations

import math

import torch

import draft_head_step_amd as _D

_I32 = torch.int32
_F32 = torch.float32
_CACHE = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2}


def _gpu(t, name):
    """Index of the device that a tensor is on."""
    i = t.get_device()
    if i < 0:
        raise ValueError(f"{name} must be a device tensor, got {t.device}")
    return i


def _arr(t, name, dtype, shape, device):
    """A dense tensor of that dtype, shape and device (index)."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on device {device}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _rows(t, name, dtypes, shape, device):
    """[N, H, D] rows: dense heads, any row stride, which is returned."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {tuple(dtypes)}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on device {device}, got {t.device}")
    n, h, d = t.stride()
    if (d != 1 and shape[2] > 1) or (h != shape[2] and shape[1] > 1):
        raise ValueError(f"{name} must have dense rows of [heads, D]")
    # a single row has no row stride of its own
    return n if shape[0] > 1 else shape[1] * shape[2]


class _Call:
    """The stream a call enqueues on, with the device of its tensors (an index) current
    meanwhile and its own allocations on that stream."""

    __slots__ = ("stream", "device", "contexts")

    def __init__(self, device, stream):
        self.stream = stream
        self.device = device
        self.contexts = ()

    def __enter__(self):
        i, s = self.device, self.stream
        if s is None and i == torch._C._cuda_getDevice():
            return torch._C._cuda_getCurrentRawStream(i)
        if s is not None and s.device.index != i:
            raise ValueError(f"the stream belongs to {s.device}, the tensors are on device {i}")
        self.contexts = (torch.cuda.device(i),) if s is None else (torch.cuda.device(i), torch.cuda.stream(s))
        for c in self.contexts:
            c.__enter__()
        return torch._C._cuda_getCurrentRawStream(i)

    def __exit__(self, *exc):
        for c in reversed(self.contexts):
            c.__exit__(*exc)
        return False


def _pool(t, name, device):
    _arr(t, name, _I32, (4,), device)


def dspark_page_map(cur_len, cu_seqlens, block_table, ring, pool, page_size, max_tokens=None, *,
                    slots=None, new_len=None, pool_out=None, stream=None):
    """Pages and slots for the new elements of every request.

    cur_len [R], cu_seqlens [R + 1], block_table [R, max_pages] (updated), ring
    [num_pages] and pool [4] = (head, count, refused, 0) are int32 device tensors.
    ``max_tokens`` is the room for elements (slots' length; needed if slots is not
    given).  Returns (slots [max_tokens] int64, new_len [R], pool_out [4]); slots
    beyond cu_seqlens[R] are not written."""
    dev = _gpu(cur_len, "cur_len")
    R, = cur_len.shape
    if block_table.dim() != 2:
        raise ValueError("block_table must be [R, max_pages]")
    mp = block_table.shape[1]
    _arr(cur_len, "cur_len", _I32, (R,), dev)
    _arr(cu_seqlens, "cu_seqlens", _I32, (R + 1,), dev)
    _arr(block_table, "block_table", _I32, (R, mp), dev)
    _arr(ring, "ring", _I32, (ring.numel(),), dev)
    _pool(pool, "pool", dev)
    if slots is not None:
        max_tokens = slots.numel()
    elif max_tokens is None:
        raise ValueError("max_tokens or slots must be given")
    with _Call(dev, stream) as s:
        if slots is None:
            slots = cur_len.new_empty((max_tokens,), dtype=torch.int64)
        if new_len is None:
            new_len = cur_len.new_empty((R,), dtype=_I32)
        if pool_out is None:
            pool_out = cur_len.new_empty((4,), dtype=_I32)
        _arr(slots, "slots", torch.int64, (max_tokens,), dev)
        _arr(new_len, "new_len", _I32, (R,), dev)
        _pool(pool_out, "pool_out", dev)
        st = (_D._LIB or _D.lib()).dspark_page_map(
            cur_len.data_ptr(), cu_seqlens.data_ptr(), R, max_tokens, page_size, mp, ring.numel(),
            block_table.data_ptr(), ring.data_ptr(), pool.data_ptr(), pool_out.data_ptr(),
            slots.data_ptr(), new_len.data_ptr(), s)
    if st:
        _D._check(st, "dspark_page_map")
    return slots, new_len, pool_out


def dspark_page_trim(cur_len, keep_len, block_table, ring, pool, page_size, *, pool_out=None,
                     stream=None):
    """The pages behind keep_len [R] of cur_len [R] tokens back to the ring (updated).
    Returns pool_out [4]."""
    dev = _gpu(cur_len, "cur_len")
    R, = cur_len.shape
    if block_table.dim() != 2:
        raise ValueError("block_table must be [R, max_pages]")
    mp = block_table.shape[1]
    _arr(cur_len, "cur_len", _I32, (R,), dev)
    _arr(keep_len, "keep_len", _I32, (R,), dev)
    _arr(block_table, "block_table", _I32, (R, mp), dev)
    _arr(ring, "ring", _I32, (ring.numel(),), dev)
    _pool(pool, "pool", dev)
    with _Call(dev, stream) as s:
        if pool_out is None:
            pool_out = cur_len.new_empty((4,), dtype=_I32)
        _pool(pool_out, "pool_out", dev)
        st = (_D._LIB or _D.lib()).dspark_page_trim(
            cur_len.data_ptr(), keep_len.data_ptr(), R, page_size, mp, ring.numel(),
            block_table.data_ptr(), ring.data_ptr(), pool.data_ptr(), pool_out.data_ptr(), s)
    if st:
        _D._check(st, "dspark_page_trim")
    return pool_out


def _cache_shape(k_cache, v_cache, lead=0):
    """(num_pages, Hk, D, P) of a pair of caches (behind `lead` leading dimensions)."""
    if k_cache.dtype not in _CACHE or v_cache.dtype != k_cache.dtype:
        raise TypeError("k_cache and v_cache must both be bfloat16, float16 or float8_e4m3fn")
    if k_cache.dim() != 5 + lead or v_cache.dim() != 4 + lead:
        raise ValueError("k_cache must be [pages, Hk, D / c, P, c] and v_cache [pages, Hk, D, P]")
    n, hk, d, p = v_cache.shape[lead:]
    c = 16 // k_cache.element_size()
    if k_cache.shape[lead:] != (n, hk, d // c, p, c) or k_cache.shape[:lead] != v_cache.shape[:lead]:
        raise ValueError(f"k_cache must be {(n, hk, d // c, p, c)} for v_cache {(n, hk, d, p)}, got "
                         f"{tuple(k_cache.shape)}")
    if v_cache.get_device() != k_cache.get_device():
        raise ValueError("k_cache and v_cache must be on one device")
    return n, hk, d, p


def _dense(t, name):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _scales(k_cache, k_scale, v_scale, hk, dev):
    if (k_scale is None) != (v_scale is None):
        raise ValueError("k_scale and v_scale go together")
    if k_scale is None:
        return 0, 0
    _arr(k_scale, "k_scale", _F32, (hk,), dev)
    _arr(v_scale, "v_scale", _F32, (hk,), dev)
    return k_scale.data_ptr(), v_scale.data_ptr()


def dspark_kv_store(k, v, slots, k_cache, v_cache, *, count=None, k_scale=None, v_scale=None,
                    stream=None):
    """Keys and values [N, Hk, D] (bfloat16 or float16, dense heads, any row stride)
    into slots [N] of the caches (updated).  ``count`` [1] int32 (for example
    cu_seqlens[R:]) limits the elements to those that the device knows of."""
    dev = _gpu(k, "k")
    n, hk, d, p = _cache_shape(k_cache, v_cache)
    _dense(k_cache, "k_cache")
    _dense(v_cache, "v_cache")
    if k_cache.get_device() != dev:
        raise ValueError(f"the caches must be on device {dev}, got {k_cache.device}")
    N = slots.numel()
    ks = _rows(k, "k", (torch.bfloat16, torch.float16), (N, hk, d), dev)
    vs = _rows(v, "v", (k.dtype,), (N, hk, d), dev)
    _arr(slots, "slots", torch.int64, (N,), dev)
    if count is not None:
        _arr(count, "count", _I32, (1,), dev)
    sk, sv = _scales(k_cache, k_scale, v_scale, hk, dev)
    with _Call(dev, stream) as s:
        st = (_D._LIB or _D.lib()).dspark_kv_store(
            k.data_ptr(), v.data_ptr(), ks, vs, _CACHE[k.dtype], slots.data_ptr(),
            0 if count is None else count.data_ptr(), N, hk, d, p, n, _CACHE[k_cache.dtype], sk,
            sv, k_cache.data_ptr(), v_cache.data_ptr(), s)
    if st:
        _D._check(st, "dspark_kv_store")


def dspark_kv_commit(k_cache, v_cache, block_table, ctx_len, path, accepted, *, mapped_len=None,
                     new_len=None, stream=None):
    """The accepted paths' keys and values to the front, in place.

    The caches are [pages, ...] or [layers, pages, ...] (layers may be strided);
    path [R, max_nodes] and accepted [R] as dspark_verify_tree returns them.
    ``mapped_len`` [R] is new_len of dspark_page_map, needed wherever that call can
    turn a request down: no position from there on is touched.  Returns new_len [R]
    = ctx_len + 1 + accepted; a request whose path is refused moves nothing and
    gets ctx_len with mapped_len, -1 without."""
    dev = _gpu(k_cache, "k_cache")
    lead = v_cache.dim() - 4
    if lead not in (0, 1):
        raise ValueError("the caches must be [pages, ...] or [layers, pages, ...]")
    n, hk, d, p = _cache_shape(k_cache, v_cache, lead)
    layers = v_cache.shape[0] if lead else 1
    if layers == 0:
        raise ValueError("the caches must have a layer")
    _dense(k_cache[0] if lead else k_cache, "k_cache (each layer)")
    _dense(v_cache[0] if lead else v_cache, "v_cache (each layer)")
    # layers that share memory would race
    kl, vl = (k_cache.stride(0), v_cache.stride(0)) if layers > 1 else (0, 0)
    if layers > 1 and (abs(kl) < n * hk * d * p or abs(vl) < n * hk * d * p):
        raise ValueError("the layers of a cache may not overlap")
    R, = ctx_len.shape
    if block_table.dim() != 2 or path.dim() != 2:
        raise ValueError("block_table must be [R, max_pages] and path [R, max_nodes]")
    mp, nodes = block_table.shape[1], path.shape[1]
    _arr(block_table, "block_table", _I32, (R, mp), dev)
    _arr(ctx_len, "ctx_len", _I32, (R,), dev)
    _arr(path, "path", _I32, (R, nodes), dev)
    _arr(accepted, "accepted", _I32, (R,), dev)
    if mapped_len is not None:
        _arr(mapped_len, "mapped_len", _I32, (R,), dev)
    with _Call(dev, stream) as s:
        if new_len is None:
            new_len = ctx_len.new_empty((R,), dtype=_I32)
        _arr(new_len, "new_len", _I32, (R,), dev)
        st = (_D._LIB or _D.lib()).dspark_kv_commit_ex(
            k_cache.data_ptr(), v_cache.data_ptr(), kl, vl, layers, _CACHE[k_cache.dtype],
            block_table.data_ptr(), ctx_len.data_ptr(),
            0 if mapped_len is None else mapped_len.data_ptr(), path.data_ptr(),
            accepted.data_ptr(), R, nodes, hk, d, p, mp, n, new_len.data_ptr(), s)
    if st:
        _D._check(st, "dspark_kv_commit")
    return new_len


def dspark_tree_attention_workspace(R: int, max_tokens: int, Hq: int, Hk: int, D: int) -> int:
    return int((_D._LIB or _D.lib()).dspark_tree_attention_workspace(R, max_tokens, Hq, Hk, D))


def dspark_tree_attention(q, k_cache, v_cache, block_table, ctx_len, cu_seqlens, scale=None, *,
                          tree_mask=None, mapped_len=None, k_scale=None, v_scale=None, out=None,
                          lse=None, want_lse=False, workspace=None, stream=None):
    """Attention of q [N, Hq, D] (bfloat16 or float16, dense heads, any row stride) over
    each request's cached context and its own segment: causal, or by tree_mask
    [N, words] int32 / uint32.  ``scale`` is 1 / sqrt(D) by default.  ``mapped_len``
    [R] is new_len of dspark_page_map: rows of a request that it turned down are NaN.
    Returns (out [N, Hq, D], lse [N, Hq] fp32 or None); rows beyond cu_seqlens[R] are
    not written."""
    dev = _gpu(q, "q")
    n, hk, d, p = _cache_shape(k_cache, v_cache)
    _dense(k_cache, "k_cache")
    _dense(v_cache, "v_cache")
    if k_cache.get_device() != dev:
        raise ValueError(f"the caches must be on device {dev}, got {k_cache.device}")
    if q.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q must be [N, Hq, D] and block_table [R, max_pages]")
    N, hq = q.shape[0], q.shape[1]
    R, mp = block_table.shape
    qs = _rows(q, "q", (torch.bfloat16, torch.float16), (N, hq, d), dev)
    _arr(block_table, "block_table", _I32, (R, mp), dev)
    _arr(ctx_len, "ctx_len", _I32, (R,), dev)
    _arr(cu_seqlens, "cu_seqlens", _I32, (R + 1,), dev)
    if mapped_len is not None:
        _arr(mapped_len, "mapped_len", _I32, (R,), dev)
    words = 0
    if tree_mask is not None:
        words = tree_mask.shape[-1]
        _arr(tree_mask, "tree_mask", torch.uint32 if tree_mask.dtype == torch.uint32 else _I32,
             (N, words), dev)
    sk, sv = _scales(k_cache, k_scale, v_scale, hk, dev)
    L = _D._LIB or _D.lib()
    with _Call(dev, stream) as s:
        if out is None:
            out = q.new_empty((N, hq, d), dtype=q.dtype)
            os_ = hq * d
        else:
            os_ = _rows(out, "out", (q.dtype,), (N, hq, d), dev)
        if lse is None and want_lse:
            lse = q.new_empty((N, hq), dtype=_F32)
        elif lse is not None:
            _arr(lse, "lse", _F32, (N, hq), dev)
        if workspace is None:
            need = L.dspark_tree_attention_workspace(R, N, hq, hk, d)
            workspace = q.new_empty((max(need, 1),), dtype=torch.uint8)
        elif workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on device {dev}")
        st = L.dspark_tree_attention_ex(
            q.data_ptr(), qs, _CACHE[q.dtype], k_cache.data_ptr(), v_cache.data_ptr(),
            _CACHE[k_cache.dtype], sk, sv, block_table.data_ptr(), ctx_len.data_ptr(),
            0 if mapped_len is None else mapped_len.data_ptr(), cu_seqlens.data_ptr(),
            0 if tree_mask is None else tree_mask.data_ptr(), words, R, N, hq, hk, d, p, mp, n,
            1.0 / math.sqrt(d) if scale is None else scale, out.data_ptr(), os_,
            0 if lse is None else lse.data_ptr(), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), s)
    if st:
        _D._check(st, "dspark_tree_attention")
    return out, lse


def dspark_tree_pack(parents, cu_seqlens, mask_words, pos0=None, *, mask=None, flat_pos=None,
                     flat_req=None, want_pos=True, want_req=False, stream=None):
    """Ancestor masks and positions of drafted trees: parents [N] int32 (segment-local,
    -1 for a root), cu_seqlens [R + 1], pos0 [R].  Returns (mask [N, mask_words]
    int32, flat_pos [N]), and flat_req [N] behind them with want_req."""
    dev = _gpu(parents, "parents")
    N, = parents.shape
    R = cu_seqlens.numel() - 1
    _arr(parents, "parents", _I32, (N,), dev)
    _arr(cu_seqlens, "cu_seqlens", _I32, (R + 1,), dev)
    if pos0 is not None:
        _arr(pos0, "pos0", _I32, (R,), dev)
    with _Call(dev, stream) as s:
        if mask is None:
            mask = parents.new_empty((N, mask_words), dtype=_I32)
        if flat_pos is None and want_pos:
            flat_pos = parents.new_empty((N,), dtype=_I32)
        if flat_req is None and want_req:
            flat_req = parents.new_empty((N,), dtype=_I32)
        _arr(mask, "mask", torch.uint32 if mask.dtype == torch.uint32 else _I32, (N, mask_words), dev)
        for t, name in ((flat_pos, "flat_pos"), (flat_req, "flat_req")):
            if t is not None:
                _arr(t, name, _I32, (N,), dev)
        st = (_D._LIB or _D.lib()).dspark_tree_pack(
            parents.data_ptr(), cu_seqlens.data_ptr(), 0 if pos0 is None else pos0.data_ptr(), R, N,
            mask_words, mask.data_ptr(), 0 if flat_pos is None else flat_pos.data_ptr(),
            0 if flat_req is None else flat_req.data_ptr(), s)
    if st:
        _D._check(st, "dspark_tree_pack")
    return (mask, flat_pos, flat_req) if flat_req is not None else (mask, flat_pos)


def dspark_verify_tree(target_logits, cu_seqlens, tokens, parents, max_nodes, *, ctx_len=None,
                       mapped_len=None, target_argmax=None, accepted=None, path=None,
                       next_token=None, stream=None):
    """Greedy verification of trees over a flattened batch: target_logits [N, V] fp32,
    tokens and parents [N] int32, node 0 of each segment its anchor.  With ``ctx_len`` and
    ``mapped_len`` [R] (cur_len and new_len of dspark_page_map) a request that it
    turned down counts as an empty segment.  Returns
    (accepted [R], path [R, max_nodes], next_token [R], target_argmax [N])."""
    dev = _gpu(tokens, "tokens")
    N, = tokens.shape
    R = cu_seqlens.numel() - 1
    _arr(tokens, "tokens", _I32, (N,), dev)
    _arr(parents, "parents", _I32, (N,), dev)
    _arr(cu_seqlens, "cu_seqlens", _I32, (R + 1,), dev)
    if target_logits.dim() != 2:
        raise ValueError("target_logits must be [N, V]")
    V = target_logits.shape[1]
    _arr(target_logits, "target_logits", _F32, (N, V), dev)
    if (ctx_len is None) != (mapped_len is None):
        raise ValueError("ctx_len and mapped_len go together")
    if mapped_len is not None:
        _arr(ctx_len, "ctx_len", _I32, (R,), dev)
        _arr(mapped_len, "mapped_len", _I32, (R,), dev)
    with _Call(dev, stream) as s:
        if target_argmax is None:
            target_argmax = tokens.new_empty((N,), dtype=_I32)
        if accepted is None:
            accepted = tokens.new_empty((R,), dtype=_I32)
        if path is None:
            path = tokens.new_empty((R, max_nodes), dtype=_I32)
        if next_token is None:
            next_token = tokens.new_empty((R,), dtype=_I32)
        _arr(target_argmax, "target_argmax", _I32, (N,), dev)
        _arr(accepted, "accepted", _I32, (R,), dev)
        _arr(path, "path", _I32, (R, max_nodes), dev)
        _arr(next_token, "next_token", _I32, (R,), dev)
        st = (_D._LIB or _D.lib()).dspark_verify_tree_ex(
            target_logits.data_ptr(), cu_seqlens.data_ptr(), tokens.data_ptr(), parents.data_ptr(),
            0 if mapped_len is None else ctx_len.data_ptr(),
            0 if mapped_len is None else mapped_len.data_ptr(), R, N, max_nodes, V,
            target_argmax.data_ptr(), accepted.data_ptr(), path.data_ptr(), next_token.data_ptr(), s)
    if st:
        _D._check(st, "dspark_verify_tree")
    return accepted, path, next_token, target_argmax
