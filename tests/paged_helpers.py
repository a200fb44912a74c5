"""Inputs for the tests of the verification over a paged cache."""
from __future__ import annotations

import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}


def half_step(dtype):
    """Largest relative rounding error of a type: half a step."""
    return torch.finfo(dtype).eps / 2


def starts(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def caches(rng, pages, Hk, D, P, name, device, std=1.0):
    t = TYPES[name]
    c = 16 if name == "e4m3" else 8
    k = torch.from_numpy(rng.normal(0, std, (pages, Hk, D // c, P, c)).astype(np.float32))
    v = torch.from_numpy(rng.normal(0, std, (pages, Hk, D, P)).astype(np.float32))
    return k.to(t).to(device), v.to(t).to(device)


def tables(rng, lens, P, pages, width=None):
    """Rows of distinct pages in random order; behind a row's end, ids that no one may use."""
    need = [-(-int(x) // P) for x in lens]
    assert sum(need) <= pages
    width = max(1, max(need)) if width is None else width
    order = rng.permutation(pages)
    t = np.full((len(lens), width), -1, np.int32)
    at = 0
    for r, k in enumerate(need):
        t[r, :k] = order[at:at + k]
        at += k
    t[:, :][t == -1] = rng.choice([-1, pages, 2 ** 31 - 1, -2 ** 31], size=int((t == -1).sum()))
    return t


def random_parents(rng, n, roots=False):
    p = np.full(n, -1, np.int32)
    for i in range(1, n):
        p[i] = rng.integers(-1 if roots else 0, i)
    return p


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)
