"""Plain CPU oracle of the paged-serving operators (numpy float64, Python integers).

TEST INFRASTRUCTURE ONLY, like fia_oracle.py, whose rules it keeps: the CUDA
library never imports it and it imports nothing from the library.

  * a query token at position p sees key j when j <= p and (j >= p - pre_tokens
    or j < sink_tokens); token i of n new tokens has p = L - n + i (L: keys of
    its sequence, the new tokens among them); a row that sees no key gives 0 and
    an lse of +inf;
  * a block id outside the pool stands for rows of zeros;
  * request b holds ceil(context / block_size) blocks and needs ceil((context +
    new) / block_size); the lacking ones come off the free list in request order.
"""
from __future__ import annotations

import numpy as np

from .fia_oracle import f64


def window_see(n: int, L: int, pre: int, sink: int) -> np.ndarray:
    """(n, L) bool: what the last n of L tokens see."""
    p = np.arange(n)[:, None] + (L - n)
    j = np.arange(L)[None, :]
    return (j <= p) & ((j >= p - pre) | (j < sink))


def cache_rows(pool: np.ndarray, ids, L: int, n2: int) -> np.ndarray:
    """The first L rows (L, n2, D) of a sequence with the given block ids."""
    if pool.ndim == 3:
        pool = pool.reshape(pool.shape[0], pool.shape[1], n2, -1)
    else:
        pool = pool.transpose(0, 2, 1, 3)
    bs = pool.shape[1]
    rows = np.zeros((L,) + pool.shape[2:], dtype=np.float64)
    for i in range(-(-L // bs)):
        blk = int(ids[i])
        e = min(L, (i + 1) * bs)
        if 0 <= blk < pool.shape[0]:
            rows[i * bs:e] = pool[blk, :e - i * bs]
    return rows


def attend(q, k, v, see, scale):
    """q (n, N1, D), k / v (L, N2, D), see (n, L) -> out (n, N1, D), lse (n, N1), and what bounds of rounding need:
    sum of w |v| (n, N1, D) and the largest scale * sum |q| |k| over the seen keys (n, N1).  Rows of k and v that
    nobody sees do not enter (they may be NaN)."""
    n, N1, D = q.shape
    used = see.any(0)
    k, v, see = k[used], v[used], see[:, used]
    g = N1 // k.shape[1]
    out, lse = np.zeros((n, N1, v.shape[2])), np.full((n, N1), np.inf)
    av, big = np.zeros_like(out), np.zeros((n, N1))
    some = see.any(1)
    if not some.any():
        return out, lse, av, big
    for h in range(N1):
        kh, vh, qh = k[:, h // g], v[:, h // g], q[some][:, h]
        s = np.where(see[some], scale * (qh @ kh.T), -np.inf)
        top = s.max(1, keepdims=True)
        e = np.exp(s - top)
        w = e / e.sum(1, keepdims=True)
        out[some, h], av[some, h] = w @ vh, w @ np.abs(vh)
        lse[some, h] = np.log(e.sum(1)) + top[:, 0]
        big[some, h] = np.where(see[some], scale * (np.abs(qh) @ np.abs(kh).T), 0.0).max(1)
    return out, lse, av, big


def decode(q, rows, lens, pre, sink, scale):
    """q (B, N1, Q, D) tensor, rows[b] = (k, v) of at least lens[b] rows -> out, lse (B, N1, Q, 1), bounds as attend."""
    q = f64(q)
    parts = []
    for b, L in enumerate(lens):
        n = q.shape[2]
        k, v = (x[:L] for x in rows[b])
        see = window_see(n, L, pre, sink)
        parts.append([x.swapaxes(0, 1) for x in attend(q[b].swapaxes(0, 1), k, v, see, scale)])
    return tuple(np.stack([p[i] for p in parts]) for i in range(4))


def assert_close(out, lse, ref, what=""):
    """Every output within what its roundings allow.  h: half a step of the output's type, relative.
      out: the output's rounding h |out|, the weights' rounding for the second product h sum w |v|, and the scores'
           error d (products exact, a sum of D + 8 roundings of at most 2^-24 sum |q| |k| scale), which moves a weight
           by at most 2 d, and its normalisation by as much again; 2^-20 for exponentials and the joins of partials.
      lse: 2 d, and the roundings of the logarithm, the maximum and their sum (2^-22 each, relative to what they hold)."""
    import torch
    o, l, av, big = ref
    h = torch.finfo(out.dtype).eps / 2
    D = o.shape[-1]
    g = out.detach().double().cpu().numpy()
    assert g.shape == o.shape, (what, g.shape, o.shape)
    d = big * (D + 8) * 2.0 ** -24
    tol = h * (np.abs(o) + av) * (1 + h) + (4 * d[..., None] + 2.0 ** -20) * av
    if out.dtype == torch.float16:
        tol = tol + 2.0 ** -25          # half of the smallest subnormal
    bad = ~(np.abs(g - o) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} outputs off, first at {np.argwhere(bad)[0]}: " \
                          f"{g[bad][0]} vs {o[bad][0]} (allowed {tol[bad][0]:.2e})"
    if lse is not None:
        gl = lse.detach().double().cpu().numpy().reshape(l.shape)
        assert np.array_equal(np.isposinf(gl), np.isposinf(l)), f"{what}: rows without keys differ"
        f = np.isfinite(l)
        ltol = 2 * d + 2.0 ** -19 * np.maximum(1.0, np.abs(np.where(f, l, 0.0)))
        assert (np.abs(gl[f] - l[f]) <= ltol[f]).all(), f"{what}: lse off by {np.abs(gl[f] - l[f]).max()}"


def block_table_append(context, new, free, table, bs, n_tokens):
    """Lists and a (B, W) integer array -> (table, slots, kv_lens, cu, blocks)."""
    table = np.array(table, dtype=np.int64)
    slots = [-1] * n_tokens
    at, t, cu, kv = 0, 0, [], []
    for b, (c, a) in enumerate(zip(context, new)):
        c, a = max(c, 0), max(a, 0)
        have, need = -(-c // bs), -(-(c + a) // bs)
        for i in range(a):
            page, off = (c + i) // bs, (c + i) % bs
            if t < n_tokens and page < table.shape[1]:
                if page >= have and off == 0:
                    f = at + page - have
                    table[b, page] = free[f] if f < len(free) else -1
                # a page's first new token may lie past n_tokens: then no later token of it is written either
                if table[b, page] >= 0 and (page < have or at + page - have < len(free)):
                    slots[t] = int(table[b, page]) * bs + off
            t += 1
        at += need - have
        cu.append(t)
        kv.append(c + a)
    return table, slots, kv, cu, at


def cache_write(x, cache, slots):
    """x (T, N, D) and a pool as float64 arrays -> the pool with the rows written."""
    out = cache.copy()
    for t, s in enumerate(slots):
        bs = out.shape[1] if out.ndim == 3 else out.shape[2]
        if 0 <= s < out.shape[0] * bs:
            if out.ndim == 4:
                out[s // bs, :, s % bs] = x[t]
            else:
                out[s // bs, s % bs] = x[t].reshape(-1)
    return out
