"""Oracle for the attention operators and the cache read.  Test infrastructure only (see
the package docstring).

packed_attention: for query token i (head h) of a sequence with Lq queries and Lk keys,
    out[i, h] = sum_j w_j v[j, h // g],  w = softmax_j(scale * q[i, h] . k[j, h // g]),
over the sequence's keys j, with ``causal`` those with j <= i + Lk - Lq; g is the number
of query heads per key head.  No visible key: zeros, lse -inf.  lse is the log of the sum
of exp(scale * q . k).

paged_attention: the same with k and v read through a block table from the caches of
KvRmsNormRopeCache (position j of sequence b: page table[b, j // block_size], offset
j % block_size; Norm mode: row j of sequence b), the Lq query tokens being the sequence's
last positions.  V1's key is the ckv row followed by the k row, its value the ckv row.
A page outside the cache is left out.

kv_cache_read: rows gathered by the slots of kv_rms_norm_rope_cache's index (-1 and slots
outside the cache give zeros).

A quantised element is read as (code - offset) / scale.  Everything is float64.  The
attention functions also return what their rounding bounds are made of: ``spread`` =
sum_j w_j |v_j| and ``reach`` = max_j scale * sum_c |q_c| |k_jc| per row, the latter on
the operands as stored (q / scale against codes, for a quantised cache).
"""
from __future__ import annotations

import numpy as np

from .codes import decode_bf16, decode_e4m3, decode_e5m2, decode_fp16
from .kv_cache import token_slots

_DECODE = {"bf16": decode_bf16, "fp16": decode_fp16, "e4m3": decode_e4m3, "e5m2": decode_e5m2,
           "int8": lambda x: np.asarray(x, np.float64)}


def attend(q, k, v, scale, causal, hidden=None):
    """One sequence and head: q [Lq, Dk], k [Lk, Dk], v [Lk, Dv] float64.  ``hidden``
    marks keys that no query sees.  Returns out [Lq, Dv], lse [Lq], spread [Lq, Dv]."""
    Lq, Lk = q.shape[0], k.shape[0]
    out, spread = np.zeros((Lq, v.shape[1])), np.zeros((Lq, v.shape[1]))
    lse = np.full(Lq, -np.inf)
    for i in range(Lq):
        n = min(Lk, max(0, i + Lk - Lq + 1)) if causal else Lk
        keep = np.arange(n) if hidden is None else np.nonzero(~hidden[:n])[0]
        if keep.size == 0:
            continue
        s = k[keep] @ q[i] * scale
        top = s.max()
        e = np.exp(s - top)
        w = e / e.sum()
        out[i] = w @ v[keep]
        spread[i] = w @ np.abs(v[keep])
        lse[i] = top + np.log(e.sum())
    return out, lse, spread


def packed_attention(q, k, v, *, starts_q, starts_k, scale, causal) -> dict:
    """q [Tq, heads, d], k and v [Tk, kv_heads, d] float64; starts [B + 1].  Rows outside
    every sequence are NaN in the results."""
    g = q.shape[1] // k.shape[1]
    res = {"out": np.full(q.shape[:2] + (v.shape[2],), np.nan), "lse": np.full(q.shape[:2], np.nan),
           "spread": np.full(q.shape[:2] + (v.shape[2],), np.nan), "reach": np.zeros(q.shape[:2])}
    for b in range(len(starts_q) - 1):
        a, z = slice(starts_q[b], starts_q[b + 1]), slice(starts_k[b], starts_k[b + 1])
        for h in range(q.shape[1]):
            o, l, s = attend(q[a, h], k[z, h // g], v[z, h // g], scale, causal)
            res["out"][a, h], res["lse"][a, h], res["spread"][a, h] = o, l, s
            if k[z].shape[0] and q[a].shape[0]:
                res["reach"][a, h] = (np.abs(q[a, h]) @ np.abs(k[z, h // g]).T).max(axis=1) * scale
    return res


def _dequantise(codes, scale, offset, n):
    """Codes [L, D] of head n to values; scale / offset [N, D], [D] or [1]."""
    if scale is None:
        return codes
    s = np.asarray(scale, np.float64)
    o = np.zeros_like(s) if offset is None else np.asarray(offset, np.float64)
    if s.ndim == 2:
        s, o = s[n], o[n]
    return (codes - o) / s


def _rows(cache, cache_mode, block_size, b, n, L, table):
    """The first L rows of sequence b, head n: [L, D] as stored (decoded), and which lie in
    a page outside the cache."""
    pos = np.arange(L)
    if cache_mode == "Norm":
        return cache[b, n, pos], np.zeros(L, bool)
    page = np.asarray(table[b], np.int64)[pos // block_size]
    bad = (page < 0) | (page >= cache.shape[0])
    page = np.where(bad, 0, page)
    if cache_mode == "PA":
        return cache[page, pos % block_size, n], bad
    return cache[page, n, pos % block_size], bad


def paged_attention(q, k_cache, ckv_cache, *, variant, seq_lens, starts_q, scale, causal, cache_mode="PA_BNSD",
                    block_size=0, table=None, k_type="bf16", v_type="bf16", k_scale=None, k_offset=None,
                    v_scale=None, v_offset=None) -> dict:
    """q [Tq, heads, Dk] float64; caches as stored (bit patterns, codes)."""
    kc, vc = _DECODE[k_type](k_cache), _DECODE[v_type](ckv_cache)
    N = kc.shape[2] if cache_mode == "PA" else kc.shape[1]
    g, Dv = q.shape[1] // N, vc.shape[-1]
    res = {"out": np.full(q.shape[:2] + (Dv,), np.nan), "lse": np.full(q.shape[:2], np.nan),
           "spread": np.full(q.shape[:2] + (Dv,), np.nan), "reach": np.zeros(q.shape[:2])}
    for b, L in enumerate(seq_lens):
        a = slice(starts_q[b], starts_q[b + 1])
        for n in range(N):
            ks, bad = _rows(kc, cache_mode, block_size, b, n, L, table)
            vs, _ = _rows(vc, cache_mode, block_size, b, n, L, table)
            k = _dequantise(ks, k_scale, k_offset, n)
            v = _dequantise(vs, v_scale, v_offset, n)
            one = lambda s, w: np.ones(w) if s is None else np.broadcast_to(np.asarray(s)[n] if np.ndim(s) == 2 else s, w)
            stored, div = ks, one(k_scale, ks.shape[1])
            if variant == 1:
                k = np.concatenate([v, k], axis=1)
                stored = np.concatenate([vs, ks], axis=1)
                div = np.concatenate([one(v_scale, vs.shape[1]), div])
            for h in range(n * g, (n + 1) * g):
                o, l, s = attend(q[a, h], k, v, scale, causal, bad)
                res["out"][a, h], res["lse"][a, h], res["spread"][a, h] = o, l, s
                if L and q[a].shape[0]:
                    res["reach"][a, h] = (np.abs(q[a, h] / div) @ np.abs(np.where(bad[:, None], 0, stored)).T).max(axis=1) * scale
    return res


def kv_cache_read(index, cache, *, B, N, S, cache_mode, block_size, stored="bf16", scale=None, offset=None):
    """One cache's rows: float64 [B, N, S, D], and the number of slots outside the cache."""
    c = _DECODE[stored](cache)
    out = np.zeros((B, N, S, c.shape[-1]))
    limit = c.shape[2] if cache_mode == "Norm" else c.shape[0] * block_size
    bad = 0
    for b in range(B):
        slots = token_slots(index, cache_mode, np.full(S, b), np.arange(S), S, block_size)
        for s, p in enumerate(slots):
            if p == -1:
                continue
            if p < 0 or p >= limit:
                bad += 1
                continue
            for n in range(N):
                if cache_mode == "Norm":
                    row = c[b, n, p]
                elif cache_mode == "PA":
                    row = c[p // block_size, p % block_size, n]
                else:
                    row = c[p // block_size, n, p % block_size]
                out[b, n, s] = _dequantise(row[None], scale, offset, n)[0]
    return out, bad
