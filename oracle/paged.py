"""The paged cache operators on the CPU, from their definitions: plain loops
for the plan, float64 for attention.  Test infrastructure, sharing no code
with the GPU path.

Attention also returns the largest error that each output may have from
float32 sums and one rounding each of the probabilities and of the result
(``attention_tolerance`` states the terms).
"""
from __future__ import annotations

from typing import NamedTuple

import numpy as np


class Plan(NamedTuple):
    cu_new: np.ndarray
    kv_len: np.ndarray
    slot_map: np.ndarray
    positions: np.ndarray
    page_count: np.ndarray
    stack: list                # the free stack, bottom first
    block_table: np.ndarray
    no_pages: bool
    clipped: bool
    bad_length: bool


def plan(seq_len, num_new, page_count, block_table, stack, page, max_tokens) -> Plan:
    """One request after the other: pages are given back first, then taken."""
    B, width = block_table.shape
    table, held = block_table.copy(), list(page_count)
    cu, fresh, clipped, bad_length, refused = [0], [0] * B, False, False, [False] * B
    for b in range(B):
        s, n = int(seq_len[b]), int(num_new[b])
        if s < 0 or n < 0 or not 0 <= held[b] <= width or s + n > width * page:
            refused[b] = bad_length = True
        elif n and (clipped or cu[-1] + n > max_tokens):
            refused[b] = clipped = True
        else:
            fresh[b] = n
        cu.append(cu[-1] + fresh[b])
    want = [-(-(int(seq_len[b]) + fresh[b]) // page) for b in range(B)]
    given = [int(p) for b in range(B) if not refused[b] for p in table[b, want[b]:held[b]]]
    pool = given + [int(p) for p in stack[::-1]]   # in the order in which pages are taken
    taken, no_pages = 0, False
    for b in range(B):
        need = 0 if refused[b] else want[b] - held[b]
        if need > 0:
            if no_pages or taken + need > len(pool):
                refused[b] = no_pages = True
                continue
            table[b, held[b]:want[b]] = pool[taken:taken + need]
            taken += need
        if not refused[b]:
            held[b] = want[b]
    slots, positions = np.full(max_tokens, -1, np.int32), np.full(max_tokens, -1, np.int32)
    for b in range(B):
        for i in range(fresh[b]):
            at = int(seq_len[b]) + i
            positions[cu[b] + i] = at
            if not refused[b]:
                slots[cu[b] + i] = table[b, at // page] * page + at % page
    kv = [0 if refused[b] else int(seq_len[b]) + fresh[b] for b in range(B)]
    return Plan(np.array(cu, np.int32), np.array(kv, np.int32), slots, positions,
                np.array(held, np.int32), pool[taken:][::-1], table, no_pages, clipped, bad_length)


def append(k_new, v_new, slot_map, k_cache, v_cache):
    """Copies of the caches [n_pages, Hk, page, D] with the new tokens in place."""
    k, v = k_cache.copy(), v_cache.copy()
    page = k.shape[2]
    for t, slot in enumerate(slot_map):
        if slot >= 0:
            k[slot // page, :, slot % page] = k_new[t]
            v[slot // page, :, slot % page] = v_new[t]
    return k, v


class Attention(NamedTuple):
    out: np.ndarray        # [T, Hq, D] float64
    lse: np.ndarray        # [T, Hq]
    out_tol: np.ndarray
    lse_tol: np.ndarray


UNIT = {"bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25)}   # rounding to 8 and 11 significant bits: relative, absolute


def attention_tolerance(dtype, D, x_abs, p, v, o, lse):
    """Bounds for one head's outputs.  ``x_abs`` [n, L]: scale * sum |q||k| of
    every score; ``p`` [n, L] probabilities; ``v`` [L, D].

    A float32 score of D terms is within (D + 4) 2^-23 x_abs (a tensor core's
    sum may truncate, hence a whole unit per term), plus 2^-22 |score| for
    the scale; exp2 adds 2^-21.  A probability therefore has relative error
    e, the normaliser as much, and each is rounded once to the type (relative
    u, or the type's smallest step where it is subnormal); the sums over the
    keys add L 2^-23 at the very worst, 2^-23 sqrt(L) 8 with room."""
    u, tiny = UNIT[dtype]
    L = p.shape[1]
    e = (D + 8) * 2.0 ** -23 * x_abs.max(-1, keepdims=True, initial=0) + 2.0 ** -20 + 2.0 ** -20 * L ** 0.5
    spread = p @ np.abs(v)
    out_tol = u * np.abs(o) + (u + 2 * e) * spread + tiny * np.abs(v).sum(0) + tiny
    lse_tol = e[:, 0] + 2.0 ** -21 * (1 + np.where(np.isfinite(lse), np.abs(lse), 0))
    return out_tol * 1.01, lse_tol


def attention(q, k_cache, v_cache, block_table, cu_new, kv_len, scale, dtype) -> Attention:
    """float64 arrays in, request by request and head by head."""
    T, Hq, D = q.shape
    Hk, page = k_cache.shape[1], k_cache.shape[2]
    out, tol = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, lse_tol = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for b in range(len(kv_len)):
        begin, end, L = int(cu_new[b]), int(cu_new[b + 1]), int(kv_len[b])
        n = end - begin
        if n == 0 or L == 0:
            continue
        ids = block_table[b, :-(-L // page)]
        last = L - n + np.arange(n)
        seen = np.arange(L)[None] <= last[:, None]
        for h in range(Hq):
            k = k_cache[ids, h * Hk // Hq].reshape(-1, D)[:L]
            v = v_cache[ids, h * Hk // Hq].reshape(-1, D)[:L]
            qh = q[begin:end, h]
            x = np.where(seen, qh @ k.T * scale, -np.inf)
            top = np.max(x, -1, keepdims=True)
            w = np.exp(x - np.where(np.isfinite(top), top, 0))
            total = w.sum(-1, keepdims=True)
            p = w / np.where(total > 0, total, 1)
            o = p @ v
            with np.errstate(divide="ignore"):
                z = (np.where(np.isfinite(top), top, 0) + np.log(total))[:, 0]
            x_abs = np.where(seen, np.abs(qh) @ np.abs(k).T * scale, 0)
            out[begin:end, h], lse[begin:end, h] = o, z
            tol[begin:end, h], lse_tol[begin:end, h] = attention_tolerance(dtype, D, x_abs, p, v, o, z)
    return Attention(out, lse, tol, lse_tol)
