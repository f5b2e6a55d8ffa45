"""Plain 64-bit forms of the paged-cache operators, request by request, for the tests.

Written from the definitions in include/ditattn.h; shares no code with the library.
"""
import math

import numpy as np
import torch


def plan(new_lens, seq_lens, table, free_pages, n_free, P, n_pages, max_tokens):
    """(lens, n_free, cu, slots, table) after the step; Python integers throughout."""
    B, max_pages = table.shape
    table = table.copy()
    cap = max_pages * P
    free = min(max(0, int(n_free)), len(free_pages))
    cu, lens, slots = [0], [], [-1] * max_tokens
    for b in range(B):
        s = min(max(0, int(seq_lens[b])), cap)
        t0 = cu[-1]
        t1 = min(max_tokens, t0 + max(0, int(new_lens[b])))
        cu.append(t1)
        have = -(-s // P)
        pages = have
        stored = s
        for t in range(t0, t1):
            pos = s + t - t0
            if pos >= cap:
                break
            if pos // P == pages:
                if free == 0:
                    break
                free -= 1
                table[b, pages] = free_pages[free]
                pages += 1
            stored = pos + 1
            page = int(table[b, pos // P])
            if 0 <= page < n_pages:
                slots[t] = page * P + pos % P
        lens.append(stored)
    return np.array(lens), free, np.array(cu), np.array(slots), table


def write(k_new, slots, cache, summary=None):
    """New rows [T, H, D] into a copy of the cache [n_pages, H, P, D] and of its summary."""
    cache = cache.clone()
    summary = None if summary is None else summary.clone()
    n_pages, P = cache.shape[0], cache.shape[2]
    fresh = {}
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < n_pages * P:
            cache[s // P, :, s % P] = k_new[t]
            fresh.setdefault(s // P, []).append((s % P, t))
    if summary is not None:
        for page, rows in fresh.items():
            x = k_new[[t for _, t in rows]].double()
            lo, hi = x.amin(0), x.amax(0)
            if all(r != 0 for r, _ in rows):
                lo = torch.minimum(lo, summary[page, :, 0].double())
                hi = torch.maximum(hi, summary[page, :, 1].double())
            summary[page] = torch.stack((lo, hi), 1).to(summary.dtype)
    return cache, summary


def rows_of(table, b, length, P, n_pages, selected=None):
    """(page, row) of each key that request b's query sees, in order."""
    length = min(max(0, int(length)), table.shape[1] * P)
    n = -(-length // P)
    cols = range(n) if selected is None else [int(i) for i in selected[:n]]
    out = []
    for i in cols:
        if 0 <= i < n and 0 <= int(table[b, i]) < n_pages:
            out += [(int(table[b, i]), r) for r in range(min(P, length - i * P))]
    return out


def attend(q, k_cache, v_cache, table, seq_lens, scale, selected=None):
    """(out, lse, bound): fp64 [B, Hq, D] and [B, Hq]; bound holds, per query head,
    (scale * max_j sum_d |q_d k_jd|, per channel sum_j p_j |v_j|)."""
    q, k_cache, v_cache = (x.detach().cpu().double().numpy() for x in (q, k_cache, v_cache))
    table, seq_lens = np.asarray(table.cpu()), np.asarray(seq_lens.cpu())
    selected = None if selected is None else np.asarray(selected.cpu())
    B, Hq, D = q.shape
    n_pages, Hkv, P = k_cache.shape[:3]
    o, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -math.inf)
    mag, pv = np.zeros((B, Hq)), np.zeros((B, Hq, D))
    for b in range(B):
        for g in range(Hkv):
            at = rows_of(table, b, seq_lens[b], P, n_pages, None if selected is None else selected[b, g])
            if not at:
                continue
            page, row = np.array(at).T
            k, v = k_cache[page, g, row], v_cache[page, g, row]
            for h in range(g * Hq // Hkv, (g + 1) * Hq // Hkv):
                s = scale * (k @ q[b, h])
                m = s.max()
                e = np.exp(s - m)
                o[b, h] = e @ v / e.sum()
                lse[b, h] = m + math.log(e.sum())
                mag[b, h] = scale * (np.abs(k) @ np.abs(q[b, h])).max()
                pv[b, h] = e @ np.abs(v) / e.sum()
    return o, lse, (mag, pv)


def scores(q, summary, table, seq_lens, P):
    """Per request and key/value head the list of (score, column), newest page first of all."""
    q, summary = q.detach().cpu().double().numpy(), summary.detach().cpu().double().numpy()
    table, seq_lens = np.asarray(table.cpu()), np.asarray(seq_lens.cpu())
    B, Hq, _ = q.shape
    n_pages, Hkv = summary.shape[:2]
    res = []
    for b in range(B):
        n = -(-min(max(0, int(seq_lens[b])), table.shape[1] * P) // P)
        for g in range(Hkv):
            x = np.full(n, -math.inf)
            ok = np.flatnonzero((table[b, :n] >= 0) & (table[b, :n] < n_pages))
            lo, hi = summary[table[b, ok], g, 0], summary[table[b, ok], g, 1]
            with np.errstate(invalid="ignore"):
                heads = [np.maximum(q[b, h] * lo, q[b, h] * hi).sum(1)
                         for h in range(g * Hq // Hkv, (g + 1) * Hq // Hkv)]
                heads = np.where(np.isnan(heads), math.inf, heads)
            x[ok] = heads.max(0)
            res.append(x)
    return res


def select(q, summary, table, seq_lens, P, top_k):
    Hkv = summary.shape[1]
    out = np.full((q.shape[0] * Hkv, top_k), -1, np.int64)
    for i, x in enumerate(scores(q, summary, table, seq_lens, P)):
        if len(x) == 0:
            continue
        order = sorted(range(len(x) - 1), key=lambda j: (-x[j], j))
        pick = sorted([len(x) - 1] + order[:top_k - 1])
        out[i, :len(pick)] = pick
    return out.reshape(q.shape[0], Hkv, top_k)
