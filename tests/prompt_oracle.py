"""Plain 64-bit forms of the operators for prompts over the paged cache, for the tests.

Written from the definitions in include/ditattn.h; shares no code with the library.
"""
import math

import numpy as np
import torch


def requests(cu_new, seq_lens, T, max_len, start_lens=None):
    """(first row, new tokens, cached keys, position of the first new token) of each request."""
    res = []
    for b in range(len(seq_lens)):
        lo, hi = (min(max(int(x), 0), T) for x in (cu_new[b], cu_new[b + 1]))
        n, length = max(0, hi - lo), min(max(int(seq_lens[b]), 0), max_len)
        res.append((lo, n, length, length - n if start_lens is None else int(start_lens[b])))
    return res


def places(table, b, length, P, n_pages):
    """(pages, rows) of the keys of request b by position; page -1: none."""
    j = np.arange(length)
    page = table[b, j // P] if length else np.zeros(0, np.int64)
    return np.where((page >= 0) & (page < n_pages), page, -1), j % P


def attend(q, k_cache, v_cache, table, seq_lens, cu_new, scale, causal=True, start_lens=None, device="cpu"):
    """(out, lse, owned, (mag, pv)) in fp64: owned [T] tells the rows of a request; mag [T, Hq] is
    scale max_j sum_d |q_d k_jd| over the keys that a row sees, pv [T, Hq, D] sum_j p_j |v_j|."""
    q, k_cache, v_cache = (x.detach().to(device).double() for x in (q, k_cache, v_cache))
    table = np.asarray(table.cpu()).astype(np.int64)
    host = lambda x: None if x is None else [int(y) for y in x.cpu()]  # noqa: E731
    T, Hq, D = q.shape
    n_pages, Hkv, P = k_cache.shape[:3]
    G = Hq // Hkv
    o, pv = (torch.zeros(T, Hq, D, dtype=torch.float64, device=device) for _ in range(2))
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=device)
    mag = torch.zeros(T, Hq, dtype=torch.float64, device=device)
    owned = torch.zeros(T, dtype=torch.bool)
    for b, (row, n, length, start) in enumerate(requests(host(cu_new), host(seq_lens), T, table.shape[1] * P,
                                                         host(start_lens))):
        owned[row:row + n] = True
        if n == 0 or length == 0:
            continue
        page, at = places(table, b, length, P, n_pages)
        have = torch.as_tensor(page >= 0, device=device)
        page, at = (torch.as_tensor(np.maximum(x, 0), device=device) for x in (page, at))
        see = have[None, :].expand(n, -1)
        if causal:
            pos = torch.arange(n, device=device)[:, None] + start
            see = see & (torch.arange(length, device=device)[None, :] <= pos)
        for h in range(Hq):
            k, v = k_cache[page, h // G, at], v_cache[page, h // G, at]
            x = q[row:row + n, h]
            s = scale * (x @ k.T)
            s = torch.where(see, s, -math.inf)
            m = s.amax(1, keepdim=True)
            e = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
            z = e.sum(1, keepdim=True)
            p = e / torch.where(z > 0, z, 1.0)
            o[row:row + n, h] = p @ v
            pv[row:row + n, h] = p @ v.abs()
            lse[row:row + n, h] = (m + torch.log(z))[:, 0]
            a = torch.where(see, x.abs() @ k.abs().T, 0.0)
            mag[row:row + n, h] = scale * a.amax(1)
    return o.cpu(), lse.cpu(), owned, (mag.cpu(), pv.cpu())


def norm_rope(x, weight, eps, freqs, axis_pairs, positions, interleaved, rot_scale):
    """(y, size) in fp64 of x [B, H, N, D]: norms (eps None: none), then the rotation (freqs None: none) at positions
    [axes, B, N]; size is |z_first| + |z_second| of each channel's pair, what y's errors are relative to."""
    z = x.detach().cpu().double()
    if eps is not None:
        z = z / torch.sqrt((z * z).mean(-1, keepdim=True) + eps)
        if weight is not None:
            z = z * weight.cpu().double()
    if freqs is None:
        return z, z.abs()
    f = freqs.cpu().double()
    axis = np.repeat(np.arange(len(axis_pairs)), axis_pairs)
    t = positions.cpu().double()[axis].permute(1, 2, 0)[:, None] * f  # [B, 1, N, n]
    c, s, n = torch.cos(t) * rot_scale, torch.sin(t) * rot_scale, len(f)
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    y, size = z.clone(), z.abs()
    y[..., i], y[..., j] = z[..., i] * c - z[..., j] * s, z[..., i] * s + z[..., j] * c
    both = (z[..., i].abs() + z[..., j].abs()) * abs(rot_scale)
    size[..., i], size[..., j] = both, both
    return y, size


def page_mass(q, lse, k_cache, table, seq_lens, mass, scale, cu_new=None, start_lens=None, window=0):
    """(mass_out, size) in fp64: size [n_pages, Hkv] is sum of weights times (1 + scale max |q||k|) of what was added."""
    q, lse, k_cache, out = (x.detach().cpu().double() for x in (q, lse, k_cache, mass))
    table = np.asarray(table.cpu()).astype(np.int64)
    T, Hq, D = q.shape
    n_pages, Hkv, P = k_cache.shape[:3]
    B, G = table.shape[0], Hq // Hkv
    host = lambda x: [int(y) for y in x.cpu()]  # noqa: E731
    cu = list(range(B + 1)) if cu_new is None else host(cu_new)
    size = torch.zeros_like(out)
    for b, (row, n, length, start) in enumerate(requests(cu, host(seq_lens), T, table.shape[1] * P,
                                                         None if start_lens is None else host(start_lens))):
        if n == 0 or length == 0:
            continue
        page, at = places(table, b, length, P, n_pages)
        w = min(n, window) if window > 0 else n
        for c in range(-(-length // P)):
            if page[c * P] >= 0 and c * P >= start:
                out[page[c * P]] = 0
        see = torch.arange(length)[None, :] <= (torch.arange(n - w, n) + start)[:, None]
        safe = np.maximum(page, 0)
        for h in range(Hq):
            k, x, m = k_cache[safe, h // G, at], q[row + n - w:row + n, h], lse[row + n - w:row + n, h]
            s = scale * (x @ k.T)
            e = torch.where(see & (m > -math.inf)[:, None] | (see & m.isnan()[:, None]), torch.exp(s - m[:, None]), 0.0)
            e = e * torch.as_tensor(page >= 0)
            big = 1 + scale * (x.abs() @ k.abs().T)
            add = torch.where(e > 0, e * big, 0.0).sum(0)
            ok = torch.as_tensor(page >= 0)
            out[:, h // G].index_add_(0, torch.as_tensor(page)[ok], e.sum(0)[ok])
            size[:, h // G].index_add_(0, torch.as_tensor(page)[ok], add[ok])
    return out, size


def evict(mass, table, seq_lens, free_pages, n_free, P, keep, recent):
    """(table, lens, stack, n_free) after the eviction; Python numbers throughout."""
    mass, table, stack = mass.detach().cpu().double().numpy(), table.cpu().numpy().copy(), free_pages.cpu().numpy().copy()
    n_pages = mass.shape[0]
    free, lens = min(max(0, int(n_free)), len(stack)), []
    for b in range(len(table)):
        length = min(max(0, int(seq_lens[b])), table.shape[1] * P)
        n = -(-length // P)
        if n > keep:
            def weight(i):
                page = int(table[b, i])
                if not 0 <= page < n_pages:
                    return (0, 0.0)  # below every number
                with np.errstate(invalid="ignore"):
                    x = float(sum(mass[page]))
                return (2, 0.0) if math.isnan(x) else (1, x)
            order = sorted(range(n - recent), key=lambda i: tuple(-y for y in weight(i)) + (i,))
            stay = set(order[:keep - recent]) | set(range(n - recent, n))
            kept = [int(table[b, i]) for i in range(n) if i in stay]
            for i in range(n):
                page = int(table[b, i])
                if i not in stay and 0 <= page < n_pages:
                    if free < len(stack):
                        stack[free] = page
                    free += 1
            table[b, :n] = kept + [-1] * (n - keep)
            length -= (n - keep) * P
        lens.append(length)
    return table, np.array(lens), stack, min(free, len(stack))
