"""The paged key/value cache's operators as measured cases: the step's plan (block tables and slot
maps from request lengths), the cache write, single-token attention over the pages, and the same
attention over the pages that a cheap score selects.

Four kinds of case, one operator each:

plan    new_lens, seq_lens [B] -> the pages each request is granted from a stack of free pages,
        written into its block-table row, and each new token's slot (page * page_size + row).
write   k, v of T new tokens, as slices of one fused projection, stored into their slots of the
        paged caches; each touched page's summary (per channel minimum and maximum of its keys)
        is brought up to date.
decode  o_b,h = softmax_j(scale q_b,h . k_j) v_j over the seq_lens[b] cached keys of request b;
        query heads h of one group share a key/value head; lse = ln sum_j exp(scale q . k_j).
sparse  for each request and key/value head, the score of page i is
        max over the group's heads of sum_d max(q_d lo_i,d, q_d hi_i,d), an upper bound of q . k over
        the page; the top_k pages with the highest scores (ties: the lowest index; the newest page
        always among them) are listed in ascending order, and decode runs over those pages alone.

`own` False computes each in elementary torch operations; True calls the library.
"""
import math

import numpy as np
import torch

own = False

# Each head layout is one of this repository's workloads' (24 or 40 heads of 128, 2 heads of 64)
# or a grouped form of it; lengths are its token counts (512, 1024, 4608, 27280, 75600).


def listed():
    return [
        # one token for each request of a full decode batch
        dict(name="plan decode 256", kind="plan", B=256, P=16, len_lo=1, len_hi=27280, new_lo=1, new_hi=1,
             spare=0, pool=1.25),
        # a step that mixes chunked prefills with decodes, its batch padded to a fixed token count
        dict(name="plan mixed 75600", kind="plan", B=63, P=64, len_lo=0, len_hi=4608, new_lo=1, new_hi=2398,
             spare=63, pool=1.5),
        # the keys and values of one decoded token of each of 64 requests
        dict(name="write decode 64", kind="write", B=64, Hq=24, Hkv=8, D=128, P=16, len_lo=0, len_hi=4608,
             new_lo=1, new_hi=1, spare=0, order="hnd"),
        # ragged prefill chunks in small heads, token-major pages
        dict(name="write ragged d64", kind="write", B=13, Hq=2, Hkv=2, D=64, P=48, len_lo=3, len_hi=1024,
             new_lo=1, new_hi=709, spare=29, order="nhd"),
        # one long video's keys, all heads
        dict(name="write prefill 27280", kind="write", B=1, Hq=24, Hkv=24, D=128, P=64, len_lo=0, len_hi=0,
             new_lo=27280, new_hi=27280, spare=0, order="hnd"),
        # the smallest call: a few short requests, where the launch counts
        dict(name="decode short d64", kind="decode", B=4, Hq=2, Hkv=2, D=64, P=16, len_lo=1, len_hi=1024,
             order="hnd", out="float32"),
        # one request against a long context: the keys' length is all there is to split
        dict(name="decode one 27280", kind="decode", B=1, Hq=24, Hkv=8, D=128, P=16, len_lo=27280,
             len_hi=27280, order="hnd", out="bfloat16"),
        # an ordinary ragged batch without shared heads, some rows still empty
        dict(name="decode ragged mha", kind="decode", B=48, Hq=24, Hkv=24, D=128, P=32, len_lo=0,
             len_hi=4608, order="nhd", out="float32"),
        # a full batch of long contexts
        dict(name="decode long 16x75600", kind="decode", B=16, Hq=40, Hkv=8, D=128, P=64, len_lo=30001,
             len_hi=75600, order="hnd", out="bfloat16"),
        # one long request, a 37th of its pages
        dict(name="sparse one 75600", kind="sparse", B=1, Hq=24, Hkv=8, D=128, P=16, len_lo=75600,
             len_hi=75600, order="hnd", out="bfloat16", top_k=128),
        # a ragged batch: the short requests have fewer pages than top_k
        dict(name="sparse ragged 32", kind="sparse", B=32, Hq=40, Hkv=8, D=128, P=32, len_lo=0,
             len_hi=27280, order="hnd", out="float32", top_k=48),
        # heads of 64 without sharing, larger pages
        dict(name="sparse mha d64", kind="sparse", B=7, Hq=2, Hkv=2, D=64, P=64, len_lo=513, len_hi=27280,
             order="nhd", out="bfloat16", top_k=17),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("plan", "write", "decode", "decode", "sparse", "sparse"))
    P = rng.choice((16, 32, 48, 64, 128))
    if kind == "plan":
        B = _log(rng, 1, 2048)
        most = max(1, 75600 // B)
        hi = _log(rng, 1, most)
        return dict(kind=kind, B=B, P=P, len_lo=rng.randrange(0, 20), len_hi=_log(rng, 20, 27280),
                    new_lo=rng.randrange(0, hi + 1), new_hi=hi, spare=rng.choice((0, 1, 37)),
                    pool=rng.choice((0.7, 1.0, 1.5)))
    heads = rng.choice(((24, 24, 128), (24, 8, 128), (40, 8, 128), (40, 40, 128), (2, 2, 64), (16, 1, 64),
                        (24, 2, 128), (24, 1, 128)))
    base = dict(kind=kind, Hq=heads[0], Hkv=heads[1], D=heads[2], P=P, order=rng.choice(("hnd", "nhd")))
    if kind == "write":
        B = _log(rng, 1, 64)
        most = max(1, 27280 * 24 * 128 // (B * heads[1] * heads[2]))
        hi = _log(rng, 1, min(most, 27280))
        return dict(base, B=B, len_lo=0, len_hi=_log(rng, 1, 4608), new_lo=rng.randrange(0, hi + 1), new_hi=hi,
                    spare=rng.choice((0, 1, 37)))
    # cached elements stay below the largest listed case's
    B = _log(rng, 1, 128)
    hi = _log(rng, 1, min(75600, max(1, 16 * 75600 * 8 * 128 // (B * heads[1] * heads[2]))))
    base.update(B=B, len_lo=rng.randrange(0, hi + 1), len_hi=hi, out=rng.choice(("float32", "bfloat16")))
    if kind == "sparse":
        base["top_k"] = min(_log(rng, 1, 256), (hi + P - 1) // P)
    return base


def _spread(lo, hi, n):
    """n whole numbers evenly from lo to hi (one number: hi): the lengths of a ragged batch."""
    return np.rint(np.linspace(hi if n == 1 else lo, hi, n)).astype(np.int64)


def _pages(n, P):
    return -(-n // P)


def _lengths(case, rng, what="len"):
    x = _spread(case[what + "_lo"], case[what + "_hi"], case["B"])
    return rng.permutation(x)


def _cache(n_pages, Hkv, P, D, order, gen):
    """A paged cache [n_pages, Hkv, P, D]: head-major in memory ("hnd") or token-major ("nhd"). The
    values of a page lie around a centre of their own, as neighbouring tokens' do."""
    shape = (n_pages, Hkv, P, D) if order == "hnd" else (n_pages, P, Hkv, D)
    x = torch.empty(shape, device="cuda", dtype=torch.bfloat16).normal_(generator=gen)
    c = torch.empty((n_pages, Hkv, 1, D) if order == "hnd" else (n_pages, 1, Hkv, D), device="cuda",
                    dtype=torch.bfloat16).normal_(generator=gen)
    x.add_(c, alpha=0.5)
    return x if order == "hnd" else x.transpose(1, 2)


def prepare(case, seed):
    rng = np.random.default_rng(int(seed))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    kind, B, P = case["kind"], case["B"], case["P"]
    lens = _lengths(case, rng)
    dev = lambda x, t=torch.int32: torch.as_tensor(np.ascontiguousarray(x)).to(device="cuda", dtype=t)  # noqa: E731
    have = _pages(lens, P)
    s = dict(case=case, P=P, seq_lens=dev(lens))
    if kind in ("plan", "write"):
        new = _lengths(case, rng, "new")
        need = _pages(lens + new, P) - have
        max_pages = max(1, int(_pages(case["len_hi"] + case["new_hi"], P)))
        spare = max(1, int(_pages(new, P).sum()))  # enough for any order of the lengths
        free = min(spare, max(1, int(need.sum() * case.get("pool", 1.0))))
    else:
        max_pages, spare = max(1, int(have.max())), 3
    n_pages = int(have.sum()) + spare
    # every cached page anywhere in the pool, entries past a request's pages unset
    order = rng.permutation(n_pages)
    table = np.full((B, max_pages), -1, np.int64)
    table[np.arange(max_pages)[None, :] < have[:, None]] = order[:have.sum()]
    s.update(n_pages=n_pages, block_table=dev(table))
    if kind in ("plan", "write"):
        total = int(new.sum())
        s.update(new_lens=dev(new), free_pages=dev(order[have.sum():]), n_free=dev(np.array([free])),
                 max_tokens=max(1, total + case["spare"]))
    if kind == "plan":
        return s
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    s["k_cache"] = _cache(n_pages, Hkv, P, D, case["order"], gen)
    s["v_cache"] = _cache(n_pages, Hkv, P, D, case["order"], gen)
    if kind == "write":
        s["slots"] = _plan(s)[3]
        qkv = torch.empty((s["max_tokens"], Hq + 2 * Hkv, D), device="cuda", dtype=torch.bfloat16)
        qkv.normal_(generator=gen)
        s["k_new"], s["v_new"] = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["summary"] = torch.stack((s["k_cache"].amin(2), s["k_cache"].amax(2)), 2)
        return s
    s["q"] = torch.empty((B, Hq, D), device="cuda", dtype=torch.bfloat16).normal_(generator=gen).mul_(1.5)
    s["out_dtype"] = getattr(torch, case["out"])
    if kind == "sparse":
        s["top_k"] = case["top_k"]
        # a page's summary covers its valid rows: all, but for the last page of a request
        rows = torch.full((n_pages,), P, device="cuda", dtype=torch.int64)
        last = np.flatnonzero(have)
        rows[dev(table[last, have[last] - 1], torch.int64)] = dev((lens - (have - 1) * P)[last], torch.int64)
        out = (torch.arange(P, device="cuda")[None, :] >= rows[:, None])[:, None, :, None]
        lo = s["k_cache"].masked_fill(out, math.inf).amin(2)
        hi = s["k_cache"].masked_fill(out, -math.inf).amax(2)
        s["summary"] = torch.stack((lo, hi), 2)
    return s


# ---------------------------------------------------------------- the plain forms


def _plan(s):
    """Lengths after the step, free pages left, first token of each request, slots; the block table
    gains the granted pages in place."""
    P, table, n_pages = s["P"], s["block_table"], s["n_pages"]
    cap = table.shape[1] * P
    old = s["seq_lens"].long().clamp(0, cap)
    cu = s["new_lens"].long().clamp(min=0).cumsum(0).clamp(max=s["max_tokens"])
    cu = torch.cat((cu.new_zeros(1), cu))
    want = torch.minimum(old + cu.diff(), torch.full_like(old, cap))
    have = (old + P - 1) // P
    need = (want + P - 1) // P - have
    off = need.cumsum(0) - need
    free = s["n_free"].long().clamp(0, s["free_pages"].numel())
    got = torch.minimum((free - off).clamp(min=0), need)
    lens = torch.minimum(want, (have + got) * P)
    col = torch.arange(table.shape[1], device=table.device)[None, :] - have[:, None]
    fresh = (col >= 0) & (col < got[:, None])
    at = (free - 1 - off[:, None] - col).clamp(0, max(0, s["free_pages"].numel() - 1))
    table.copy_(torch.where(fresh, s["free_pages"][at], table))
    t = torch.arange(s["max_tokens"], device=table.device)
    b = torch.searchsorted(cu, t, right=True).sub(1).clamp(max=old.numel() - 1)
    pos = old[b] + t - cu[b]
    page = table[b, (pos // P).clamp(max=table.shape[1] - 1)].long()
    ok = (t < cu[-1]) & (pos < lens[b]) & (page >= 0) & (page < n_pages)
    slots = torch.where(ok, page * P + pos % P, -1)
    return lens.int(), (free - got.sum()).int(), cu.int(), slots


def _write(s):
    P, slots = s["P"], s["slots"]
    t = torch.nonzero(slots >= 0).flatten()
    page, row = slots[t] // P, slots[t] % P
    k_new = s["k_new"][t]
    s["k_cache"][page, :, row] = k_new
    s["v_cache"][page, :, row] = s["v_new"][t]
    begun = page[row == 0]
    kf = k_new.float()
    at = page[:, None, None].expand_as(kf)
    lo, hi = s["summary"][:, :, 0].float(), s["summary"][:, :, 1].float()
    lo[begun], hi[begun] = math.inf, -math.inf
    s["summary"][:, :, 0] = lo.scatter_reduce(0, at, kf, "amin").to(torch.bfloat16)
    s["summary"][:, :, 1] = hi.scatter_reduce(0, at, kf, "amax").to(torch.bfloat16)
    return s["k_cache"], s["v_cache"], s["summary"]


def _attend(s, pages, positions, dtype):
    """Attention over the rows of `pages` [B, Hkv, n] (physical; below 0: none), which hold the
    positions [B, Hkv, n * P]."""
    q, B, Hkv, P = s["q"], s["q"].shape[0], s["k_cache"].shape[1], s["P"]
    D, G = q.shape[2], q.shape[1] // Hkv
    head = torch.arange(Hkv, device=q.device)[None, :, None]
    at = pages.clamp(min=0)
    k = s["k_cache"][at, head].reshape(B, Hkv, -1, D).to(dtype)
    v = s["v_cache"][at, head].reshape(B, Hkv, -1, D).to(dtype)
    ok = (pages >= 0).repeat_interleave(P, 2) & (positions < s["seq_lens"][:, None, None])
    x = (q.reshape(B, Hkv, G, D).to(dtype) @ k.transpose(2, 3)) / math.sqrt(D)
    x = x.masked_fill(~ok[:, :, None], -math.inf)
    m = x.amax(3, keepdim=True).clamp(min=-1e30)
    e = torch.exp(x - m)
    z = e.sum(3, keepdim=True)
    o = (e / torch.where(z > 0, z, torch.ones_like(z))) @ v
    return o.reshape(B, -1, D), (m + torch.log(z)).reshape(B, -1)


def _decode(s, dtype=torch.float32):
    table, P, Hkv = s["block_table"].long(), s["P"], s["k_cache"].shape[1]
    pos = torch.arange(table.shape[1] * P, device=table.device)[None, None].expand(table.shape[0], Hkv, -1)
    o, lse = _attend(s, table[:, None].expand(-1, Hkv, -1), pos, dtype)
    return o.to(s["out_dtype"]), lse


def _select(s):
    """The listed pages of each request and key/value head. The scores are in 64 bits: the border
    between the last page in and the first one out may be a rounding wide."""
    table, q, P, top_k = s["block_table"].long(), s["q"], s["P"], s["top_k"]
    B, D, Hkv = q.shape[0], q.shape[2], s["summary"].shape[1]
    n = ((s["seq_lens"].long() + P - 1) // P).clamp(0, table.shape[1])[:, None, None]
    both = s["summary"][table.clamp(min=0)].permute(0, 2, 1, 3, 4).double()
    qg = q.reshape(B, Hkv, -1, D).double()
    x = qg.clamp(min=0) @ both[..., 1, :].transpose(2, 3) + qg.clamp(max=0) @ both[..., 0, :].transpose(2, 3)
    x = x.amax(2)
    i = torch.arange(table.shape[1], device=q.device)
    x = torch.where(i == n - 1, math.inf, torch.where(i < n, x, -math.inf))
    best = x.sort(dim=2, descending=True, stable=True)[1][:, :, :top_k]
    best = torch.where(torch.arange(best.shape[2], device=q.device) < n, best, table.shape[1])
    best = best.sort(2)[0]
    return torch.where(best < table.shape[1], best, -1)


def _sparse(s, dtype=torch.float32):
    pick = _select(s)
    table, P = s["block_table"].long(), s["P"]
    pages = table[:, None].expand(-1, pick.shape[1], -1).gather(2, pick.clamp(min=0))
    pos = (pick[..., None] * P + torch.arange(P, device=pick.device)).flatten(2)
    o, lse = _attend(s, torch.where(pick < 0, -1, pages), pos, dtype)
    return pick.int(), o.to(s["out_dtype"]), lse


# ---------------------------------------------------------------- the library's calls


def _own_plan(s, da):
    lens, n_free, cu, slots = da.paged_plan(s["new_lens"], s["seq_lens"], s["block_table"], s["free_pages"],
                                            s["n_free"], page_size=s["P"], n_pages=s["n_pages"],
                                            max_tokens=s["max_tokens"])
    return lens, n_free, cu, slots


def _own_write(s, da):
    da.paged_kv_write(s["k_new"], s["v_new"], s["slots"], s["k_cache"], s["v_cache"], summary=s["summary"])
    return s["k_cache"], s["v_cache"], s["summary"]


def _own_decode(s, da, selected=None):
    return da.paged_attn_fwd(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"],
                             selected=selected, out_dtype=s["out_dtype"])


def _own_sparse(s, da):
    pick = da.paged_select(s["q"], s["summary"], s["block_table"], s["seq_lens"], page_size=s["P"],
                           top_k=s["top_k"])
    return (pick, *_own_decode(s, da, pick))


def run(state):
    kind = state["case"]["kind"]
    if own:
        from diffusion_transformer_long_gb300 import ditattn as da
        call = {"plan": _own_plan, "write": _own_write, "decode": _own_decode, "sparse": _own_sparse}
        r = call[kind](state, da)
    else:
        r = {"plan": _plan, "write": _write, "decode": _decode, "sparse": _sparse}[kind](state)
    return (*r, state["block_table"]) if kind == "plan" else r


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    B, P = case["B"], case["P"]
    lens = _spread(case["len_lo"], case["len_hi"], B)
    if case["kind"] == "plan":
        # lengths and new lengths in; lengths, first tokens out; every slot; every granted page read
        # from the stack and written to the table (at most: the two lists' order is the seed's)
        new = _spread(case["new_lo"], case["new_hi"], B)
        total = int(new.sum())
        grant = _pages(total, P)
        return {"bytes": 4 * (4 * B + 3) + 8 * (total + case["spare"]) + 8 * grant, "flops": total}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["kind"] == "write":
        total = int(_spread(case["new_lo"], case["new_hi"], B).sum())
        pages = _pages(total, P)
        return {"bytes": total * (8 + 2 * 2 * Hkv * D * 2) + pages * Hkv * 2 * D * 2, "flops": 2 * total * Hkv * D}
    out = 4 if case["out"] == "float32" else 2
    io = B * (Hq * D * (2 + out) + Hq * 4 + 4)
    n = _pages(lens, P)
    if case["kind"] == "decode":
        rows = int(lens.sum()) * Hkv
        return {"bytes": rows * D * 4 + io + 4 * int(n.sum()), "flops": 4 * rows * (Hq // Hkv) * D}
    k = np.minimum(n, case["top_k"])
    rows = int(np.minimum(lens, k * P).sum()) * Hkv
    pages = int(n.sum()) * Hkv
    return {"bytes": rows * D * 4 + pages * 2 * D * 2 + io + 4 * (int(n.sum()) + Hkv * B * case["top_k"]),
            "flops": 4 * rows * (Hq // Hkv) * D + 4 * pages * (Hq // Hkv) * D}


# ---------------------------------------------------------------- the definition in 64 bits


def _exact_write(s):
    """Row by row in the slots' order on flat copies, then each page's extremes from the rows it
    holds: those written now, or those and its earlier summary."""
    P, slots = s["P"], s["slots"].cpu().numpy()
    order = np.flatnonzero(slots >= 0)
    t = torch.as_tensor(order).cuda()
    res = []
    for new, cache in ((s["k_new"], s["k_cache"]), (s["v_new"], s["v_cache"])):
        flat = cache.permute(0, 2, 1, 3).double().reshape(-1, *new.shape[1:])
        flat[torch.as_tensor(slots[order]).cuda()] = new[t].double()
        res.append(flat.reshape(-1, P, *new.shape[1:]).permute(0, 2, 1, 3))
    summary = s["summary"].double()
    pages = slots[order] // P
    first = np.flatnonzero(np.diff(pages, prepend=-1))
    for i, j in zip(first, np.append(first[1:], len(order))):
        lo_row, p = int(slots[order[i]] % P), int(pages[i])
        rows = res[0][p, :, lo_row:lo_row + int(j - i)]
        ext = torch.stack((rows.amin(1), rows.amax(1)), 1)
        if lo_row:
            ext = torch.stack((torch.minimum(ext[:, 0], summary[p, :, 0]),
                               torch.maximum(ext[:, 1], summary[p, :, 1])), 1)
        summary[p] = ext
    return (*res, summary)


def _exact_request(s, b, pick):
    """One request: its keys and values by position, in 64 bits; softmax by its definition."""
    P, Hkv, D = s["P"], s["k_cache"].shape[1], s["q"].shape[2]
    n = int(s["seq_lens"][b])
    q = s["q"][b].double().reshape(Hkv, -1, D)
    pages = s["block_table"][b, :_pages(n, P)].long()
    k, v = (x[pages].permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :n] for x in (s["k_cache"], s["v_cache"]))
    listed_pages = torch.full((Hkv, s.get("top_k", 1)), -1, dtype=torch.int32, device="cuda")
    if n == 0:
        return listed_pages, q * 0, torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    w = torch.einsum("hgd,hnd->hgn", q, k.double()) * D ** -0.5
    if pick:
        lo, hi = s["summary"][pages].double().permute(2, 1, 0, 3)
        score = torch.stack([torch.maximum(q[:, g, None] * lo, q[:, g, None] * hi).sum(2)
                             for g in range(q.shape[1])]).amax(0)
        score[:, -1] = math.inf
        rank = torch.argsort(-score, dim=1, stable=True)[:, :s["top_k"]].sort(1)[0]
        listed_pages[:, :rank.shape[1]] = rank.int()
        keep = torch.zeros_like(score, dtype=torch.bool).scatter_(1, rank, True)
        w = w.masked_fill(~keep.repeat_interleave(P, 1)[:, None, :n], -math.inf)
    return listed_pages, torch.softmax(w, 2) @ v.double(), torch.logsumexp(w, 2)


def exact(case, seed):
    if case["kind"] == "plan":
        return None
    s = prepare(case, seed)
    if case["kind"] == "write":
        return _exact_write(s)
    rows = [_exact_request(s, b, case["kind"] == "sparse") for b in range(case["B"])]
    o, lse = torch.stack([r[1].flatten(0, 1) for r in rows]), torch.stack([r[2].flatten() for r in rows])
    return (torch.stack([r[0] for r in rows]), o, lse) if case["kind"] == "sparse" else (o, lse)
