"""Prompts over the paged key/value cache, as measured cases: the norms and rotary positions that
queries and keys take before the cache, the attention of a step's new tokens over the pages, the
weight that each page has drawn, and the eviction of the pages that drew least.

Four kinds of case, one operator each:

rope     y = rot(w x / sqrt(mean_d x_d^2 + eps)) of each head of q and k; rot turns pair i of the first
         2 n channels, (2 i, 2 i + 1) or (i, i + n), by the angle pos_a(i) f_i, where a(i) is the position
         axis of the pair, and scales them by one number.
prefill  the n_b newest of request b's seq_lens[b] cached tokens attend to the cache: token i at position
         p = start_b + i to the keys j <= p (causal) or to all: o = softmax_j(scale q . k_j) v_j,
         lse = ln sum_j exp(scale q . k_j); the query heads of a group share a key/value head.
mass     for each page and key/value head the attention weight exp(scale q . k_j - lse) of its keys,
         summed over the keys, the group's heads and the step's last `window` queries, added to what the
         page had drawn; a page whose first key is new starts from nothing.
evict    a request of more than `keep` pages keeps its newest `recent` ones and, of the others, those of
         most weight over all heads (ties: the lowest index), in order; the others go back to the stack.

`own` False computes each in elementary torch operations; True calls the library.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6

# Head layouts are this repository's workloads' (24 or 40 heads of 128, 2 heads of 64) or grouped forms
# of them; lengths are its token counts (512, 1024, 4608, 27280, 75600) and parts of them. The position
# axes are a token index alone, or a video's frame, row and column.


def listed():
    return [
        # the smallest rotation: one token for each request of a decode batch, queries and keys as slices of
        # one projection, half of each head rotated, positions stretched for a long context
        dict(name="rope decode 64", kind="rope", B=64, T=64, Hq=24, Hkv=8, D=128, rot=64, axes=1, inter=False, norm=True,
             order="packed", scaling="yarn", far=1000000),
        # an image's queries and keys, token-major as projected, head-major for the attention
        dict(name="rope image 4608", kind="rope", B=1, T=4608, Hq=24, Hkv=24, D=128, rot=128, axes=3, inter=True,
             norm=True, order="bhnd", scaling="none", far=64),
        # one video's queries and keys, all heads
        dict(name="rope video 75600", kind="rope", B=1, T=75600, Hq=40, Hkv=40, D=128, rot=128, axes=3, inter=True,
             norm=True, order="bhnd", scaling="none", far=80),
        # the smallest attention: a few short prompts
        dict(name="prefill short d64", kind="prefill", B=4, Hq=2, Hkv=2, D=64, P=16, old_lo=0, old_hi=512, new_lo=1,
             new_hi=64, causal=True, order="hnd", spare=0),
        # a few candidate tokens for each of several long contexts: the keys' length is what there is to split
        dict(name="prefill verify 4x75600", kind="prefill", B=4, Hq=40, Hkv=8, D=128, P=64, old_lo=30001, old_hi=75595,
             new_lo=5, new_hi=5, causal=True, order="hnd", spare=0),
        # an ordinary step: chunks of prompts behind caches of any length, its batch padded
        dict(name="prefill ragged 16", kind="prefill", B=16, Hq=24, Hkv=8, D=128, P=16, old_lo=0, old_hi=4608, new_lo=1,
             new_hi=1024, causal=True, order="nhd", spare=37),
        # one whole prompt
        dict(name="prefill one 27280", kind="prefill", B=1, Hq=24, Hkv=8, D=128, P=64, old_lo=0, old_hi=0, new_lo=27280,
             new_hi=27280, causal=True, order="hnd", spare=0),
        # a block of video tokens that sees itself and all blocks before it
        dict(name="prefill block 4608", kind="prefill", B=1, Hq=24, Hkv=24, D=128, P=128, old_lo=22672, old_hi=22672,
             new_lo=4608, new_hi=4608, causal=False, order="hnd", spare=0),
        # one token for each request of a ragged decode batch
        dict(name="mass decode 48", kind="mass", B=48, Hq=24, Hkv=8, D=128, P=32, old_lo=0, old_hi=4607, new_lo=1,
             new_hi=1, window=1, order="hnd"),
        # a prompt's last queries observe a long cache
        dict(name="mass window 2x75600", kind="mass", B=2, Hq=40, Hkv=8, D=128, P=64, old_lo=74576, old_hi=74576,
             new_lo=1024, new_hi=1024, window=16, order="hnd"),
        # a batch of long contexts down to a budget
        dict(name="evict 16x75600", kind="evict", B=16, Hkv=8, P=16, len_lo=30001, len_hi=75600, keep=2048, recent=64),
        # a large batch of short ones, some within the budget
        dict(name="evict 256x4608", kind="evict", B=256, Hkv=24, P=64, len_lo=0, len_hi=4608, keep=40, recent=4),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = ((24, 24, 128), (24, 8, 128), (40, 8, 128), (40, 40, 128), (2, 2, 64), (16, 1, 64), (24, 2, 128), (24, 1, 128))
MOST_FLOPS = 4e12   # below the largest listed prefill's
MOST_KEYS = 2 * 75600 * 8 * 128   # cached elements, at most the largest listed cases'


def draw(rng):
    kind = rng.choice(("rope", "rope", "prefill", "prefill", "prefill", "mass", "evict"))
    Hq, Hkv, D = rng.choice(HEADS)
    P = rng.choice((16, 32, 48, 64, 128))
    if kind == "rope":
        axes = rng.choice((1, 3))
        T = _log(rng, 1, min(75600, 75600 * 80 * 128 // ((Hq + Hkv) * D)))
        rot = D if axes == 3 else rng.choice((16, 32, D // 2, D - 16, D))
        return dict(kind=kind, B=_log(rng, 1, min(T, 64)) if axes == 1 else 1, T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rot,
                    axes=axes, inter=rng.choice((True, False)), norm=rng.choice((True, True, False)),
                    order="packed" if axes == 1 else "bhnd",
                    scaling=rng.choice(("none", "linear", "ntk", "yarn")) if axes == 1 else "none",
                    far=_log(rng, 16, 1000000) if axes == 1 else rng.randrange(8, 100))
    if kind == "evict":
        B = _log(rng, 1, 1024)
        hi = _log(rng, 1, min(75600, 16 * 75600 // B))
        n = -(-hi // P)
        keep = _log(rng, 1, max(1, n))
        return dict(kind=kind, B=B, Hkv=Hkv, P=P, len_lo=rng.randrange(0, hi + 1), len_hi=hi, keep=keep,
                    recent=rng.randrange(1, keep + 1))
    B = _log(rng, 1, 64)
    hi = _log(rng, 1, min(75600, max(1, MOST_KEYS // (B * Hkv * D))))
    order = rng.choice(("hnd", "nhd"))
    base = dict(kind=kind, B=B, Hq=Hq, Hkv=Hkv, D=D, P=P, order=order)
    if kind == "mass":
        new = 1 if rng.random() < 0.5 else _log(rng, 1, 512)
        window = 1 if new == 1 else _log(rng, 1, 16)
        return dict(base, old_lo=rng.randrange(0, hi + 1), old_hi=hi, new_lo=rng.randrange(1, new + 1), new_hi=new,
                    window=window)
    most = max(1, int(MOST_FLOPS / (4 * B * Hq * D * hi)))
    new = min(_log(rng, 1, 27280), most, 27280 * 24 * 128 // (B * Hq * D) + 1, max(1, hi))
    return dict(base, old_lo=rng.randrange(0, hi - new + 1), old_hi=hi - new, new_lo=rng.randrange(0, new + 1),
                new_hi=new, causal=rng.random() < 0.75, spare=rng.choice((0, 1, 37)))


def _spread(lo, hi, n):
    """n whole numbers evenly from lo to hi (one number: hi): the lengths of a ragged batch."""
    return np.rint(np.linspace(hi if n == 1 else lo, hi, n)).astype(np.int64)


def _dev(x, t=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x)).to(device="cuda", dtype=t)


def _normal(shape, gen, dtype=torch.bfloat16):
    return torch.empty(shape, device="cuda", dtype=dtype).normal_(generator=gen)


def _cache(n_pages, Hkv, P, D, order, gen):
    """A paged cache [n_pages, Hkv, P, D]: head-major in memory ("hnd") or token-major ("nhd"). The
    values of a page lie around a centre of their own, as neighbouring tokens' do."""
    hnd = order == "hnd"
    x = _normal((n_pages, Hkv, P, D) if hnd else (n_pages, P, Hkv, D), gen)
    x.add_(_normal((n_pages, Hkv, 1, D) if hnd else (n_pages, 1, Hkv, D), gen), alpha=0.5)
    return x if hnd else x.transpose(1, 2)


def _frequencies(case):
    """(angle per position of each pair, in 32 bits; the axes' pairs; the rotation's scale)."""
    n = case["rot"] // 2
    if case["axes"] == 3:  # frame, row, column: 44, 42, 42 channels of 128
        each = [n - 2 * (n // 3), n // 3, n // 3]
        return np.concatenate([10000.0 ** (-np.arange(m) / m) for m in each]), each, 1.0
    theta, i = 10000.0, np.arange(n)
    if case["scaling"] == "ntk":  # a larger base: the slowest pair is stretched eightfold, the fastest not
        theta *= 8.0 ** (n / max(1, n - 1))
    f = theta ** (-i / n)
    if case["scaling"] == "linear":
        f = f / 8
    if case["scaling"] == "yarn":  # pairs of few turns in 4096 positions are stretched, those of many not
        turns = 4096 * f / (2 * math.pi)
        keep = np.clip((turns - 1) / (32 - 1), 0, 1)
        return f * (keep + (1 - keep) / 8), [n], 0.1 * math.log(8) + 1
    return f, [n], 1.0


def prepare(case, seed):
    rng = np.random.default_rng(int(seed))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    return {"rope": _prepare_rope, "evict": _prepare_evict}.get(case["kind"], _prepare_cached)(case, rng, gen)


def _prepare_rope(case, rng, gen):
    T, Hq, Hkv, D, B = (case[x] for x in ("T", "Hq", "Hkv", "D", "B"))
    f, each, scale = _frequencies(case)
    s = dict(case=case, freqs=_dev(f, torch.float32), axis_pairs=each, rot_scale=scale)
    qkv = _normal((T, Hq + 2 * Hkv, D), gen)
    qkv.mul_(torch.rand((1, Hq + 2 * Hkv, 1), device="cuda", generator=gen).mul_(3).add_(0.3).bfloat16())
    s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
    if case["norm"]:
        s["q_weight"], s["k_weight"] = (_normal((D,), gen, torch.float32).mul_(0.2).add_(1).bfloat16() for _ in range(2))
    if case["axes"] == 3:
        # tokens of a video in raster order, rows and columns of the plane below `far`
        far = case["far"]
        t = np.arange(T)
        s["positions"] = _dev(np.stack((t // (far * far), t // far % far, t % far)))
        return s
    new = np.bincount(rng.integers(0, B, T - B), minlength=B) + 1 if T > B else np.ones(B, np.int64)
    s["cu_new"] = _dev(np.concatenate(([0], np.cumsum(new))))
    s["start_lens"] = _dev(rng.integers(0, case["far"], B))
    return s


def _table(lens, P, n_pages, rng):
    """Every request's pages anywhere in the pool; entries past them are unset."""
    have = -(-lens // P)
    order = rng.permutation(n_pages)
    table = np.full((len(lens), max(1, int(have.max()))), -1, np.int64)
    table[np.arange(table.shape[1])[None, :] < have[:, None]] = order[:have.sum()]
    return table, order[have.sum():]


def _prepare_evict(case, rng, gen):
    lens = rng.permutation(_spread(case["len_lo"], case["len_hi"], case["B"]))
    used = int((-(-lens // case["P"])).sum())
    n_pages = used + 5
    table, free = _table(lens, case["P"], n_pages, rng)
    # drawn weight: a few pages drew most of it
    mass = torch.empty((n_pages, case["Hkv"]), device="cuda").exponential_(generator=gen).pow_(3)
    stack = np.zeros(n_pages, np.int64)
    stack[:5] = free
    return dict(case=case, n_pages=n_pages, seq_lens=_dev(lens), block_table=_dev(table), mass=mass,
                free_pages=_dev(stack), n_free=_dev(np.array([5])), table_out=torch.zeros_like(_dev(table)))


def _prepare_cached(case, rng, gen):
    B, Hq, Hkv, D, P = (case[x] for x in ("B", "Hq", "Hkv", "D", "P"))
    old = rng.permutation(_spread(case["old_lo"], case["old_hi"], B))
    new = rng.permutation(_spread(case["new_lo"], case["new_hi"], B))
    n_pages = int((-(-(old + new) // P)).sum()) + 3
    table, _ = _table(old + new, P, n_pages, rng)
    T = max(1, int(new.sum()) + case.get("spare", 0))
    cu = np.concatenate(([0], np.cumsum(new)))
    s = dict(case=case, seq_lens=_dev(old + new), block_table=_dev(table), cu_new=_dev(cu),
             k_cache=_cache(n_pages, Hkv, P, D, case["order"], gen),
             # host copies, as a scheduler holds them: (first row, new tokens, cached tokens) of each request
             requests=[(int(cu[b]), int(new[b]), int(old[b] + new[b])) for b in range(B)])
    qkv = _normal((T, Hq + 2 * Hkv, D), gen)
    s["q"] = qkv[:, :Hq].mul_(1.5)
    if case["kind"] == "prefill":
        s["v_cache"] = _cache(n_pages, Hkv, P, D, case["order"], gen)
        s["out"] = torch.zeros((T, Hq, D), device="cuda", dtype=torch.bfloat16)
        s["lse"] = torch.zeros((T, Hq), device="cuda")
        return s
    # the attention's lse for the queries that observe, and the weight drawn before
    s["lse"] = torch.zeros((T, Hq), device="cuda")
    for b, (row, n, length) in enumerate(s["requests"]):
        w = min(n, case["window"])
        x = _scores(s, b, length, row + n - w, w, torch.float32)
        s["lse"][row + n - w:row + n] = torch.logsumexp(x, 3).permute(2, 0, 1).reshape(w, Hq)
    s["mass"] = torch.empty((n_pages, Hkv), device="cuda").exponential_(generator=gen)
    s["mass_out"] = s["mass"].clone()
    return s


# ---------------------------------------------------------------- the plain forms


def _rope_rows(s, x, weight):
    """x [T, H, D] normed and rotated, in 32 bits; angles in 64."""
    case = s["case"]
    x = x.float()
    if case["norm"]:
        x = x * torch.rsqrt((x * x).mean(2, keepdim=True) + EPS) * weight.float()
    n = case["rot"] // 2
    if case["axes"] == 1:
        t = torch.arange(case["T"], device=x.device)
        b = torch.searchsorted(s["cu_new"][1:].long(), t, right=True)
        at = (s["start_lens"].long()[b] + t - s["cu_new"].long()[b])[:, None].expand(-1, n)
    else:
        axis = torch.repeat_interleave(torch.tensor(s["axis_pairs"]))
        at = s["positions"].long()[axis.to(x.device)].t()
    angle = at.double() * s["freqs"].double()
    cos, sin = ((f(angle) * s["rot_scale"]).float()[:, None] for f in (torch.cos, torch.sin))
    if case["inter"]:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), 3).flatten(2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), 2)
    y = torch.cat((y, x[..., 2 * n:]), 2).to(torch.bfloat16)
    return y.transpose(0, 1).contiguous()[None] if case["order"] == "bhnd" else y


def _rope(s):
    return _rope_rows(s, s["q"], s.get("q_weight")), _rope_rows(s, s["k"], s.get("k_weight"))


def _keys(s, name, b, length, dtype):
    """Request b's cached keys or values by position: [Hkv, length, D]."""
    P = s["case"]["P"]
    pages = s["block_table"][b, :-(-length // P)].long()
    x = s[name][pages].transpose(0, 1)
    return x.reshape(x.shape[0], -1, x.shape[3])[:, :length].to(dtype)


def _scores(s, b, length, row, n, dtype, keys=None, first=0):
    """scale q . k of the n tokens from row `row` on: [Hkv, G, n, keys], -inf where a token does not see.
    The tokens' positions end `first` before the request's last one."""
    case = s["case"]
    k = _keys(s, "k_cache", b, length, dtype) if keys is None else keys
    q = s["q"][row:row + n].to(dtype).unflatten(1, (case["Hkv"], -1)).permute(1, 2, 0, 3)
    x = (q.flatten(1, 2) @ k.transpose(1, 2)).unflatten(1, (-1, n)) / math.sqrt(case["D"])
    if case.get("causal", True):
        at = torch.arange(length - first - n, length - first, device=x.device)
        x.masked_fill_(torch.arange(k.shape[1], device=x.device)[None, :] > at[:, None], -math.inf)
    return x


def _prefill(s):
    case = s["case"]
    Hq, D = case["Hq"], case["D"]
    out, lse = torch.zeros_like(s["out"]), torch.zeros_like(s["lse"])
    for b, (row, n, length) in enumerate(s["requests"]):
        if n == 0:
            continue
        k, v = (_keys(s, x, b, length, torch.float32) for x in ("k_cache", "v_cache"))
        step = max(1, min(n, (1 << 28) // (Hq * length)))  # tokens whose scores are held at once
        for i in range(0, n, step):
            m = min(step, n - i)
            end = length - n + i + m if case["causal"] else length
            x = _scores(s, b, length, row + i, m, torch.float32, k[:, :end], n - i - m)
            top = x.amax(3, keepdim=True)
            e = x.sub_(top).exp_()
            z = e.sum(3, keepdim=True)
            o = (e.flatten(1, 2) @ v[:, :end]).unflatten(1, (-1, m)) / z
            out[row + i:row + i + m] = o.permute(2, 0, 1, 3).reshape(m, Hq, D).to(out.dtype)
            lse[row + i:row + i + m] = (top + z.log())[..., 0].permute(2, 0, 1).reshape(m, Hq)
    return out, lse


def _mass(s):
    case, P = s["case"], s["case"]["P"]
    res = s["mass"].clone()
    for b, (row, n, length) in enumerate(s["requests"]):
        w = min(n, case["window"])
        x = _scores(s, b, length, row + n - w, w, torch.float32)
        lse = s["lse"][row + n - w:row + n].unflatten(1, (case["Hkv"], -1)).permute(1, 2, 0)
        e = x.sub_(lse[..., None]).exp_().sum((1, 2))  # [Hkv, length]
        e = torch.nn.functional.pad(e, (0, -length % P)).unflatten(1, (-1, P)).sum(2).t()
        pages = s["block_table"][b, :e.shape[0]].long()
        begun = torch.arange(e.shape[0], device=e.device) * P >= length - n
        res[pages] = torch.where(begun[:, None], e, res[pages] + e)
    return res


def _evict(s):
    """(table, lengths, stack, pages on it); all requests at once."""
    case, P, keep, recent = s["case"], s["case"]["P"], s["case"]["keep"], s["case"]["recent"]
    table, lens = s["block_table"].long(), s["seq_lens"].long()
    i = torch.arange(table.shape[1], device=table.device)
    n = ((lens + P - 1) // P)[:, None]
    x = s["mass"].double().sum(1)[table.clamp(min=0)]
    x = torch.where(i >= n, -math.inf, torch.where(i >= n - recent, math.inf, x))
    rank = x.sort(dim=1, descending=True, stable=True)[1].argsort(1)
    kept = (rank < keep) & (i < n)
    at = torch.where(kept, i, table.shape[1]).sort(1)[0]
    table_out = torch.where(at < table.shape[1], table.gather(1, at.clamp(max=table.shape[1] - 1)), -1)
    gone = table[(i < n) & ~kept]
    stack = s["free_pages"].clone()
    n_free = s["n_free"]
    put = n_free.long() + torch.arange(gone.shape[0], device=table.device)
    stack[put] = gone.int()
    left = lens - P * ((i < n) & ~kept).sum(1)
    return table_out.int(), left.int(), stack, n_free + gone.shape[0]


# ---------------------------------------------------------------- the library's calls


def _own_rope(s, da):
    case = s["case"]
    kw = dict(freqs=s["freqs"], interleaved=case["inter"], rot_scale=s["rot_scale"], eps=EPS if case["norm"] else None,
              q_weight=s.get("q_weight"), k_weight=s.get("k_weight"))
    if case["order"] == "bhnd":
        q, k = (x.transpose(0, 1)[None] for x in (s["q"], s["k"]))
        return da.qk_norm_rope(q, k, positions=s["positions"], axis_pairs=s["axis_pairs"], **kw)
    return da.qk_norm_rope(s["q"], s["k"], cu_new=s["cu_new"], start_lens=s["start_lens"], **kw)


def _own_prefill(s, da):
    return da.paged_prefill_fwd(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"], s["cu_new"],
                                causal=s["case"]["causal"], out=s["out"], lse=s["lse"])


def _own_mass(s, da):
    return da.paged_page_mass(s["q"], s["lse"], s["k_cache"], s["block_table"], s["seq_lens"], s["mass"],
                              cu_new=s["cu_new"], window=s["case"]["window"], mass_out=s["mass_out"])


def _own_evict(s, da):
    lens, n_free = da.paged_evict(s["mass"], s["block_table"], s["seq_lens"], s["free_pages"], s["n_free"],
                                  page_size=s["case"]["P"], keep=s["case"]["keep"], recent=s["case"]["recent"],
                                  table_out=s["table_out"])
    return s["table_out"], lens, s["free_pages"], n_free


def run(state):
    kind = state["case"]["kind"]
    if own:
        from diffusion_transformer_long_gb300 import ditattn as da
        return {"rope": _own_rope, "prefill": _own_prefill, "mass": _own_mass, "evict": _own_evict}[kind](state, da)
    return {"rope": _rope, "prefill": _prefill, "mass": _mass, "evict": _evict}[kind](state)


# ---------------------------------------------------------------- what a pass cannot do without


def _pairs(n, length, causal):
    """(query, key) pairs of n new tokens that end a request of `length`."""
    return n * length - (n * (n - 1) // 2 if causal else 0)


def work(case):
    if case["kind"] == "rope":
        T, H, D = case["T"], case["Hq"] + case["Hkv"], case["D"]
        pos = 4 * T * case["axes"] if case["axes"] > 1 else 8 * case["B"]
        return {"bytes": T * H * D * 4 + pos + 2 * case["rot"] + 4 * D, "flops": T * H * (4 * D + 3 * case["rot"])}
    B, P, Hkv = case["B"], case["P"], case["Hkv"]
    if case["kind"] == "evict":
        n = -(-_spread(case["len_lo"], case["len_hi"], B) // P)
        gone = int(np.maximum(0, n - case["keep"]).sum())
        kept = int(np.minimum(n, case["keep"]).sum())
        # every page's weight and table entry in; the kept entries and the dropped ones out, lengths in and out
        return {"bytes": int(n.sum()) * (4 * Hkv + 4) + 4 * (kept + gone) + 8 * B, "flops": int(n.sum()) * Hkv}
    Hq, D = case["Hq"], case["D"]
    old, new = (_spread(case[x + "_lo"], case[x + "_hi"], B) for x in ("old", "new"))
    lens = old + new  # (which length meets which is the seed's: the sums are of these)
    keys, pages = int(lens.sum()) * Hkv, int((-(-lens // P)).sum())
    if case["kind"] == "mass":
        w = np.minimum(new, case["window"])
        pairs = sum(_pairs(int(a), int(b), True) for a, b in zip(w, lens))
        return {"bytes": keys * D * 2 + int(w.sum()) * Hq * (2 * D + 4) + pages * (8 * Hkv + 4),
                "flops": pairs * Hq * 2 * D}
    T = int(new.sum())
    pairs = sum(_pairs(int(a), int(b), case["causal"]) for a, b in zip(new, lens))
    return {"bytes": keys * D * 4 + T * Hq * (4 * D + 4) + 4 * pages, "flops": pairs * Hq * 4 * D}


# ---------------------------------------------------------------- the definition in 64 bits


def _exact_rope(s):
    case = s["case"]
    n, T = case["rot"] // 2, case["T"]
    if case["axes"] == 1:
        cu, start = s["cu_new"].cpu().numpy().astype(np.int64), s["start_lens"].cpu().numpy().astype(np.int64)
        at = np.concatenate([start[b] + np.arange(cu[b + 1] - cu[b]) for b in range(case["B"])])
        angle = at[:, None] * s["freqs"].cpu().double().numpy()[None]
    else:
        at = np.repeat(s["positions"].cpu().numpy().astype(np.float64), s["axis_pairs"], axis=0)
        angle = at.T * s["freqs"].cpu().double().numpy()
    # a rotation is a product with a unit complex number
    turn = torch.polar(torch.full((T, n), s["rot_scale"], dtype=torch.float64), torch.as_tensor(angle)).cuda()[:, None]
    res = []
    for name in ("q", "k"):
        y = s[name].double()
        if case["norm"]:
            y = y / torch.sqrt(y.square().sum(2, keepdim=True) / case["D"] + EPS) * s[name + "_weight"].double()
        first = slice(0, 2 * n, 2) if case["inter"] else slice(0, n)
        second = slice(1, 2 * n, 2) if case["inter"] else slice(n, 2 * n)
        z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
        y[..., first], y[..., second] = z.real, z.imag
        res.append(y.permute(1, 0, 2)[None] if case["order"] == "bhnd" else y)
    return tuple(res)


def _exact_head(s, b, h, name):
    """Keys or values of request b, head h, row by row through the table, in 64 bits."""
    P, length = s["case"]["P"], s["requests"][b][2]
    j = torch.arange(length, device="cuda")
    return s[name][s["block_table"][b].long()[j // P], h, j % P].double()


def _exact_prefill(s):
    case = s["case"]
    G, D = case["Hq"] // case["Hkv"], case["D"]
    out, lse = (torch.zeros(s[x].shape, dtype=torch.float64, device="cuda") for x in ("out", "lse"))
    for b, (row, n, length) in enumerate(s["requests"]):
        j = torch.arange(length, device="cuda")
        for h in range(case["Hq"]):
            if n == 0:
                continue
            if h % G == 0:
                k, v = (_exact_head(s, b, h // G, x) for x in ("k_cache", "v_cache"))
            for i in range(0, n, 2048):
                at = torch.arange(i, min(n, i + 2048), device="cuda")
                see = j[None, :] <= (length - n + at)[:, None] if case["causal"] else (j < length)[None]
                end = min(length, length - n + int(at.numel()) + i) if case["causal"] else length
                w = (s["q"][row + at, h].double() @ k[:end].T) * D ** -0.5
                w = torch.where(see[:, :end], w, -math.inf)
                out[row + at, h] = torch.softmax(w, 1) @ v[:end]
                lse[row + at, h] = torch.logsumexp(w, 1)
    return out, lse


def _exact_mass(s):
    case, P = s["case"], s["case"]["P"]
    G = case["Hq"] // case["Hkv"]
    res = s["mass"].double()
    for b, (row, n, length) in enumerate(s["requests"]):
        page = s["block_table"][b].long()[torch.arange(-(-length // P), device="cuda")]
        res[page[-(-(length - n) // P):]] = 0  # pages whose first key is new
        for g in range(case["Hkv"]):
            k = _exact_head(s, b, g, "k_cache")
            total = torch.zeros(length, dtype=torch.float64, device="cuda")
            for t in range(n - min(n, case["window"]), n):
                seen = length - n + t + 1
                for h in range(g * G, (g + 1) * G):
                    w = (k[:seen] @ s["q"][row + t, h].double()) * case["D"] ** -0.5
                    total[:seen] += torch.exp(w - s["lse"][row + t, h].double())
            res[:, g].index_add_(0, page[torch.arange(length, device="cuda") // P], total)
    return res


def exact(case, seed):
    if case["kind"] == "evict":
        return None
    s = prepare(case, seed)
    return {"rope": _exact_rope, "prefill": _exact_prefill, "mass": _exact_mass}[case["kind"]](s)
