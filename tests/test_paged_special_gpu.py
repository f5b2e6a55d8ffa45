"""The paged attention and selection where scores or values are no ordinary numbers, or of very different sizes: what
the definition makes of them, whatever launch, grid and split of the keys a call gets."""
import math

import numpy as np
import pytest
import torch

import paged_oracle as po
from diffusion_transformer_long_gb300 import ditattn as da
from test_paged_gpu import check_attn, dev, launch, make_case, rand, tables, widened  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[0, 1000, 1, 3, 50], ids=lambda g: f"grid {g}")
def grid(request):
    """The launch that the sizes choose (0), the one for many items, and that on capped grids."""
    da.set_grid_limit(request.param)
    yield request.param
    da.set_grid_limit(0)


def check_with_nan(o, lse, ref):
    """NaN where the 64-bit form has it (whole rows: a score is NaN), its values elsewhere."""
    o_ref, lse_ref, (mag, pv) = ref
    none = np.isnan(lse_ref)
    assert np.array_equal(np.isnan(lse.cpu().numpy()), none)
    assert o.isnan().cpu().numpy()[none].all() and not o.isnan().cpu().numpy()[~none].any()
    o, lse = o.masked_fill(torch.as_tensor(none, device=o.device)[..., None], 0), lse.nan_to_num(0, math.inf, -math.inf)
    for x in (o_ref, lse_ref, mag, pv):
        x[none] = 0
    check_attn(o, lse, ref)


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("what", ["query", "key", "page", "first part", "last part", "all keys", "infinite"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,P", [([1, 40, 0], 4, 2, 64, 16), ([4000, 300, 17], 6, 2, 128, 16),
                                             ([9000], 3, 1, 64, 64), ([700, 90], 24, 1, 128, 32)])
def test_nan_scores_show(lens, Hq, Hkv, D, P, what, selected, grid):
    q, k, v, table, sl = make_case(lens, Hq, Hkv, D, P, seed=len(lens))
    n = -(-lens[0] // P)  # request 0's pages
    pages = table[0, :n].long()
    if what == "query":
        q[0, 1, 3] = float("nan")
        q[-1, Hq - 1, D - 1] = float("nan")  # (in a request without keys: not seen)
    elif what == "key":
        k[pages[n // 2], 0, 0, 5] = float("nan")
    elif what == "infinite":  # a score of +inf: inf - inf
        q[0, :, 5] = 1.0
        k[pages[n // 2], 0, 0, 5] = float("inf")
    else:
        part = dict(page=pages[n // 2:n // 2 + 1])
        part.update({"first part": pages[:(n + 2) // 3], "last part": pages[n // 3:], "all keys": pages})
        k[part[what], Hkv - 1, :, 7] = float("nan")
    sel = None
    if selected:
        m = table.shape[1]
        sel = torch.arange(m, device=q.device, dtype=torch.int32).expand(len(lens), Hkv, m).contiguous()
    with np.errstate(invalid="ignore"):
        ref = po.attend(q, k, v, table, sl, D ** -0.5, selected=sel)
    assert np.isnan(ref[1][0]).any()
    check_with_nan(*da.paged_attn_fwd(q, k, v, table, sl, selected=sel), ref)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("lens,Hq,Hkv,D,P", [([40, 1], 4, 2, 64, 16), ([4000, 300], 6, 2, 128, 16), ([9000], 3, 1, 64, 64)])
def test_values_behind_scores_of_minus_infinity(lens, Hq, Hkv, D, P, bad, grid):
    """A request none of whose keys scores above -inf has no output, whatever its values hold; where another key
    counts, 0 times such a value shows in its channel."""
    q, k, v, table, sl = make_case(lens, Hq, Hkv, D, P, seed=3)
    q[:, :, 0] = 1.0
    n = -(-lens[0] // P)
    pages = table[0, :n].long()
    k[pages, :, :, 0] = -float("inf")
    v[pages, 0, :, 5] = bad
    o, lse = da.paged_attn_fwd(q, k, v, table, sl)
    cut = table.clone()
    cut[0] = -1
    check_attn(o, lse, po.attend(q, k.nan_to_num(neginf=0), v.nan_to_num(0, 0, 0), cut, sl, D ** -0.5))
    assert (o[0] == 0).all() and (lse[0] == -math.inf).all()
    # one page of keys that count, the last
    k[pages[-1], :, :, 0] = 0
    v[pages[-1], 0, :, 5] = 0
    cut[0, n - 1] = table[0, n - 1]
    o, lse = da.paged_attn_fwd(q, k, v, table, sl)
    if n > 1:
        assert o[0, :Hq // Hkv, 5].isnan().all()
        o[0, :Hq // Hkv, 5] = 0
    kept = v.nan_to_num(0, 0, 0)
    kept[pages, 0, :, 5] = 0
    check_attn(o, lse, po.attend(q, k.nan_to_num(neginf=0), kept, cut, sl, D ** -0.5))


@pytest.mark.parametrize("lens,Hq,Hkv,D,P", [([4000, 300, 17], 6, 2, 128, 16), ([9000], 3, 1, 64, 64),
                                             ([700, 90], 24, 1, 128, 32), ([64], 2, 2, 64, 16), ([1500], 40, 1, 128, 16)])
def test_float_output_keeps_all_parts_of_the_weights(lens, Hq, Hkv, D, P, launch):
    """fp32 output, flat scores: the 2-norm of the error is that of 32-bit weights.  Their relative errors, of random sign
    from key to key, are the exponential's (at most 2^-22) and a few roundings (2^-24 each): below 8e-7 together.
    Weights in two bf16 parts would be off by up to 2^-18 evenly, 2^-18 / sqrt(3) = 2.2e-6 in the mean."""
    q, k, v, table, sl = make_case(lens, Hq, Hkv, D, P, seed=1, q_scale=0.25)
    o = da.paged_attn_fwd(q, k, v, table, sl)[0].double().cpu().numpy()
    want = po.attend(q, k, v, table, sl, D ** -0.5)[0]
    assert np.linalg.norm(o - want) <= 8e-7 * np.linalg.norm(want)


# ------------------------------------------------------------------ selection


@pytest.mark.parametrize("n", [40, 700, 2047, 9001])
@pytest.mark.parametrize("kind", ["both", "positive", "negative", "newest", "unused", "every page"])
@pytest.mark.parametrize("e", [20, 40, 70, 100])
def test_select_beside_pages_of_another_scale(n, kind, e, launch):
    """One page far larger than the others (or each page of its own size): the others keep their order."""
    P, Hq, Hkv, D = 16, 3, 1, 64 if n % 2 else 128
    lens = [n * P, n * P - 5]
    table, n_pages = tables(lens, P, seed=n)
    q = rand(2, Hq, D, seed=1)
    a, b = rand(n_pages, Hkv, 1, D, seed=2), rand(n_pages, Hkv, 1, D, seed=3)
    summary = torch.cat((torch.minimum(a, b), torch.maximum(a, b)), 2)
    at = table[0, n - 1 if kind == "newest" else n // 3]
    if kind in ("both", "newest"):
        summary[at] *= 2.0 ** e
    elif kind == "positive":
        summary[at] = (q[0, 0] * 2.0 ** e).expand(Hkv, 2, D)
    elif kind == "negative":
        summary[at] = (q[0, 0] * -2.0 ** e).expand(Hkv, 2, D)
    elif kind == "unused":  # minima that no product of a positive query takes
        q = q.abs()
        summary[at, :, 0] = -2.0 ** e
    else:
        g = torch.Generator(device="cuda").manual_seed(5)
        x = torch.randint(-e // 2, e // 2 + 1, (n_pages, 1, 1, 1), generator=g, device="cuda")
        summary *= torch.exp2(x.float()).to(torch.bfloat16)
    t = dev(table)
    t, sl = (widened(t, launch) if n < 2100 else t), dev(lens)
    for top_k in (2, n // 3, n - 2):
        got = da.paged_select(q, summary, t, sl, P, top_k)
        assert np.array_equal(got.cpu().numpy(), po.select(q, summary, t, sl, P, top_k)), top_k


@pytest.mark.parametrize("n", [100, 1500, 9001])
def test_select_pages_without_keys_tie_with_scores_of_minus_infinity(n, launch):
    """Both score -inf: the lower index first, whichever it is."""
    P, Hq, Hkv, D = 16, 2, 1, 64
    table, n_pages = tables([n * P], P, seed=n, extra_cols=0)
    q = rand(1, Hq, D, seed=1).abs()
    summary = rand(n_pages, Hkv, 1, D, seed=2).repeat(1, 1, 2, 1)
    kind = np.random.default_rng(3).integers(0, 4, n)
    summary[dev(table[0, :n][kind == 1], torch.int64), :, :, 0] = -float("inf")
    table[0, :n][kind == 2] = -1
    t = dev(table)
    t, sl = (widened(t, launch) if n < 2100 else t), dev([n * P])
    for top_k in (n // 4, n // 2, n * 5 // 8, n * 3 // 4, n - 1):
        got = da.paged_select(q, summary, t, sl, P, top_k)
        assert np.array_equal(got.cpu().numpy(), po.select(q, summary, t, sl, P, top_k)), top_k


@pytest.mark.parametrize("kind", ["some", "empty"])
@pytest.mark.parametrize("n", [100, 1500, 4000])
def test_select_takes_either_order_of_the_extremes(n, kind, launch):
    """Summaries of which some have the larger value first, or are those of no key at all (+inf, -inf)."""
    P, Hq, Hkv, D = 16, 6, 2, 128
    table, n_pages = tables([n * P, n * P - 5], P, seed=n)
    q, summary = rand(2, Hq, D, seed=1), rand(n_pages, Hkv, 2, D, seed=2)
    if kind == "empty":
        some = torch.as_tensor(np.random.default_rng(3).random(n_pages) < 0.1)
        summary[some, :, 0], summary[some, :, 1] = float("inf"), -float("inf")
    t = dev(table)
    t, sl = (widened(t, launch) if n < 2100 else t), dev([n * P, n * P - 5])
    for top_k in (2, n // 20, n // 3):
        got = da.paged_select(q, summary, t, sl, P, top_k)
        assert np.array_equal(got.cpu().numpy(), po.select(q, summary, t, sl, P, top_k)), top_k


@pytest.mark.parametrize("n", [100, 1500, 9001])
@pytest.mark.parametrize("e", [-30, -60, -90, -120])
def test_select_zeros_among_scores_that_underflow(n, e, launch):
    """Pages of zeros tie with each other only: products that vanish in 32 bits still have their order in 64."""
    P, Hq, Hkv, D = 16, 2, 1, 64 if n % 2 else 128
    table, n_pages = tables([n * P], P, seed=n, extra_cols=0)
    q = rand(1, Hq, D, seed=1) * 2.0 ** e
    a, b = rand(n_pages, Hkv, 1, D, seed=2), rand(n_pages, Hkv, 1, D, seed=3)
    summary = torch.cat((torch.minimum(a, b), torch.maximum(a, b)), 2) * 2.0 ** e
    kind = torch.as_tensor(np.random.default_rng(3).integers(0, 4, n_pages))
    summary[kind == 1] = 0
    summary[kind == 2] *= -1  # minima above maxima: scores below 0
    t = dev(table)
    t, sl = (widened(t, launch) if n < 2100 else t), dev([n * P])
    for top_k in (n // 4, n // 2, n * 5 // 8, n * 3 // 4, n - 1):
        got = da.paged_select(q, summary, t, sl, P, top_k)
        assert np.array_equal(got.cpu().numpy(), po.select(q, summary, t, sl, P, top_k)), top_k


def test_select_of_the_newest_page_scores_nothing():
    """top_k = 1: nothing goes through the workspace."""
    lens, P, Hq, Hkv, D = [40000, 0, 17], 16, 4, 2, 64
    table, n_pages = tables(lens, P)
    q, summary = rand(3, Hq, D, seed=1), rand(n_pages, Hkv, 2, D, seed=2)
    need = da.lib().dit_paged_select_workspace_bytes(3, Hkv, table.shape[1])
    ws = torch.full((need,), 0x5A, dtype=torch.uint8, device="cuda")
    assert need > 0
    got = da.paged_select(q, summary, dev(table), dev(lens), P, 1, workspace=ws)
    assert got.flatten().tolist() == [2499] * Hkv + [-1] * Hkv + [1] * Hkv
    assert (ws == 0x5A).all()
