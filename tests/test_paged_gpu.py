"""GPU parity of the paged key/value cache: dit_paged_plan, dit_paged_kv_write, dit_paged_select and
dit_paged_attn_fwd against their plain 64-bit forms (paged_oracle), and a run of them together.

Tolerances of the attention, from its arithmetic (S = scale max_j sum_d |q_d k_jd| for the row,
A = sum_j p_j |v_j| for the channel):
  - a score is a sum of D exact products in 32 bits, in D / 16 steps of 16 products and the running
    sum, each term kept to within 2^-23 of the step's largest: off by at most
    (D / 16) * 17 * 2^-23 * S =: E;
  - a weight is off by a factor of at most exp(E) (score) and 2^-21 (exponential, in 32 bits), its
    two or three 8-bit parts by 2^-17, a sum of them by 2^-20; numerator and denominator both:
    |o - o_ref| <= (2 E + 2^-16) A, and half a step of the output's type;
  - |lse - lse_ref| <= E + 2^-19 + 2^-23 |lse|.
These are worst cases; over a whole output the errors are of random sign, so the 2-norm of the error
is also held to 1e-5 (fp32 output) of the result's.
"""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_oracle as po
from diffusion_transformer_long_gb300 import ditattn as da

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(DEV, dtype)


def rand(*shape, seed=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def cache_view(n_pages, H, P, D, order, seed=0, scale=1.0):
    """A [n_pages, H, P, D] view: head-major, token-major, or a part of a larger allocation."""
    if order == "hnd":
        return rand(n_pages, H, P, D, seed=seed, scale=scale)
    if order == "nhd":
        return rand(n_pages, P, H, D, seed=seed, scale=scale).transpose(1, 2)
    return rand(n_pages, H + 1, P + 3, 2 * D, seed=seed, scale=scale)[:, 1:, 2:P + 2, D:]


def tables(lens, P, seed=0, extra_pages=2, extra_cols=1):
    """(block table with shuffled pages, -1 past each length; n_pages)."""
    rng = np.random.default_rng(seed)
    n = [-(-max(0, x) // P) for x in lens]
    n_pages = sum(n) + extra_pages
    order = rng.permutation(n_pages)
    t = np.full((len(lens), max(1, max(n) + extra_cols)), -1, np.int64)
    at = 0
    for b, m in enumerate(n):
        t[b, :m] = order[at:at + m]
        at += m
    return t, n_pages


@pytest.fixture(params=["as chosen", "many items"])
def launch(request):
    """The launch that the sizes choose (a cluster for each of few items), and the one for many items."""
    da.set_grid_limit(1000 if request.param == "many items" else 0)
    yield request.param
    da.set_grid_limit(0)


def widened(table, launch):
    """For the selection: the same table with room for more pages than a cluster takes on."""
    if launch == "as chosen":
        return table
    wide = torch.full((table.shape[0], 2100), -1, device=DEV, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    return wide


# ------------------------------------------------------------------ plan


def check_plan(new, old, table, free_pages, n_free, P, n_pages, max_tokens, in_place=False):
    want = po.plan(new, old, table, free_pages, n_free, P, n_pages, max_tokens)
    td, sd, fd = dev(table), dev(old), dev([n_free])
    kw = dict(seq_lens_out=sd, n_free_out=fd) if in_place else {}
    got = da.paged_plan(dev(new), sd, td, dev(free_pages), fd, P, n_pages, max_tokens, **kw)
    names = ("lens", "n_free", "cu", "slots")
    for name, g, w in zip(names, got, want):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), name
    assert np.array_equal(td.cpu().numpy(), want[4]), "table"
    if not in_place:
        assert np.array_equal(sd.cpu().numpy(), np.asarray(old)) and int(fd) == n_free


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,P,old_hi,new_lo,new_hi,pool", [
    (1, 16, 40, 1, 1, 1.0), (1, 16, 0, 27280, 27280, 1.0), (5, 48, 200, 0, 90, 1.0),
    (64, 16, 600, 1, 1, 1.0), (33, 32, 100, 0, 500, 0.6), (1000, 16, 70, 0, 3, 1.0),
    (8192, 16, 40, 0, 2, 0.9), (3, 1024, 5000, 0, 3000, 1.0), (2047, 64, 300, 0, 40, 1.3)])
def test_plan(B, P, old_hi, new_lo, new_hi, pool, in_place):
    rng = np.random.default_rng(B + P)
    old = rng.integers(0, old_hi + 1, B)
    new = rng.integers(new_lo, new_hi + 1, B)
    have = -(-old // P)
    need = -(-(old + new) // P) - have
    max_pages = int((-(-(old + new) // P)).max()) + 1
    n_free = int(need.sum() * pool)
    n_pages = int(have.sum()) + n_free + 4
    order = rng.permutation(n_pages)
    table = np.full((B, max_pages), -7, np.int64)
    at = 0
    for b in range(B):
        table[b, :have[b]] = order[at:at + have[b]]
        at += have[b]
    free_pages = order[at:]
    for max_tokens in {max(1, int(new.sum())), int(new.sum()) + 77, max(1, int(new.sum()) * 2 // 3)}:
        check_plan(new, old, table, free_pages, n_free, P, n_pages, max_tokens, in_place)


def test_plan_unusual_contents():
    """Negative and huge lengths, a full table row, no free pages, a count past the stack, table and
    stack entries outside the pool, a strided table."""
    big = 2 ** 31 - 1
    table = np.array([[3, -1, -1], [0, 99, -1], [1, 2, 4], [-5, -1, -1]])
    free_pages = np.array([5, 77, 6, -2, 8])
    for new, old in (([4, 20, 7, 9], [16, 20, 48, 3]), ([-3, 0, big, 1], [-8, 33, 40, 16]),
                     ([big, big, big, big], [0, 0, 0, 0]), ([1, 1, 1, 1], [big, -big, 16, 32])):
        for n_free in (0, 2, 5, 50, -4):
            check_plan(new, old, table, free_pages, n_free, 16, 9, 100)
    wide = torch.full((4, 10), -1, dtype=torch.int32, device=DEV)
    wide[:, :3] = dev(table)
    new, old = [4, 20, 7, 9], [16, 20, 40, 3]
    got = da.paged_plan(dev(new), dev(old), wide[:, :3], dev(free_pages), dev([5]), 16, 9, 64)
    want = po.plan(new, old, table, free_pages, 5, 16, 9, 64)
    assert np.array_equal(got[3].cpu().numpy(), want[3])
    assert np.array_equal(wide[:, :3].cpu().numpy(), want[4]) and (wide[:, 3:] == -1).all()


# ------------------------------------------------------------------ write


def check_write(T, H, D, P, order, slots, n_pages, with_summary, seed=0, k_new=None):
    qkv = rand(T, 3 * H, D, seed=seed)
    k_new = qkv[:, H:2 * H] if k_new is None else k_new
    v_new = qkv[:, 2 * H:]
    k, v = (cache_view(n_pages, H, P, D, order, seed=seed + i) for i in (1, 2))
    summary = rand(n_pages, H, 2, D, seed=seed + 3) if with_summary else None
    sl = dev(slots, torch.int64)
    want_k, want_s = po.write(k_new.cpu(), sl.cpu(), k.cpu(), None if summary is None else summary.cpu())
    want_v, _ = po.write(v_new.cpu(), sl.cpu(), v.cpu())
    da.paged_kv_write(k_new, v_new, sl, k, v, summary=summary)
    bits = lambda x: x.contiguous().cpu().view(torch.int16)  # noqa: E731
    assert torch.equal(bits(k), bits(want_k)) and torch.equal(bits(v), bits(want_v))
    if with_summary:  # values: the zero of a page that holds both has either sign
        s = summary.cpu()
        assert torch.equal(s.isnan(), want_s.isnan())
        assert torch.equal(s.nan_to_num(), want_s.nan_to_num())


def plan_slots(old, new, P, seed=0, spare=0):
    rng = np.random.default_rng(seed)
    n_pages = sum(-(-(o + n) // P) for o, n in zip(old, new)) + 3
    order = list(rng.permutation(n_pages))
    slots = []
    for o, n in zip(old, new):
        pages = [order.pop() for _ in range(-(-(o + n) // P))]
        slots += [pages[i // P] * P + i % P for i in range(o, o + n)]
    return np.array(slots + [-1] * spare, np.int64), n_pages


@pytest.mark.parametrize("with_summary", [False, True])
@pytest.mark.parametrize("H,D,P,order,old,new,spare", [
    (1, 64, 16, "hnd", [0], [1], 0), (8, 128, 16, "hnd", [0, 15, 16, 17, 31], [1, 1, 1, 1, 1], 3),
    (2, 64, 48, "nhd", [3, 0, 47, 48, 100], [200, 1, 2, 90, 0], 5),
    (3, 128, 16, "nhd", [5], [333], 0), (5, 128, 128, "part", [0, 100], [300, 57], 31),
    (2, 64, 1024, "hnd", [1000], [1100], 1), (40, 128, 16, "hnd", list(range(70)), [1] * 70, 0),
    (24, 128, 64, "hnd", [0], [5000], 0), (1, 64, 32, "part", [7] * 33, [35] * 33, 2)])
def test_write(H, D, P, order, old, new, spare, with_summary):
    slots, n_pages = plan_slots(old, new, P, seed=len(old), spare=spare)
    check_write(len(slots), H, D, P, order, slots, n_pages, with_summary)


@pytest.mark.parametrize("shape,dims,keys", [
    ((2, 9, 3, 32, 64), (0, 1, 2, 3, 4), 0), ((9, 2, 3, 32, 64), (1, 0, 2, 3, 4), 0),
    ((9, 2, 3, 32, 64), (1, 0, 2, 3, 4), 1), ((9, 32, 2, 3, 64), (2, 0, 3, 1, 4), 0),
    ((9, 32, 3, 2, 64), (3, 0, 2, 1, 4), 1), ((9, 3, 2, 32, 64), (2, 0, 1, 3, 4), 0),
    ((9, 3, 32, 2, 64), (3, 0, 1, 2, 4), 0)])
def test_keys_and_values_in_one_allocation(shape, dims, keys):
    """Pages, heads or rows of keys and values in turn: written and attended to as in two allocations."""
    both = rand(*shape, seed=1)
    pair = both.permute(*dims)  # [2, n_pages, H, P, D]
    k, v = pair[keys], pair[1 - keys]
    n_pages, H, P, D = k.shape
    apart = [x.clone(memory_format=torch.contiguous_format) for x in (k, v)]
    lens = [50, 0, 32, 97]
    table, _ = tables(lens, P, extra_pages=n_pages - 7)
    slots = np.concatenate([table[b, np.arange(n) // P] * P + np.arange(n) % P for b, n in enumerate(lens)])
    new = rand(len(slots), 2 * H, D, seed=2)
    q, td, sl = rand(len(lens), 2 * H, D, seed=3), dev(table), dev(lens)
    res = []
    for kc, vc in ((k, v), apart):
        summary = torch.zeros(n_pages, H, 2, D, device=DEV, dtype=torch.bfloat16)
        da.paged_kv_write(new[:, :H], new[:, H:], dev(slots, torch.int64), kc, vc, summary=summary)
        sel = da.paged_select(q, summary, td, sl, P, 2)
        res.append((kc, vc, summary, sel, *da.paged_attn_fwd(q, kc, vc, td, sl),
                    *da.paged_attn_fwd(q, kc, vc, td, sl, selected=sel)))
    for a, b in zip(*res):
        assert torch.equal(a, b)
    check_attn(*res[0][4:6], po.attend(q, k, v, td, sl, D ** -0.5))


def test_write_skips_and_nan():
    """Slots outside the pool are skipped wherever they stand (a page's run goes on behind them, as a
    run of its own rows), and a NaN key shows in its page's summary."""
    P, n_pages, H, D = 16, 6, 2, 128
    slots = [-1, 16, 17, 18, -9, 32, 96, 33 + 2 ** 40, 80, 81, 95, -1]
    slots[10] = 82
    k_new = rand(len(slots), H, D, seed=9)
    k_new[2, 1, 7] = float("nan")
    k_new[9, 0, 3] = float("inf")
    for summary in (False, True):
        check_write(len(slots), H, D, P, "hnd", slots, n_pages, summary, k_new=k_new)
    check_write(4, H, D, P, "hnd", [-1, -1, 96, 2 ** 62], n_pages, True)


# ------------------------------------------------------------------ attention


def check_attn(o, lse, ref, bf16=False):
    o_ref, lse_ref, (mag, pv) = ref
    D = o_ref.shape[2]
    E = (D // 16) * 17 * 2.0 ** -23 * mag
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    tol = (2 * E + 2.0 ** -16)[..., None] * pv + (2.0 ** -8 if bf16 else 2.0 ** -23) * np.abs(o_ref) + 1e-37
    err = np.abs(o - o_ref)
    assert (err <= tol).all(), f"out: {(err / tol).max():.3g} times its bound, {err.max():.3g}"
    none = np.isinf(lse_ref)
    assert (lse[none] == -math.inf).all() and (o[none] == 0).all()
    lerr = np.abs(lse[~none] - lse_ref[~none])
    ltol = E[~none] + 2.0 ** -19 + 2.0 ** -23 * np.abs(lse_ref[~none])
    assert (lerr <= ltol).all(), f"lse: {(lerr / ltol).max():.3g} times its bound"
    if not bf16 and np.abs(o_ref).max() > 0:
        rel = np.linalg.norm(o - o_ref) / np.linalg.norm(o_ref)
        assert rel <= 1e-5, f"2-norm of the error: {rel:.3g}"


def make_case(lens, Hq, Hkv, D, P, order="hnd", seed=0, q_scale=1.5, k_scale=1.0):
    table, n_pages = tables(lens, P, seed)
    q = rand(len(lens), Hq, D, seed=seed + 1, scale=q_scale)
    k = cache_view(n_pages, Hkv, P, D, order, seed=seed + 2, scale=k_scale)
    v = cache_view(n_pages, Hkv, P, D, order, seed=seed + 3)
    return q, k, v, dev(table), dev(lens)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Hq,Hkv,D,P,order,lens", [
    (2, 2, 64, 16, "hnd", [1]), (2, 2, 64, 16, "nhd", [0, 1, 15, 16, 17, 63, 64, 65, 1024]),
    (24, 8, 128, 16, "hnd", [0, 0, 1, 2, 4608]), (24, 24, 128, 32, "nhd", [31, 32, 33, 700]),
    (40, 8, 128, 64, "hnd", [5, 1000, 63]), (16, 1, 64, 48, "part", [47, 48, 49, 2000]),
    (24, 2, 128, 128, "hnd", [129, 1, 300]), (24, 1, 128, 16, "nhd", [513, 16]),
    (40, 1, 128, 16, "hnd", [700, 3]), (70, 2, 64, 32, "nhd", [333, 0, 64]),
    (64, 2, 64, 1024, "hnd", [1500, 1023]), (9, 1, 128, 16, "part", [100]),
    (1, 1, 128, 16, "hnd", [27280]), (8, 8, 64, 16, "hnd", list(range(130)))])
def test_attn(Hq, Hkv, D, P, order, lens, out_dtype, launch):
    q, k, v, table, sl = make_case(lens, Hq, Hkv, D, P, order, seed=Hq + len(lens))
    o, lse = da.paged_attn_fwd(q, k, v, table, sl, out_dtype=out_dtype)
    da.check()
    ref = po.attend(q, k, v, table, sl, 1 / math.sqrt(D))
    check_attn(o, lse, ref, out_dtype == torch.bfloat16)
    o2, none = da.paged_attn_fwd(q, k, v, table, sl, out_dtype=out_dtype, with_lse=False)
    assert none is None and torch.equal(o, o2)  # and equal calls give equal bits


@pytest.mark.parametrize("D,P", [(64, 16), (128, 48)])
def test_attn_ignores_what_no_request_holds(D, P, launch):
    """Rows past a length and pages of nobody hold NaN and infinities; table entries past a length
    are wild; entries inside a length that are outside the pool hold no keys."""
    lens = [0, 1, P - 1, P, P + 1, 5 * P + 3, 777, 16, 3 * P]
    q, k, v, table, sl = make_case(lens, 6, 2, D, P, seed=3)
    used = torch.zeros(k.shape[0], P, dtype=torch.bool, device=DEV)
    for b, n in enumerate(lens):
        for page, row in po.rows_of(table.cpu().numpy(), b, n, P, k.shape[0]):
            used[page, row] = True
    for x, bad in ((k, float("nan")), (v, float("inf"))):
        x.masked_fill_(~used[:, None, :, None], bad)
    wild = table.clone()
    wild[table < 0] = 2 ** 31 - 1
    scale = 1 / math.sqrt(D)
    ref = po.attend(q, k.nan_to_num(0, 0, 0), v.nan_to_num(0, 0, 0), table, sl, scale)
    check_attn(*da.paged_attn_fwd(q, k, v, wild, sl), ref)
    wild[5, 1] = -4                 # a page in the middle
    wild[6, 777 // P] = k.shape[0]  # the last page
    wild[3, 0] = 2 ** 30            # the only page: no keys at all
    ref = po.attend(q, k.nan_to_num(0, 0, 0), v.nan_to_num(0, 0, 0), wild, sl, scale)
    assert np.isinf(ref[1][3]).all()
    check_attn(*da.paged_attn_fwd(q, k, v, wild, sl), ref)
    # lengths below 0, and past the table (counted as the table's last row)
    odd = sl.clone()
    odd[1] = -(2 ** 31)
    odd[2] = 2 ** 31 - 1
    full = table.clone()
    full[2] = torch.arange(table.shape[1], device=DEV, dtype=torch.int32) % k.shape[0]
    kk, vv = k.nan_to_num(0, 0, 0), v.nan_to_num(0, 0, 0)
    check_attn(*da.paged_attn_fwd(q, kk, vv, full, odd), po.attend(q, kk, vv, full, odd, scale))


def test_attn_nan_and_infinite_keys_reach_their_own_row_only(launch):
    q, k, v, table, sl = make_case([40, 40, 40], 4, 2, 64, 16, seed=5)
    k[table[0, 1], 0, 3] = float("nan")
    v[table[1, 2], 1, 7, 5] = float("inf")
    o, lse = (x.cpu() for x in da.paged_attn_fwd(q, k, v, table, sl))
    assert o[0, :2].isnan().all() and lse[0, :2].isnan().all()
    assert o[0, 2:].isfinite().all() and o[2].isfinite().all() and lse[1:].isfinite().all()
    bad = torch.zeros(4, 64, dtype=torch.bool)
    bad[2:, 5] = True
    assert torch.equal(~o[1].isfinite(), bad)


@pytest.mark.parametrize("q_scale,k_scale", [(8.0, 4.0), (0.0, 1.0), (1e-3, 1e-3)])
def test_attn_peaked_and_flat(q_scale, k_scale, launch):
    q, k, v, table, sl = make_case([3000, 33, 1], 24, 8, 128, 16, seed=7, q_scale=q_scale, k_scale=k_scale)
    check_attn(*da.paged_attn_fwd(q, k, v, table, sl), po.attend(q, k, v, table, sl, 128 ** -0.5))


def test_attn_growing_scores(launch):
    """Every key beats the ones before it: the running maximum moves at each step."""
    n, D, P = 2000, 64, 16
    table, n_pages = tables([n], P, extra_pages=0, extra_cols=0)
    q = torch.ones(1, 2, D, device=DEV, dtype=torch.bfloat16)
    k, v = torch.zeros(n_pages, 2, P, D, device=DEV, dtype=torch.bfloat16), rand(n_pages, 2, P, D, seed=1)
    at = dev(table[0], torch.int64)
    ramp = torch.linspace(-80, 80, n, device=DEV).reshape(-1, P)
    k[at, 0, :, 0] = ramp.to(torch.bfloat16)
    k[at, 1, :, 0] = -ramp.to(torch.bfloat16)
    t, sl = dev(table), dev([n])
    for scale in (1.0, 10.0):
        check_attn(*da.paged_attn_fwd(q, k, v, t, sl, scale=scale), po.attend(q, k, v, t, sl, scale))


def test_attn_views_streams_workspace():
    """Strided queries and tables, caller's outputs, a poisoned workspace of the exact size with a
    guard behind it, another stream."""
    lens = [100, 0, 3000, 17]
    q, k, v, table, sl = make_case(lens, 10, 2, 128, 32, "part", seed=11)
    fused = torch.zeros(4, 14, 192, device=DEV, dtype=torch.bfloat16)
    fused[:, 2:12, 64:] = q
    wide = torch.full((4, 160), 12345, device=DEV, dtype=torch.int32)
    wide[:, 2:2 + table.shape[1]] = table
    need = da.lib().dit_paged_attn_workspace_bytes(4, 10, 2, 128, 32, 150)
    assert need > 0
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full((5, 10, 128), 7.0, device=DEV)
    lse = torch.full((5, 10), 7.0, device=DEV)
    da.paged_attn_fwd(fused[:, 2:12, 64:], k, v, wide[:, 2:152], sl, out=out[:4], lse=lse[:4],
                      workspace=ws[:need])
    da.check()
    ref = po.attend(q, k, v, table, sl, 128 ** -0.5)
    check_attn(out[:4], lse[:4], ref)
    assert (ws[need:] == 0xFF).all() and (out[4] == 7).all() and (lse[4] == 7).all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, l2 = da.paged_attn_fwd(q, k, v, wide[:, 2:152], sl, stream=s)
    s.synchronize()
    assert torch.equal(o2, out[:4]) and torch.equal(l2, lse[:4])
    # few keys at most: clusters, and no workspace
    assert da.lib().dit_paged_attn_workspace_bytes(4, 10, 2, 128, 32, table.shape[1]) == 0
    check_attn(*da.paged_attn_fwd(fused[:, 2:12, 64:], k, v, table, sl, stream=s), ref)


@pytest.mark.parametrize("B", [700, 5000])
def test_attn_many_requests(B):
    """More requests than a block has threads: lengths 0 to 40, one longer; rows in a strided query."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 41, B)
    lens[B // 3] = 900
    q, k, v, table, sl = make_case(list(lens), 4, 2, 64, 16, seed=81)
    check_attn(*da.paged_attn_fwd(q, k, v, table, sl), po.attend(q, k, v, table, sl, 0.125))


def test_attn_scores_without_a_finite_one(launch):
    """Keys that score -inf weigh nothing; a request all of whose keys do is one without keys."""
    q, k, v, table, sl = make_case([40, 20], 2, 2, 64, 16, seed=83)
    q[:, :, 0] = 1.0
    k[table[0, 1], :, :, 0] = -float("inf")
    k[table[1, :2].long(), :, :, 0] = -float("inf")
    o, lse = da.paged_attn_fwd(q, k, v, table, sl)
    cut = table.clone()
    cut[0, 1] = -1
    cut[1] = -1
    check_attn(o, lse, po.attend(q, k.nan_to_num(neginf=0), v, cut, sl, 0.125))
    assert (lse[1] == -float("inf")).all() and (o[1] == 0).all()


def test_attn_two_streams_at_once(launch):
    cases = [make_case([2000 + i, 900, 5], 24, 8, 128, 16, seed=20 + i) for i in range(2)]
    alone = [da.paged_attn_fwd(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = [da.paged_attn_fwd(*c, stream=s) for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for (o, lse), (o1, l1) in zip(got, alone):
            assert torch.equal(o, o1) and torch.equal(lse, l1)


def test_captured_between_copies_and_two_graphs_of_one_workspace(launch):
    """Captured behind a copy, a fill and each other; two graphs that share the workspaces, replayed
    in turn, and one call captured twice into the same graph."""
    P, top_k = 16, 9
    q, k, v, table, sl = make_case([1500, 40, 0, 333], 6, 2, 64, P, seed=61)
    table = widened(table, launch)
    summary = torch.stack((k.amin(2), k.amax(2)), 2)
    src = torch.empty_like(q)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    wsel = torch.empty(da.lib().dit_paged_select_workspace_bytes(4, 2, 5000), dtype=torch.uint8, device=DEV)
    ws.fill_(0x5A)
    wsel.fill_(0xA5)
    x = q.clone()

    def step(out, lse):
        x.copy_(src)
        sel = da.paged_select(x, summary, table, sl, P, top_k, workspace=wsel)
        out.fill_(3)
        da.paged_attn_fwd(x, k, v, table, sl, selected=sel, out=out, lse=lse, workspace=ws)
        return sel

    graphs, outs = [], []
    for _ in range(2):
        out, lse = torch.empty(2, 4, 6, 64, device=DEV), torch.empty(2, 4, 6, device=DEV)
        src.copy_(q)
        step(out[0], lse[0])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sel = [step(out[i], lse[i]) for i in range(2)]
        graphs.append(g)
        outs.append((out, lse, sel))
    for i in range(12):
        src.copy_(rand(4, 6, 64, seed=70 + i, scale=1.5))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        out, lse, sel = outs[i % 2]
        want = po.select(src, summary, table, sl, P, top_k)
        ref = po.attend(src, k, v, table, sl, 64 ** -0.5, selected=dev(want))
        for c in range(2):
            assert np.array_equal(sel[c].cpu().numpy(), want)
            check_attn(out[c], lse[c], ref)


def test_attn_capped_grid():
    """A capped grid walks many items per block: the same values up to the order of the joins."""
    lens = [0, 700, 33, 1, 2500, 64]
    q, k, v, table, sl = make_case(lens, 12, 4, 64, 16, seed=31)
    ref = po.attend(q, k, v, table, sl, 64 ** -0.5)
    try:
        for cap in (1, 2, 7, 50):
            da.set_grid_limit(cap)
            check_attn(*da.paged_attn_fwd(q, k, v, table, sl), ref)
    finally:
        da.set_grid_limit(0)


def test_attn_reports_a_wait_that_runs_out(launch):
    """With the copies withheld every wait runs out after its limit, the launch ends and the check
    says so; the next call is right again."""
    q, k, v, table, sl = make_case([500, 0, 40], 8, 2, 128, 16, seed=33)
    good = da.paged_attn_fwd(q, k, v, table, sl)
    da.check()
    try:
        da.inject_stall(True, 200_000)
        da.paged_attn_fwd(q, k, v, table, sl)
        with pytest.raises(da.DitError) as e:
            da.check()
        assert e.value.status == da.DIT_ERR_TIMEOUT
    finally:
        da.inject_stall(False)
    o, lse = da.paged_attn_fwd(q, k, v, table, sl)
    da.check()
    assert torch.equal(o, good[0]) and torch.equal(lse, good[1])


def test_attn_offsets_past_32_bits(launch):
    """Pages that begin more than 2^32 bytes and more than 2^31 elements into the cache."""
    H, P, D = 2, 64, 128
    n_pages = 2 ** 31 // (H * P * D) + 40
    k = torch.empty(n_pages, H, P, D, device=DEV, dtype=torch.bfloat16)
    k[:3] = rand(3, H, P, D, seed=1)
    k[-3:] = rand(3, H, P, D, seed=2)
    pages = [n_pages - 1, 0, n_pages - 3, 2, n_pages - 2, 1]
    table, sl = dev([pages]), dev([6 * P - 5])
    q = rand(1, 4, D, seed=3)
    o, lse = da.paged_attn_fwd(q, k, k, table, sl)
    small = torch.cat((k[:3], k[-3:]))
    small_table = dev([[i if i < 3 else i - n_pages + 6 for i in pages]])
    check_attn(o, lse, po.attend(q, small, small, small_table, sl, D ** -0.5))
    # the write reaches the same pages
    new = rand(3, H, D, seed=4)
    slots = torch.tensor([(n_pages - 1) * P + 5, 2 * P + 1, n_pages * P], device=DEV)
    v = torch.zeros(n_pages, H, P, D, device=DEV, dtype=torch.bfloat16)
    da.paged_kv_write(new, new, slots, k, v)
    assert torch.equal(k[-1, :, 5], new[0]) and torch.equal(v[-1, :, 5], new[0])
    assert torch.equal(k[2, :, 1], new[1]) and torch.equal(v[2, :, 1], new[1])


# ------------------------------------------------------------------ selection


@pytest.mark.parametrize("Hq,Hkv,D,P,lens,top_k", [
    (2, 2, 64, 16, [1], 1), (24, 8, 128, 16, [0, 1, 16, 17, 500, 4608], 8),
    (40, 8, 128, 32, [3000, 40], 1), (16, 1, 64, 16, [9000, 100, 5], 33),
    (24, 24, 128, 48, [1000, 2000], 21), (24, 1, 128, 16, [700], 44), (64, 2, 64, 16, [1600, 320], 20),
    (2, 2, 64, 16, [75600], 100), (4, 4, 128, 16, [27280, 27264], 1000)])
def test_select(Hq, Hkv, D, P, lens, top_k, launch):
    table, n_pages = tables(lens, P, seed=top_k)
    q = rand(len(lens), Hq, D, seed=1, scale=1.5)
    a, b = rand(n_pages, Hkv, 1, D, seed=2), rand(n_pages, Hkv, 1, D, seed=3)
    summary = torch.cat((torch.minimum(a, b), torch.maximum(a, b)), 2)
    t, sl = widened(dev(table), launch) if table.shape[1] < 2100 else dev(table), dev(lens)
    top_k = min(top_k, table.shape[1])
    got = da.paged_select(q, summary, t, sl, P, top_k)
    assert np.array_equal(got.cpu().numpy(), po.select(q, summary, t, sl, P, top_k))


@pytest.mark.parametrize("kind", ["equal", "few values", "near", "nan", "inf", "overflow", "tiny", "zero q",
                                  "bad entries", "inf q"])
def test_select_borders(kind, launch):
    """Scores that tie, that differ by less than a 32-bit sum resolves, that are no numbers, that pass
    the range of 32 bits at either end."""
    lens, P, Hq, Hkv, D, top_k = [2000, 1999, 130, 16], 16, 6, 2, 128, 37
    table, n_pages = tables(lens, P, seed=8)
    q = rand(len(lens), Hq, D, seed=1)
    a, b = rand(n_pages, Hkv, 1, D, seed=2), rand(n_pages, Hkv, 1, D, seed=3)
    summary = torch.cat((torch.minimum(a, b), torch.maximum(a, b)), 2)
    g = torch.Generator(device=DEV).manual_seed(4)
    some = torch.rand(n_pages, Hkv, generator=g, device=DEV) < 0.2
    if kind == "equal":
        summary[:] = summary[:1].clone()
    elif kind == "few values":
        summary[:] = summary[torch.arange(n_pages, device=DEV) % 3]
    elif kind == "near":  # one channel of a tiny query differs: the sums agree to about 2^-30
        summary[:] = summary[:1].clone()
        q[:, :, 5] = 2.0 ** -24
        summary[:, :, :, 5] = rand(n_pages, Hkv, 1, seed=6)
    elif kind == "nan":
        summary[some, 1, 9] = float("nan")
    elif kind == "inf":
        summary[some, 0, 9] = -float("inf")
        summary[~some, 1, 3] = float("inf")
    elif kind == "overflow":
        q *= 2.0 ** 70
        summary *= 2.0 ** 66
    elif kind == "tiny":
        q *= 2.0 ** -75
        summary *= 2.0 ** -70
    elif kind == "zero q":
        q.zero_()
    elif kind == "bad entries":
        table[0, 3:50] = -1
        table[1, ::2] = n_pages
        table[2, -2] = 2 ** 31 - 1
    else:
        q[0, 0, 0] = float("inf")
        q[1, 4, 7] = float("nan")
    t, sl = widened(dev(table), launch), dev(lens)
    for k in (1, 2, top_k, table.shape[1]):
        got = da.paged_select(q, summary, t, sl, P, k)
        assert np.array_equal(got.cpu().numpy(), po.select(q, summary, t, sl, P, k)), k


@pytest.mark.parametrize("n,kind", [(700, "equal"), (700, "nan"), (2047, "two values"), (3000, "two values"), (9001, "random"),
                                    (9001, "equal"), (9001, "two values"), (9001, "inf")])
def test_select_among_many_pages(n, kind):
    """More pages at the border than are ranked pair by pair, and more pages than shared memory holds."""
    P, Hq, Hkv, D = 16, 3, 1, 64
    table, n_pages = tables([n * P, n * P - 5], P, seed=n)
    q = rand(2, Hq, D, seed=1)
    a, b = rand(n_pages, Hkv, 1, D, seed=2), rand(n_pages, Hkv, 1, D, seed=3)
    summary = torch.cat((torch.minimum(a, b), torch.maximum(a, b)), 2)
    some = torch.rand(n_pages, generator=torch.Generator(device=DEV).manual_seed(4), device=DEV) < 0.4
    if kind == "equal":
        summary[:] = summary[:1].clone()
    elif kind == "two values":
        summary[:] = summary[some.int()]
    elif kind == "nan":
        summary[some, 0, 1, 9] = float("nan")
    elif kind == "inf":
        summary[some, 0, 0, 9] = -float("inf")
    t, sl = dev(table), dev([n * P, n * P - 5])
    for k in (2, 17, n // 3, n - 1):
        got = da.paged_select(q, summary, t, sl, P, k)
        assert np.array_equal(got.cpu().numpy(), po.select(q, summary, t, sl, P, k)), k


def test_tables_far_wider_than_the_requests():
    """Room for 2^20 pages a request, a few of them held: nothing takes the room for the length."""
    lens, P = [100, 0, 3000], 16
    q, k, v, table, sl = make_case(lens, 6, 2, 64, P, seed=91)
    wide = torch.full((3, 1 << 20), -1, device=DEV, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    summary = torch.stack((k.amin(2), k.amax(2)), 2)
    sel = da.paged_select(q, summary, wide, sl, P, 20)
    assert np.array_equal(sel.cpu().numpy(), po.select(q, summary, table, sl, P, 20))
    check_attn(*da.paged_attn_fwd(q, k, v, wide, sl), po.attend(q, k, v, table, sl, 0.125))
    check_attn(*da.paged_attn_fwd(q, k, v, wide, sl, selected=sel),
               po.attend(q, k, v, table, sl, 0.125, selected=sel))
    free = dev(np.arange(40))
    got = da.paged_plan(dev([20, 5, 1]), sl, wide, free, dev([40]), P, 500, 26)
    want = po.plan([20, 5, 1], lens, table.cpu().numpy(), np.arange(40), 40, P, 500, 26)
    assert np.array_equal(got[3].cpu().numpy(), want[3]) and np.array_equal(got[0].cpu().numpy(), want[0])


def test_first_calls_of_a_process_can_be_captured():
    """A fresh process captures its first calls: nothing of their setup is forbidden in a capture."""
    code = """
import torch
from diffusion_transformer_long_gb300 import ditattn as da
i32 = dict(dtype=torch.int32, device="cuda")
B, H, D, P, n = 3, 2, 64, 16, 30
new, lens, table = torch.full((B,), 5, **i32), torch.zeros(B, **i32), torch.full((B, 8), -1, **i32)
free, n_free = torch.arange(n, **i32), torch.full((1,), n, **i32)
k, v = (torch.zeros(n, H, P, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
s = torch.zeros(n, H, 2, D, dtype=torch.bfloat16, device="cuda")
x = torch.randn(15, 3 * H, D, device="cuda").bfloat16()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    _, _, _, slots = da.paged_plan(new, lens, table, free, n_free, P, n, 15, seq_lens_out=lens, n_free_out=n_free)
    da.paged_kv_write(x[:, H:2 * H], x[:, 2 * H:], slots, k, v, summary=s)
    sel = da.paged_select(x[:B, :H], s, table, lens, P, 2)
    o, lse = da.paged_attn_fwd(x[:B, :H], k, v, table, lens, selected=sel)
g.replay()
da.check()
assert lens.tolist() == [5] * B and o.isfinite().all() and lse.isfinite().all() and o.abs().sum() > 0
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("Hq,Hkv,D,P,order", [(24, 8, 128, 16, "hnd"), (2, 2, 64, 48, "nhd"), (16, 1, 64, 64, "part")])
def test_attn_over_selected_pages(Hq, Hkv, D, P, order, launch):
    """Lists as paged_select writes them, and any other list: skipped, repeated, unsorted entries."""
    lens = [0, 1, P, P + 1, 40 * P - 3, 2000]
    q, k, v, table, sl = make_case(lens, Hq, Hkv, D, P, order, seed=41)
    rng = np.random.default_rng(5)
    n = 6
    sel = rng.integers(-2, 45, (len(lens), Hkv, n))
    sel[4] = [[0, 39, 3, 3, -1, 38]] * Hkv
    sel[3] = [[1, 0, -1, 7, 7, 7]] * Hkv
    sd = dev(sel)
    check_attn(*da.paged_attn_fwd(q, k, v, table, sl, selected=sd),
               po.attend(q, k, v, table, sl, D ** -0.5, selected=sd))
    every = dev(np.broadcast_to(np.arange(table.shape[1]), (len(lens), Hkv, table.shape[1])).copy())
    ref = po.attend(q, k, v, table, sl, D ** -0.5)
    check_attn(*da.paged_attn_fwd(q, k, v, table, sl, selected=every), ref)


# ------------------------------------------------------------------ a run of them together


@pytest.mark.parametrize("sparse", [False, True])
def test_replayed_steps_are_in_order(sparse, launch):
    """Three decode steps captured back to back, each kernel behind the last with nothing between: every
    step sees what the one before wrote (the lengths, the table, the new keys), replay after replay."""
    B, Hq, Hkv, D, P, n_pages, steps = 4, 6, 2, 64, 16, 40, 3
    k, v = (torch.zeros(n_pages, Hkv, P, D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    summary = torch.zeros(n_pages, Hkv, 2, D, device=DEV, dtype=torch.bfloat16)
    table = widened(torch.full((B, 10), -1, device=DEV, dtype=torch.int32), launch)
    free, n_free, lens = dev(np.arange(n_pages)), dev([n_pages]), dev([0] * B)
    new, qkv = dev([1] * B), rand(steps, B, Hq + 2 * Hkv, D, seed=1)

    def step(i):
        da.paged_plan(new, lens, table, free, n_free, P, n_pages, B, seq_lens_out=lens, n_free_out=n_free, slots=slots)
        da.paged_kv_write(qkv[i, :, Hq:Hq + Hkv], qkv[i, :, Hq + Hkv:], slots, k, v, summary=summary)
        sel = da.paged_select(qkv[i, :, :Hq], summary, table, lens, P, 3) if sparse else None
        return (*da.paged_attn_fwd(qkv[i, :, :Hq], k, v, table, lens, selected=sel), sel)

    slots = torch.empty(B, dtype=torch.int64, device=DEV)
    step(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = [step(i) for i in range(steps)]
    for it in range(12):
        qkv.copy_(rand(steps, B, Hq + 2 * Hkv, D, seed=it))
        before = lens.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(lens, before + steps)
        for i, (o, lse, sel) in enumerate(res):
            # the last steps' rows are there already; each step's own length hides them
            then = before + i + 1
            if sparse and i < steps - 1:
                continue  # later rows of the same page are in its summary by now
            if sparse:
                want = po.select(qkv[i, :, :Hq], summary, table, then, P, 3)
                assert np.array_equal(sel.cpu().numpy(), want)
            check_attn(o, lse, po.attend(qkv[i, :, :Hq], k, v, table, then, D ** -0.5, selected=sel))


def test_steps_together_eager_and_replayed(launch):
    """A batch that prefills, then decodes token by token: plan, write with summaries, select,
    attention over all and over the selected pages, eagerly and as one captured step replayed as the
    lengths grow; a request that is idle for some steps and one that runs out of pages."""
    B, Hq, Hkv, D, P, top_k, n_pages, max_pages = 4, 6, 2, 64, 16, 3, 30, 12
    scale = D ** -0.5
    k, v = (torch.full((n_pages, Hkv, P, D), float("nan"), device=DEV, dtype=torch.bfloat16) for _ in range(2))
    summary = torch.full((n_pages, Hkv, 2, D), float("nan"), device=DEV, dtype=torch.bfloat16)
    table = torch.full((B, max_pages), -1, device=DEV, dtype=torch.int32)
    free = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).to(DEV, torch.int32)
    n_free, lens = dev([n_pages]), dev([0] * B)
    keys = [[torch.zeros(0, Hkv, D), torch.zeros(0, Hkv, D)] for _ in range(B)]  # what each request holds

    def step(new, qkv, max_tokens):
        _, _, cu, slots = da.paged_plan(new, lens, table, free, n_free, P, n_pages, max_tokens,
                                        seq_lens_out=lens, n_free_out=n_free)
        da.paged_kv_write(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], slots, k, v, summary=summary)
        q = qkv[:B, :Hq]
        sel = da.paged_select(q, summary, table, lens, P, top_k)
        return (cu, sel, *da.paged_attn_fwd(q, k, v, table, lens),
                *da.paged_attn_fwd(q, k, v, table, lens, selected=sel))

    def follow(new, qkv, res):
        cu, sel, o, lse, os_, ls = res
        da.check()
        cu, x = cu.cpu(), qkv.cpu()
        for b in range(B):
            for i in range(2):
                rows = x[cu[b]:cu[b + 1], Hq + i * Hkv:Hq + (i + 1) * Hkv].float()
                keys[b][i] = torch.cat((keys[b][i], rows))[:int(lens[b])]
        # what the requests hold, gathered by position, attended to as one page each
        t = np.arange(B)[:, None]
        most = max(1, int(lens.max()))
        dense = [torch.zeros(B, Hkv, most, D) for _ in range(2)]
        for b in range(B):
            for i in range(2):
                n = len(keys[b][i])
                assert n == int(lens[b])
                dense[i][b, :, :n] = keys[b][i].transpose(0, 1)
        q = qkv[:B, :Hq]
        check_attn(o, lse, po.attend(q, *dense, torch.as_tensor(t), lens, scale))
        assert np.array_equal(sel.cpu().numpy(), po.select(q, summary, table, lens, P, top_k))
        kk, vv = k.nan_to_num(0, 0, 0), v.nan_to_num(0, 0, 0)
        check_attn(os_, ls, po.attend(q, kk, vv, table, lens, scale, selected=sel))

    new = dev([40, 0, 75, 16])
    qkv = rand(140, Hq + 2 * Hkv, D, seed=50)
    follow(new, qkv, step(new, qkv, 140))
    new = dev([1, 1, 1, 1])
    qkv = rand(5, Hq + 2 * Hkv, D, seed=51)
    follow(new, qkv, step(new, qkv, 5))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(new, qkv, 5)
    expect = np.array([41, 1, 76, 17])
    for i in range(60):
        fresh = [1, int(i % 3 == 0), 1, int(i < 9) * 2 - int(i == 4)]
        new.copy_(dev(fresh))
        qkv.copy_(rand(5, Hq + 2 * Hkv, D, seed=100 + i))
        graph.replay()
        torch.cuda.synchronize()
        follow(new, qkv, res)
        expect += np.maximum(fresh, 0)
        if int(n_free) > 0:
            assert np.array_equal(lens.cpu().numpy(), np.minimum(expect, max_pages * P))
