"""GPU parity of dit_paged_prefill_fwd against its plain 64-bit form (prompt_oracle).

Tolerances, from the arithmetic (S = scale max_j sum_d |q_d k_jd| over the keys that the row sees,
A = sum_j p_j |v_j| for the channel):
  - a score is a sum of D exact products in 32 bits, in D / 16 steps of 16 products and the running
    sum, each term kept to within 2^-23 of the step's largest: off by at most
    (D / 16) * 17 * 2^-23 * S =: E;
  - a weight is off by a factor of at most exp(E) (score), 2^-21 (exponential), and in the product by 2^-8 (its
    rounding to bf16); the sum that divides it is of the rounded weights, so that a channel is off by at most
    2 (E + 2^-8 + 2^-20) A for those, n 2^-23 A for the product's accumulation over n keys in 32 bits, and half a step
    of the output's type;
  - |lse - lse_ref| <= E + 2^-19 + n 2^-26 + 2^-23 |lse| (a row's sum of n terms runs in 8 chains of 32 bits).
These are worst cases; the roundings of many weights are of random sign, so the 2-norm of the error over a whole
output of many keys is also held to 2^-8 of the norm of A (bf16 output: 2^-7).
"""
import math

import numpy as np
import pytest
import torch

import prompt_oracle as po
from diffusion_transformer_long_gb300 import ditattn as da
from test_paged_gpu import cache_view, rand, tables

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(DEV, dtype)


@pytest.fixture(autouse=True)
def no_timeouts():
    yield
    da.set_grid_limit(0)
    da.check(DEV)


class Step:
    """A step of requests with `old` cached and `new` new tokens each, its cache and queries."""

    def __init__(self, old, new, Hq, Hkv, D, P, order="hnd", spare=0, seed=0, room=0, scale=1.5):
        old, new = np.asarray(old), np.asarray(new)
        self.lens_h, self.new_h, self.P = old + new, new, P
        t, n_pages = tables(self.lens_h, P, seed=seed)
        if room:  # room for so many keys: the table's width decides the launch
            t = np.concatenate((t, np.full((len(t), max(0, room // P - t.shape[1])), -1)), 1)
        self.table, self.n_pages = dev(t), n_pages
        self.lens, self.cu = dev(self.lens_h), dev(np.concatenate(([0], np.cumsum(new))))
        self.T = max(1, int(new.sum()) + spare)
        self.q = rand(self.T, Hq + 2 * Hkv, D, seed=seed + 1, scale=scale)[:, :Hq]
        self.k, self.v = (cache_view(n_pages, Hkv, P, D, order, seed=seed + 2 + i) for i in range(2))
        self.shape = (self.T, Hq, D)
        self.scale = D ** -0.5

    def run(self, causal=True, out_dtype=torch.float32, start=None, fill=None, **kw):
        out = lse = None
        if fill is not None:
            out = torch.full(self.shape, fill, device=DEV, dtype=out_dtype)
            lse = torch.full(self.shape[:2], fill, device=DEV)
        return da.paged_prefill_fwd(self.q, self.k, self.v, self.table, self.lens, self.cu, start_lens=start,
                                    causal=causal, out=out, lse=lse, out_dtype=out_dtype, **kw)

    def check(self, causal=True, out_dtype=torch.float32, start=None, device="cpu", got=None):
        out, lse = got or self.run(causal, out_dtype, start, fill=7.0)
        da.check(DEV)
        o, l, owned, (mag, pv) = po.attend(self.q, self.k, self.v, self.table, self.lens, self.cu, self.scale, causal,
                                           start, device)
        compare(out, lse, o, l, owned, mag, pv, int(max(1, self.lens_h.max())), got is None)
        return out, lse


def compare(out, lse, o, l, owned, mag, pv, n, filled=True, ok=None):
    """ok: elements of `out` to look at (all by default)."""
    D = out.shape[2]
    E = D / 16 * 17 * 2.0 ** -23 * mag
    half = 0 if out.dtype == torch.float32 else 2.0 ** -8
    got, got_l = out.double().cpu(), lse.double().cpu()
    if filled and not owned.all():
        assert (got[~owned] == 7).all() and (got_l[~owned] == 7).all(), "rows of no request were written"
    tol = 2 * (E[..., None] + 2.0 ** -8 + 2.0 ** -20) * pv + n * 2.0 ** -23 * pv
    tol = tol + half * (o.abs() + tol) + 1e-30
    good = (got - o).abs() <= tol
    if ok is not None:
        good |= ~ok
    good = good[owned]
    assert good.all(), f"{(~good).sum()} of {good.numel()} outputs off, first at {torch.nonzero(~good)[0].tolist()}"
    none = l == -math.inf
    assert (got_l[owned & none.all(1)] == -math.inf).all()
    tl = E + 2.0 ** -19 + n * 2.0 ** -26 + 2.0 ** -23 * l.abs().nan_to_num(posinf=0)
    bad = ~(((got_l - l).abs() <= tl) | (none & (got_l == l)))
    assert not bad[owned].any(), f"lse off at {torch.nonzero(bad & owned[:, None])[0].tolist()}"
    if ok is None and owned.any() and n > 512:
        err = (got - o)[owned].norm() / pv[owned].norm()
        assert err <= (2.0 ** -8 if out.dtype == torch.float32 else 2.0 ** -7), float(err)


HEADS = [(1, 1, 64), (2, 2, 64), (3, 1, 128), (6, 2, 128), (10, 2, 64), (16, 1, 64), (24, 1, 128), (40, 1, 128), (128, 1, 64)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_one_request(Hq, Hkv, D, causal):
    """Every group size at the lengths around a tile's and an item's ends, whole items."""
    tt = 128 // (Hq // Hkv)
    for old, new in ((0, 1), (5, 2), (0, tt), (120, tt + 1), (0, 2 * tt), (130, 2 * tt + 1), (300, 1)):
        Step([old], [new], Hq, Hkv, D, 16, seed=old + new).check(causal, torch.bfloat16 if old else torch.float32)


@pytest.mark.parametrize("order", ["hnd", "nhd", "part"])
@pytest.mark.parametrize("P", [16, 32, 48, 64, 80, 128, 192, 1024])
def test_page_sizes(P, order):
    for causal in (True, False):
        Step([0, 100, 513, 0, 7], [300, 1, 77, 0, 130], 6, 2, 128, P, order, spare=3, seed=P).check(causal)
    Step([200, 0], [19, 40], 2, 1, 64, P, order, seed=P).check(out_dtype=torch.bfloat16)


@pytest.mark.parametrize("limit", [0, 1, 2, 7])
@pytest.mark.parametrize("D", [64, 128])
def test_split_items(D, limit):
    """Items of many key tiles, dealt out over all blocks, and over few that walk many items each."""
    da.set_grid_limit(limit)
    for Hq, Hkv in ((2, 2), (6, 2), (16, 1)):
        for old, new in (([3000], [5]), ([2000, 0, 900], [1, 700, 0]), ([0, 31, 5000], [129, 1, 300])):
            s = Step(old, new, Hq, Hkv, D, 32, seed=limit, spare=2, room=6000)
            s.check(True, torch.bfloat16 if limit else torch.float32)
            s.check(False)


@pytest.mark.parametrize("room", [0, 4096])
def test_many_requests(room):
    rng = np.random.default_rng(3)
    for B, hi in ((200, 40), (33, 300)):
        new = rng.integers(0, hi, B) * (rng.random(B) < 0.7)
        s = Step(rng.integers(0, 400, B), new, 4, 2, 64, 16, spare=11, seed=B, room=room)
        s.check(True, torch.bfloat16)


@pytest.mark.parametrize("order", ["hnd", "nhd", "part", "kv in one", "rows of both"])
@pytest.mark.parametrize("P", [16, 48])
def test_copies_of_both_channel_blocks(P, order):
    """Wide tables of small pages: one copy brings both channel blocks of 16 rows, where the strides allow it."""
    for Hq, Hkv in ((6, 2), (4, 1), (3, 3)):
        s = Step([0, 700, 77], [200, 90, 1], Hq, Hkv, 128, P, "part" if order == "part" else "hnd", room=9000, seed=P)
        n = s.n_pages
        if order == "nhd":
            s.k, s.v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (s.k, s.v))
        elif order == "kv in one":
            both = torch.stack((s.k, s.v), 1)
            s.k, s.v = both[:, 0], both[:, 1]
        elif order == "rows of both":
            both = torch.stack((s.k.transpose(1, 2), s.v.transpose(1, 2)), 2).contiguous()
            s.k, s.v = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
        s.table[1, 4], s.table[0, 1] = n + 5, -1
        s.check(True)
        s.check(False)
        page, row = int(s.table[1, (789 - 30) // P]), (789 - 30) % P  # a value that the first 59 tokens do not see
        s.v[page, :, row, 65] = math.inf
        got, _ = s.run()
        first = int(s.cu[1])
        assert got[first:first + 59].isfinite().all() and not got[first + 59:first + 90, :, 65].isfinite().any()


def test_one_page():
    for P in (16, 128):
        for Hq, Hkv in ((2, 1), (4, 2)):
            s = Step([0], [P], Hq, Hkv, 128, P, room=9000)
            k, v = s.k[int(s.table[0, 0])][None].clone(), s.v[int(s.table[0, 0])][None].clone()
            s.table[0, 0] = 0
            s.k, s.v, s.n_pages = k, v, 1
            s.check()


def test_no_tokens_and_no_keys():
    for room in (0, 2048):
        s = Step([0, 40, 0], [0, 0, 0], 2, 1, 64, 16, spare=5, room=room)
        s.check()
        s = Step([0, 0], [3, 4], 2, 1, 64, 16, room=room)
        s.lens = dev([0, -5])
        out, lse = s.run(fill=7.0)
        assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("room", [0, 2048])
def test_unusual_contents(room):
    """Lengths below 0 and past the table, entries outside the pool, first rows out of range and descending,
    positions anywhere."""
    s = Step([64, 300, 10, 500], [40, 33, 6, 200], 6, 2, 64, 32, spare=9, room=room)
    s.table[1, 2] = -1
    s.table[1, 5] = s.n_pages
    s.table[3, 0] = 2 ** 31 - 1
    s.table[3, 7:9] = -9
    for causal in (True, False):
        s.check(causal)
    big = 2 ** 31 - 1
    for start in ([0, 0, 0, 0], [-20, 310, 4, -big - 1], [big, -3, 16, 450], [60, 250, -1000000, 400]):
        s.check(True, start=dev(start))
    s.lens = dev([-4, big, 7, 600])
    s.lens_h = np.array([0, s.table.shape[1] * 32, 7, 600])
    if room == 0:  # (the columns past the pages are -1: no keys)
        s.check(True)
    s.lens, s.lens_h = dev([104, 333, 16, 700]), np.array([104, 333, 16, 700])
    for cu in ([-5, 40, 40, 30, 200], [3, 60, 60, 61, big], [0, 0, 0, 0, s.T]):
        s.cu = dev(cu)
        s.check(True)


def test_values_that_are_not_finite():
    """Infinities and NaN behind a request's last key, or at keys that a row does not see, change nothing; a
    row that sees one has it in its channel."""
    for P, room, Hq, Hkv in ((16, 0, 2, 2), (64, 4096, 6, 2), (48, 4096, 16, 1)):
        s = Step([37, 260, 1000], [300, 77, 130], Hq, Hkv, 128, P, room=room)
        cols = lambda b, j: (int(s.table[b, j // P]), j % P)  # noqa: E731
        clean_v, clean_k = s.v.clone(), s.k.clone()
        for b, n in enumerate(s.lens_h):
            page, row = cols(b, int(n) - 1)
            s.k[page, :, row + 1:] = math.nan
            s.v[page, :, row + 1:] = math.inf
        used = {int(x) for b in range(3) for x in s.table[b, :-(-int(s.lens_h[b]) // P)]}
        for page in set(range(s.n_pages)) - used:
            s.k[page], s.v[page] = math.nan, math.nan
        s.check(True)
        s.check(False)
        want, _ = s.run()
        # one value of the new tokens' own, one of the cached ones
        marks = [(0, 200, 0, 5, math.inf), (0, 300, Hkv - 1, 70, math.nan), (1, 262, 0, 0, -math.inf), (2, 1100, 0, 127, math.nan),
                 (2, 1001, Hkv - 1, 64, math.inf), (1, 3, 0, 9, math.nan)]
        saved = s.v.clone()
        for b, j, h, d, x in marks:
            page, row = cols(b, j)
            s.v[page, h, row, d] = x
        got, _ = s.run()
        touched = torch.zeros(s.shape, dtype=torch.bool, device=DEV)
        G = Hq // Hkv
        for b, j, h, d, x in marks:
            row0, first = int(s.cu[b]), int(s.lens_h[b] - s.new_h[b])
            touched[row0 + max(0, j - first):row0 + int(s.new_h[b]), h * G:(h + 1) * G, d] = True
        assert not got[touched].isfinite().any()
        assert torch.equal(got[~touched], want[~touched])
        # a key that is not finite, seen by the later rows only
        s.v.copy_(saved)
        page, row = cols(0, 250)
        s.k[page, 0, row, 3] = math.nan
        got, lse = s.run()
        hit = torch.zeros(s.shape[:2], dtype=torch.bool, device=DEV)
        hit[250 - 37:300, :G] = True
        assert got[hit].isnan().all() and lse[hit].isnan().all()
        assert torch.equal(got[~hit], want[~hit]) and lse[~hit].isfinite().all()
        s.v.copy_(clean_v)
        s.k.copy_(clean_k)


def test_scores_at_infinity():
    """Scores of -inf weigh nothing, a row of them alone gives 0; +inf makes its row NaN."""
    for room in (0, 4096):
        s = Step([100, 0], [50, 200], 2, 1, 64, 16, room=room)
        s.q.copy_(torch.ones_like(s.q))
        for j in (0, 20, 149):
            s.k[int(s.table[0, j // 16]), 0, j % 16] = -math.inf
        for j in range(130):
            s.k[int(s.table[1, j // 16]), 0, j % 16] = -math.inf
        s.v[int(s.table[1, 0])] = math.nan
        out, lse = s.run()
        first = out[50:50 + 130]
        assert (first == 0).all() and (lse[50:180] == -math.inf).all()
        assert out[:50].isfinite().all() and lse[:50].isfinite().all()
        s.k[int(s.table[0, 7]), 0, 3] = math.inf  # key 115: seen from new token 15 on
        out, lse = s.run()
        assert out[15:50].isnan().all() and lse[15:50].isnan().all() and out[:15].isfinite().all()


def test_single_tokens_agree_with_the_decode_call():
    s = Step([0, 37, 4000, 511], [1, 1, 1, 1], 24, 8, 128, 16, room=5000)
    a, la = s.run()
    b, lb = da.paged_attn_fwd(s.q, s.k, s.v, s.table, s.lens)
    assert (la - lb).abs().max() < 1e-4
    assert (a - b).norm() / b.norm() < 2.0 ** -8  # the weights' rounding


def test_equal_bits_streams_and_graphs():
    """Equal calls give equal bits: again, on another stream, captured and replayed with grown lengths; two graphs with
    workspaces of their own run at once."""
    s = Step([3000, 0, 700], [40, 500, 1], 6, 2, 128, 16, room=8192)
    want = s.run(out_dtype=torch.bfloat16)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(s.run(out_dtype=torch.bfloat16), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = s.run(out_dtype=torch.bfloat16, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(s.run(out_dtype=torch.bfloat16))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for lens in (s.lens_h, s.lens_h - np.array([1000, 0, 600])):
        s.lens.copy_(dev(lens))
        want = s.run(out_dtype=torch.bfloat16)
        torch.cuda.synchronize()
        for _ in range(4):
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for got in outs:
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_past_32_bits():
    """Pages and query rows whose elements lie past 2^31."""
    n_pages, Hkv, P, D = 70000, 4, 64, 128
    assert n_pages * Hkv * P * D > 2 ** 31
    s = Step([1300], [70], 8, Hkv, D, P, room=4096)
    k, v = (torch.empty(n_pages, Hkv, P, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    to = torch.arange(s.table.shape[1], device=DEV, dtype=torch.int32) * 997 + n_pages - 997 * s.table.shape[1]
    n = -(-int(s.lens_h[0]) // P)
    for i in range(n):
        k[int(to[i])], v[int(to[i])] = s.k[int(s.table[0, i])], s.v[int(s.table[0, i])]
    want = s.run()
    got = da.paged_prefill_fwd(s.q, k, v, to[None], s.lens, s.cu)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_expired_wait_is_reported():
    s = Step([300], [40], 2, 1, 64, 16, room=2048)
    try:
        da.inject_stall(True, 2_000_000)
        s.run()
        with pytest.raises(da.DitError) as e:
            da.check(DEV)
        assert e.value.status == da.DIT_ERR_TIMEOUT
    finally:
        da.inject_stall(False)
    s.check()


@pytest.mark.parametrize("limit", [0, 1, 3])
@pytest.mark.parametrize("Hq,Hkv,D,P,room", [(6, 2, 128, 16, 9000), (6, 2, 128, 64, 4096), (8, 1, 64, 32, 0), (3, 3, 64, 16, 3000)])
def test_few_tokens(Hq, Hkv, D, P, room, limit):
    """Steps of few tokens a request: items in turn on the two halves of a block, empty ones and long ones among them."""
    da.set_grid_limit(limit)
    rng = np.random.default_rng(limit)
    old, new = rng.integers(0, 500, 90), rng.integers(0, 6, 90)
    new[7], old[11] = 150, 2900 if room else 900
    s = Step(old, new, Hq, Hkv, D, P, spare=3, seed=P, room=room)
    s.check(True, torch.bfloat16)
    s.check(False)
    none = rng.random(90) < 0.3  # requests without a key
    s.lens_h = np.where(none, 0, s.lens_h)
    s.lens = dev(s.lens_h)
    s.check(True)


@pytest.mark.parametrize("Hq,Hkv", [(40, 1), (64, 1), (33, 1), (96, 2)])
def test_few_tokens_of_large_groups(Hq, Hkv):
    for D in (64, 128):
        for new in ([1], [2], [1] * 20, [0, 3, 0, 0, 1, 0, 0, 0]):
            Step([300] * len(new), new, Hq, Hkv, D, 32, seed=len(new), room=2048).check()


def test_few_tokens_values_that_are_not_finite():
    new = [3, 1, 0, 5, 2, 1]
    s = Step([127, 300, 5, 1000, 62, 0], new, 6, 2, 128, 16, room=4096)
    want = s.run()[0]
    for b in (0, 3, 4):  # the request's last key: its last token sees it
        at = int(s.lens_h[b]) - 1
        s.v[int(s.table[b, at // 16]), 1, at % 16, 9] = math.nan
        if at % 16 < 15:
            s.v[int(s.table[b, at // 16]), :, at % 16 + 1:] = math.inf  # behind the length
    got = s.run()[0]
    mark = torch.zeros_like(got, dtype=torch.bool)
    for b in (0, 3, 4):
        mark[int(s.cu[b + 1]) - 1, 3:, 9] = True
    assert got[mark].isnan().all() and torch.equal(got[~mark], want[~mark])


def test_few_tokens_streams_and_graphs():
    rng = np.random.default_rng(8)
    steps = [Step(rng.integers(0, 3000, 40), rng.integers(1, 5, 40), 6, 2, 128, 64, seed=i, room=4096) for i in range(2)]
    want = [s.run() for s in steps]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in steps]
    for _ in range(5):  # two calls at once
        got = [s.run(stream=st) for s, st in zip(steps, side)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
    graphs = []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = s.run()
        graphs.append((g, out))
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for (_, o), w in zip(graphs, want) for a, b in zip(o, w))


def test_few_tokens_expired_wait_is_reported():
    s = Step([300] * 9, [1] * 9, 2, 1, 64, 16, room=2048)
    try:
        da.inject_stall(True, 2_000_000)
        s.run()
        with pytest.raises(da.DitError) as e:
            da.check(DEV)
        assert e.value.status == da.DIT_ERR_TIMEOUT
    finally:
        da.inject_stall(False)
    s.check()
