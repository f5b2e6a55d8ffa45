"""GPU parity of dit_paged_page_mass and dit_paged_evict against their plain forms (prompt_oracle), and a run of all the
operators for prompts together.

Tolerance of the weights: a score is off by at most (D / 16) 17 2^-23 of scale sum_d |q_d k_d| (as in test_prefill_gpu), its
difference to the lse and the exponential by 2^-21 of 1 and of the score's size, sums of up to 2^17 weights in 32 bits,
in chains of at most 2^12, by 2^-12 of the sum in the worst case and its root in practice: each weight's size (1 +
scale sum |q k|) times 2^-17, plus 2^-18 of the page's sum, old weight included, covers the sizes here (chains of 2^6)."""
import math

import numpy as np
import pytest
import torch

import prompt_oracle as po
from diffusion_transformer_long_gb300 import ditattn as da
from test_paged_gpu import cache_view, rand, tables
from test_prefill_gpu import Step

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(DEV, dtype)


def check_mass(s, window=0, decode=False, start=None):
    """s: a Step; its attention's lse, then the weights."""
    out, lse = s.run(True, start=start, fill=0.0)
    mass = torch.rand(s.n_pages, s.k.shape[1], device=DEV, generator=torch.Generator(DEV).manual_seed(1)) * 3
    kw = dict(cu_new=None if decode else s.cu, start_lens=start, window=window)
    res = torch.full_like(mass, -5.0)
    got = da.paged_page_mass(s.q, lse, s.k, s.table, s.lens, mass, mass_out=res, **kw)
    assert got is res
    want, size = po.page_mass(s.q, lse, s.k, s.table, s.lens, mass, s.scale, **kw)
    touched = torch.zeros(s.n_pages, dtype=torch.bool)
    cu = np.arange(len(s.lens_h) + 1) if decode else np.asarray(s.cu.cpu())
    lens = s.lens.cpu().numpy()
    for b in range(len(lens)):
        if min(cu[b + 1], s.T) > max(0, cu[b]):
            t = s.table[b, :-(-min(max(0, int(lens[b])), s.table.shape[1] * s.P) // s.P)].cpu()
            touched[t[(t >= 0) & (t < s.n_pages)].long()] = True
    got = got.cpu().double()
    assert (got[~touched] == -5).all()
    tol = 2.0 ** -17 * size + 2.0 ** -18 * want.abs() + 1e-30
    bad = ~((got - want).abs() <= tol) & touched[:, None]
    assert not bad.any(), f"{bad.sum()} off, worst {float(((got - want).abs() / tol)[touched].max())}"
    again = mass.clone()  # in place: the same sums, other pages untouched
    da.paged_page_mass(s.q, lse, s.k, s.table, s.lens, again, **kw)
    assert torch.equal(again.cpu()[touched], res.cpu()[touched]) and torch.equal(again.cpu()[~touched], mass.cpu()[~touched])


@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (6, 2, 128), (16, 1, 64), (24, 1, 128), (40, 1, 128), (130, 1, 64)])
@pytest.mark.parametrize("P", [16, 48, 64, 80, 128, 512, 1024])
def test_mass_of_single_tokens(P, Hq, Hkv, D):
    s = Step([0, 15, 100, 1000, 3 * P - 1, 2 * P], [1] * 6, min(Hq, 128), Hkv, D, P, seed=P)
    check_mass(s, decode=True)
    check_mass(s, window=3)


@pytest.mark.parametrize("order", ["hnd", "nhd", "part"])
@pytest.mark.parametrize("window", [0, 1, 7, 40, 1000])
def test_mass_of_windows(window, order):
    for P, Hq, Hkv, D in ((16, 6, 2, 128), (64, 4, 4, 64), (128, 5, 1, 128)):
        s = Step([0, 300, 77, 0, 512], [130, 45, 1, 0, 64], Hq, Hkv, D, P, order, spare=3, seed=window)
        check_mass(s, window)


def test_mass_many_requests():
    rng = np.random.default_rng(5)
    for B in (70, 300):
        s = Step(rng.integers(0, 200, B), rng.integers(0, 3, B), 4, 2, 64, 16, seed=B)
        check_mass(s)


@pytest.mark.parametrize("columns,P", [(0, 64), (2048, 64), (2500, 48), (150, 1024)])
def test_mass_runs_of_pages(columns, P):
    """The table's room sets how many pages a block takes at a time."""
    s = Step([9000, 4097, 0, 2100], [33, 20, 30, 1], 6, 2, 128, P, seed=columns)
    if columns:
        s.table = torch.cat([s.table, torch.full((4, columns), -1, dtype=torch.int32, device=DEV)], 1).contiguous()
    check_mass(s, 20)


def test_mass_unusual_contents():
    """Positions anywhere, entries outside the pool, lengths below 0, rows without a key, keys that are not finite."""
    s = Step([64, 300, 10], [40, 33, 6], 6, 2, 64, 32, spare=4)
    s.table[1, 2], s.table[1, 5], s.table[0, 0] = -1, s.n_pages, 2 ** 31 - 1
    check_mass(s)
    check_mass(s, 5)
    for start in ([0, 0, 0], [-30, 310, 4], [2 ** 31 - 1, -2 ** 31, 16]):
        check_mass(s, start=dev(start))
    s.lens = dev([-4, 333, 16])
    check_mass(s)
    s = Step([90], [20], 2, 1, 64, 16)
    s.lens, page = dev([110]), int(s.table[0, 6])
    s.k[page, :, 14:] = math.nan  # behind the last key
    check_mass(s)
    out, lse = s.run()
    lse[3, 1] = -math.inf
    lse[7, 0] = math.nan
    got = da.paged_page_mass(s.q, lse, s.k, s.table, s.lens, torch.zeros(s.n_pages, 1, device=DEV), cu_new=s.cu)
    seen = s.table[0, :7].long()  # token 7, at position 97, sees the pages up to its own
    assert got[seen].isnan().all()
    got = da.paged_page_mass(s.q, lse, s.k, s.table, s.lens, torch.zeros(s.n_pages, 1, device=DEV), cu_new=s.cu, window=5)
    assert got.isfinite().all()


def test_mass_streams_graphs_and_large_offsets():
    s = Step([3000, 40], [40, 7], 6, 2, 128, 16)
    _, lse = s.run()
    mass = torch.rand(s.n_pages, 2, device=DEV)
    want = da.paged_page_mass(s.q, lse, s.k, s.table, s.lens, mass, cu_new=s.cu, mass_out=mass.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mass.clone()
    side.wait_stream(torch.cuda.current_stream())
    da.paged_page_mass(s.q, lse, s.k, s.table, s.lens, got, cu_new=s.cu, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    res, g = mass.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        da.paged_page_mass(s.q, lse, s.k, s.table, s.lens, mass, cu_new=s.cu, mass_out=res)
    g.replay()
    assert torch.equal(res, want)
    n_pages, Hkv, P, D = 270000, 2, 64, 64
    assert n_pages * Hkv * P * D > 2 ** 31
    s = Step([1300], [70], 4, Hkv, D, P)
    _, lse = s.run()
    k = torch.empty(n_pages, Hkv, P, D, dtype=torch.bfloat16, device=DEV)
    to = torch.arange(s.table.shape[1], device=DEV, dtype=torch.int32) * 997 + n_pages - 997 * s.table.shape[1]
    n = -(-int(s.lens_h[0]) // P)
    for i in range(n):
        k[int(to[i])] = s.k[int(s.table[0, i])]
    small = da.paged_page_mass(s.q, lse, s.k, s.table, s.lens, torch.zeros(s.n_pages, Hkv, device=DEV), cu_new=s.cu)
    big = da.paged_page_mass(s.q, lse, k, to[None], s.lens, torch.zeros(n_pages, Hkv, device=DEV), cu_new=s.cu)
    assert torch.equal(big[to[:n].long()], small[s.table[0, :n].long()])


# ------------------------------------------------------------------ eviction


def evict_state(lens, P, H, seed=0, extra_cols=2, capacity=None, n_free=3):
    t, n_pages = tables(lens, P, seed=seed, extra_pages=4, extra_cols=extra_cols)
    g = torch.Generator(DEV).manual_seed(seed)
    mass = torch.rand(n_pages, H, device=DEV, generator=g) ** 4
    stack = np.full(n_pages if capacity is None else capacity, -9)
    stack[:n_free] = np.arange(n_free)
    return mass, dev(t), dev(lens), dev(stack), dev([n_free])


def check_evict(mass, table, lens, stack, n_free, P, keep, recent):
    want = po.evict(mass, table, lens, stack, n_free, P, keep, recent)
    before = [x.clone() for x in (mass, table, lens, n_free)]
    t_out, st = torch.full_like(table, 77), stack.clone()
    got_lens, got_free = da.paged_evict(mass, table, lens, st, n_free, P, keep, recent, table_out=t_out)
    for name, g, w in (("table", t_out, want[0]), ("lens", got_lens, want[1]), ("stack", st, want[2])):
        assert np.array_equal(g.cpu().numpy(), w), name
    assert int(got_free) == want[3]
    same = lambda a, b: torch.equal(a.view(torch.int32), b.view(torch.int32))  # noqa: E731 (NaN too)
    assert all(same(a, b) for a, b in zip(before, (mass, table, lens, n_free)))
    t2, l2, s2, f2 = table.clone(), lens.clone(), stack.clone(), n_free.clone()  # in place
    da.paged_evict(mass, t2, l2, s2, f2, P, keep, recent, seq_lens_out=l2, n_free_out=f2)
    assert np.array_equal(t2.cpu().numpy(), want[0]) and np.array_equal(l2.cpu().numpy(), want[1])
    assert np.array_equal(s2.cpu().numpy(), want[2]) and int(f2) == want[3]


@pytest.mark.parametrize("keep,recent", [(1, 1), (2, 1), (7, 7), (7, 3), (40, 4), (600, 1), (5000, 5000)])
@pytest.mark.parametrize("P,H", [(16, 1), (16, 8), (64, 24)])
def test_evict(P, H, keep, recent):
    for seed, lens in enumerate(([1], [0, 17, 300, 5000], [P * 40, P * 40 + 1, P * 41, P * 7, P * 7 + 1], [P * 20000 + 3, 9])):
        check_evict(*evict_state(lens, P, H, seed), P, keep, recent)


def test_evict_many_requests():
    rng = np.random.default_rng(2)
    for B in (300, 2500, 8192):
        check_evict(*evict_state(rng.integers(0, 400, B), 16, 2, B), 16, 9, 2)


def test_evict_equal_and_unusual_weights():
    """Ties go to the lower index; NaN stays, infinities in their places, -0 is 0, entries outside the pool go first."""
    mass, table, lens, stack, n_free = evict_state([16 * 500, 16 * 30], 16, 4)
    for value in (0.0, 1.5):
        mass.fill_(value)
        check_evict(mass, table, lens, stack, n_free, 16, 20, 5)
    mass[::2] *= -1
    mass[::7, 1] = -0.0
    check_evict(mass, table, lens, stack, n_free, 16, 20, 5)
    mass.copy_(torch.randint(0, 3, mass.shape, device=DEV).float())
    check_evict(mass, table, lens, stack, n_free, 16, 100, 5)
    mass.uniform_()
    mass[table[0, 10].long(), 2], mass[table[0, 400].long(), 0] = math.nan, math.nan
    mass[table[0, 20].long(), 1], mass[table[0, 30].long(), 1] = math.inf, -math.inf
    mass[table[0, 40].long(), :2] = torch.tensor([math.inf, -math.inf], device=DEV)
    mass[table[0, 50].long()] = 3e38  # more than 32 bits hold, in sum
    mass[table[0, 60].long()] = 1e-42
    for keep, recent in ((6, 1), (3, 1), (2, 2), (499, 1)):
        check_evict(mass, table, lens, stack, n_free, 16, keep, recent)
    table[0, 3:200:5], table[1, 0], table[0, 499] = -1, mass.shape[0], -7
    for keep, recent in ((6, 2), (450, 3), (480, 1), (28, 1)):
        check_evict(mass, table, lens, stack, n_free, 16, keep, recent)
    # equal weights but for their last bit in 64 bits
    m2, t2, l2, s2, f2 = evict_state([16 * 100], 16, 2)
    m2[:, 0], m2[:, 1] = 1.0, 0.0
    for i in (3, 50, 71):
        m2[t2[0, i].long(), 1] = 2.0 ** -40
    check_evict(m2, t2, l2, s2, f2, 16, 3, 1)


def test_evict_unusual_lengths_and_stacks():
    mass, table, lens, stack, n_free = evict_state([16 * 50, 16 * 60, 5], 16, 2)
    for ls in ([-3, 16 * 60, 5], [2 ** 31 - 1, -2 ** 31, 16 * 61]):
        check_evict(mass, table, dev(ls), stack, n_free, 16, 10, 2)
    for free in (-4, 0, 10 ** 6):
        check_evict(mass, table, lens, stack, dev([free]), 16, 10, 2)
    check_evict(mass, table, lens, stack[:20].clone(), n_free, 16, 10, 2)  # too small a stack
    wide = torch.full((3, table.shape[1] + 9), 5, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    want = po.evict(mass, table, lens, stack, n_free, 16, 10, 2)
    da.paged_evict(mass, wide[:, :table.shape[1]], lens, stack.clone(), n_free, 16, 10, 2)
    assert np.array_equal(wide[:, :table.shape[1]].cpu().numpy(), want[0]) and (wide[:, table.shape[1]:] == 5).all()


def test_evict_graphs_and_streams():
    mass, table, lens, stack, n_free = evict_state([16 * 300, 16 * 100 + 3, 40], 16, 8)
    bufs = [x.clone() for x in (table, lens, stack, n_free)]
    t, l, s, f = bufs
    g = torch.cuda.CUDAGraph()
    da.paged_evict(mass, t.clone(), l, s.clone(), f, 16, 50, 4)
    with torch.cuda.graph(g):
        da.paged_evict(mass, t, l, s, f, 16, 50, 4, seq_lens_out=l, n_free_out=f)
    for seed in (1, 2):
        mass.uniform_()
        for x, y in zip(bufs, (table, lens, stack, n_free)):
            x.copy_(y)
        want = po.evict(mass, table, lens, stack, n_free, 16, 50, 4)
        g.replay()
        for x, w in zip(bufs, want):
            assert np.array_equal(x.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))
        g.replay()  # within the budget now: nothing changes
        for x, w in zip(bufs, want):
            assert np.array_equal(x.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))


# ------------------------------------------------------------------ all together


def test_a_step_of_prompts_captured_and_replayed():
    """Plan, norms and positions, write, attention, weights, eviction as one captured step, replayed as the lengths grow
    and shrink, against the same caches kept by hand; then a decode step on what is left."""
    B, Hq, Hkv, D, P, n_pages, T = 3, 6, 2, 128, 16, 120, 96
    freqs, _, scale = da.rope_freqs(D)
    k_cache, v_cache = (torch.zeros(n_pages, Hkv, P, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    summary, mass = torch.zeros(n_pages, Hkv, 2, D, dtype=torch.bfloat16, device=DEV), torch.zeros(n_pages, Hkv, device=DEV)
    table = torch.full((B, 80), -1, dtype=torch.int32, device=DEV)
    lens, at, new = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(3))
    stack, n_free = torch.arange(n_pages, dtype=torch.int32, device=DEV), dev([n_pages])
    qkv = torch.zeros(T, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)
    qw, kw = (rand(D, seed=i).float() * 0.1 + 1 for i in (1, 2))
    out = torch.zeros(T, Hq, D, device=DEV)
    lse = torch.zeros(T, Hq, device=DEV)
    seen = torch.zeros(B, dtype=torch.int32, device=DEV)

    def step():
        before = lens.clone()
        _, _, cu, slots = da.paged_plan(new, lens, table, stack, n_free, P, n_pages, T, seq_lens_out=lens, n_free_out=n_free)
        seen.copy_(lens)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        q, k = da.qk_norm_rope(q, k, freqs=freqs, eps=1e-6, q_weight=qw, k_weight=kw, cu_new=cu, start_lens=at)
        da.paged_kv_write(k, v, slots, k_cache, v_cache, summary=summary)
        da.paged_prefill_fwd(q, k_cache, v_cache, table, lens, cu, start_lens=before, out=out, lse=lse)
        da.paged_page_mass(q, lse, k_cache, table, lens, mass, cu_new=cu, start_lens=before, window=8)
        at.add_(new)
        da.paged_evict(mass, table, lens, stack, n_free, P, keep=10, recent=2, seq_lens_out=lens, n_free_out=n_free)

    state = (k_cache, v_cache, summary, mass, table, lens, at, stack, n_free)
    fresh = [x.clone() for x in state]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for x, y in zip(state, fresh):
        x.copy_(y)
    rows = [[] for _ in range(B)]  # by hand: (position, key, value, page) of each cached token
    weight = {}
    for i, ns in enumerate(([50, 0, 7], [40, 30, 20], [1, 80, 1], [60, 1, 30], [1, 1, 1], [30, 30, 30])):
        new.copy_(dev(ns))
        qkv.copy_(rand(T, Hq + 2 * Hkv, D, seed=100 + i))
        first = at.cpu().tolist()
        g.replay()
        da.check(DEV)
        row = 0
        for b, n in enumerate(ns):
            if n == 0:
                continue
            part = qkv[row:row + n].transpose(0, 1)[None]
            pos = torch.arange(first[b], first[b] + n)[None, None]
            q, _ = po.norm_rope(part[:, :Hq], qw, 1e-6, freqs, [D // 2], pos, False, scale)
            k, _ = po.norm_rope(part[:, Hq:Hq + Hkv], kw, 1e-6, freqs, [D // 2], pos, False, scale)
            q, k, v = q.bfloat16().double()[0], k.bfloat16().double()[0], part[0, Hq + Hkv:].cpu().double()
            old = len(rows[b])
            rows[b] += [(k[:, j], v[:, j]) for j in range(n)]
            assert int(seen[b]) == len(rows[b])
            K, V = (torch.stack([r[c] for r in rows[b]], 1).repeat_interleave(Hq // Hkv, 0) for c in range(2))
            s = q @ K.transpose(1, 2) / math.sqrt(D)
            s = s.masked_fill(torch.arange(len(rows[b]))[None, :] > old + torch.arange(n)[:, None], -math.inf)
            w = torch.softmax(s, 2)
            err = (out[row:row + n].cpu().double().transpose(0, 1) - w @ V).abs().max()
            # keys and queries may be rounded to the other side (2^-8 of scores up to a few), weights by 2^-8
            assert err < 0.1, float(err)
            drawn = w[:, max(0, n - 8):].sum((0, 1))
            m = weight.setdefault(b, [])
            m += [0.0] * (-(-len(rows[b]) // P) - len(m))
            for c in range(len(m)):
                x = float(drawn[c * P:(c + 1) * P].sum())
                m[c] = x if c * P >= old else m[c] + x
            row += n
        # eviction by hand, by the weights on the device (the hand's differ in their last bits)
        for b in range(B):
            m = weight.get(b, [])
            if len(m) <= 10:
                continue
            order = sorted(range(len(m) - 2), key=lambda c: (-m[c], c))
            stay = sorted(order[:8]) + [len(m) - 2, len(m) - 1]
            border = m[order[7]] - m[order[8]]
            assert border > 1e-3 * m[order[7]], "inputs too even to tell the kept pages by hand"
            rows[b] = [r for c in stay for r in rows[b][c * P:(c + 1) * P]]
            weight[b] = [m[c] for c in stay]
        assert lens.cpu().tolist() == [len(r) for r in rows]
        used = sum(-(-len(r) // P) for r in rows)
        assert int(n_free) == n_pages - used
        live = torch.cat([table[b, :-(-len(rows[b]) // P)] for b in range(B)]).cpu().tolist()
        assert sorted(live + stack[:int(n_free)].cpu().tolist()) == list(range(n_pages))
    q = rand(B, Hq, D, seed=9)
    got, _ = da.paged_attn_fwd(q, k_cache, v_cache, table, lens)
    for b in range(B):
        K, V = (torch.stack([r[c] for r in rows[b]], 1).repeat_interleave(Hq // Hkv, 0) for c in range(2))
        w = torch.softmax((q[b].cpu().double()[:, None] @ K.transpose(1, 2)) / math.sqrt(D), 2)
        assert ((w @ V)[:, 0] - got[b].cpu().double()).abs().max() < 0.1
