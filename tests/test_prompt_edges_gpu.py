"""Calls of the operators for prompts at the edges of what their documentation allows, on the GPU."""
import numpy as np
import pytest
import torch

import prompt_oracle as po
from diffusion_transformer_long_gb300 import ditattn as da
from test_mass_evict_gpu import evict_state
from test_paged_gpu import rand
from test_prefill_gpu import Step
from test_qk_norm_rope_gpu import close, weight

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(DEV, dtype)


@pytest.fixture(autouse=True)
def no_timeouts():
    yield
    da.set_grid_limit(0)
    da.check(DEV)


# ------------------------------------------------------------------ norms and positions


@pytest.mark.parametrize("inter", [False, True])
def test_interleaved_views_in_place(inter):
    """Slices of one head-major allocation, halves of its tokens: turned in place, what lies beside them as it was."""
    B, N, D = 3, 29, 128
    freqs, pairs, _ = da.rope_freqs(64)
    pos = dev(np.random.default_rng(0).integers(0, 5000, (1, B, N)))
    qw, kw = weight(D, 1), weight(D, 2)
    for which in ("heads", "tokens"):
        x = rand(B, 9, 2 * N if which == "tokens" else N, D, seed=7)
        cut = (lambda t: (t[:, 1:5], t[:, 5:8])) if which == "heads" else (lambda t: (t[:, 2:9, :N], t[:, 2:9, N:]))
        before, (q, k) = x.clone(), cut(x)
        got = da.qk_norm_rope(q, k, pos, freqs, pairs, inter, 1.0, 1e-6, qw, kw, q_out=q, k_out=k)
        assert got[0] is q and got[1] is k
        for y, old, w in zip((q, k), cut(before), (qw, kw)):
            close(y, old, w, 1e-6, freqs, pairs, pos, inter, 1.0)
            old.copy_(y)
        assert torch.equal(x, before)


# ------------------------------------------------------------------ eviction


def test_tables_in_one_allocation():
    """The old and the new table's rows in turn: the result of tables apart."""
    mass, table, lens, stack, n_free = evict_state([16 * 50, 16 * 60 + 3, 5, 16 * 9], 16, 2)
    want = po.evict(mass, table, lens, stack, n_free, 16, 10, 2)
    n = table.shape[1]
    both = torch.full((4, 2, n + 3), 5, dtype=torch.int32, device=DEV)
    for i in (0, 1):
        both.fill_(5)
        old, new = both[:, i, :n], both[:, 1 - i, :n]
        old.copy_(table)
        got_lens, got_free = da.paged_evict(mass, old, lens, stack.clone(), n_free, 16, 10, 2, table_out=new)
        assert np.array_equal(new.cpu().numpy(), want[0]) and torch.equal(old, table) and (both[:, :, n:] == 5).all()
        assert np.array_equal(got_lens.cpu().numpy(), want[1]) and int(got_free) == want[3]


# ------------------------------------------------------------------ attention of new tokens


@pytest.mark.parametrize("n", [1, 100, 300])
def test_items_that_outlast_a_wait(n):
    """The limit of a wait is one of no progress: an item of 1500 key tiles (over 500 us) under a limit of 100 us a step
    ends in order.  All pages are one, so that the outputs are the short request's."""
    P, keys, repeat = 1024, 1024, 190
    q, k, v = rand(n, 1, 64, seed=1), rand(1, 1, P, 64, seed=2), rand(1, 1, P, 64, seed=3)
    table = torch.zeros(1, repeat, dtype=torch.int32, device=DEV)
    cu, want = dev([0, n]), da.paged_prefill_fwd(q, k, v, table[:, :1], dev([keys]), dev([0, n]), causal=False)
    try:
        da.set_grid_limit(1)  # (one block has it all)
        da.inject_stall(False, 200_000)
        out, lse = da.paged_prefill_fwd(q, k, v, table, dev([repeat * keys]), cu, causal=False)
        da.check(DEV)
    finally:
        da.inject_stall(False)
        da.set_grid_limit(0)
    # Sums of 190 times as many equal terms in 32 bits, 2^18 keys: off by at most 2^18 2^-23 of them, twice, in the worst case.
    assert (out - want[0]).abs().max() <= 2.0 ** -4 * v.abs().max()
    assert (lse - want[1] - np.log(repeat)).abs().max() <= 2.0 ** -4


# ------------------------------------------------------------------ page weights


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("old,new", [([300], [40]), ([4000, 0, 700], [100, 30, 1]), ([20000], [300])])
def test_mass_expired_wait_is_reported(old, new, D):
    """With the keys' copies withheld every block's wait runs out, also one of several column blocks and runs; the next
    call is right again."""
    s = Step(old, new, 6, 2, D, 16)
    _, lse = s.run()
    mass = torch.rand(s.n_pages, 2, device=DEV)
    call = lambda: da.paged_page_mass(s.q, lse, s.k, s.table, s.lens, mass, cu_new=s.cu, mass_out=mass.clone())  # noqa: E731
    want = call()
    da.check(DEV)
    try:
        da.inject_stall(True, 2_000_000)
        call()
        with pytest.raises(da.DitError) as e:
            da.check(DEV)
        assert e.value.status == da.DIT_ERR_TIMEOUT
    finally:
        da.inject_stall(False)
    assert torch.equal(call(), want)
