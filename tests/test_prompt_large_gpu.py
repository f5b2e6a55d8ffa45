"""The operators for prompts where their caches and groups are large: requests whose items go head by head, page weights of
groups of more than 128 heads, and the whole step behind inputs that are written late."""
import math

import numpy as np
import pytest
import torch

import prompt_oracle as po
from diffusion_transformer_long_gb300 import ditattn as da
from test_paged_order_gpu import late_copy  # noqa: F401 (a fixture)
from test_prefill_gpu import Step, compare
from test_prompt_order_gpu import B, D, DEV, Hkv, Hq, Inputs, N_PAGES, P, T

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_timeouts():
    yield
    da.set_grid_limit(0)
    da.check(DEV)


BORDER = 192 << 20  # bytes of a request's keys and values, above which its items go head by head


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,over,new", [
    ((24, 24, 128), [5], [2000]),                       # more items than blocks
    ((24, 24, 128), [0, 1, None, None], [300, 5, 40, 200]),   # at the border, one key past it, short ones
    ((72, 24, 128), [700, None, 1], [130, 1, 90]),      # a group of three
    ((80, 40, 128), [1, 0, None, 900], [5, 1, 3, 0]),   # few tokens a request: items of one Q tile
    ((40, 40, 64), [1, None, -1], [7, 1, 600])])
def test_items_head_by_head(heads, over, new, causal):
    """Requests of so many keys (more than the border by `over`; None: few), alone and in one batch with others, whole and
    in parts, on the whole GPU and on few blocks."""
    Hq, Hkv, D = heads
    at = BORDER // (4 * Hkv * D)
    lens = [n + 333 if o is None else at + o for o, n in zip(over, new)]
    s = Step(np.array(lens) - np.array(new), new, Hq, Hkv, D, 64, spare=2, seed=len(new))
    assert any(n * 4 * Hkv * D > BORDER for n in lens)
    ref = po.attend(s.q, s.k, s.v, s.table, s.lens, s.cu, s.scale, causal, device=DEV)
    for limit in (0, 1, 7, 40):
        da.set_grid_limit(limit)
        out, lse = s.run(causal, torch.bfloat16 if limit == 7 else torch.float32, fill=7.0)
        compare(out, lse, *ref[:3], *ref[3], max(lens))
        da.check(DEV)


@pytest.mark.parametrize("Hq,Hkv,D", [(129, 1, 64), (129, 1, 128), (200, 1, 64), (400, 2, 128), (256, 1, 128), (512, 2, 64)])
def test_mass_of_large_groups(Hq, Hkv, D):
    """Groups of more heads than the attention of new tokens takes, up to a product's 256 columns, so that each token is a
    column block of its own; the lse is the plain form's."""
    for old, new in (([0, 15, 1000, 77], [1, 1, 1, 1]), ([0, 300, 1000, 77], [5, 3, 40, 0])):
        s = Step(old, new, Hq, Hkv, D, 32, spare=2, seed=Hq)
        single = all(n == 1 for n in new)
        lse = po.attend(s.q, s.k, s.k, s.table, s.lens, s.cu, s.scale)[1].float().to(DEV)
        mass = torch.rand(s.n_pages, Hkv, device=DEV)
        if single:
            s.q, lse = s.q[:4], lse[:4].contiguous()
        for window in (0, 1, 3):
            kw = dict(cu_new=None if single and window < 3 else s.cu, window=window)
            got = da.paged_page_mass(s.q, lse, s.k, s.table, s.lens, mass, mass_out=mass.clone(), **kw)
            want, size = po.page_mass(s.q, lse, s.k, s.table, s.lens, mass, s.scale, **kw)
            # (as in test_mass_evict_gpu: chains of sums of the length there, 64 columns a thread)
            tol = 2.0 ** -17 * size + 2.0 ** -18 * want.abs() + 1e-30
            assert ((got.cpu().double() - want).abs() <= tol).all(), (new, window)


class Late(Inputs):
    """The step's inputs before its plan: lengths without the new tokens, whose numbers are in pos[2]; and its outputs."""

    def __init__(self, max_pages):
        super().__init__(max_pages)
        self.out, self.lse_out = torch.zeros(T, Hq, D, device=DEV), torch.zeros(T, Hq, device=DEV)

    def clear(self):
        self.out.zero_()
        self.lse_out.zero_()

    def fill(self, seed):
        super().fill(seed)
        new = self.cu[1:] - self.cu[:-1]
        self.pos[2, :B].copy_(new)
        self.lens.sub_(new)
        self.clear()
        return self


def whole_step(x):
    """(No kernel but the library's in front of the last call.)"""
    lens, n_free, cu, slots = da.paged_plan(x.pos[2, :B], x.lens, x.table, x.free, x.n_free[:1], P, N_PAGES, T)
    q, k = x.q, x.qkv[:, Hq:Hq + Hkv]
    da.qk_norm_rope(q, k, freqs=x.freqs, eps=1e-6, cu_new=cu, start_lens=x.start, q_out=q, k_out=k)
    da.paged_kv_write(k, x.qkv[:, Hq + Hkv:], slots, x.k, x.v)
    da.paged_prefill_fwd(q, x.k, x.v, x.table, lens, cu, start_lens=x.lens, out=x.out, lse=x.lse_out)
    da.paged_page_mass(q, x.lse_out, x.k, x.table, lens, x.mass, cu_new=cu, start_lens=x.lens, window=16)
    left, free_left = da.paged_evict(x.mass, x.table, lens, x.free, n_free, P, 20, 3)
    return x.out.clone(), x.lse_out.clone(), x.raw.clone(), lens, left, free_left


@pytest.mark.parametrize("room", [50, 400], ids=["whole items", "items in parts"])
def test_whole_step_with_inputs_written_late(late_copy, room):  # noqa: F811
    """Plan, norms and positions, write, attention, weights and eviction behind a kernel that lets them start early and
    writes their inputs late: eagerly and captured."""
    x, fresh = Late(room), Late(room).fill(0)
    graph = torch.cuda.CUDAGraph()
    whole_step(x.fill(1))
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        late_copy(fresh.raw, x.raw)
        res = whole_step(x)
    for i in range(6):
        fresh.fill(10 + i)
        x.raw.copy_(fresh.raw)
        x.clear()
        torch.cuda.synchronize()
        want = [y.clone() for y in whole_step(x)]
        torch.cuda.synchronize()
        assert want[0].isfinite().all() and (want[1] != 0).any() and math.isfinite(float(x.mass.sum()))
        for replayed in (False, True):
            x.fill(100 + i)
            torch.cuda.synchronize()
            if replayed:
                graph.replay()
                got = res
            else:
                late_copy(fresh.raw, x.raw)
                got = whole_step(x)
            torch.cuda.synchronize()
            da.check()
            for j, (a, b) in enumerate(zip(got, want)):
                assert torch.equal(a, b), (i, replayed, j)
