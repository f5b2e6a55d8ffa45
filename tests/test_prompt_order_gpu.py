"""The operators for prompts behind a kernel that lets them start early and writes their inputs late (as
test_paged_order_gpu has it for the others): every call must see what that kernel wrote, eagerly and captured."""
import numpy as np
import pytest
import torch

from diffusion_transformer_long_gb300 import ditattn as da
from test_paged_order_gpu import late_copy  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
B, Hq, Hkv, D, P, N_PAGES, T = 5, 6, 2, 64, 16, 260, 200


class Inputs:
    """All inputs as views of one allocation."""

    def __init__(self, max_pages):
        bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
        shapes = dict(lens=((B,), i32), cu=((B + 1,), i32), start=((B,), i32), n_free=((4,), i32), free=((N_PAGES,), i32),
                      table=((B, max_pages), i32), pos=((3, T), i32), freqs=((32,), f32), w=((D,), f32), lse=((T, Hq), f32),
                      mass=((N_PAGES, Hkv), f32), qkv=((T, Hq + 2 * Hkv, D), bf), k=((N_PAGES, Hkv, P, D), bf),
                      v=((N_PAGES, Hkv, P, D), bf))
        at, places = 0, {}
        for name, (shape, t) in shapes.items():
            n = int(np.prod(shape)) * t.itemsize
            places[name] = (at, n, shape, t)
            at += -(-n // 256) * 256
        self.raw = torch.zeros(at, dtype=torch.uint8, device=DEV)
        for name, (lo, n, shape, t) in places.items():
            setattr(self, name, self.raw[lo:lo + n].view(t).view(shape))

    def fill(self, seed):
        rng = np.random.default_rng(seed)
        put = lambda x, y: x.copy_(torch.as_tensor(np.asarray(y)))  # noqa: E731
        new = rng.integers(0, 40, B)
        put(self.cu, np.concatenate(([0], np.cumsum(new))))
        put(self.lens, new + rng.integers(0, 50 * P - 40, B))
        put(self.start, rng.integers(0, 100000, B))
        order = rng.permutation(N_PAGES)
        put(self.free[:10], order[250:])
        put(self.n_free, [int(rng.integers(4, 11))] * 4)
        self.table.fill_(-1)
        put(self.table[:, :50], order[:250].reshape(B, 50))
        put(self.pos, rng.integers(0, 1000, (3, T)))
        put(self.freqs, rng.random(32, np.float32))
        put(self.w, 1 + rng.standard_normal(D, np.float32))
        put(self.lse, 6 + rng.random((T, Hq), np.float32))
        put(self.mass, rng.random((N_PAGES, Hkv), np.float32))
        for x in (self.qkv, self.k, self.v):
            x.copy_(torch.as_tensor(rng.standard_normal(tuple(x.shape), np.float32)))
        return self

    @property
    def q(self):
        return self.qkv[:, :Hq]


def rope_packed(x):
    out = [torch.zeros(T, h, D, dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv)]
    return da.qk_norm_rope(x.q, x.qkv[:, Hq:Hq + Hkv], freqs=x.freqs, eps=1e-6, q_weight=x.w, k_weight=x.w, cu_new=x.cu,
                           start_lens=x.start, q_out=out[0], k_out=out[1])


def rope_axes_in_place(x):
    q, k = x.q, x.qkv[:, Hq:Hq + Hkv]
    da.qk_norm_rope(q, k, positions=x.pos, freqs=x.freqs, axis_pairs=(8, 8, 16), interleaved=True, q_out=q, k_out=k)
    return (x.qkv,)


def prefill(x):
    out, lse = torch.zeros(T, Hq, D, device=DEV), torch.zeros(T, Hq, device=DEV)
    return da.paged_prefill_fwd(x.q, x.k, x.v, x.table, x.lens, x.cu, out=out, lse=lse)


def mass(x):
    return (da.paged_page_mass(x.q, x.lse, x.k, x.table, x.lens, x.mass, cu_new=x.cu),)


def mass_few(x):
    return (da.paged_page_mass(x.q, x.lse, x.k, x.table, x.lens, x.mass, cu_new=x.cu, window=2),)


def evict(x):
    return (*da.paged_evict(x.mass, x.table, x.lens, x.free, x.n_free[:1], P, 20, 3, seq_lens_out=x.lens,
                            n_free_out=x.n_free[:1]), x.table, x.free)


def step(x):
    q, k = x.q, x.qkv[:, Hq:Hq + Hkv]
    da.qk_norm_rope(q, k, freqs=x.freqs, eps=1e-6, cu_new=x.cu, start_lens=x.start, q_out=q, k_out=k)
    out, lse = prefill(x)
    da.paged_page_mass(q, lse, x.k, x.table, x.lens, x.mass, cu_new=x.cu, window=16)
    return (out, lse, x.mass.clone(), *evict(x))


@pytest.mark.parametrize("room", [50, 400], ids=["whole items", "items in parts"])
@pytest.mark.parametrize("call", [rope_packed, rope_axes_in_place, prefill, mass, mass_few, evict, step],
                         ids=lambda f: f.__name__)
def test_inputs_written_late(late_copy, call, room):  # noqa: F811
    x = Inputs(room)
    graph, res = torch.cuda.CUDAGraph(), None
    fresh = Inputs(room).fill(0)
    call(x.fill(1))
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        late_copy(fresh.raw, x.raw)
        res = call(x)
    for i in range(6):
        fresh.fill(10 + i)
        x.raw.copy_(fresh.raw)
        torch.cuda.synchronize()
        want = [y.clone() for y in call(x)]
        torch.cuda.synchronize()
        for replayed in (False, True):
            x.fill(100 + i)
            torch.cuda.synchronize()
            if replayed:
                graph.replay()
                got = res
            else:
                late_copy(fresh.raw, x.raw)
                got = call(x)
            torch.cuda.synchronize()
            da.check()
            for j, (a, b) in enumerate(zip(got, want)):
                assert torch.equal(a, b), (i, replayed, j)
