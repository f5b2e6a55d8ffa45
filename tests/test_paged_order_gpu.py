"""The paged operators behind a kernel that lets them start early and writes their inputs late: lengths,
tables, slots, lists, queries, summaries and the caches themselves.  Every call must see what that kernel
wrote, eagerly and in a captured graph, though the old contents were in the caches and are valid inputs."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from diffusion_transformer_long_gb300 import build as dbuild
from diffusion_transformer_long_gb300 import ditattn as da

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
B, Hq, Hkv, D, P, TOP = 5, 6, 2, 64, 16, 7
N_PAGES, T = 130, 90
CYCLES = 60_000  # about 30 us: longer than a launch takes


@pytest.fixture(scope="module")
def late_copy(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("late") / "late_copy.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "late_copy.cu")
    subprocess.run([os.path.join(dbuild.cuda_home(), "bin", "nvcc"), *dbuild.ARCH, "-O2", "-shared", "-Xcompiler",
                    "-fPIC", "-cudart", "shared", "-o", so, src], check=True)
    fn = ctypes.CDLL(so).late_copy_launch
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_longlong, ctypes.c_int, ctypes.c_longlong,
                   ctypes.c_void_p, ctypes.c_void_p]
    sink = torch.zeros(1, dtype=torch.int32, device=DEV)

    def launch(src, dst):
        assert fn(src.data_ptr(), dst.data_ptr(), dst.numel() // 16, 152, CYCLES, sink.data_ptr(),
                  torch.cuda.current_stream().cuda_stream) == 0
    return launch


class Inputs:
    """All inputs of a step as views of one allocation, small ones first."""

    def __init__(self, max_pages):
        bf, i32 = torch.bfloat16, torch.int32
        shapes = dict(lens=((B,), i32), new=((B,), i32), n_free=((4,), i32), free=((N_PAGES,), i32),
                      table=((B, max_pages), i32), slots=((T,), torch.int64), sel=((B, Hkv, TOP), i32),
                      q=((B, Hq, D), bf), kv=((T, 2 * Hkv, D), bf), summary=((N_PAGES, Hkv, 2, D), bf),
                      k=((N_PAGES, Hkv, P, D), bf), v=((N_PAGES, Hkv, P, D), bf))
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
        put(self.lens, rng.integers(0, 20 * P, B))
        put(self.new, rng.integers(0, 18, B))
        order = rng.permutation(N_PAGES)  # the requests' pages, and ten free ones
        put(self.free[:10], order[120:])
        put(self.n_free, [int(rng.integers(4, 11))] * 4)
        self.table.fill_(-1)
        put(self.table[:, :24], order[:120].reshape(B, 24))
        # a page's tokens in ascending slots, as a plan lays them out
        pages, slots = rng.permutation(N_PAGES)[:T // 15], []
        for p in pages:
            first = int(rng.integers(0, 2))
            slots += [p * P + r for r in range(first, first + 15)]
        put(self.slots, (slots + [-1] * T)[:T])
        put(self.sel, np.sort(rng.integers(0, 20, (B, Hkv, TOP)), 2))
        for x in (self.q, self.kv, self.k, self.v):
            x.copy_(torch.as_tensor(rng.standard_normal(tuple(x.shape), np.float32)))
        self.summary.copy_(torch.stack((self.k.amin(2), self.k.amax(2)), 2))
        return self


def plan(x):
    return da.paged_plan(x.new, x.lens, x.table, x.free, x.n_free[:1], P, N_PAGES, T) + (x.table,)


def plan_in_place(x):
    return da.paged_plan(x.new, x.lens, x.table, x.free, x.n_free[:1], P, N_PAGES, 5000, seq_lens_out=x.lens,
                         n_free_out=x.n_free[:1]) + (x.table,)


def write(x):
    da.paged_kv_write(x.kv[:, :Hkv], x.kv[:, Hkv:], x.slots, x.k, x.v)
    return x.k, x.v


def write_summary(x):
    da.paged_kv_write(x.kv[:, :Hkv], x.kv[:, Hkv:], x.slots, x.k, x.v, summary=x.summary)
    return x.k, x.v, x.summary


def select(x):
    return (da.paged_select(x.q, x.summary, x.table, x.lens, P, TOP),)


def attn(x):
    return da.paged_attn_fwd(x.q, x.k, x.v, x.table, x.lens)


def attn_selected(x):
    return da.paged_attn_fwd(x.q, x.k, x.v, x.table, x.lens, selected=x.sel)


def step(x):
    lens, _, _, slots = da.paged_plan(x.new, x.lens, x.table, x.free, x.n_free[:1], P, N_PAGES, T)
    da.paged_kv_write(x.kv[:, :Hkv], x.kv[:, Hkv:], slots, x.k, x.v, summary=x.summary)
    sel = da.paged_select(x.q, x.summary, x.table, lens, P, TOP)
    return (lens, slots, sel, *da.paged_attn_fwd(x.q, x.k, x.v, x.table, lens, selected=sel),
            *da.paged_attn_fwd(x.q, x.k, x.v, x.table, lens))


@pytest.mark.parametrize("many", [False, True], ids=["few items", "many items"])
@pytest.mark.parametrize("call", [plan, plan_in_place, write, write_summary, select, attn, attn_selected, step],
                         ids=lambda f: f.__name__)
def test_inputs_written_late(late_copy, call, many):
    """`many`: the launches for many items (a table with room for more pages, a capped grid)."""
    da.set_grid_limit(1000 if many else 0)
    try:
        x = Inputs(2100 if many else 24)
        graph, res = torch.cuda.CUDAGraph(), None
        fresh = Inputs(2100 if many else 24).fill(0)
        call(x.fill(1))
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            late_copy(fresh.raw, x.raw)
            res = call(x)
        for i in range(8):
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
    finally:
        da.set_grid_limit(0)


def test_step_captured_behind_a_projection():
    """A step whose rows come straight out of a matrix product, captured and replayed with other inputs."""
    x = Inputs(24).fill(3)
    wide = torch.randn(512, (Hq + 2 * Hkv) * D, device=DEV).to(torch.bfloat16)
    rows = torch.randn(T, 512, device=DEV).to(torch.bfloat16)
    keep = x.raw.clone()

    def calls(qkv):
        lens, _, _, slots = da.paged_plan(x.new, x.lens, x.table, x.free, x.n_free[:1], P, N_PAGES, T)
        da.paged_kv_write(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], slots, x.k, x.v, summary=x.summary)
        q = qkv[:B, :Hq]
        sel = da.paged_select(q, x.summary, x.table, lens, P, TOP)
        return (lens, slots, sel, *da.paged_attn_fwd(q, x.k, x.v, x.table, lens, selected=sel))

    calls((rows @ wide).view(T, Hq + 2 * Hkv, D))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qkv = (rows @ wide).view(T, Hq + 2 * Hkv, D)
        got = calls(qkv)
    for i in range(8):
        rows.copy_(torch.randn(T, 512, device=DEV))
        x.raw.copy_(keep)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        product = (rows.double() @ wide.double()).view_as(qkv)  # bf16 out: half a step, and the fp32 sum's error
        assert (qkv - product).abs().max() <= 2.0 ** -8 * product.abs().max() * 1.01
        x.raw.copy_(keep)
        torch.cuda.synchronize()
        for a, b in zip(got, calls(qkv.clone())):
            assert torch.equal(a, b)
