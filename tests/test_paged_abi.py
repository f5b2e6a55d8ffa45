"""Argument checks of the paged-cache entry points that need no GPU: every call here is refused with
the documented status before any CUDA call, and the binding refuses wrong tensors."""
import ctypes
import math

import pytest
import torch

from diffusion_transformer_long_gb300 import build as dbuild
from diffusion_transformer_long_gb300 import ditattn as da

INVALID, UNSUPPORTED = da.DIT_ERR_INVALID_ARG, da.DIT_ERR_UNSUPPORTED

# Fake, well separated device addresses: validation never dereferences them.
A = [i << 44 for i in range(1, 14)]


@pytest.fixture(scope="module")
def lib():
    dbuild.build()
    return da.lib()


def plan(lib, **kw):
    a = dict(new=A[0], old=A[1], table=A[2], stride=10, free=A[3], n_free=A[4], old_out=A[5], free_out=A[6],
             cu=A[7], slots=A[8], B=4, max_pages=10, P=16, n_pages=50, cap=20, tokens=64)
    a.update(kw)
    return lib.dit_paged_plan(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), INVALID), (dict(B=8193), UNSUPPORTED), (dict(tokens=0), INVALID),
    (dict(tokens=(1 << 30) + 1), INVALID), (dict(cap=-1), INVALID), (dict(P=0), INVALID),
    (dict(P=24), UNSUPPORTED), (dict(P=2048), UNSUPPORTED), (dict(n_pages=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(max_pages=1 << 28, stride=1 << 28), INVALID),
    (dict(stride=9), INVALID), (dict(stride=1 << 60), INVALID), (dict(new=None), INVALID),
    (dict(old=None), INVALID), (dict(table=None), INVALID), (dict(free=None), INVALID),
    (dict(n_free=None), INVALID), (dict(old_out=None), INVALID), (dict(free_out=None), INVALID),
    (dict(cu=None), INVALID), (dict(slots=None), INVALID), (dict(slots=A[8] + 4), INVALID),
    (dict(cu=A[7] + 2), INVALID), (dict(table=A[2] + 1), INVALID),
    (dict(old_out=A[1] + 4), INVALID),          # shifted, not in place
    (dict(free_out=A[3] + 8), INVALID),         # inside the stack
    (dict(cu=A[0]), INVALID), (dict(slots=A[2] + 64), INVALID), (dict(old_out=A[2] + 80), INVALID),
    (dict(free_out=A[7] + 16), INVALID), (dict(cu=A[1] + 12), INVALID)])
def test_plan_validation(lib, kw, status):
    assert plan(lib, **kw) == status


def S(b, h, n):
    return da.Strides(b, h, n)


def write(lib, **kw):
    a = dict(k=A[0], ks=None, v=A[1], vs=None, slots=A[2], kc=A[3], kcs=None, vc=A[4], vcs=None, summary=A[5],
             T=7, H=2, D=64, P=16, n_pages=9)
    a.update(kw)
    return lib.dit_paged_kv_write(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), INVALID), (dict(H=0), INVALID), (dict(D=96), UNSUPPORTED), (dict(P=8), UNSUPPORTED),
    (dict(n_pages=0), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(slots=None), INVALID),
    (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(k=A[0] + 2), INVALID), (dict(slots=A[2] + 4), INVALID),
    (dict(summary=A[5] + 8), INVALID), (dict(ks=S(64, 64, 132)), INVALID), (dict(ks=S(64, 0, 128)), INVALID),
    (dict(kcs=S(2048, 1024, 60)), INVALID),      # rows not 16-byte strided
    (dict(kcs=S(2048, 1024, 32)), INVALID),      # rows overlap
    (dict(kcs=S(1024, 1024, 64)), INVALID),      # pages overlap
    (dict(kcs=S(1 << 39, 1024, 64)), INVALID), (dict(vc=A[3] + 4096), INVALID), (dict(summary=A[4] + 64), INVALID),
    # interleaved caches: not by whole halves, by less than a head, of other strides, with the summary or the rows inside
    (dict(kcs=S(4096, 1024, 64), vc=A[3] + 2048, vcs=S(4096, 1024, 64)), INVALID),
    (dict(kcs=S(4096, 128, 256), vc=A[3] + 64, vcs=S(4096, 128, 256)), INVALID),
    (dict(kcs=S(4096, 1024, 64), vc=A[3] + 4096, vcs=S(4096, 64, 128)), INVALID),
    (dict(kcs=S(4096, 1024, 64), vc=A[3], vcs=S(4096, 1024, 64)), INVALID),
    (dict(kcs=S(6144, 1024, 64), vc=A[3] + 4096, vcs=S(6144, 1024, 64), summary=A[3] + 8192), INVALID),
    (dict(kcs=S(6144, 1024, 64), vc=A[3] + 4096, vcs=S(6144, 1024, 64), k=A[3] + 8192), INVALID),
    (dict(kc=A[0] + 512), INVALID), (dict(vc=A[2]), INVALID), (dict(H=1 << 20, n_pages=1 << 30), INVALID)])
def test_write_validation(lib, kw, status):
    assert write(lib, **kw) == status


@pytest.mark.parametrize("T", [(1 << 30) + 1, (1 << 31) - 1])
def test_write_token_count_validation(lib, T):
    """Past 2^30 tokens their indexes would pass 32 bits inside a launch."""
    few = dict(ks=S(64, 64, 8), vs=S(64, 64, 8), H=1, summary=None)  # rows that overlap: they fit a GPU's memory
    assert write(lib, T=T, **few) == INVALID
    assert write(lib, T=1 << 30, **few) != INVALID  # (no GPU here: the launch fails)


NEED = 1 << 30


def attn(lib, **kw):
    a = dict(q=A[0], qs=None, k=A[1], ks=None, v=A[2], vs=None, table=A[3], stride=10, lens=A[4], sel=None, n_sel=0,
             out=A[5], lse=A[6], B=3, Hq=8, Hkv=2, D=128, P=16, n_pages=9, max_pages=10, scale=0.088, dt=0,
             ws=A[7], ws_bytes=NEED)
    a.update(kw)
    return lib.dit_paged_attn_fwd(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=9), INVALID), (dict(Hq=1), INVALID), (dict(D=80), UNSUPPORTED),
    (dict(P=20), UNSUPPORTED), (dict(n_pages=0), INVALID), (dict(max_pages=0), INVALID), (dict(stride=9), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(table=None), INVALID),
    (dict(lens=None), INVALID), (dict(out=None), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=64), INVALID),
    (dict(ws=A[7] + 128), INVALID), (dict(out=A[5] + 8), INVALID), (dict(lse=A[6] + 2), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=math.nan), INVALID), (dict(dt=3), INVALID),
    (dict(sel=A[8], n_sel=0), INVALID), (dict(sel=A[8], n_sel=11), INVALID), (dict(sel=A[8] + 2, n_sel=2), INVALID),
    (dict(qs=S(1024, 100, 0)), INVALID), (dict(ks=S(1 << 38, 1 << 38, 128), B=1, Hq=1 << 23, Hkv=1 << 23), INVALID), (dict(ks=S(0, 2048, 128)), INVALID), (dict(out=A[0] + 1024), INVALID),
    (dict(lse=A[4]), INVALID), (dict(ws=A[2] + 256), INVALID), (dict(out=A[7] + 4096), INVALID),
    (dict(lse=A[5] + 64), INVALID), (dict(B=1 << 16, Hq=1 << 16), INVALID)])
def test_attn_validation(lib, kw, status):
    assert attn(lib, **kw) == status


def test_attn_scale_validation(lib):
    """Scores are held in base 2: a scale that is finite only without that factor would make them all infinite."""
    assert attn(lib, scale=2.4e38) == INVALID and attn(lib, scale=math.inf) == INVALID
    assert attn(lib, scale=2.3e38) != INVALID  # (no GPU here: the launch fails)


def select(lib, **kw):
    a = dict(q=A[0], qs=None, summary=A[1], table=A[2], stride=10, lens=A[3], sel=A[4], B=3, Hq=8, Hkv=2, D=128, P=16,
             n_pages=9, max_pages=10, top_k=4, ws=A[5], ws_bytes=NEED)
    a.update(kw)
    return lib.dit_paged_select(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), INVALID), (dict(Hkv=3), INVALID), (dict(D=32), UNSUPPORTED), (dict(P=40), UNSUPPORTED),
    (dict(top_k=0), INVALID), (dict(top_k=11), INVALID), (dict(q=None), INVALID), (dict(summary=None), INVALID),
    (dict(summary=A[1] + 8), INVALID), (dict(table=None), INVALID), (dict(stride=3), INVALID), (dict(lens=None), INVALID),
    (dict(sel=None), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=16), INVALID), (dict(ws=A[5] + 16), INVALID),
    (dict(sel=A[5]), INVALID), (dict(sel=A[3]), INVALID), (dict(ws=A[1]), INVALID),
    (dict(Hkv=1 << 20, Hq=1 << 20, n_pages=1 << 30, B=1), INVALID)])
def test_select_validation(lib, kw, status):
    assert select(lib, **kw) == status


def test_workspace_sizes(lib):
    assert lib.dit_paged_attn_workspace_bytes(0, 8, 2, 128, 16, 9) == 0
    assert lib.dit_paged_attn_workspace_bytes(1, 8, 0, 128, 16, 9) == 0
    assert lib.dit_paged_attn_workspace_bytes(1, 8, 2, 128, 0, 9) == 0
    assert lib.dit_paged_attn_workspace_bytes(64, 8, 2, 128, 16, 900) > 0
    assert lib.dit_paged_select_workspace_bytes(1, 0, 5) == 0
    assert lib.dit_paged_select_workspace_bytes(64, 8, 1 << 20) >= 64 * 8 * (1 << 20)  # no 32-bit wrap


def test_binding_refuses_host_tensors():
    i, x = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    c, t = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        da.paged_plan(i, i, t, i, i[:1], 16, 3, 8)
    with pytest.raises(ValueError):
        da.paged_kv_write(x, x, torch.zeros(2, dtype=torch.int64), c, c)
    with pytest.raises(ValueError):
        da.paged_attn_fwd(x, c, c, t, i)
    with pytest.raises(ValueError):
        da.paged_select(x, torch.zeros(3, 2, 2, 64, dtype=torch.bfloat16), t, i, 16, 2)


@pytest.mark.gpu
def test_binding_refusals():
    """What the binding itself must stop: the C ABI sees pointers and sizes, not buffers."""
    dev = "cuda"
    i, t = torch.zeros(2, dtype=torch.int32, device=dev), torch.zeros(2, 4, dtype=torch.int32, device=dev)
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=dev)
    c = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16, device=dev)
    s = torch.zeros(3, 2, 2, 64, dtype=torch.bfloat16, device=dev)
    slots = torch.zeros(2, dtype=torch.int64, device=dev)
    ok = lambda **kw: da.paged_attn_fwd(**{**dict(q=x, k_cache=c, v_cache=c, block_table=t, seq_lens=i), **kw})  # noqa: E731
    ok()
    for kw, e in ((dict(q=x.float()), TypeError), (dict(q=x[0]), ValueError), (dict(q=x[..., ::2]), ValueError),
                  (dict(v_cache=c[:2]), ValueError), (dict(k_cache=c.float()), TypeError),
                  (dict(block_table=t.long()), TypeError), (dict(block_table=t[:1]), ValueError),
                  (dict(block_table=t.t().contiguous().t()), ValueError), (dict(seq_lens=i[:1]), ValueError),
                  (dict(seq_lens=i.cpu()), ValueError), (dict(selected=t), ValueError),
                  (dict(selected=torch.zeros(2, 2, 5, dtype=torch.int32, device=dev)), da.DitError),
                  (dict(out=torch.zeros(2, 4, 32, device=dev)), ValueError), (dict(lse=torch.zeros(2, 5, device=dev)), ValueError),
                  (dict(workspace=torch.zeros(64, dtype=torch.uint8, device=dev),
                        block_table=torch.zeros(2, 500, dtype=torch.int32, device=dev)), ValueError), (dict(scale=-1.0), da.DitError),
                  (dict(out_dtype=torch.float16), TypeError),
                  (dict(q=torch.zeros(2, 3, 64, dtype=torch.bfloat16, device=dev)), da.DitError)):
        with pytest.raises(e):
            ok(**kw)
    with pytest.raises(ValueError):
        da.paged_kv_write(x, x, slots, c, c.clone())              # 4 heads into 2
    y = x[:, :2]
    with pytest.raises(da.DitError):
        da.paged_kv_write(y, y, slots, c, c)                      # one buffer for keys and values
    with pytest.raises(TypeError):
        da.paged_kv_write(y, y, slots.int(), c, c.clone())
    with pytest.raises(ValueError):
        da.paged_kv_write(y, y, slots, c, c.clone(), summary=s[:2])
    with pytest.raises(da.DitError):
        da.paged_select(x, s, t, i, 16, 5)
    with pytest.raises(da.DitError):
        da.paged_select(x, s, t, i, 20, 2)
    with pytest.raises(TypeError):
        da.paged_plan(i.long(), i, t, i, i[:1], 16, 3, 8)
    with pytest.raises(ValueError):
        da.paged_plan(i, i, t, i, i, 16, 3, 8)
    with pytest.raises(da.DitError):
        da.paged_plan(i, i, t, i, i[:1], 16, 3, 0)
