"""Argument checks of the entry points for prompts that need no GPU: every call here is refused with the documented
status before any CUDA call, and the binding refuses wrong tensors."""
import ctypes
import math

import pytest
import torch

from diffusion_transformer_long_gb300 import build as dbuild
from diffusion_transformer_long_gb300 import ditattn as da

INVALID, UNSUPPORTED = da.DIT_ERR_INVALID_ARG, da.DIT_ERR_UNSUPPORTED

# Made-up, well separated device addresses: refused calls never look at them, and no GPU is to.
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up device addresses: run where there is no GPU")
A = [i << 44 for i in range(1, 18)]


@pytest.fixture(scope="module")
def lib():
    dbuild.build()
    return da.lib()


def S(b, h, n):
    return da.Strides(b, h, n)


def rope(lib, pairs=(8, 8, 16), **kw):
    a = dict(q=A[0], qs=None, qo=A[1], qos=None, Hq=4, k=A[2], ks=None, ko=A[3], kos=None, Hk=2, norm=1, eps=1e-6, qw=A[4],
             kw=A[5], wdt=1, freqs=A[6], pairs=None, axes=None, inter=0, scale=1.0, pos=A[7], pos_b=0, pos_axis=50, cu=None,
             start=None, requests=0, B=2, N=50, D=128)
    a.update(kw)
    if a["axes"] is None:
        a["axes"] = len(pairs)
    a["pairs"] = (ctypes.c_int * max(1, len(pairs)))(*pairs) if pairs is not None else None
    return lib.dit_qk_norm_rope(*a.values(), None)


QKV = S(50 * 8 * 128, 128, 8 * 128)  # token-major rows of 8 heads


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(Hq=0), INVALID), (dict(D=96), UNSUPPORTED), (dict(Hk=0), INVALID),
    (dict(k=None), INVALID), (dict(k=None, Hk=0), INVALID), (dict(k=None, Hk=0, ko=None), INVALID), (dict(q=None), INVALID), (dict(qo=None), INVALID),
    (dict(q=A[0] + 8), INVALID), (dict(ko=A[3] + 2), INVALID), (dict(norm=2), INVALID), (dict(norm=0), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID), (dict(wdt=2), INVALID),
    (dict(qw=A[4] + 1), INVALID), (dict(wdt=0, kw=A[5] + 2), INVALID), (dict(freqs=None), INVALID), (dict(pairs=()), INVALID),
    (dict(pairs=(8, -8, 16)), INVALID), (dict(pairs=(32, 40)), INVALID), (dict(pairs=(9, 8)), UNSUPPORTED),
    (dict(pairs=(8, 8, 8, 8, 8)), UNSUPPORTED), (dict(pairs=(0, 0)), INVALID), (dict(axes=-1), INVALID), (dict(freqs=A[6] + 2), INVALID),
    (dict(inter=3), INVALID), (dict(scale=math.nan), INVALID), (dict(pos=None), INVALID), (dict(pos=A[7] + 2), INVALID),
    (dict(pos_b=-1), INVALID), (dict(pos_axis=1 << 60), INVALID), (dict(cu=A[8], start=A[9]), INVALID),
    (dict(pos=None, cu=A[8], start=A[9], requests=3), INVALID),                       # packed: one batch, one axis
    (dict(pos=None, cu=A[8], start=A[9], requests=3, B=1), INVALID),
    (dict(pos=None, cu=A[8], start=A[9], requests=0, B=1, pairs=(16,)), INVALID),
    (dict(pos=None, cu=A[8], start=None, requests=3, B=1, pairs=(16,)), INVALID),
    (dict(norm=0, qw=None, kw=None, freqs=None, pairs=(), pos=None), INVALID),         # nothing to do
    (dict(freqs=None, pairs=()), INVALID),                                            # positions without a rotation
    (dict(N=1 << 30), INVALID), (dict(qs=S(51200, 12800, 60)), INVALID), (dict(qos=S(25600, 12800, 64)), INVALID),
    (dict(qo=A[0] + 256), INVALID), (dict(qo=A[2]), INVALID), (dict(ko=A[1]), INVALID), (dict(ko=A[6] - 512), INVALID), (dict(qo=A[7] - 1024), INVALID),
    # in place: not with other strides; slices of one projection: not when they share heads
    (dict(qo=A[0], qos=QKV), INVALID),
    (dict(qs=QKV, qos=QKV, qo=A[0], ks=QKV, kos=QKV, k=A[0] + 768, ko=A[0] + 768), INVALID),
    (dict(qs=QKV, qos=QKV, qo=A[0], ks=QKV, kos=QKV, k=A[0] + 7 * 256, ko=A[0] + 7 * 256), INVALID)])
def test_rope_validation(lib, kw, status):
    assert rope(lib, **kw) == status


def test_rope_accepts_slices_in_place(lib):
    at = dict(qs=QKV, qos=QKV, qo=A[0], ks=QKV, kos=QKV, k=A[0] + 4 * 256, ko=A[0] + 4 * 256)
    assert rope(lib, **at) not in (INVALID, UNSUPPORTED)  # (no GPU here: the launch fails)
    assert rope(lib, k=None, Hk=0, ko=None, kw=None) not in (INVALID, UNSUPPORTED)


NEED = 1 << 30


def prefill(lib, **kw):
    a = dict(q=A[0], qs=None, k=A[1], ks=None, v=A[2], vs=None, table=A[3], stride=100, lens=A[4], cu=A[5], start=A[6],
             out=A[7], lse=A[8], T=7, B=3, Hq=8, Hkv=2, D=128, P=16, n_pages=9, max_pages=100, causal=1, scale=0.088, dt=0,
             ws=A[9], ws_bytes=NEED)
    a.update(kw)
    return lib.dit_paged_prefill_fwd(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), INVALID), (dict(T=(1 << 30) + 1), INVALID), (dict(B=0), INVALID), (dict(B=2 ** 31 - 1), INVALID),
    (dict(Hkv=0), INVALID), (dict(Hq=9), INVALID), (dict(Hq=1), INVALID), (dict(D=80), UNSUPPORTED), (dict(P=20), UNSUPPORTED),
    (dict(Hq=258), UNSUPPORTED), (dict(P=2048), UNSUPPORTED), (dict(n_pages=0), INVALID), (dict(max_pages=0), INVALID), (dict(stride=99), INVALID),
    (dict(max_pages=1 << 27, stride=1 << 27), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(cu=None), INVALID), (dict(out=None), INVALID),
    (dict(ws=None), INVALID), (dict(ws_bytes=64), INVALID), (dict(ws=A[9] + 128), INVALID), (dict(out=A[7] + 8), INVALID),
    (dict(lse=A[8] + 2), INVALID), (dict(cu=A[5] + 2), INVALID), (dict(start=A[6] + 1), INVALID), (dict(causal=2), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=2.4e38), INVALID), (dict(dt=3), INVALID),
    (dict(qs=S(0, 100, 1024)), INVALID), (dict(qs=S(0, 128, 1 << 39)), INVALID), (dict(qs=S(0, 1 << 38, 128)), INVALID),
    (dict(ks=S(0, 2048, 128)), INVALID), (dict(out=A[0] + 1024), INVALID), (dict(lse=A[4]), INVALID), (dict(out=A[5] - 64), INVALID),
    (dict(ws=A[2] + 256), INVALID), (dict(out=A[9] + 4096), INVALID), (dict(lse=A[7] + 64), INVALID), (dict(lse=A[6]), INVALID),
    (dict(T=1 << 20, Hq=1 << 14, Hkv=1 << 13), INVALID)])
def test_prefill_validation(lib, kw, status):
    assert prefill(lib, **kw) == status


def test_prefill_workspace(lib):
    need = lib.dit_paged_prefill_workspace_bytes
    assert need(128, 16, 64) == 0 and need(128, 16, 65) > 0 and need(128, 0, 5) == 0 and need(0, 16, 500) == 0
    assert prefill(lib, max_pages=64, stride=64, ws=None, ws_bytes=0) not in (INVALID, UNSUPPORTED)


def mass(lib, **kw):
    a = dict(q=A[0], qs=None, lse=A[1], k=A[2], ks=None, table=A[3], stride=10, lens=A[4], cu=A[5], start=A[6], mass=A[7],
             out=A[8], T=7, B=3, Hq=8, Hkv=2, D=128, P=16, n_pages=9, max_pages=10, window=0, scale=0.088)
    a.update(kw)
    return lib.dit_paged_page_mass(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), INVALID), (dict(B=0), INVALID), (dict(window=-1), INVALID), (dict(cu=None), INVALID),
    (dict(cu=None, T=3), INVALID), (dict(Hq=9), INVALID), (dict(D=32), UNSUPPORTED), (dict(P=8), UNSUPPORTED), (dict(n_pages=0), INVALID),
    (dict(stride=9), INVALID), (dict(q=None), INVALID), (dict(lse=None), INVALID), (dict(k=None), INVALID), (dict(table=None), INVALID),
    (dict(lens=None), INVALID), (dict(mass=None), INVALID), (dict(out=None), INVALID), (dict(lse=A[1] + 2), INVALID),
    (dict(mass=A[7] + 2), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=math.inf), INVALID), (dict(out=A[7] + 4), INVALID),
    (dict(out=A[1]), INVALID), (dict(out=A[2] + 64), INVALID), (dict(out=A[3]), INVALID), (dict(out=A[0]), INVALID)])
def test_mass_validation(lib, kw, status):
    assert mass(lib, **kw) == status


def test_mass_in_place_is_accepted(lib):
    assert mass(lib, out=A[7]) not in (INVALID, UNSUPPORTED)
    assert mass(lib, cu=None, start=None, T=3) not in (INVALID, UNSUPPORTED)


def evict(lib, **kw):
    a = dict(mass=A[0], table=A[1], stride=10, out=A[2], out_stride=12, lens=A[3], lens_out=A[4], free=A[5], n_free=A[6],
             n_free_out=A[7], B=4, Hkv=2, P=16, n_pages=50, max_pages=10, cap=20, keep=5, recent=2, ws=A[8], ws_bytes=1 << 20)
    a.update(kw)
    return lib.dit_paged_evict(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), INVALID), (dict(B=8193), UNSUPPORTED), (dict(Hkv=0), INVALID), (dict(cap=-1), INVALID), (dict(keep=0), INVALID),
    (dict(recent=0), INVALID), (dict(recent=6), INVALID), (dict(P=24), UNSUPPORTED), (dict(n_pages=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(stride=9), INVALID), (dict(out_stride=9), INVALID), (dict(mass=None), INVALID), (dict(table=None), INVALID),
    (dict(out=None), INVALID), (dict(lens=None), INVALID), (dict(lens_out=None), INVALID), (dict(free=None), INVALID),
    (dict(n_free=None), INVALID), (dict(n_free_out=None), INVALID), (dict(ws=None), INVALID), (dict(ws=A[8] + 64), INVALID),
    (dict(ws_bytes=32), INVALID), (dict(mass=A[0] + 2), INVALID), (dict(free=A[5] + 1), INVALID),
    (dict(out=A[1]), INVALID),                                  # in place with another stride
    (dict(out=A[1] + 40, out_stride=10), INVALID), (dict(lens_out=A[3] + 4), INVALID), (dict(n_free_out=A[3]), INVALID),
    (dict(free=A[0] + 8), INVALID), (dict(n_free_out=A[5] + 76), INVALID), (dict(ws=A[5]), INVALID), (dict(lens_out=A[1] + 20), INVALID)])
def test_evict_validation(lib, kw, status):
    assert evict(lib, **kw) == status


def test_evict_in_place_is_accepted(lib):
    assert evict(lib, out=A[1], out_stride=10, lens_out=A[3], n_free_out=A[6]) not in (INVALID, UNSUPPORTED)
    assert lib.dit_paged_evict_workspace_bytes(0, 5) == 0 and lib.dit_paged_evict_workspace_bytes(3, 5) > 0


def test_frequencies():
    f, pairs, scale = da.rope_freqs(8, theta=100.0, device="cpu")
    assert pairs == [4] and scale == 1.0 and f.dtype == torch.float32
    assert torch.allclose(f, torch.tensor([1.0, 100 ** -0.25, 0.1, 100 ** -0.75]))
    lin = da.rope_freqs(8, theta=100.0, scaling="linear", factor=4, device="cpu")[0]
    assert torch.allclose(lin, f / 4)
    ntk = da.rope_freqs(8, theta=100.0, scaling="ntk", factor=4, device="cpu")[0]
    assert ntk[0] == 1 and torch.allclose(ntk[3], f[3] / 4)
    yarn, _, s = da.rope_freqs(64, scaling="yarn", factor=8, original_len=4096, device="cpu")
    plain = da.rope_freqs(64, device="cpu")[0]
    turns = 4096 * plain.double() / (2 * math.pi)
    assert torch.equal(yarn[turns > 32], plain[turns > 32]) and torch.allclose(yarn[turns < 1], plain[turns < 1] / 8)
    assert s == pytest.approx(0.1 * math.log(8) + 1)
    f3, pairs, _ = da.rope_freqs((44, 42, 42), device="cpu")
    assert pairs == [22, 21, 21] and len(f3) == 64 and f3[0] == f3[22] == f3[43] == 1
    for bad in (dict(rot=7), dict(rot=()), dict(rot=(4, 3)), dict(rot=8, scaling="x"), dict(rot=8, factor=0.5), dict(rot=8, theta=0.0)):
        with pytest.raises(ValueError):
            da.rope_freqs(**{"device": "cpu", **bad})


def test_binding_refuses_wrong_tensors():
    x, i = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    c = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        da.qk_norm_rope(x, eps=1e-6)
    with pytest.raises(ValueError):
        da.qk_norm_rope([1.0], eps=1e-6)
    with pytest.raises(ValueError):
        da.paged_prefill_fwd(x, c, c, i[None], i, i)
    with pytest.raises(ValueError):
        da.paged_page_mass(x, x, c, i[None], i, x)
    with pytest.raises(ValueError):
        da.paged_evict(torch.zeros(3, 2), i[None], i, i, i, 16, 2)


@pytest.mark.parametrize("B", [(1 << 20) + 1, (1 << 30) + 1, (1 << 31) - 2])
def test_request_limit(lib, B):
    """Request indexes stay in 32 bits in a warp's step past the last one, and sums over the requests in milliseconds."""
    assert prefill(lib, B=B) == INVALID and mass(lib, B=B) == INVALID
    assert rope(lib, pos=None, cu=A[8], start=A[9], requests=B, B=1, pairs=(16,)) == INVALID


@pytest.mark.parametrize("call", [prefill, mass])
def test_room_limit(lib, call):
    """Key indexes stay in 32 bits in a full row's last tile."""
    at = dict(B=1, T=1, cu=A[5], P=16)
    assert call(lib, max_pages=(1 << 26) + 1, **at) == UNSUPPORTED
    assert call(lib, max_pages=1 << 20, P=1024, **{k: v for k, v in at.items() if k != "P"}) not in (INVALID, UNSUPPORTED)
