"""dit_qk_norm_rope takes any views that share no element, however they interleave, and refuses those that do: checked
against the sets of elements themselves, without a GPU (an accepted call fails at its launch)."""
import ctypes
import random

import numpy as np
import pytest
import torch

from diffusion_transformer_long_gb300 import build as dbuild
from diffusion_transformer_long_gb300 import ditattn as da

INVALID, UNSUPPORTED = da.DIT_ERR_INVALID_ARG, da.DIT_ERR_UNSUPPORTED

# Made-up device addresses: no GPU is to look at them.
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up device addresses: run where there is no GPU")
A, FAR = 1 << 44, [i << 45 for i in range(1, 9)]
D = 64


@pytest.fixture(scope="module")
def lib():
    dbuild.build()
    return da.lib()


class V:
    """A [B, H, N, D] view `at` elements into the allocation."""

    def __init__(self, at, b, h, n, H):
        self.at, self.strides, self.H = at, (b, h, n), H

    def addr(self):
        return A + 2 * self.at

    def s(self):
        return da.Strides(*self.strides)

    def pieces(self, B, N):
        """Where its 8-element pieces lie (strides and offsets are multiples of 8)."""
        b, h, n = self.strides
        x = (np.arange(B)[:, None, None, None] * b + np.arange(self.H)[:, None, None] * h + np.arange(N)[:, None] * n
             + np.arange(0, D, 8))
        return (x.ravel() + self.at) // 8


def call(lib, q, k, qo, ko, B, N):
    """Accepted or not; None in place of an output: an allocation of its own."""
    out = [(None if v is None else v.s(), FAR[i] if v is None else v.addr()) for i, v in enumerate((qo, ko))]
    st = lib.dit_qk_norm_rope(q.addr(), q.s(), out[0][1], out[0][0], q.H, k.addr(), k.s(), out[1][1], out[1][0], k.H, 1, 1e-6,
                              None, None, 1, None, (ctypes.c_int * 1)(), 0, 0, 1.0, None, 0, 0, None, None, 0, B, N, D, None)
    assert st != UNSUPPORTED
    return st != INVALID


@pytest.mark.parametrize("B", [1, 2, 5])
def test_head_major_slices(lib, B):
    """Slices of one [B, heads, N, D] allocation: in place, and as outputs."""
    for Hq, Hk, heads, N in ((4, 4, 12, 50), (24, 8, 40, 7), (1, 1, 2, 3), (3, 5, 8, 1)):
        q, k = V(0, heads * N * D, N * D, D, Hq), V(Hq * N * D, heads * N * D, N * D, D, Hk)
        apart = V(1 << 40, D * 8, D, D, Hq), V(1 << 41, D * 8, D, D, Hk)
        assert call(lib, q, k, q, k, B, N) and call(lib, k, q, k, q, B, N)
        if B == 1:
            apart = V(1 << 40, Hq * N * D, N * D, D, Hq), V(1 << 41, Hk * N * D, N * D, D, Hk)
            assert call(lib, *apart, q, k, B, N)
        else:
            apart = V(1 << 38, Hq * N * D, N * D, D, Hq), V(1 << 39, Hk * N * D, N * D, D, Hk)
            assert call(lib, *apart, q, k, B, N)
        # one head too many, or half a head off
        if Hq > 1:
            k1 = V((Hq - 1) * N * D, heads * N * D, N * D, D, Hk)
            assert not call(lib, q, k1, q, k1, B, N) and not call(lib, *apart, q, k1, B, N)
        k2 = V(Hq * N * D - 8, heads * N * D, N * D, D, Hk)
        assert not call(lib, q, k2, q, k2, B, N)


@pytest.mark.parametrize("B", [1, 3])
def test_halves_of_the_tokens_and_mixed_layouts(lib, B):
    H, N = 4, 10
    whole = (H * 2 * N * D, 2 * N * D, D)  # [B, H, 2 N, D]: the first N tokens of each head, and the others
    assert call(lib, V(0, *whole, H), V(N * D, *whole, H), V(0, *whole, H), V(N * D, *whole, H), B, N)
    assert not call(lib, V(0, *whole, H), V((N - 1) * D, *whole, H), V(0, *whole, H), V((N - 1) * D, *whole, H), B, N)
    # a block for each batch, queries head-major, keys token-major behind them
    b = (H + 2) * N * D
    q, k = V(0, b, N * D, D, H), V(H * N * D, b, D, 2 * D, 2)
    assert call(lib, q, k, q, k, B, N)
    k = V(H * N * D - D, b, D, 2 * D, 2)
    assert not call(lib, q, k, q, k, B, N)
    # channels beside channels: rows of 2 D, a half each
    q, k = V(0, H * N * 2 * D, N * 2 * D, 2 * D, H), V(D, H * N * 2 * D, N * 2 * D, 2 * D, H)
    assert call(lib, q, k, q, k, B, N)


def test_views_at_random(lib):
    """Whether any two of them share an element, and none of the outputs itself, is what is accepted."""
    rng = random.Random(5)
    seen = [0, 0]
    for _ in range(4000):
        B, N, heads = rng.randint(1, 3), rng.randint(1, 4), rng.randint(2, 6)
        rows = N * rng.choice((1, 1, 2))
        wide = D * rng.choice((1, 1, 2))
        order = rng.choice(("bhn", "bnh", "hbn", "nbh"))
        extent, stride, at = dict(b=B, h=heads, n=rows), {}, wide
        for x in reversed(order):
            stride[x], at = at, at * extent[x]
        strides = stride["b"], stride["h"], stride["n"]

        def some(H):
            off = rng.choice((0, wide - D, (rows - N) * strides[2])) + rng.randint(0, heads - H) * strides[1]
            return V(off if rng.random() < 0.8 else max(0, off - 8), *strides, H)

        Hq, Hk = rng.randint(1, heads - 1), rng.randint(1, heads - 1)
        q, k = some(Hq), some(Hk)
        qo, ko = (q if rng.random() < 0.6 else some(Hq)), (k if rng.random() < 0.6 else some(Hk))
        p = [set(x.pieces(B, N).tolist()) for x in (q, k, qo, ko)]
        same = lambda a, b: a.at == b.at  # noqa: E731 (of one layout)
        good = not p[2] & p[3] and not p[2] & p[1] and not p[3] & p[0]
        good &= (same(q, qo) or not p[2] & p[0]) and (same(k, ko) or not p[3] & p[1])
        assert call(lib, q, k, qo, ko, B, N) == good, (B, N, strides, q.at, k.at, qo.at, ko.at, Hq, Hk)
        seen[good] += 1
    assert min(seen) > 400


def test_views_of_different_layouts_at_random(lib):
    """Queries and keys of unlike strides in one allocation, in place: accepted as long as they share nothing."""
    rng = random.Random(6)
    seen = [0, 0]
    for _ in range(4000):
        B, N = rng.randint(1, 3), rng.randint(1, 4)

        def some(block):
            H = rng.randint(1, 4)
            extent, stride, at = dict(b=B, h=H, n=N), {}, D
            for x in rng.choice(("bhn", "bnh", "hbn", "nbh"))[::-1]:
                stride[x] = at
                at = at * extent[x] + rng.choice((0, 0, D, 3 * D))
            if rng.random() < 0.5 and stride["b"] <= block:  # a block of its own for each batch
                stride["b"] = block
            return V(D * rng.randint(0, 40), stride["b"], stride["h"], stride["n"], H)

        block = D * rng.randint(8, 64)
        q, k = some(block), some(block)
        p = [x.pieces(B, N).tolist() for x in (q, k)]
        if any(len(set(x)) < len(x) for x in p):
            continue  # (an output that meets itself)
        good = not set(p[0]) & set(p[1])
        got = call(lib, q, k, q, k, B, N)
        assert not got or good, (B, N, q.at, q.strides, q.H, k.at, k.strides, k.H)
        if got != good:  # refused although apart: an output whose own dimensions do not nest
            assert any(not nested(v, B, N) for v in (q, k)), (B, N, q.at, q.strides, q.H, k.at, k.strides, k.H)
        seen[good] += 1
    assert min(seen) > 400


def nested(v, B, N):
    """Whether each dimension's stride clears what the shorter ones span, as outputs have to."""
    b, h, n = v.strides
    at = D
    for stride, extent in sorted(((b, B), (h, v.H), (n, N))):
        if extent > 1:
            if stride < at:
                return False
            at += stride * (extent - 1)
    return True


def test_views_that_take_long_to_tell_apart(lib):
    """Layouts that have nothing in common are told apart as far as that goes quickly, and refused else; never accepted
    where they meet."""
    H, N = 8, 4096
    q = V(0, 8 * N * D * 3, D, 3 * H * D, H)  # token-major in every third row
    for off, good in ((H * D, True), (0, False), (H * D - 8, False)):
        k = V(off, 8 * N * D * 3, D, 3 * H * D, H)
        assert call(lib, q, k, q, k, 2, N) == good
    k = V(8, 8 * N * D * 3, N * D, D, H)  # head-major across all of them
    assert not call(lib, q, k, q, k, 2, N)
