"""GPU parity of dit_qk_norm_rope against its plain 64-bit form (prompt_oracle).

Tolerance: y is computed in 32 bits (a cosine and sine off by 2^-22 with their angle's rounding, the norm's factor by
2^-21 with the sum of D squares, six more roundings) from values of size |z_first| + |z_second|: off by at most 2^-19 of
that, and by half a step of bf16, 2^-8 of the value."""
import math

import numpy as np
import pytest
import torch

import prompt_oracle as po
from diffusion_transformer_long_gb300 import ditattn as da
from test_paged_gpu import rand

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(DEV, dtype)


def weight(D, seed, dtype=torch.bfloat16):
    return (1 + rand(D, seed=seed, scale=0.3).float()).to(dtype)


def close(got, x, w, eps, freqs, pairs, positions, inter, scale):
    y, size = po.norm_rope(x, w, eps, freqs, pairs, positions, inter, scale)
    E = 2.0 ** -19 * size
    got = got.double().cpu()
    bad = ~((got - y).abs() <= E + 2.0 ** -8 * (y.abs() + E))
    assert not bad.any(), f"{bad.sum()} of {bad.numel()} off, first at {torch.nonzero(bad)[0].tolist()}"


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 16), (64, 64), (64, 48), (128, 128), (128, 16), (128, 112), (128, 64)])
@pytest.mark.parametrize("B,Hq,Hk,N", [(1, 1, 1, 1), (2, 3, 1, 5), (1, 24, 8, 64), (1, 40, 40, 33), (3, 5, 0, 700), (1, 2, 2, 2050)])
def test_layouts_and_sizes(B, Hq, Hk, N, D, rot, inter):
    rng = np.random.default_rng(rot + N)
    x = rand(B, N, Hq + 2 * Hk + 1, D, seed=N, scale=3).transpose(1, 2)  # token-major, as projected
    q, k = x[:, :Hq], x[:, Hq:Hq + Hk] if Hk else None
    freqs, pairs, scale = da.rope_freqs(rot, scaling="yarn", factor=4)
    qw, kw = weight(D, 1), weight(D, 2) if Hk else None
    pos = dev(rng.integers(-1000, 1 << 20, (1, B, N)))
    yq, yk = da.qk_norm_rope(q, k, pos, freqs, pairs, inter, scale, 1e-6, qw, kw)
    assert yq.is_contiguous() and yq.shape == q.shape and (yk is None) == (not Hk)
    close(yq, q, qw, 1e-6, freqs, pairs, pos, inter, scale)
    if Hk:
        close(yk, k, kw, 1e-6, freqs, pairs, pos, inter, scale)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dims", [(44, 42, 42), (16, 56, 56), (32, 32, 32, 32), (0, 16, 48), (128,)])
def test_position_axes(dims, inter):
    B, H, N, D = 2, 4, 37, 128
    x, k = rand(B, H, N, D, seed=5), rand(B, 2, N, D, seed=6)
    fs = [da.rope_freqs(d)[0] for d in dims if d]
    freqs, pairs = torch.cat(fs), [d // 2 for d in dims]
    pos = dev(np.random.default_rng(1).integers(0, 200, (len(dims), B, N)))
    for shared in (False, True):
        p = pos[:, 0].contiguous() if shared else pos
        y, yk = da.qk_norm_rope(x, k, p, freqs, pairs, inter, 1.0)
        want = pos[:, :1].expand(-1, B, -1) if shared else pos
        close(y, x, None, None, freqs, pairs, want, inter, 1.0)
        close(yk, k, None, None, freqs, pairs, want, inter, 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_parts_alone(dtype):
    """Norms without a rotation (weights of either type, or none), a rotation without norms, one position for all."""
    q, k = rand(9, 6, 64, seed=1), rand(9, 2, 64, seed=2)
    w = weight(64, 3, dtype)
    y, yk = da.qk_norm_rope(q, k, eps=1e-5, q_weight=w)
    view = lambda t: t.transpose(0, 1)[None]  # noqa: E731
    close(view(y), view(q), w, 1e-5, None, None, None, False, 1)
    close(view(yk), view(k), None, 1e-5, None, None, None, False, 1)
    freqs, pairs, _ = da.rope_freqs(32)
    pos = dev(np.full(9, 12345))
    y, none = da.qk_norm_rope(q, positions=pos, freqs=freqs)
    assert none is None
    close(view(y), view(q), None, None, freqs, pairs, pos[None, None], False, 1)


@pytest.mark.parametrize("inter", [False, True])
def test_packed_requests_in_place(inter):
    """Positions from the requests' first ones; the slices of one projection in place; rows of no request, and what
    lies beside the slices, are left as they are."""
    rng = np.random.default_rng(0)
    for R, hi in ((1, 40), (7, 5), (40, 3), (1500, 3), (5000, 1)):
        new = rng.integers(0, hi + 1, R)
        lead, spare = 3, 5
        cu = lead + np.concatenate(([0], np.cumsum(new)))
        T = int(cu[-1]) + spare
        start = rng.integers(-5, 1 << 22, R)
        pos = np.zeros(T, np.int64)
        for r in range(R):
            pos[cu[r]:cu[r + 1]] = start[r] + np.arange(new[r])
        x = rand(T, 9, 128, seed=R)
        before = x.clone()
        freqs, pairs, _ = da.rope_freqs(64, scaling="ntk", factor=8)
        qw, kw = weight(128, 1), weight(128, 2)
        q, k = x[:, 1:6], x[:, 6:8]
        da.qk_norm_rope(q, k, freqs=freqs, interleaved=inter, eps=1e-6, q_weight=qw, k_weight=kw, cu_new=dev(cu),
                        start_lens=dev(start), q_out=q, k_out=k)
        own = torch.zeros(T, dtype=torch.bool)
        own[lead:int(cu[-1])] = True
        assert torch.equal(x[~own.to(DEV)], before[~own.to(DEV)]) and torch.equal(x[:, [0, 8]], before[:, [0, 8]])
        at = dev(pos[None, None, own.numpy()])
        for new_x, old, w in ((q, before[:, 1:6], qw), (k, before[:, 6:8], kw)):
            close(new_x[own.to(DEV)].transpose(0, 1)[None], old[own.to(DEV)].transpose(0, 1)[None], w, 1e-6, freqs, pairs, at,
                  inter, 1)


def test_far_positions_are_exact():
    """Angles to the last position of 32 bits: against whole-number arithmetic."""
    from fractions import Fraction
    pi = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)
    pos = [0, 1, -1, 2 ** 24 + 1, 75600, 2 ** 31 - 1, -2 ** 31, 123456789, -987654321]
    freqs, pairs, _ = da.rope_freqs(64, theta=500000.0)
    x = rand(len(pos), 1, 64, seed=3)
    y, _ = da.qk_norm_rope(x, positions=dev(pos), freqs=freqs)
    y, x = y.double().cpu(), x.double().cpu()
    for a, p in enumerate(pos):
        for i, f in enumerate(freqs.tolist()):
            t = Fraction(f) * p / (2 * pi)
            angle = float((t - round(t)) * 2 * pi)
            c, s = math.cos(angle), math.sin(angle)
            u, v = float(x[a, 0, i]), float(x[a, 0, i + 32])
            for got, want in ((y[a, 0, i], u * c - v * s), (y[a, 0, i + 32], u * s + v * c)):
                assert abs(float(got) - want) <= 2.0 ** -8 * abs(want) + 2.0 ** -19 * (abs(u) + abs(v)), (p, i)


def test_unusual_frequencies_and_values():
    x = rand(4, 2, 64, seed=3)
    for f in (0.0, -0.7, 1e-30, 1e-42, 3.5, 70000.0, 2.0 ** 60):
        freqs = torch.full((16,), f, device=DEV)
        y, _ = da.qk_norm_rope(x, positions=dev([0, 1, 7, -12]), freqs=freqs)
        if abs(f) < 100:
            close(y.transpose(0, 1)[None], x.transpose(0, 1)[None], None, None, freqs, [16], dev([[[0, 1, 7, -12]]]), False, 1)
        assert y.isfinite().all()
    for f in (math.nan, math.inf):
        y, _ = da.qk_norm_rope(x, positions=dev([0, 1, 7, -12]), freqs=torch.full((16,), f, device=DEV))
        assert y[..., :32].isnan().all() and torch.equal(y[..., 32:], x[..., 32:])
    # a value that is not finite stays in its pair without norms, and in its head with them
    for inter in (False, True):
        z = x.clone()
        z[1, 0, 3], z[2, 1, 40], z[3, 0, 63] = math.nan, math.inf, math.nan
        freqs = da.rope_freqs(32)[0]
        y, _ = da.qk_norm_rope(z, positions=dev([0, 1, 7, -12]), freqs=freqs, interleaved=inter)
        want, _ = da.qk_norm_rope(x, positions=dev([0, 1, 7, -12]), freqs=freqs, interleaved=inter)
        hit = torch.zeros_like(x, dtype=torch.bool)
        hit[1, 0, [3, 2] if inter else [3, 19]] = True
        hit[2, 1, 40] = hit[3, 0, 63] = True
        assert not y[hit].isfinite().any() and torch.equal(y[~hit], want[~hit])
        y, _ = da.qk_norm_rope(z, eps=1e-6)
        want, _ = da.qk_norm_rope(x, eps=1e-6)
        clean = z.isfinite().all(2)
        assert torch.equal(y[clean], want[clean]) and not y[~clean].isfinite().all(1).any()
    zero, _ = da.qk_norm_rope(torch.zeros_like(x), eps=1e-6)
    assert (zero == 0).all()


def test_streams_graphs_and_views():
    """Another stream; a captured step replayed with other positions; outputs of other strides."""
    q, k = rand(2, 4, 300, 128, seed=1), rand(2, 2, 300, 128, seed=2)
    freqs, pairs, _ = da.rope_freqs(128)
    pos = dev(np.arange(300))
    want = da.qk_norm_rope(q, k, pos, freqs, eps=1e-6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = da.qk_norm_rope(q, k, pos, freqs, eps=1e-6, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    big = torch.full((2, 300, 7, 256), 5.0, device=DEV, dtype=torch.bfloat16)
    qo, ko = big[:, :, 1:5, 128:].transpose(1, 2), big[:, :, 5:7, :128].transpose(1, 2)
    g = torch.cuda.CUDAGraph()
    da.qk_norm_rope(q, k, pos, freqs, eps=1e-6, q_out=qo, k_out=ko)
    with torch.cuda.graph(g):
        da.qk_norm_rope(q, k, pos, freqs, eps=1e-6, q_out=qo, k_out=ko)
    for shift in (0, 1000):
        pos.copy_(dev(np.arange(300) + shift))
        want = da.qk_norm_rope(q, k, pos, freqs, eps=1e-6)
        g.replay()
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    assert (big[:, :, 0] == 5).all() and (big[:, :, 1:5, :128] == 5).all() and (big[:, :, 5:, 128:] == 5).all()


def test_attention_sees_only_distances():
    """Queries and keys turned by their positions score by their distance: the same prompt further along gives the
    same outputs, up to the roundings of its queries and keys."""
    q, k, v = (rand(1, 2, 300, 128, seed=i) for i in (1, 2, 3))
    freqs = da.rope_freqs(128)[0]
    outs = []
    for far in (0, 100000):
        a, b = da.qk_norm_rope(q, k, dev(np.arange(300) + far), freqs, eps=1e-6)
        outs.append(da.attn_fwd(a, b, v)[0])
    # scores are off by 2 x 2^-8 of q's and k's roundings, up to sqrt(128) in size: outputs by a few percent of |v|'s mean
    assert (outs[0] - outs[1]).abs().max() < 4 * 2.0 ** -8 * math.sqrt(128) * v.abs().max().item()
    assert (outs[0] - outs[1]).norm() < 0.05 * outs[0].norm()
