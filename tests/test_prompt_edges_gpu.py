"""Calls of the operators for prompts at the edges of what their documentation allows, on the GPU."""
import numpy as np
import pytest
import torch

from diffusion_transformer_long_gb300 import ditattn as da
from test_paged_gpu import rand
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
