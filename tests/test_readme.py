"""The README's Python, run: every call of the library binds to its parameters, and what rope_freqs returns reaches the
rotation whole."""
import inspect
import os
import re
from types import SimpleNamespace
from unittest.mock import MagicMock

import numpy as np
import pytest
import torch

from diffusion_transformer_long_gb300 import ditattn as da

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
BLOCKS = re.findall(r"```python\n(.*?)```", open(README, encoding="utf-8").read(), re.S)
ROPE = [b for b in BLOCKS if "qk_norm_rope" in b]
STEP = [b for b in ROPE if "paged_plan" in b]


class Names(dict):
    """What a block takes as given."""

    def __missing__(self, name):
        if name in ("int", "len", "range", "print"):
            raise KeyError(name)
        self[name] = MagicMock(name=name)
        return self[name]


def yarn(real, device):
    """rope_freqs for a context that is stretched, whose scale is not 1."""
    return lambda rot, **kw: real(rot, **{"scaling": "yarn", "factor": 8, "device": device, **kw})


@pytest.mark.parametrize("block", ROPE, ids=lambda b: re.findall(r"da\.(\w+)", b)[-1])
def test_calls_bind_and_the_rotation_is_whole(block):
    tables, turned = [], 0

    def fake(name):
        real = getattr(da, name)
        results = dict(paged_plan=4, qk_norm_rope=2, paged_prefill_fwd=2, paged_attn_fwd=2, paged_evict=2, attn_fwd=2,
                       chunk_attention=2, attention=2).get(name, 1)

        def call(*args, **kw):
            nonlocal turned
            bound = inspect.signature(real).bind(*args, **kw)
            if name == "rope_freqs":
                tables.append(yarn(real, "cpu")(*args, **kw))
                return tables[-1]
            if name == "qk_norm_rope":
                bound.apply_defaults()
                freqs, pairs, scale = tables[-1]
                assert bound.arguments["freqs"] is freqs
                assert bound.arguments["rot_scale"] == scale
                assert (bound.arguments["axis_pairs"] or [len(freqs)]) == pairs
                turned += 1
            return tuple(MagicMock() for _ in range(results)) if results > 1 else MagicMock()
        return call

    names = Names(da=SimpleNamespace(**{x: fake(x) for x in set(re.findall(r"da\.(\w+)", block))}))
    exec(compile(block, README, "exec"), names)
    assert turned == len(re.findall("qk_norm_rope", block)) > 0


@pytest.mark.gpu
def test_the_step_runs():
    """The step of requests as it stands, with frequencies of a stretched context: its queries are turned and scaled, and
    the attention is over the keys that were."""
    import prompt_oracle as po
    dev, i32, bf16 = torch.device("cuda:0"), torch.int32, torch.bfloat16
    B, Hq, Hkv, D, n_pages = 2, 6, 2, 128, 80
    new = [70, 300]
    T = sum(new)
    gen = torch.Generator(dev).manual_seed(3)
    normal = lambda *shape: torch.randn(*shape, device=dev, generator=gen).to(bf16)  # noqa: E731
    q, k = normal(T, Hq, D), normal(T, Hkv, D)
    qw, kw = (1 + 0.2 * normal(D).float() for _ in range(2))
    names = dict(
        da=SimpleNamespace(**{x: getattr(da, x) for x in dir(da)}), q=q, k=k, v=normal(T, Hkv, D), qw=qw, kw=kw, T=T, n_pages=n_pages,
        q1=normal(B, Hq, D), new_lens=torch.tensor(new, dtype=i32, device=dev), seq_lens=torch.zeros(B, dtype=i32, device=dev),
        positions=torch.tensor([7, 5000], dtype=i32, device=dev), block_table=torch.full((B, 70), -1, dtype=i32, device=dev),
        free_pages=torch.arange(n_pages, dtype=i32, device=dev), n_free=torch.tensor([n_pages], dtype=i32, device=dev),
        k_cache=torch.zeros(n_pages, Hkv, 64, D, dtype=bf16, device=dev), v_cache=torch.zeros(n_pages, Hkv, 64, D, dtype=bf16, device=dev),
        summary=torch.zeros(n_pages, Hkv, 2, D, dtype=bf16, device=dev), mass=torch.zeros(n_pages, Hkv, device=dev))
    names["da"].rope_freqs = yarn(da.rope_freqs, dev)
    exec(compile(STEP[0], README, "exec"), names)
    da.check(dev)
    freqs, pairs, scale = da.rope_freqs(D, scaling="yarn", factor=8, device=dev)
    at = torch.tensor(np.concatenate([start + np.arange(n) for start, n in zip((7, 5000), new)]))[None, None]
    for got, x, w in ((names["q"], q, qw), (names["k"], k, kw)):
        y, size = po.norm_rope(x.transpose(0, 1)[None], w, 1e-6, freqs, pairs, at, False, scale)
        y, size = y[0].transpose(0, 1), size[0].transpose(0, 1)
        # (as in test_qk_norm_rope_gpu)
        E = 2.0 ** -19 * size
        assert ((got.double().cpu() - y).abs() <= E + 2.0 ** -8 * (y.abs() + E)).all()
    # the weight that the last 32 tokens of each request gave, all heads: their rows' weights add up to 1
    assert abs(names["mass"].sum().item() - B * 32 * Hq) < 1e-3 * B * 32 * Hq
    assert names["out"].isfinite().all() and names["seq_lens"].tolist() == new
