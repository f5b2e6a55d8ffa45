"""Argument checks of the operators for prompts at the edges of what their documentation allows, without a GPU."""
import pytest
import torch

from test_prompt_abi import A, INVALID, UNSUPPORTED, evict, lib, mass, prefill  # noqa: F401 (lib: a fixture)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up device addresses: run where there is no GPU")


@pytest.mark.parametrize("B", [1, 2, 8192])
def test_evict_takes_tables_in_one_allocation(lib, B):  # noqa: F811
    """Rows of the old and the new table in turn: [B, 2, max_pages], or columns of a wider buffer."""
    rows = lambda at, stride: {at + r * stride + i for r in range(B) for i in range(10)}  # noqa: E731
    for at, stride, out_stride in ((10, 20, 20), (14, 24, 24), (-10, 20, 20), (9, 20, 20), (11, 20, 20), (-9, 24, 24),
                                   (20, 20, 20), (5, 10, 10), (10, 40, 20), (5, 40, 20), (20, 20, 40)):
        got = evict(lib, B=B, stride=stride, out=A[1] + 4 * at, out_stride=out_stride)
        assert got != UNSUPPORTED and (got == INVALID) == bool(rows(0, stride) & rows(at, out_stride)), (at, stride)


@pytest.mark.parametrize("Hkv", [1, 2, 8])
def test_group_limits(lib, Hkv):  # noqa: F811
    """Page weights of at most 256 heads a group, attention of at most 128."""
    for cu in (A[5], None):
        at = dict(Hkv=Hkv, cu=cu, **(dict(T=3, start=None) if cu is None else {}))
        assert mass(lib, Hq=257 * Hkv, **at) == UNSUPPORTED
        assert mass(lib, Hq=256 * Hkv, **at) not in (INVALID, UNSUPPORTED)
    assert prefill(lib, Hq=129 * Hkv, Hkv=Hkv) == UNSUPPORTED
    assert prefill(lib, Hq=128 * Hkv, Hkv=Hkv) not in (INVALID, UNSUPPORTED)
