"""The layer for a few tokens with grouped routing over few large groups: the groups' scores and choice are the
same whatever their size."""
import ctypes

import pytest
import torch

from tests.test_layer_few import Layer
from tests.test_serve_abi import UNSUPPORTED, few, moe  # noqa: F401


def test_groups_of_one_expert_and_uneven_ones_are_refused(moe):  # noqa: F811
    for kw in (dict(E=8, n_group=8), dict(E=8, n_group=3), dict(E=64, n_group=33), dict(E=8, n_group=0)):
        assert few(moe, method=2, **kw) == UNSUPPORTED
    # moe_route keeps its own limit
    r = moe.MoeRouteParams(256, 8, 2, 4, 2, 1.0)
    assert moe._lib.moe_route(None, 4, None, ctypes.byref(r), None, None, None) == UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
@pytest.mark.parametrize("E,n_group,topk_group,k", [(256, 4, 2, 8), (256, 2, 1, 8), (132, 4, 3, 5), (256, 1, 1, 8), (70, 2, 2, 3)])
@pytest.mark.parametrize("T", [3, 16])
def test_large_groups(moe, T, E, n_group, topk_group, k):  # noqa: F811
    layer = Layer(moe, T, 96, 64, E, k, 2, "16", "bf16", n_group=n_group, topk_group=topk_group, rsf=2.5, seed=E)
    layer.check(layer())
    # keys that are equal: the lowest groups and experts
    layer.x.zero_()
    layer.bias.zero_()
    y, ids, sc = layer()
    assert ids.tolist() == [list(range(k))] * T and not y.any()
    assert torch.allclose(sc, torch.full_like(sc, 2.5 / k), rtol=2.0 ** -22)
