"""Edges of the gradient norm and clipping: infinite limits, and lists of the
sizes that training has, against 64 bits on the GPU."""
import numpy as np
import pytest

from tests.test_gpu_grad import _clip

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", [False, True])
def test_infinite_limit(out):
    """A limit of infinity asks for the norm alone; an infinite norm has
    coefficient 0 beside it too."""
    import torch

    g = torch.full((3000,), 2.0, device="cuda")
    to = [torch.full_like(g, 7.0)] if out else None
    _, stats = _clip([g], to, float("inf"))
    assert stats[0] == np.float32(12000 ** 0.5) and stats[1] == 1.0
    assert (to[0] if out else g).eq(2.0).all()
    g[17] = float("inf")
    _, stats = _clip([g], to, float("inf"))
    assert np.isinf(stats[0]) and stats[1] == 0.0
    got = to[0] if out else g
    assert torch.isnan(got[17]) and int((got == 0).sum()) == 2999
    g = torch.full((30,), float("nan"), device="cuda")
    _, stats = _clip([g], None, float("inf"))
    assert np.isnan(stats).all()
