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


@pytest.mark.parametrize("swap", ["data", "set_"])
def test_list_keeps_its_memory(swap):
    """A list means the memory that its tensors had: a tensor that is given
    other memory does not free it for others."""
    import torch

    import orthogonal_fine_tuning_amd as oft

    n = 5 << 20  # (large tensors have blocks of their own, which the next of that size would get)
    grads, out = [torch.ones(n, device="cuda")], [torch.zeros(n, device="cuda")]
    lst = oft.grad_list(grads, out)
    nb = oft.oft_grad_workspace_bytes(lst)
    ws, sumsq = torch.empty(nb, dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.float64, device="cuda")
    stats = torch.zeros(2, device="cuda")
    was = [grads[0].data_ptr(), out[0].data_ptr()]
    for t in (grads[0], out[0]):
        other = torch.full((8,), 3.0, device="cuda")
        if swap == "data":
            t.data = other
        else:
            t.set_(other)
    others = [torch.full((n,), 5.0, device="cuda") for _ in range(4)]
    assert not {t.data_ptr() for t in others} & set(was)
    oft.oft_grad_sumsq(lst, sumsq, ws=ws, ws_bytes=nb)
    oft.oft_grad_clip(lst, sumsq, 1.0, stats)
    assert float(sumsq) == n and all(bool((t == 5).all()) for t in others)
