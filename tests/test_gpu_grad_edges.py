"""Edges of the gradient norm and clipping: infinite limits, and lists of the
sizes that training has, against 64 bits on the GPU."""
import numpy as np
import pytest

from tests.adapter_cases import HALF, U
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


LISTS = {  # elements of each tensor
    "few": [9000001, 17, 4099],           # 8192 elements a workgroup
    "many": [600011] * 15 + [3],
    "few_streamed": [20000003, 0, 5, 70001],  # past 64 MB as fp32; as bf16 twice as many
    "many_streamed": [1500007] * 14,
}


def _views(sizes, dtype, odd, seed):
    """Tensors cut from one buffer of ones, starting anywhere if odd."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.ones(sum(sizes) + 64 * len(sizes), dtype=dtype, device="cuda")
    out, at = [], 0
    for i, n in enumerate(sizes):
        at += 1 + i % 7 if odd else 0
        out.append(buf[at:at + n])
        out[-1].copy_(0.01 * torch.randn(n, generator=g, device="cuda"))
        at += n if odd else (n + 15) & ~15
    return buf, out


@pytest.mark.parametrize("max_norm", [0.5, 1e6])
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", LISTS)
def test_lists_of_training(name, dtype, odd, max_norm):
    import torch

    import orthogonal_fine_tuning_amd as oft

    kind = torch.float32 if dtype == "f32" else torch.bfloat16
    sizes = [2 * n if dtype == "bf16" and "streamed" in name else n for n in LISTS[name]]
    buf, grads = _views(sizes, kind, odd, 1)
    mark, outs = _views(sizes, kind, odd, 2)
    before = buf.clone()
    total = sum(float(t.double().square().sum()) for t in grads)
    norm = total ** 0.5
    coef = min(1.0, max_norm / (norm + 1e-6))

    def clip(lst):
        nb = oft.oft_grad_workspace_bytes(lst)
        ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
        sumsq, stats = torch.full((1,), float("nan"), dtype=torch.float64, device="cuda"), torch.zeros(2, device="cuda")
        oft.oft_grad_sumsq(lst, sumsq, ws=ws, ws_bytes=nb)
        oft.oft_grad_clip(lst, sumsq, max_norm, stats)
        return float(sumsq), stats.double().cpu().numpy()

    sumsq, stats = clip(oft.grad_list(grads, outs))
    assert abs(sumsq - total) <= 1e-9 * total
    assert abs(stats[0] - norm) <= 2 * U * norm and abs(stats[1] - coef) <= 8 * U * coef
    for g, o in zip(grads, outs):
        want = g.double() * coef
        off = (o.double() - want).abs() - (want.abs() * (10 * U + HALF[dtype] * (1 + 10 * U)) + 2.0 ** -126)
        assert not bool((off > 0).any())
    assert torch.equal(buf, before)
    clip(oft.grad_list(grads))
    for g, o in zip(grads, outs):
        assert torch.equal(g, o)
        g.fill_(1.0)
        o.fill_(1.0)
    assert bool((buf == 1).all()) and bool((mark == 1).all())  # nothing between the tensors
