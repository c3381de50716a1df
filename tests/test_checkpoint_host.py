"""Autograd functions over 8-bit checkpoints, without a GPU: which torch operations they
call, and when they make codes.  A frozen weight needs no codes, so these calls run on the CPU."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from integer_quantized_nn_amd import checkpoint as C
from integer_quantized_nn_amd import layers as L


class Ops(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.names = set()

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.names.add(func.overloadpacket.__name__)
        return func(*args, **(kwargs or {}))


@pytest.mark.parametrize("transposed_w", [False, True])
@pytest.mark.parametrize("bias", [False, True])
def test_linear_makes_no_batched_products(bias, transposed_w):
    """torch multiplies a batch whose axes are not in memory order by bmm, with the weight as a
    transposed view on its right; the layer's products have two axes."""
    g = torch.Generator().manual_seed(1)
    w = torch.randn(16, 8, generator=g).t() if transposed_w else torch.randn(8, 16, generator=g)
    b = torch.randn(8, generator=g) if bias else None
    x = torch.randn(5, 3, 16, generator=g).transpose(0, 1).requires_grad_()
    dy = torch.randn(5, 3, 8, generator=g).transpose(0, 1)
    with Ops() as ops:
        y = C.linear(x, w, b)
        dx, = torch.autograd.grad(y, x, dy)
    assert not any("bmm" in n for n in ops.names), ops.names
    x64, w64, b64 = x.detach().double(), w.double(), torch.zeros(8).double() if b is None else b.double()
    want, mag = x64 @ w64.t() + b64, x64.abs() @ w64.abs().t() + b64.abs()
    # 16 (8) products and additions in binary32, a rounding each
    assert y.shape == (3, 5, 8) and dx.shape == x.shape
    assert torch.all((y.double() - want).abs() <= 34 * 2.0 ** -24 * mag)
    assert torch.all((dx.double() - dy.double() @ w64).abs() <= 16 * 2.0 ** -24 * (dy.double().abs() @ w64.abs()))


@pytest.mark.parametrize("shape", [(16,), (4, 16), (2, 3, 16), (3, 0, 16)])
def test_linear_results_may_be_changed_in_place(shape):
    w = torch.randn(8, 16, generator=torch.Generator().manual_seed(2))
    x = torch.ones(shape, requires_grad=True)
    y = C.linear(x, w)
    y.add_(1.0).mul_(2.0)
    y.sum().backward()
    assert y.shape == shape[:-1] + (8,) and x.grad.shape == shape
    assert torch.all((x.grad.double() - 2 * w.double().sum(0)).abs() <= 10 * 2.0 ** -23 * 2 * w.double().abs().sum(0))


def test_linear_makes_no_codes_without_a_gradient(monkeypatch):
    """Evaluation of a trained layer quantizes nothing; with gradients on, it does."""
    def quantize_groups(*args, **kw):
        raise RuntimeError("codes made")

    monkeypatch.setattr(L, "quantize_groups", quantize_groups)
    x, w = torch.ones(3, 16), torch.ones(8, 16, requires_grad=True)
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            y = C.linear(x, w)
        assert torch.equal(y, torch.full((3, 8), 16.0)) and not y.requires_grad
    assert torch.equal(C.linear(x, w.detach()), torch.full((3, 8), 16.0))
    with pytest.raises(RuntimeError, match="codes made"):
        C.linear(x, w)
