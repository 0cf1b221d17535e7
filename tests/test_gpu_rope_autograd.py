"""pkv_rope of tensors that require a gradient.

A rotation in 32 bits is within 4e-7 factor (|x_a| + |x_b|) of the 64-bit one and
is rounded once to the tensor's type (eps / 2 of the value, f16 below 2^-14 by
2^-25); a gradient is a rotation of the incoming one.
"""
import numpy as np
import pytest
import torch

from test_gpu_rope import close, formula, inputs

pytestmark = pytest.mark.gpu

import paged_kv_cache_406_b200 as P  # noqa: E402


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("n,heads,d,rot", [(1, 2, 64, 64), (33, 3, 128, 44), (9, 4, 80, 80)])
def test_gradient(native, dtype, interleaved, transpose, n, heads, d, rot):
    x, pos, inv = inputs(n, heads, d, rot, dtype, n)
    dy, _, _ = inputs(n, heads, d, rot, dtype, n + 1)
    leaf = x.clone().requires_grad_()
    y = P.pkv_rope(leaf, pos, inv, interleaved, 1.5, transpose)
    assert y.requires_grad and torch.equal(y, P.pkv_rope(x, pos, inv, interleaved, 1.5, transpose))
    (grad,) = torch.autograd.grad(y, leaf, dy)
    want, mag = formula(dy, pos, inv, 1.5, interleaved, not transpose)
    assert grad.dtype == x.dtype
    close(grad, want, mag, 1.5, x.dtype)


def test_gradient_against_differences(native):
    """y is linear in x, so the difference of a sum of y over x +- u is exact up to roundings."""
    x, pos, inv = inputs(20, 3, 64, 44, "f32", 4)
    u, _, _ = inputs(20, 3, 64, 44, "f32", 6)
    leaf = x.clone().requires_grad_()
    y = P.pkv_rope(leaf, pos, inv)
    loss = lambda t: float((P.pkv_rope(t, pos, inv).double() ** 2).sum())  # noqa: E731
    (y.double() ** 2).sum().backward()
    step = 2.0 ** -6
    diff = (loss(x + step * u) - loss(x - step * u)) / (2 * step)  # a square's central difference is exact
    got = float((leaf.grad.double() * u.double()).sum())
    # each y is off by at most 4e-7 (|x_a| + |x_b|) + 2^-24 |y|, relative to step: sums of 3840 such terms
    pair = x.abs().double() + u.abs().double()
    tol = float((2 * pair * 8 * 6e-7 * pair).sum() / step)
    assert abs(diff - got) <= tol


def test_views_expanded_gradients_and_second_derivatives(native):
    x, pos, inv = inputs(12, 8, 64, 64, "f32", 3)
    leaf = x.clone().requires_grad_()
    y = P.pkv_rope(leaf[:, 2:5], pos, inv)  # heads of a wider projection
    y.sum().backward()                      # an expanded gradient of ones
    ones = torch.ones_like(y)
    want, mag = formula(ones, pos, inv, 1.0, False, True)
    close(leaf.grad[:, 2:5], want, mag, 1.0, torch.float32)
    assert not bool(leaf.grad[:, :2].any()) and not bool(leaf.grad[:, 5:].any())
    a, g = x.clone().requires_grad_(), torch.ones_like(x).requires_grad_()
    (dx,) = torch.autograd.grad(P.pkv_rope(a, pos, inv), a, g, create_graph=True)
    (back,) = torch.autograd.grad(dx, g, x)  # the derivative by g of R^T g along x: R x
    assert torch.equal(back, P.pkv_rope(x, pos, inv))
    empty = torch.empty(0, 8, 64, device="cuda", requires_grad=True)
    P.pkv_rope(empty, pos[:0], inv).sum().backward()
    assert empty.grad.shape == (0, 8, 64)


def test_where_no_gradient_is_recorded(native):
    x, pos, inv = inputs(4, 8, 64, 64, "bf16", 3)
    leaf = x.clone().requires_grad_()
    with torch.no_grad():
        y = P.pkv_rope(leaf, pos, inv)
        assert not y.requires_grad
        assert torch.equal(P.pkv_rope(leaf, pos, inv, out=torch.empty_like(x)), y)
    for out in (torch.empty_like(x), leaf.detach()):
        with pytest.raises(RuntimeError):
            P.pkv_rope(leaf, pos, inv, out=out)
    assert torch.equal(leaf.detach(), x)  # nothing was written in place
    with torch.inference_mode():
        assert torch.equal(P.pkv_rope(leaf, pos, inv), y)
    moved = pos.clone()
    y = P.pkv_rope(leaf, moved, inv)
    moved += 1
    with pytest.raises(RuntimeError):  # the positions of the forward pass are gone
        y.sum().backward()
    assert np.isfinite(float(y.detach().float().sum()))


def test_captured_forward_and_backward(native):
    """Both passes in one graph, replayed on new contents."""
    x, pos, inv = inputs(40, 8, 128, 128, "bf16", 2)
    dy, _, _ = inputs(40, 8, 128, 128, "bf16", 3)
    leaf = x.clone().requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(P.pkv_rope(leaf, pos, inv), leaf, dy)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = P.pkv_rope(leaf, pos, inv)
        (grad,) = torch.autograd.grad(y, leaf, dy)
    for sign in (1, -1):
        with torch.no_grad():
            leaf.copy_(sign * x)
            dy.mul_(sign)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.detach(), P.pkv_rope(sign * x, pos, inv))
        assert torch.equal(grad, P.pkv_rope(dy, pos, inv, transpose=True))
