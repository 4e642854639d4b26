"""rotary under autograd: the recorded gradient against the formula in 64 bits
and against differences, through views, twice, and with in-place writes seen.

Bounds as in test_gpu_kv.py: sine and cosine good to 2^-19 of |a| + |b|, results
rounded once to their type."""
import pytest
import torch

from test_gpu_kv import BF, DEV, F32, HF, UNIT, gen, randn, rotary_want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("layout,rd", [("half", 64), ("interleaved", 64), ("half", 32), ("interleaved", 30)])
def test_autograd_gives_the_turn_back(uz, layout, rd, dtype):
    rates, factor = uz.rotary_rates(rd, scaling="ramp", factor=4.0, original_length=512)
    plan = uz.rotary_plan(rd, layout=layout, scaling="ramp", factor=4.0, original_length=512)
    g = gen(rd)
    pos = torch.randint(0, 1 << 16, (2, 11), generator=g, device=DEV).to(torch.int32)
    w = randn(g, 2, 11, 3, 64, dtype=dtype)
    for f, sign in ((uz.rotary, -1.0), (uz.rotary_backward, 1.0)):
        base = randn(g, 2, 11, 5, 64, dtype=dtype).requires_grad_()
        y = f(base[:, :, 1:4], pos, plan)  # heads of a projection: a strided view
        assert y.requires_grad
        with torch.no_grad():
            assert torch.equal(y, f(base[:, :, 1:4], pos, plan))
        y.backward(w)
        want, bound = rotary_want(w, pos, rates, factor, rd, layout, sign)
        got = base.grad[:, :, 1:4]
        assert torch.all((got.double() - want).abs() <= bound + 2 * UNIT[dtype] * want.abs() + 2.0 ** -25)
        assert torch.all(base.grad[:, :, :1] == 0) and torch.all(base.grad[:, :, 4:] == 0)


def test_autograd_against_differences_and_twice(uz):
    plan = uz.rotary_plan(48, layout="interleaved")
    g = gen(7)
    x, w, u = (randn(g, 13, 3, 96) for _ in range(3))
    pos = torch.randint(0, 5000, (13,), generator=g, device=DEV).to(torch.int32)
    x.requires_grad_()
    loss = (uz.rotary(x, pos, plan).square() * w).sum() / 2
    (grad,) = torch.autograd.grad(loss, x, create_graph=True)
    with torch.no_grad():
        f = lambda z: (uz.rotary(z, pos, plan).double().square() * w.double()).sum() / 2
        diff = (f(x + u) - f(x - u)) / 2  # of a quadratic: exact at any step
        # y is off by 2^-19 (|a| + |b|), so f by less than 2^-17 max|w| |z|^2 of its argument z
        size = w.abs().max().double() * (x.double().norm() + u.double().norm()) ** 2
    assert abs(diff - (grad.double() * u.double()).sum()) <= 2.0 ** -16 * size
    (twice,) = torch.autograd.grad((grad * u).sum(), x)  # the second derivative along u: R^T w R u
    with torch.no_grad():
        want = uz.rotary_backward(w * uz.rotary(u, pos, plan), pos, plan)
    assert torch.allclose(twice, want, rtol=2.0 ** -18, atol=2.0 ** -18)


def test_autograd_of_a_sum_and_of_nothing(uz):
    plan = uz.rotary_plan(8)
    pos = torch.arange(4, dtype=torch.int32, device=DEV)
    x = torch.ones(4, 2, 8, device=DEV, requires_grad=True)
    uz.rotary(x, pos, plan).sum().backward()  # the gradient arrives as one element expanded
    assert torch.equal(x.grad, uz.rotary_backward(torch.ones(4, 2, 8, device=DEV), pos, plan))
    e = torch.ones(0, 2, 8, device=DEV, requires_grad=True)
    uz.rotary(e, pos[:0], plan).sum().backward()
    assert e.grad.shape == e.shape


def test_in_place_writes_are_seen(uz):
    plan = uz.rotary_plan(8)
    pos = torch.arange(4, dtype=torch.int32, device=DEV)
    x = torch.ones(4, 2, 8, device=DEV, requires_grad=True)
    y = x * 2
    z = y * y  # keeps y
    with torch.no_grad():
        uz.rotary(y, pos, plan, out=y)
    with pytest.raises(RuntimeError, match="in-?place"):
        z.sum().backward()
    positions = pos.clone()
    z = uz.rotary(x, positions, plan)
    positions += 1
    with pytest.raises(RuntimeError, match="in-?place"):
        z.sum().backward()
    with pytest.raises(ValueError, match="gradient"):
        uz.rotary(x, pos, plan, out=torch.empty_like(x))
    with torch.inference_mode():  # tensors without versions
        a = torch.ones(4, 2, 8, device=DEV)
        assert uz.rotary(a, pos, plan, out=a) is a
