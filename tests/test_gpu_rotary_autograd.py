"""sv.rotary in a graph: the gradient that reaches its input."""
import pytest
import torch

from speculative_decoding_verification_rows_gb300 import build as sv_build
from speculative_decoding_verification_rows_gb300 import sv
from tests.attention_cases import rotate64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv_build.build()
    sv.load()


def inputs(tokens, heads, d, rot, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x, dy = (torch.randn((tokens, heads, d), generator=g).to(dtype) for _ in range(2))
    pos = torch.randint(0, 9000, (tokens,), generator=g, dtype=torch.int32)
    return x, dy, pos, sv.rotary_frequencies(rot, device="cpu")[0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved,inverse", [(False, False), (True, False), (False, True)])
def test_the_gradient_is_the_formulas(dtype, interleaved, inverse):
    x, dy, pos, freq = inputs(21, 3, 64, 32, dtype, 1)
    want, tol = rotate64(dy, pos, freq, interleaved, inverse=not inverse, mscale=1.3)
    leaf = x.cuda().requires_grad_()
    y = sv.rotary(leaf, pos.cuda(), freq.cuda(), interleaved=interleaved, inverse=inverse, mscale=1.3)
    assert y.requires_grad
    y.backward(dy.cuda())
    assert ((leaf.grad.double().cpu() - want).abs() <= tol).all()
    plain = sv.rotary(x.cuda(), pos.cuda(), freq.cuda(), interleaved=interleaved, inverse=inverse, mscale=1.3)
    assert torch.equal(y.detach(), plain) and not plain.requires_grad


def test_the_gradient_is_the_slope():
    x, w, pos, freq = inputs(9, 2, 64, 64, torch.float32, 2)
    leaf = x.cuda().requires_grad_()
    (sv.rotary(leaf, pos.cuda(), freq.cuda(), mscale=0.7) * w.cuda()).sum().backward()
    f = lambda z: float((rotate64(z, pos, freq, mscale=0.7)[0] * w.double()).sum())     # noqa: E731
    _, tol = rotate64(w, pos, freq, inverse=True, mscale=0.7)
    g = torch.Generator().manual_seed(3)
    for _ in range(3):
        step = torch.randn(x.shape, generator=g, dtype=torch.float64)
        slope = (f(x.double() + 1e-3 * step) - f(x.double() - 1e-3 * step)) / 2e-3      # exact: the map is linear
        along = float((leaf.grad.double().cpu() * step).sum())
        assert abs(slope - along) <= float((tol * step.abs()).sum()) + 1e-9 * abs(slope) + 1e-9


def test_shared_heads_views_and_broadcast_gradients():
    x, _, pos, freq = inputs(11, 5, 64, 64, torch.float32, 4)
    ones = torch.ones((11, 6, 64))
    want, tol = rotate64(ones, pos, freq, inverse=True)
    # one head for six: the gradients of the copies add up (six roundings of sums of up to six parts)
    one = x[:, :1].cuda().requires_grad_()
    sv.rotary(one.expand(-1, 6, -1), pos.cuda(), freq.cuda()).sum().backward()
    total = want.sum(1, keepdim=True)
    assert ((one.grad.double().cpu() - total).abs() <= 6 * tol[:, :1] + 6 * 2.0 ** -24 * want.abs().sum(1, keepdim=True)).all()
    # a view of a packed projection, in the middle of a graph
    packed = torch.randn((11, 9, 64), generator=torch.Generator().manual_seed(5)).cuda().requires_grad_()
    sv.rotary((packed * 2.0)[:, 2:8], pos.cuda(), freq.cuda()).sum().backward()
    got = packed.grad.double().cpu()
    assert ((got[:, 2:8] - 2 * want).abs() <= 2 * tol).all()
    assert (got[:, :2] == 0).all() and (got[:, 8:] == 0).all()


def test_a_gradient_of_the_gradient_and_calls_that_record_nothing():
    x, dy, pos, freq = (z.cuda() for z in inputs(7, 2, 64, 64, torch.float32, 6))
    leaf, seed = x.requires_grad_(), dy.requires_grad_()
    y = sv.rotary(leaf, pos, freq, mscale=1.1)
    (dx,) = torch.autograd.grad(y, leaf, seed, create_graph=True)
    (back,) = torch.autograd.grad(dx, seed, torch.ones_like(dx))              # the map itself, of ones
    assert torch.equal(back, sv.rotary(torch.ones_like(dx), pos, freq, mscale=1.1))
    with torch.no_grad():
        assert not sv.rotary(leaf, pos, freq).requires_grad
    out = torch.empty_like(x, requires_grad=False)
    assert sv.rotary(leaf, pos, freq, out=out) is out and not out.requires_grad


def test_positions_changed_before_the_gradient_are_noticed():
    x, dy, pos, freq = (z.cuda() for z in inputs(7, 2, 64, 64, torch.float32, 7))
    y = sv.rotary(x.requires_grad_(), pos, freq)
    pos += 1
    with pytest.raises(RuntimeError):
        y.backward(dy)
