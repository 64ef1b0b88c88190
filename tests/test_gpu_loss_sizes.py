"""The cross entropy of logits beyond what a softmax tells apart, up to float32's range:
a logit times log2(e) is rounded by half of its last place, many powers of two.  Losses
are of the formula's size, gradients the difference of two rows.

Logits of one product that is exact and of small ones: a loss of z - z_y is off by
the float32 rounding of z and of log2(e) z and its way back, 8 E of it."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from entropy_decoding_df11_amd import df11  # noqa: E402
from test_gpu_loss import DEV, E, U, gen  # noqa: E402

SIZES = [2.0 ** 22, 2.0 ** 27, 2.0 ** 31, 2.0 ** 33, 1e12, 1e20, 1e37]


def run(w, x, t):
    head = df11.compress(w, layout="mfma_tiles")
    y = x.to(DEV).requires_grad_()
    loss = df11.linear_cross_entropy(head, y, t.to(DEV), reduction="none")
    dx, = torch.autograd.grad(loss.sum(), y)
    plain = df11.linear_cross_entropy(head, x.to(DEV), t.to(DEV), reduction="none")
    return loss.detach().double().cpu(), plain.double().cpu(), dx.double().cpu()


@pytest.mark.parametrize("tokens", [9, 60])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_one_logit_far_off(tokens, size, sign):
    """Another class's far above the target's, or the target's far below all others."""
    w = (torch.randn(320, 64, generator=gen(70)) * 0.05).bfloat16()
    w[:, 0] = 0
    w[200, 0] = sign * 2.0 ** 10
    x = torch.randn(tokens, 64, generator=gen(71))
    x[:, 0] = size * 2.0 ** -10 * (1 + torch.rand(tokens, generator=gen(72)))
    x = x.bfloat16()
    t = torch.randint(0, 200, (tokens,), generator=gen(73))
    if sign < 0:
        t[:] = 200
    z = x.double() @ w.double().t()
    want = z.logsumexp(1) - z.gather(1, t[:, None])[:, 0]
    p = z.softmax(1)
    want_dx = p @ w.double() - w[t].double()
    loss, plain, dx = run(w, x, t)
    for got in (loss, plain):
        assert bool(((got - want).abs() <= 8 * E * want.abs() + 1e-3).all())
    # (a logit is off by 2 d: where other classes share the probability that moves it among them)
    d = 68 * E * (x.double()[:, 1:].abs() @ w.double()[:, 1:].abs().t()).amax(1, keepdim=True)
    size_ = p @ w.double().abs() + w[t].double().abs()
    assert bool(((dx - want_dx).abs() <= 1.02 * (2 * U + 2 * d + 200 * E) * size_).all())


@pytest.mark.parametrize("tokens", [9, 60])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_all_logits_alike(tokens, size, sign):
    """Of any size: the logarithm of their number, as far as float32 can tell it, and finite."""
    w = torch.full((320, 64), 0.0).bfloat16()
    w[:, 0] = sign * 2.0 ** 10
    x = torch.zeros(tokens, 64)
    x[:, 0] = size * 2.0 ** -10 * (1 + torch.rand(tokens, generator=gen(74)))
    x = x.bfloat16()
    t = torch.randint(0, 320, (tokens,), generator=gen(75))
    z = (x.double() @ w.double().t())[:, 0].abs()
    loss, plain, dx = run(w, x, t)
    for got in (loss, plain):
        assert bool(got.isfinite().all()) and bool((got >= 0).all())
        assert bool(((got - 5.7683).abs() <= 8 * E * z + 1e-3).all())
    assert bool(dx.isfinite().all())
