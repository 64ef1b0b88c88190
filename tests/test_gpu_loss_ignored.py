"""Tokens that the cross entropy ignores, where the losses' own gradient is not finite."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from entropy_decoding_df11_amd import df11  # noqa: E402
from test_gpu_loss import DEV, Head  # noqa: E402


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_ignored_tokens_stay_zero(value):
    """As where the losses' logarithm is taken: an ignored token's is minus infinity, and so is its slope."""
    head = Head(40, 320, 64, seed=43)
    x = head.dx_.clone().requires_grad_()
    ignored = head.dt == -100
    dy = torch.ones(40, device=DEV)
    want, = torch.autograd.grad(head.run_on(x), x, dy)
    dx, = torch.autograd.grad(head.run_on(x), x, torch.where(ignored, value, dy))
    assert bool(ignored.any()) and torch.equal(dx, want) and bool((dx[ignored] == 0).all())


def test_scored_tokens_do_not():
    """A token whose gradient is zero because its target is certain carries what is not finite on."""
    head = Head(40, 320, 64, seed=44, lean=0.0)
    head.x = (60 * head.w[torch.where(head.targets < 0, 0, head.targets)].float() / 0.05).bfloat16() * 8
    x = head.x.to(DEV).requires_grad_()
    loss = head.run_on(x)
    certain = (loss.detach() == 0) & (head.dt != -100)
    assert bool(certain.any())
    dx, = torch.autograd.grad(loss, x, torch.full_like(loss, math.nan))
    assert bool(dx[head.dt != -100].isnan().all()) and bool((dx[head.dt == -100] == 0).all())
