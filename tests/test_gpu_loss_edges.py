"""The cross entropy where the target's logit is not finite."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from entropy_decoding_df11_amd import df11  # noqa: E402
from test_gpu_loss import DEV, Head  # noqa: E402


@pytest.mark.parametrize("tokens", [9, 50])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_targets_whose_logit_overflows(tokens, sign):
    """No other logit of theirs does.  The other tokens' losses and gradients are those without it."""
    head = Head(tokens, 192, 64, 150, seed=40)
    w = head.w.clone()
    w[:, 0] = 0
    head.x[:, 0] = 0
    head.targets[head.targets == 7] = 8
    far, ignored = 1, 7
    assert int(head.targets[ignored]) == -100
    head.targets[far] = 7
    dt = head.targets.to(DEV)
    results = []
    for value in (sign * 2.0 ** 110, 0.0):
        w[7, 0] = value
        x0 = head.x.clone()
        x0[[far, ignored], 0] = 2.0 ** 20
        c = df11.compress(w, layout="mfma_tiles")
        x = x0.to(DEV).requires_grad_()
        loss = df11.linear_cross_entropy(c, x, dt, vocab=150, reduction="none")
        dx, = torch.autograd.grad(loss.sum(), x)
        plain = df11.linear_cross_entropy(c, x.detach(), dt, vocab=150, reduction="none")
        results.append((loss.detach(), dx, plain))
    (loss, dx, plain), (want, want_dx, want_plain) = results
    assert bool(loss[far].isnan()) and bool(plain[far].isnan()) and bool(dx[far].isnan().all())
    others = torch.arange(tokens, device=DEV) != far
    assert torch.equal(loss[others], want[others]) and torch.equal(plain[others], want_plain[others])
    assert torch.equal(dx[others, 1:], want_dx[others, 1:]) and bool((dx[ignored] == 0).all())


@pytest.mark.parametrize("tokens", [12, 60])
def test_one_class_of_states_that_are_not_finite(tokens):
    head = Head(tokens, 64, 32, 1, seed=41)
    head.targets[:] = 0
    x0 = head.x.clone()
    for row, value in ((1, math.nan), (2, math.inf), (3, -math.inf)):
        x0[row, 3] = value
    bad = torch.zeros(tokens, dtype=torch.bool, device=DEV)
    bad[1:4] = True
    for grad in (False, True):
        x = x0.to(DEV).requires_grad_(grad)
        loss = df11.linear_cross_entropy(head.head, x, head.targets.to(DEV), vocab=1, reduction="none")
        assert torch.equal(loss.isnan(), bad) and bool((loss[~bad] == 0).all())
        if grad:
            dx, = torch.autograd.grad(loss.sum(), x)
            assert bool(dx[bad].isnan().all()) and bool((dx[~bad] == 0).all())
