"""The largest sizes of the cache's operators and the loss that their launches hold,
through the C ABI: refusals before any launch, which run without a GPU."""

import pytest

from test_cache_and_loss_refusals import A, B, C, E, TOO_LARGE, _load, _loss, _loss_grad, _stream


@pytest.mark.parametrize("tokens", [1 << 24, (1 << 25) - 8, 1 << 26])
def test_loss_with_a_gradient(tokens):
    far = 0x4000000000  # (the gradient spans more than the other addresses are apart)
    head = _stream(rows=256, cols=32)
    assert _loss(w=head, x=A, xs=32, t=tokens, inf=32, outf=256, vocab=256, targets=B, loss=C, grad=far,
                 ws=2 * far, nbytes=1 << 60) == TOO_LARGE
    assert _load().df11_cross_entropy_workspace(head, tokens, 1) == 0


@pytest.mark.parametrize("tokens", [1 << 24, 1 << 26])
def test_the_gradient_itself(tokens):
    far = 0x4000000000
    assert _loss_grad(t=tokens, inf=32, grad=far, dx=2 * far, dxs=32, dy=E) == TOO_LARGE
