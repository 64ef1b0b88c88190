"""The loss at the most tokens that it takes with its gradient, and more without it."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from entropy_decoding_df11_amd import df11  # noqa: E402
from test_gpu_loss import DEV, E, U, gen  # noqa: E402


@pytest.mark.parametrize("tokens,grad", [((1 << 24) - 1, True), ((1 << 25) + 3, False)])
def test_loss_of_many_tokens(tokens, grad):
    """The first, some and the last tokens against the formula in 64 bits (tolerances of test_gpu_loss.py)."""
    w = (torch.randn(64, 32, generator=gen(61)) * 0.3).bfloat16()
    head = df11.compress(w, layout="mfma_tiles")
    g = torch.Generator(device=DEV).manual_seed(62)
    x = torch.randn(tokens, 32, device=DEV, generator=g, dtype=torch.bfloat16)
    t = torch.randint(0, 64, (tokens,), device=DEV, generator=g)
    x.requires_grad_(grad)
    loss = df11.linear_cross_entropy(head, x, t, reduction="none")
    some = torch.cat([torch.arange(500), torch.arange(tokens // 2, tokens // 2 + 500), torch.arange(tokens - 500, tokens)]).to(DEV)
    wd, xs, ts = w.to(DEV).double(), x.detach()[some].double(), t[some]
    z = xs @ wd.t()
    lse, zy = z.logsumexp(1), z.gather(1, ts[:, None])[:, 0]
    d = (36 * E * (xs.abs() @ wd.abs().t())).amax(1)
    big = d + 4 * E + 81 * E + 8 * E * (lse.abs() + zy.abs())
    assert bool(((loss.detach()[some].double() - (lse - zy)).abs() <= 2.02 * big).all())
    if grad:
        dx, = torch.autograd.grad(loss, x, torch.ones_like(loss))
        p = (z - lse[:, None]).exp().scatter(1, ts[:, None], 0)
        s, wy = p.sum(1, keepdim=True), wd[ts]
        want, size = p @ wd - s * wy, p @ wd.abs()
        far = 1.02 * ((U + 66 * E) * size + (2 * big[:, None] + 8 * E) * (size + s * wy.abs())) + U * want.abs()
        assert bool(((dx[some].double() - want).abs() <= far + 4 * E * want.abs()).all())
    else:
        with pytest.raises(RuntimeError, match="TOO_LARGE"):
            df11.linear_cross_entropy(head, x[:1 << 24].requires_grad_(), t[:1 << 24])
