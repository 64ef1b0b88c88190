"""Attention's quotient: numerator and denominator have the same weights, as they are
rounded to the cache's type, and the logarithm of the sum has them unrounded."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from test_gpu_attention import Case  # noqa: E402
from test_gpu_attention_weights import scored  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,places", [(1, 40), (1, 900), (1, 5000), (3, 700), (40, 300), (70, 5000)])
def test_equal_values(tokens, places, dtype):
    """Where all values are alike the output is that value.
    (One place of eight has a weight of one; the others' is rounded down to a half from almost half a step above
    it.  Those and the values have few bits, so that the sums are exact.)"""
    case = Case([places], [tokens], dtype, 4, 1, 64, page=16, seed=31)
    low = math.log(0.5 * (1 + 0.49 * torch.finfo(dtype).eps))
    scored(case, lambda p: torch.where(p % 8 == 0, 0.0, torch.tensor(low, dtype=torch.float64)))
    p = torch.arange(places + tokens)
    value = torch.tensor([1 + 126 / 128, 1.0, -3.96875, 0.25]).repeat(16).to(dtype)
    case.v[case.table[0].long()[p // case.page], p % case.page] = value
    case.upload()
    _, _, lse, lse_tol = case.expect(scale=0.125)
    got, got_lse = case.attend(scale=0.125, return_lse=True)
    assert torch.equal(got.cpu(), value.expand(got.shape))
    assert bool(((got_lse.cpu().double() - lse).abs() <= lse_tol).all())
    assert torch.equal(case.attend(scale=0.125), got)
