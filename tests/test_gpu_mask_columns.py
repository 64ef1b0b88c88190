"""Attention under a mask without columns: a sequence's new tokens see what is cached of
it and none of each other.  Cases and tolerances are those of test_gpu_attention.py."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from test_gpu_attention import DEV, Case  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.bool, torch.uint8])
@pytest.mark.parametrize("tokens", [[9, 20, 2], [1, 1, 1], [200, 90, 3]])
def test_no_columns(tokens, dtype):
    case = Case([3, 50, 0], tokens, torch.bfloat16, 4, 2, 64, seed=7)
    out = case.check(mask=torch.zeros(case.total, 0, dtype=dtype))
    assert bool((out[case.starts[2]:] == 0).all())
    _, lse = case.attend(mask=torch.ones(case.total, 5, dtype=dtype, device=DEV)[:, :0], return_lse=True)
    assert bool((lse[case.starts[2]:] == -math.inf).all()) and bool(lse[:case.starts[2]].isfinite().all())
