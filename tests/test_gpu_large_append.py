"""The cache's append at the most tokens that it takes."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from entropy_decoding_df11_amd import df11  # noqa: E402
from test_gpu_loss import DEV, gen  # noqa: E402


def test_append_of_2_to_24_tokens():
    """Most of them without a place; the second sequence's are the last ones."""
    tokens, heads, dim = 1 << 24, 8, 256
    page, pages = 16, 4
    row = torch.randn(1, heads, dim, generator=gen(60)).bfloat16().to(DEV)
    k, v = row.expand(tokens, -1, -1), (2 * row).expand(tokens, -1, -1)
    cache = [torch.zeros(pages, page, heads, dim, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, tokens - 3, tokens], dtype=torch.int32, device=DEV)
    df11.append_kv(k, v, *cache, table, starts, torch.tensor([5, 9], dtype=torch.int32, device=DEV))
    want = torch.zeros(pages * page, dtype=torch.bool, device=DEV)
    want[5:32] = True
    want[32 + 9:32 + 12] = True
    for got, of in zip(cache, (row, 2 * row)):
        got = got.view(-1, heads, dim)
        assert torch.equal(got[want], of.expand(30, -1, -1)) and bool((got[~want] == 0).all())
