"""Attention whose outputs replace their queries, and tiles with rows to spare behind a
sequence's last one.  Cases and tolerances are those of test_gpu_attention.py."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from test_gpu_attention import DEV, Case, tree  # noqa: E402


# tiles of 16, 64, 128 and 256 rows, the last one of a sequence with rows to spare, some cut over workgroups
IN_PLACE = [(8, 1, 128, [0, 3, 900, 40, 0, 5, 5, 5, 300], [1, 1, 9, 1, 1, 1, 1, 1, 1]), (6, 2, 64, [70, 0], [21, 33]),
            (4, 1, 128, [2000, 100], [70, 25]), (4, 1, 128, [0, 500, 30], [130, 71, 333]), (7, 1, 256, [90, 40], [39, 20])]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("heads,kv_heads,dim,lengths,tokens", IN_PLACE)
def test_outputs_on_their_queries(heads, kv_heads, dim, lengths, tokens, masked, dtype):
    """The same bits as with outputs of their own, whichever tile of a sequence is done first."""
    case = Case(lengths, tokens, dtype, heads, kv_heads, dim, seed=20)
    for first in case.starts[:-1]:
        case.q[first] *= 6  # (a first token whose scores move references)
    mask = tree(case).to(DEV) if masked else None
    want, want_lse = case.attend(mask=mask, return_lse=True)
    for _ in range(4):
        q = case.q.to(DEV)
        got, lse = case.attend(q=q, out=q, mask=mask, return_lse=True)
        assert got is q and torch.equal(got, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("heads,kv_heads,dim,lengths,tokens", IN_PLACE)
def test_tiles_with_rows_to_spare(heads, kv_heads, dim, lengths, tokens, masked):
    case = Case(lengths, tokens, torch.bfloat16, heads, kv_heads, dim, seed=21)
    case.check(mask=tree(case) if masked else None)
