"""Attention whose outputs replace their queries, and tiles with rows to spare behind a
sequence's last one.  Cases and tolerances are those of test_gpu_attention.py."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from test_gpu_attention import DEV, E, Case, tree  # noqa: E402


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


@pytest.mark.parametrize("group", [3, 5, 7])
@pytest.mark.parametrize("lengths,tokens", [([100], [1500]), ([0, 300, 40], [700, 333, 1])])
def test_prompts_of_odd_groups(group, lengths, tokens):
    Case(lengths, tokens, torch.bfloat16, group, 1, 64, seed=22).check()


@pytest.mark.parametrize("group", [3, 4])
def test_prompts_longer_than_their_pages(group):
    """New tokens without a place see the places that there are, in every one of a sequence's tiles."""
    case = Case([700], [900], torch.bfloat16, group, 1, 64, seed=23)
    width = 1300 // case.page
    case.batch = (case.table[:, :width].contiguous().to(DEV), *case.batch[1:])
    got, lse = case.attend(return_lse=True)
    p = torch.arange(width * case.page)
    pages = case.table[0].long()[p // case.page]
    k, v = (half[pages, p % case.page, 0].double() for half in (case.k, case.v))
    for h in range(group):
        z = torch.where(case.seen(0, None)[:, :len(p)], 0.125 * case.q[:, h].double() @ k.t(), -torch.inf)
        far = (got[:, h].cpu().double() - z.softmax(1) @ v).abs()
        assert bool((far <= 2.1 * 2.0 ** -8 * (z.softmax(1) @ v.abs())).all())
        d = 0.125 * (64 + 4) * E * (case.q[:, h].double().abs() @ k.abs().t()).amax(1) + 8 * E * z.abs().nan_to_num(0, 0, 0).amax(1)
        most = 1.01 * (2 * d + (8 + len(p)) * E + 4 * E * z.logsumexp(1).abs())
        assert bool(((lse[:, h].cpu().double() - z.logsumexp(1)).abs() <= most).all())
