"""Attention's weights in the cache's type: a tail far below a row's largest weight.

A weight is rounded to the cache's type relative to a reference of which the largest
weight seen when the reference was last taken is 2^7 (fp16) and no weight more than
2^15, so that a place's rounding is at most u of it, or where fp16 is subnormal half
of its least step, 2^-25: 2^-32 of that largest weight, which is a part of the
sum.  Over the places that adds 2^-32 sum |v| to the tolerance of
test_gpu_attention.py (the last sequence's sum |v|, half as much again for the others').  (bfloat16 has float32's range: nothing is added.)"""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from test_gpu_attention import Case  # noqa: E402


def scored(case, scores):
    """Sets keys and queries so that with a scale of 1/8 every query's score of place p is scores[p], in two parts."""
    case.q.zero_()
    case.q[..., :2] = 8
    for s, a in enumerate(case.lengths_):
        p = torch.arange(a + case.tokens[s])
        at = case.table[s].long()[p // case.page], p % case.page
        case.k[at] = 0
        high = scores(p).double().to(case.dtype)
        case.k[(*at, slice(None), 0)] = high[:, None]
        case.k[(*at, slice(None), 1)] = (scores(p).double() - high.double()).to(case.dtype)[:, None]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("gap", [10, 14, 16, 17, 18, 20])
@pytest.mark.parametrize("seqs,tokens,kv_heads,places", [(1, 1, 1, 131072), (1, 40, 1, 30000), (1, 3, 1, 600), (32, 40, 8, 2000)])
def test_one_place_far_ahead(seqs, tokens, kv_heads, places, gap, dtype):
    """An early place that takes most of the weight and adds nothing: the output is the others'."""
    case = Case([places] * seqs, [tokens] * seqs, dtype, 4 if seqs == 1 else kv_heads, kv_heads, 64, page=64, seed=30)
    scored(case, lambda p: torch.where(p == 2, float(gap), 0.0))
    p = torch.arange(places + tokens)
    for s in range(seqs):
        at = case.table[s].long()[p // case.page], p % case.page
        case.v[at] = (case.v[at].float() / 4 + 1).to(dtype)
        case.v[case.table[s, 0], 2] = 0
    case.upload()
    o, tol, lse, lse_tol = case.expect(scale=0.125)
    if dtype == torch.float16:
        tol = tol + 2.0 ** -32 * float(case.v[at].double().abs().sum(0).max()) * 1.5
    got, got_lse = case.attend(scale=0.125, return_lse=True)
    assert bool(((got.cpu().double() - o).abs() <= tol).all()), float(((got.cpu().double() - o).abs() / tol).max())
    assert bool(((got_lse.cpu().double() - lse).abs() <= lse_tol).all())
