"""Attention where scores are far beyond what a softmax tells apart, up to float32's
range: a score times c is rounded by half of its last place, which is then many
powers of two.  Places with such scores below the others add nothing, one above all
others takes all, and no output is NaN."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from test_gpu_attention import E, Case  # noqa: E402


def far(dtype):
    """Keys whose scores (queries of 8 in one dimension, a scale of 1/8) are these, and their number's roundings of either sign."""
    return [-1e38, -1.7e38, -2.3e38, -3e38, -1e20, -3e12] if dtype == torch.bfloat16 else [-65000.0, -50000.0, -41111.0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,places", [(1, 700), (1, 5000), (3, 300), (40, 300), (70, 3000)])
def test_places_far_below(tokens, places, dtype):
    """A sequence's first 512 places, or all but the last 40, with such keys: the output is that of the others."""
    for low in far(dtype):
        case = Case([places], [tokens], dtype, 4, 1, 64, page=16, seed=32)
        lost = min(512, places - 40)
        size = 1.0 if dtype == torch.bfloat16 else 60000.0  # (of the query: float16 has no larger keys)
        p = torch.arange(places + tokens)
        at = case.table[0].long()[p // case.page], p % case.page
        case.q[..., 0] = size
        case.k[(*at, slice(None), 0)] = 0
        early = p[:lost]
        case.k[(case.table[0].long()[early // case.page], early % case.page)] = 0
        case.k[(case.table[0].long()[early // case.page], early % case.page, slice(None), 0)] = low
        case.upload()
        got, lse = (t.cpu().double() for t in case.attend(return_lse=True))
        o, tol, want, lse_tol = near(case, lost)
        assert bool(got.isfinite().all()) and bool(((got - o).abs() <= tol).all())
        assert bool(((lse - want).abs() <= lse_tol).all())


def near(case, lost):
    """What the case expects of the places from `lost` on (the others' keys made zero and not seen)."""
    seen = case.seen

    def without(s, mask):
        out = seen(s, mask)
        out[:, :lost] = False
        return out

    case.seen = without
    return case.expect()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,places", [(1, 700), (1, 5000), (40, 300), (70, 3000)])
def test_one_place_far_above(tokens, places, dtype):
    for high in far(dtype):
        case = Case([places], [tokens], dtype, 4, 1, 64, page=16, seed=33)
        case.q[..., 0] = -1.0 if dtype == torch.bfloat16 else -60000.0
        p = torch.arange(places + tokens)
        at = case.table[0].long()[p // case.page], p % case.page
        case.k[(*at, slice(None), 0)] = 0
        one = 137
        case.k[case.table[0, one // case.page], one % case.page, :, 0] = high
        case.upload()
        got = case.attend().cpu()
        value = case.v[case.table[0, one // case.page], one % case.page, 0]
        assert torch.equal(got, value.expand(got.shape))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,places", [(1, 700), (1, 5000), (40, 3000), (70, 3000)])
def test_large_scores_alike(tokens, places, dtype):
    """Places of one score have one weight, whichever block they are in: the output is the values' mean.
    (Weights are alike to the last bit, so that their rounding cancels: u of the result and the sums' n e are left.)"""
    for score in (9e3, -9e3, 1.1e5, -1.3e5, 1.1e6, -1.7e6, 7.1e6, -1.1e7):
        case = Case([places], [tokens], dtype, 4, 1, 64, page=16, seed=34)
        p = torch.arange(places + tokens)
        at = case.table[0].long()[p // case.page], p % case.page
        case.q.zero_()
        case.k[at] = 0
        case.q[..., 0] = 8000
        case.k[(*at, slice(None), 0)] = score / 1000  # (of a scale of 1/8)
        case.upload()
        got = case.attend().cpu().double()
        v = case.v[at][:, 0].double()
        for t in range(tokens):
            mean, size = v[:places + t + 1].mean(0), v[:places + t + 1].abs().mean(0)
            u = torch.finfo(dtype).eps / 2
            assert bool(((got[t] - mean).abs() <= u * mean.abs() + 2 * (places + tokens) * E * size).all()), (score, t)
