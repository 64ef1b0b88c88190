"""append_kv and tree_attention on queries, keys and values that are parts of one
tensor's rows, as a fused product leaves them: the queries are rotated and replaced
in place."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from entropy_decoding_df11_amd import df11  # noqa: E402
from test_gpu_attention import DEV, Case, gen  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads,kv_heads,dim,tokens", [(4, 2, 64, [1, 1, 1]), (8, 2, 128, [5, 33, 1]), (3, 3, 80, [7, 0, 2])])
def test_one_tensor_of_rows(heads, kv_heads, dim, tokens, dtype):
    case = Case([0, 90, 31], tokens, dtype, heads, kv_heads, dim, seed=50)
    rows = torch.randn(case.total, (heads + 2 * kv_heads) * dim, generator=gen(51)).to(dtype).to(DEV)
    rotary = df11.rotary_table(300, dim)

    def step(rows, in_place):
        q, k, v = (t.unflatten(-1, (-1, dim)) for t in rows.split([heads * dim, kv_heads * dim, kv_heads * dim], 1))
        if not in_place:
            q, k, v = (t.clone() for t in (q, k, v))
        case.upload()
        got = df11.append_kv(k, v, case.dk, case.dv, *case.batch, q=q, rotary=rotary, q_out=q if in_place else None)
        out = df11.tree_attention(got, case.dk, case.dv, *case.batch, out=got if in_place else None)
        return out, case.dk, case.dv

    fused = rows.clone()
    want, got = step(rows, False), step(fused, True)
    assert got[0].data_ptr() == fused.data_ptr()
    for a, b in zip(got, want):
        assert torch.equal(a.nan_to_num(7), b.nan_to_num(7))
    assert torch.equal(fused[:, heads * dim:], rows[:, heads * dim:])
