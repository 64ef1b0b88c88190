"""A step without tokens through blocks on a cache and the scores (test_gpu_generation.py's model)."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from entropy_decoding_df11_amd import df11, runtime  # noqa: E402
from test_gpu_generation import DEV, DIM, HEADS, HIDDEN, KV, VOCAB, Cache, ints, model  # noqa: E402,F401


def test_no_tokens(model):  # noqa: F811
    cache = Cache()
    before = [[t.clone() for t in pair] for pair in cache.pairs]
    step = runtime.Step(cache.table, ints(0, 0, 0, 0), ints(5, 0, 7), model["rotary"])
    x = torch.zeros(0, HIDDEN, dtype=torch.bfloat16, device=DEV)
    targets = torch.zeros(0, dtype=torch.int64, device=DEV)
    scores = runtime.score_tokens(x, model["blocks"], model["head"], targets, cache.pairs, step, vocab=VOCAB)
    assert scores.shape == (0,) and scores.dtype == torch.float32
    k, q = (torch.zeros(0, n, DIM, dtype=torch.bfloat16, device=DEV) for n in (KV, HEADS))
    where = (*cache.pairs[0], cache.table, step.starts, step.lengths)
    assert df11.append_kv(k, k, *where, q=q, rotary=model["rotary"]).shape == (0, HEADS, DIM)
    assert df11.append_kv(k, k, *where, q=q, q_out=q) is q and df11.append_kv(k, k, *where) is None
    out, lse = df11.tree_attention(q, *where, return_lse=True)
    assert out.shape == q.shape and lse.shape == (0, HEADS)
    for pair, old in zip(cache.pairs, before):
        for t, o in zip(pair, old):
            assert torch.equal(t.nan_to_num(3), o.nan_to_num(3))
