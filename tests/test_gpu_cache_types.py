"""A bfloat16 model on a float16 cache, against the model written out in torch
(test_gpu_generation.py, whose tolerance holds: float16 rounds keys, values and the
attention's outputs, of about one, finer than the bfloat16 that the written-out model
has there)."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from entropy_decoding_df11_amd import runtime  # noqa: E402
from test_gpu_generation import (DEV, FAR, VOCAB, Cache, model, prefill, tree_step, written_out)  # noqa: E402,F401


def test_float16_cache(model):  # noqa: F811
    cache = Cache()
    cache.pairs = [tuple(t.half() for t in pair) for pair in cache.pairs]
    texts, scores = prefill(model, cache)
    want = [written_out(model, t)[:-1].log_softmax(1).gather(1, t[1:, None])[:, 0] for t in texts]
    assert float((scores.cpu().double() - torch.cat(want)).abs().max()) <= FAR
    x, step, targets, paths = tree_step(model, cache, texts)
    y = runtime.operator_model_forward(x, model["blocks"], cache.pairs, step)
    assert y.dtype == torch.bfloat16 and y.shape == x.shape
    scores = runtime.score_tokens(x, model["blocks"], model["head"], targets, cache.pairs, step, vocab=VOCAB)
    want = torch.stack([written_out(model, p)[-1].log_softmax(0)[t] for p, t in zip(paths, targets.cpu())])
    assert float((scores.cpu().double() - want).abs().max()) <= FAR
