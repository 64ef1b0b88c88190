"""Queries, keys and values that are parts of one tensor's rows, and outputs on or beside
them, through the C ABI (as in test_cache_places.py)."""

import pytest

from test_cache_and_loss_refusals import D, INVALID, _append, _attend

# 5 tokens of 4 query heads and 2 of keys and values of 64, two bytes: rows of 512
ROWS = dict(q=D, k=D + 2 * 256, v=D + 2 * 384, q_stride=512, k_stride=512, v_stride=512, q_head_stride=64, q_heads=4)
# the same by heads: (heads, tokens, dim)
HEADS = dict(q=D, k=D + 2 * 4 * 320, v=D + 2 * 6 * 320, q_stride=64, k_stride=64, v_stride=64, q_head_stride=320,
             k_head_stride=320, v_head_stride=320, q_heads=4)


def _taken(call, **k):
    import torch
    assert call(batch=dict(tokens=0), **k) == 0
    if not torch.cuda.is_available():  # (a launch would read what is not there)
        assert call(**k) not in (0, INVALID)


@pytest.mark.parametrize("rows", [ROWS, HEADS])
def test_queries_in_place(rows):
    out = dict(q_out=rows["q"], q_out_stride=rows["q_stride"], q_out_head_stride=rows["q_head_stride"])
    _taken(_append, **rows, **out)
    for bad in (dict(q_out=rows["k"]), dict(q_out=rows["v"]), dict(q_out=rows["q"] + 2 * 64), dict(q_out=rows["k"] - 2),
                dict(dtype=1), dict(k=D), dict(k=D + 2 * 200) if rows is ROWS else dict(v=D + 2 * 300),
                dict(q_out_stride=1024)):
        assert _append(**dict(rows, **out) | bad) == INVALID


def test_outputs_beside_their_queries():
    both = dict(q=D, out=D + 2 * 256, q_stride=512, out_stride=512)
    _taken(_attend, **both)
    _taken(_attend, **dict(both, out=D))
    for bad in (dict(out=D + 2 * 248), dict(out=D + 2 * 8), dict(out=D + 2 * 256, out_stride=1024),
                dict(out=D + 2 * (512 - 64)), dict(q_stride=248, out=D + 2 * 256 * 8, out_stride=512, q=D + 2 * 2000)):
        assert _attend(**dict(both) | bad) == INVALID
