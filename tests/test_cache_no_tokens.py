"""append_kv and tree_attention of no tokens, whose tensors have no address: nothing to do,
and nothing refused (as in test_cache_and_loss_refusals.py, without a GPU)."""

from test_cache_and_loss_refusals import INVALID, Q, _append, _attend

NONE = dict(k=None, v=None, q=None, q_out=None, q_heads=4, q_stride=256, q_head_stride=64, q_out_stride=256,
            q_out_head_stride=64)


def test_no_tokens():
    assert _append(batch=dict(tokens=0), **NONE) == 0
    assert _append(batch=dict(tokens=0), **dict(NONE, rotary=None)) == 0
    assert _append(batch=dict(tokens=1), **dict(Q, q=None, q_out=None)) == INVALID
    assert _attend(batch=dict(tokens=0), q=None, out=None) == 0
