"""Forward-mode derivatives, which the operators do not carry, are refused and not dropped.
(A dual tensor does not require a gradient, and torch.no_grad does not turn it off.)"""

import types

import pytest

from entropy_decoding_df11_amd import df11

torch = pytest.importorskip("torch")
from torch.autograd import forward_ad  # noqa: E402

CACHE = torch.zeros(8, 16, 2, 64, dtype=torch.bfloat16)
BATCH = dict(page_table=torch.zeros(3, 4).int(), starts=torch.zeros(4).int(), lengths=torch.zeros(3).int())
KV, Q = torch.zeros(5, 2, 64, dtype=torch.bfloat16), torch.zeros(5, 4, 64, dtype=torch.bfloat16)
HEAD = types.SimpleNamespace(shape=(128, 64), tile_cols=64, decode_table_bits=11, _bufs={"enc": torch.zeros(1)})
X, T = torch.zeros(5, 64, dtype=torch.bfloat16), torch.zeros(5, dtype=torch.int64)

CALLS = [
    (df11.append_kv, dict(BATCH, k=KV, v=KV.clone(), k_cache=CACHE, v_cache=CACHE.clone(), q=Q, rotary=torch.zeros(9, 64)),
     ("k", "v", "q", "k_cache", "v_cache", "rotary")),
    (df11.tree_attention, dict(BATCH, q=Q, k_cache=CACHE, v_cache=CACHE.clone(), out=Q.clone()),
     ("q", "k_cache", "v_cache", "out")),
    (df11.linear_cross_entropy, dict(w=HEAD, x=X, targets=T), ("x",)),
    (df11.rms_norm, dict(x=X, weight=torch.ones(64), residual=X.clone()), ("x", "weight", "residual")),
    (df11.matmul_epilogue, dict(w=HEAD, x=X, bias=torch.zeros(128), residual=torch.zeros(5, 128)), ("x", "bias", "residual")),
    (df11.gated_matmul, dict(gate=HEAD, up=HEAD, x=X), ("x",)),
]


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("call,given,names", CALLS)
def test_dual_tensors(call, given, names, grad):
    with torch.set_grad_enabled(grad), forward_ad.dual_level():
        for name in names:
            dual = forward_ad.make_dual(given[name], torch.ones_like(given[name]))
            with pytest.raises(ValueError, match="forward-mode"):
                call(**dict(given, **{name: dual}))
        with pytest.raises(ValueError, match="GPU"):  # (and others pass)
            call(**given)
    with pytest.raises(ValueError, match="GPU"):
        call(**given)
