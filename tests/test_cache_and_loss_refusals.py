"""Argument checks of the paged cache's operators and of the cross entropy,
through the C ABI and the binding.  Every refusal comes before any launch, so
these run without a GPU; the addresses are never read."""

import ctypes
import os

import pytest

from entropy_decoding_df11_amd import _lib

INVALID, SMALL, TOO_LARGE, HIP = -1, -5, -7, -8

# (far apart, 256-byte aligned)
A, B, C, D, E, F, G, H, I, J = (0x100000000 * (i + 1) for i in range(10))


def _load():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libdf11.so is not built")
    return _lib.load()


def _pack(format, fields, given):
    assert not set(given) - set(fields)
    return format.pack(*((given.get(n) or 0) for n in fields))


def _cache(**k):
    """Eight pages of 16 places, two heads of 64."""
    a = dict(k=A, v=B, kp=2048, kl=128, kh=64, vp=2048, vl=128, vh=64, n=8, page=16, heads=2, dim=64, t=0)
    a.update(k)
    return _lib.KV_CACHE.pack(a["k"] or 0, a["v"] or 0, a["kp"], a["kl"], a["kh"], a["vp"], a["vl"], a["vh"], a["n"], a["page"],
                              a["heads"], a["dim"], a["t"], 0)


def _batch(**k):
    a = dict(starts=C, lengths=C + 0x1000, table=C + 0x2000, stride=4, seqs=3, pages=4, tokens=5)
    a.update(k)
    return _lib.KV_BATCH.pack(a["starts"] or 0, a["lengths"] or 0, a["table"] or 0, a["stride"], a["seqs"], a["pages"],
                              a["tokens"], 0)


def _append(cache=None, batch=None, **k):
    a = dict(k=D, v=E, k_stride=128, k_head_stride=64, v_stride=128, v_head_stride=64, dtype=0)
    a.update(k)
    return _load().df11_append_kv(_cache(**(cache or {})), _batch(**(batch or {})), _pack(_lib.APPEND, _lib.APPEND_FIELDS, a), None)


Q = dict(q=F, q_stride=256, q_head_stride=64, q_heads=4, q_out=G, q_out_stride=256, q_out_head_stride=64)
ROT = dict(rotary=H, rotary_rows=100, rotary_dims=64)

BAD_CACHES = [dict(k=None), dict(v=None), dict(k=A + 8), dict(v=B + 2), dict(kp=2049), dict(kl=4), dict(vh=1),
              dict(kp=1 << 40), dict(n=0), dict(n=1 << 31), dict(page=0), dict(page=(1 << 20) + 1), dict(heads=0),
              dict(heads=4097), dict(dim=0), dict(dim=60), dict(dim=264), dict(t=2), dict(t=7),
              dict(n=(1 << 31) - 1, kp=1 << 39)]
BAD_BATCHES = [dict(starts=None), dict(starts=C + 2), dict(lengths=None), dict(lengths=C + 1), dict(table=None),
               dict(table=C + 3), dict(tokens=(1 << 24) + 1), dict(seqs=(1 << 24) + 1), dict(pages=(1 << 26) + 1),
               dict(stride=1 << 40)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_caches_are_checked(bad):
    assert _append(cache=bad) == INVALID
    assert _attend(cache=bad) == INVALID


@pytest.mark.parametrize("bad", BAD_BATCHES)
def test_batches_are_checked(bad):
    assert _append(batch=bad) == INVALID
    assert _attend(batch=bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=None), dict(k=D + 1), dict(v=E + 1), dict(dtype=3), dict(dtype=2, k=D + 2),
    dict(k_stride=1 << 40), dict(v_head_stride=1 << 32),
    dict(Q, q_out=None), dict(Q, q=None), dict(Q, q_heads=0), dict(Q, q_heads=4097), dict(q_heads=4), dict(Q, q=F + 1),
    dict(Q, q_out=G + 1), dict(Q, q_out_stride=255), dict(Q, q_out_head_stride=63), dict(Q, q_out_head_stride=1 << 32),
    dict(ROT, rotary=H + 2), dict(ROT, rotary_dims=0), dict(ROT, rotary_dims=63), dict(ROT, rotary_dims=66),
    dict(ROT, rotary_rows=0), dict(ROT, rotary_rows=1 << 41), dict(ROT, interleaved=2), dict(positions=I + 2),
    dict(k=A), dict(v=A), dict(k=B + 64), dict(Q, q=A), dict(Q, q_out=A), dict(Q, q_out=D), dict(Q, q_out=E),
    dict(Q, q_out=F + 2), dict(Q, q_out=F, q_out_stride=512), dict(Q, q_out=F, dtype=1), dict(Q, q_out=C),
    dict(Q, **dict(ROT, q_out=H)), dict(Q, q_out=I, positions=I), dict(ROT, rotary=A), dict(positions=B),
])
def test_append_refuses(bad):
    assert _append(**bad) == INVALID


@pytest.mark.parametrize("bad", [dict(k=C), dict(v=C + 0x2000)])
def test_append_refuses_a_cache_on_the_batch(bad):
    assert _append(cache=bad) == INVALID


@pytest.mark.parametrize("bad", [dict(kp=0), dict(vp=56), dict(kl=0), dict(vl=8), dict(kh=0), dict(vh=56), dict(v=A)])
def test_append_refuses_places_on_each_other(bad):
    """An expanded cache, or one tensor for both halves; attention, which only reads, takes them."""
    assert _append(cache=bad) == INVALID
    assert _attend(cache=bad, batch=dict(seqs=0)) == 0


def test_append_takes_nothing():
    assert _append(batch=dict(tokens=0)) == 0
    assert _append(batch=dict(tokens=0), k=None, v=None) == 0
    assert _append(batch=dict(seqs=0, lengths=None, table=None)) == 0
    assert _load().df11_append_kv(None, _batch(), _pack(_lib.APPEND, _lib.APPEND_FIELDS, {}), None) == INVALID
    assert _load().df11_append_kv(_cache(), None, _pack(_lib.APPEND, _lib.APPEND_FIELDS, {}), None) == INVALID
    assert _load().df11_append_kv(_cache(), _batch(), None, None) == INVALID


def _attend(cache=None, batch=None, ws=J, nbytes=1 << 30, entry="run", **k):
    a = dict(q=D, out=E, q_stride=256, q_head_stride=64, out_stride=256, out_head_stride=64, q_heads=4, scale=0.125)
    a.update(k)
    lib, s = _load(), (_cache(**(cache or {})), _batch(**(batch or {})), _pack(_lib.ATTENTION, _lib.ATTENTION_FIELDS, a))
    return lib.df11_tree_attention_workspace(*s) if entry == "size" else lib.df11_tree_attention(*s, ws, nbytes, None)


BAD_ATTENTION = [
    dict(q=None), dict(out=None), dict(q=D + 8), dict(out=E + 2), dict(q_stride=257), dict(q_head_stride=4),
    dict(out_stride=260), dict(out_head_stride=1 << 40), dict(q_stride=1 << 40), dict(q_heads=0), dict(q_heads=3),
    dict(q_heads=4098), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")),
    dict(out_stride=248), dict(out_head_stride=56), dict(lse=F + 2), dict(mask=G, mask_stride=1 << 40),
]


@pytest.mark.parametrize("bad", BAD_ATTENTION)
def test_attention_refuses(bad):
    assert _attend(**bad) == INVALID
    assert _attend(entry="size", **bad) == 0


@pytest.mark.parametrize("bad", [
    dict(out=A), dict(out=B + 64), dict(out=C), dict(out=D + 16), dict(out=D, out_stride=512), dict(lse=A), dict(lse=D),
    dict(lse=E), dict(lse=C + 0x2000), dict(mask=E, mask_cols=4, mask_stride=4), dict(lse=G, mask=G, mask_cols=9, mask_stride=9),
])
def test_attention_refuses_overlaps(bad):
    assert _attend(**bad) == INVALID


def test_attention_takes_nothing():
    for batch in (dict(tokens=0), dict(seqs=0, lengths=None, table=None)):
        assert _attend(batch=batch) == 0
        assert _attend(batch=batch, q=None, out=None, ws=None, nbytes=0) == 0
        assert _attend(batch=batch, entry="size") == 0
    lib = _load()
    assert lib.df11_tree_attention(None, _batch(), _pack(_lib.ATTENTION, _lib.ATTENTION_FIELDS, {}), None, 0, None) == INVALID
    assert lib.df11_tree_attention(_cache(), _batch(), None, None, 0, None) == INVALID


def test_strides_of_one_element_are_not_used():
    """Whatever they are: one page of one place, one token, one head."""
    one = dict(n=1, page=1, heads=1, kp=3, kl=5, kh=1 << 50, vp=1, vl=7, vh=9)
    few = dict(tokens=1)
    assert _append(cache=one, batch=few, k_stride=1 << 45, k_head_stride=1 << 40, v_stride=3, k=1) == INVALID  # (k itself)
    assert _append(cache=one, batch=dict(tokens=0), k_stride=1 << 45, k_head_stride=1 << 40, v_stride=3) == 0
    assert _attend(cache=one, batch=dict(few, seqs=0), q_stride=3, out_stride=5, q_heads=1, q_head_stride=1, out_head_stride=3) == 0


def _layout(name, fields):
    """Offsets and size of a struct of the header, by the C compiler."""
    import subprocess
    import tempfile
    repo = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with tempfile.TemporaryDirectory() as d:
        src = os.path.join(d, "s.c")
        with open(src, "w") as f:
            f.write('#include <stddef.h>\n#include <stdio.h>\n#include "df11.h"\nint main(void) {\n')
            for n in fields:
                f.write(f'    printf("%zu ", offsetof({name}, {n}));\n')
            f.write(f'    printf("%zu\\n", sizeof({name}));\n    return 0;\n}}\n')
        subprocess.run(["gcc", f"-I{os.path.join(repo, 'include')}", src, "-o", os.path.join(d, "s")], check=True)
        return [int(v) for v in subprocess.run([os.path.join(d, "s")], capture_output=True, text=True,
                                               check=True).stdout.split()]


@pytest.mark.parametrize("name,format,fields", [
    ("df11_kv_cache", "KV_CACHE", "KV_CACHE_FIELDS"), ("df11_kv_batch", "KV_BATCH", "KV_BATCH_FIELDS"),
    ("df11_append", "APPEND", "APPEND_FIELDS"), ("df11_attention", "ATTENTION", "ATTENTION_FIELDS")])
def test_packed_structures(name, format, fields):
    import struct
    format, fields = getattr(_lib, format), getattr(_lib, fields)
    *offsets, size = _layout(name, fields)
    assert size == format.size
    kinds = []
    for n, c in __import__("re").findall(r"(\d*)([QIf])", format.format):
        kinds += [c] * int(n or 1)
    at = 0
    for offset, kind in zip(offsets, kinds):
        assert offset == at
        at += struct.calcsize("=" + kind)
    assert len(kinds) == len(fields) and at == size


def test_loss_structure():
    fields = [n for n, _ in _lib.Loss._fields_]
    *offsets, size = _layout("df11_loss", fields)
    assert [getattr(_lib.Loss, n).offset for n in fields] == offsets and ctypes.sizeof(_lib.Loss) == size


def test_cache_binding_refuses():
    import torch
    from entropy_decoding_df11_amd import df11
    kc = torch.zeros(8, 16, 2, 64, dtype=torch.bfloat16)
    q, x = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    table, starts, lengths = torch.zeros(3, 4).int(), torch.zeros(4).int(), torch.zeros(3).int()
    good = dict(k_cache=kc, v_cache=kc.clone(), page_table=table, starts=starts, lengths=lengths)
    both = [dict(k_cache=kc.float()), dict(v_cache=kc.half()), dict(v_cache=kc[:7]), dict(k_cache=kc[0]),
            dict(k_cache=kc[..., :60], v_cache=kc[..., :60]), dict(k_cache=kc[:0], v_cache=kc[:0]),
            dict(k_cache=kc.transpose(2, 3), v_cache=kc.transpose(2, 3)), dict(page_table=table.long()),
            dict(page_table=table[:2]), dict(page_table=table.t()), dict(starts=starts[:3]), dict(starts=starts.long()),
            dict(lengths=lengths.float()), dict(lengths=torch.zeros(6).int()[::2]), dict(page_table=table[0]),
            dict(starts=torch.zeros(4, device="meta").int())]
    for bad in both + [dict(k=x[0]), dict(k=x.double()), dict(v=x.float()), dict(v=x[:4]), dict(k=x[..., :32]),
                       dict(k=q, v=q), dict(q=q.half()), dict(q=q[:4]), dict(q=q[:, :0]), dict(q_out=q),
                       dict(q=q, q_out=q.half()), dict(q=q, q_out=q[:4]), dict(rotary=torch.zeros(9, 64).half()),
                       dict(rotary=torch.zeros(9, 63)), dict(rotary=torch.zeros(9, 66)), dict(rotary=torch.zeros(0, 64)),
                       dict(rotary=torch.zeros(64)), dict(rotary=torch.zeros(64, 9).t()),
                       dict(positions=torch.zeros(5)), dict(positions=torch.zeros(4).int()),
                       dict(positions=torch.zeros(10).int()[::2]), dict(k=x.float().requires_grad_(), v=x.float()),
                       dict(k=x.transpose(1, 2).contiguous().transpose(1, 2))]:
        with pytest.raises(ValueError):
            df11.append_kv(**(dict(good, k=x, v=x) | bad))
    for bad in both + [dict(q=q.half()), dict(q=q[0]), dict(q=q[:, :3]), dict(q=q[:, :0]), dict(q=q[..., :32]),
                       dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                       dict(mask=torch.zeros(5, 4)), dict(mask=torch.zeros(4, 4).bool()), dict(mask=torch.zeros(5).bool()),
                       dict(mask=torch.zeros(4, 5).bool().t()), dict(out=q[:4]), dict(out=q.half()),
                       dict(q=q.clone().requires_grad_()), dict(q=q.clone().requires_grad_(), out=q)]:
        with pytest.raises(ValueError):
            df11.tree_attention(**(dict(good, q=q) | bad))
    for call in (lambda: df11.append_kv(x, x, **good), lambda: df11.tree_attention(q, **good)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for bad in ((-1, 64), (10, 0), (10, 7)):
        with pytest.raises(ValueError):
            df11.rotary_table(*bad, device="cpu")


def _stream(rows=128, cols=64, at=0x2000000000, tile=True):
    """A device stream whose header is sound and whose addresses are never read."""
    import numpy as np
    from entropy_decoding_df11_amd import df11, workloads
    w = workloads.f32_to_bf16_bits(np.random.default_rng(0).standard_normal(rows * cols) * 0.02)
    s = _lib.DeviceStream()
    s.h = df11.encode(w).header
    for i, name in enumerate(("enc", "sm", "gaps", "out_pos", "luts", "code_lengths", "decode_table")):
        setattr(s, name, at + i * 0x1000000)
    s.decode_table_bits = 11
    s.tile_cols = cols if tile else 0
    return s


def _loss(w="sound", x=A, xs=64, t=40, inf=64, outf=128, ws=J, nbytes=1 << 40, given=True, **k):
    lib = _load()
    a = dict(targets=B, loss=C, vocab=128, ignore_index=-100)
    a.update(k)
    w = _stream() if w == "sound" else w
    return lib.df11_cross_entropy(None if w is None else ctypes.byref(w), x, xs, t, inf, outf,
                                  ctypes.byref(_lib.Loss(**a)) if given else None, ws, nbytes, None)


@pytest.mark.parametrize("bad", [
    dict(w=None), dict(inf=32), dict(outf=64), dict(inf=60), dict(outf=0), dict(given=False), dict(vocab=0),
    dict(vocab=129), dict(mean=2), dict(x=None), dict(x=A + 8), dict(xs=60), dict(xs=(1 << 22) + 8), dict(targets=None),
    dict(targets=B + 4), dict(loss=None), dict(loss=C + 2), dict(total=D + 2), dict(count=D + 1), dict(grad=E + 8),
    dict(loss=A), dict(loss=B), dict(total=C), dict(total=D, count=D), dict(grad=A), dict(grad=B), dict(grad=C),
    dict(grad=D, total=D + 64), dict(loss=0x2000000000), dict(grad=0x2000000000), dict(count=0x2001000000),
])
def test_loss_refuses(bad):
    assert _loss(**bad) == INVALID


def test_loss_refuses_sizes():
    assert _loss(w=_stream(tile=False)) == INVALID
    assert _loss(t=1 << 26) == TOO_LARGE
    lib = _load()
    s = _stream()
    assert lib.df11_cross_entropy_workspace(None, 4, 0) == 0
    assert lib.df11_cross_entropy_workspace(s, 0, 1) == 0
    assert lib.df11_cross_entropy_workspace(_stream(tile=False), 4, 1) == 0
    assert lib.df11_cross_entropy_workspace(s, 1 << 26, 0) == 0


def _loss_grad(**k):
    a = dict(grad=A, dy=B, dys=1, count=None, t=4, inf=64, dx=C, dxs=64, dt=0)
    a.update(k)
    return _load().df11_cross_entropy_grad(a["grad"], a["dy"], a["dys"], a["count"], a["t"], a["inf"], a["dx"], a["dxs"],
                                           a["dt"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(dt=1), INVALID), (dict(dt=9), INVALID), (dict(inf=0), INVALID), (dict(inf=40), INVALID),
    (dict(inf=1 << 23), TOO_LARGE), (dict(t=1 << 26), TOO_LARGE), (dict(grad=None), INVALID), (dict(grad=A + 4), INVALID),
    (dict(dy=None), INVALID), (dict(dy=B + 1), INVALID), (dict(dys=1 << 32), INVALID), (dict(dx=None), INVALID),
    (dict(dx=C + 1), INVALID), (dict(dxs=60), INVALID), (dict(dxs=1 << 32), INVALID), (dict(count=D + 2), INVALID),
    (dict(dx=A), INVALID), (dict(dx=B), INVALID), (dict(dx=D, count=D), INVALID),
])
def test_loss_grad_refuses(bad, status):
    assert _loss_grad(**bad) == status


def test_loss_grad_takes_no_tokens():
    assert _loss_grad(t=0) == 0
    assert _loss_grad(t=0, grad=None, dy=None, dx=None) == 0


def test_loss_binding_refuses():
    import types

    import torch
    from entropy_decoding_df11_amd import df11
    head = lambda **k: types.SimpleNamespace(**{"shape": (128, 64), "tile_cols": 64,  # noqa: E731
                                                "_bufs": {"enc": torch.zeros(1)}, **k})
    x, t = torch.zeros(5, 64, dtype=torch.bfloat16), torch.zeros(5, dtype=torch.int64)
    for bad in (dict(w=head(tile_cols=0)), dict(w=head(shape=(128,))), dict(w=head(shape=(0, 64))), dict(x=x.float()),
                dict(x=x[:, :32]), dict(x=torch.zeros((), dtype=torch.bfloat16)), dict(targets=t.int()),
                dict(targets=t[:4]), dict(targets=t[:, None]), dict(vocab=0), dict(vocab=129), dict(reduction="average"),
                dict(targets=t.to("meta")), dict(x=torch.zeros(1, 64, dtype=torch.bfloat16).expand(1 << 26, 64),
                                                 targets=t[:1].expand(1 << 26))):
        with pytest.raises(ValueError):
            df11.linear_cross_entropy(**(dict(w=head(), x=x, targets=t) | bad))
    with pytest.raises(ValueError, match="GPU"):
        df11.linear_cross_entropy(head(), x, t)
