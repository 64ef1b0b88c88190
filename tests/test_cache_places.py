"""Which caches append_kv takes for its two halves: those whose places lie apart.  Through
the C ABI, before any launch: what is taken ends with the missing GPU's error, or with
nothing to do."""

import pytest

from test_cache_and_loss_refusals import A, B, D, INVALID, _append, _load  # noqa: F401

ODD = [  # places on each other though every stride passes a head
    dict(kl=64), dict(vl=64), dict(kh=128), dict(kp=128), dict(vp=1024), dict(kp=2040), dict(kl=120, kh=64),
    dict(kp=64, kl=512, kh=8192 - 64), dict(kp=64, vp=64),
    # halves on each other: shifted by pages, by places, within a head's row
    dict(v=A + 2 * 2048), dict(v=A + 2 * 4 * 2048), dict(v=A + 2 * 128), dict(v=A + 2 * 64), dict(v=A + 16),
    dict(v=A + 2 * 2048, kp=4096, vp=4096, kl=256, vl=256),  # (the second half's heads between the first one's pages)
    dict(v=A + 2 * 1024, kp=2048, vp=4096),
]


@pytest.mark.parametrize("bad", ODD)
def test_places_on_each_other(bad):
    assert _append(cache=bad) == INVALID


FINE = [  # (8 pages of 16 places of 2 heads of 64)
    dict(), dict(kp=2048, kl=64, kh=1024, vp=2048, vl=64, vh=1024), dict(kh=1 << 20, kl=64, kp=1024),
    dict(kp=64, kl=8 * 64, kh=16 * 8 * 64), dict(kp=4096), dict(kl=128 + 8, kp=16 * 136),
    # halves of one tensor: (pages, 2, page, heads, dim), (pages, page, 2, heads, dim), (pages, page, heads, 2, dim),
    # (2, pages, ..), every second page, and of either order of places and heads
    dict(v=A + 2 * 2048, kp=4096, vp=4096), dict(v=A + 2 * 128, kp=4096, vp=4096, kl=256, vl=256),
    dict(v=A + 2 * 64, kp=4096, vp=4096, kl=256, vl=256, kh=128, vh=128), dict(v=A + 2 * 8 * 2048),
    dict(v=A - 2 * 2048, kp=4096, vp=4096), dict(v=A + 2 * 2048, kp=4096, vp=4096, kl=64, kh=1024),
    dict(v=A + 2 * (2048 + 4096 * 3), kp=4096, vp=4096),
    # one of each
    dict(n=1, page=1, heads=1, kp=8, kl=8, kh=8, vp=8, vl=8, vh=8), dict(n=1, kp=8, vp=8), dict(page=1, kl=0, vl=0, kp=128, vp=128),
]


@pytest.mark.parametrize("cache", FINE)
def test_places_apart(cache):
    assert _append(cache=cache, batch=dict(tokens=0)) == 0
    import torch
    if not torch.cuda.is_available():  # (a launch would read what is not there)
        assert _append(cache=cache) not in (0, INVALID)
