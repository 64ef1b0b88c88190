"""The paged cache's operators against plain implementations in 64 bits: keys and
values appended with the rotation on the way, and attention of new tokens over
the cache.

Tolerances.  u = eps / 2 of the type is the most that a rounding is off, e =
2^-24 that of float32.  An append rounds once, from float32 products of two
terms: 4 e of the terms and u of the result.  Attention: a score of D products
is off by at most d = scale (D + 4) e sum |q k|, and so is its place in the
exponent, twice with the row's largest, 8 e |scale s| more for the change of
base; the exponential itself 4 e; the weights are rounded to the cache's type, u,
and the sums over n places lose n e.  All of it reaches an output in proportion
to sum p |v|, and the output is rounded once more."""

import math
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from entropy_decoding_df11_amd import df11  # noqa: E402

E = 2.0 ** -24
DEV = "cuda:0"


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Case:
    """A cache with random pages, every place that no sequence holds filled with NaN, and a batch."""

    def __init__(self, lengths, tokens, dtype=torch.bfloat16, heads=4, kv_heads=2, dim=64, page=16, seed=0, first=0,
                 spare=0, by_head=False):
        g = gen(seed)
        self.lengths_, self.tokens, self.page, self.dim = list(lengths), list(tokens), page, dim
        self.heads, self.kv_heads, self.dtype = heads, kv_heads, dtype
        need = [-(-(a + b) // page) for a, b in zip(lengths, tokens)]
        n_pages = sum(need) + 2
        order = torch.randperm(n_pages, generator=g)
        width = max(need, default=0)
        table, at = torch.zeros(len(need), width, dtype=torch.int32), 0
        for s, n in enumerate(need):
            table[s, :n] = order[at:at + n].int()
            at += n
        shape = (n_pages, kv_heads, page, dim) if by_head else (n_pages, page, kv_heads, dim)
        self.k = torch.full(shape, math.nan, dtype=dtype)
        self.v = torch.full(shape, math.nan, dtype=dtype)
        if by_head:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        for s, (a, b) in enumerate(zip(lengths, tokens)):
            p = torch.arange(a + b)
            for half in (self.k, self.v):
                half[table[s].long()[p // page], p % page] = torch.randn(a + b, kv_heads, dim, generator=g).to(dtype)
        starts = [first]
        for b in tokens:
            starts.append(starts[-1] + b)
        self.total = starts[-1] + spare
        self.q = (1.5 * torch.randn(self.total, heads, dim, generator=g)).to(dtype)
        self.table, self.starts = table, starts
        self.upload()

    def upload(self):
        self.dk, self.dv = self.on_gpu(self.k), self.on_gpu(self.v)
        self.batch = (self.table.to(DEV), torch.tensor(self.starts, dtype=torch.int32, device=DEV),
                      torch.tensor(self.lengths_, dtype=torch.int32, device=DEV))

    @staticmethod
    def on_gpu(t):
        """A copy with t's strides."""
        if t.is_contiguous():
            return t.to(DEV)
        return t.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)

    def attend(self, q=None, **more):
        return df11.tree_attention(self.q.to(DEV) if q is None else q, self.dk, self.dv, *self.batch, **more)

    def seen(self, s, mask):
        a, b = self.lengths_[s], self.tokens[s]
        out = torch.ones(b, a + b, dtype=torch.bool)
        if mask is None:
            out[:, a:] = torch.ones(b, b, dtype=torch.bool).tril()
        else:
            out[:, a:] = False
            w = min(b, mask.shape[1])
            out[:, a:a + w] = mask[self.starts[s]:self.starts[s] + b, :w] != 0
        return out

    def expect(self, mask=None, scale=None):
        """(out, its tolerance, lse, its tolerance) of every row in 64 bits; rows of no sequence zero."""
        scale = self.dim ** -0.5 if scale is None else scale
        u, group = half_step(self.dtype), self.heads // self.kv_heads
        o = torch.zeros(self.total, self.heads, self.dim, dtype=torch.float64)
        tol, lse, lse_tol = torch.zeros_like(o), torch.zeros(self.total, self.heads, dtype=torch.float64), \
            torch.zeros(self.total, self.heads, dtype=torch.float64)
        for s, (a, b) in enumerate(zip(self.lengths_, self.tokens)):
            if not b:
                continue
            p = torch.arange(a + b)
            pages = self.table[s].long()[p // self.page]
            rows = slice(self.starts[s], self.starts[s] + b)
            seen = self.seen(s, mask)
            for h in range(self.heads):
                k = self.k[pages, p % self.page, h // group].double()
                v = self.v[pages, p % self.page, h // group].double()
                q = self.q[rows, h].double()
                z = torch.where(seen, scale * (q @ k.nan_to_num(0, 0, 0).t()), -math.inf)
                d = scale * (self.dim + 4) * E * (q.abs() @ k.nan_to_num(0, 0, 0).abs().t())
                d = torch.where(seen, d + 8 * E * z.abs().nan_to_num(0, 0, 0), 0).amax(1, keepdim=True)
                top = z.amax(1, keepdim=True).clamp(min=-1e300)
                w = (z - top).exp()
                total = w.sum(1, keepdim=True)
                pr = torch.where(total > 0, w / total, 0)
                o[rows, h] = pr @ v.nan_to_num(0, 0, 0)
                each = 2 * d + 8 * E + (a + b) * E
                tol[rows, h] = 1.01 * ((u + each) * (pr @ v.nan_to_num(0, 0, 0).abs()) + u * o[rows, h].abs()) + 1e-30
                lse[rows, h] = (total.log() + top.where(total > 0, torch.tensor(-math.inf, dtype=torch.float64)))[:, 0]
                lse_tol[rows, h] = (each[:, 0] + 4 * E * lse[rows, h].abs().nan_to_num(0, 0, 0)) * 1.01
        return o, tol, lse, lse_tol

    def check(self, mask=None, scale=None, **more):
        """Runs the case with guarded rows and compares it."""
        g = gen(99)
        out = torch.randn(self.q.shape, generator=g).to(self.dtype).to(DEV)
        before = out.clone()
        got, lse = self.attend(mask=None if mask is None else mask.to(DEV), scale=scale, out=out, return_lse=True, **more)
        torch.cuda.synchronize()
        assert got is out
        o, tol, want_lse, lse_tol = self.expect(mask, scale)
        rows = slice(self.starts[0], self.starts[-1])
        far = (out.cpu().double() - o).abs()[rows]
        assert bool((far <= tol[rows]).all()), f"off by {(far / tol[rows]).max():.3g} tolerances"
        lse = lse.cpu().double()[rows]
        empty = want_lse[rows] == -math.inf
        assert torch.equal(lse == -math.inf, empty)
        assert bool(((lse - want_lse[rows]).abs()[~empty] <= lse_tol[rows][~empty]).all())
        for part in (slice(0, self.starts[0]), slice(self.starts[-1], None)):
            assert torch.equal(out[part], before[part])
        return out


def tree(case, seed=0, width=None):
    """A random tree's mask for every sequence of the case."""
    g = gen(seed)
    width = max(case.tokens) if width is None else width
    mask = torch.zeros(case.total, width, dtype=torch.bool)
    for s, n in enumerate(case.tokens):
        rows = torch.zeros(n, width, dtype=torch.bool)
        for i in range(n):
            parent = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
            if parent >= 0:
                rows[i] = rows[parent]
            if i < width:
                rows[i, i] = True
        mask[case.starts[s]:case.starts[s] + n] = rows
    return mask


SHAPES = [(1, 1, 64), (4, 2, 64), (8, 1, 128), (7, 1, 80), (6, 2, 96), (5, 5, 8), (16, 2, 256), (3, 1, 136)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads,kv_heads,dim", SHAPES)
def test_decode(dtype, heads, kv_heads, dim):
    """One token after none, one, and up to a few steps of cached places."""
    Case([0, 1, 31, 32, 127, 128, 300, 1000], [1] * 8, dtype, heads, kv_heads, dim).check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page", [1, 3, 16, 24, 40, 128, 1000])
def test_page_sizes(dtype, page):
    Case([5, 90, 257, 0], [3, 1, 17, 40], dtype, 4, 2, 64, page, seed=1).check()


@pytest.mark.parametrize("heads,kv_heads,dim", SHAPES)
@pytest.mark.parametrize("tokens", [[2, 7, 1], [33, 64, 5], [130, 0, 71]])
def test_prompt_pieces(heads, kv_heads, dim, tokens):
    Case([0, 200, 77], tokens, torch.bfloat16, heads, kv_heads, dim, seed=2).check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads,kv_heads,dim", SHAPES)
def test_trees(dtype, heads, kv_heads, dim):
    case = Case([0, 130, 515], [24, 61, 1], dtype, heads, kv_heads, dim, seed=3)
    case.check(mask=tree(case))


@pytest.mark.parametrize("page", [7, 16])
def test_long_context(page):
    """Tiles that many workgroups share, and a reference that moves."""
    case = Case([20000, 3000], [1, 9], torch.bfloat16, 8, 2, 128, page, seed=4)
    # scores that grow along the places
    for s, a in enumerate(case.lengths_):
        p = torch.arange(a)
        at = case.table[s].long()[p // page], p % page
        case.k[at] = (case.k[at].float() * (0.2 + 3 * p / a)[:, None, None]).to(case.dtype)
    case.upload()
    case.check()


@pytest.mark.parametrize("scale", [0.003, 1.0, 30.0])
def test_scales(scale):
    case = Case([64, 300], [5, 40], torch.bfloat16, 4, 2, 64, seed=5)
    case.check(scale=scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rows_that_see_nothing(dtype):
    case = Case([0, 0, 40], [5, 1, 3], dtype, 4, 2, 64, seed=6)
    mask = tree(case)
    mask[1] = False
    mask[5] = False
    mask[6] = False  # (its cached places stay)
    out = case.check(mask=mask)
    assert bool((out[1] == 0).all()) and bool((out[5] == 0).all())


def test_mask_columns():
    """Fewer columns than new tokens, more of them, bytes other than one, rows apart."""
    case = Case([3, 50], [9, 20], torch.bfloat16, 4, 2, 64, seed=7)
    case.check(mask=tree(case, width=6))
    case.check(mask=tree(case, width=31))
    case.check(mask=tree(case).to(torch.uint8) * 2)
    wide = torch.zeros(case.total, 64, dtype=torch.bool)
    wide[:, :20] = tree(case)
    mask = wide.to(DEV)[:, :20]
    o, tol, _, _ = case.expect(wide[:, :20])
    got = case.attend(mask=mask).cpu().double()
    assert bool(((got - o).abs() <= tol).all())


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128])
def test_values_of_places_that_a_row_does_not_see(dtype, value, dim):
    """A drafted token with infinities or NaN reaches its descendants alone."""
    case = Case([37, 0], [20, 40], dtype, 4, 2, dim, seed=8)
    mask = tree(case)
    bad = [(0, 4), (1, 7)]
    for s, j in bad:
        p = case.lengths_[s] + j
        at = int(case.table[s, p // case.page]), p % case.page
        case.k[at][..., 3] = value
        case.v[at][..., 5] = value
    case.upload()
    out = case.attend(mask=mask.to(DEV)).cpu().double()
    o, tol, _, _ = case.expect(mask)
    touched = torch.zeros(case.total, dtype=torch.bool)
    for s, j in bad:
        rows = slice(case.starts[s], case.starts[s + 1])
        touched[rows] = mask[rows, j]
    assert bool(touched.any()) and not bool(touched.all())
    assert bool(((out - o).abs()[~touched] <= tol[~touched]).all())
    assert not bool(out[touched][..., 5].isfinite().any()) or not math.isnan(value)


def test_lowest_keys():
    """Keys of the type's lowest value: scores of float32's range, sums still of the others."""
    case = Case([40], [4], torch.bfloat16, 2, 1, 64, seed=9)
    p = torch.arange(0, 40, 3)
    at = case.table[0].long()[p // case.page], p % case.page
    case.k[at] = torch.finfo(torch.bfloat16).min
    case.q = case.q.abs()  # every such score is -inf or nearly
    case.upload()
    out = case.attend().cpu().double()
    assert bool(out.isfinite().all())
    for half in (case.k, case.v):
        half[at] = 0
    keep = torch.ones(44, dtype=torch.bool)
    keep[p] = False
    z = torch.where(case.seen(0, None) & keep, 0.125 * torch.einsum(
        "qhd,kd->hqk", case.q.double(), case.k[case.table[0].long()[torch.arange(44) // 16], torch.arange(44) % 16, 0].double()),
        -math.inf)
    v = case.v[case.table[0].long()[torch.arange(44) // 16], torch.arange(44) % 16, 0].double()
    want = (z.softmax(2) @ v).transpose(0, 1)
    assert bool(((out - want).abs() <= 2.0 ** -6 * (z.softmax(2) @ v.abs()).transpose(0, 1)).all())


@pytest.mark.parametrize("page", [5, 16])
def test_pages_that_do_not_exist(page):
    """Places in them are not seen, read or counted, and neither are places beyond the table."""
    case = Case([70, 20], [3, 2], torch.bfloat16, 4, 2, 64, page, seed=10)
    table = case.table.clone()
    lost = [1, 3]
    for j, bad in zip(lost, (-1, case.k.shape[0])):
        table[0, j] = bad
    kept = torch.tensor([p // page not in lost for p in range(73)])
    case.batch = (table.to(DEV), *case.batch[1:])
    out = case.attend().cpu().double()
    u = half_step(case.dtype)
    p = torch.arange(73)
    pages = case.table[0].long()[p // page]
    for h in range(4):
        k, v = (half[pages, p % page, h // 2].double() for half in (case.k, case.v))
        z = torch.where(case.seen(0, None) & kept, 0.125 * case.q[:3, h].double() @ k.t(), -math.inf)
        far = (out[:3, h] - z.softmax(1) @ v).abs()
        assert bool((far <= 2.1 * u * (z.softmax(1) @ v.abs())).all())
    o, tol, _, _ = case.expect()
    assert bool(((out - o).abs()[3:] <= tol[3:]).all())
    # a table that ends before the sequence does
    short = Case([70], [3], torch.bfloat16, 4, 2, 64, page, seed=11)
    width = 70 // page
    short.batch = (short.table[:, :width].contiguous().to(DEV), *short.batch[1:])
    got = short.attend().cpu().double()
    p = torch.arange(width * page)
    pages = short.table[0].long()[p // page]
    for h in range(4):
        k, v = (half[pages, p % page, h // 2].double() for half in (short.k, short.v))
        z = 0.125 * short.q[:, h].double() @ k.t()
        z = torch.where(short.seen(0, None)[:, :width * page], z, -math.inf)
        assert bool(((got[:, h] - z.softmax(1) @ v).abs() <= 2.1 * u * (z.softmax(1) @ v.abs())).all())


def test_rows_of_no_sequence():
    case = Case([9, 40, 3], [2, 0, 5], torch.bfloat16, 4, 2, 64, first=3, spare=4)
    case.check()
    case = Case([9, 40, 3], [2, 0, 35], torch.bfloat16, 4, 2, 64, first=3, spare=4)
    case.check(mask=tree(case))


def test_strides():
    """Queries that are a part of a fused product's rows, heads apart, outputs between others, pages by head."""
    case = Case([33, 260], [5, 1], torch.bfloat16, 4, 2, 64, by_head=True, seed=12)
    case.check()
    fused = torch.zeros(case.total, 4 * 64 + 128 + 8, dtype=case.dtype, device=DEV)
    q = fused[:, 8:8 + 256].view(case.total, 4, 64)
    q.copy_(case.q)
    by_head = torch.empty(4, case.total, 64, dtype=case.dtype, device=DEV).transpose(0, 1)
    by_head.copy_(case.q)
    plain = case.attend()
    assert torch.equal(case.attend(q=q), plain) and torch.equal(case.attend(q=by_head), plain)
    out = torch.full((case.total, 7, 80), 5.0, dtype=case.dtype, device=DEV)
    case.attend(out=out[:, 1:5, 8:72])
    assert torch.equal(out[:, 1:5, 8:72], plain)
    out[:, 1:5, 8:72] = 5
    assert bool((out == 5).all())
    on_q = case.q.to(DEV)
    case.attend(q=on_q, out=on_q)
    assert torch.equal(on_q, plain)


def test_nothing_to_do():
    case = Case([9], [1], torch.bfloat16, 4, 2, 64)
    empty = case.attend(q=case.q[:0].to(DEV))
    assert empty.shape == (0, 4, 64)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    out = torch.full((3, 4, 64), 7.0, dtype=case.dtype, device=DEV)
    df11.tree_attention(case.q[:1].expand(3, 4, 64).to(DEV).contiguous(), case.dk, case.dv, torch.zeros(0, 4, dtype=torch.int32, device=DEV),
                        torch.zeros(1, dtype=torch.int32, device=DEV), none, out=out)
    assert bool((out == 7).all())


def test_many_sequences():
    """More sequences than a workgroup's threads, most of them short."""
    g = gen(13)
    lengths = torch.randint(0, 90, (601,), generator=g).tolist()
    lengths[300] = 5000
    tokens = torch.randint(0, 4, (601,), generator=g).tolist()
    Case(lengths, tokens, torch.float16, 2, 1, 64, seed=13).check()


def test_far_pages():
    """Places past 32 bits of bytes and of elements."""
    case = Case([100], [2], torch.bfloat16, 4, 2, 64, seed=14)
    n, stride = case.k.shape[0], (1 << 32) // (case.k.shape[0] - 1) // 8 * 8 + 4096
    halves = []
    for half in (case.k, case.v):
        big = torch.empty(stride * n, dtype=case.dtype, device=DEV)
        far = big.as_strided((n, 16, 2, 64), (stride, 128, 64, 1))
        far.copy_(half)
        halves.append(far)
    got = df11.tree_attention(case.q.to(DEV), *halves, *case.batch)
    assert torch.equal(got, case.attend())


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [(4, 2, 64, 16), (4, 2, 64, 9), (7, 1, 80, 16), (6, 2, 96, 24),
                                                      (3, 1, 136, 5), (4, 2, 256, 16), (4, 2, 256, 11)])
def test_cut_tiles(heads, kv_heads, dim, page, masked):
    """Tiles of many rows that many workgroups share, of every padded width, with pages of whole and of odd loads."""
    case = Case([7000, 1500, 0], [70, 1, 33], torch.float16, heads, kv_heads, dim, page, seed=31, first=2, spare=3)
    case.check(mask=tree(case, seed=31) if masked else None)


def test_shared_pages():
    """Two sequences with one prefix: the same pages in both tables."""
    case = Case([320, 330], [3, 20], torch.bfloat16, 8, 2, 128, seed=32)
    case.table[1, :20] = case.table[0, :20]
    case.upload()
    case.check()


@pytest.mark.parametrize("tokens", [[1, 2], [40, 3]])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_queries_that_are_not_finite(tokens, value):
    """They spoil their own rows only."""
    case = Case([2000, 90], tokens, torch.bfloat16, 4, 2, 64, seed=33)
    q = case.q.clone()
    q[0, 1, 5] = value
    out, lse = case.attend(q=q.to(DEV), return_lse=True)
    o, tol, want, lse_tol = case.expect()
    others = torch.ones(case.total, case.heads, dtype=torch.bool)
    others[0, 1] = False
    assert bool(((out.cpu().double() - o).abs() <= tol)[others].all())
    assert bool(((lse.cpu().double() - want).abs() <= lse_tol)[others].all())
    assert bool(out[0, 1].isnan().all()) and bool(lse[0, 1].isnan())


def test_far_pages_of_many_rows():
    case = Case([100], [40], torch.bfloat16, 4, 2, 64, seed=34)
    n, stride = case.k.shape[0], (1 << 32) // (case.k.shape[0] - 1) // 8 * 8 + 4096
    halves = []
    for half in (case.k, case.v):
        big = torch.empty(stride * n, dtype=case.dtype, device=DEV)
        far = big.as_strided((n, 16, 2, 64), (stride, 128, 64, 1))
        far.copy_(half)
        halves.append(far)
    got = df11.tree_attention(case.q.to(DEV), *halves, *case.batch)
    assert torch.equal(got, case.attend())


def test_threads():
    """Calls from threads at once, each on a stream of its own."""
    cases = [Case([4000, 17], [1, 5 + 30 * s], torch.bfloat16, 8, 2, 128, seed=35 + s) for s in range(3)]
    qs = [c.q.to(DEV) for c in cases]
    want = [c.attend(q=q) for c, q in zip(cases, qs)]
    torch.cuda.synchronize()
    got = [[] for _ in cases]

    def work(i):
        stream = torch.cuda.Stream()
        for _ in range(5):
            got[i].append(cases[i].attend(q=qs[i], stream=stream))
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for outs, w in zip(got, want):
        assert len(outs) == 5 and all(torch.equal(o, w) for o in outs)


def test_same_bits_again():
    case = Case([3000, 17, 900], [1, 30, 7], torch.bfloat16, 8, 2, 128, seed=15)
    mask = tree(case).to(DEV)
    first = case.attend(mask=mask, return_lse=True)
    for _ in range(3):
        again = case.attend(mask=mask, return_lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ---------------------------------------------------------------------------
# Append.
# ---------------------------------------------------------------------------

def rotate(x, table, interleaved):
    """(values, sum of the terms' magnitudes) of x (tokens, heads, dim) rotated by table's rows, in 64 bits."""
    half = table.shape[1] // 2
    cos, sin = table[:, None, :half].double(), table[:, None, half:].double()
    out, size = x.double().clone(), x.double().abs()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    va, vb = x.double()[..., a], x.double()[..., b]
    out[..., a], out[..., b] = va * cos - vb * sin, vb * cos + va * sin
    size[..., a] = (va * cos).abs() + (vb * sin).abs()
    size[..., b] = (vb * cos).abs() + (va * sin).abs()
    return out, size


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,dims", [(64, 64), (128, 64), (80, 80), (96, 36), (8, 2), (256, 256), (64, 0)])
@pytest.mark.parametrize("source", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_append(dtype, source, dim, dims, interleaved):
    case = Case([0, 37, 5, 200], [3, 1, 0, 20], dtype, 6, 2, dim, page=24, seed=16, first=2, spare=3)
    g = gen(17)
    q = torch.randn(case.total, 6, dim, generator=g).to(source)
    k, v = (torch.randn(case.total, 2, dim, generator=g).to(source) for _ in range(2))
    table = df11.rotary_table(400, dims, 500000.0, device="cpu") if dims else None
    positions = torch.randint(0, 400, (case.total,), generator=g).int() if interleaved else None
    q_out = torch.full(q.shape, 3.0, dtype=dtype, device=DEV)
    got = df11.append_kv(k.to(DEV), v.to(DEV), case.dk, case.dv, *case.batch, q=q.to(DEV),
                         rotary=None if table is None else table.to(DEV),
                         positions=None if positions is None else positions.to(DEV), interleaved=interleaved, q_out=q_out)
    assert got is q_out
    got, new_k, new_v = got.cpu(), case.dk.cpu(), case.dv.cpu()
    u = half_step(dtype)
    mine = torch.zeros(case.k.shape[:2], dtype=torch.bool)
    for s, (a, b) in enumerate(zip(case.lengths_, case.tokens)):
        rows, place = slice(case.starts[s], case.starts[s] + b), torch.arange(a, a + b)
        at = case.table[s].long()[place // 24], place % 24
        mine[at] = True
        where = place if positions is None else positions[rows].long()
        for name, x, y in (("q", q[rows], got[rows]), ("k", k[rows], new_k[at])):
            want, size = rotate(x, table[where], interleaved) if dims else (x.double(), 0 * x.double())
            assert bool(((y.double() - want).abs() <= 4 * E * size + u * want.abs() * 1.01 + 2.0 ** -24).all()), name
        assert torch.equal(new_v[at], v[rows].to(dtype))
    for new, old in ((new_k, case.k), (new_v, case.v)):  # the rest of the cache, NaN included
        assert torch.equal(new[~mine].view(torch.int16), old[~mine].view(torch.int16))
    assert bool((got[:2] == 3).all()) and bool((got[case.starts[-1]:] == 3).all())


def test_append_strides():
    """Parts of a fused product's rows, odd strides, pages by head, in place, halves of one tensor."""
    dtype = torch.bfloat16
    plain = Case([5, 60], [4, 2], dtype, 4, 2, 64, seed=18)
    g = gen(19)
    for width, at in ((4 * 64 + 2 * 128, 0), (4 * 64 + 2 * 128 + 5, 3)):
        fused = torch.randn(6, width, generator=g).to(dtype).to(DEV)
        q, k, v = (fused[:, at + i:at + j].unflatten(1, (-1, 64)) for i, j in ((0, 256), (256, 384), (384, 512)))
        table = df11.rotary_table(100, 64, device=DEV)
        results = []
        for by_head in (False, True):
            case = Case([5, 60], [4, 2], dtype, 4, 2, 64, seed=18, by_head=by_head)
            results.append((df11.append_kv(k, v, case.dk, case.dv, *case.batch, q=q, rotary=table), case.dk, case.dv))
        both = torch.full((*plain.k.shape[:1], 2, *plain.k.shape[1:]), math.nan, dtype=dtype, device=DEV)
        both[:, 0], both[:, 1] = plain.k.to(DEV), plain.v.to(DEV)
        contiguous = (t.contiguous() for t in (k, v))
        results.append((df11.append_kv(*contiguous, both[:, 0], both[:, 1], *plain.batch, q=q.contiguous(), rotary=table),
                        both[:, 0], both[:, 1]))
        on_q = q.contiguous()
        df11.append_kv(k, v, plain.dk, plain.dv, *plain.batch, q=on_q, rotary=table, q_out=on_q)
        results.append((on_q, plain.dk, plain.dv))
        for other in results[1:]:
            for a, b in zip(results[0], other):
                assert torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))
        plain.upload()


def test_append_what_does_not_exist():
    """Positions beyond the table give NaN; places beyond the page table or in no page are not written."""
    dtype = torch.bfloat16
    case = Case([30, 14], [4, 4], dtype, 2, 1, 64, seed=20)
    x = torch.randn(8, 1, 64, generator=gen(21)).to(dtype).to(DEV)
    q = torch.randn(8, 2, 64, generator=gen(22)).to(dtype).to(DEV)
    table = case.table.clone()
    table[0, 2] = case.k.shape[0]     # places 32 .. 47 of sequence 0
    table[1, 1] = -5                  # 16 .. of sequence 1
    before = case.dk.clone(), case.dv.clone()
    positions = torch.tensor([0, 99, 100, -1, 5, 6, 2 ** 31 - 1, 7], dtype=torch.int32, device=DEV)
    got = df11.append_kv(x, x, case.dk, case.dv, table.to(DEV), *case.batch[1:], q=q, rotary=df11.rotary_table(100, 64),
                         positions=positions)
    bad = torch.tensor([False, False, True, True, False, False, True, False], device=DEV)
    assert torch.equal(got.isnan().flatten(1).all(1), bad) and torch.equal(got.isnan().flatten(1).any(1), bad)
    changed = (case.dv.view(torch.int16) != before[1].view(torch.int16)).flatten(2).any(2).nonzero().tolist()
    want = sorted([int(case.table[0, 1]), p] for p in (14, 15)) + [[int(case.table[1, 0]), p] for p in (14, 15)]
    assert sorted(changed) == sorted(want)
    # a table that ends before the new tokens do, and no columns at all
    for width in (1, 0):
        case.upload()
        df11.append_kv(x, x, case.dk, case.dv, case.table[:, :width].contiguous().to(DEV), *case.batch[1:])
        changed = (case.dv.view(torch.int16) != case.v.to(DEV).view(torch.int16)).flatten(2).any(2).nonzero().tolist()
        assert sorted(changed) == ([[int(case.table[1, 0]), 14], [int(case.table[1, 0]), 15]] if width else [])


def test_append_far_positions():
    """Angles of far positions, from a table in 64 bits."""
    table = df11.rotary_table(1 << 20, 64, 10000.0)
    p = (1 << 20) - 1
    angle = p * 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    assert bool(((table[p].cpu().double() - torch.cat([angle.cos(), angle.sin()])).abs() <= 2 * E + p * 2.0 ** -51).all())


# ---------------------------------------------------------------------------
# Both, as a step uses them.
# ---------------------------------------------------------------------------

def test_append_then_attend():
    """What is appended is what is attended to, whether in one go or token by token."""
    dtype = torch.bfloat16
    g = gen(23)
    n, heads, kv_heads, dim = 70, 4, 2, 64
    q, k, v = (torch.randn(n, h, dim, generator=g).to(dtype).to(DEV) for h in (heads, kv_heads, kv_heads))
    table = df11.rotary_table(n, dim)
    pages = torch.randperm(6, generator=g).int().to(DEV)[None, :5]
    outs = []
    for pieces in ([n], [40, 30], [1] * n):
        kc, vc = (torch.full((6, 16, kv_heads, dim), math.nan, dtype=dtype, device=DEV) for _ in range(2))
        at, rows = 0, []
        for m in pieces:
            batch = (pages, torch.tensor([0, m], dtype=torch.int32, device=DEV),
                     torch.tensor([at], dtype=torch.int32, device=DEV))
            part = slice(at, at + m)
            turned = df11.append_kv(k[part], v[part], kc, vc, *batch, q=q[part], rotary=table)
            rows.append(df11.tree_attention(turned, kc, vc, *batch))
            at += m
        outs.append(torch.cat(rows))
    for other in outs[1:]:
        assert bool(((other - outs[0]).abs().float() <= 2.0 ** -6 * (1 + outs[0].abs().float())).all())


def test_captured_step():
    """A step in a graph, replayed with other lengths, pages, starts and masks."""
    case = Case([50, 300, 7], [3, 2, 4], torch.bfloat16, 4, 2, 64, seed=24, spare=2)
    other = Case([280, 20, 90], [2, 4, 3], torch.bfloat16, 4, 2, 64, seed=25, spare=2)
    width = 20
    static = [torch.zeros(3, width, dtype=torch.int32, device=DEV), case.batch[1].clone(), case.batch[2].clone()]
    mask = torch.zeros(case.total, 4, dtype=torch.bool, device=DEV)
    q = torch.zeros_like(case.q).to(DEV)
    pages = max(case.k.shape[0], other.k.shape[0])
    kc, vc = (torch.zeros(pages, 16, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k, v = (torch.zeros(case.total, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table = df11.rotary_table(400, 64)

    def fill(c):
        static[0].zero_()
        static[0][:, :c.table.shape[1]] = c.batch[0]
        static[1].copy_(c.batch[1])
        static[2].copy_(c.batch[2])
        mask.copy_(tree(c, seed=26, width=4))
        q.copy_(c.q)
        kc[:c.k.shape[0]], vc[:c.k.shape[0]] = c.dk, c.dv
        k.copy_(torch.randn(c.total, 2, 64, generator=gen(27)))
        v.copy_(torch.randn(c.total, 2, 64, generator=gen(28)))

    def step():
        turned = df11.append_kv(k, v, kc, vc, *static, q=q, rotary=table)
        return df11.tree_attention(turned, kc, vc, *static, mask=mask)

    fill(case)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for c in (case, other, case, other):
        fill(c)
        rows = slice(c.starts[0], c.starts[-1])
        graph.replay()
        torch.cuda.synchronize()
        got, gk = out[rows].clone(), kc.clone()
        fill(c)
        want = step()[rows]
        assert torch.equal(got, want) and torch.equal(gk.view(torch.int16), kc.view(torch.int16))


def test_streams():
    """Two calls at once, on streams of their own, inputs freed before the streams get to them."""
    a, b = (Case([4000, 17], [1, 40], torch.bfloat16, 8, 2, 128, seed=s) for s in (29, 30))
    want = [c.attend() for c in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        outs = []
        for c, stream in zip((a, b), streams):
            q = c.q.to(DEV)
            stream.wait_stream(torch.cuda.current_stream())
            outs.append(c.attend(q=q, stream=stream))
            del q
            torch.randn(c.q.shape, device=DEV)  # takes a freed input's place, were it free
        torch.cuda.synchronize()
        for got, w in zip(outs, want):
            assert torch.equal(got, w)


def test_versions():
    """Outputs that are given tell autograd that they have changed."""
    case = Case([9], [2], torch.bfloat16, 4, 2, 64)
    out = torch.empty_like(case.q, device=DEV)
    before = out._version, case.dk._version
    case.attend(out=out)
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    df11.append_kv(x, x, case.dk, case.dv, *case.batch)
    assert out._version > before[0] and case.dk._version > before[1]
