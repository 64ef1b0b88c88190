"""The softmax cross entropy through a compressed head against its formula in
64 bits.

Tolerances.  E = 2^-24 is half a step of float32, U = 2^-8 of bfloat16.  A logit
of C exact products is off by at most d = (C + 4) E sum |x w|, and so is its
place in an exponent; the exponential adds 4 E, a token's sum over V classes, added
in chains of 8, 6 across lanes and then panel by panel, (V / 64 + 80) E, and
the loss's own terms 8 E (|lse| + |z|).  With D the sum of those for the
largest d among the classes, a loss is off by at most 2 D, and so is u, the
others' logarithm against the target, whose logistic s scales the gradient:
2 D s (sum p |W| + s |W_y|).  The gradient's exponentials are rounded to
bfloat16, U, and their product's sums, of V / 32 steps, lose (V / 32 + 64) E; the
result is rounded once more."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from entropy_decoding_df11_amd import df11  # noqa: E402

E, U = 2.0 ** -24, 2.0 ** -8
DEV = "cuda:0"


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Head:
    """A head of random rows, compressed, and tokens whose states lean towards their targets."""

    def __init__(self, tokens, rows, cols, vocab=None, seed=0, size=1.0, lean=4.0, scale=None):
        g = gen(seed)
        self.vocab = rows if vocab is None else vocab
        w = torch.randn(rows, cols, generator=g) * 0.05
        if scale is not None:
            w = w * scale(torch.arange(rows))[:, None]
        self.w = w.bfloat16()
        self.head = df11.compress(self.w, layout="mfma_tiles")
        self.targets = torch.randint(0, self.vocab, (tokens,), generator=g)
        lean = lean * torch.rand(tokens, 1, generator=g) / (0.0025 * cols)
        x = size * torch.randn(tokens, cols, generator=g) + lean * 0.05 * self.w[self.targets].float() / 0.05
        self.x = x.bfloat16()
        self.targets[::7] = -100
        if tokens:
            self.targets[0] = self.vocab - 1
        self.dx_, self.dt = self.x.to(DEV), self.targets.to(DEV)

    def run(self, **more):
        return df11.linear_cross_entropy(self.head, self.dx_, self.dt, vocab=self.vocab, **more)

    def expect(self, dy=None):
        """(loss, its tolerance, dx for the losses' gradients dy, its tolerance) in 64 bits on the GPU."""
        w, x = self.w.to(DEV)[:self.vocab].double(), self.dx_.double()
        z = x @ w.t()
        scored = self.dt != -100
        target = torch.where(scored, self.dt, 0)[:, None]
        lse = z.logsumexp(1)
        zy = z.gather(1, target)[:, 0]
        p = (z - lse[:, None]).exp()
        d = ((x.shape[1] + 4) * E * (x.abs() @ w.abs().t())).amax(1)
        big = d + 4 * E + (self.vocab / 64 + 80) * E + 8 * E * (lse.abs() + zy.abs())
        # (lse - zy would lose a loss far below one in 64 bits too)
        u = (z - zy[:, None]).scatter(1, target, -math.inf).logsumexp(1)
        exact = u.clamp(min=0) + (-u.abs()).exp().log1p()
        loss, tol = torch.where(scored, exact, 0), torch.where(scored, 2.02 * big, 0)
        if dy is None:
            return loss, tol, None, None
        others = p.scatter(1, target, 0)
        s = others.sum(1, keepdim=True)
        wy, g = w[target[:, 0]], torch.where(scored, dy.to(DEV).double(), 0)[:, None]
        part, size = others @ w, others @ w.abs()
        grad = g * (part - s * wy)
        each = U + (self.vocab / 32 + 64) * E
        far = g.abs() * 1.02 * (each * size + 2 * big[:, None] * (size + s * wy.abs()) + 8 * E * (size + s * wy.abs()))
        return loss, tol, grad, far + U * grad.abs() + 1e-37

    def run_on(self, x, reduction="none"):
        return df11.linear_cross_entropy(self.head, x, self.dt, vocab=self.vocab, reduction=reduction)

    def check(self, reduction="none", seed=1):
        loss, tol, _, _ = self.expect()
        got = self.run(reduction="none")
        assert bool(((got.double() - loss).abs() <= tol).all()), float(((got.double() - loss).abs() / tol).nan_to_num(0).max())
        count = int((self.targets != -100).sum())
        g = torch.rand(self.targets.shape, generator=gen(seed)) + 0.5
        x = self.dx_.clone().requires_grad_()
        out = df11.linear_cross_entropy(self.head, x, self.dt, vocab=self.vocab, reduction=reduction)
        if reduction == "none":
            dy = g
            assert bool(((out.detach().double() - loss).abs() <= tol).all())
            dx, = torch.autograd.grad(out, x, g.to(DEV))
        else:
            f = 1.0 / count if reduction == "mean" else 1.0
            dy = torch.full_like(g, 0.75 * f)
            out_ = out.detach()
            assert abs(float(out_) - float(loss.sum()) * f) <= float(tol.sum()) * f + 2 * E * abs(float(out_))
            assert abs(float(self.run(reduction=reduction)) - float(loss.sum()) * f) <= float(tol.sum()) * f + \
                2 * E * abs(float(out_))
            dx, = torch.autograd.grad(out, x, torch.tensor(0.75, device=DEV))
        _, _, want, far = self.expect(dy)
        off = ((dx.double() - want).abs() / (far + 4 * E * want.abs())).max()
        assert dx.dtype == torch.bfloat16 and float(off) <= 1, float(off)
        assert bool((dx[self.dt == -100] == 0).all())


# one token and one panel, tokens about the fused product's limit, widths of one
# and an odd number of k-steps, padding within the last panel and beyond it, a
# second piece of one panel and of many
SIZES = [(1, 64, 32, None), (3, 128, 64, 100), (31, 640, 96, 601), (32, 4160, 64, 4100), (33, 4160, 160, None),
         (130, 9024, 128, 9000), (257, 256, 256, 129), (64, 20032, 32, 19968)]


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("tokens,rows,cols,vocab", SIZES)
def test_loss_and_gradient(tokens, rows, cols, vocab, reduction):
    Head(tokens, rows, cols, vocab).check(reduction)


def test_many_pieces():
    """More exponentials than a piece holds, also where the second piece moves the references."""
    Head(4100, 33024, 32, 33000, seed=2).check()
    Head(4100, 33024, 32, 33000, seed=2, size=8.0, lean=0.0, scale=lambda v: torch.where(v < 16384, 0.05, 1 + v / 4000)).check()


@pytest.mark.parametrize("tokens", [9, 50])
def test_references_move(tokens):
    """Logits that grow far past what the first pieces had, and others that stay far below."""
    Head(tokens, 4096 * 3, 64, seed=3, size=8.0, lean=0.0, scale=lambda v: torch.where(v < 4096, 0.05, 1.0) * (1 + v / 500)).check()
    Head(tokens, 4096 * 3, 64, seed=4, size=8.0, lean=0.0, scale=lambda v: torch.where(v > 4096, 0.05, 30.0)).check()


@pytest.mark.parametrize("tokens", [9, 50])
def test_certain_targets(tokens):
    """Losses and gradients far below one keep their relative accuracy."""
    head = Head(tokens, 1024, 64, seed=5, lean=0.0)
    head.x = (60 * head.w[torch.where(head.targets < 0, 0, head.targets)].float() / 0.05).bfloat16() / 4
    head.dx_ = head.x.to(DEV)
    loss, _, want, _ = head.expect(torch.ones(tokens))
    assert float(loss[1:7].max()) < 1e-6
    d = float(((64 + 4) * E * (head.dx_.double().abs() @ head.w.to(DEV).double().abs().t())).max())
    got = head.run(reduction="none").double()
    kept = loss > 1e-36
    assert bool(((got - loss).abs()[kept] <= (2.1 * d + 200 * E) * loss[kept]).all())
    x = head.dx_.clone().requires_grad_()
    dx, = torch.autograd.grad(head.run_on(x).sum(), x)
    rows = kept & (head.dt != -100) & (loss > 1e-30)
    size = want.abs().amax(1, keepdim=True)
    assert bool(rows.any()) and bool(((dx.double() - want).abs()[rows] <= 4 * U * size[rows]).all())


def test_one_class():
    head = Head(40, 64, 32, 1, seed=6)
    x = head.dx_.clone().requires_grad_()
    loss = head.run_on(x)
    dx, = torch.autograd.grad(loss.sum(), x)
    assert bool((loss == 0).all()) and bool((dx == 0).all())
    assert bool((head.run(reduction="none")[:3] == 0).all())


@pytest.mark.parametrize("tokens", [12, 60])
def test_targets_that_are_no_class(tokens):
    """Ignored ones are zero, others beyond the vocabulary NaN; so is what an infinity or a NaN in x gives."""
    head = Head(tokens, 192, 64, 150, seed=7)
    want = head.run(reduction="none")
    for t, v in ((1, 150), (2, 191), (3, -1), (4, 2 ** 40), (5, -2 ** 63), (6, 192)):
        head.targets[t] = v
    head.targets[9] = -100
    head.dt = head.targets.to(DEV)
    head.x[8, 3], head.x[10, 5], head.x[9, 1] = math.inf, math.nan, math.nan
    head.dx_ = head.x.to(DEV)
    bad = torch.zeros(tokens, dtype=torch.bool)
    bad[[1, 2, 3, 4, 5, 6, 8, 10]] = True
    bad = bad.to(DEV)
    for grad in (False, True):
        x = head.dx_.clone().requires_grad_(grad)
        loss = head.run_on(x)
        assert torch.equal(loss.isnan(), bad)
        fine = ~bad
        fine[9] = False
        assert bool(((loss - want)[fine].abs() <= 100 * E * (1 + want[fine])).all())
        if grad:
            dx, = torch.autograd.grad(loss.sum(), x)
            assert torch.equal(dx.isnan().all(1), bad) and torch.equal(dx.isnan().any(1), bad)
            assert bool((dx[9] == 0).all())
    other = df11.linear_cross_entropy(head.head, head.dx_, torch.full_like(head.dt, 3), vocab=150, ignore_index=3)
    assert bool(other.isnan())  # nothing to take a mean of


@pytest.mark.parametrize("tokens", [9, 50])
def test_states_that_are_not_finite(tokens):
    """They spoil their own tokens only: the others keep their bits."""
    head = Head(tokens, 4160, 64, seed=17)
    x = head.dx_.clone()
    for row, value in ((1, math.nan), (2, math.inf), (8, -math.inf)):
        x[row, 3] = value
    assert all(int(head.targets[row]) != -100 for row in (1, 2, 8))
    others = torch.ones(tokens, dtype=torch.bool, device=DEV)
    others[[1, 2, 8]] = False
    for gradient in (False, True):
        results = []
        for states in (x, head.dx_):
            states = states.clone().requires_grad_(gradient)
            loss = head.run_on(states)
            results.append((loss.detach(), torch.autograd.grad(loss.sum(), states)[0] if gradient else loss))
        for got, want in zip(*results):
            assert torch.equal(got[others], want[others])
            assert not bool(got[[1, 2, 8]].isfinite().flatten(1).all(1).any() if got.dim() == 2 else
                            got[[1, 2, 8]].isfinite().any())


def test_nothing_to_score():
    head = Head(40, 64, 32, seed=8)
    head.dt.fill_(-100)
    x = head.dx_.clone().requires_grad_()
    loss = head.run_on(x, "mean")
    dx, = torch.autograd.grad(loss, x)
    assert bool(loss.isnan()) and bool((dx == 0).all())
    none = torch.zeros(0, 32, dtype=torch.bfloat16, device=DEV, requires_grad=True)
    t = torch.zeros(0, dtype=torch.int64, device=DEV)
    assert df11.linear_cross_entropy(head.head, none, t, reduction="none").shape == (0,)
    total = df11.linear_cross_entropy(head.head, none, t, reduction="sum")
    assert float(total.detach()) == 0 and torch.autograd.grad(total, none)[0].shape == (0, 32)
    assert bool(df11.linear_cross_entropy(head.head, none.detach(), t).isnan())


def test_shapes_and_strides():
    head = Head(60, 320, 64, seed=9)
    want, one = head.run(reduction="none"), head.run(reduction="none")[4]
    assert torch.equal(df11.linear_cross_entropy(head.head, head.dx_.view(3, 20, 64), head.dt.view(3, 20), reduction="none"),
                       want.view(3, 20))
    single = df11.linear_cross_entropy(head.head, head.dx_[4], head.dt[4], reduction="none")
    assert single.shape == () and abs(float(single - one)) <= 100 * E * (1 + float(one))
    wide = torch.zeros(60, 200, dtype=torch.bfloat16, device=DEV)
    wide[:, 8:72] = head.dx_
    assert torch.equal(df11.linear_cross_entropy(head.head, wide[:, 8:72], head.dt, reduction="none"), want)
    t = torch.stack([head.dt, head.dt], 1)[:, 0]
    assert torch.equal(df11.linear_cross_entropy(head.head, head.dx_, t, reduction="none"), want)
    x = head.dx_.view(3, 20, 64).clone().requires_grad_()
    g = torch.rand(20, device=DEV).expand(3, 20)
    dx, = torch.autograd.grad(df11.linear_cross_entropy(head.head, x, head.dt.view(3, 20), reduction="none"), x, g)
    flat = head.dx_.clone().requires_grad_()
    want_dx, = torch.autograd.grad(head.run_on(flat), flat, g.reshape(-1))
    assert torch.equal(dx.view(60, 64), want_dx)


def test_gradient_against_differences():
    """Central differences of the operator's own losses: with dz the change of the
    logits along a direction, the third derivative is at most (max dz - min dz)^3."""
    head = Head(40, 640, 64, 600, seed=10)
    head.x = (torch.randint(-24, 25, head.x.shape, generator=gen(11)) / 8).bfloat16()
    head.dx_ = head.x.to(DEV)
    h = 0.125
    x = head.dx_.clone().requires_grad_()
    dx, = torch.autograd.grad(head.run_on(x).sum(), x)
    _, tol, _, far = head.expect(torch.ones(40))
    for seed in range(4):
        way = (torch.randint(0, 2, head.x.shape, generator=gen(20 + seed)) * 2 - 1).to(DEV)
        up, down = ((head.dx_.float() + s * h * way).bfloat16() for s in (1, -1))
        assert torch.equal(up.float() - down.float(), 2 * h * way.float())
        slope = (df11.linear_cross_entropy(head.head, up, head.dt, vocab=600, reduction="none").double()
                 - df11.linear_cross_entropy(head.head, down, head.dt, vocab=600, reduction="none").double()) / (2 * h)
        dz = way.double() @ head.w.to(DEV)[:600].double().t()
        third = (dz.amax(1) - dz.amin(1)) ** 3
        most = h * h / 6 * third + 1.5 * tol / h + far.sum(1)
        assert bool(((dx.double() * way).sum(1) - slope).abs().le(most).all())


def test_same_bits_again():
    head = Head(300, 9024, 64, seed=12)
    x = head.dx_.clone().requires_grad_()
    first = head.run_on(x, "mean")
    grad, = torch.autograd.grad(first, x)
    few = df11.linear_cross_entropy(head.head, head.dx_[:20], head.dt[:20], reduction="none")
    for _ in range(3):
        again = head.run_on(x, "mean")
        assert torch.equal(again, first) and torch.equal(torch.autograd.grad(again, x)[0], grad)
        assert torch.equal(df11.linear_cross_entropy(head.head, head.dx_[:20], head.dt[:20], reduction="none"), few)


@pytest.mark.parametrize("tokens", [5, 100])
def test_captured(tokens):
    """A scoring and a training step in one graph, replayed on other tokens."""
    a, b = (Head(tokens, 4416, 64, 4400, seed=s) for s in (13, 14))
    head = a.head
    x = a.dx_.clone().requires_grad_()
    t = a.dt.clone()

    def step():
        score = df11.linear_cross_entropy(head, x.detach(), t, vocab=4400, reduction="none")
        loss = df11.linear_cross_entropy(head, x, t, vocab=4400)
        return score, loss.detach(), torch.autograd.grad(loss, x)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for c in (a, b, a, b):
        with torch.no_grad():
            x.copy_(c.dx_)
            t.copy_(c.dt)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        y = c.dx_.clone().requires_grad_()
        loss = df11.linear_cross_entropy(head, y, c.dt, vocab=4400)
        want = (df11.linear_cross_entropy(head, c.dx_, c.dt, vocab=4400, reduction="none"), loss.detach(),
                torch.autograd.grad(loss, y)[0])
        for g, w in zip(got, want):
            assert torch.equal(g, w)


def test_streams():
    """Calls of one head at once, on streams of their own, inputs freed before the streams get to them."""
    heads = [Head(n, 4416, 64, seed=15) for n in (20, 200)]
    want = [h.run(reduction="none") for h in heads]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        outs = []
        for h, stream in zip(heads, streams):
            x, t = h.x.to(DEV), h.targets.to(DEV)
            stream.wait_stream(torch.cuda.current_stream())
            outs.append(df11.linear_cross_entropy(heads[0].head if h is heads[0] else h.head, x, t, reduction="none",
                                                  stream=stream))
            del x, t
            torch.randn(h.x.shape, device=DEV)
        torch.cuda.synchronize()
        for got, w in zip(outs, want):
            assert torch.equal(got, w)


def test_loss_kept_by_its_graph():
    """The loss may be changed in place, and the gradient asked for twice."""
    head = Head(50, 320, 64, seed=16)
    x = head.dx_.clone().requires_grad_()
    loss = head.run_on(x, "mean")
    first, = torch.autograd.grad(loss, x, retain_graph=True)
    twice, = torch.autograd.grad(2 * loss, x, retain_graph=True)
    assert bool(((twice.float() - 2 * first.float()).abs() <= 2 * U * first.float().abs()).all())
    again, = torch.autograd.grad(loss.add_(1.0), x)
    assert torch.equal(again, first)
    with pytest.raises(ValueError):
        df11.linear_cross_entropy(head.head, x, head.dt, stream=torch.cuda.Stream())
