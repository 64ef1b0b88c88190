"""A small model's steps through all of the operators on a paged cache: a prompt,
a tree of drafted tokens attended to and scored through the compressed head, and
the accepted path, against the model written out in torch.

The written-out model rounds to bfloat16 where an operator's output does; every
other sum is 64 bits.  A sum that falls on the other side of a rounding differs
by a step, 2^-7 of the value at most.  Scores are logarithms of a softmax of logits
with a standard deviation of about one: a logit is a sum of 256 products of a
normed state (each off by a few steps at random, 2^-6 of about one) with weights of
0.06, off by 2^-6 * 0.06 * 16 = 0.015 or so; twice for the target and the
logarithm of the sum, four times for the largest of a hundred: 0.12."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from entropy_decoding_df11_amd import df11, runtime, workloads  # noqa: E402

DEV = "cuda:0"
HIDDEN, HEADS, KV, DIM, MLP, VOCAB, ROWS, PAGE = 256, 8, 2, 64, 512, 1000, 1024, 16
SHAPES = [("q_proj", (HEADS * DIM, HIDDEN)), ("k_proj", (KV * DIM, HIDDEN)), ("v_proj", (KV * DIM, HIDDEN)),
          ("o_proj", (HIDDEN, HEADS * DIM)), ("gate_proj", (MLP, HIDDEN)), ("up_proj", (MLP, HIDDEN)),
          ("down_proj", (HIDDEN, MLP))]
FAR = 0.12


def bits(rng, *shape, size=0.06):
    return workloads.f32_to_bf16_bits(rng.standard_normal(shape) * size)


def bf16(b):
    return torch.from_numpy(b.view(np.int16).copy()).view(torch.bfloat16)


@pytest.fixture(scope="module")
def model():
    rng = np.random.default_rng(0)
    raw = [{nm: bits(rng, *s) for nm, s in SHAPES} for _ in range(2)]
    blocks = [df11.compress_block({nm: bf16(b) for nm, b in w.items()}, device=DEV, codebook="per_weight",
                                  layout="mfma_tiles") for w in raw]
    head = bits(rng, ROWS, HIDDEN)
    return dict(blocks=blocks, raw=[{nm: bf16(b).double() for nm, b in w.items()} for w in raw],
                head=df11.compress(bf16(head), layout="mfma_tiles"), head_raw=bf16(head).double()[:VOCAB],
                embed=bf16(bits(rng, VOCAB, HIDDEN, size=1.0)), rotary=df11.rotary_table(400, DIM))


def r(x):
    return x.float().bfloat16().double()


def norm(x):
    return r(x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5))


def written_out(model, tokens):
    """Logits of every token of one sequence."""
    x = model["embed"][tokens].double()
    n = len(tokens)
    table = model["rotary"][:n].cpu().double()
    cos, sin = table[:, None, :DIM // 2], table[:, None, DIM // 2:]

    def turn(y):
        a, b = y[..., :DIM // 2], y[..., DIM // 2:]
        return r(torch.cat([a * cos - b * sin, b * cos + a * sin], -1))

    for w in model["raw"]:
        h = norm(x)
        q, k, v = (h @ w[nm].t() for nm in ("q_proj", "k_proj", "v_proj"))
        q, k, v = turn(q.view(n, HEADS, DIM)), turn(k.view(n, KV, DIM)), r(v).view(n, KV, DIM)
        z = torch.einsum("qhd,khd->hqk", q, k.repeat_interleave(HEADS // KV, 1)) / DIM ** 0.5
        z = z.masked_fill(~torch.ones(n, n, dtype=torch.bool).tril(), -torch.inf)
        a = r(torch.einsum("hqk,khd->qhd", z.softmax(-1), v.repeat_interleave(HEADS // KV, 1))).reshape(n, -1)
        x = r(a @ w["o_proj"].t() + x)
        h = norm(x)
        g, u = h @ w["gate_proj"].t(), h @ w["up_proj"].t()
        x = r(r(torch.nn.functional.silu(g) * u) @ w["down_proj"].t() + x)
    return norm(x) @ model["head_raw"].t()


class Cache:
    def __init__(self, pages=40):
        self.pairs = [tuple(torch.full((pages, PAGE, KV, DIM), float("nan"), dtype=torch.bfloat16, device=DEV)
                            for _ in range(2)) for _ in range(2)]
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(3)).int()
        self.table = order[:36].view(3, 12).to(DEV)


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


PROMPTS = [37, 5, 90]


def prompts():
    g = torch.Generator().manual_seed(4)
    return [torch.randint(0, VOCAB, (n,), generator=g) for n in PROMPTS]


def prefill(model, cache):
    """All prompts but their last tokens, scored against the next ones."""
    texts = prompts()
    ids = torch.cat([t[:-1] for t in texts])
    starts = np.concatenate([[0], np.cumsum([n - 1 for n in PROMPTS])])
    step = runtime.Step(cache.table, ints(*starts), ints(0, 0, 0), model["rotary"])
    scores = runtime.score_tokens(model["embed"][ids].to(DEV), model["blocks"], model["head"],
                                  torch.cat([t[1:] for t in texts]).to(DEV), cache.pairs, step, vocab=VOCAB)
    return texts, scores


def test_prompts(model):
    texts, scores = prefill(model, Cache())
    want = [written_out(model, t)[:-1].log_softmax(1).gather(1, t[1:, None])[:, 0] for t in texts]
    assert float((scores.cpu().double() - torch.cat(want)).abs().max()) <= FAR


# of every sequence the parents of its drafted tokens; -1: the prompt's last token, itself the first new one
TREES = [[-1, 0, 0, 1, 1, 2, 5], [-1, 0, 1], [-1, 0, 0, 0, 2, 4, 4, 1, 7]]


def drafted(texts, seed=5):
    """(ids, paths to each new token, mask, depths) of a step that verifies the trees."""
    g = torch.Generator().manual_seed(seed)
    ids, paths, depths = [], [], []
    mask = torch.zeros(sum(map(len, TREES)), max(map(len, TREES)), dtype=torch.bool)
    for text, parents in zip(texts, TREES):
        own = [int(text[-1])] + torch.randint(0, VOCAB, (len(parents) - 1,), generator=g).tolist()
        first, seen = len(ids), []
        for i, p in enumerate(parents):
            seen.append((seen[p] if p >= 0 else []) + [i])
            mask[first + i, seen[i]] = True
            depths.append(len(seen[i]) - 1)
            paths.append(torch.cat([text[:-1], torch.tensor([own[j] for j in seen[i]])]))
        ids += own
    return torch.tensor(ids), paths, mask, depths


def tree_step(model, cache, texts, seed=5):
    ids, paths, mask, depths = drafted(texts, seed)
    cached = [n - 1 for n in PROMPTS]
    seq = [s for s, t in enumerate(TREES) for _ in t]
    step = runtime.Step(cache.table, ints(*np.concatenate([[0], np.cumsum([len(t) for t in TREES])])), ints(*cached),
                        model["rotary"], ints(*[cached[s] + d for s, d in zip(seq, depths)]), mask.to(DEV))
    targets = torch.randint(0, VOCAB, (len(ids),), generator=torch.Generator().manual_seed(seed + 1))
    return model["embed"][ids].to(DEV), step, targets.to(DEV), paths


def test_drafted_trees(model):
    """Every drafted token is scored as at the end of its own path."""
    cache = Cache()
    texts, _ = prefill(model, cache)
    x, step, targets, paths = tree_step(model, cache, texts)
    scores = runtime.score_tokens(x, model["blocks"], model["head"], targets, cache.pairs, step, vocab=VOCAB)
    want = torch.stack([written_out(model, p)[-1].log_softmax(0)[t] for p, t in zip(paths, targets.cpu())])
    assert float((scores.cpu().double() - want).abs().max()) <= FAR


def test_accepted_path(model):
    """After a tree, the accepted path's tokens are appended again and generation goes on from them."""
    cache = Cache()
    texts, _ = prefill(model, cache)
    x, step, targets, paths = tree_step(model, cache, texts)
    runtime.score_tokens(x, model["blocks"], model["head"], targets, cache.pairs, step, vocab=VOCAB)
    ends = [6, 9, 18]  # the deepest accepted token of each sequence, by row
    lengths, news = [n - 1 for n in PROMPTS], [paths[e][n - 1:] for e, n in zip(ends, PROMPTS)]
    ids = torch.cat(news)
    starts = np.concatenate([[0], np.cumsum([len(t) for t in news])])
    again = runtime.Step(cache.table, ints(*starts), ints(*lengths), model["rotary"])
    targets = torch.randint(0, VOCAB, (len(ids),), generator=torch.Generator().manual_seed(9))
    scores = runtime.score_tokens(model["embed"][ids].to(DEV), model["blocks"], model["head"], targets.to(DEV), cache.pairs,
                                  again, vocab=VOCAB)
    want = torch.cat([written_out(model, paths[e])[n - 1:].log_softmax(1) for e, n in zip(ends, PROMPTS)])
    want = want.gather(1, targets[:, None])[:, 0]
    assert float((scores.cpu().double() - want).abs().max()) <= FAR


def test_captured_step(model):
    """One graph, replayed on other drafts: embeddings, masks and positions change in place."""
    cache = Cache()
    texts, _ = prefill(model, cache)
    x, step, targets, _ = tree_step(model, cache, texts)
    forward = runtime.CapturedForward(
        lambda y: runtime.score_tokens(y, model["blocks"], model["head"], targets, cache.pairs, step, vocab=VOCAB), x)
    for seed in (5, 6, 7, 5):
        y, _, new, paths = tree_step(model, cache, texts, seed)
        targets.copy_(new)
        got = forward(y)
        want = torch.stack([written_out(model, p)[-1].log_softmax(0)[t] for p, t in zip(paths, new.cpu())])
        assert float((got.cpu().double() - want).abs().max()) <= FAR


def test_what_goes_together(model):
    x = torch.zeros(2, 3, HIDDEN, dtype=torch.bfloat16, device=DEV)
    cache = Cache()
    step = runtime.Step(cache.table, ints(0, 3, 3, 3), ints(0, 0, 0))
    with pytest.raises(ValueError):
        runtime.operator_block_forward(x, model["blocks"][0], cache=cache.pairs[0], step=step)
    with pytest.raises(ValueError):
        runtime.operator_block_forward(x[0], model["blocks"][0], cache=cache.pairs[0])
    with pytest.raises(ValueError):
        runtime.operator_block_forward(x[0], model["blocks"][0], step=step)
    with pytest.raises(ValueError):  # no gradients through the cache
        runtime.operator_block_forward(x[0].clone().requires_grad_(), model["blocks"][0], cache=cache.pairs[0], step=step)
