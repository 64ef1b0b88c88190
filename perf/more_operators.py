"""Measured cases of the operators that a step of generation and its scoring need
beside the compressed products: keys and values appended to a paged cache with the
position rotation on the way, attention of drafted tokens over that cache, and the
softmax cross entropy through a compressed output head, with its gradient.

A cache is pages of (page, kv_heads, dim); page_table[s] lists sequence s's pages.
Sequence s holds lengths[s] tokens and brings tokens starts[s] .. starts[s + 1] - 1
of the batch, its i-th going to place lengths[s] + i.  Where `own` is false the
operators run in their plain form, elementary torch operations in 32 bits.

    append  (a, b) -> (a cos - b sin, b cos + a sin) of q and k, at each token's
            position; k and v to their places in the cache
    attend  o = sum_j p_j v_j,  p = softmax over the visible j of scale q . k_j: all
            lengths[s] cached places, and of the new tokens those that the mask (a
            drafted token's ancestors and itself) or, without one, their order allows
    loss    -log softmax(x W^T)[target], W the output head; dx through the same head
"""

import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
IGNORED = -100

# Stored bits of one weight: sign and mantissa verbatim, about 2.6 bits of
# exponent entropy.
WEIGHT_BYTES = 10.6 / 8


def _case(op, name, **more):
    if op == "loss":
        case = {"op": op, "tokens": 1, "cols": 4096, "rows": 32000, "vocab": 32000, "mean": False, "grad": False}
    else:
        case = {"op": op, "seqs": 1, "tokens": 1, "context": 1024, "heads": 32, "kv_heads": 8, "dim": 128, "page": 16,
                "type": "bf16"}
        case.update({"from": "bf16", "rotated": 128, "pairs": False} if op == "append" else {"tree": False, "lse": False})
    case.update(more)
    if name:
        case["name"] = name
    return case


def listed():
    return [
        # One token of one sequence: the call's latency.
        _case("append", "append_one_token", context=700),
        # Drafted trees of a serving batch, straight from the products' float sums.
        _case("append", "append_trees", seqs=64, tokens=24, context=1000, **{"from": "fp32"}),
        # Ragged prompts; half of each head rotated, in neighbouring pairs, pages of an odd size.
        _case("append", "append_prompts", seqs=7, tokens=1531, context=300, page=40, type="fp16", rotated=64, pairs=True,
              **{"from": "fp16"}),
        # One token over a short context: the call's latency.
        _case("attend", "attend_one_token", context=700),
        # One token of each of a batch of sequences of many lengths.
        _case("attend", "attend_batch", seqs=64, context=8192),
        # A tree of drafted tokens over one long context.
        _case("attend", "attend_long_tree", tokens=64, context=131072, page=64, tree=True),
        # Drafted trees of a batch: narrow heads, seven to a key head, pages that end inside a tile.
        _case("attend", "attend_trees", seqs=24, tokens=25, context=4096, heads=28, kv_heads=4, dim=64, page=40,
              type="fp16", tree=True, lse=True),
        # Pieces of two prompts after what is cached of them.
        _case("attend", "attend_prompts", seqs=2, tokens=1531, context=2500, page=32),
        # Drafted tokens scored.
        _case("loss", "loss_drafts", tokens=24),
        # A prompt's perplexity through the largest head.
        _case("loss", "loss_prompt", tokens=1000, rows=128256, vocab=128256),
        # A training step of what is below a frozen head.
        _case("loss", "loss_train", tokens=2048, mean=True, grad=True),
        # The same of a smaller model: rows of padding behind the vocabulary, an odd batch.
        _case("loss", "loss_train_small", tokens=333, cols=1024, rows=50304, vocab=50257, grad=True),
    ]


def _spread(rng, low, high):
    """A whole number in [low, high], even over its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "loss"])
    if op == "loss":
        cols, rows = 32 * _spread(rng, 8, 160), 64 * _spread(rng, 4, 800)
        while cols * rows > 1 << 27:
            cols, rows = 32 * _spread(rng, 8, 160), 64 * _spread(rng, 4, 800)
        return _case(op, None, tokens=_spread(rng, 1, 2048), cols=cols, rows=rows,
                     vocab=rows - rng.choice([0, 0, rng.randrange(64)]), mean=rng.random() < 0.5,
                     grad=rng.random() < 0.5)
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8])
    dim, page, kind = rng.choice([64, 64, 80, 96, 128, 128, 128, 256]), rng.choice([16, 16, 24, 32, 64, 128]), \
        rng.choice(["bf16", "bf16", "fp16"])
    seqs = _spread(rng, 1, 64)
    tokens = rng.choice([1, 1, _spread(rng, 2, 128), _spread(rng, 2, 1000)])
    common = {"seqs": seqs, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "type": kind}
    if op == "append":
        return _case(op, None, tokens=min(tokens, 8192 // seqs), context=_spread(rng, 1, 1000), **common,
                     rotated=rng.choice([dim, dim, dim // 2]), pairs=rng.random() < 0.3,
                     **{"from": rng.choice([kind, "fp32"])})
    tokens = min(tokens, max(1, 1000 // seqs))
    # (keys of all sequences and heads, and products of queries with them, as in the listed cases)
    most = min((1 << 27) // (seqs * kv_heads * dim), (1 << 35) // (seqs * tokens * heads * dim))
    return _case(op, None, tokens=tokens, context=_spread(rng, 1, max(1, min(65536, most - tokens))), **common,
                 tree=1 < tokens <= 128 and rng.random() < 0.7, lse=rng.random() < 0.3)


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------

def _layout(case):
    """(tokens cached, tokens new) of every sequence, the longest first of each: plain numbers of the case."""
    rng = random.Random(case["seqs"] * 7919 + case["context"] * 31 + case["tokens"])
    cached = [case["context"]] + [rng.randint(0, case["context"]) for _ in range(case["seqs"] - 1)]
    new = [case["tokens"]] + [rng.randint((case["tokens"] + 1) // 2, case["tokens"]) for _ in range(case["seqs"] - 1)]
    return cached, new


def _parents(case, n, rng):
    """Parents of n drafted tokens (-1: the last cached one), several to a level as drafting gives them."""
    return [-1 if i < 2 else rng.randint(max(-1, i // 2 - 3), i - 1) for i in range(n)]


def _trees(case, new):
    """Of every new token (its depth, the list of its ancestors and itself), sequence by sequence."""
    rng, out = random.Random(case["tokens"]), []
    for n in new:
        seen = []
        for i, p in enumerate(_parents(case, n, rng)):
            seen.append((seen[p] if p >= 0 else []) + [i])
        out += seen
    return out


def _head(g, rows, cols):
    """Trained-weight statistics: N(0, 0.02^2) with one entry in 10^4 an outlier from N(0, 1)."""
    w = torch.randn(rows, cols, device="cuda", generator=g)
    far = torch.rand(rows, cols, device="cuda", generator=g) < 1e-4
    return torch.where(far, w, w * 0.02).bfloat16()


def _prepare_loss(case, g):
    w = _head(g, case["rows"], case["cols"])
    t = case["tokens"]
    target = torch.randint(0, case["vocab"], (t,), device="cuda", generator=g)
    # A trained model's hidden states lean towards what comes next, some more, some less.
    lean = 8 * torch.rand(t, 1, device="cuda", generator=g) * (4096 / case["cols"])
    x = 2 * torch.randn(t, case["cols"], device="cuda", generator=g) * (4096 / case["cols"]) ** 0.5
    state = {"case": case, "x": (x + lean * w[target].float()).bfloat16()}
    state["target"] = torch.where(torch.rand(t, device="cuda", generator=g) < 0.1, IGNORED, target)
    state["target"][0] = target[0]
    if case["grad"]:
        shape = () if case["mean"] else (t,)
        state["dy"] = 0.5 + torch.rand(shape, device="cuda", generator=g)
    if own:
        # A program keeps its head compressed; it is compressed once.
        from entropy_decoding_df11_amd import df11
        w = df11.compress(w.cpu(), layout="mfma_tiles")
    state["w"] = w
    return state


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "loss":
        return _prepare_loss(case, g)
    cached, new = _layout(case)
    page, kind, total = case["page"], TYPES[case["type"]], sum(new)
    need = [-(-(c + n) // page) for c, n in zip(cached, new)]
    width, pages = -(-(case["context"] + case["tokens"]) // page), sum(need) + 3
    order = torch.randperm(pages, device="cuda", generator=g).int()
    starts = torch.zeros(case["seqs"] + 1, dtype=torch.int64)
    starts[1:] = torch.tensor(new).cumsum(0)
    first = torch.zeros(case["seqs"], dtype=torch.int64)
    first[1:] = torch.tensor(need[:-1]).cumsum(0)
    at = first[:, None] + torch.arange(width)
    held = torch.arange(width) < torch.tensor(need)[:, None]
    table = torch.where(held.cuda(), order[at.clamp(max=pages - 1).cuda()], 0).int()
    state = {"case": case, "starts": starts.int().cuda(), "lengths": torch.tensor(cached).int().cuda(), "page_table": table}
    for name in ("k_cache", "v_cache"):
        state[name] = torch.randn(pages, page, case["kv_heads"], case["dim"], device="cuda", generator=g).to(kind)
    q = torch.randn(total, case["heads"], case["dim"], device="cuda", generator=g)
    if case["op"] == "attend":
        # Normed queries, a little sharper than chance.
        state["q"] = (1.5 * q).to(kind)
        if case["tree"]:
            mask = torch.zeros(total, case["tokens"], dtype=torch.bool)
            for i, seen in enumerate(_trees(case, new)):
                mask[i, seen] = True
            state["mask"] = mask.cuda()
        return state
    source = TYPES[case["from"]]
    state["q"] = q.to(source)
    for name in ("k", "v"):
        state[name] = torch.randn(total, case["kv_heads"], case["dim"], device="cuda", generator=g).to(source)
    # Drafted trees' positions are their depths; up to 2^17 positions are in the table.
    seq = torch.repeat_interleave(torch.arange(case["seqs"]), torch.tensor(new))
    depth = torch.arange(total) - starts[:-1][seq]
    if case["tokens"] <= 128:
        depth = torch.tensor([len(seen) - 1 for seen in _trees(case, new)])
    state["positions"] = (torch.tensor(cached)[seq] + depth).int().cuda()
    half = case["rotated"] // 2
    angle = torch.arange(1 << 17, device="cuda", dtype=torch.float64)[:, None] * \
        500000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    state["rotary"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    return state


# ---------------------------------------------------------------------------
# Plain forms.
# ---------------------------------------------------------------------------

def _rotate(x, table, pairs):
    half = table.shape[1] // 2
    cos, sin = table[:, None, :half], table[:, None, half:]
    head, rest = x[..., :2 * half], x[..., 2 * half:]
    if pairs:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = head[..., :half], head[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, rest], -1)


def _places(s, total):
    """(sequence, place among its new tokens) of every token of the batch."""
    at = torch.arange(total, device="cuda")
    seq = torch.searchsorted(s["starts"][1:].contiguous(), at, right=True)
    return seq, at - s["starts"].long()[seq]


def _plain_append(s):
    case, kind = s["case"], s["k_cache"].dtype
    table = s["rotary"][s["positions"].long()]
    seq, i = _places(s, s["k"].shape[0])
    place = s["lengths"].long()[seq] + i
    page, offset = s["page_table"].long()[seq, place // case["page"]], place % case["page"]
    s["k_cache"][page, offset] = _rotate(s["k"].float(), table, case["pairs"]).to(kind)
    s["v_cache"][page, offset] = s["v"].to(kind)
    return {"q": _rotate(s["q"].float(), table, case["pairs"]).to(kind), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s):
    case = s["case"]
    seqs, n, hk, d = case["seqs"], case["tokens"], case["kv_heads"], case["dim"]
    total, group = s["q"].shape[0], case["heads"] // hk
    seq, i = _places(s, total)
    q = torch.zeros(seqs, n, hk, group, d, device="cuda")
    q[seq, i] = s["q"].float().view(total, hk, group, d)
    q = q.permute(0, 2, 3, 1, 4).reshape(seqs, hk, group * n, d)
    table = s["page_table"].long()
    k = s["k_cache"][table].flatten(1, 2).float().permute(0, 2, 3, 1)  # seqs, kv_heads, dim, places
    score = (q @ k).view(seqs, hk, group, n, -1) / math.sqrt(d)
    place = torch.arange(score.shape[-1], device="cuda")
    j = place - s["lengths"].long()[:, None]  # a place's number among the new tokens
    if case["tree"]:
        among = torch.zeros(seqs, n, n, dtype=torch.bool, device="cuda")
        among[seq, i] = s["mask"]
        seen = among.gather(2, j.clamp(0, n - 1)[:, None].expand(seqs, n, -1)) & (j < n)[:, None] | (j < 0)[:, None]
    else:
        seen = j[:, None] <= torch.arange(n, device="cuda")[:, None]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = score.sub_(top).exp_()
    total_p = p.sum(-1, keepdim=True)
    v = s["v_cache"][table].flatten(1, 2).float().transpose(1, 2)
    o = (p.view(seqs, hk, group * n, -1) @ v).view(seqs, hk, group, n, d)
    o = torch.where(total_p > 0, o / total_p, 0.0)
    out = {"o": o.permute(0, 3, 1, 2, 4)[seq, i].flatten(1, 2).to(s["q"].dtype)}
    if case["lse"]:
        lse = (total_p.log() + top)[..., 0]
        out["lse"] = lse.permute(0, 3, 1, 2)[seq, i].flatten(1, 2)
    return out


def _plain_loss(s):
    case = s["case"]
    w = s["w"][:case["vocab"]].float()
    z = s["x"].float() @ w.t()
    counted = s["target"] != IGNORED
    target = torch.where(counted, s["target"], 0)[:, None]
    top = z.amax(1, keepdim=True)
    e = (z - top).exp()
    total = e.sum(1, keepdim=True)
    loss = torch.where(counted, (total.log() + top - z.gather(1, target))[:, 0], 0.0)
    out = {"loss": loss.sum() / counted.sum() if case["mean"] else loss}
    if case["grad"]:
        g = torch.where(counted, s["dy"] / counted.sum() if case["mean"] else s["dy"], 0.0)[:, None]
        dz = e.div_(total).scatter_add_(1, target, torch.full_like(top, -1.0)).mul_(g)
        out["dx"] = (dz @ w).to(s["x"].dtype)
    return out


# ---------------------------------------------------------------------------
# The framework's operators.
# ---------------------------------------------------------------------------

def _own_append(s):
    from entropy_decoding_df11_amd import df11
    q = df11.append_kv(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["starts"], s["lengths"], q=s["q"],
                       rotary=s["rotary"], positions=s["positions"], interleaved=s["case"]["pairs"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attend(s):
    from entropy_decoding_df11_amd import df11
    got = df11.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["starts"], s["lengths"],
                              mask=s.get("mask"), return_lse=s["case"]["lse"])
    return dict(zip(("o", "lse"), got)) if s["case"]["lse"] else {"o": got}


def _own_loss(s):
    from entropy_decoding_df11_amd import df11
    case = s["case"]
    x = s["x"].detach().requires_grad_() if case["grad"] else s["x"]
    loss = df11.linear_cross_entropy(s["w"], x, s["target"], vocab=case["vocab"], ignore_index=IGNORED,
                                     reduction="mean" if case["mean"] else "none")
    if not case["grad"]:
        return {"loss": loss}
    return {"loss": loss.detach(), "dx": torch.autograd.grad(loss, x, s["dy"])[0]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "attend": _own_attend, "loss": _own_loss}[op](state)
    return {"append": _plain_append, "attend": _plain_attend, "loss": _plain_loss}[op](state)


def work(case):
    if case["op"] == "loss":
        t, c, r = case["tokens"], case["cols"], case["vocab"]
        total, flops = 2 * t * c + WEIGHT_BYTES * r * c + 8 * t + 4 * t, 2 * t * r * c
        if case["grad"]:  # dx, and the product that gives it
            total, flops = total + 2 * t * c + 4 * t, 2 * flops
        return {"bytes": int(total), "flops": flops}
    cached, new = _layout(case)
    total, each = sum(new), case["heads"] + 2 * case["kv_heads"]
    if case["op"] == "append":
        moved = case["dim"] * total * each * (SIZE[case["from"]] + SIZE[case["type"]])
        return {"bytes": moved + total * (4 + 4 * case["rotated"]),
                "flops": 3 * case["rotated"] * total * (each - case["kv_heads"])}
    size = SIZE[case["type"]]
    held = sum(cached) + total
    seen = sum(c * n for c, n in zip(cached, new))
    if case["tree"]:
        seen += sum(len(t) for t in _trees(case, new))
    else:
        seen += sum(n * (n + 1) // 2 for n in new)
    return {"bytes": size * case["dim"] * (2 * held * case["kv_heads"] + 2 * total * case["heads"])
            + total * (case["tokens"] * case["tree"] + 4 * case["heads"] * case["lse"]),
            "flops": 4 * case["dim"] * case["heads"] * seen}


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------

def _exact_append(case, s):
    half = case["rotated"] // 2
    turn = torch.complex(*s["rotary"].double()[s["positions"].long()].split(half, 1))[:, None]
    got = {}
    for name in ("q", "k"):
        x = s[name].double().clone()
        lanes = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["pairs"] else \
            (slice(0, half), slice(half, 2 * half))
        z = torch.complex(x[..., lanes[0]], x[..., lanes[1]]) * turn
        x[..., lanes[0]], x[..., lanes[1]] = z.real, z.imag
        got[name] = x
    k, v = s["k_cache"].double(), s["v_cache"].double()
    cached, new = _layout(case)
    first = 0
    for b, (c, n) in enumerate(zip(cached, new)):
        slots = torch.arange(c, c + n, device="cuda")
        pages = s["page_table"][b].long()[slots // case["page"]]
        k[pages, slots % case["page"]] = got["k"][first:first + n]
        v[pages, slots % case["page"]] = s["v"][first:first + n].double()
        first += n
    return {"q": got["q"], "k_cache": k, "v_cache": v}


def _exact_attend(case, s):
    cached, new = _layout(case)
    group = case["heads"] // case["kv_heads"]
    outs, lses, first = [], [], 0
    for b, (c, n) in enumerate(zip(cached, new)):
        places = torch.arange(c + n, device="cuda")
        pages = s["page_table"][b].long()[places // case["page"]]
        visible = torch.ones(n, c + n, dtype=torch.bool, device="cuda")
        visible[:, c:] = s["mask"][first:first + n, :n] if case["tree"] else \
            torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        o = torch.zeros(n, case["heads"], case["dim"], dtype=torch.float64, device="cuda")
        lse = torch.zeros(n, case["heads"], dtype=torch.float64, device="cuda")
        for h in range(case["kv_heads"]):
            k = s["k_cache"][:, :, h][pages, places % case["page"]].double()
            v = s["v_cache"][:, :, h][pages, places % case["page"]].double()
            for m in range(h * group, h * group + group):
                z = s["q"][first:first + n, m].double() @ k.t() * case["dim"] ** -0.5
                z = z.masked_fill(~visible, -math.inf)
                lse[:, m] = z.logsumexp(1)
                o[:, m] = torch.nan_to_num(z.softmax(1)) @ v
        outs.append(o)
        lses.append(lse)
        first += n
    got = {"o": torch.cat(outs)}
    if case["lse"]:
        got["lse"] = torch.cat(lses)
    return got


def _exact_loss(case, s):
    x, kept = s["x"].double(), s["target"] != IGNORED
    pieces = [(at, min(case["vocab"], at + 8192)) for at in range(0, case["vocab"], 8192)]
    logits = [x @ s["w"][a:b].double().t() for a, b in pieces]
    lse = torch.stack([z.logsumexp(1) for z in logits], 1).logsumexp(1)
    loss = torch.zeros_like(lse)
    for (a, b), z in zip(pieces, logits):
        here = kept & (s["target"] >= a) & (s["target"] < b)
        rows = here.nonzero()[:, 0]
        loss[rows] = lse[rows] - z[rows, s["target"][rows] - a]
    got = {"loss": loss.sum() / kept.sum() if case["mean"] else loss}
    if case["grad"]:
        g = s["dy"].double() * kept
        g = (g / kept.sum() if case["mean"] else g)[:, None]
        dx = torch.zeros_like(x)
        for (a, b), z in zip(pieces, logits):
            dx += (z - lse[:, None]).exp() @ s["w"][a:b].double()
        got["dx"] = g * (dx - s["w"][s["target"].clamp(min=0)].double())
    return got


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"append": _exact_append, "attend": _exact_attend, "loss": _exact_loss}[case["op"]](case, s)
