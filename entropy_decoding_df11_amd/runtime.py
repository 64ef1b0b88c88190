"""Decompress transformer blocks just before use, or fuse the decode into
each projection.

GeekNews, "DFloat11: Kompresi inferensi GPU lossless yang mengecilkan LLM
menjadi 70% ukurannya", sections "Dekompresi yang disesuaikan untuk inferensi
GPU" and "Dekompresi per transformer block": weights stay compressed in HBM,
each block is decompressed into a scratch buffer right before its forward
pass and discarded after it.  BlockDecoder does that on the caller's stream,
or, with overlap=True, decodes block i + 1 on a side stream into the other of
two scratch buffers while the caller computes with block i.
"""

from __future__ import annotations

import dataclasses
from typing import Dict, Iterator, List, Optional, Sequence, Tuple, Union

from .attention import append_kv, tree_attention
from .df11 import DF11Block, DF11BlockBatch
from .loss import linear_cross_entropy
from .operators import gated_matmul, matmul_epilogue, rms_norm

Block = Union[DF11Block, DF11BlockBatch]


class BlockDecoder:
    """Iterate over compressed blocks, yielding (index, {name: bf16 weight})
    with every weight already decoded in the caller's stream order.

    By default each block is decoded on the caller's stream right before it
    is yielded.  With overlap=True, block i + 1 is decoded on a side stream
    while the caller enqueues block i's work; an event recorded on the
    caller's stream when it asks for the next block marks block i's scratch
    buffer free again.  Either way the weights of block i are valid until the
    caller asks for block i + 2 (two scratch buffers alternate), so the caller
    must finish enqueuing block i's work before advancing.

    Overlap rarely pays on one GPU: the decoder's persistent grid fills every
    CU and is bound by HBM, and so are the caller's GEMMs at small batch.
    decode_workgroups caps the workgroups of an overlapped decode (0: fill the
    GPU) so the caller's kernels find room beside it.
    """

    def __init__(self, blocks: Sequence[Block], device="cuda", overlap: bool = False, decode_workgroups: int = 0):
        import torch
        self.blocks = list(blocks)
        self.device = torch.device(device)
        self.overlap = overlap
        self.decode_workgroups = decode_workgroups
        n = max((b.n_elements for b in self.blocks), default=0)
        self._scratch = [torch.empty(max(n, 1), dtype=torch.bfloat16, device=self.device) for _ in range(2)]
        # Default priority: streams of different priorities are avoided.
        self._side = torch.cuda.Stream(self.device) if overlap else None

    def __len__(self) -> int:
        return len(self.blocks)

    def _decode(self, i: int, stream, cap: int = 0) -> Dict:
        b = self.blocks[i]
        if cap:
            b.set_max_workgroups(cap)
        try:
            return b.decompress(scratch=self._scratch[i % 2], stream=stream)
        finally:
            if cap:
                b.set_max_workgroups(0)

    def __iter__(self) -> Iterator[Tuple[int, Dict]]:
        import torch
        if not self.blocks:
            return
        main = torch.cuda.current_stream(self.device)
        if not self.overlap:
            for i in range(len(self.blocks)):
                yield i, self._decode(i, main)
            return
        side = self._side
        free = [None, None]      # event: the caller has finished with scratch[k]
        ready = [None] * len(self.blocks)

        def launch(i: int):
            side.wait_stream(main) if free[i % 2] is None else side.wait_event(free[i % 2])
            views = self._decode(i, side, self.decode_workgroups)
            ev = torch.cuda.Event()
            ev.record(side)
            ready[i] = ev
            return views

        pending = launch(0)
        for i in range(len(self.blocks)):
            views = pending
            main.wait_event(ready[i])
            if i + 1 < len(self.blocks):
                pending = launch(i + 1)
            yield i, views
            # the caller has enqueued block i's work on `main`
            ev = torch.cuda.Event()
            ev.record(main)
            free[i % 2] = ev


def block_forward(x, w: Dict, eps: float = 1e-5, operators: bool = False):
    """A synthetic Llama-style block forward on BF16 weights (no attention
    mixing, which needs no weights): RMS-normed projections q, k, v and o
    with a residual, then the gated MLP (gate, up, down) with a residual.
    Used to show the decompressed weights in use; shapes follow the weights.

    operators: the norms run as rms_norm (the second one with the residual's
    addition), one launch each in place of torch's elementwise ones.  They
    round once where torch's chain rounds the reciprocal root and each
    product to x's dtype, so the last bits differ."""
    import torch
    import torch.nn.functional as F

    def rms(h):
        return h * torch.rsqrt(h.float().pow(2).mean(-1, keepdim=True) + eps).to(h.dtype)

    h = rms_norm(x, eps=eps) if operators else rms(x)
    q = F.linear(h, w["q_proj"])
    k = F.linear(h, w["k_proj"])
    v = F.linear(h, w["v_proj"])
    rep = q.shape[-1] // k.shape[-1]
    a = q + (k * v).repeat_interleave(rep, dim=-1)
    if operators:
        h, x = rms_norm(F.linear(a, w["o_proj"]), residual=x, eps=eps)
    else:
        x = x + F.linear(a, w["o_proj"])
        h = rms(x)
    x = x + F.linear(F.silu(F.linear(h, w["gate_proj"])) * F.linear(h, w["up_proj"]), w["down_proj"])
    return x


# Token counts up to which the fused products beat decoding the block first
# and calling torch's GEMM (Llama-3-8B block, measured): the matrix-core
# product sweeps the stream once per 64 tokens, the row-order product takes
# up to 8 tokens.
FUSED_MAX_TOKENS_TILES = 64
FUSED_MAX_TOKENS_ROWS = 8


@dataclasses.dataclass
class Step:
    """What a step of generation brings beside its tokens, the same for every
    block (attention.py): where the batch's sequences stand in a paged cache
    (page_table, starts, lengths), the rotation of their positions, and the mask
    of drafted trees.  The tensors may be changed in place between the replays
    of a captured step."""

    page_table: "torch.Tensor"  # noqa: F821
    starts: "torch.Tensor"  # noqa: F821
    lengths: "torch.Tensor"  # noqa: F821
    rotary: Optional["torch.Tensor"] = None  # noqa: F821
    positions: Optional["torch.Tensor"] = None  # noqa: F821
    mask: Optional["torch.Tensor"] = None  # noqa: F821
    interleaved: bool = False


def cached_attention(q, k, v, cache: Tuple, step: Step):
    """The attention of a block: k and v (tokens, kv_heads * head_dim) appended
    to cache, a pair of (pages, page, kv_heads, head_dim) tensors, and q (tokens,
    heads * head_dim) attending over it; float32 (a product's sums) or the
    cache's type.  Returns (tokens, heads * head_dim) of the cache's type."""
    k_cache, v_cache = cache
    dim = k_cache.shape[-1]
    where = (k_cache, v_cache, step.page_table, step.starts, step.lengths)
    q = append_kv(k.unflatten(-1, (-1, dim)), v.unflatten(-1, (-1, dim)), *where, q=q.unflatten(-1, (-1, dim)),
                  rotary=step.rotary, positions=step.positions, interleaved=step.interleaved)
    return tree_attention(q, *where, mask=step.mask, out=q).flatten(1)


def operator_block_forward(x, blk: DF11BlockBatch, eps: float = 1e-5, cache: Optional[Tuple] = None,
                           step: Optional[Step] = None):
    """block_forward through the operators around the products, for x of any
    leading dimensions: rms_norm, q, k and v (one matmul_batch up to
    FUSED_MAX_TOKENS_TILES tokens, else and under autograd matmul_epilogue),
    o and down with the residual in their epilogue (matmul_epilogue), gate and
    up as one gated product (gated_matmul).  blk holds one DF11 stream per
    weight in MFMA tile order (compress_block(..., codebook="per_weight",
    layout="mfma_tiles")).  Every operator computes in float32 and rounds its
    output once.  matmul_batch adds with float atomics and uses the weights'
    work counters: with it the last bits may differ from call to call, and
    calls on one block must not overlap; the other operators repeat theirs and
    may.  Differentiable with respect to x (the weights are frozen).

    With cache, the block's pair of paged keys and values, and step, x is
    (tokens, features) and the block attends over the cache (cached_attention;
    no gradients), whose output of the cache's type is taken in x's; without them
    it has no attention mixing, as block_forward."""
    import torch
    from .df11 import matmul_batch

    if (cache is None) != (step is None):
        raise ValueError("cache and step go together")
    if cache is not None and x.dim() != 2:
        raise ValueError("x must be (tokens, features) for a block that attends")
    w = {nm: t for (nm, _, _), t in zip(blk.views, blk.tensors)}
    qkv = [w[nm] for nm in ("q_proj", "k_proj", "v_proj")]
    h = rms_norm(x, eps=eps)
    tokens = x.numel() // x.shape[-1]
    if not 0 < tokens <= FUSED_MAX_TOKENS_TILES or (torch.is_grad_enabled() and x.requires_grad):
        q, k, v = (matmul_epilogue(t, h) for t in qkv)
    else:
        q, k, v = matmul_batch(qkv, [h.view(tokens, x.shape[-1])] * 3)
        if cache is None:
            q, k, v = (y.to(x.dtype).view(*x.shape[:-1], -1) for y in (q, k, v))
    if cache is None:
        a = q + (k * v).repeat_interleave(q.shape[-1] // k.shape[-1], dim=-1)
    else:
        a = cached_attention(q, k, v, cache, step).to(x.dtype)
    x = matmul_epilogue(w["o_proj"], a, residual=x)
    h = gated_matmul(w["gate_proj"], w["up_proj"], rms_norm(x, eps=eps))
    return matmul_epilogue(w["down_proj"], h, residual=x)


def operator_model_forward(x, blocks: Sequence[DF11BlockBatch], caches: Optional[Sequence[Tuple]] = None,
                           step: Optional[Step] = None):
    """operator_block_forward over every block in order, with caches (one pair
    for each block) and step attending over them."""
    for i, blk in enumerate(blocks):
        x = operator_block_forward(x, blk, cache=None if caches is None else caches[i], step=step)
    return x


def score_tokens(x, blocks: Sequence[DF11BlockBatch], head, targets, caches: Optional[Sequence[Tuple]] = None,
                 step: Optional[Step] = None, norm=None, eps: float = 1e-5, vocab: Optional[int] = None):
    """The logarithm of the probability that the model gives each token's target,
    float32 (tokens,): operator_model_forward, the last norm (weight norm) and the
    compressed output head, whose logits are not kept (linear_cross_entropy).  What
    drafted tokens are accepted by, and a text's perplexity.  Targets of -100 give
    zero."""
    h = rms_norm(operator_model_forward(x, blocks, caches, step), weight=norm, eps=eps)
    return -linear_cross_entropy(head, h, targets, vocab=vocab, reduction="none")


def fused_block_forward(x, blk: DF11BlockBatch, eps: float = 1e-5, scratch=None):
    """block_forward with each projection's decode fused into its product:
    blk holds one DF11 stream per weight, and no weight is ever decompressed
    to HBM.  Weights in MFMA tile order (compress_block(..., layout=
    "mfma_tiles")) go through the matrix-core product (df11_matmul_batch:
    q, k and v in one launch, o, gate and up in one, down), for any token
    count; weights in row order through the row-order product
    (df11_linear_batch / df11_linear), for 1..8 tokens.  The products
    accumulate in float32 and are rounded to x's dtype, like the resident
    path's outputs, but in another order, so the last bits can differ from
    block_forward's.  Above FUSED_MAX_TOKENS_TILES (tile order) or
    FUSED_MAX_TOKENS_ROWS (row order) tokens the block is decoded (into
    scratch, if given) and block_forward runs on it: there the GEMM's reuse
    of W across tokens outweighs the decode."""
    import torch
    import torch.nn.functional as F
    from .df11 import linear_batch, matmul_batch

    w = {nm: t for (nm, _, _), t in zip(blk.views, blk.tensors)}
    tiled = all(t.tile_cols for t in blk.tensors)
    if x.shape[0] > (FUSED_MAX_TOKENS_TILES if tiled else FUSED_MAX_TOKENS_ROWS):
        return block_forward(x, blk.decompress(scratch=scratch), eps)

    def products(names_, xin, outs):
        ts = [w[nm] for nm in names_]
        if tiled:
            matmul_batch(ts, [xin] * len(ts), outs=outs, accumulate=True)
        elif len(ts) == 1:
            ts[0].linear(xin, out=outs[0], accumulate=True)
        else:
            linear_batch(ts, xin, outs=outs, accumulate=True)

    def rms(h):
        return h * torch.rsqrt(h.float().pow(2).mean(-1, keepdim=True) + eps).to(h.dtype)

    # The seven products accumulate into views of one buffer, zeroed by one
    # fill, rather than each zeroing its own output (df11_linear_acc).
    names = ("q_proj", "k_proj", "v_proj", "o_proj", "gate_proj", "up_proj", "down_proj")
    tokens = x.shape[0]
    sizes = [tokens * w[nm].shape[0] for nm in names]
    buf = torch.zeros(sum(sizes), dtype=torch.float32, device=x.device)
    y = {nm: part.view(tokens, w[nm].shape[0]) for nm, part in zip(names, torch.split(buf, sizes))}

    h = rms(x).contiguous()
    products(("q_proj", "k_proj", "v_proj"), h, [y["q_proj"], y["k_proj"], y["v_proj"]])
    q, k, v = (y[nm].to(x.dtype) for nm in ("q_proj", "k_proj", "v_proj"))
    rep = q.shape[-1] // k.shape[-1]
    a = q + (k * v).repeat_interleave(rep, dim=-1)
    products(("o_proj",), a.contiguous(), [y["o_proj"]])
    x = x + y["o_proj"].to(x.dtype)
    h = rms(x).contiguous()
    products(("gate_proj", "up_proj"), h, [y["gate_proj"], y["up_proj"]])
    g, u = (y[nm].to(x.dtype) for nm in ("gate_proj", "up_proj"))
    products(("down_proj",), (F.silu(g) * u).contiguous(), [y["down_proj"]])
    x = x + y["down_proj"].to(x.dtype)
    return x


def fused_model_forward(x, blocks: Sequence[DF11BlockBatch]):
    """fused_block_forward over every block in order."""
    for blk in blocks:
        x = fused_block_forward(x, blk)
    return x


class CapturedForward:
    """A forward captured once into a HIP graph and replayed.

    At a few tokens a forward is many small launches (per block: the
    products, or decodes and products, plus norms, activations and residual
    adds); a graph replay issues all of them at once.  forward(x) must run on
    the current stream and keep its shapes: this wrapper runs it `warmup`
    times on a side stream (so that launch-time queries, torch's allocations
    and the decode tables' caches are settled), then captures one call into a
    graph that reads a static copy of x and writes a static output.
    __call__(x) copies x in, replays, and returns that output, which the next
    call overwrites.  Every DF11 kernel launches without memsets or host
    synchronisation and leaves its work counters zero, so replays are
    independent.  The forward's own buffers (weights, BlockDecoder scratch)
    must stay alive as long as this object."""

    def __init__(self, forward, example_x, warmup: int = 2):
        import torch
        self._forward = forward
        self.x = example_x.clone()
        side = torch.cuda.Stream(self.x.device)
        side.wait_stream(torch.cuda.current_stream(self.x.device))
        with torch.cuda.stream(side):
            for _ in range(warmup):
                forward(self.x)
        torch.cuda.current_stream(self.x.device).wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.y = forward(self.x)

    def __call__(self, x):
        if x.shape != self.x.shape or x.dtype != self.x.dtype:
            raise ValueError("a captured forward takes inputs of the captured shape and dtype")
        self.x.copy_(x)
        self.graph.replay()
        return self.y


def model_forward(x, blocks: Union[BlockDecoder, List[Dict]], operators: bool = False):
    """Run block_forward over every block in order, taking the weights from a
    BlockDecoder (compressed) or from a list of dicts (resident BF16)."""
    items = iter(blocks) if isinstance(blocks, BlockDecoder) else enumerate(blocks)
    for _, w in items:
        x = block_forward(x, w, operators=operators)
    return x
