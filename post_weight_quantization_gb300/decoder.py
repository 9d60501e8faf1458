"""A quantized decoder, with the serving operators as they are used together. `Attention`: packed q, k, v
and o projections with per-token adapters, head norms with the rotation, the 4-bit paged cache and
attention over it. `Layer`: the norms with the residual stream around it and the gated MLP, whose
tokens may be 8-bit ones. `Decoder`: embedding, layers, the head's logits and the choice of the next
token. Each takes the new tokens of a batch of sequences, whole prompts, pieces of them and single
tokens alike.

    python -m post_weight_quantization_gb300.decoder        # prompts, then tokens one by one
"""
from dataclasses import dataclass, field
from typing import Dict, List, Optional, Tuple

import torch

from . import gptq


class Batch:
    """Running sequences and the pages that hold them: `lens` tokens each, `tables[b]` their pages in
    order. `extend` finds places for new tokens and lays out what the operators read."""

    def __init__(self, num_pages: int, page_size: int, device="cuda"):
        self.page_size, self.device = page_size, torch.device(device)
        self.free: List[int] = list(range(num_pages))[::-1]
        self.lens: List[int] = []
        self.tables: List[List[int]] = []

    def add(self) -> int:
        """A new sequence without tokens; returns its number."""
        self.lens.append(0)
        self.tables.append([])
        return len(self.lens) - 1

    def release(self, b: int) -> None:
        """Give the pages of sequence b back; its number stays, with no tokens."""
        self.free += self.tables[b][::-1]
        self.lens[b], self.tables[b] = 0, []

    def extend(self, new: List[int], width: int = 0) -> "Step":
        """Places for new[b] more tokens of each sequence b; the table of pages has at least `width`
        columns. Raises MemoryError, with nothing changed, when there are not enough free pages."""
        if len(new) != len(self.lens) or min(new, default=0) < 0:
            raise ValueError(f"one count per sequence, none negative: {len(self.lens)} sequences, got {new}")
        p = self.page_size
        need = [-(-(n + k) // p) - len(t) for n, k, t in zip(self.lens, new, self.tables)]
        if sum(need) > len(self.free):
            raise MemoryError(f"{sum(need)} pages needed, {len(self.free)} free")
        slots, positions, cu = [], [], [0]
        for b, k in enumerate(new):
            self.tables[b] += [self.free.pop() for _ in range(need[b])]
            places = range(self.lens[b], self.lens[b] + k)
            positions += places
            slots += [self.tables[b][j // p] * p + j % p for j in places]
            self.lens[b] += k
            cu.append(cu[-1] + k)
        width = max([len(t) for t in self.tables] + [1, width])
        table = [t + [0] * (width - len(t)) for t in self.tables]
        # one copy for the 32-bit numbers of a step
        ints = torch.tensor(positions + cu + self.lens + sum(table, []), dtype=torch.int32).to(self.device)
        return Step(torch.tensor(slots, dtype=torch.int64).to(self.device), ints, len(new), max(new, default=0))


class Step:
    """What a step's operators read beside the tokens: slots (T,) int64, the new tokens' places in the
    cache; positions (T,), cu_q (batch + 1,), kv_lens (batch,), the new tokens included, and
    block_table (batch, pages), all int32; max_q, the most new tokens of a sequence."""

    def __init__(self, slots: torch.Tensor, ints: torch.Tensor, batch: int, max_q: int):
        T = slots.shape[0]
        self.slots, self.ints, self.max_q = slots, ints, max_q
        self.positions, self.cu_q, self.kv_lens, table = ints.split([T, batch + 1, batch, ints.shape[0] - T - 2 * batch - 1])
        self.block_table = table.view(batch, table.shape[0] // max(batch, 1))

    def copy_(self, other: "Step") -> "Step":
        """Take over a step of the same shape in place, for a captured graph that reads this one."""
        shape = lambda s: (s.max_q, s.slots.shape, s.block_table.shape)
        if shape(self) != shape(other):
            raise ValueError("the steps have different shapes")
        self.slots.copy_(other.slots)
        self.ints.copy_(other.ints)
        return self


@dataclass
class Attention:
    """The block: packed projections (q, k, v: hidden -> heads; o: heads -> hidden), adapters by
    projection as (A, B) with one alpha per adapter, norm weights, rotation tables, cache."""
    q: gptq.QuantizedLayer
    k: gptq.QuantizedLayer
    v: gptq.QuantizedLayer
    o: gptq.QuantizedLayer
    heads: int
    cache: gptq.KVCache
    cos: torch.Tensor
    sin: torch.Tensor
    wq: Optional[torch.Tensor] = None
    wk: Optional[torch.Tensor] = None
    eps: float = 1e-6
    window: int = 0
    alpha: Optional[torch.Tensor] = None
    adapters: Dict[str, Tuple[torch.Tensor, torch.Tensor]] = field(default_factory=dict)

    def _project(self, name: str, X, m: int, ids, Y=None):
        A, B = self.adapters.get(name, (None, None))
        if A is None or ids is None:
            return gptq.gptq_adapter_linear(getattr(self, name), X, m, Y=Y, out_bf16=True)
        return gptq.gptq_adapter_linear(getattr(self, name), X, m, A, B, ids, self.alpha, Y=Y, out_bf16=True)

    def forward(self, X: torch.Tensor, step: Step, ids: Optional[torch.Tensor] = None) -> torch.Tensor:
        """X (T, hidden) bf16, the new tokens of all sequences one after another; ids (T,) int32, each
        token's adapter (negative: none). Appends their keys and values and returns the block's
        output (T, hidden) bf16."""
        c, T = self.cache, X.shape[0]
        nq, nk = self.heads * c.head_dim, c.n_kv_heads * c.head_dim
        qkv = torch.empty((T, nq + 2 * nk), dtype=torch.bfloat16, device=X.device)
        parts = qkv.split([nq, nk, nk], dim=1)
        for name, Y in zip("qkv", parts):
            self._project(name, X, Y.shape[1], ids, Y)
        Q, K, V = (Y.view(T, Y.shape[1] // c.head_dim, c.head_dim) for Y in parts)
        gptq.gptq_qk_norm_rope(Q, K, step.positions, self.cos, self.sin, self.wq, self.wk, self.eps, Q_out=Q, K_out=K)
        gptq.gptq_kv_append(c, K, V, step.slots)
        O = gptq.gptq_kv_attention(c, Q, step.cu_q, step.kv_lens, step.block_table, step.max_q, window=self.window)
        return self._project("o", O.view(T, nq), X.shape[1], ids)


@dataclass
class Layer:
    """A decoder layer: norm, attention, norm, gated MLP, the residual stream beside them in bf16. gate and up
    (hidden -> wide) and down (wide -> hidden) are packed layers; w_attn and w_mlp the norms' weights. With
    `eight_bit` the MLP's tokens are e4m3 with a scale each (up to 4-bit layers are read as such for many)."""
    attention: Attention
    gate: gptq.QuantizedLayer
    up: gptq.QuantizedLayer
    down: gptq.QuantizedLayer
    w_attn: torch.Tensor
    w_mlp: torch.Tensor
    act: str = "silu"
    eps: float = 1e-6
    eight_bit: bool = False

    def mlp(self, X: torch.Tensor, scale: Optional[torch.Tensor], residual: torch.Tensor) -> torch.Tensor:
        """down(act(gate(x)) * up(x)) + residual for normed tokens X, bf16 or e4m3 with their scale."""
        wide = self.gate.qweight.shape[0]
        U = gptq.gptq_linear(self.up, X, wide, x_scale=scale, out_bf16=True)
        H = gptq.gptq_linear(self.gate, X, wide, x_scale=scale, act=self.act, mul=U, Y=U, out_bf16=True)
        return gptq.gptq_linear(self.down, H, residual.shape[1], residual=residual, out_bf16=True)

    def forward(self, X: torch.Tensor, step: Step, ids: Optional[torch.Tensor] = None) -> torch.Tensor:
        """X (T, hidden) bf16, the residual stream of the new tokens; returns it behind the layer."""
        N, _, _ = gptq.gptq_add_rms_norm(X, None, self.w_attn, eps=self.eps)
        A = self.attention.forward(N, step, ids)
        N, R, scale = gptq.gptq_add_rms_norm(A, X, self.w_mlp, eps=self.eps, R_out=A,
                                             out_dtype=torch.float8_e4m3fn if self.eight_bit else torch.bfloat16)
        return self.mlp(N, scale, R)


@dataclass
class Decoder:
    """Embedding (vocab, hidden) bf16, layers, the last norm's weights and the packed head (hidden -> vocab)."""
    embedding: torch.Tensor
    layers: List[Layer]
    w: torch.Tensor
    head: gptq.QuantizedLayer
    eps: float = 1e-6

    def logits(self, tokens: torch.Tensor, step: Step, ids: Optional[torch.Tensor] = None) -> torch.Tensor:
        """tokens (T,) int32 or int64, the new tokens of all sequences one after another; returns (batch, vocab)
        float32, the logits behind each sequence's last new token (of no meaning for a sequence without one). A
        token outside the vocabulary, such as the -1 of a row that could not be drawn from, has NaN for its
        embedding: the logits of its sequence are NaN, its next token is -1, and no other sequence is touched."""
        inside = tokens.clamp(0, self.embedding.shape[0] - 1)
        X = self.embedding.index_select(0, inside).masked_fill_((tokens != inside)[:, None], float("nan"))
        for layer in self.layers:
            X = layer.forward(X, step, ids)
        last = (step.cu_q[1:] - 1).clamp(min=0)
        last = X.index_select(0, last) if X.shape[0] else X.new_zeros((last.shape[0], X.shape[1]))
        N, _, _ = gptq.gptq_add_rms_norm(last, None, self.w, eps=self.eps)
        return gptq.gptq_linear(self.head, N, self.embedding.shape[0])

    def forward(self, tokens: torch.Tensor, step: Step, u: torch.Tensor, ids: Optional[torch.Tensor] = None,
                **settings: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
        """The next token of each sequence and its log probability; u and `settings` (temperature, top_k, top_p,
        min_p) as gptq_sample takes them, one number per sequence."""
        return gptq.gptq_sample(self.logits(tokens, step, ids), u, **settings)


def rotation_tables(n: int, dim: int, base: float = 10000.0, device="cuda"):
    """cos and sin (n, dim / 2) float32 of position * base^(-2 i / dim)."""
    freq = base ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    a = torch.arange(n, dtype=torch.float64)[:, None] * freq
    return a.cos().float().to(device), a.sin().float().to(device)


def random_block(hidden: int, heads: int, kv_heads: int, head_dim: int, num_pages: int, page_size: int = 64,
                 positions: int = 4096, bits: int = 4, group_size: int = 128, adapters: int = 0, rank: int = 16,
                 tokens: int = 512, seed: int = 0) -> Attention:
    """A block of random weights, quantized on random calibration tokens."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape, scale=1.0: scale * torch.randn(shape, generator=gen, device="cuda")
    shapes = {"q": (heads * head_dim, hidden), "k": (kv_heads * head_dim, hidden), "v": (kv_heads * head_dim, hidden),
              "o": (hidden, heads * head_dim)}
    layers, pairs = {}, {}
    for name, (m, d) in shapes.items():
        layers[name] = gptq.quantize_layer(rand(m, d, scale=d ** -0.5), [rand(tokens, d).bfloat16()], bits=bits,
                                           group_size=group_size)[0]
        if adapters:
            pairs[name] = (rand(adapters, rank, d, scale=d ** -0.5).bfloat16(), rand(adapters, m, rank, scale=0.1).bfloat16())
    cos, sin = rotation_tables(positions, head_dim)
    return Attention(heads=heads, cache=gptq.KVCache.empty(num_pages, page_size, kv_heads, head_dim), cos=cos, sin=sin,
                     wq=1 + rand(head_dim, scale=0.1), wk=1 + rand(head_dim, scale=0.1), adapters=pairs,
                     alpha=torch.linspace(0.5, 1.5, adapters, device="cuda") if adapters else None, **layers)


def random_decoder(vocab: int, hidden: int, wide: int, layers: int, heads: int, kv_heads: int, head_dim: int, num_pages: int,
                   page_size: int = 64, bits: int = 4, group_size: int = 128, eight_bit: bool = False, tokens: int = 512,
                   seed: int = 0, **block) -> Decoder:
    """A decoder of random weights, quantized on random calibration tokens (the head at 8 bits)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape, scale=1.0: scale * torch.randn(shape, generator=gen, device="cuda")

    def packed(m, d, b):
        return gptq.quantize_layer(rand(m, d, scale=d ** -0.5), [rand(tokens, d).bfloat16()], bits=b, group_size=group_size)[0]

    stack = []
    for i in range(layers):
        attention = random_block(hidden, heads, kv_heads, head_dim, num_pages, page_size, bits=bits, group_size=group_size,
                                 tokens=tokens, seed=seed + 1 + i, **block)
        stack.append(Layer(attention, packed(wide, hidden, bits), packed(wide, hidden, bits), packed(hidden, wide, bits),
                           1 + rand(hidden, scale=0.1), 1 + rand(hidden, scale=0.1), eight_bit=eight_bit))
    return Decoder(rand(vocab, hidden).bfloat16(), stack, 1 + rand(hidden, scale=0.1), packed(vocab, hidden, 8))


def run_decoder(steps: int = 32) -> None:
    """Prompts through a decoder of two layers, then tokens drawn one by one, by calls and by a captured graph."""
    model = random_decoder(32000, 4096, 11008, 2, heads=32, kv_heads=8, head_dim=128, num_pages=256, eight_bit=True)
    batch = Batch(256, 64)
    lens = [1500, 700, 331, 1]
    for _ in lens:
        batch.add()
    n = len(lens)
    gen = torch.Generator(device="cuda").manual_seed(0)
    rows = lambda v, dtype=torch.float32: torch.full((n,), v, dtype=dtype, device="cuda")
    settings = dict(temperature=rows(0.8), top_k=rows(50, torch.int32), top_p=rows(0.95))
    u = torch.rand((2 * steps + 1, n), generator=gen, device="cuda")
    tokens = torch.randint(0, 32000, (sum(lens),), generator=gen, device="cuda", dtype=torch.int32)
    step = batch.extend(lens)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    model.forward(tokens, step, u[0], **settings)          # again below: the same tokens into the same places
    start.record()
    token, _ = model.forward(tokens, step, u[0], **settings)
    end.record()
    torch.cuda.synchronize()
    prompts = start.elapsed_time(end) * 1e3
    width = len(batch.free) // n
    plans = [batch.extend([1] * n, width) for _ in range(2 * steps)]
    out = [token]
    torch.cuda.synchronize()
    start.record()
    for i, plan in enumerate(plans[:steps]):
        out.append(model.forward(out[-1], plan, u[1 + i], **settings)[0])
    end.record()
    torch.cuda.synchronize()
    calls = start.elapsed_time(end) * 1e3 / steps
    at, token, v = plans[steps], out[-1].clone(), u[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        drawn, _ = model.forward(token, at, v, **settings)
    start.record()
    for i, plan in enumerate(plans[steps:]):
        at.copy_(plan)
        v.copy_(u[1 + steps + i])
        graph.replay()
        token.copy_(drawn)
        out.append(drawn.clone())
    end.record()
    torch.cuda.synchronize()
    replays = start.elapsed_time(end) * 1e3 / steps
    gptq.gptq_device_check()
    print(f"decoder of 2 layers, prompts {lens}: {prompts:.0f} us; {2 * steps} tokens of each sequence: {calls:.0f} us a step by calls, "
          f"{replays:.0f} us by a graph; the first sequence's begin {[int(t[0]) for t in out[:6]]}")


def main() -> None:
    block = random_block(hidden=4096, heads=32, kv_heads=8, head_dim=128, num_pages=256, adapters=4, rank=16)
    batch = Batch(256, block.cache.page_size)
    lens, steps = [1500, 700, 331, 1], 64
    for _ in lens:
        batch.add()
    seq = torch.arange(len(lens), dtype=torch.int32, device="cuda")
    which = seq - 1                              # sequence 0 has no adapter
    X = torch.randn((sum(lens), 4096), device="cuda").bfloat16()
    step = batch.extend(lens)
    ids = torch.repeat_interleave(which, torch.tensor(lens, device="cuda")).int()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    block.forward(X, step, ids)                  # again below: the same tokens into the same places
    start.record()
    Y = block.forward(X, step, ids)
    end.record()
    torch.cuda.synchronize()
    print(f"prompts {lens}: {start.elapsed_time(end) * 1e3:.0f} us, mean |y| {Y.float().abs().mean().item():.4f}")
    last = (step.cu_q[1:] - 1).long()
    X = Y[last]
    width = len(batch.free) // len(lens)
    plans = [batch.extend([1] * len(lens), width) for _ in range(2 * steps)]
    torch.cuda.synchronize()
    start.record()
    for plan in plans[:steps]:
        X = block.forward(X, plan, which)
    end.record()
    torch.cuda.synchronize()
    calls = start.elapsed_time(end) * 1e3 / steps
    # the same as one captured graph, whose tokens, places and lengths are copied into it
    at = plans[steps]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y = block.forward(X, at, which)
    start.record()
    for plan in plans[steps:]:
        at.copy_(plan)
        graph.replay()
        X.copy_(Y)
    end.record()
    torch.cuda.synchronize()
    replays = start.elapsed_time(end) * 1e3 / steps
    gptq.gptq_device_check()
    print(f"{2 * steps} tokens of each sequence, one by one: {calls:.0f} us a step by calls, {replays:.0f} us by a graph, "
          f"mean |y| {X.float().abs().mean().item():.4f}")
    run_decoder()


if __name__ == "__main__":
    main()
