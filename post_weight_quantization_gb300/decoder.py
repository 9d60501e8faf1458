"""One attention block of a quantized decoder, with the serving operators as they are used together:
packed q, k, v and o projections with per-token adapters, head norms with the rotation, the 4-bit
paged cache and attention over it. `Attention.forward` takes the new tokens of a batch of sequences,
whole prompts, pieces of them and single tokens alike.

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


if __name__ == "__main__":
    main()
