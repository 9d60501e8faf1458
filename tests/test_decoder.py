"""The attention block that runs the serving operators together, and the batch of sequences that
feeds it.

Tolerance: the block rounds q, k, v and the attention's output to bf16 where the oracle does not. A
rounding moves a value by at most 2^-8 of itself, which moves a cached code by one step (a fifteenth
of a row's range, about a third of its standard deviation) with a probability of at most 2^-8 * 15 *
|x| / range, about 3 %: a relative error of at most sqrt(0.03) / 3 = 0.06 in k and v, and of a few
2^-8 besides. The outputs' relative error in the Euclidean norm is to be at most 0.08.
"""
import numpy as np
import pytest
import torch

from oracle import gptq_oracle as orc
from oracle import serving_oracle as so


@pytest.fixture(scope="module")
def dec():
    from post_weight_quantization_gb300 import build as b
    b.build()
    from post_weight_quantization_gb300 import decoder
    return decoder


def test_batch_places(dec):
    batch = dec.Batch(10, 4, device="cpu")
    assert [batch.add() for _ in range(3)] == [0, 1, 2]
    step = batch.extend([5, 0, 4])
    assert step.cu_q.tolist() == [0, 5, 5, 9] and step.kv_lens.tolist() == [5, 0, 4] and step.max_q == 5
    assert step.positions.tolist() == [0, 1, 2, 3, 4, 0, 1, 2, 3]
    step = batch.extend([1, 2, 1])
    assert step.positions.tolist() == [5, 0, 1, 4] and step.kv_lens.tolist() == [6, 2, 5] and step.max_q == 2
    slots = [t[j // 4] * 4 + j % 4 for t, n in zip(batch.tables, batch.lens) for j in range(n)]
    assert len(set(slots)) == 13 and max(slots) < 40
    assert step.slots.tolist() == [batch.tables[0][1] * 4 + 1, batch.tables[1][0] * 4, batch.tables[1][0] * 4 + 1,
                                   batch.tables[2][1] * 4]
    assert [len(t) for t in batch.tables] == [2, 1, 2] and step.block_table.shape == (3, 2)
    for b, t in enumerate(batch.tables):
        assert step.block_table[b, :len(t)].tolist() == t


def test_batch_refusals_and_release(dec):
    batch = dec.Batch(3, 4, device="cpu")
    batch.add()
    batch.add()
    batch.extend([4, 4])
    lens, tables, free = list(batch.lens), [list(t) for t in batch.tables], list(batch.free)
    with pytest.raises(MemoryError):
        batch.extend([1, 5])
    with pytest.raises(ValueError):
        batch.extend([1])
    with pytest.raises(ValueError):
        batch.extend([1, -1])
    assert (batch.lens, batch.tables, batch.free) == (lens, tables, free)
    batch.release(0)
    assert batch.lens == [0, 4] and len(batch.free) == 2
    step = batch.extend([8, 0])
    assert step.kv_lens.tolist() == [8, 4] and not batch.free and step.slots.tolist() != []


def f64(t):
    return t.detach().cpu().double().numpy()


def _oracle(block, X, which, lens):
    """The block over whole sequences at once, in 64 bits."""
    c = block.cache
    def project(name, x, ids):
        q = getattr(block, name)
        words = q.qweight.cpu().numpy().view(np.uint32)
        A, B = (f64(t) for t in block.adapters[name])
        return so.adapter_linear(x, words, f64(q.scales), f64(q.zeros), q.bits, q.group_size, A, B, ids, f64(block.alpha))
    out = []
    for x, a in zip(X, which):
        x, ids, pos, n = f64(x), [a] * len(x), np.arange(len(x)), len(x)
        q, k, v = (project(name, x, ids).reshape(n, -1, c.head_dim) for name in "qkv")
        cos, sin = f64(block.cos), f64(block.sin)
        q = so.norm_rope(q, pos, cos, sin, f64(block.wq), block.eps)
        k = so.norm_rope(k, pos, cos, sin, f64(block.wk), block.eps)
        kv = [[], []]
        for i, rows in enumerate((k, v)):
            for h in range(c.n_kv_heads):
                got = [so.quantize_row(r) for r in rows[:, h]]
                kv[i].append(np.array([cd * float(s) + float(lo) for cd, s, lo in got]))
        G = block.heads // c.n_kv_heads
        o = np.stack([so.attention(q[:, h], kv[0][h // G], kv[1][h // G], 0, c.head_dim ** -0.5, True, block.window)[0]
                      for h in range(block.heads)], axis=1)
        out.append(project("o", o.reshape(n, -1), ids))
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("hidden,heads,kv_heads,dim,page,window", [(512, 8, 2, 64, 16, 0), (384, 3, 3, 128, 64, 20),
                                                                   (256, 16, 1, 64, 32, 0)])
def test_block_prompts_then_tokens(dec, hidden, heads, kv_heads, dim, page, window):
    """Prompts of several lengths, a piece more for some, then tokens one by one."""
    block = dec.random_block(hidden, heads, kv_heads, dim, num_pages=40, page_size=page, positions=200, adapters=2, rank=8,
                             seed=hidden)
    block.window = window
    rounds = [[100, 1, 37, 0], [30, 2, 0, 5], [1, 1, 1, 1], [1, 1, 1, 1]]
    which = [0, -1, 1, 0]
    batch = dec.Batch(40, page)
    for _ in which:
        batch.add()
    gen = torch.Generator().manual_seed(1)
    X, Y = [[] for _ in which], [[] for _ in which]
    for new in rounds:
        xs = [torch.randn((n, hidden), generator=gen).bfloat16() for n in new]
        ids = torch.tensor([a for a, n in zip(which, new) for _ in range(n)], dtype=torch.int32).cuda()
        y = block.forward(torch.cat(xs).cuda(), batch.extend(new), ids)
        for b, part in enumerate(y.split(new)):
            X[b].append(xs[b])
            Y[b].append(part)
    torch.cuda.synchronize()
    from post_weight_quantization_gb300 import gptq
    gptq.gptq_device_check()
    want = _oracle(block, [torch.cat(x) for x in X], which, rounds)
    for got, ref in zip(Y, want):
        err = np.linalg.norm(f64(torch.cat(got)) - ref) / np.linalg.norm(ref)
        assert err <= 0.08, err


@pytest.mark.gpu
def test_block_in_a_graph(dec):
    """Single tokens through a captured graph: the bits of the calls, step after step."""
    block = dec.random_block(256, 8, 2, 64, num_pages=24, page_size=16, positions=100, adapters=2, rank=8)
    which = torch.tensor([1, -1, 0], dtype=torch.int32).cuda()
    gen = torch.Generator().manual_seed(2)
    prompt = torch.randn((60, 256), generator=gen).bfloat16().cuda()
    tokens = [torch.randn((3, 256), generator=gen).bfloat16().cuda() for _ in range(20)]
    def start():
        batch = dec.Batch(24, 16)
        for _ in which:
            batch.add()
        step = batch.extend([40, 17, 3])
        block.forward(prompt, step, torch.repeat_interleave(which, torch.tensor([40, 17, 3]).cuda()))
        return [batch.extend([1, 1, 1], 6) for _ in tokens]
    want = [block.forward(X, step, which) for X, step in zip(tokens, start())]
    steps = start()
    X, at = tokens[0].clone(), dec.Step(steps[0].slots.clone(), steps[0].ints.clone(), 3, 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y = block.forward(X, at, which)
    for x, step, ref in zip(tokens, steps, want):
        X.copy_(x)
        at.copy_(step)
        graph.replay()
        assert torch.equal(Y, ref)
    with pytest.raises(ValueError):
        at.copy_(dec.Step(at.slots, at.ints, 3, 2))


@pytest.mark.gpu
def test_example_runs(dec, capsys):
    dec.main()
    out = capsys.readouterr().out
    assert "us a step" in out and "nan" not in out


@pytest.mark.gpu
def test_empty_step(dec):
    """A step without new tokens, one without sequences, and the next one as if it had not been."""
    block = dec.random_block(256, 4, 2, 64, num_pages=8, page_size=16, positions=50, adapters=2, rank=8)
    gen = torch.Generator().manual_seed(3)
    X = [torch.randn((n, 256), generator=gen).bfloat16().cuda() for n in (20, 2)]
    outs = []
    for empty in (False, True):
        batch = dec.Batch(8, 16)
        if empty:
            assert block.forward(X[0][:0], batch.extend([])).shape == (0, 256)
        for _ in range(2):
            batch.add()
        ids = torch.zeros(20, dtype=torch.int32, device="cuda")
        outs.append([block.forward(X[0], batch.extend([15, 5]), ids)])
        if empty:
            for some in (None, ids[:0]):
                Y = block.forward(X[0][:0], batch.extend([0, 0]), some)
                assert Y.shape == (0, 256) and Y.dtype == torch.bfloat16
        outs[-1].append(block.forward(X[1], batch.extend([1, 1]), ids[:2]))
    torch.cuda.synchronize()
    from post_weight_quantization_gb300 import gptq
    gptq.gptq_device_check()
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_copy_refuses_steps_of_other_shapes(dec):
    """... before it writes anything: another number of tokens, sequences, pages or most new tokens."""
    def step(new, width=3):
        batch = dec.Batch(20, 4, device="cpu")
        for _ in new:
            batch.add()
        return batch.extend(new, width)
    at = step([1, 1, 1])
    slots, ints = at.slots.clone(), at.ints.clone()
    for other in (step([1, 0, 0]), step([1, 1, 0]), step([1, 1, 1, 1]), step([1, 1, 1], 4), step([2, 1, 0])):
        with pytest.raises(ValueError):
            at.copy_(other)
        assert torch.equal(at.slots, slots) and torch.equal(at.ints, ints)
    other = step([0, 0, 0])
    same = dec.Step(slots + 5, ints + 1, 3, 1)
    with pytest.raises(ValueError):
        at.copy_(other)
    assert torch.equal(at.copy_(same).slots, slots + 5) and torch.equal(at.ints, ints + 1)
