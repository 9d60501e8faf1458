"""Packed projections whose CTAs take several tiles one after another, so that every count that a tile hands to the next one is
used: places of slabs and codes, which set of warps has which slab, batches of scales and zeros, rows that end in a half block.

Tolerances as for the operator's other tests, against 64 bits on the GPU: z is off by (unit + G + 2) 2^-23 sum |x w|, G sums of
`unit` columns; a token's scale adds 2 roundings, bias, gate and residual one each; silu and relu have a slope of at most 1.1, and the
exponential and the quotient add (16 + 4 |z|) 2^-23 |act|; the output's rounding is half a unit in its last place.
"""
import math

import numpy as np
import pytest
import torch

from oracle import gptq_oracle as orc

pytestmark = pytest.mark.gpu

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def g():
    from post_weight_quantization_gb300 import build as b
    b.build()
    from post_weight_quantization_gb300 import gptq
    return gptq


def layer(g, rng, m, d, bits, group):
    G = 1 if group == -1 else d // group
    gs = d // G
    codes = rng.integers(0, 2 ** bits, (m, d))
    words = torch.from_numpy(orc.pack_codes(codes, bits).astype(np.uint32).view(np.int32)).cuda()
    scales = torch.from_numpy(((0.5 + rng.random((m, G))) * 4 / 2 ** bits / math.sqrt(d)).astype(np.float32)).cuda()
    zeros = torch.from_numpy(rng.integers(0, 2 ** bits, (m, G)).astype(np.float32)).cuda()
    W = (torch.from_numpy(codes).cuda().double() - zeros.double().repeat_interleave(gs, 1)) * scales.double().repeat_interleave(gs, 1)
    return g.QuantizedLayer(words, scales, zeros, None, bits, group, d), W


def tokens(rng, T, d, eight):
    x = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).cuda()
    if not eight:
        return x.bfloat16(), None, x.bfloat16().double()
    xs = x.abs().amax(1) / 448
    x = (x / xs[:, None]).clamp(-448, 448).to(E4M3)
    return x, xs, x.double() * xs.double()[:, None]


def check(W, X, d, group, eight, bias, act, mul, res, Y):
    gs = d if group == -1 else group
    unit = 128 if gs % 128 == 0 else 64 if gs % 64 == 0 else 32
    z = X @ W.T
    err = (unit + -(-d // unit) + 2) * 2.0 ** -23 * (X.abs() @ W.abs().T)
    if eight:
        err += 2.0 ** -23 * z.abs()
    if bias is not None:
        z = z + bias.double()
        err += 2.0 ** -23 * (z.abs() + bias.double().abs())
    y = z * torch.sigmoid(z) if act == "silu" else z.clamp(min=0) if act == "relu" else z
    if act == "silu":
        err = 1.1 * err + (16 + 4 * z.abs()) * 2.0 ** -23 * y.abs()
    if mul is not None:
        y = y * mul.double()
        err = err * mul.double().abs() + 2.0 ** -23 * y.abs()
    if res is not None:
        y = y + res.double()
        err += 2.0 ** -23 * y.abs()
    bound = err + U[Y.dtype] * (1 + 2.0 ** -8) * y.abs() + 1e-37
    off = (Y.double() - y).abs() / bound
    assert bool((off <= 1).all()), (float(off.max()), [tuple(i) for i in (off > 1).nonzero()[:5].tolist()], int((off > 1).sum()))


def run(g, rng, T, m, d, bits, group, eight, act, out, bias=False, mul=False, res=False):
    q, W = layer(g, rng, m, d, bits, group)
    x, xs, X = tokens(rng, T, d, eight)
    b = torch.from_numpy(rng.standard_normal(m).astype(np.float32)).cuda() if bias else None
    a = torch.randn((T, m), device="cuda").to(out) if mul else None
    r = torch.randn((T, m), device="cuda").to(out) if res else None
    n = g.gptq_launch_count()
    Y = g.gptq_linear(q, x, m, x_scale=xs, bias=b, act=act, mul=a, residual=r, out_bf16=out is torch.bfloat16)
    n = g.gptq_launch_count() - n
    torch.cuda.synchronize()
    g.gptq_device_check()
    check(W, X, d, group, eight, b, act, a, r, Y)
    return n


# 20 x 17 tiles: three one after another on a CTA. An odd number of blocks, rows that end in a quarter, half and three quarters
# of a block, one block, half a block; whole rows as a group
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("d,bits,group", [(640, 4, 128), (1152, 4, 128), (320, 4, 64), (448, 4, 64), (416, 4, 32), (480, 4, 32), (96, 4, 32),
                                          (64, 4, 64), (1056, 4, -1), (1088, 4, -1), (128, 4, 128),
                                          (640, 3, 128), (320, 3, 64), (416, 3, 32), (128, 3, -1), (448, 3, -1),
                                          (640, 2, 128), (448, 2, 64), (416, 2, 32), (192, 2, -1), (1216, 2, 64),
                                          (640, 8, 128), (320, 8, 64), (416, 8, 32), (384, 8, -1), (224, 8, -1)])
def test_three_tiles_of_a_cta(g, d, bits, group, eight):
    rng = np.random.default_rng(d * 10 + bits)
    run(g, rng, 4200, 2500, d, bits, group, eight, ("none", "silu", "relu")[(d // 32 + bits) % 3], torch.bfloat16 if d % 128 else torch.float32,
        bias=bits % 2 == 0, mul=d % 3 == 0, res=eight)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("d,bits,group", [(320, 4, 64), (384, 4, 128), (96, 4, 32), (320, 3, 64), (96, 2, 32), (192, 8, 64)])
def test_many_tiles_of_a_cta(g, d, bits, group, eight):
    """51 x 20 tiles: seven one after another."""
    rng = np.random.default_rng(d + bits)
    run(g, rng, 13000, 2500, d, bits, group, eight, "none", torch.bfloat16)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("T", [66, 128, 200, 256])
@pytest.mark.parametrize("d,bits,group", [(640, 4, 128), (320, 4, 64), (640, 3, 128), (448, 2, 64), (640, 8, 128)])
def test_one_tile_of_tokens(g, T, d, bits, group, eight):
    """Up to 256 tokens of a wide layer: the tiles' kernel, which takes up to 4 bits with 8-bit tokens by one launch."""
    rng = np.random.default_rng(T + d + bits)
    n = run(g, rng, T, 11007, d, bits, group, eight, "silu", torch.bfloat16, mul=True)
    assert n == (2 if eight and bits == 8 else 1)


@pytest.mark.parametrize("eight", [False, True])
def test_long_rows_repeat_themselves(g, eight):
    """The same input gives the same bits, pass after pass, with another between: 64 x 24 tiles of 32 blocks."""
    rng = np.random.default_rng(7)
    q, _ = layer(g, rng, 8192, 4096, 4, 128)
    a, b = tokens(rng, 6000, 4096, eight), tokens(rng, 6000, 4096, eight)
    call = lambda t: g.gptq_linear(q, t[0], 8192, x_scale=t[1], out_bf16=True)
    want = call(a)
    for _ in range(20):
        call(b)
        assert torch.equal(call(a), want)
    g.gptq_device_check()


# 20 x 20 tiles of 256 tokens with adapters: runs of one adapter's tokens in every number, so that a tile has an odd or an even
# number of blocks more; ranks of one block and of two, rows of an odd number of blocks. U = alpha A x has d products of fp32 sums,
# then enters as two bf16 parts (2^-16), with `rank` products more.
@pytest.mark.parametrize("call", ["adapter_linear", "linear"])
@pytest.mark.parametrize("d,bits,group,rank", [(640, 4, 128, 16), (512, 4, 64, 72), (384, 8, 128, 8), (416, 8, 32, 128), (640, 3, 128, 16), (320, 2, 64, 64)])
def test_three_tiles_of_a_cta_with_adapters(g, d, bits, group, rank, call):
    rng = np.random.default_rng(d + bits + rank)
    T, m, n = 5003, 2500, 7
    q, W = layer(g, rng, m, d, bits, group)
    x, _, X = tokens(rng, T, d, False)
    A = (torch.from_numpy(rng.standard_normal((n, rank, d))).cuda() * d ** -0.5).bfloat16()
    B = (torch.from_numpy(rng.standard_normal((n, m, rank))).cuda() * rank ** -0.5).bfloat16()
    alpha = torch.from_numpy((0.5 + rng.random(n)).astype(np.float32)).cuda()
    runs = rng.choice([1, 17, 90, 200, 256, 700], 400)
    ids = torch.from_numpy(np.repeat(rng.integers(-1, n, 400), runs)[:T].astype(np.int32)).cuda()
    z, mag = X @ W.T, X.abs() @ W.abs().T
    unit = 128 if group % 128 == 0 else 64 if group % 64 == 0 else 32
    err = (unit + -(-d // unit) + 2) * 2.0 ** -23 * mag
    for a in range(n):
        at = (ids == a).nonzero()[:, 0]
        z[at] += alpha[a].double() * ((X[at] @ A[a].double().T) @ B[a].double().T)
        err[at] += ((d + rank) * 2.0 ** -23 + 2.0 ** -16) * alpha[a].double() * ((X[at].abs() @ A[a].double().abs().T) @ B[a].double().abs().T)
    y = z
    if call == "linear":
        res = torch.randn((T, m), device="cuda")
        Y = g.gptq_linear(q, x, m, A=A, B=B, ids=ids, alpha=alpha, act="silu", residual=res)
        y = z * torch.sigmoid(z)
        err = 1.1 * err + (16 + 4 * z.abs()) * 2.0 ** -23 * y.abs()
        y = y + res.double()
        err += 2.0 ** -23 * y.abs()
    else:
        Y = g.gptq_adapter_linear(q, x, m, A, B, ids, alpha)
    torch.cuda.synchronize()
    g.gptq_device_check()
    off = (Y.double() - y).abs() / (err + 2.0 ** -24 * y.abs() + 1e-37)
    assert bool((off <= 1).all()), (float(off.max()), (off > 1).nonzero()[:5].tolist(), int((off > 1).sum()))
