"""The serving operators against the float64 oracle: head norms with the rotation, rows of
the 4-bit cache, attention over the cache, adapters beside a packed layer. Inputs are made
on the CPU; the cache that attention reads is written by the oracle, so each operator is
checked on its own.

Tolerances (u: half a unit in the last place, relative: 2^-8 bf16, 2^-11 fp16, 2^-24 fp32):
  norm_rope   a head's mean of squares is a sum of D positive terms in at most 8 + 5 steps
              and enters as its square root, the norm, weight and rotation add at most 8
              roundings: 16 * 2^-24 * (|n_i c| + |n_j s|) + u |y|
  cache rows  bit-equal codes, scales and lowest values
  attention   a score is a sum of D exact products in fp32 (tensor-core accumulation may
              truncate: 2^-22 a step), scaled: d_s = (D + 8) 2^-22 sm_scale sum |q| (15 scale +
              |low|); the probabilities' product with the codes may round them to fp16
              (2^-11): (2^-11 + 2 max d_s + 2^-18) sum_j p_j (|v_j| + 2 |low_j|) + u |o|
  adapters    the packed layer as its own tests have it, (unit + G + 2) 2^-23 sum |x w|; the
              low-rank part in fp32 with the inner product carried as two bf16 parts:
              ((d + rank) 2^-23 + 2^-16) |alpha| |B| (|A| |x|); + u |y|
"""
import numpy as np
import pytest
import torch

from oracle import gptq_oracle as orc
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu

HALF_ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-37, torch.bfloat16: 1e-37, torch.float16: 2.0 ** -25}


@pytest.fixture(scope="module")
def g():
    from post_weight_quantization_gb300 import build as b
    b.build()
    from post_weight_quantization_gb300 import gptq
    return gptq


def f64(t):
    return t.detach().cpu().double().numpy()


def randn(rng, shape, dtype, scale=1.0):
    return torch.from_numpy(scale * rng.standard_normal(shape)).to(dtype)


def done(g):
    torch.cuda.synchronize()
    g.gptq_device_check()


# ------------------------------------------------------------------ norm and rotation
def _tables(n, rot):
    freq = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(n)[:, None] * freq
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def _check_norm_rope(x, got, positions, cos, sin, w, eps, interleaved):
    ref = so.norm_rope(f64(x), positions, cos, sin, w, eps, interleaved)
    n = np.abs(so.norm_rope(f64(x), w=w, eps=eps))
    mag = n.copy()
    if cos is not None:
        mag = so.norm_rope(n, positions, np.abs(cos), -np.abs(sin), None, eps, interleaved)
        half = cos.shape[1]
        pairs = [(2 * i, 2 * i + 1) if interleaved else (i, i + half) for i in range(half)]
        for i, (a, b) in enumerate(pairs):          # |n_j c| + |n_i s| for the second of a pair
            c, s = np.abs(cos)[positions, i][:, None], np.abs(sin)[positions, i][:, None]
            mag[..., b] = n[..., b] * c + n[..., a] * s
    bound = 16 * 2.0 ** -24 * mag + HALF_ULP[got.dtype] * np.abs(ref) * (1 + 2.0 ** -8) + TINY[got.dtype]
    assert np.all(np.abs(f64(got) - ref) <= bound), float(np.max(np.abs(f64(got) - ref) / bound))


@pytest.mark.parametrize("T,hq,hk,D,rot", [(1, 32, 32, 128, 128), (7, 64, 8, 128, 64), (33, 5, 1, 64, 64),
                                           (3, 28, 4, 256, 64), (2, 3, 2, 80, 80), (5, 2, 0, 8, 0),
                                           (4, 9, 3, 96, 32), (130, 8, 1, 16, 16), (19, 1, 1, 248, 240)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("din,dout", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
                                      (torch.float32, torch.bfloat16), (torch.float32, torch.float32),
                                      (torch.bfloat16, torch.float16)])
def test_norm_rope(g, T, hq, hk, D, rot, interleaved, din, dout):
    rng = np.random.default_rng(T * 1000 + D + rot)
    pad = 16
    qkv = randn(rng, (T, (hq + 2 * hk) * D + pad), din, 2.0).cuda()         # a fused projection's rows
    Q, K = qkv[:, :hq * D].view(T, hq, D), qkv[:, hq * D:(hq + hk) * D].view(T, hk, D)
    wq, wk = (1 + 0.2 * rng.standard_normal((2, D))).astype(np.float32)
    n_pos = 300
    pos = rng.integers(0, n_pos, T).astype(np.int32)
    cos, sin = _tables(n_pos, rot) if rot else (None, None)
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()
    Qo, Ko = g.gptq_qk_norm_rope(Q, K if hk else None, dev(pos) if rot else None, dev(cos), dev(sin), wq=dev(wq),
                                 wk=dev(wk) if hk else None, eps=1e-5, interleaved=interleaved, out_dtype=dout)
    done(g)
    _check_norm_rope(Q, Qo, pos, cos, sin, wq, 1e-5, interleaved)
    if hk:
        _check_norm_rope(K, Ko, pos, cos, sin, wk, 1e-5, interleaved)


@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (64, 32, True), (256, 256, False)])
def test_norm_rope_in_place_and_without_norm(g, D, rot, interleaved):
    rng = np.random.default_rng(D)
    T, hq, hk = 11, 6, 2
    cos, sin = _tables(64, rot)
    pos = rng.integers(0, 64, T).astype(np.int32)
    args = [torch.from_numpy(a).cuda() for a in (pos, cos, sin)]
    Q, K = randn(rng, (T, hq, D), torch.bfloat16).cuda(), randn(rng, (T, hk, D), torch.bfloat16).cuda()
    want = g.gptq_qk_norm_rope(Q, K, *args, interleaved=interleaved)
    _check_norm_rope(Q, want[0], pos, cos, sin, None, 1e-6, interleaved)
    qkv = torch.cat([Q.reshape(T, -1), K.reshape(T, -1)], dim=1).contiguous()
    q, k = qkv[:, :hq * D].view(T, hq, D), qkv[:, hq * D:].view(T, hk, D)
    g.gptq_qk_norm_rope(q, k, *args, interleaved=interleaved, Q_out=q, K_out=k)
    done(g)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_norm_rope_zero_rows_nan_and_bad_position(g):
    T, h, D = 4, 2, 128
    x = torch.zeros((T, h, D), dtype=torch.bfloat16)
    x[1] = 3.0
    x[2, 0, 5] = float("nan")
    x[3] = 1.0
    cos, sin = (torch.from_numpy(a).cuda() for a in _tables(8, D))
    w = torch.ones(D, device="cuda")
    pos = torch.tensor([0, 7, 3, 8], dtype=torch.int32, device="cuda")          # 8 is out of range
    y, _ = g.gptq_qk_norm_rope(x.cuda(), None, pos, cos, sin, wq=w)
    torch.cuda.synchronize()
    with pytest.raises(g.GPTQError) as e:
        g.gptq_device_check()
    assert e.value.status == g.GPTQ_ERR_INVALID_ARG
    g.gptq_device_check()                                                        # read once, then clear
    y = y.float().cpu()
    assert torch.all(y[0] == 0) and torch.isnan(y[2, 0]).all() and torch.isfinite(y[2, 1]).all()
    assert torch.allclose(y[3], torch.ones(h, D), atol=2.0 ** -8)                # written without rotation


# ------------------------------------------------------------------ cache rows
def _rows(rng, shape, dtype, kind):
    x = rng.standard_normal(shape)
    if kind == "offset":
        x = 0.01 * x + 5.0 * rng.standard_normal(shape[:-1])[..., None]
    elif kind == "wide":
        x = x * np.exp(8 * rng.standard_normal(shape))
    elif kind == "steps":                                                        # quotients on ties
        x = rng.integers(0, 31, shape) * 0.25 - 2.0
    x = torch.from_numpy(x).to(dtype)
    if kind == "special":
        x.view(-1, shape[-1])[0] = 0.0
        x.view(-1, shape[-1])[1] = 7.25
        x.view(-1, shape[-1])[2, 3] = float("inf")
        x.view(-1, shape[-1])[3, 1] = -float("inf")
        x.view(-1, shape[-1])[4, 0] = float("nan")
        x.view(-1, shape[-1])[5] = 1e-7
        x.view(-1, shape[-1])[6] *= 1e-6
        if dtype != torch.float16:
            x.view(-1, shape[-1])[7] *= 1e7
    return x


@pytest.mark.parametrize("kind", ["normal", "offset", "wide", "steps", "special"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("H,D,page", [(8, 128, 64), (3, 64, 16), (1, 256, 48)])
def test_kv_append_and_read(g, kind, dtype, H, D, page):
    rng = np.random.default_rng(D + page)
    T, pages = 29, 7
    K, V = _rows(rng, (T, H, D), dtype, kind), _rows(rng, (T, H, D), dtype, kind)
    slots = rng.choice(pages * page, T, replace=False).astype(np.int64)
    slots[[4, 20]] = -1
    pool = rng.integers(0, 256, (pages, H, so.block_bytes(page, D))).astype(np.uint8)
    want = pool.copy()
    for t in range(T):
        if slots[t] >= 0:
            for h in range(H):
                so.write_slot(want, page, D, slots[t], h, f64(K[t, h]), f64(V[t, h]))
    kv = torch.stack([K, V], dim=1).reshape(T, 2 * H * D).cuda()                 # side by side, strided
    k, v = kv[:, :H * D].view(T, H, D), kv[:, H * D:].view(T, H, D)
    cache = g.KVCache(torch.from_numpy(pool.copy()).cuda(), page, H, D)
    g.gptq_kv_append(cache, k, v, torch.from_numpy(slots).cuda())
    done(g)
    got = cache.pool.cpu().numpy()
    if kind == "special":                       # a NaN scale's payload is free
        half = got[..., page * D:].copy().view(np.float16), want[..., page * D:].copy().view(np.float16)
        same = (half[0] == half[1]) | (np.isnan(half[0]) & np.isnan(half[1]))
        assert same.all() and np.array_equal(got[..., :page * D], want[..., :page * D])
    else:
        assert np.array_equal(got, want)
    for out in (torch.float32, torch.bfloat16, torch.float16):
        rk, rv = g.gptq_kv_read(cache, torch.from_numpy(slots).cuda(), dtype=out)
        for t in range(T):
            for h in range(H):
                ref = so.read_slot(got, page, D, slots[t], h) if slots[t] >= 0 else (np.zeros(D), np.zeros(D))
                for r, x in zip(ref, (rk, rv)):
                    assert torch.allclose(x[t, h].cpu().double(), torch.from_numpy(r), rtol=2 * HALF_ULP[out],
                                          atol=2 * TINY[out], equal_nan=True), (t, h)
    done(g)


def test_kv_append_out_of_range_slots(g):
    H, D, page, pages = 2, 64, 16, 3
    cache = g.KVCache(torch.zeros((pages, H, so.block_bytes(page, D)), dtype=torch.uint8, device="cuda"), page, H, D)
    K = torch.randn((2, H, D), device="cuda")
    slots = torch.tensor([pages * page, 1 << 40], dtype=torch.int64, device="cuda")
    g.gptq_kv_append(cache, K, K, slots)
    torch.cuda.synchronize()
    with pytest.raises(g.GPTQError):
        g.gptq_device_check()
    assert not cache.pool.any()
    k, v = g.gptq_kv_read(cache, slots)
    torch.cuda.synchronize()
    with pytest.raises(g.GPTQError):
        g.gptq_device_check()
    assert not k.any() and not v.any()


# ------------------------------------------------------------------ attention
class Batch:
    """Sequences of the given lengths and numbers of query tokens over one random cache whose
    unused places hold NaN scales."""

    def __init__(self, lens, new, hq, h, D, page, dtype, seed, q_scale=1.5, v_scale=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.new, self.hq, self.h, self.D, self.page = lens, new, hq, h, D, page
        per = [-(-n // page) for n in lens]
        pages = sum(per) + 2
        self.pool = np.full((pages, h, so.block_bytes(page, D)), 0xFF, dtype=np.uint8)   # fp16 0xFFFF is NaN
        width = max(per + [1]) + 1
        order = rng.permutation(pages)
        self.table = np.full((len(lens), width), pages + 9, dtype=np.int32)              # never read
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            at += n
            for j in range(lens[b]):
                slot = int(self.table[b, j // page]) * page + j % page
                for x in range(h):
                    so.write_slot(self.pool, page, D, slot, x, rng.standard_normal(D) + 0.5,
                                  v_scale * np.exp(rng.standard_normal()) * rng.standard_normal(D))
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.Q = randn(rng, (int(self.cu[-1]), hq, D), dtype, q_scale)

    def gpu(self, g):
        self.cache = g.KVCache(torch.from_numpy(self.pool).cuda(), self.page, self.h, self.D)
        dev = [torch.from_numpy(a).cuda() for a in (self.cu, np.array(self.lens, np.int32), self.table)]
        return self.cache, self.Q.cuda(), *dev

    def check(self, O, lse=None, sm=None, causal=True, window=0, heads=None):
        sm = self.D ** -0.5 if sm is None else sm
        G = self.hq // self.h
        for b, n in enumerate(self.lens):
            for x in range(self.h):
                k, v = so.read_sequence(self.pool, self.page, self.D, self.table[b], n, x)
                ks, kl, vs, vl = self._numbers(b, n, x)
                for y in range(x * G, (x + 1) * G):
                    if heads is not None and y not in heads:
                        continue
                    q = f64(self.Q[self.cu[b]:self.cu[b + 1], y])
                    first = n - self.new[b]
                    o, l = so.attention(q, k, v, first, sm, causal, window)
                    got = f64(O[self.cu[b]:self.cu[b + 1], y])
                    for i in range(q.shape[0]):
                        d_s = ((self.D + 8) * 2.0 ** -22 * sm * np.abs(q[i]).sum() * np.max(15 * ks + np.abs(kl))) if n else 0.0
                        mag, _ = so.attention(q[i:i + 1], k, np.abs(v) + 2 * np.abs(vl)[:, None], first + i, sm, causal, window)
                        bound = ((2.0 ** -11 + 2 * d_s + 2.0 ** -18) * mag[0]
                                 + HALF_ULP[O.dtype] * np.abs(o[i]) * (1 + 2.0 ** -6) + TINY[O.dtype])
                        err = np.abs(got[i] - o[i])
                        assert np.all(err <= bound), (b, y, i, float(np.max(err / bound)))
                        if lse is not None:
                            a = float(lse[self.cu[b] + i, y])
                            assert a == l[i] or abs(a - l[i]) <= d_s + 2.0 ** -18 + 2.0 ** -22 * abs(l[i]), (a, l[i])

    def _numbers(self, b, n, x):
        out = np.zeros((4, n))
        for j in range(n):
            page, at = int(self.table[b][j // self.page]), j % self.page
            s = self.page * self.D + 8 * at
            out[:, j] = self.pool[page, x, s:s + 8].copy().view(np.float16)
        return out


@pytest.mark.parametrize("hq,h,D,page", [(4, 4, 128, 16), (8, 1, 128, 64), (7, 1, 64, 32), (16, 2, 256, 48),
                                         (40, 1, 128, 16), (6, 2, 64, 256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attention_one_token(g, hq, h, D, page, dtype):
    """Decoding: lengths of zero, one, around a page and around the tiles, and several tiles."""
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 127, 129, 300]
    t = Batch(lens, [1] * len(lens), hq, h, D, page, dtype, seed=hq + D)
    lse = torch.full((len(lens), hq), 7.0, device="cuda")
    O = g.gptq_kv_attention(*t.gpu(g), 1, lse=lse)
    done(g)
    assert not O[0].any() and torch.isinf(lse[0]).all()
    t.check(O, lse)


@pytest.mark.parametrize("hq,h,D,page", [(8, 1, 128, 16), (3, 3, 64, 32), (4, 2, 256, 16)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 5), (False, 0), (False, 9), (True, 1)])
def test_attention_several_tokens(g, hq, h, D, page, causal, window):
    """A few new tokens each (none for one sequence), some of them more than the cache holds
    (rows that see nothing)."""
    lens, new = [70, 2, 33, 9, 0], [5, 4, 0, 9, 2]
    t = Batch(lens, new, hq, h, D, page, torch.bfloat16, seed=D + window)
    lse = torch.empty((sum(new), hq), device="cuda")
    O = g.gptq_kv_attention(*t.gpu(g), max(new), causal=causal, window=window, lse=lse)
    done(g)
    t.check(O, lse, causal=causal, window=window)


@pytest.mark.parametrize("hq,h,D,page,dtype", [(8, 2, 128, 64, torch.bfloat16), (2, 2, 64, 16, torch.float16),
                                               (3, 1, 256, 32, torch.bfloat16), (16, 1, 128, 128, torch.bfloat16)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 100), (False, 0)])
def test_attention_piece_of_a_prompt(g, hq, h, D, page, dtype, causal, window):
    """Many new tokens over a longer cache, ragged, one sequence shorter than its new tokens."""
    lens, new = [331, 140, 100], [150, 140, 130]
    t = Batch(lens, new, hq, h, D, page, dtype, seed=D + page)
    lse = torch.empty((sum(new), hq), device="cuda")
    O = g.gptq_kv_attention(*t.gpu(g), max(new), causal=causal, window=window, lse=lse)
    done(g)
    t.check(O, lse, causal=causal, window=window, heads=(0, hq - 1))


@pytest.mark.parametrize("new", [1, 3, 70])
def test_attention_scales_of_every_size(g, new):
    """Large and tiny queries (fp16's whole range and beyond it in bf16) and values."""
    for q_scale, v_scale, dtype in ((1e-6, 1e-4, torch.bfloat16), (300.0, 2e3, torch.float16), (1e6, 1.0, torch.bfloat16),
                                    (1e-30, 1.0, torch.bfloat16)):
        t = Batch([150, 80], [new, new], 4, 2, 128, 16, dtype, seed=5, q_scale=q_scale, v_scale=v_scale)
        sm = 128 ** -0.5 if q_scale < 1 else 128 ** -0.5 / q_scale
        O = g.gptq_kv_attention(*t.gpu(g), new, sm_scale=sm)
        done(g)
        t.check(O, sm=sm)


@pytest.mark.parametrize("new", [2, 40])
def test_attention_nan_in_unseen_keys(g, new):
    """A NaN in a key that only later tokens see leaves the earlier ones as they are."""
    t = Batch([90], [new], 8, 1, 128, 16, torch.bfloat16, seed=3)
    clean = g.gptq_kv_attention(*t.gpu(g), new)
    slot = int(t.table[0, 89 // 16]) * 16 + 89 % 16
    so.write_slot(t.pool, 16, 128, slot, 0, np.full(128, np.nan), np.full(128, np.nan))
    O = g.gptq_kv_attention(*t.gpu(g), new)
    done(g)
    assert torch.equal(O[:-1], clean[:-1]) and torch.isnan(O[-1]).all()


def test_attention_long_split_cache(g):
    """A length that is split over many blocks and joined, with a flat and a peaked row."""
    page, D, h, hq, n = 64, 128, 2, 16, 20011
    gen = torch.Generator(device="cuda").manual_seed(3)
    pages = -(-n // page)
    cache = g.KVCache.empty(pages, page, h, D)
    K = torch.randn((n, h, D), device="cuda", generator=gen)
    V = torch.randn((n, h, D), device="cuda", generator=gen) + 0.3
    order = torch.randperm(pages, device="cuda", generator=gen)
    at = torch.arange(n, device="cuda")
    slots = order[at // page] * page + at % page
    g.gptq_kv_append(cache, K, V, slots)
    k, v = (x.double() for x in g.gptq_kv_read(cache, slots, dtype=torch.float32))
    Q = torch.randn((1, hq, D), device="cuda", generator=gen).to(torch.bfloat16)
    Q[0, 0] = 0.0
    Q[0, 1] *= 12.0
    for new_lens in (n, 7777):
        O = g.gptq_kv_attention(cache, Q, torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                                torch.tensor([new_lens], dtype=torch.int32, device="cuda"),
                                order.to(torch.int32)[None], 1)
        done(g)
        for x in range(hq):
            p = torch.softmax(k[:new_lens, x // 8] @ Q[0, x].double() * D ** -0.5, 0)
            ref = p @ v[:new_lens, x // 8]
            # the bound of the other tests with every |v| + 2 |low| below 3 * 6
            mag = p @ (v[:new_lens, x // 8].abs() + 12.0)
            assert torch.all((O[0, x].double() - ref).abs() <= (2.0 ** -11 + 2.0 ** -12) * mag + 2.0 ** -8 * ref.abs())


def test_attention_query_strides_and_uncovered_tokens(g):
    """Queries inside wider rows, outputs too; tokens outside every sequence keep what was there."""
    t = Batch([40, 9], [2, 1], 4, 2, 64, 16, torch.bfloat16, seed=11)
    cache, Q, cu, lens, table = t.gpu(g)
    cu = cu + 1
    wide = torch.zeros((6, 5 * 64 + 8), dtype=torch.bfloat16, device="cuda")
    wide[1:4, :256] = Q.reshape(3, 256)
    out = torch.full((6, 4 * 64 + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    g.gptq_kv_attention(cache, wide[:, :256].view(6, 4, 64), cu, lens, table, 2, O=out[:, :256].view(6, 4, 64))
    done(g)
    t.check(out[1:4, :256].reshape(3, 4, 64))
    assert torch.all(out[:, 256:] == 3) and torch.all(out[0] == 3) and torch.all(out[4:] == 3)


def test_attention_bad_lengths_and_pages_are_reported(g):
    for new in (1, 40):
        t = Batch([64, 64], [new, new], 4, 2, 64, 16, torch.bfloat16, seed=12)
        for bad in ("length", "page"):
            cache, Q, cu, lens, table = t.gpu(g)
            if bad == "length":
                lens[1] = table.shape[1] * 16 + 5
                table[1, 4:] = table[1, 0]
            else:
                table[1, 1] = cache.pool.shape[0]
            O = g.gptq_kv_attention(cache, Q, cu, lens, table, new)
            torch.cuda.synchronize()
            with pytest.raises(g.GPTQError) as e:
                g.gptq_device_check()
            assert e.value.status == g.GPTQ_ERR_INVALID_ARG
            assert torch.isfinite(O[:new].float()).all()             # the other sequence is untouched


# ------------------------------------------------------------------ adapters
def _layer(rng, m, d, bits, gs):
    G = 1 if gs == -1 else d // gs
    codes = rng.integers(0, 2 ** bits, size=(m, d))
    zeros = rng.integers(0, 2 ** bits, size=(m, G)).astype(np.float32)
    scales = (0.02 * (0.5 + rng.random((m, G)))).astype(np.float32)
    return orc.pack_codes(codes, bits), scales, zeros


def _check_adapter(g, m, d, bits, gs, T, n, rank, ids, out_bf16, seed, alpha=True, ldx=0):
    rng = np.random.default_rng(seed)
    words, sc, ze = _layer(rng, m, d, bits, gs)
    q = g.QuantizedLayer(torch.from_numpy(words.view(np.int32)).cuda(), torch.from_numpy(sc).cuda(),
                         torch.from_numpy(ze).cuda(), None, bits, gs, d)
    X = randn(rng, (T, d + ldx), torch.bfloat16)[:, :d]
    A, B = randn(rng, (n, rank, d), torch.bfloat16, d ** -0.5), randn(rng, (n, m, rank), torch.bfloat16)
    al = (0.5 + rng.random(n)).astype(np.float32) if alpha else None
    ids = np.asarray(ids, dtype=np.int32)
    Y = g.gptq_adapter_linear(q, X.cuda(), m, A.cuda(), B.cuda(), torch.from_numpy(ids).cuda(),
                              alpha=None if al is None else torch.from_numpy(al).cuda(), out_bf16=out_bf16)
    done(g)
    ref = so.adapter_linear(f64(X), words, sc, ze, bits, gs, f64(A), f64(B), ids, al)
    W = np.abs(orc.dequantize_packed(words, sc, ze, bits, d, gs, None))
    G = 1 if gs == -1 else d // gs
    unit = min(256, d if gs == -1 else gs)
    bound = (unit + G + 2) * 2.0 ** -23 * (np.abs(f64(X)) @ W.T)
    for t, a in enumerate(ids):
        if a >= 0:
            low = np.abs(f64(B[a])) @ (np.abs(f64(A[a])) @ np.abs(f64(X[t])))
            bound[t] += ((d + rank) * 2.0 ** -23 + 2.0 ** -16) * (1.0 if al is None else al[a]) * low
    bound += HALF_ULP[Y.dtype] * np.abs(ref) * (1 + 2.0 ** -7) + 1e-30
    err = np.abs(f64(Y) - ref)
    assert np.all(err <= bound), float(np.max(err / bound))


@pytest.mark.parametrize("bits,gs", [(4, 128), (4, 32), (4, -1), (2, 64), (2, 32), (3, 128), (3, 64), (8, 128), (8, 32)])
@pytest.mark.parametrize("T", [1, 2, 9, 17, 40])
@pytest.mark.parametrize("out_bf16", [False, True])
def test_adapter_linear_decoding(g, bits, gs, T, out_bf16):
    """Each token its own adapter, some none, out of order."""
    rng = np.random.default_rng(T)
    _check_adapter(g, 200, 768, bits, gs, T, 6, 16, rng.integers(-1, 6, T), out_bf16, seed=bits * 100 + T)


@pytest.mark.parametrize("rank", [8, 24, 64, 128])
@pytest.mark.parametrize("T", [1, 5, 70, 150])
def test_adapter_linear_ranks(g, rank, T):
    rng = np.random.default_rng(rank + T)
    _check_adapter(g, 136, 512, 4, 128, T, 5, rank, np.sort(rng.integers(-1, 5, T)), T % 2 == 0, seed=rank, alpha=T > 1,
                   ldx=8)


@pytest.mark.parametrize("T,ids", [(300, "runs"), (129, "one"), (257, "mixed"), (140, "none")])
@pytest.mark.parametrize("m,d,bits,gs", [(300, 512, 4, 128), (64, 1056, 8, 32), (257, 768, 2, 64), (520, 640, 3, -1)])
def test_adapter_linear_prompts(g, T, ids, m, d, bits, gs):
    rng = np.random.default_rng(T + m)
    ids = {"runs": np.sort(rng.integers(-1, 7, T)), "one": np.full(T, 3), "mixed": rng.integers(-1, 7, T),
           "none": np.full(T, -1)}[ids]
    _check_adapter(g, m, d, bits, gs, T, 7, 16, ids, T % 2 == 0, seed=T)


@pytest.mark.parametrize("d,bits,gs,rank,ids", [(256, 4, 128, 16, "runs"), (416, 4, 32, 8, "mixed"), (512, 8, 64, 64, "runs"),
                                                (384, 2, 64, 40, "one"), (640, 3, 128, 72, "runs"), (320, 3, -1, 128, "mixed"),
                                                (96, 8, 96, 16, "none"), (1024, 4, -1, 16, "sparse")])
def test_adapter_linear_many_tokens(g, d, bits, gs, rank, ids):
    """Enough rows and tokens for the tiles of 256 tokens, partial ones among them."""
    m, T = 2500, 1300
    rng = np.random.default_rng(d + rank)
    ids = {"runs": np.sort(rng.integers(-1, 6, T)), "mixed": rng.integers(-1, 6, T), "one": np.full(T, 2),
           "none": np.full(T, -1), "sparse": np.where(rng.random(T) < 0.01, 1, -1)}[ids]
    _check_adapter(g, m, d, bits, gs, T, 6, rank, ids, rank % 16 == 0, seed=rank, ldx=16)


@pytest.mark.parametrize("m,d,bits,gs", [(130, 96, 2, 32), (70, 160, 3, 32), (257, 1120, 3, -1), (64, 32, 4, 32),
                                         (129, 1056, 2, 96), (1, 224, 8, -1), (300, 800, 4, 160)])
@pytest.mark.parametrize("T", [1, 33, 140])
def test_adapter_linear_odd_widths(g, m, d, bits, gs, T):
    """Widths whose packed rows are no multiple of 16 bytes, widths that end inside a block,
    groups that no power of two above 32 divides."""
    rng = np.random.default_rng(m + T)
    _check_adapter(g, m, d, bits, gs, T, 3, 8, rng.integers(-1, 3, T), T == 33, seed=d + T)


def test_adapter_linear_without_adapters_and_bad_ids(g):
    rng = np.random.default_rng(1)
    m, d, T = 100, 256, 7
    words, sc, ze = _layer(rng, m, d, 4, 128)
    q = g.QuantizedLayer(torch.from_numpy(words.view(np.int32)).cuda(), torch.from_numpy(sc).cuda(),
                         torch.from_numpy(ze).cuda(), None, 4, 128, d)
    for T in (7, 200):
        X = randn(rng, (T, d), torch.bfloat16).cuda()
        plain = g.gptq_adapter_linear(q, X, m)
        A, B = randn(rng, (2, 16, d), torch.bfloat16).cuda(), randn(rng, (2, m, 16), torch.bfloat16).cuda()
        none = g.gptq_adapter_linear(q, X, m, A, B, torch.full((T,), -1, dtype=torch.int32, device="cuda"))
        done(g)
        assert torch.equal(plain, none)
        ids = torch.full((T,), -1, dtype=torch.int32, device="cuda")
        ids[3] = 2                                                     # out of range: no adapter, reported
        bad = g.gptq_adapter_linear(q, X, m, A, B, ids)
        torch.cuda.synchronize()
        with pytest.raises(g.GPTQError) as e:
            g.gptq_device_check()
        assert e.value.status == g.GPTQ_ERR_INVALID_ARG
        assert torch.equal(bad, plain)


def test_serving_on_another_stream(g):
    """Every call goes to the stream it is given, behind the work queued there."""
    s = torch.cuda.Stream()
    t = Batch([200], [1], 8, 1, 128, 16, torch.bfloat16, seed=21)
    cache, Q, cu, lens, table = t.gpu(g)
    torch.cuda.synchronize()
    late = torch.zeros_like(Q)
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        late.copy_(Q)
    O = g.gptq_kv_attention(cache, late, cu, lens, table, 1, stream=s)
    s.synchronize()
    t.check(O)


@pytest.mark.parametrize("hq,h,D,page", [(8, 2, 128, 64), (16, 2, 64, 32)])
def test_attention_piece_with_cold_caches(g, hq, h, D, page):
    """The same call with everything evicted in between gives the same bits: what a warp reads of a
    tile is read before the next tile takes its place, however late the warp comes."""
    t = Batch([331, 140], [150, 140], hq, h, D, page, torch.bfloat16, seed=7 * D)
    args = t.gpu(g)
    evict = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    want = None
    for i in range(40):
        evict.fill_(i)
        O = g.gptq_kv_attention(*args, 150)
        if want is None:
            want = O
        assert torch.equal(O, want), i
    done(g)
    t.check(want, heads=(0, hq - 1))


# ------------------------------------------------------------------ attention over long caches
class Long:
    """One long sequence's cache, which all sequences of a batch share through their tables (sequence b
    sees its first lens[b] tokens), and attention over it in float64 on the GPU. The cached values
    are those that gptq_kv_read gives; the bounds are the ones above, with 2^-11 sm sum |q| |k| more for a
    score of the kernel for many rows, which rounds k to fp16. Values of V move with their tile of
    128 keys, so that a tile that is lost or counted twice moves the output, and lse moves by the tile's
    share of the softmax."""

    def __init__(self, g, n, h, D, page, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.n, self.h, self.D, self.page = n, h, D, page
        pages = -(-n // page)
        self.order = torch.randperm(pages, device="cuda", generator=gen)
        self.cache = g.KVCache(torch.full((pages, h, page * (D + 8)), 0xFF, dtype=torch.uint8, device="cuda"), page, h, D)
        at = torch.arange(n, device="cuda")
        slots = self.order[at // page] * page + at % page
        K = torch.randn((n, h, D), device="cuda", generator=gen)
        V = torch.randn((n, h, D), device="cuda", generator=gen) + 3 * torch.randn((n // 128 + 1, 1, D), device="cuda",
                                                                                   generator=gen)[at // 128]
        g.gptq_kv_append(self.cache, K, V, slots)
        self.k, self.v = (x.double() for x in g.gptq_kv_read(self.cache, slots, dtype=torch.float32))
        num = self.cache.pool[..., page * D:].contiguous().view(torch.float16).view(pages, h, page, 4).double()
        self.num = num[slots // page, :, slots % page]                       # (n, h, 4)
        self.gen = gen

    def batch(self, lens, new, hq, dtype=torch.bfloat16):
        """Queries of a batch and what the call reads beside them."""
        self.lens, self.hq, self.cu = lens, hq, [0]
        for x in new:
            self.cu.append(self.cu[-1] + x)
        self.Q = torch.randn((self.cu[-1], hq, self.D), device="cuda", generator=self.gen).to(dtype)
        self.Q[::3] *= 4                                                    # some rows are peaked
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        return self.cache, self.Q, ints(self.cu), ints(lens), self.order.int()[None].repeat(len(lens), 1)

    def check(self, O, lse, seqs, heads, causal=True, window=0, sm=None, many=False):
        sm, G = self.D ** -0.5 if sm is None else sm, self.hq // self.h
        for b in seqs:
            n, a, z = self.lens[b], self.cu[b], self.cu[b + 1]
            pos = torch.arange(n - (z - a), n, device="cuda")[:, None]
            key = torch.arange(n, device="cuda")[None]
            see = (key <= pos if causal else key >= 0) & ((key > pos - window) if window else (key >= 0))
            for y in heads:
                k, v, num = self.k[:n, y // G], self.v[:n, y // G], self.num[:n, y // G]
                q = self.Q[a:z, y].double()
                s = (sm * (q @ k.T)).masked_fill(~see, -float("inf"))
                l = torch.logsumexp(s, 1)
                p = torch.where(see, torch.exp(s - l[:, None]), 0.0)
                ref, mag = p @ v, p @ (v.abs() + 2 * num[:, 3:].abs())
                d_s = (self.D + 8) * 2.0 ** -22 * sm * q.abs().sum(1, keepdim=True) * (15 * num[:, 0] + num[:, 1].abs()).max()
                if many:
                    d_s = d_s + 2.0 ** -11 * sm * (q.abs() @ k.abs().T).max(1, keepdim=True).values
                bound = ((2.0 ** -11 + 2 * d_s + 2.0 ** -18) * mag + HALF_ULP[O.dtype] * ref.abs() * (1 + 2.0 ** -6)
                         + TINY[O.dtype])
                err = (O[a:z, y].double() - ref).abs()
                assert (err <= bound).all(), (b, y, float((err / bound).max()))
                dl = (lse[a:z, y].double() - l).abs()
                assert (dl <= d_s[:, 0] + 2.0 ** -18 + 2.0 ** -22 * l.abs()).all(), (b, y, float(dl.max()))


@pytest.mark.parametrize("hq,h,D,page,new", [(4, 4, 64, 16, 1), (32, 4, 64, 32, 1), (4, 4, 128, 16, 1), (32, 4, 128, 64, 1),
                                             (4, 4, 256, 32, 1), (32, 4, 256, 16, 1), (16, 4, 64, 64, 8), (12, 4, 256, 64, 5)])
def test_attention_few_rows_with_cold_caches(g, hq, h, D, page, new):
    """The kernel of few rows a head, whose ring of tiles is filled anew several times by every CTA, with
    everything evicted in between: the same bits each time, one row a head and more."""
    t = Long(g, 9001, h, D, page, seed=D + hq)
    lens = [9001 - 61 * i for i in range(24)]
    args = t.batch(lens, [new] * 24, hq)
    evict = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    lse = torch.empty((24 * new, hq), device="cuda")
    want = None
    for i in range(30):
        evict.fill_(i)
        O = g.gptq_kv_attention(*args, new, lse=lse)
        if want is None:
            want = O
        assert torch.equal(O, want), i
    done(g)
    t.check(want, lse, (0, 9, 23), (0, hq - 1))


# ------------------------------------------------------------------ memory of calls on another stream
def _on_another_stream(call, sizes):
    """call(stream) while the current stream is still to write blocks of the sizes that the call
    allocates, blocks that have been given back already. Returns call's result. (A first round loads
    the kernels and gets the memory, which can wait for the device.)"""
    side = torch.cuda.Stream()
    for cycles in (1000, 400_000_000):
        torch.cuda.synchronize()
        blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
        torch.cuda._sleep(cycles)
        for b in blocks:
            b.fill_(0x55)
        del blocks, b
        out = call(side)
        side.synchronize()
        early = not torch.cuda.current_stream().query()         # what it queued is still to come
        torch.cuda.synchronize()
    assert early
    return out


def test_serving_memory_of_another_stream(g):
    """Outputs and workspaces of calls on another stream than the current one are not memory that
    the current stream has yet to write."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()
    T, hq, hk, D, page, m, d, rank = 300, 8, 2, 64, 16, 256, 512, 16
    Q, K, V, X = rnd(T, hq, D), rnd(T, hk, D), rnd(T, hk, D), rnd(T, d)
    w = torch.rand(D, generator=gen, device="cuda")
    cache = g.KVCache.empty(20, page, hk, D)
    slots = torch.arange(T, device="cuda")
    g.gptq_kv_append(cache, K, V, slots)
    cu, lens = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, T], [T]))
    table = torch.arange(20, dtype=torch.int32, device="cuda")[None]
    q = g.QuantizedLayer(torch.randint(-2 ** 31, 2 ** 31 - 1, (m, d // 8), generator=gen, dtype=torch.int32, device="cuda"),
                         torch.rand((m, 4), generator=gen, device="cuda"), torch.full((m, 4), 8.0, device="cuda"), None, 4, 128, d)
    A, B, ids = rnd(3, rank, d), rnd(3, m, rank), torch.arange(T, dtype=torch.int32, device="cuda") // 100
    lib = g.library()
    calls = {
        "norm": (lambda s: g.gptq_qk_norm_rope(Q, K, wq=w, wk=w, stream=s), [2 * T * hq * D, 2 * T * hk * D]),
        "read": (lambda s: g.gptq_kv_read(cache, slots, stream=s), [2 * T * hk * D]),
        "attention": (lambda s: (g.gptq_kv_attention(cache, Q, cu, lens, table, T, stream=s),),
                      [2 * T * hq * D, lib.gptq_kv_attention_workspace_size(T, hq, hk, D, 1, T)]),
        "adapter": (lambda s: (g.gptq_adapter_linear(q, X, m, A, B, ids, stream=s),),
                    [4 * T * m, lib.gptq_adapter_workspace_size(m, d, 4, 128, T, rank)]),
    }
    for name, (call, sizes) in calls.items():
        want = call(None)
        for a, b in zip(want, _on_another_stream(call, sizes)):
            assert torch.equal(a, b), name
    done(g)


def test_layer_memory_of_another_stream(g):
    """The same for the calls that make a packed layer and use it alone."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    T, m, d = 300, 256, 512
    X = torch.randn((T, d), generator=gen, device="cuda").bfloat16()
    W = torch.randn((m, d), generator=gen, device="cuda")
    q, H, Hinv1, _ = g.quantize_layer(W, [X])
    fields = lambda q: (q.qweight, q.scales, q.zeros, q.col_losses)
    size = g.gptq_workspace_size
    calls = {
        "factor": (lambda s: g.gptq_factor(H, act_order=True, sync=False, stream=s)[:2],
                   [4 * d * d, 4 * d, size(g.GPTQ_WS_FACTOR, 0, d)]),
        "layer": (lambda s: fields(g.gptq_quantize_layer(W, Hinv1, stream=s)),
                  [m * d // 2, 4 * m * d // 128, 4 * d, size(g.GPTQ_WS_QUANTIZE, m, d)]),
        "codes": (lambda s: (g.gptq_unpack_codes(q.qweight, m, d, 4, stream=s),), [m * d]),
        "gemv": (lambda s: (g.gptq_dequant_gemv(q, X[:4], m, stream=s),), [4 * 4 * m]),
        "gemm": (lambda s: (g.gptq_dequant_gemm(q, X, m, out_bf16=True, stream=s),),
                 [2 * T * m, size(g.GPTQ_WS_DEQUANT_GEMM, m, d)]),
    }
    for name, (call, sizes) in calls.items():
        want = call(None)
        for a, b in zip(want, _on_another_stream(call, sizes)):
            assert torch.equal(a, b), name
    done(g)


@pytest.mark.parametrize("hq,h,D,max_q,n,lens", [(4, 2, 64, 1, 40, [200, 64]), (8, 8, 128, 1, 300, [400] * 24),
                                                 (8, 2, 128, 40, 60, [90, 80])])
def test_attention_counts_past_max_q_are_reported(g, hq, h, D, max_q, n, lens):
    """cu_q with more tokens for a sequence than max_q says, or fewer than none: reported, the sequence
    taken as its first max_q tokens (or none), the others as they are."""
    t = Long(g, max(lens), h, D, 16, seed=D)
    new = [max_q] * len(lens)
    cache, Q, cu, kv, table = t.batch(lens, new, hq)
    total = Q.shape[0]
    wide = torch.cat([Q, torch.randn((n, hq, D), device="cuda").bfloat16()])
    cu = cu.clone()
    cu[-1] += n                                                  # the last sequence: n tokens too many
    fill = lambda: (torch.full_like(wide, 5.0), torch.full((total + n, hq), 5.0, device="cuda"))
    O, lse = fill()
    g.gptq_kv_attention(cache, wide, cu, kv, table, max_q, O=O, lse=lse)
    torch.cuda.synchronize()
    with pytest.raises(g.GPTQError) as e:
        g.gptq_device_check()
    assert e.value.status == g.GPTQ_ERR_INVALID_ARG
    t.check(O, lse, range(len(lens)), (0, hq - 1))
    assert torch.all(O[total:] == 5) and torch.all(lse[total:] == 5)
    cu[-1] = cu[-2] - 1                                          # a step below zero: no tokens
    O, lse = fill()
    g.gptq_kv_attention(cache, wide, cu, kv, table, max_q, O=O, lse=lse)
    torch.cuda.synchronize()
    with pytest.raises(g.GPTQError):
        g.gptq_device_check()
    t.check(O, lse, range(len(lens) - 1), (0,))
    assert torch.all(O[total - max_q:] == 5)


def test_adapter_linear_a_million_tokens(g):
    """More groups of 16 tokens than a grid's second dimension holds."""
    m, d, rank, n, T = 8, 32, 8, 5, 65536 * 16 + 9
    rng = np.random.default_rng(8)
    words, sc, ze = _layer(rng, m, d, 4, 32)
    q = g.QuantizedLayer(torch.from_numpy(words.view(np.int32)).cuda(), torch.from_numpy(sc).cuda(),
                         torch.from_numpy(ze).cuda(), None, 4, 32, d)
    gen = torch.Generator(device="cuda").manual_seed(8)
    rnd = lambda *s: torch.randn(s, device="cuda", generator=gen).bfloat16()
    X, A, B = rnd(T, d), rnd(n, rank, d), rnd(n, m, rank)
    ids = (torch.arange(T, device="cuda") // 1000 % (n + 1) - 1).int()
    Y = g.gptq_adapter_linear(q, X, m, A, B, ids)
    done(g)
    W = torch.from_numpy(orc.dequantize_packed(words, sc, ze, 4, d, 32, None)).cuda()
    x = X.double()
    ref, bound = x @ W.T, 35 * 2.0 ** -23 * (x.abs() @ W.abs().T)
    for a in range(n):
        t = ids == a
        ref[t] += x[t] @ A[a].double().T @ B[a].double().T
        bound[t] += ((d + rank) * 2.0 ** -23 + 2.0 ** -16) * (x[t].abs() @ A[a].double().abs().T @ B[a].double().abs().T)
    bound += HALF_ULP[torch.float32] * ref.abs() + 1e-30
    assert ((Y.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("new", [1, 3, 70])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 20), (False, 9)])
def test_attention_scores_that_vanish(g, new, causal, window):
    """Scale and queries so small that their product is below every fp32 number: each row is the
    mean of the keys it sees."""
    t = Batch([150, 80], [new, new], 4, 2, 128, 16, torch.bfloat16, seed=5, q_scale=1e-35)
    lse = torch.empty((2 * new, 4), device="cuda")
    O = g.gptq_kv_attention(*t.gpu(g), new, sm_scale=1e-8, causal=causal, window=window, lse=lse)
    done(g)
    t.check(O, lse, sm=1e-8, causal=causal, window=window)


@pytest.mark.parametrize("new", [1, 3, 70])
def test_attention_largest_queries(g, new):
    """bf16 queries up to the largest finite one, whose plain sum over a head is beyond fp32."""
    t = Long(g, 150, 2, 128, 16, seed=6)
    args = t.batch([150, 80], [new, new], 4)
    big = torch.finfo(torch.bfloat16).max
    t.Q[:, 0::2] = 0.0
    t.Q[:, 0::2, 5] = big
    t.Q[:, 0::2, 60] = 3.1e38
    t.Q[:, 1::2] = (1e38 * t.Q[:, 1::2].float()).clamp(-big, big).bfloat16()
    t.Q[:, 1::2, 7] = -big
    lse = torch.empty((2 * new, 4), device="cuda")
    O = g.gptq_kv_attention(*args, new, sm_scale=2e-38, lse=lse)
    done(g)
    t.check(O, lse, (0, 1), range(4), sm=float(np.float32(2e-38)), many=new == 70)


@pytest.mark.parametrize("T", [40, 300, 1300])
def test_adapter_linear_extreme_inner_products(g, T):
    """An inner product that is infinite, that is a NaN, and one that is finite in fp32 but rounds to an
    infinite bf16: the same in every tile size."""
    m, d, rank = 2500, 64, 8
    rng = np.random.default_rng(T)
    words, sc, ze = _layer(rng, m, d, 4, 64)
    q = g.QuantizedLayer(torch.from_numpy(words.view(np.int32)).cuda(), torch.from_numpy(sc).cuda(),
                         torch.from_numpy(ze).cuda(), None, 4, 64, d)
    X = torch.zeros((T, d), dtype=torch.bfloat16)
    X[:, :3] = torch.tensor([1.0, 1.0, 2.0])
    A, B = torch.zeros((4, rank, d), dtype=torch.bfloat16), torch.zeros((4, m, rank), dtype=torch.bfloat16)
    big = torch.finfo(torch.bfloat16).max
    A[0, 3, 0], A[0, 3, 2] = big, big                              # 3 big: infinite
    A[1, 3, 0], A[1, 3, 1] = big, 8e35                             # above bf16's largest, below fp32's
    A[2, 3, 0] = float("nan")
    A[3] = -A[1]
    B[0, :, 3] = torch.from_numpy(np.where(np.arange(m) % 2, 2.0, -0.5))
    B[1:, :, 3] = 2.0 ** -120
    ids = np.repeat(np.arange(4), -(-T // 4))[:T].astype(np.int32)
    Y = g.gptq_adapter_linear(q, X.cuda(), m, A.cuda(), B.cuda(), torch.from_numpy(ids).cuda())
    done(g)
    W = orc.dequantize_packed(words, sc, ze, 4, d, 64, None)
    base = f64(X[0]) @ W.T
    y, inner = f64(Y), float(A[1, 3, 0]) + float(A[1, 3, 1])
    assert inner < np.finfo(np.float32).max
    assert np.array_equal(y[ids == 0], np.broadcast_to(np.where(np.arange(m) % 2, np.inf, -np.inf), y[ids == 0].shape))
    assert np.isnan(y[ids == 2]).all()
    for a, sign in ((1, 1.0), (3, -1.0)):
        ref = base + sign * inner * 2.0 ** -120
        assert (np.abs(y[ids == a] - ref) <= 2.0 ** -15 * (np.abs(ref) + inner * 2.0 ** -120)).all()


@pytest.mark.parametrize("hq,new", [(2, 5), (8, 40)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_windows_of_any_size(g, hq, new, causal):
    """A window past every position is no window, up to the largest one, for rows before the first key too."""
    t = Batch([1, 90, 0], [new] * 3, hq, 2, 64, 16, torch.bfloat16, seed=9)
    want = g.gptq_kv_attention(*t.gpu(g), new, causal=causal)
    done(g)
    t.check(want, causal=causal)
    for window in (200, 2 ** 31 - 1, 2 ** 31, 2 ** 40, 2 ** 63 - 1):
        assert torch.equal(g.gptq_kv_attention(*t.gpu(g), new, causal=causal, window=window), want), window
    done(g)


MANY_ROWS = [                                    # hq, h, D, page, lens, new, causal, window
    (6, 2, 128, 64, [9001], [500], True, 0),                     # groups of 3, a partial row tile, more than four parts
    (24, 8, 128, 64, [9001], [500], True, 0),                    # two to four parts
    (14, 2, 64, 16, [9001, 3000, 1500], [300, 37, 130], True, 2000),
    (10, 2, 64, 32, [5000, 1200], [200, 199], False, 0),
    (16, 1, 128, 48, [131, 4097, 2000], [2, 17, 0], True, 0),
    (4, 4, 128, 16, [2300], [2300], True, 0),                    # a prompt from an empty cache
    (4, 2, 64, 256, [3001, 700], [1100, 700], True, 900),
    (40, 1, 128, 128, [9001] * 3, [1, 1, 1], True, 0),           # wide groups of one token
    (9, 1, 64, 64, [6000, 6000], [300, 7], False, 1500),
]
FEW_ROWS = [
    (2, 2, 64, 16, [9001], [1], True, 0),                        # one row an item; many parts
    (32, 2, 64, 32, [9001, 1500], [1, 1], True, 0),              # 16 rows
    (14, 2, 64, 48, [9001, 8000], [4, 3], True, 0),              # 28 rows, of 32
    (8, 1, 128, 64, [9001, 40], [1, 1], True, 5000),
    (12, 1, 128, 128, [9001], [1], True, 0),                     # 12 rows, of 16
    (10, 2, 128, 16, [9001, 2100, 4000], [3, 1, 2], False, 0),
    (4, 2, 256, 32, [9001], [1], True, 0),
    (6, 1, 256, 64, [9001, 3300], [50, 33], True, 0),            # many items of 16 rows
    (16, 2, 256, 16, [9001] * 8, [3] * 8, True, 3000),
    (24, 8, 128, 64, [2500 - 61 * i for i in range(40)], [1] * 40, True, 0),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", MANY_ROWS + FEW_ROWS, ids=lambda c: "-".join(map(str, (c[0], c[1], c[2], sum(c[5])))))
def test_attention_of_items_that_are_cut(g, case, dtype):
    """More than 1024 keys, so that the line of tiles cuts items between CTAs: output and log-sum-exp of
    every part's join, and the same bits again."""
    hq, h, D, page, lens, new, causal, window = case
    t = Long(g, max(lens), h, D, page, seed=hq + D + sum(new))
    args = t.batch(lens, new, hq, dtype)
    lse, again = torch.empty((2, sum(new), hq), device="cuda")
    O = g.gptq_kv_attention(*args, max(new), causal=causal, window=window, lse=lse)
    O2 = g.gptq_kv_attention(*args, max(new), causal=causal, window=window, lse=again)
    done(g)
    assert torch.equal(O, O2) and torch.equal(lse, again)
    rows = max(new) * (hq // h)
    t.check(O, lse, range(0, len(lens), 1 + len(lens) // 4), sorted({0, 1, hq // 2, hq - 1}), causal, window,
            many=D != 256 and rows > (32 if D == 64 else 16))


def test_kv_append_every_scale(g):
    """Every fp16 scale that a row can have (up to twice the largest number over 15), with values on
    and next to the ties between codes: the bits of a true division."""
    D, page = 64, 16
    s = np.arange(1, 0x7C00, dtype=np.uint16).view(np.float16).astype(np.float32)
    s = s[s <= np.float32(2 * 65504 / 15)]
    low = np.where(15 * s <= 65504, np.float32(0), np.float32(-65504))
    low[::2] = np.where(15 * s[::2] <= 65504, -np.minimum(15 * s[::2], 65504).astype(np.float16).astype(np.float32), low[::2])
    ties = (s[:, None] * (np.arange(15, dtype=np.float32) + np.float32(0.5)) + low[:, None]).astype(np.float32)
    inf = np.float32(np.inf)
    x = np.concatenate([low[:, None], (15 * s + low)[:, None], ties, np.nextafter(ties, inf), np.nextafter(ties, -inf),
                        np.random.default_rng(1).random((len(s), 15), dtype=np.float32) * (15 * s)[:, None] + low[:, None]], axis=1)
    x = np.concatenate([x, x[:, :D - x.shape[1]]], axis=1).astype(np.float32)
    T = len(s)
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        K = torch.from_numpy(x).to(dtype)
        y = np.clip(K.float().numpy(), -65504, 65504)                    # 65504 is 65536 in bf16
        lo, hi = y.min(1), y.max(1)
        scale = ((hi - lo) / np.float32(15)).astype(np.float16)
        low16 = lo.astype(np.float16)
        if dtype == torch.float32:
            assert len(set(scale.view(np.uint16).tolist())) > 28000         # nearly every one of them
        with np.errstate(divide="ignore", invalid="ignore"):
            q = (y - low16.astype(np.float32)[:, None]) / scale.astype(np.float32)[:, None]
        codes = np.where(scale[:, None] == 0, 0, np.clip(np.rint(q), 0, 15)).astype(np.uint8)
        cache = g.KVCache(torch.zeros((-(-T // page), 1, page * (D + 8)), dtype=torch.uint8, device="cuda"), page, 1, D)
        V = K.flip(0).contiguous()
        g.gptq_kv_append(cache, K[:, None].cuda(), V[:, None].cuda(), torch.arange(T, device="cuda"))
        done(g)
        pool = cache.pool.cpu().numpy()[:, 0]
        half = page * D // 2
        num = np.ascontiguousarray(pool[:, 2 * half:]).view(np.float16).reshape(-1, 4)[:T]
        for kv, order in ((0, slice(None)), (1, slice(None, None, -1))):
            b = pool[:, kv * half:(kv + 1) * half].reshape(-1, D // 2)[:T]
            got = np.stack([b & 15, b >> 4], axis=-1).reshape(T, D)
            assert np.array_equal(got, codes[order]) and np.array_equal(num[:, 2 * kv], scale[order])
            assert np.array_equal(num[:, 2 * kv + 1], low16[order])


@pytest.mark.parametrize("D,new", [(64, 1), (128, 40), (256, 2)])
def test_attention_steps_and_lengths_of_any_bits(g, D, new):
    """cu_q and kv_lens with numbers far out of range: reported, outputs of the other sequences as they
    are, nothing written outside them."""
    t = Long(g, 300, 2, D, 16, seed=D)
    cache, Q, cu, kv, table = t.batch([200, 64, 300], [new] * 3, 4)
    for at, value in ((1, -2 ** 31), (1, 2 ** 31 - 1), (2, -2 ** 31), (3, 2 ** 31 - 1), (3, -1), (0, -2 ** 31), (0, 2 ** 31 - 1)):
        bad = cu.clone()
        bad[at] = value
        O, lse = torch.full_like(Q, 5.0), torch.full(Q.shape[:2], 5.0, device="cuda")
        g.gptq_kv_attention(cache, Q, bad, kv, table, new, O=O, lse=lse)
        torch.cuda.synchronize()
        with pytest.raises(g.GPTQError):
            g.gptq_device_check()
        assert torch.isfinite(O.float()).all()
        t.check(O, lse, [b for b in range(3) if at not in (b, b + 1)], (0, 3))
    for b, value in ((1, -1), (1, -2 ** 31), (2, 2 ** 31 - 1)):
        bad = kv.clone()
        bad[b] = value
        O, lse = torch.full_like(Q, 5.0), torch.full(Q.shape[:2], 5.0, device="cuda")
        g.gptq_kv_attention(cache, Q, cu, bad, table, new, O=O, lse=lse)
        torch.cuda.synchronize()
        with pytest.raises(g.GPTQError):
            g.gptq_device_check()
        t.check(O, lse, [x for x in range(3) if x != b], (0, 3))


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("D,hq,new", [(64, 8, 2), (128, 8, 2), (256, 8, 2), (64, 8, 40), (128, 8, 40), (256, 8, 40)])
def test_attention_nan_in_one_row_of_a_key(g, which, D, hq, new):
    """A NaN in a key's K row alone or V row alone makes NaN of every value of the rows that see the key,
    and of no other row's, whatever tile it is in."""
    for place in (700, 899):
        t = Batch([900], [new], hq, 1, D, 16, torch.bfloat16, seed=D)
        lse, lse2 = torch.empty((2, new, hq), device="cuda")
        clean = g.gptq_kv_attention(*t.gpu(g), new, window=150, lse=lse)
        slot = int(t.table[0, place // 16]) * 16 + place % 16
        row = np.full(D, np.nan)
        k, v = so.read_slot(t.pool, 16, D, slot, 0)
        so.write_slot(t.pool, 16, D, slot, 0, row if which == "k" else k, row if which == "v" else v)
        O = g.gptq_kv_attention(*t.gpu(g), new, window=150, lse=lse2)
        done(g)
        pos = torch.arange(900 - new, 900)
        sees = ((pos >= place) & (pos - 150 < place)).cuda()
        assert sees.any() == (place == 899) and torch.isnan(O[sees]).all()
        assert torch.equal(O[~sees], clean[~sees]) and torch.equal(lse2[~sees], lse[~sees])
        if which == "k":
            assert torch.isnan(lse2[sees]).all()


def test_streams_by_handle(g):
    """A stream as a handle: torch's own, the default stream's two (0 and 1) and the thread's own (2), with the
    current stream another one."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    X = torch.randn((40, 256), generator=gen, device="cuda").bfloat16()
    q = g.quantize_layer(torch.randn((64, 256), generator=gen, device="cuda"), [X])[0]
    calls = (lambda s: g.gptq_adapter_linear(q, X, 64, stream=s), lambda s: g.gptq_dequant_gemm(q, X, 64, stream=s),
             lambda s: g.gptq_qk_norm_rope(X.view(40, 2, 128), None, stream=s)[0])
    want = [c(None) for c in calls]
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    for handle in (other.cuda_stream, 0, 1, 2):
        for current in (torch.cuda.default_stream(), side):
            with torch.cuda.stream(current):
                got = [c(handle) for c in calls]
                torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), handle
    done(g)


def _fp16_error(g, D, hq, h, n, new, window):
    """The error of fp16 outputs over values without a mean, where no rounding is averaged away, in the
    2-norm and in units of the rounding of the exact output."""
    gen = torch.Generator(device="cuda").manual_seed(n + D)
    page, batch = 16, 4
    pages = -(-n // page)
    cache = g.KVCache.empty(batch * pages, page, h, D)
    at = torch.arange(n, device="cuda")
    table = torch.arange(batch * pages, device="cuda").view(batch, pages)
    Q = (1.5 * torch.randn((batch * new, hq, D), device="cuda", generator=gen)).half()
    want = []
    for b in range(batch):
        slots = table[b, at // page] * page + at % page
        g.gptq_kv_append(cache, *(torch.randn((n, h, D), device="cuda", generator=gen) for _ in range(2)), slots)
        k, v = (x.double() for x in g.gptq_kv_read(cache, slots, dtype=torch.float32))
        pos = torch.arange(n - new, n, device="cuda")[:, None]
        see = (at <= pos) & ((at > pos - window) if window else (at >= 0))
        q = Q[b * new:(b + 1) * new].double()
        s = torch.einsum("ihd,khd->ihk", q, k.repeat_interleave(hq // h, 1)) * D ** -0.5
        p = torch.softmax(s.masked_fill(~see[:, None], -float("inf")), -1)
        want.append(torch.einsum("ihk,khd->ihd", p, v.repeat_interleave(hq // h, 1)))
    want = torch.cat(want)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    O = g.gptq_kv_attention(cache, Q, ints([new * i for i in range(batch + 1)]), ints([n] * batch), table.int(), new, window=window)
    done(g)
    return float((O.double() - want).norm() / (want.half().double() - want).norm())


# One more rounding as large as the output's would make it sqrt(2); with 6 % for the scatter 1.5.
@pytest.mark.parametrize("D,hq,h,new", [(64, 4, 1, 2), (64, 16, 1, 1), (64, 28, 1, 1), (128, 8, 8, 1), (128, 16, 1, 1), (256, 8, 1, 1),
                                        (256, 16, 2, 3), (256, 16, 2, 100)])
@pytest.mark.parametrize("n,window", [(3, 0), (100, 11), (128, 0), (600, 0)])
def test_attention_fp16_output_of_few_rows(g, D, hq, h, n, new, window):
    assert _fp16_error(g, D, hq, h, n, min(new, n), window) <= 1.5


@pytest.mark.parametrize("D,hq,h", [(64, 16, 1), (128, 16, 1), (64, 28, 4), (128, 8, 8)])
@pytest.mark.parametrize("n,new,window", [(3, 3, 0), (8, 5, 4), (24, 20, 11), (128, 64, 0), (400, 100, 30), (600, 100, 128)])
def test_attention_fp16_output_of_many_rows_over_few_keys(g, D, hq, h, n, new, window):
    assert _fp16_error(g, D, hq, h, n, new, window) <= 1.5
