"""The serving operators without a GPU: the C ABI refuses bad arguments before anything is
launched, the binding passes on the pointers, sizes and strides it is given and refuses
tensors of other shapes, and the float64 oracle meets cases worked out by hand."""
import os

import numpy as np
import pytest
import torch

from oracle import serving_oracle as so


@pytest.fixture(scope="module")
def g():
    from post_weight_quantization_gb300 import build as b
    if not os.path.exists(b.LIB_PATH):
        b.build()
    from post_weight_quantization_gb300 import gptq
    return gptq


# fake, aligned, never dereferenced device addresses: validation must fail first
P = 0x10000000


def test_norm_rope_refusals(g):
    lib, bad = g.library(), g.GPTQ_ERR_INVALID_ARG
    before = g.gptq_launch_count()

    def call(Q=P, K=P, din=1, T=4, hq=8, hk=2, D=128, ldq=1024, ldk=256, wq=P, wk=P, eps=1e-6, c=P, s=P, n=16, rot=128,
             inter=0, pos=P, Qo=P, Ko=P, dout=1, ldqo=1024, ldko=256):
        return lib.gptq_qk_norm_rope(Q, K, din, T, hq, hk, D, ldq, ldk, wq, wk, eps, c, s, n, rot, inter, pos, Qo, Ko,
                                     dout, ldqo, ldko, None)

    for kw in (dict(Q=None), dict(K=None), dict(Qo=None), dict(Ko=None), dict(din=3), dict(dout=-1), dict(T=-1),
               dict(T=1 << 31), dict(hq=0), dict(hk=-1), dict(D=4), dict(D=12), dict(D=264), dict(ldq=1016),
               dict(ldk=255), dict(ldq=1028), dict(ldqo=1000), dict(ldko=260), dict(Q=P + 8), dict(Ko=P + 4),
               dict(wq=P + 4), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(c=None),
               dict(s=None), dict(pos=None), dict(n=0), dict(rot=136), dict(rot=8), dict(rot=-16), dict(c=P + 8)):
        assert call(**kw) == bad, kw
        assert g.gptq_last_error()
    assert call(T=0, Q=None) == g.GPTQ_OK
    assert call(din=0, ldq=1026) == bad                       # fp32 rows 8 bytes off
    assert g.gptq_launch_count() == before


def test_cache_refusals(g):
    lib, bad = g.library(), g.GPTQ_ERR_INVALID_ARG
    before = g.gptq_launch_count()

    def append(K=P, V=P, dt=1, T=4, H=8, D=128, ldk=1024, ldv=1024, slots=P, pool=P, pages=4, page=64):
        return lib.gptq_kv_append(K, V, dt, T, H, D, ldk, ldv, slots, pool, pages, page, None)

    def read(pool=P, pages=4, page=64, H=8, D=128, slots=P, T=4, K=P, V=P, dt=1, ldk=1024, ldv=1024):
        return lib.gptq_kv_read(pool, pages, page, H, D, slots, T, K, V, dt, ldk, ldv, None)

    for call in (append, read):
        for kw in (dict(K=None), dict(V=None), dict(slots=None), dict(pool=None), dict(pool=P + 8), dict(dt=3),
                   dict(T=-1), dict(T=1 << 31), dict(H=0), dict(ldk=1023), dict(ldv=1016), dict(ldk=1028),
                   dict(K=P + 2), dict(pages=0), dict(pages=1 << 31), dict(page=8), dict(page=24), dict(page=272)):
            assert call(**kw) == bad, kw
        for D in (32, 96, 100, 512):
            assert call(D=D, ldk=8192, ldv=8192) == g.GPTQ_ERR_UNSUPPORTED
        assert call(T=0, K=None, slots=None) == g.GPTQ_OK
    assert g.gptq_launch_count() == before


def test_attention_refusals(g):
    lib, bad = g.library(), g.GPTQ_ERR_INVALID_ARG
    before = g.gptq_launch_count()

    def call(Q=P, dt=1, total=4, hq=8, h=2, D=128, ldq=1024, cu=P, lens=P, table=P, ldt=8, width=8, batch=4, max_q=1,
             pool=P, pages=64, page=16, sm=0.1, causal=1, window=0, O=P, ldo=1024, lse=None, ws=P, wsb=1 << 40):
        return lib.gptq_kv_attention(Q, dt, total, hq, h, D, ldq, cu, lens, table, ldt, width, batch, max_q, pool, pages,
                                     page, sm, causal, window, O, ldo, lse, ws, wsb, None)

    for kw in (dict(Q=None), dict(O=None), dict(dt=0), dict(dt=3), dict(total=-1), dict(hq=7), dict(hq=1), dict(h=0),
               dict(ldq=1000), dict(ldo=1028), dict(Q=P + 8), dict(cu=None), dict(lens=None), dict(table=None),
               dict(ldt=7), dict(width=-1), dict(width=1 << 28), dict(batch=65536), dict(batch=-1), dict(max_q=-1),
               dict(pool=None), dict(pages=0), dict(page=20), dict(sm=0.0), dict(sm=-1.0), dict(sm=float("nan")),
               dict(sm=float("inf")), dict(window=-1), dict(ws=None), dict(ws=P + 128), dict(wsb=0)):
        assert call(**kw) == bad, kw
    assert call(D=96, ldq=8192, ldo=8192) == g.GPTQ_ERR_UNSUPPORTED
    for kw in (dict(total=0), dict(batch=0), dict(max_q=0)):
        assert call(Q=None, cu=None, ws=None, **kw) == g.GPTQ_OK
    size = lib.gptq_kv_attention_workspace_size
    assert size(4, 8, 2, 128, 4, 1) > 0 and size(4, 8, 3, 128, 4, 1) == 0 and size(4, 8, 2, 96, 4, 1) == 0
    assert call(wsb=size(4, 8, 2, 128, 4, 1) - 1) == bad
    assert g.gptq_launch_count() == before


def test_adapter_refusals(g):
    lib, bad = g.library(), g.GPTQ_ERR_INVALID_ARG
    before = g.gptq_launch_count()

    def call(q=P, s=P, z=P, m=64, d=256, bits=4, gs=128, X=P, T=3, ldx=256, A=P, B=P, al=P, n=2, rank=16, ids=P, Y=P,
             yd=0, ldy=64, ws=P, wsb=1 << 40):
        return lib.gptq_adapter_linear(q, s, z, m, d, bits, gs, X, T, ldx, A, B, al, n, rank, ids, Y, yd, ldy, ws, wsb,
                                       None)

    for kw in (dict(q=None), dict(s=None), dict(z=None), dict(q=P + 8), dict(m=0), dict(d=250, ldx=256), dict(bits=5),
               dict(gs=96), dict(gs=16), dict(X=None), dict(X=P + 8), dict(T=-1), dict(T=1 << 31), dict(ldx=252),
               dict(ldx=260), dict(A=None), dict(B=None), dict(ids=None), dict(A=P + 8), dict(B=P + 2), dict(n=-1),
               dict(rank=0), dict(rank=12), dict(rank=136), dict(Y=None), dict(yd=2), dict(ldy=63), dict(ws=None),
               dict(ws=P + 64), dict(wsb=0)):
        assert call(**kw) == bad, kw
    assert call(T=0, X=None, Y=None, ws=None) == g.GPTQ_OK
    size = lib.gptq_adapter_workspace_size
    assert size(64, 256, 4, 128, 3, 16) > 0 and size(64, 256, 4, 96, 3, 16) == 0 and size(64, 256, 4, 128, 3, 12) == 0
    assert call(wsb=size(64, 256, 4, 128, 3, 16) - 1) == bad
    assert g.gptq_launch_count() == before


# ------------------------------------------------------------------ the binding
class _Recorder:
    REAL = ("gptq_kv_attention_workspace_size", "gptq_adapter_workspace_size", "gptq_status_string", "gptq_last_error")

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name in self.REAL:
            return getattr(self.real, name)

        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def fake(g, monkeypatch):
    rec = _Recorder(g.library())
    monkeypatch.setattr(g, "_lib", rec)

    def need_cuda(t, name, dtypes):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")
        if t.dtype not in dtypes:
            raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    monkeypatch.setattr(g, "_need_cuda", need_cuda)
    monkeypatch.setattr(g, "_stream", lambda s: None)
    return rec


def test_norm_rope_marshalling(g, fake):
    T, hq, hk, D = 5, 4, 2, 64
    qkv = torch.zeros((T, (hq + 2 * hk) * D), dtype=torch.bfloat16)
    Q, K = qkv[:, :hq * D].view(T, hq, D), qkv[:, hq * D:(hq + hk) * D].view(T, hk, D)
    cos = torch.zeros((9, 16))
    pos = torch.zeros(T, dtype=torch.int32)
    Qo, Ko = g.gptq_qk_norm_rope(Q, K, pos, cos, cos, wq=torch.zeros(D), eps=1e-5, out_dtype=torch.float16)
    a = fake.calls[-1][1]
    assert a[2:9] == (1, T, hq, hk, D, 512, 512) and a[10] is None and a[14:17] == (9, 32, 0) and a[20:23] == (2, 256, 128)
    assert a[1] - a[0] == 2 * hq * D
    assert Qo.dtype == Ko.dtype == torch.float16 and Ko.shape == (T, hk, D)
    Qo, Ko = g.gptq_qk_norm_rope(Q[:1], None)
    assert Ko is None and fake.calls[-1][1][5] == 0 and fake.calls[-1][1][15] == 0
    n = len(fake.calls)
    for kw in (dict(cos=cos), dict(cos=cos, sin=cos), dict(positions=pos), dict(positions=pos[:4], cos=cos, sin=cos),
               dict(wq=torch.zeros(D + 1)), dict(Q_out=torch.zeros((T, hq, D + 1), dtype=torch.bfloat16)),
               dict(positions=pos, cos=cos, sin=torch.zeros((9, 15)))):
        with pytest.raises(ValueError):
            g.gptq_qk_norm_rope(Q, K, **kw)
    with pytest.raises(ValueError):
        g.gptq_qk_norm_rope(Q, None, wk=torch.zeros(D))
    with pytest.raises(ValueError):
        g.gptq_qk_norm_rope(Q.transpose(0, 1), None)                 # heads not dense in a token's row
    with pytest.raises(TypeError):
        g.gptq_qk_norm_rope(Q, K.float())
    with pytest.raises(TypeError):
        g.gptq_qk_norm_rope(Q, K, positions=pos.long(), cos=cos, sin=cos)
    with pytest.raises(TypeError):
        g.gptq_qk_norm_rope(Q, K, out_dtype=torch.float64)
    assert len(fake.calls) == n


def test_cache_and_attention_marshalling(g, fake):
    H, D, page, pages, T = 2, 64, 16, 5, 6
    cache = g.KVCache.empty(pages, page, H, D, device="cpu")
    assert cache.pool.shape == (pages, H, 16 * 72)
    kv = torch.zeros((T, 2 * H * D), dtype=torch.float16)
    K, V = kv[:, :H * D].view(T, H, D), kv[:, H * D:].view(T, H, D)
    slots = torch.zeros(T, dtype=torch.int64)
    g.gptq_kv_append(cache, K, V, slots)
    a = fake.calls[-1][1]
    assert a[2:8] == (2, T, H, D, 256, 256) and a[10:12] == (pages, page)
    k, v = g.gptq_kv_read(cache, slots, dtype=torch.float32)
    assert k.shape == (T, H, D) and v.dtype == torch.float32 and fake.calls[-1][1][9] == 0
    Q = torch.zeros((3, 4, D), dtype=torch.bfloat16)
    cu, lens = torch.tensor([0, 1, 3], dtype=torch.int32), torch.tensor([4, 9], dtype=torch.int32)
    table = torch.zeros((2, 8), dtype=torch.int32)[:, :3]
    O = g.gptq_kv_attention(cache, Q, cu, lens, table, 2, window=4)
    a = fake.calls[-1][1]
    assert a[1:7] == (1, 3, 4, H, D, 256) and a[10:14] == (8, 3, 2, 2) and a[15:20] == (pages, page, D ** -0.5, 1, 4)
    assert O.shape == Q.shape and O.dtype == Q.dtype and a[22] is None
    n = len(fake.calls)
    bad = [lambda: g.gptq_kv_append(cache, K, V, slots[:5]), lambda: g.gptq_kv_append(cache, K[:, :1], V, slots),
           lambda: g.gptq_kv_append(g.KVCache(cache.pool, 32, H, D), K, V, slots),
           lambda: g.gptq_kv_read(cache, slots, K=K[:3].float(), dtype=torch.float32),
           lambda: g.gptq_kv_attention(cache, Q, cu[:2], lens, table, 2),
           lambda: g.gptq_kv_attention(cache, Q, cu, lens[:1], table, 2),
           lambda: g.gptq_kv_attention(cache, Q, cu, lens, table[0], 2),
           lambda: g.gptq_kv_attention(cache, Q, cu, lens, table, 2, O=torch.zeros((3, 4, 32), dtype=torch.bfloat16)),
           lambda: g.gptq_kv_attention(cache, Q, cu, lens, table, 2, lse=torch.zeros((3, 3))),
           lambda: g.gptq_kv_attention(cache, Q, cu, lens, table, 2, ws=torch.zeros(8, dtype=torch.uint8))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: g.gptq_kv_append(cache, K, V.float(), slots),
                 lambda: g.gptq_kv_attention(cache, Q.float(), cu, lens, table, 2),
                 lambda: g.gptq_kv_attention(cache, Q, cu.long(), lens, table, 2)):
        with pytest.raises(TypeError):
            call()
    assert len(fake.calls) == n


def test_adapter_marshalling(g, fake):
    m, d, T, n, r = 48, 256, 5, 3, 16
    q = g.QuantizedLayer(torch.zeros((m, 32), dtype=torch.int32), torch.zeros((m, 2)), torch.zeros((m, 2)), None, 4, 128, d)
    X = torch.zeros((T, d + 8), dtype=torch.bfloat16)[:, :d]
    A, B = torch.zeros((n, r, d), dtype=torch.bfloat16), torch.zeros((n, m, r), dtype=torch.bfloat16)
    ids, al = torch.zeros(T, dtype=torch.int32), torch.zeros(n)
    Y = g.gptq_adapter_linear(q, X, m, A, B, ids, alpha=al, out_bf16=True)
    a = fake.calls[-1][1]
    assert a[3:7] == (m, d, 4, 128) and a[8:10] == (T, d + 8) and a[13:15] == (n, r) and a[17:19] == (1, m)
    assert Y.shape == (T, m) and Y.dtype == torch.bfloat16
    g.gptq_adapter_linear(q, X, m)
    assert fake.calls[-1][1][10:14] == (None, None, None, 0)
    calls = len(fake.calls)
    bad = [lambda: g.gptq_adapter_linear(q, X, m, A, None, ids), lambda: g.gptq_adapter_linear(q, X, m, None, B),
           lambda: g.gptq_adapter_linear(q, X, m, A, B[:2], ids), lambda: g.gptq_adapter_linear(q, X, m, A, B, ids[:3]),
           lambda: g.gptq_adapter_linear(q, X, m, A[..., :8], B, ids), lambda: g.gptq_adapter_linear(q, X, m + 1, A, B, ids),
           lambda: g.gptq_adapter_linear(q, X, m, A, B, ids, alpha=al[:2]),
           lambda: g.gptq_adapter_linear(q, X[:, :128], m, A, B, ids),
           lambda: g.gptq_adapter_linear(q, X, m, A, B, ids, Y=torch.zeros((T, m + 1)))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        g.gptq_adapter_linear(q, X, m, A.float(), B, ids)
    with pytest.raises(TypeError):
        g.gptq_adapter_linear(q, X, m, A, B, ids.long())
    assert len(fake.calls) == calls


# ------------------------------------------------------------------ the oracle
def test_oracle_cache_row_by_hand():
    codes, scale, low = so.quantize_row(np.array([-1.0, 0.0, 0.25, 2.75]))
    assert scale == 0.25 and low == -1.0 and codes.tolist() == [0, 4, 5, 15]
    codes, scale, _ = so.quantize_row(np.array([0.0, 7.5, 1.25, 0.75]))          # quotients 2.5 and 1.5: ties to even
    assert scale == 0.5 and codes.tolist() == [0, 15, 2, 2]
    assert so.quantize_row(np.full(4, 3.0))[0].tolist() == [0] * 4 and so.quantize_row(np.full(4, 3.0))[1] == 0
    codes, scale, low = so.quantize_row(np.array([np.inf, -np.inf, 0.0]))
    assert low == -65504.0 and codes.tolist()[:2] == [15, 0]
    assert np.isnan(so.quantize_row(np.array([1.0, np.nan]))[1])
    pool = np.zeros((2, 1, so.block_bytes(16, 64)), np.uint8)
    k = np.arange(64.0)
    so.write_slot(pool, 16, 64, 17, 0, k, -k)
    got = so.read_slot(pool, 16, 64, 17, 0)
    assert np.abs(got[0] - k).max() <= 4.2 / 2 + 0.01 and np.abs(got[1] + k).max() <= 4.2 / 2 + 0.01
    assert not pool[0].any() and pool[1, 0, 32:64].any() and pool[1, 0, 512 + 32:512 + 64].any()


def test_oracle_attention_masks():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((4, 8)), rng.standard_normal((6, 8)), rng.standard_normal((6, 8))
    o, lse = so.attention(q, k, v, 2, 0.3)
    for i in range(4):
        e = np.exp(0.3 * k[:3 + i] @ q[i])
        assert np.allclose(o[i], e @ v[:3 + i] / e.sum()) and np.isclose(lse[i], np.log(e.sum()))
    o, lse = so.attention(q, k, v, -2, 1.0)                                      # the first two see nothing
    assert not o[:2].any() and np.isinf(lse[:2]).all() and np.allclose(o[2], v[0])
    o, _ = so.attention(q, k, v, 2, 1.0, window=1)
    assert np.allclose(o, v[2:])


def test_oracle_norm_rope_turns():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    c, s = np.array([[0.0, 1.0]]), np.array([[1.0, 0.0]])
    assert np.allclose(so.norm_rope(x, [0], c, s), [[[0, 4, 3, 0]]])             # pair (0, 2) turned by 90 degrees
    assert np.allclose(so.norm_rope(x, [0], c, s, interleaved=True), [[[-4, 3, 0, 0]]])
    assert np.allclose(so.norm_rope(x, w=np.ones(4), eps=0.0), x / 2.5)
    rng = np.random.default_rng(1)
    y = rng.standard_normal((3, 2, 16))
    a = rng.random((5, 8))
    assert np.allclose((so.norm_rope(y, [0, 2, 4], np.cos(a), np.sin(a)) ** 2).sum(-1), (y ** 2).sum(-1))


def test_act_order_layers_of_several_groups_are_refused(g):
    """The adapter projection reads natural groups; a layer that was quantized in the act-order
    permutation says so."""
    q = lambda gs, act: g.QuantizedLayer(torch.zeros((8, 8), dtype=torch.int32), torch.zeros((8, 1 if gs == -1 else 64 // gs)),
                                         torch.zeros((8, 1 if gs == -1 else 64 // gs)), None, 4, gs, 64, act_order=act)
    X = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="act-order"):
        g.gptq_adapter_linear(q(32, True), X, 8)
    for gs, act in ((32, False), (-1, True), (64, True)):          # on to the next check: not a CUDA tensor
        with pytest.raises(TypeError):
            g.gptq_adapter_linear(q(gs, act), X, 8)


@pytest.mark.gpu
def test_layers_say_whether_they_are_act_order(g):
    W, X = torch.randn((64, 256), device="cuda"), torch.randn((300, 256), device="cuda").bfloat16()
    plain, act = (g.quantize_layer(W, [X], act_order=a)[0] for a in (False, True))
    assert (plain.act_order, act.act_order) == (False, True)
    g.gptq_adapter_linear(plain, X[:3], 64)
    with pytest.raises(ValueError, match="act-order"):
        g.gptq_adapter_linear(act, X[:3], 64)
    one = g.quantize_layer(W, [X], group_size=-1, act_order=True)[0]
    assert torch.allclose(g.gptq_adapter_linear(one, X[:3], 64), g.gptq_dequant_gemv(one, X[:3], 64), rtol=1e-4, atol=1e-4)
    pipe = g.HostPipeline(64, 256, act_order=True)
    assert pipe.host_out.act_order and not g.HostPipeline(64, 256).host_out.act_order


def test_attention_refuses_lengths_whose_tiles_pass_31_bits(g):
    lib = g.library()

    def call(width, page):
        st = lib.gptq_kv_attention(P, 1, 4, 8, 2, 128, 1024, P, P, P, width, width, 4, 1, P, 64, page, 0.1, 1, 0, P, 1024, None,
                                   P, 0, None)
        assert st == g.GPTQ_ERR_INVALID_ARG
        return g.gptq_last_error()

    for page in (16, 48, 256):
        most = (2 ** 31 - 256) // page
        assert "workspace" in call(most, page)                     # the next check
        assert "table_width" in call(most + 1, page) and "table_width" in call((2 ** 31 - 1) // page + 1, page)
