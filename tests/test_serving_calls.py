"""The serving operators' two ways from Python to the library: the module that takes what a decoding
loop passes, and the binding's own checks for everything else. Both give the same bits, and what
the module declines the binding refuses, or allows, as it says."""
import sys

import pytest
import torch


@pytest.fixture(scope="module")
def g():
    from post_weight_quantization_gb300 import build as b
    b.build()
    from post_weight_quantization_gb300 import gptq
    return gptq


NAMES = ("adapter_linear", "qk_norm_rope", "kv_append", "kv_read", "kv_attention")


class Spy:
    """The module, noting which calls it took."""

    def __init__(self, calls):
        self.taken = []
        for name in NAMES:
            def call(*args, f=getattr(calls, name), name=name):
                got = f(*args)
                self.taken.append((name, got is not None))
                return got
            setattr(self, name, call)


@pytest.fixture
def spy(g, monkeypatch):
    s = Spy(g._calls)
    monkeypatch.setattr(g, "_calls", s)
    return s


def test_declines_what_is_not_on_the_gpu(g):
    c = g._calls
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    assert c.qk_norm_rope(x, None, None, None, None, None, None, 1e-6, False, None, None, None) is None
    pool = torch.zeros((2, 4, 16 * 72), dtype=torch.uint8)
    slots = torch.zeros(2, dtype=torch.int64)
    assert c.kv_append(pool, 16, 4, 64, x, x, slots) is None
    assert c.kv_read(pool, 16, 4, 64, slots, torch.bfloat16, None, None) is None
    assert c.kv_attention(pool, 16, 4, 64, x, None, None, None, 1, None, True, 0, None, None, None) is None
    assert c.adapter_linear(*[None] * 15) is None
    assert c.qk_norm_rope(*["x"] * 12) is None
    with pytest.raises(TypeError):
        c.kv_append(pool)


def _all_calls(g, stream, given):
    """Every operator once; with `given`, into the caller's outputs and workspaces."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    T, hq, hk, D, page, m, d = 5, 8, 2, 64, 16, 96, 256
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()
    Q, K, V, X = rnd(T, hq, D), rnd(T, hk, D), rnd(T, hk, D), rnd(T, d)
    cos, sin = torch.rand((2, 50, D // 2), generator=gen, device="cuda")
    w = torch.rand(D, generator=gen, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    out = {}
    kw = dict(Q_out=torch.empty_like(Q), K_out=torch.empty_like(K)) if given else {}
    out["norm"] = g.gptq_qk_norm_rope(Q, K, pos, cos, sin, w, w, eps=1e-5, stream=stream, **kw)
    if given:
        assert out["norm"][0] is kw["Q_out"] and out["norm"][1] is kw["K_out"]
    out["only q"] = g.gptq_qk_norm_rope(Q, None, out_dtype=torch.float32, wq=w, stream=stream)
    assert out["only q"][1] is None
    cache = g.KVCache(torch.zeros((3, hk, page * (D + 8)), dtype=torch.uint8, device="cuda"), page, hk, D)
    slots = torch.arange(20, 20 + T, device="cuda")
    assert g.gptq_kv_append(cache, K, V, slots, stream=stream) is None
    out["pool"] = (cache.pool,)
    kw = dict(K=torch.empty_like(K), V=torch.empty_like(V)) if given else {}
    out["read"] = g.gptq_kv_read(cache, slots, stream=stream, **kw)
    cu, lens = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 2, T], [5, 9]))
    table = torch.tensor([[1, 0], [1, 2]], dtype=torch.int32, device="cuda")
    need = g._lib.gptq_kv_attention_workspace_size(T, hq, hk, D, 2, 3)
    kw = dict(O=torch.empty_like(Q), ws=torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")) if given else {}
    lse = torch.empty((T, hq), device="cuda")
    out["attention"] = (g.gptq_kv_attention(cache, Q, cu, lens, table, 3, window=4, lse=lse, stream=stream, **kw), lse)
    if given:
        assert out["attention"][0] is kw["O"]
    q = g.QuantizedLayer(torch.randint(-2 ** 31, 2 ** 31 - 1, (m, d // 8), generator=gen, dtype=torch.int32, device="cuda"),
                         torch.rand((m, 2), generator=gen, device="cuda"), torch.full((m, 2), 8.0, device="cuda"), None, 4, 128, d)
    A, B = rnd(3, 8, d), rnd(3, m, 8)
    ids = torch.tensor([0, 2, -1, 1, 2], dtype=torch.int32, device="cuda")
    kw = dict(Y=torch.empty((T, m), device="cuda")) if given else {}
    out["adapter"] = (g.gptq_adapter_linear(q, X, m, A, B, ids, torch.rand(3, generator=gen, device="cuda"), stream=stream, **kw),)
    out["layer"] = (g.gptq_adapter_linear(q, X[:1], m, out_bf16=True, stream=stream),)
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("given", [False, True])
def test_both_ways_give_the_same(g, spy, given):
    short = _all_calls(g, None, given)
    assert len(spy.taken) == 7 and all(took for _, took in spy.taken) and {n for n, _ in spy.taken} == set(NAMES)
    long = _all_calls(g, torch.cuda.current_stream(), given)
    assert len(spy.taken) == 7
    torch.cuda.synchronize()
    g.gptq_device_check()
    for name, ts in short.items():
        for a, b in zip(ts, long[name]):
            assert (a is None and b is None) or torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name


@pytest.mark.gpu
def test_unusual_arguments_go_the_long_way(g, spy):
    Q = torch.randn((3, 2, 64), device="cuda").bfloat16()
    g.gptq_qk_norm_rope(Q, None, eps=1)                        # an int for a float: allowed
    assert spy.taken[-1] == ("qk_norm_rope", False)
    X = torch.randn((2, 256), device="cuda").bfloat16()
    q = g.QuantizedLayer(torch.zeros((8, 32), dtype=torch.int32, device="cuda"), torch.ones((8, 2), device="cuda"),
                         torch.zeros((8, 2), device="cuda"), None, 4, 128, 256)
    a, b = g.gptq_adapter_linear(q, X.view(torch.int16), 8), g.gptq_adapter_linear(q, X, 8)
    assert spy.taken[-2:] == [("adapter_linear", False), ("adapter_linear", True)] and torch.equal(a, b)
    for bad in (lambda: g.gptq_qk_norm_rope(Q.double(), None), lambda: g.gptq_qk_norm_rope(Q.transpose(0, 1), None),
                lambda: g.gptq_adapter_linear(q, X, 9), lambda: g.gptq_adapter_linear(q, X.float(), 8),
                lambda: g.gptq_adapter_linear(q, X, 8, ws=torch.zeros(8, dtype=torch.uint8, device="cuda"),
                                              A=torch.zeros((1, 8, 256), dtype=torch.bfloat16, device="cuda"),
                                              B=torch.zeros((1, 8, 8), dtype=torch.bfloat16, device="cuda"),
                                              ids=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            bad()
        assert not spy.taken[-1][1]
    # a group size the library does not take: declined, then refused with the library's reason
    q3 = g.QuantizedLayer(q.qweight, torch.ones((8, 16), device="cuda"), torch.zeros((8, 16), device="cuda"), None, 4, 16, 256)
    with pytest.raises(g.GPTQError):
        g.gptq_adapter_linear(q3, X, 8)
    torch.cuda.synchronize()
    g.gptq_device_check()


@pytest.mark.gpu
def test_references_and_memory_are_given_back(g):
    Q = torch.randn((3, 2, 64), device="cuda").bfloat16()
    out = torch.empty_like(Q)
    for _ in range(10):
        g.gptq_qk_norm_rope(Q, None, Q_out=out)
        g.gptq_qk_norm_rope(Q, None)
    torch.cuda.synchronize()
    refs, held = [sys.getrefcount(x) for x in (Q, out, None)], torch.cuda.memory_allocated()
    for _ in range(200):
        g.gptq_qk_norm_rope(Q, None, Q_out=out)
        g.gptq_qk_norm_rope(Q, None)
    assert [sys.getrefcount(x) for x in (Q, out)] == refs[:2] and torch.cuda.memory_allocated() == held
    assert abs(sys.getrefcount(None) - refs[2]) < 100


@pytest.mark.gpu
def test_other_threads_go_on_while_a_launch_waits(g):
    """A launch waits while the stream's queue is full; other Python threads run meanwhile."""
    import threading
    import time
    Q = torch.randn((3, 2, 64), device="cuda").bfloat16()
    out = torch.empty_like(Q)
    for _ in range(3):
        g.gptq_qk_norm_rope(Q, None, Q_out=out)
    torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    gaps, stop = [], threading.Event()

    def tick():
        at = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps.append(now - at)
            at = now
    thread = threading.Thread(target=tick)
    thread.start()
    start = time.perf_counter()
    torch.cuda._sleep(2_000_000_000)                               # about a second
    for _ in range(6000):                                          # more than a queue holds
        g.gptq_qk_norm_rope(Q, None, Q_out=out)
    waited = time.perf_counter() - start
    stop.set()
    thread.join()
    torch.cuda.synchronize()
    assert waited > 0.4, waited                                    # the launches did wait
    assert max(gaps) < waited / 2, (max(gaps), waited)
