"""(0, rank, d) adapters are none, by both ways into the library and both packed projections."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    from post_weight_quantization_gb300 import build as b
    b.build()
    from post_weight_quantization_gb300 import gptq
    return gptq


@pytest.mark.parametrize("T", [0, 1, 30, 300])
def test_no_adapters_to_choose_from(g, T):
    m, d, rank = 96, 256, 16
    q = g.QuantizedLayer(torch.randint(-2 ** 31, 2 ** 31, (m, d // 8), device="cuda", dtype=torch.int64).int(),
                         torch.full((m, 2), 0.01, device="cuda"), torch.full((m, 2), 8.0, device="cuda"), None, 4, 128, d)
    X = torch.randn((T, d), device="cuda").bfloat16()
    none = dict(A=torch.empty((0, rank, d), dtype=torch.bfloat16, device="cuda"), B=torch.empty((0, m, rank), dtype=torch.bfloat16, device="cuda"),
                ids=torch.full((T,), -1, dtype=torch.int32, device="cuda"), alpha=torch.empty(0, device="cuda"))
    want, base = g.gptq_linear(q, X, m, act="silu"), g.gptq_adapter_linear(q, X, m)
    for stream in (None, torch.cuda.current_stream()):
        assert torch.equal(g.gptq_linear(q, X, m, act="silu", stream=stream, **none), want)
        assert torch.equal(g.gptq_adapter_linear(q, X, m, stream=stream, **none), base)
        with pytest.raises(ValueError):                     # 8-bit tokens take no adapters, not even none
            g.gptq_linear(q, X.to(torch.float8_e4m3fn), m, x_scale=torch.ones(T, device="cuda"), stream=stream, **none)
    torch.cuda.synchronize()
    g.gptq_device_check()
