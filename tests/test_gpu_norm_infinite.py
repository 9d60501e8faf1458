"""8-bit rows whose product with the weights is infinite: no number for a scale or a code."""
import pytest
import torch

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def g():
    from post_weight_quantization_gb300 import build as b
    b.build()
    from post_weight_quantization_gb300 import gptq
    return gptq


@pytest.mark.parametrize("d", [64, 1024, 4096, 20000])
def test_infinite_products_with_weights(g, d):
    x = torch.ones((5, d))
    x[1] = 1e15
    x[2, 7] = 0.0                                            # times the infinite weight: no number
    x[4] = 0.0
    w = torch.ones(d)
    w[7], w[9] = float("inf"), 1e30                          # 1e15 * 1e30 passes fp32's range
    for weights, nan in ((w, [0, 1, 2, 3, 4]), (torch.where(torch.isinf(w), torch.ones(d), w), [1])):
        Q, _, scale = g.gptq_add_rms_norm(x.cuda(), w=weights.cuda(), eps=1e-6, out_dtype=E4M3)
        torch.cuda.synchronize()
        g.gptq_device_check()
        Q, scale = Q.float().cpu(), scale.cpu()
        for i in range(5):
            if i in nan:
                assert torch.isnan(scale[i]) and torch.isnan(Q[i]).all(), (i, scale[i])
            else:
                assert torch.isfinite(scale[i]) and torch.isfinite(Q[i]).all()
        if len(nan) == 1:
            assert scale[4] == 0 and Q[0, 9] == 448 and abs(scale[0] * 448 / 1e30 - 1) < 1e-5
