"""The activations' own arithmetic, in each of the three kernels that a packed projection may take, in fp32: tokens of zeros, so that
the bias alone is z, exactly. Against 64 bits, in 2^-23 of |act(z)| (the exponential errs by 2 + 1.2 y units of the last place, y the
exponent's size, the quotient by 2, erfcf by 4):
  silu       its divisor rounds once: 5 + 1.2 |z|
  gelu_tanh  the exponent y = 1.6 |z| (1 + 0.045 z^2) is off by six roundings, 3 y units: 5 + 4.2 y
  gelu       the argument's two roundings move erfc by z^2 + |z|: 5 + z^2 + |z|
and for positive z, where the exponential is the smaller part of the divisor, or erfc next to 2, 5. Where the divisor passes 2^126
the quotient is 0: 2^-126 |z|, which also covers what is below fp32's normal range.
"""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    from post_weight_quantization_gb300 import build as b
    b.build()
    from post_weight_quantization_gb300 import gptq
    return gptq


@pytest.mark.parametrize("T", [1, 20, 2600])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_activations_alone(g, T, act):
    m, d = 6000, 128
    rng = np.random.default_rng(T)
    z = np.concatenate([np.linspace(-100, 100, 2000), np.linspace(-8, 8, 2000), rng.standard_normal(1000), 1e-6 * rng.standard_normal(998),
                        [0.0, -0.0]]).astype(np.float32)
    q = g.QuantizedLayer(torch.zeros((m, d // 8), dtype=torch.int32, device="cuda"), torch.ones((m, 1), device="cuda"),
                         torch.zeros((m, 1), device="cuda"), None, 4, 128, d)
    x = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    Y = g.gptq_linear(q, x, m, bias=torch.from_numpy(z).cuda(), act=act)
    torch.cuda.synchronize()
    g.gptq_device_check()
    assert torch.equal(Y, Y[:1].expand_as(Y))
    got, z = Y[0].cpu().double().numpy(), z.astype(np.float64)
    want, a = so.activation(z, act), np.abs(z)
    n = {"relu": 0 * z, "silu": 5 + 1.2 * a, "gelu": 5 + z * z + a, "gelu_tanh": 5 + 4.2 * 1.6 * a * (1 + 0.045 * z * z)}[act]
    bound = np.where(z > 0, np.minimum(n, 5), n) * 2.0 ** -23 * np.abs(want) + 2.0 ** -126 * a
    assert np.all(np.abs(got - want) <= bound), float(np.max(np.abs(got - want) / np.maximum(bound, 1e-300)))
