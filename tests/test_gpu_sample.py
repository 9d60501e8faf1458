"""The sampler's clusters: rows that several CTAs share, in batches of every size, and beside other work."""
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


def settings(rng, n, dtype=torch.float32):
    dev = lambda a, t: torch.from_numpy(np.asarray(a, t)).cuda()
    return dict(temperature=dev(rng.uniform(0.3, 1.5, n), np.float32), top_k=dev(rng.integers(0, 300, n), np.int32),
                top_p=dev(rng.uniform(0.3, 1.05, n), np.float32), min_p=dev(0.1 * rng.random(n) ** 2, np.float32))


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("n", [1, 19, 150])
def test_rows_of_several_ctas_beside_other_work(g, n, cut):
    """Clusters that start while another stream fills the SMs, time after time: the same tokens each time."""
    rng = np.random.default_rng(n)
    v = 60000
    x = torch.from_numpy(2.5 * rng.standard_normal((n, v)).astype(np.float32)).cuda()
    u = torch.from_numpy(rng.random(n).astype(np.float32) * np.float32(1 - 2.0 ** -24)).cuda()
    s = settings(rng, n) if cut else {}
    want, lp = g.gptq_sample(x, u, **s)
    host = {k: t.cpu().tolist() for k, t in s.items()}
    for i in range(min(n, 6)):
        assert int(want[i]) == so.sample_row(x[i].cpu().double().numpy(), float(u[i]), **{k: t[i] for k, t in host.items()})[0]
    side, a = torch.cuda.Stream(), torch.randn((2048, 2048), device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(60):
        with torch.cuda.stream(side):
            b = a @ a
            b.add_(1.0)
        tokens, l = g.gptq_sample(x, u, **s)
        assert torch.equal(tokens, want) and torch.equal(l, lp)
    torch.cuda.synchronize()
    g.gptq_device_check()


def test_rows_with_bad_settings_end_in_clusters_too(g):
    """Rows of eight CTAs whose settings are refused beside ones that are drawn."""
    n, v = 6, 128000
    x = torch.randn((n, v), device="cuda")
    u = torch.tensor([0.5, 1.0, 0.25, -1.0, float("nan"), 0.75], device="cuda")
    tokens, lp = g.gptq_sample(x, u, top_p=torch.full((n,), 0.9, device="cuda"))
    torch.cuda.synchronize()
    with pytest.raises(g.GPTQError):
        g.gptq_device_check()
    g.gptq_device_check()
    t = tokens.tolist()
    assert t[1] == t[3] == t[4] == -1 and min(t[0], t[2], t[5]) >= 0 and torch.isnan(lp[[1, 3, 4]]).all()
