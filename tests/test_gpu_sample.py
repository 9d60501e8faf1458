"""The sampler's clusters: rows that several CTAs share, in batches of every size, and beside other work."""
import math

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


# ------------------------------------------------------------------ the border of top_p
def flat(rng, n, v):
    """Rows whose tokens each have a share of about 1 / v: fp32 sums of so many are off by more than that."""
    return torch.from_numpy((0.05 * rng.standard_normal((n, v))).astype(np.float32))


def kept_of(x, p, T, k=0):
    """The tokens that top_p keeps of a row, by falling logit, from 64 bits, and how far the border is from either neighbour, as a
    share of the mass."""
    order = np.argsort(-x, kind="stable")
    if k:
        order = order[:k]
    w = np.exp((x[order] - x[order[0]]) / T)
    c = np.cumsum(w)
    p = float(np.float32(p))
    n = int(np.searchsorted(c - w, p * c[-1], side="left"))
    gap = np.abs(np.concatenate([(c - w)[max(n - 1, 0):n + 1], c[n - 1:n]]) / c[-1] - p).min()
    return order[:n], gap


@pytest.mark.parametrize("k", [0, 100000])
@pytest.mark.parametrize("v", [150000, 262144])
def test_the_border_of_top_p_in_flat_rows(g, v, k):
    """Each row's u draws the last kept token by index, and the border's token is the last one there is: drawn if it is kept. Weights
    are exact to 2^-30, so a border may fall either way within that share of the mass from a token's end; here none is so near."""
    rng = np.random.default_rng(v + k)
    n = 12
    x = flat(rng, n, v)
    p = rng.uniform(0.2, 0.98, n).astype(np.float32)
    T = rng.uniform(0.5, 2.0, n).astype(np.float32)
    for rows in (range(n), [0], [5]):
        rows = list(rows)
        dev = lambda a, t: torch.from_numpy(np.asarray(a, t)[rows]).cuda()
        u = np.full(n, 1 - 2.0 ** -24, np.float32)
        # the token at the border is the last by index where it is moved there
        y = x.clone()
        want = []
        for i in range(n):
            kept, gap = kept_of(x[i].double().numpy(), p[i], float(T[i]), k)
            assert gap > 2.0 ** -30
            last, end = int(kept[-1]), v - 1
            y[i, last], y[i, end] = x[i, end], x[i, last]
            kept, _ = kept_of(y[i].double().numpy(), p[i], float(T[i]), k)
            assert int(kept[-1]) == end
            want.append(end)
        s = dict(temperature=dev(T, np.float32), top_p=dev(p, np.float32))
        if k:
            s["top_k"] = torch.full((len(rows),), k, dtype=torch.int32, device="cuda")
        tokens, lp = g.gptq_sample(y[rows].cuda(), dev(u, np.float32), **s)
        torch.cuda.synchronize()
        g.gptq_device_check()
        got = tokens.cpu().tolist()
        for j, i in enumerate(rows):
            exact, _ = so.sample_row(y[i].double().numpy(), float(u[i]), float(T[i]), k, float(p[i]))
            assert exact == want[i] and got[j] == exact, (i, got[j], exact)
            # one token less, or more, moves the share of the mass by about 1 / v
            kept = so.sample_row(y[i].double().numpy(), float(u[i]), float(T[i]), k, float(p[i]))[1]
            assert abs(lp[j].item() - kept) <= 2.0 ** -21 * (1 + math.log(v))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("k", [0, 4000])
def test_a_row_alone_and_in_a_batch(g, dtype, k):
    """The same rows alone, by threes and in a batch of 200, which share them out among 8, 8 and 2 CTAs: the same tokens, bit by
    bit the same log probabilities."""
    rng = np.random.default_rng(k)
    n, v = 200, 40000
    x = torch.from_numpy(np.where(np.arange(n)[:, None] % 2, 0.02, 2.0) * rng.standard_normal((n, v))).to(dtype).cuda()
    dev = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()
    u, s = dev(rng.random(n) * (1 - 2.0 ** -24)), dict(top_p=dev(rng.uniform(0.1, 0.999, n)), temperature=dev(rng.uniform(0.5, 3.0, n)))
    if k:
        s["top_k"] = torch.full((n,), k, dtype=torch.int32, device="cuda")
    tokens, lp = g.gptq_sample(x, u, **s)
    for rows in [slice(i, i + 1) for i in range(0, 20)] + [slice(i, i + 3) for i in range(20, 60, 3)]:
        t, l = g.gptq_sample(x[rows], u[rows], **{a: b[rows] for a, b in s.items()})
        assert torch.equal(t, tokens[rows]) and torch.equal(l, lp[rows])
    for i in range(0, n, 25):
        want = so.sample_row(x[i].cpu().double().numpy(), float(u[i]), float(s["temperature"][i]), k, float(s["top_p"][i]))
        assert int(tokens[i]) == want[0]
    torch.cuda.synchronize()
    g.gptq_device_check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["steps", "two", "tail", "near zero", "far below"])
def test_the_border_of_top_p_among_equal_and_close_logits(g, kind, dtype):
    """Values of which many share a place but not a key, many share both, and tails that weigh next to nothing."""
    rng = np.random.default_rng(len(kind))
    n, v = 8, 30000
    x = {"steps": np.round(4 * rng.standard_normal((n, v))) / 4, "two": np.where(rng.random((n, v)) < 0.4, 1.0, 0.75),
         "tail": np.where(rng.random((n, v)) < 1e-3, 3.0, -26.0 + rng.standard_normal((n, v))),
         "near zero": 20.0 * (rng.random((n, v)) < 1e-4) + 1e-5 * rng.standard_normal((n, v)),
         "far below": -1000.0 + 1e-3 * rng.standard_normal((n, v))}[kind]
    x = torch.from_numpy(x).to(dtype)
    u = (rng.random(n) * (1 - 2.0 ** -24)).astype(np.float32)
    for p in (0.1, 0.5, 0.9, 0.999, 1 - 2.0 ** -24, 0.0, -1.0):
        for k in (0, 700, 20000):
            s = dict(top_p=torch.full((n,), p, device="cuda"))
            if k:
                s["top_k"] = torch.full((n,), k, dtype=torch.int32, device="cuda")
            tokens, _ = g.gptq_sample(x.cuda(), torch.from_numpy(u).cuda(), **s)
            got = tokens.cpu().tolist()
            for i in range(n):
                assert got[i] == so.sample_row(x[i].double().numpy(), float(u[i]), 1.0, k, float(np.float32(p)))[0], (kind, p, k, i)
    torch.cuda.synchronize()
    g.gptq_device_check()
