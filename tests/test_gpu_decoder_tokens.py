"""A decoder's steps at their edges: tokens outside the vocabulary, and no tokens at all."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dec():
    from post_weight_quantization_gb300 import build as b
    b.build()
    from post_weight_quantization_gb300 import decoder
    return decoder


def model_of(dec, eight_bit):
    return dec.random_decoder(vocab=300, hidden=256, wide=512, layers=2, heads=4, kv_heads=2, head_dim=64, num_pages=40, page_size=16,
                              group_size=64, eight_bit=eight_bit, positions=200, seed=11)


@pytest.mark.parametrize("eight_bit", [False, True])
@pytest.mark.parametrize("bad", [-1, 300, 2 ** 31 - 1, -2 ** 31])
def test_tokens_outside_the_vocabulary(dec, bad, eight_bit):
    """Their sequence has NaN for logits and -1 for its next tokens; the others have what they have without it."""
    model = model_of(dec, eight_bit)
    lens = [40, 1, 17]
    tokens = torch.randint(0, 300, (sum(lens),), generator=torch.Generator().manual_seed(1)).int().cuda()
    u = torch.rand((3, 3), generator=torch.Generator().manual_seed(2)).cuda()
    runs = []
    for wrong in (False, True):
        t = tokens.clone()
        if wrong:
            t[40] = bad                                     # the second sequence's only token
        for layer in model.layers:
            layer.attention.cache.pool.zero_()
        batch = dec.Batch(40, 16)
        for _ in lens:
            batch.add()
        step, out = batch.extend(lens, 8), []
        for i in range(3):
            logits = model.logits(t, step)
            token, lp = dec.gptq.gptq_sample(logits, u[i])
            out.append((logits, token, lp))
            t, step = token, batch.extend([1, 1, 1], 8)
        runs.append(out)
    torch.cuda.synchronize()
    dec.gptq.gptq_device_check()
    for (l0, t0, p0), (l1, t1, p1) in zip(*runs):
        assert torch.isfinite(l0).all() and int(t0.min()) >= 0
        for i in (0, 2):
            assert torch.equal(l0[i], l1[i]) and t0[i] == t1[i] and p0[i] == p1[i]
        assert torch.isnan(l1[1]).all() and int(t1[1]) == -1 and torch.isnan(p1[1])


def test_a_step_without_tokens(dec):
    model = model_of(dec, False)
    batch = dec.Batch(40, 16)
    for _ in range(2):
        batch.add()
    prompt = torch.arange(30, dtype=torch.int32, device="cuda")
    before = model.logits(prompt, batch.extend([20, 10], 4))
    pools = [layer.attention.cache.pool.clone() for layer in model.layers]
    u = torch.zeros(2, device="cuda")
    token, _ = model.forward(prompt[:0], batch.extend([0, 0], 4), u)
    assert token.shape == (2,) and model.logits(prompt[:0], batch.extend([0, 0], 4)).shape == before.shape
    assert all(torch.equal(layer.attention.cache.pool, p) for layer, p in zip(model.layers, pools))
    one = model.logits(prompt[:1], batch.extend([0, 1], 4))
    assert torch.isfinite(one).all()
    torch.cuda.synchronize()
    dec.gptq.gptq_device_check()
