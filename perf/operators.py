"""The serving operators' workloads: what is timed, on which inputs, and their plain forms.

Four operators of a decoder block whose projections are stored as packed codes:

  adapter    a packed projection with the low-rank adapters of many requests beside it
  norm_rope  the norm of each query and key head and the position rotation, in one pass
  append     K and V rows quantized to 4 bits into the pages of a cache, and read back
  attention  attention over that cache through a page table

Shapes are those of the layers that this package quantizes: a 4096-wide projection with 32
heads of 128, and a block of hidden width 8192 with 64 query heads, 8 key/value heads of 128
and 28672-wide MLP layers.

`run` computes an operator in elementary torch operations in fp32, or, with `own` set, by
the package's entry points. A cache is one uint8 tensor (pages, heads, page_size * (D + 8)):
per page and head first the K codes of its tokens (D / 2 bytes each, two codes per byte, the
lower half first), then the V codes, then four float16 per token: K scale, K lowest value,
V scale, V lowest value. A value is code * scale + lowest.
"""
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one request through a 4096-wide projection with its adapter: latency
        dict(name="adapter 1 token 4096", op="adapter", m=4096, d=4096, bits=4, group=128, tokens=1, rank=16,
             adapters=8, requests=1, out="float32"),
        # a decoding batch: 48 requests, one token each, most with an adapter of their own
        dict(name="adapter 48 tokens 8192", op="adapter", m=8192, d=8192, bits=4, group=128, tokens=48, rank=16,
             adapters=64, requests=48, out="bfloat16"),
        # the 2-bit variant of the grouped key projection, a few requests, wider adapters
        dict(name="adapter 2-bit 13 tokens", op="adapter", m=1024, d=8192, bits=2, group=64, tokens=13, rank=64,
             adapters=16, requests=13, out="bfloat16"),
        # prompts of nine requests run together, of uneven lengths
        dict(name="adapter prompts 3001 tokens", op="adapter", m=4096, d=4096, bits=4, group=128, tokens=3001, rank=16,
             adapters=32, requests=9, out="bfloat16"),
        # a decoding batch's queries and keys
        dict(name="norm_rope 33 tokens", op="norm_rope", tokens=33, heads=64, kv_heads=8, dim=128, rot=128,
             interleaved=False, weights=True, kind="bfloat16"),
        # a prompt's queries and keys
        dict(name="norm_rope 16381 tokens", op="norm_rope", tokens=16381, heads=64, kv_heads=8, dim=128, rot=128,
             interleaved=False, weights=True, kind="bfloat16"),
        # a decoding batch's keys and values into the cache
        dict(name="append 33 tokens", op="append", tokens=33, kv_heads=8, dim=128, page=64, kind="bfloat16"),
        # a long prompt's keys and values into the cache
        dict(name="append 30011 tokens", op="append", tokens=30011, kv_heads=8, dim=128, page=64, kind="bfloat16"),
        # one short conversation of the 4096-wide model: latency
        dict(name="attention 1 x 331", op="attention", heads=32, kv_heads=32, dim=128, page=16, batch=1, new=1,
             shortest=331, longest=331, window=0, kind="bfloat16"),
        # an ordinary decoding batch of ragged lengths
        dict(name="attention 48 ragged 4096", op="attention", heads=64, kv_heads=8, dim=128, page=64, batch=48, new=1,
             shortest=60, longest=4099, window=0, kind="bfloat16"),
        # two long documents, each split over the whole GPU
        dict(name="attention 2 x 131000", op="attention", heads=64, kv_heads=8, dim=128, page=64, batch=2, new=1,
             shortest=120000, longest=131001, window=0, kind="bfloat16"),
        # a piece of a long prompt: its new tokens over what the cache holds already
        dict(name="attention piece of 1024 over 8192", op="attention", heads=64, kv_heads=8, dim=128, page=64, batch=1,
             new=1024, shortest=8187, longest=8187, window=0, kind="bfloat16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adapter", "adapter", "norm_rope", "append", "attention", "attention", "attention"])
    if op == "adapter":
        bits, group = rng.choice([(4, 128), (4, 128), (2, 64), (3, 128), (8, 128)])
        m, d = rng.choice([(4096, 4096), (8192, 8192), (1024, 8192), (11008, 4096), (4096, 11008), (1000, 4096)])
        few = rng.random() < 0.7
        tokens = _log(rng, 1, 128) if few else _log(rng, 129, 3001)
        if m * d * tokens > 4096 * 4096 * 3001:
            tokens = 4096 * 4096 * 3001 // (m * d)
        requests = tokens if few else rng.randint(1, 16)
        return dict(op=op, m=m, d=d, bits=bits, group=group, tokens=tokens, rank=rng.choice([8, 16, 16, 32, 64]),
                    adapters=rng.randint(1, 64), requests=requests, out=rng.choice(["bfloat16", "bfloat16", "float32"]))
    kind = rng.choice(["bfloat16", "bfloat16", "float16"])
    dim = rng.choice([64, 128, 128, 256])
    if op == "norm_rope":
        heads, kv_heads = rng.choice([(32, 32), (64, 8), (8, 1), (28, 4)])
        tokens = _log(rng, 1, max(1, 16381 * 72 * 128 // ((heads + kv_heads) * dim)))
        return dict(op=op, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, dim // 4]), interleaved=rng.random() < 0.3,
                    weights=rng.random() < 0.8, kind=kind)
    page = rng.choice([16, 32, 64, 64, 128])
    if op == "append":
        kv_heads = rng.choice([1, 4, 8, 32])
        tokens = _log(rng, 1, max(1, 30011 * 8 * 128 // (kv_heads * dim)))
        return dict(op=op, tokens=tokens, kv_heads=kv_heads, dim=dim, page=page, kind=kind)
    heads, kv_heads = rng.choice([(32, 32), (64, 8), (32, 8), (28, 4), (16, 1)])
    new = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 1024)])
    if new <= 8:
        batch = _log(rng, 1, 96)
        longest = _log(rng, 17, max(18, min(131001, 2 * 131001 * 8 * 128 // (batch * kv_heads * dim))))
        longest = max(new, min(longest, 2 * 131001 * 64 * 128 // (batch * heads * dim * new)))
    else:
        batch = rng.randint(1, 4)
        longest = max(new, _log(rng, new, max(new + 1, 1024 * 8187 * 64 * 128 // (new * batch * heads * dim))))
        longest = min(longest, max(new, 131001 * 8 * 128 // (batch * kv_heads * dim)))
    shortest = max(new, rng.choice([longest, longest // 3, 1]))
    return dict(op=op, heads=heads, kv_heads=kv_heads, dim=dim, page=page, batch=batch, new=new, shortest=shortest,
                longest=longest, window=rng.choice([0, 0, 0, max(1, longest // 2)]), kind=kind)


def _lengths(case):
    """The lengths of a batch's sequences: spread evenly from the shortest to the longest."""
    n, lo, hi = case["batch"], case["shortest"], case["longest"]
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def work(case):
    op = case["op"]
    if op == "adapter":
        m, d, t, r = case["m"], case["d"], case["tokens"], case["rank"]
        used = min(case["adapters"], case["requests"])
        size = 4 if case["out"] == "float32" else 2
        return {"bytes": m * d * case["bits"] // 8 + 8 * m * (d // case["group"]) + 2 * t * d + 2 * used * r * (m + d)
                + 4 * t + size * t * m,
                "flops": 2 * t * m * d + 2 * t * r * (m + d)}
    if op == "norm_rope":
        t, n, dim = case["tokens"], case["heads"] + case["kv_heads"], case["dim"]
        return {"bytes": 4 * t * n * dim + 4 * t * case["rot"] + 4 * t, "flops": t * n * (4 * dim + 3 * case["rot"])}
    if op == "append":
        t, h, dim = case["tokens"], case["kv_heads"], case["dim"]
        return {"bytes": 4 * t * h * dim + t * h * (dim + 8) + 4 * t * h * dim + 8 * t, "flops": 10 * t * h * dim}
    h, hq, dim, new, w = case["kv_heads"], case["heads"], case["dim"], case["new"], case["window"]
    read = pairs = 0
    for n in _lengths(case):
        read += min(n, w + new - 1) if w else n
        # token i of the new ones sees n - new + i + 1 keys, at most w of them
        seen = [n - new + 1, n]
        if w and seen[1] > w:
            full = seen[1] - max(seen[0], w) + 1
            pairs += full * w + ((w - 1 + seen[0]) * (w - seen[0]) // 2 if seen[0] < w else 0)
        else:
            pairs += (seen[0] + seen[1]) * new // 2
    return {"bytes": read * h * (dim + 8) + 4 * case["batch"] * new * hq * dim, "flops": 4 * pairs * hq * dim}


# ---------------------------------------------------------------------------- inputs
def _quantize(x):
    """Codes, scale and lowest value (float16) of the rows of x (..., D) in fp32."""
    x = x.float().clamp(-65504.0, 65504.0)
    low, high = x.amin(-1), x.amax(-1)
    scale = ((high - low) / torch.full_like(low, 15.0)).half()
    low = low.half()
    s = scale.float()[..., None]
    codes = torch.where(s > 0, (x - low.float()[..., None]) / s, torch.zeros_like(x))
    codes = torch.round(codes).clamp(0.0, 15.0)
    return codes, scale, low


def _pack(codes):
    c = codes.to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _rows(gen, shape, dtype):
    """Keys or values: unit normal with a few channels well off zero, as projections give."""
    x = torch.randn(shape, device=DEV, generator=gen)
    offset = torch.randn(shape[-2:], device=DEV, generator=gen)
    return (x + torch.where(offset > 1.8, 3.0 * offset, 0.2 * offset)).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed * 7919 + 17)
    op = case["op"]
    s = {"op": op}
    if op == "adapter":
        m, d, bits, t = case["m"], case["d"], case["bits"], case["tokens"]
        groups = d // case["group"]
        s.update(m=m, d=d, bits=bits, group=case["group"], out=getattr(torch, case["out"]))
        s["qweight"] = torch.randint(-2 ** 31, 2 ** 31, (m, d * bits // 32), device=DEV, dtype=torch.int64,
                                     generator=gen).to(torch.int32)
        s["scales"] = (0.5 + torch.rand((m, groups), device=DEV, generator=gen)) * (0.12 / 2 ** bits)
        s["zeros"] = torch.full((m, groups), 2.0 ** (bits - 1), device=DEV) - torch.randint(
            0, 2, (m, groups), device=DEV, generator=gen)
        s["X"] = torch.randn((t, d), device=DEV, generator=gen).to(torch.bfloat16)
        n, r = case["adapters"], case["rank"]
        s["A"] = (torch.randn((n, r, d), device=DEV, generator=gen) / d ** 0.5).to(torch.bfloat16)
        s["B"] = (torch.randn((n, m, r), device=DEV, generator=gen) / r ** 0.5).to(torch.bfloat16)
        s["alpha"] = 0.5 + torch.rand((n,), device=DEV, generator=gen)
        # each request is a run of tokens with one adapter; now and then a request has none
        ends = torch.sort(torch.rand((case["requests"] - 1,), device=DEV, generator=gen) * t)[0]
        of = torch.searchsorted(ends, torch.arange(t, device=DEV) + 0.5) if case["requests"] < t else torch.arange(
            t, device=DEV)
        first = int(torch.randint(0, n, (1,), device=DEV, generator=gen))
        ids = (of + first) % n
        none = torch.rand((case["requests"],), device=DEV, generator=gen) < 0.1
        none[0] = False
        s["ids"] = torch.where(none[of], torch.full_like(ids, -1), ids).to(torch.int32)
    elif op == "norm_rope":
        t, dim, kind = case["tokens"], case["dim"], getattr(torch, case["kind"])
        hq, hk = case["heads"], case["kv_heads"]
        # queries, keys and values come out of one projection, side by side
        qkv = torch.randn((t, (hq + 2 * hk) * dim), device=DEV, generator=gen).to(kind)
        s["Q"] = qkv[:, :hq * dim].view(t, hq, dim)
        s["K"] = qkv[:, hq * dim:(hq + hk) * dim].view(t, hk, dim)
        s["wq"] = s["wk"] = None
        if case["weights"]:
            s["wq"] = 1.0 + 0.1 * torch.randn((dim,), device=DEV, generator=gen)
            s["wk"] = 1.0 + 0.1 * torch.randn((dim,), device=DEV, generator=gen)
        span = max(4096, t)
        freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"])
        angle = torch.arange(span, device=DEV, dtype=torch.float64)[:, None] * freq
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        start = torch.randint(0, span - t + 1, (1,), device=DEV, generator=gen)
        s["positions"] = (torch.arange(t, device=DEV) + start).to(torch.int32)
        s["interleaved"], s["eps"] = case["interleaved"], 1e-6
    elif op == "append":
        t, h, dim, page = case["tokens"], case["kv_heads"], case["dim"], case["page"]
        kind = getattr(torch, case["kind"])
        s.update(page=page, dim=dim, kv_heads=h, kind=kind)
        pages = -(-t // page) + 7
        s["pool"] = torch.zeros((pages, h, page * (dim + 8)), device=DEV, dtype=torch.uint8)
        s["K"], s["V"] = _rows(gen, (t, h, dim), kind), _rows(gen, (t, h, dim), kind)
        order = torch.randperm(pages, device=DEV, generator=gen)
        at = torch.arange(t, device=DEV) + int(torch.randint(0, page, (1,), device=DEV, generator=gen))
        s["slots"] = order[at // page] * page + at % page
    else:
        h, hq, dim, page, new = case["kv_heads"], case["heads"], case["dim"], case["page"], case["new"]
        kind = getattr(torch, case["kind"])
        lens = _lengths(case)
        wide = -(-max(lens) // page)
        pages = sum(-(-n // page) for n in lens) + 3
        parts = [_quantize(_rows(gen, (pages, page, h, dim), torch.bfloat16).transpose(1, 2)) for _ in range(2)]
        numbers = torch.stack([x for p in parts for x in p[1:]], dim=-1)          # (pages, h, page, 4) float16
        s["pool"] = torch.cat([_pack(p[0]).reshape(pages, h, -1) for p in parts]
                              + [numbers.view(torch.uint8).reshape(pages, h, -1)], dim=-1)
        s.update(page=page, dim=dim, kv_heads=h, new=new, window=case["window"], longest=max(lens))
        order = torch.randperm(pages, device=DEV, generator=gen).to(torch.int32)
        table = torch.zeros((len(lens), wide), device=DEV, dtype=torch.int32)
        at = 0
        for b, n in enumerate(lens):
            k = -(-n // page)
            table[b, :k] = order[at:at + k]
            at += k
        s["table"] = table
        s["lens"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
        s["cu_q"] = torch.arange(0, (len(lens) + 1) * new, new, device=DEV, dtype=torch.int32)
        s["Q"] = (1.5 * torch.randn((len(lens) * new, hq, dim), device=DEV, generator=gen)).to(kind)
    return s


# ---------------------------------------------------------------------------- plain forms
def _codes(qweight, bits, d):
    """Codes (m, d) of a little-endian bitstream of int32 words."""
    w = qweight.to(torch.int64) & 0xFFFFFFFF
    w = torch.cat([w, torch.zeros_like(w[:, :1])], dim=1)
    at = torch.arange(d, device=qweight.device) * bits
    lo, off = at // 32, at % 32
    return ((w[:, lo] | (w[:, lo + 1] << 32)) >> off) & (2 ** bits - 1)


def _plain_adapter(s):
    m, d = s["m"], s["d"]
    groups = d // s["group"]
    codes = _codes(s["qweight"], s["bits"], d).float().view(m, groups, s["group"])
    W = ((codes - s["zeros"][..., None]) * s["scales"][..., None]).view(m, d)
    X, A, B, ids = s["X"].float(), s["A"], s["B"], s["ids"].long()
    n, r, _ = A.shape
    t = X.shape[0]
    has, at = ids >= 0, ids.clamp(min=0)
    weight = torch.where(has, s["alpha"][at], torch.zeros_like(s["alpha"][at]))
    Y = X @ W.T
    if t <= n:                                  # the adapters that the tokens use
        U = (X[:, None, :] * A[at].float()).sum(-1) * weight[:, None]
        Y = Y + (B[at].float() * U[:, None, :]).sum(-1)
    else:                                       # all adapters, each token keeps its own
        U = (X @ A.float().reshape(n * r, d).T).view(t, n, r)
        U = U * ((torch.arange(n, device=DEV) == at[:, None]) * weight[:, None])[..., None]
        Y = Y + U.view(t, n * r) @ B.float().transpose(0, 1).reshape(m, n * r).T
    return Y.to(s["out"])


def _plain_norm_rope(s):
    def one(x, w):
        kind, x = x.dtype, x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w
        cos, sin = s["cos"][s["positions"].long()][:, None, :], s["sin"][s["positions"].long()][:, None, :]
        half = cos.shape[-1]
        if s["interleaved"]:
            a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:2 * half]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        return torch.cat([turned, x[..., 2 * half:]], dim=-1).to(kind)

    return one(s["Q"], s["wq"]), one(s["K"], s["wk"])


def _split(blocks, page, dim):
    """Codes of K and V (..., page, dim) in fp32 and the four numbers (..., page, 4) of cache blocks."""
    half = page * dim // 2
    lead = blocks.shape[:-1]

    def codes(x):
        x = x.reshape(*lead, page, dim // 2)
        return torch.stack([x & 15, x >> 4], dim=-1).flatten(-2).float()

    numbers = blocks[..., 2 * half:].contiguous().view(torch.float16).view(*lead, page, 4).float()
    return codes(blocks[..., :half]), codes(blocks[..., half:2 * half]), numbers


def _plain_append(s):
    page, dim, pool = s["page"], s["dim"], s["pool"]
    pages, h = pool.shape[:2]
    half = page * dim // 2
    at, off = s["slots"] // page, s["slots"] % page
    codes, scale, low = _quantize(torch.stack([s["K"], s["V"]], dim=2))                # (tokens, h, 2, ...)
    pool[..., :2 * half].view(pages, h, 2, page, dim // 2)[at, :, :, off] = _pack(codes)
    numbers = pool[..., 2 * half:].view(torch.float16).view(pages, h, page, 2, 2)
    numbers[at, :, off] = torch.stack([scale, low], dim=-1)
    values = (codes * scale.float()[..., None] + low.float()[..., None]).to(s["kind"])
    return values[:, :, 0], values[:, :, 1]


def _plain_attention(s):
    page, dim, h, new, table = s["page"], s["dim"], s["kv_heads"], s["new"], s["table"]
    batch, wide = table.shape
    kc, vc, numbers = _split(s["pool"][table.long()], page, dim)          # (batch, wide, h, page, ...)

    def values(c, k):
        x = c * numbers[..., 2 * k, None] + numbers[..., 2 * k + 1, None]
        return x.transpose(1, 2).reshape(batch, h, wide * page, dim)

    q = s["Q"].float().view(batch, new, h, -1, dim).permute(0, 2, 3, 1, 4).reshape(batch, h, -1, dim)
    scores = (q @ values(kc, 0).transpose(-1, -2)).view(batch, h, -1, new, wide * page) * dim ** -0.5
    key = torch.arange(wide * page, device=DEV)
    last = s["lens"][:, None].long() - new + torch.arange(new, device=DEV)     # position of each new token
    seen = key <= last[..., None]
    if s["window"]:
        seen = seen & (key > last[..., None] - s["window"])
    scores = scores.masked_fill_(~seen[:, None, None], -math.inf)
    scores = scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    total = scores.sum(-1, keepdim=True)
    o = (scores.view(batch, h, -1, wide * page) @ values(vc, 1)).view(batch, h, -1, new, dim) / total
    return o.permute(0, 3, 1, 2, 4).reshape(batch * new, -1, dim).to(s["Q"].dtype)


# ---------------------------------------------------------------------------- one pass
def run(s):
    op = s["op"]
    if not own:
        return {"adapter": _plain_adapter, "norm_rope": _plain_norm_rope, "append": _plain_append,
                "attention": _plain_attention}[op](s)
    from post_weight_quantization_gb300 import gptq as g
    if op == "adapter":
        layer = g.QuantizedLayer(s["qweight"], s["scales"], s["zeros"], None, s["bits"], s["group"], s["d"])
        return g.gptq_adapter_linear(layer, s["X"], s["m"], s["A"], s["B"], s["ids"], alpha=s["alpha"],
                                     out_bf16=s["out"] == torch.bfloat16)
    if op == "norm_rope":
        return g.gptq_qk_norm_rope(s["Q"], s["K"], s["positions"], s["cos"], s["sin"], wq=s["wq"], wk=s["wk"],
                                   eps=s["eps"], interleaved=s["interleaved"])
    cache = g.KVCache(s["pool"], s["page"], s["kv_heads"], s["dim"])
    if op == "append":
        g.gptq_kv_append(cache, s["K"], s["V"], s["slots"])
        return g.gptq_kv_read(cache, s["slots"], dtype=s["kind"])
    return g.gptq_kv_attention(cache, s["Q"], s["cu_q"], s["lens"], s["table"], s["new"], window=s["window"])


# ---------------------------------------------------------------------------- in 64 bits
def _exact_adapter(s):
    m, d, bits, group = s["m"], s["d"], s["bits"], s["group"]
    bit = torch.arange(32, device=DEV, dtype=torch.int32)
    W = torch.empty((m, d), device=DEV, dtype=torch.float64)
    for r in range(0, m, 1024):
        stream = ((s["qweight"][r:r + 1024, :, None] >> bit) & 1).flatten(1).view(-1, d, bits).double()
        codes = stream @ (2.0 ** torch.arange(bits, device=DEV, dtype=torch.float64))
        z = s["zeros"][r:r + 1024].double().repeat_interleave(group, dim=1)
        W[r:r + 1024] = (codes - z) * s["scales"][r:r + 1024].double().repeat_interleave(group, dim=1)
    X = s["X"].double()
    Y = X @ W.T
    for a in torch.unique(s["ids"]).tolist():
        if a >= 0:
            rows = (s["ids"] == a).nonzero()[:, 0]
            Y[rows] += float(s["alpha"][a].double()) * ((X[rows] @ s["A"][a].double().T) @ s["B"][a].double().T)
    return Y


def _exact_norm_rope(s):
    got = []
    for x, w in ((s["Q"], s["wq"]), (s["K"], s["wk"])):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * w.double()
        turn = torch.complex(s["cos"].double(), s["sin"].double())[s["positions"].long()][:, None]
        n = turn.shape[-1]
        head = x[..., :2 * n]
        pairs = head.unflatten(-1, (n, 2)) if s["interleaved"] else head.unflatten(-1, (2, n)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.flatten(-2) if s["interleaved"] else z.transpose(-1, -2).flatten(-2)
        got.append(torch.cat([z, x[..., 2 * n:]], dim=-1))
    return tuple(got)


def _exact_append(s):
    got = []
    for x in (s["K"], s["V"]):
        x = x.double().clamp(-65504, 65504)
        low = x.min(-1, keepdim=True).values
        scale = ((x.max(-1, keepdim=True).values - low) / 15).half().double()
        low = low.half().double()
        codes = torch.where(scale > 0, (x - low) / scale.clamp(min=1e-30), torch.zeros_like(x)).round().clamp(0, 15)
        got.append(codes * scale + low)
    return tuple(got)


def _exact_attention(s):
    page, dim, h, new = s["page"], s["dim"], s["kv_heads"], s["new"]
    lens, out = s["lens"].tolist(), []
    for b, n in enumerate(lens):
        blocks = s["pool"][s["table"][b, :-(-n // page)].long()].transpose(0, 1)        # (h, pages, bytes)
        q = s["Q"][b * new:(b + 1) * new].double().unflatten(1, (h, -1))                # (new, h, g, dim)
        heads = []
        for j in range(h):
            raw = blocks[j]
            numbers = raw[:, page * dim:].contiguous().view(torch.float16).view(-1, 4).double()[:n]
            byte = raw[:, :page * dim].reshape(-1, 2, page, dim // 2).transpose(0, 1).reshape(2, -1, dim // 2)[:, :n]
            c = torch.empty((2, n, dim), device=DEV, dtype=torch.float64)
            c[..., 0::2], c[..., 1::2] = (byte % 16).double(), (byte // 16).double()
            k = c[0] * numbers[:, 0:1] + numbers[:, 1:2]
            v = c[1] * numbers[:, 2:3] + numbers[:, 3:4]
            z = torch.einsum("igd,kd->igk", q[:, j], k) / math.sqrt(dim)
            at = torch.arange(n, device=DEV)
            pos = torch.arange(n - new, n, device=DEV)[:, None]
            hide = at > pos
            if s["window"]:
                hide = hide | (at <= pos - s["window"])
            z = z.masked_fill(hide[:, None], -math.inf)
            heads.append(torch.einsum("igk,kd->igd", torch.softmax(z, dim=-1), v))
        out.append(torch.stack(heads, dim=1).flatten(1, 2))
    return torch.cat(out)


def exact(case, seed):
    s = prepare(case, seed)
    return {"adapter": _exact_adapter, "norm_rope": _exact_norm_rope, "append": _exact_append,
            "attention": _exact_attention}[s["op"]](s)
