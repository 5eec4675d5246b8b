"""Cases of the feed-forward sublayer and the head in 8 bits: RMSNorm with the residual's addition and an 8-bit output, the product of
8-bit rows with 8-bit weights, the gated product (gate and up projections, activation, product), and log probabilities of given tokens
with the entropy and the most likely alternatives; in a plain form and through the library's entry points."""

import torch

own = False

DEV = "cuda"
BLOCK = 128  # values that share a scale: 128 along a row; 128 x 128 of a weight matrix


def listed():
    return [
        # one step of 64 tokens at width 5120: what the reading half hands to the feed-forward sublayer, in 8 bits: latency
        norm("norm step", 64, 5120, False, False),
        # a chunk of a prompt at an odd width, residual and gains
        norm("norm odd", 1027, 2000, True, True),
        # prefill batch of 4 x 4096 tokens
        norm("norm prefill", 16384, 5120, True, True),
        # one token through a square projection: latency, the weights' bytes
        mul("mul token", 1, 5120, 5120, "bf16"),
        # the decode batch of 256 sequences, back from the wide side of the feed-forward sublayer
        mul("mul decode", 256, 20480, 5120, "bf16"),
        # the vocabulary's logits of 33 sequences
        mul("mul head", 33, 5120, 100003, "f32"),
        # prefill batch of 4 x 4096 tokens, back from the wide side
        mul("mul prefill", 16384, 20480, 5120, "bf16"),
        # a few tokens of one sequence through a narrow block: latency
        gated("gated token", 3, 5120, 2048, "silu", "e4m3"),
        # the decode batch of 256 sequences
        gated("gated decode", 256, 5120, 20480, "silu", "e4m3"),
        # one prompt of 4099 tokens, bf16 handed on
        gated("gated prefill", 4099, 5120, 20480, "gelu", "bf16"),
        # what a decode step of 256 sequences answers with: the drawn token's log probability and 20 alternatives
        logprobs("logprobs decode", 256, 131072, 20, "bf16", 1.25, True),
        # every token of a prompt scored
        logprobs("logprobs prompt", 4097, 100003, 5, "f32", 1.0, False),
    ]


def norm(name, tokens, dim, residual, gains):
    c = dict(op="norm", tokens=tokens, dim=dim, residual=residual, gains=gains)
    return dict(c, name=name) if name else c


def mul(name, tokens, k, features, out):
    c = dict(op="mul", tokens=tokens, k=k, features=features, out=out)
    return dict(c, name=name) if name else c


def gated(name, tokens, k, features, act, out):
    c = dict(op="gated", tokens=tokens, k=k, features=features, act=act, out=out)
    return dict(c, name=name) if name else c


def logprobs(name, tokens, vocab, top, dtype, scale, banned):
    c = dict(op="logprobs", tokens=tokens, vocab=vocab, top=top, dtype=dtype, scale=scale, banned=banned)
    return dict(c, name=name) if name else c


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))

    op = rng.choice(("norm", "mul", "mul", "gated", "gated", "logprobs"))
    if op == "norm":
        kind = rng.choice(((False, False), (False, True), (True, True)))
        return norm(None, spread(1, 8000), 16 * spread(4, 512), *kind)
    if op == "mul":
        return mul(None, spread(1, 4000), 16 * spread(8, 1024), spread(48, 20000), rng.choice(("bf16", "f32")))
    if op == "gated":
        return gated(None, spread(1, 4000), 16 * spread(8, 512), 16 * spread(4, 1024), rng.choice(("silu", "gelu")), rng.choice(("e4m3", "bf16")))
    vocab = spread(500, 200000)
    return logprobs(None, spread(1, max(2, min(4000, 200000000 // vocab))), vocab, rng.choice((0, 1, 5, 8, 20, 32)), rng.choice(("bf16", "f32")),
                    rng.choice((0.7, 1.0, 1.0, 1.5)), rng.random() < 0.5)


# ---- what the cases are made of ---------------------------------------------------------------------


def blocks(n):
    return -(-n // BLOCK)


def in_blocks(x):
    """[..., n] as [..., blocks, 128], zeros behind the last value."""
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % BLOCK)).unflatten(-1, (-1, BLOCK))


def quantise(x):
    """8-bit codes and fp32 scales of 128 values along the last dimension: scale = largest magnitude / 448, code = x * (448 / largest magnitude), rounded to even."""
    b = in_blocks(x)
    top = b.abs().amax(-1).clamp(min=2.0 ** -64)
    codes = (b * (448.0 / top)[..., None]).flatten(-2)[..., :x.shape[-1]]
    return codes.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), top / 448.0


def weights(g, rows, cols):
    """A weight matrix in 8 bits with a scale for each 128 x 128 block; the blocks' sizes differ as they do in trained matrices."""
    size = 0.02 * torch.exp(0.3 * torch.randn((blocks(rows), blocks(cols)), generator=g, device=DEV))
    codes = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty((blocks(rows), blocks(cols)), device=DEV)
    for i in range(0, rows, 8192):
        n = min(8192, rows - i)
        part = slice(i // BLOCK, i // BLOCK + blocks(n))
        x = torch.randn((n, cols), generator=g, device=DEV)
        top = torch.nn.functional.pad(x.abs(), (0, -cols % BLOCK, 0, -n % BLOCK)).unflatten(1, (-1, BLOCK)).unflatten(0, (-1, BLOCK)).amax((1, 3))
        codes[i:i + n] = (x * spread_out(448.0 / top, n, cols)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        scales[part] = top / 448.0 * size[part]
    return codes, scales


def spread_out(scales, rows, cols):
    """A block's scale at each of its 128 x 128 places."""
    return scales.repeat_interleave(BLOCK, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]


def activations(g, *shape):
    """Rows as they leave a norm or an activation: a few strong columns, tokens of several sizes."""
    x = torch.randn(shape, generator=g, device=DEV)
    x *= torch.where(torch.rand(shape[-1], generator=g, device=DEV) < 0.02, 8.0, 1.0)
    return x * torch.exp(0.5 * torch.randn((shape[0], 1), generator=g, device=DEV))


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 1000003 + 29)
    st = dict(case)
    n = case["tokens"]
    if case["op"] == "norm":
        st["x"] = activations(g, n, case["dim"]).to(torch.bfloat16)
        st["res"] = (3 * activations(g, n, case["dim"])).to(torch.bfloat16) if case["residual"] else None
        st["w"] = 1 + 0.1 * torch.randn(case["dim"], generator=g, device=DEV) if case["gains"] else None
    elif case["op"] == "logprobs":
        pitch = -(-case["vocab"] // 8) * 8  # rows of a wider buffer
        logits = 3 * torch.randn((n, pitch), generator=g, device=DEV)
        likely = torch.randint(0, case["vocab"], (n, 8), generator=g, device=DEV)
        logits.scatter_add_(1, likely, 4 + 6 * torch.rand((n, 8), generator=g, device=DEV))
        if case["banned"]:  # what a grammar rules out
            logits.masked_fill_(torch.rand(pitch, generator=g, device=DEV) < 0.1, float("-inf"))
        st["logits"] = logits.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)[:, :case["vocab"]]
        any_token = torch.randint(0, case["vocab"], (n,), generator=g, device=DEV)
        st["tokens_given"] = torch.where(torch.rand(n, generator=g, device=DEV) < 0.7, likely[:, 0], any_token)
    else:
        st["x"], st["x_scales"] = quantise(activations(g, n, case["k"]))
        st["w"], st["w_scales"] = weights(g, case["features"], case["k"])
        if case["op"] == "gated":
            st["up"], st["up_scales"] = weights(g, case["features"], case["k"])
    return st


# ---- one pass -------------------------------------------------------------------------------------


def run(st):
    if own:
        return {"norm": own_norm, "mul": own_mul, "gated": own_gated, "logprobs": own_logprobs}[st["op"]](st)
    return {"norm": plain_norm, "mul": plain_mul, "gated": plain_gated, "logprobs": plain_logprobs}[st["op"]](st)


def own_norm(st):
    import hyper_connection_residual_hc_gb300 as hc
    x, res = st["x"], st["res"]
    n, d = x.shape
    codes = torch.empty((n, d), dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty((n, blocks(d)), dtype=torch.float32, device=DEV)
    out = None if res is None else torch.empty_like(x)
    hc.hc_norm_quant8(x, d, res, d, st["w"], hc.quant8(n, d, norm=st["gains"], norm_eps=1e-6), out, d, codes, d, scales)
    return (codes, scales) if out is None else (codes, scales, out)


def own_mul(st):
    import hyper_connection_residual_hc_gb300 as hc
    n, k, features, wide = st["tokens"], st["k"], st["features"], st["out"] == "f32"
    pitch = (features + 7) // 8 * 8
    out = torch.empty((n, pitch), dtype=torch.float32 if wide else torch.bfloat16, device=DEV)
    hc.hc_mul8(st["x"], k, st["x_scales"], st["w"], k, st["w_scales"], n, hc.mul8(features, k, hc.HC_F32 if wide else hc.HC_BF16), out, pitch)
    return out[:, :features]


def own_gated(st):
    import hyper_connection_residual_hc_gb300 as hc
    n, k, features, short = st["tokens"], st["k"], st["features"], st["out"] == "e4m3"
    out = torch.empty((n, features), dtype=torch.float8_e4m3fn if short else torch.bfloat16, device=DEV)
    scales = torch.empty((n, blocks(features)), dtype=torch.float32, device=DEV) if short else None
    s = hc.gated8(features, k, hc.HC_ACT_SILU if st["act"] == "silu" else hc.HC_ACT_GELU, hc.HC_E4M3 if short else hc.HC_BF16)
    hc.hc_gated_mul8(st["x"], k, st["x_scales"], st["w"], st["w_scales"], st["up"], st["up_scales"], k, n, s, out, features, scales)
    return (out, scales) if short else out


def own_logprobs(st):
    import hyper_connection_residual_hc_gb300 as hc
    z, top = st["logits"], st["top"]
    n, vocab = z.shape
    given = torch.empty(n, dtype=torch.float32, device=DEV)
    entropy = torch.empty(n, dtype=torch.float32, device=DEV)
    best = torch.empty((n, top), dtype=torch.float32, device=DEV) if top else None
    which = torch.empty((n, top), dtype=torch.int32, device=DEV) if top else None
    s = hc.logprobs(n, vocab, top, st["scale"], hc.HC_BF16 if st["dtype"] == "bf16" else hc.HC_F32)
    hc.hc_token_logprobs(z, z.stride(0), st["tokens_given"], s, given, entropy, best, which)
    return (given, entropy, best, which) if top else (given, entropy)


def plain_norm(st):
    y = st["x"].float()
    total = None
    if st["residual"]:
        total = (y + st["res"].float()).to(torch.bfloat16)
        y = total.float()
    if st["gains"]:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * st["w"]
    codes, scales = quantise(y)
    return (codes, scales) if total is None else (codes, scales, total)


def values(codes, scales):
    """The values of 8-bit rows, in fp32."""
    return codes.float() * scales.repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def plain_product(st, w, scales):
    w = w.float() * spread_out(scales, *w.shape)
    return values(st["x"], st["x_scales"]) @ w.T


def plain_mul(st):
    y = plain_product(st, st["w"], st["w_scales"])
    return y if st["out"] == "f32" else y.to(torch.bfloat16)


def plain_gated(st):
    a = plain_product(st, st["w"], st["w_scales"])
    if st["act"] == "silu":
        a = a / (1 + torch.exp(-a))
    else:
        a = 0.5 * a * (1 + torch.tanh(0.7978845608028654 * (a + 0.044715 * a * a * a)))
    h = a * plain_product(st, st["up"], st["up_scales"])
    return quantise(h) if st["out"] == "e4m3" else h.to(torch.bfloat16)


def plain_logprobs(st):
    x, top = st["logits"].float(), st["top"]
    t = (x - x.amax(-1, keepdim=True)) * st["scale"]
    e = torch.exp(t)
    total = e.sum(-1, keepdim=True)
    log_total = total.log()
    entropy = log_total - torch.where(e > 0, e * t, e).sum(-1, keepdim=True) / total
    given = t.gather(1, st["tokens_given"][:, None]) - log_total
    out = (given.squeeze(1), entropy.squeeze(1))
    if not top:
        return out
    # whole numbers that rise with the logits, of two equal ones the lower index first
    bits = (x + 0.0).contiguous().view(torch.int32)
    key = ((bits ^ (bits >> 31 & 0x7FFFFFFF)).long() << 32) - torch.arange(x.shape[1], device=DEV)
    key = key.topk(top, -1).values
    which = -key & 0xFFFFFFFF
    return out + (t.gather(1, which) - log_total, which.int())


# ---- what a pass cannot do without ------------------------------------------------------------------


def work(case):
    n = case["tokens"]
    if case["op"] == "norm":
        d = case["dim"]
        each = (7 if case["residual"] else 3) * d + 4 * blocks(d)
        return {"bytes": n * each + 4 * d * case["gains"], "flops": (8 if case["gains"] else 3) * n * d}
    if case["op"] == "logprobs":
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * (case["vocab"] * size + 16 + 8 * case["top"]), "flops": 6 * n * case["vocab"]}
    k, f = case["k"], case["features"]
    size = {"f32": 4, "bf16": 2, "e4m3": 1}[case["out"]]
    both = 2 if case["op"] == "gated" else 1
    more = 4 * n * blocks(f) if case["out"] == "e4m3" else 0
    return {"bytes": n * (k + 4 * blocks(k)) + both * (f * k + 4 * blocks(f) * blocks(k)) + size * n * f + more, "flops": 2 * both * n * k * f}


# ---- the definitions in 64 bits -----------------------------------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": exact_norm, "mul": exact_mul, "gated": exact_gated, "logprobs": exact_logprobs}[case["op"]](st)


def exact_codes(y):
    """What the codes and scales of rows in 64 bits round."""
    scales = torch.stack([part.abs().amax(-1) for part in y.split(BLOCK, -1)], -1).clamp(min=2.0 ** -64) / 448
    return torch.cat([part / scales[:, i:i + 1] for i, part in enumerate(y.split(BLOCK, -1))], -1), scales


def exact_norm(st):
    y = st["x"].double()
    total = None
    if st["residual"]:
        total = y + st["res"].double()
        y = total.to(torch.bfloat16).double()
    if st["gains"]:
        y = y / ((y * y).sum(-1, keepdim=True) / y.shape[-1] + 1e-6).sqrt() * st["w"].double()
    codes, scales = exact_codes(y)
    return (codes, scales) if total is None else (codes, scales, total)


def exact_product(st, w, scales):
    """The sum over the blocks of 128 of the products of codes, each block's times both scales."""
    out = torch.zeros((st["tokens"], w.shape[0]), dtype=torch.float64, device=DEV)
    each = scales.double().repeat_interleave(BLOCK, 0)[:w.shape[0]]
    step = 16 * BLOCK
    for i in range(0, w.shape[1], step):
        b = slice(i // BLOCK, (i + step) // BLOCK)
        xs = st["x"][:, i:i + step].double() * st["x_scales"][:, b].double().repeat_interleave(BLOCK, 1)[:, :w.shape[1] - i]
        out += xs @ (w[:, i:i + step].double() * each[:, b].repeat_interleave(BLOCK, 1)[:, :w.shape[1] - i]).T
    return out


def exact_mul(st):
    return exact_product(st, st["w"], st["w_scales"])


def exact_gated(st):
    a = exact_product(st, st["w"], st["w_scales"])
    if st["act"] == "silu":
        a = a * torch.sigmoid(a)
    else:
        a = a * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (a + 0.044715 * a ** 3))  # (1 + tanh x) / 2 = sigmoid(2 x)
    h = a * exact_product(st, st["up"], st["up_scales"])
    return exact_codes(h) if st["out"] == "e4m3" else h


def exact_logprobs(st):
    rows, top = [], st["top"]
    for x, token in zip(st["logits"].split(512), st["tokens_given"].split(512)):
        x = x.double()
        lp = torch.log_softmax(x * st["scale"], -1)
        entropy = -(lp.exp() * lp.masked_fill(lp == float("-inf"), 0.0)).sum(-1)
        row = [lp[torch.arange(len(x), device=DEV), token], entropy]
        if top:
            which = x.sort(dim=-1, descending=True, stable=True).indices[:, :top]
            row += [lp.gather(1, which), which.int()]
        rows.append(row)
    return tuple(torch.cat(part) for part in zip(*rows))
