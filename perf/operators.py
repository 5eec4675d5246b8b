"""Cases of the attention-sublayer operators: per-head norms with the position rotation, the 4-bit key/value cache
(write and read back) and the attention over it, in a plain form and through the library's entry points."""

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # the magnitudes of codes 0..7; bit 3 is the sign


def listed():
    return [
        # one step of 64 tokens at width 5120 (40 heads of 128): latency
        rope("rope step", 64, 40, 8, 128, 128, 0, "half", 1, 65536),
        # decode batch deep in a long context, the last half of each head rotated, adjacent pairs
        rope("rope decode far", 257, 32, 4, 128, 64, 64, "pairs", 1, 1 << 20),
        # image and video patches: time, height and width positions, odd head width, as many key heads as query heads
        rope("rope images", 4097, 16, 16, 80, 80, 0, "half", 3, 4096),
        # prefill batch of 4 x 4096 tokens
        rope("rope prefill", 16384, 40, 8, 128, 128, 0, "half", 1, 16384),
        # one new token for each of 256 sequences
        cache("cache decode", 256, 1, 0, 8, 128, 64),
        # a prefill of 4 prompts of up to 4096 tokens, written and handed on in bf16
        cache("cache prefill", 4, 4096, 0, 8, 128, 64),
        # a few new tokens behind a cached prefix, the whole prefix read back; small pages, odd lengths
        cache("cache prefix", 9, 33, 5003, 4, 64, 16),
        # a small decode batch in short contexts: latency
        attn("attend short", 8, 1, 509, 40, 8, 128, 64, 0),
        # the decode batch of 256 sequences, contexts of up to 4096
        attn("attend decode", 256, 1, 4096, 40, 8, 128, 64, 0),
        # a few sequences with long contexts: the keys of one sequence spread over the whole GPU
        attn("attend long", 3, 1, 131072, 40, 8, 128, 128, 0),
        # five drafted tokens checked at once for 64 sequences, sliding window
        attn("attend drafts", 64, 5, 4001, 32, 8, 128, 32, 1024),
        # a chunk of two long prompts behind what was prefilled before
        attn("attend prefill", 2, 2048, 8192, 40, 8, 128, 64, 0),
    ]


def rope(name, tokens, q_heads, k_heads, dim, rot, start, style, axes, furthest):
    c = dict(op="rope", tokens=tokens, q_heads=q_heads, k_heads=k_heads, dim=dim, rot=rot, start=start, style=style, axes=axes, furthest=furthest)
    return dict(c, name=name) if name else c


def cache(name, seqs, new, context, heads, dim, page_size):
    c = dict(op="cache", seqs=seqs, new=new, context=context, heads=heads, dim=dim, page_size=page_size)
    return dict(c, name=name) if name else c


def attn(name, seqs, q_len, kv_len, q_heads, kv_heads, dim, page_size, window):
    c = dict(op="attention", seqs=seqs, q_len=q_len, kv_len=kv_len, q_heads=q_heads, kv_heads=kv_heads, dim=dim, page_size=page_size, window=window)
    return dict(c, name=name) if name else c


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))

    op = rng.choice(("rope", "cache", "attention", "attention"))
    dim = rng.choice((64, 128, 128, 256))
    if op == "rope":
        dim = rng.choice((64, 80, 96, 128, 128, 192, 256))
        rot = rng.choice([r for r in (32, 64, 80, 96, 128, 192, 256) if r <= dim])
        k_heads = rng.choice((1, 2, 4, 8))
        return rope(None, spread(1, 8000), k_heads * rng.choice((1, 3, 5, 8)), k_heads, dim, rot, rng.choice((0, dim - rot)), rng.choice(("half", "pairs")),
                    rng.choice((1, 1, 3)), spread(64, 1 << 20))
    if op == "cache":
        seqs = spread(1, 256)
        return cache(None, seqs, spread(1, max(1, 8000 // seqs)), spread(1, max(1, 20000 // seqs)) - 1, rng.choice((1, 3, 4, 8)), dim, rng.choice((16, 32, 64, 128)))
    kv_heads = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 4, 5, 7, 8, 16))
    if rng.random() < 0.3:  # a prefill chunk
        seqs, q_len = rng.randint(1, 3), spread(17, 1000)
        return attn(None, seqs, q_len, q_len + spread(1, 5000) - 1, kv_heads * min(group, 5), kv_heads, dim, rng.choice((16, 32, 64, 128)), rng.choice((0, 0, spread(100, 2000))))
    seqs = spread(1, 256)
    q_len = rng.choice((1, 1, 2, 4, 7))
    return attn(None, seqs, q_len, q_len + spread(1, 500000 // seqs) - 1, kv_heads * group, kv_heads, dim, rng.choice((16, 32, 64, 128)), rng.choice((0, 0, 0, spread(64, 4000))))


# ---- what the cases are made of ---------------------------------------------------------------------


def lengths(case):
    """[(keys, queries)] of each sequence of a case: ragged down to about half the longest, the same for every seed."""
    if case["op"] == "cache":
        most, least, q = case["context"] + case["new"], case["new"], case["new"]
    else:
        most, least, q = case["kv_len"], case["q_len"], case["q_len"]
    return [(max(least, most - (i * 37 % case["seqs"]) * most // (2 * case["seqs"])), q) for i in range(case["seqs"])]


def block_bytes(dim):
    """Bytes of 16 tokens of one head: key codes, key scales, value codes, value scales."""
    return 18 * dim


def e4m3(x):
    """The nearest 8-bit float (4 exponent, 3 mantissa bits), as its bits; at most 448."""
    return x.clamp(max=448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def quantise(x):
    """4-bit codes and the 8-bit scales of 16 values along the last dimension: scale = amax / 6 rounded, code = x / scale rounded, ties to the even code."""
    b = x.float().unflatten(-1, (-1, 16))
    bits = e4m3(b.abs().amax(-1) / 6.0)
    s = bits.view(torch.float8_e4m3fn).float()
    a = torch.where(s[..., None] > 0, b.abs() / s[..., None], torch.zeros_like(b))
    code = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    return (code + 8 * torch.signbit(b)).to(torch.uint8).flatten(-2), bits


def pack(k, v):
    """Keys and values [blocks, heads, 16, dim] as the cache holds them: [blocks, heads, 18 * dim] bytes."""
    n, h, _, dim = k.shape
    kc, ks = quantise(k)
    vc, vs = quantise(v)
    # keys: token = 8 hw + r, column = c (dim / 4) + 16 quad + 4 s + 2 e + nibble; byte [quad][r][c][s][hw][e]
    kc = kc.view(n, h, 2, 8, 4, dim // 64, 4, 2, 2)
    kc = (kc[..., 0] + 16 * kc[..., 1]).permute(0, 1, 5, 3, 4, 6, 2, 7).reshape(n, h, -1)
    ks = ks.view(n, h, 2, 8, 4, dim // 64).permute(0, 1, 3, 4, 2, 5).reshape(n, h, -1)
    # values: token = 8 hi + 2 c + odd, column = r (dim / 8) + 8 quad + 2 m + nibble; byte [quad][r][c][m][hi][odd]
    vc = vc.view(n, h, 2, 4, 2, 8, dim // 64, 4, 2)
    vc = (vc[..., 0] + 16 * vc[..., 1]).permute(0, 1, 6, 5, 3, 7, 2, 4).reshape(n, h, -1)
    vs = vs.view(n, h, 2, 4, 2, dim // 16).permute(0, 1, 5, 3, 2, 4).reshape(n, h, -1)
    return torch.cat((kc, ks, vc, vs), -1)


def unpack(raw, dim):
    """Keys and values [..., 16, dim] in fp32 of cache blocks [..., 18 * dim]."""
    lead, n = raw.shape[:-1], raw[..., 0].numel()
    level = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=raw.device)
    kc, ks, vc, vs = raw.reshape(n, -1).split((8 * dim, dim, 8 * dim, dim), -1)
    kc = torch.stack((kc & 15, kc >> 4), -1).view(n, dim // 64, 8, 4, 4, 2, 2, 2).permute(0, 5, 2, 3, 1, 4, 6, 7).reshape(n, 16, dim // 16, 16)
    ks = ks.reshape(n, 8, 4, 2, dim // 64).permute(0, 3, 1, 2, 4).reshape(n, 16, dim // 16)
    vc = torch.stack((vc & 15, vc >> 4), -1).view(n, dim // 64, 8, 4, 4, 2, 2, 2).permute(0, 5, 3, 6, 2, 1, 4, 7).reshape(n, 16, dim // 16, 16)
    vs = vs.reshape(n, dim // 16, 4, 2, 2).permute(0, 3, 2, 4, 1).reshape(n, 16, dim // 16)
    k = level[kc.int()] * ks.contiguous().view(torch.float8_e4m3fn).float()[..., None]
    v = level[vc.int()] * vs.contiguous().view(torch.float8_e4m3fn).float()[..., None]
    return k.view(*lead, 16, dim), v.view(*lead, 16, dim)


def byte_places(dim):
    """[16, 18 dim / 16]: where the bytes of each of a block's 16 tokens lie in it: key codes, key scales, value codes, value scales, by column."""
    t = torch.arange(16, device=DEV)[:, None]
    c2, c16 = torch.arange(0, dim, 2, device=DEV)[None], torch.arange(0, dim, 16, device=DEV)[None]
    col, row = c2 % (dim // 4), c2 % (dim // 8)
    kc = col // 16 * 512 + (t % 8) * 64 + c2 // (dim // 4) * 16 + col // 4 % 4 * 4 + t // 8 * 2 + col // 2 % 2
    ks = (t % 8) * (dim // 8) + c16 // (dim // 4) * (dim // 32) + t // 8 * (dim // 64) + c16 % (dim // 4) // 16
    vc = row // 8 * 512 + c2 // (dim // 8) * 64 + t % 8 // 2 * 16 + row // 2 % 4 * 4 + t // 8 * 2 + t % 2
    vs = c16 // 16 * 16 + t % 8 // 2 * 4 + t // 8 * 2 + t % 2
    return torch.cat((kc, 8 * dim + ks, 9 * dim + vc, 17 * dim + vs), 1)


def keys_and_values(g, *shape):
    """Keys as they come from a norm and a rotation, with a few strong columns; values a little smaller."""
    k = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    k *= torch.where(torch.rand(shape[-1], generator=g, device=DEV) < 0.05, 4.0, 1.0).to(torch.bfloat16)
    return k, torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16) * 0.5


def paged(case, g, heads):
    """A cache whose sequences lie on pages in no order: its bytes, the page table (-1 where a sequence has no page) and the keys of each sequence."""
    size, lens = case["page_size"], [kv for kv, _ in lengths(case)]
    pages = [-(-n // size) for n in lens]
    order = torch.randperm(sum(pages) + 3, generator=g, device=DEV).int()
    table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, p in enumerate(pages):
        table[i, :p] = order[at:at + p]
        at += p
    k, v = keys_and_values(g, (sum(pages) + 3) * size // 16, heads, 16, case["dim"])
    raw = torch.cat([pack(a, b) for a, b in zip(k.split(4096), v.split(4096))])
    raw = raw.view(sum(pages) + 3, size // 16, heads, -1).transpose(1, 2).contiguous()  # [pages, heads, blocks, bytes]
    return raw, table, torch.tensor(lens, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 1000003 + 17)
    st = dict(case)
    dim = case["dim"]
    if case["op"] == "rope":
        n, hq, hk, axes = case["tokens"], case["q_heads"], case["k_heads"], case["axes"]
        qkv = torch.randn((n, (hq + 2 * hk) * dim), generator=g, device=DEV, dtype=torch.bfloat16)  # the fused projection's output
        st["q"], st["k"] = qkv[:, :hq * dim], qkv[:, hq * dim:(hq + hk) * dim]
        st["q_w"] = 1 + 0.1 * torch.randn(dim, generator=g, device=DEV)
        st["k_w"] = 1 + 0.1 * torch.randn(dim, generator=g, device=DEV)
        st["positions"] = torch.randint(0, case["furthest"], (axes, n), generator=g, device=DEV)
        freq = [10000.0 ** (-2.0 * j / case["rot"]) for j in range(case["rot"] // 2)]
        axis = [j * axes // (case["rot"] // 2) for j in range(case["rot"] // 2)]
        st["freq"] = torch.tensor(freq, dtype=torch.float64, device=DEV)
        st["axis"] = torch.tensor(axis, device=DEV)
        if own:
            import hyper_connection_residual_hc_gb300 as hc
            st["table"] = torch.empty(hc.hc_rope_table_size(case["rot"]), dtype=torch.uint8, device=DEV)
            hc.hc_prepare_rope(freq, axis, case["rot"], axes, st["table"])
        return st
    heads = case["heads"] if case["op"] == "cache" else case["kv_heads"]
    st["cache"], st["table"], st["kv_len"] = paged(case, g, heads)
    lens = lengths(case)
    if case["op"] == "cache":
        n = sum(q for _, q in lens)
        k, v = keys_and_values(g, n, heads, dim)
        st["kv"] = torch.cat((k.flatten(1), v.flatten(1)), 1)  # one projection's output: a token's keys, then its values
        size, table = case["page_size"], st["table"].long()
        spots = [(i, torch.arange(kv, device=DEV)) for i, (kv, _) in enumerate(lens)]
        every = [table[i, p // size] * size + p % size for i, p in spots]
        st["slots"] = torch.cat([s[len(s) - case["new"]:] for s in every])
        st["read"] = torch.cat(every)
        st["places"] = byte_places(dim)
        return st
    n = sum(q for _, q in lens)
    st["q"] = torch.randn((n, case["q_heads"], dim), generator=g, device=DEV, dtype=torch.bfloat16)
    st["q_start"] = torch.arange(0, n + 1, case["q_len"], dtype=torch.int32, device=DEV)
    if own:
        import hyper_connection_residual_hc_gb300 as hc
        st["workspace"] = hc.new_kv_workspace()
    return st


# ---- one pass -------------------------------------------------------------------------------------


def run(st):
    if own:
        return {"rope": own_rope, "cache": own_cache, "attention": own_attention}[st["op"]](st)
    return {"rope": plain_rope, "cache": plain_cache, "attention": plain_attention}[st["op"]](st)


def own_rope(st):
    import hyper_connection_residual_hc_gb300 as hc
    n, hq, hk, dim = st["tokens"], st["q_heads"], st["k_heads"], st["dim"]
    q_out = torch.empty((n, hq, dim), dtype=torch.bfloat16, device=DEV)
    k_out = torch.empty((n, hk, dim), dtype=torch.bfloat16, device=DEV)
    r = hc.rope(st["table"], st["rot"], st["start"], st["axes"], hc.HC_ROPE_HALF if st["style"] == "half" else hc.HC_ROPE_PAIRS)
    hc.hc_qk_norm_rope(st["q"], st["q"].stride(0), st["k"], st["k"].stride(0), st["q_w"], st["k_w"], st["positions"], r, n, hc.heads(hq, hk, dim, 1e-6),
                       q_out, hq * dim, k_out, hk * dim)
    return q_out, k_out


def own_cache(st):
    import hyper_connection_residual_hc_gb300 as hc
    heads, dim, m = st["heads"], st["dim"], st["read"].numel()
    s = hc.kv_shape(st["cache"].shape[0], st["page_size"], heads, dim)
    k, v, stride = st["kv"][:, :heads * dim], st["kv"][:, heads * dim:], st["kv"].stride(0)
    hc.hc_kv_write(k, stride, v, stride, st["slots"], st["slots"].numel(), s, st["cache"])
    k_out = torch.empty((m, heads, dim), dtype=torch.bfloat16, device=DEV)
    v_out = torch.empty((m, heads, dim), dtype=torch.bfloat16, device=DEV)
    hc.hc_kv_read(st["cache"], st["read"], m, s, k_out, heads * dim, v_out, heads * dim)
    return k_out, v_out


def own_attention(st):
    import hyper_connection_residual_hc_gb300 as hc
    n, hq, dim = st["q"].shape
    s = hc.kv_shape(st["cache"].shape[0], st["page_size"], st["kv_heads"], dim)
    a = hc.attention(n, st["seqs"], st["q_len"], st["table"].shape[1], hq, dim ** -0.5, causal=True, window=st["window"])
    out = torch.empty((n, hq, dim), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((n, hq), dtype=torch.float32, device=DEV)
    hc.hc_kv_attention(st["q"], hq * dim, st["q_start"], st["kv_len"], st["table"], st["cache"], a, s, out, hq * dim, lse, st["workspace"])
    return out, lse


def plain_rope(st):
    phi = st["positions"][st["axis"]].double() * st["freq"][:, None]  # [rot / 2, tokens]: far positions need 64 bits
    cos, sin = phi.cos().float().T[:, None], phi.sin().float().T[:, None]
    return (plain_rope_one(st, st["q"], st["q_w"], st["q_heads"], cos, sin), plain_rope_one(st, st["k"], st["k_w"], st["k_heads"], cos, sin))


def plain_rope_one(st, x, w, heads, cos, sin):
    x = x.unflatten(-1, (heads, st["dim"])).float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
    before, turned, after = x.split((st["start"], st["rot"], st["dim"] - st["start"] - st["rot"]), -1)
    if st["style"] == "half":
        a, b = turned.chunk(2, -1)
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((before, turned, after), -1).to(torch.bfloat16)


def slot_bytes(st, slots):
    """The places [slots, heads, bytes] in the cache of the bytes of the tokens in `slots`."""
    heads, size, dim = st["heads"], st["page_size"], st["dim"]
    blocks = (slots // size)[:, None] * heads + torch.arange(heads, device=DEV)
    first = (blocks * (size // 16) + (slots % size // 16)[:, None]) * block_bytes(dim)
    return first[..., None] + st["places"][slots % 16][:, None]


def plain_cache(st):
    heads, dim = st["heads"], st["dim"]
    codes, scales = quantise(st["kv"].view(-1, 2, heads, dim))
    codes = codes[..., 0::2] + 16 * codes[..., 1::2]
    new = torch.cat((codes[:, 0], scales[:, 0], codes[:, 1], scales[:, 1]), -1)
    flat = st["cache"].view(-1)
    flat[slot_bytes(st, st["slots"])] = new
    level = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=DEV)
    raw = flat[slot_bytes(st, st["read"])].view(-1, heads, 2, 9 * dim // 16)
    c, s = raw.split((dim // 2, dim // 16), -1)
    x = level[torch.stack((c & 15, c >> 4), -1).int()].view(-1, heads, 2, dim // 16, 16) * s.contiguous().view(torch.float8_e4m3fn).float()[..., None]
    x = x.view(-1, heads, 2, dim).to(torch.bfloat16)
    return x[:, :, 0].contiguous(), x[:, :, 1].contiguous()


def plain_attention(st):
    seqs, q_len, hk, dim = st["seqs"], st["q_len"], st["kv_heads"], st["dim"]
    raw = st["cache"][st["table"].clamp(min=0).long()]  # [seqs, pages, heads, blocks, bytes]
    k, v = unpack(raw.transpose(1, 2), dim)
    k, v = k.reshape(seqs, hk, -1, dim), v.reshape(seqs, hk, -1, dim)
    q = st["q"].float().view(seqs, q_len, hk, -1, dim).permute(0, 2, 3, 1, 4) * dim ** -0.5  # [seqs, kv heads, group, queries, dim]
    z = (q.flatten(2, 3) @ k.transpose(-1, -2)).unflatten(2, (-1, q_len))
    p = torch.arange(k.shape[2], device=DEV)
    pos = (st["kv_len"].long()[:, None] - q_len + torch.arange(q_len, device=DEV))[:, :, None]  # [seqs, queries, 1]
    hidden = (p > pos) | (p <= pos - st["window"] if st["window"] else p < 0)
    z = z.masked_fill(hidden[:, None, None], float("-inf"))
    top = z.amax(-1, keepdim=True)
    w = torch.exp(z - top)
    total = w.sum(-1, keepdim=True)
    out = (w.flatten(2, 3) @ v).unflatten(2, (-1, q_len)) / total
    lse = (top + total.log()).squeeze(-1)
    return out.permute(0, 3, 1, 2, 4).reshape(seqs * q_len, -1, dim).to(torch.bfloat16), lse.permute(0, 3, 1, 2).reshape(seqs * q_len, -1)


# ---- what a pass cannot do without ------------------------------------------------------------------


def work(case):
    dim = case["dim"]
    if case["op"] == "rope":
        values = case["tokens"] * (case["q_heads"] + case["k_heads"]) * dim
        return {"bytes": 4 * values + 8 * case["tokens"] * case["axes"] + 8 * dim, "flops": 10 * values}
    if case["op"] == "cache":
        row = case["heads"] * dim
        new, read = sum(q for _, q in lengths(case)), sum(kv for kv, _ in lengths(case))
        return {"bytes": (new + read) * (4 * row + 9 * row // 8 + 8), "flops": 4 * new * row + 2 * read * row}
    keys = pairs = rows = 0
    for kv, q in lengths(case):
        w = case["window"] or kv
        keys += min(kv, w + q - 1)
        pairs += sum(min(w, kv - q + i + 1) for i in range(q))
        rows += q * case["q_heads"]
    return {"bytes": keys * case["kv_heads"] * dim * 9 // 8 + rows * (4 * dim + 4), "flops": 4 * dim * pairs * case["q_heads"]}


# ---- the definitions in 64 bits -----------------------------------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": exact_rope, "cache": exact_cache, "attention": exact_attention}[case["op"]](st)


def exact_rope(st):
    out = []
    angle = torch.stack([st["positions"][int(a)].double() * f for a, f in zip(st["axis"].cpu(), st["freq"])], 1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]  # [tokens, 1, rot / 2] on the unit circle
    half, s = st["rot"] // 2, st["start"]
    first = torch.arange(half, device=DEV) + s if st["style"] == "half" else 2 * torch.arange(half, device=DEV) + s
    second = first + (half if st["style"] == "half" else 1)
    for x, w, heads in ((st["q"], st["q_w"], st["q_heads"]), (st["k"], st["k_w"], st["k_heads"])):
        x = x.double().reshape(-1, heads, st["dim"])
        y = x / ((x * x).sum(-1, keepdim=True) / st["dim"] + 1e-6).sqrt() * w.double()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    return tuple(out)


def nearest(x, levels):
    """The index of the level nearest to each x >= 0 (levels rising from 0), of two as near the even one."""
    levels = torch.tensor(levels, dtype=torch.float64, device=DEV)
    middle = (levels[1:] + levels[:-1]) / 2
    low = torch.searchsorted(middle, x.contiguous())
    high = torch.searchsorted(middle, x.contiguous(), right=True)
    return torch.where(low % 2 == 0, low, high)


def scale_levels():
    """The values of the 8-bit scales: 4 exponent bits with bias 7, 3 mantissa bits, none above 448."""
    return [m / 512 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]


def exact_values(raw, dim):
    """The values [blocks, 2, 16, dim] that cache blocks [blocks, 18 * dim] stand for, by the places of their bytes."""
    places = byte_places(dim)
    kc, ks, vc, vs = places.split((dim // 2, dim // 16, dim // 2, dim // 16), 1)
    code = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device=DEV)
    scale = torch.tensor(scale_levels() + [float("nan")], dtype=torch.float64, device=DEV)
    out = []
    for c, s in ((kc, ks), (vc, vs)):
        b = raw[:, c.flatten()].view(-1, 16, dim // 2).int()
        x = torch.empty((len(raw), 16, dim), dtype=torch.float64, device=DEV)
        x[..., 0::2], x[..., 1::2] = code[b % 16], code[b // 16]
        out.append(x * scale[raw[:, s.flatten()].view(-1, 16, dim // 16).int()].repeat_interleave(16, -1))
    return torch.stack(out, 1)


def exact_cache(st):
    heads, dim, size = st["heads"], st["dim"], st["page_size"]
    pages = st["cache"].shape[0]
    held = exact_values(st["cache"].view(-1, block_bytes(dim)), dim).view(pages, heads, size // 16, 2, 16, dim)
    held = held.permute(0, 2, 4, 3, 1, 5).reshape(pages * size, 2, heads, dim)
    x = st["kv"].double().view(-1, 2, heads, dim // 16, 16)
    levels = torch.tensor(scale_levels(), dtype=torch.float64, device=DEV)
    s = levels[nearest(x.abs().amax(-1) / 6, scale_levels())][..., None]
    code = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    y = code[nearest(x.abs() / torch.where(s > 0, s, torch.ones_like(s)), E2M1)] * s * torch.sign(x)
    held[st["slots"]] = y.view(-1, 2, heads, dim)
    got = held[st["read"]]
    return got[:, 0], got[:, 1]


def exact_attention(st):
    hk, dim, q_len = st["kv_heads"], st["dim"], st["q_len"]
    group = st["q_heads"] // hk
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device=DEV)
    for i, n in enumerate(st["kv_len"].tolist()):
        used = st["table"][i, :-(-n // st["page_size"])].long()
        rows = slice(i * q_len, (i + 1) * q_len)
        pos = torch.arange(n - q_len, n, device=DEV)[:, None]
        p = torch.arange(n, device=DEV)[None]
        seen = (p <= pos) & (p > pos - (st["window"] or n + q_len))
        for h in range(hk):
            kv = exact_values(st["cache"][used, h].view(-1, block_bytes(dim)), dim).transpose(0, 1).reshape(2, -1, dim)[:, :n]
            z = torch.einsum("qgd,kd->gqk", st["q"][rows, h * group:(h + 1) * group].double(), kv[0]) / dim ** 0.5
            z = torch.where(seen, z, torch.full_like(z, float("-inf")))
            total = torch.logsumexp(z, -1)
            out[rows, h * group:(h + 1) * group] = torch.einsum("gqk,kd->qgd", torch.exp(z - total[..., None]), kv[1])
            lse[rows, h * group:(h + 1) * group] = total.T
    return out, lse
