"""Cases and plain forms of the operators that make a decode step's selection, in the order in which a program calls them:

  queries  the heads' queries from a projection: norm of each head, rotation, rounded to bf16 or to 8 bits with block scales
  keys     the new tokens' index keys: norm, rotation, quantised to 8 or 4 bits with block scales into the cache
  score    every key of a token's context scored against its queries: the sum over the heads of weight * max(0, q . k)
  select   the positions with the k best scores, ties to the lowest, ascending: what a resolve takes

``run`` computes a case with elementary torch operations, or (``own``) with the framework's kernels; ``exact`` computes
it from the definitions in 64 bits.
"""
import math

import torch

own = False

BLOCK = 32       # values under one scale
EPS = 1e-6
THETA = 10000.0  # base of the rotation's frequencies
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of a 4-bit value


def listed():
    return [
        # the index queries of one decode step, a token for each of 256 requests, in 8 bits
        dict(name="queries_256tok_h32_8bit", op="queries", n=256, heads=32, dim=128, rope=64, at=0, norm="none", bits=8,
             halves=False, pad=0),
        # a prompt's attention queries: each head normed, its last part rotated, in bf16
        dict(name="queries_8192tok_h16", op="queries", n=8192, heads=16, dim=192, rope=64, at=128, norm="rms", bits=16,
             halves=True, pad=0),
        # a few tokens with sizes off every power of two, the batch padded as a captured graph needs it
        dict(name="queries_37tok_h20_d96", op="queries", n=37, heads=20, dim=96, rope=32, at=64, norm="layer", bits=8,
             halves=True, pad=11),
        # one new key for each of 256 requests in 4 bits: what every decode step stores
        dict(name="keys_256req_decode_4bit", op="keys", R=256, shortest=1, longest=1, least=0, past=2000, dim=128, rope=64,
             at=0, norm="layer", bits=4, halves=False, pad=0),
        # prompts of uneven lengths, 8-bit keys
        dict(name="keys_8req_prompt_8bit", op="keys", R=8, shortest=2000, longest=8192, least=0, past=0, dim=128, rope=64,
             at=0, norm="layer", bits=8, halves=True, pad=100),
        # one user's step over a short context: all latency
        dict(name="score_1req_4096_h16_8bit", op="score", R=1, shortest=1, longest=1, least=4095, past=4095, dim=64,
             heads=16, bits=8),
        # a moderate batch of very uneven contexts
        dict(name="score_32req_ragged_h20_8bit", op="score", R=32, shortest=1, longest=1, least=0, past=32767, dim=128,
             heads=20, bits=8),
        # high concurrency over long contexts, 4-bit keys: the largest step
        dict(name="score_256req_40960_h32_4bit", op="score", R=256, shortest=1, longest=1, least=32768, past=40959, dim=128,
             heads=32, bits=4),
        # prompt chunks behind contexts of up to 16384
        dict(name="score_4req_chunk128_h32_4bit", op="score", R=4, shortest=128, longest=128, least=3968, past=15872,
             dim=128, heads=32, bits=4),
        # a single user's selection
        dict(name="select_1row_4096_k256", op="select", rows=1, least=4096, length=4096, k=256, recent=1, ties=False),
        # high concurrency over long contexts
        dict(name="select_256rows_40960_k2048", op="select", rows=256, least=32768, length=40960, k=2048, recent=1,
             ties=False),
        # a few requests with contexts of up to a million tokens, scores with few digits and so with many ties
        dict(name="select_2rows_1M_k2048_ties", op="select", rows=2, least=700_001, length=1_000_000, k=2048, recent=64,
             ties=True),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["queries", "keys", "score", "score", "score", "select", "select"])
    if op == "queries":
        dim = 32 * rng.randint(1, 8)
        heads = rng.choice([1, 8, 16, 20, 32, 48])
        rope = rng.choice([r for r in (0, 32, 64, 64) if r <= dim])
        return dict(op=op, n=_spread(rng, 1, min(8192, 8192 * 16 * 192 // (heads * dim))), heads=heads, dim=dim, rope=rope,
                    at=rng.choice([0, dim - rope]), norm=rng.choice(["none", "rms", "layer"]), bits=rng.choice([8, 16]),
                    halves=rng.random() < 0.5, pad=rng.choice([0, _spread(rng, 1, 50)]))
    if op == "keys":
        longest = _spread(rng, 1, 8192)
        R = _spread(rng, 1, max(1, min(256, (1 << 15) // longest)))
        return dict(op=op, R=R, shortest=_spread(rng, 1, longest), longest=longest, least=0,
                    past=_spread(rng, 1, max(1, min(1 << 17, (1 << 20) // R))), dim=rng.choice([64, 128, 128]),
                    rope=rng.choice([0, 32, 64]), at=0, norm=rng.choice(["none", "rms", "layer", "layer"]),
                    bits=rng.choice([4, 8]), halves=rng.random() < 0.5, pad=rng.choice([0, _spread(rng, 1, 200)]))
    if op == "score":
        past = _spread(rng, 1, 131_072)
        longest = rng.choice([1, 1, 1, _spread(rng, 2, 256)])
        heads = rng.choice([1, 8, 16, 20, 32, 40])
        dim, bits = rng.choice([64, 128, 128]), rng.choice([4, 8])
        # (pairs of a token and a key, and bytes of keys, as many as in the largest listed case at most)
        most = min(256 * 36_000 * 32 // (longest * max(heads, 32)), 256 * 36_000 * 512 // (dim * bits))
        return dict(op=op, R=_spread(rng, 1, max(1, min(256, most // (past + longest)))),
                    shortest=_spread(rng, 1, longest), longest=longest, least=rng.choice([0, past]), past=past, dim=dim,
                    heads=heads, bits=bits)
    length = _spread(rng, 64, 1_000_000)
    k = _spread(rng, 1, min(2048, length // 2))
    return dict(op=op, rows=_spread(rng, 1, max(1, min(256, 256 * 36_864 // length))), least=rng.choice([0, length]),
                length=length, k=k, recent=rng.choice([0, min(1, k // 2), _spread(rng, 1, max(1, k)) // 2]),
                ties=rng.random() < 0.4)


def _even(lo, hi, count):
    """Numbers from lo to hi, spread evenly, out of order, the same for every seed (a case's work does not go by it)."""
    even = [hi if count == 1 else lo + (hi - lo) * i // (count - 1) for i in range(count)]
    step = next(s for s in range(count // 2 + 1, count + 2) if math.gcd(s, count) == 1)
    return [even[i * step % count] for i in range(count)]


def _tokens(case):
    """Of each request its new tokens and those that it has, and of each new token its request and position."""
    new, old = _even(case["shortest"], case["longest"], case["R"]), _even(case["least"], case["past"], case["R"])[::-1]
    pad = case.get("pad", 0)
    req = [r for r, m in enumerate(new) for _ in range(m)] + [-1] * pad
    pos = [o + i for o, m in zip(old, new) for i in range(m)] + [-1] * pad
    return new, old, req, pos, case["past"] + case["longest"]


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, gen, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(torch.bfloat16)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _frequencies(rope):
    i = torch.arange(rope // 2, dtype=torch.float64, device="cuda")
    return THETA ** (-2.0 * i / max(rope, 1))


def _context(R, H, k=1):
    """The handle that a program keeps (its rows play no part here)."""
    import hierarchical_memory_amd as hm
    return hm.SwapIn(hm.config(R, k, k, 0.0, 16, H, 0))


def _exponents(y, bits):
    """For each block of 32 values in the last dimension, the least e with every value at most 448 * 2^e (448 is the
    largest 8-bit value, 0.875 * 2^9) or 6 * 2^e (the largest 4-bit value, 0.75 * 2^3), and -100 at least."""
    top = y.abs().unflatten(-1, (-1, BLOCK)).amax(-1)
    m, e = torch.frexp(top)
    e = e - 9 + (m > 0.875).to(e.dtype) if bits == 8 else e - 3 + (m > 0.75).to(e.dtype)
    return torch.where(top > 0, e, torch.full_like(e, -100)).clamp(min=-100)


def _quantised(y, bits):
    """Bytes of the values and of the scales for y (float32). 4-bit values lie in pairs, the even one in the low bits."""
    e = _exponents(y, bits)
    x = torch.ldexp(y.unflatten(-1, (-1, BLOCK)), -e.unsqueeze(-1)).flatten(-2)
    if bits == 8:
        return x.to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)
    a = x.abs()  # between two magnitudes to the nearer one, half way to the one of even number
    code = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    code = code + 8 * torch.signbit(x).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _values(codes, scales, bits, dtype):
    """What the bytes of values and scales stand for."""
    if bits == 8:
        v = codes.view(torch.float8_e4m3fn).to(dtype)
    else:
        grid = torch.tensor([*GRID, *(-g for g in GRID)], dtype=dtype, device=codes.device)
        v = grid[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    return (v.unflatten(-1, (-1, BLOCK)) * torch.exp2(scales.to(dtype) - 127).unsqueeze(-1)).flatten(-2)


def _weights(case, gen):
    """A norm's weight and bias."""
    dim, norm = case["dim"], case["norm"]
    w = (1 + 0.1 * torch.randn((dim,), generator=gen, device="cuda")).to(torch.bfloat16)
    b = _normal((dim,), gen, 0.1)
    return w if norm != "none" else None, b if norm == "layer" else None


def _head_format(case):
    import hierarchical_memory_amd as hm
    return hm.head_format(case["dim"], case["rope"], case["at"], hm.HS_ROPE_HALVES if case["halves"] else hm.HS_ROPE_PAIRS,
                          {"none": hm.HS_NORM_NONE, "rms": hm.HS_NORM_RMS, "layer": hm.HS_NORM_LAYER}[case["norm"]], EPS)


def _key_format(case):
    import hierarchical_memory_amd as hm
    return hm.key_format(case["dim"], hm.HS_KEY_MXFP8 if case["bits"] == 8 else hm.HS_KEY_MXFP4)


def _prepare_queries(case, gen):
    n, heads, dim = case["n"], case["heads"], case["dim"]
    s = {"case": case, "freqs": _frequencies(case["rope"]) if case["rope"] else None}
    # the projection of a program that computes the heads' queries and more in one product: rows wider than the queries
    s["x"] = _normal((n + case["pad"], heads * dim + 64), gen, 2.0)[:, :heads * dim].unflatten(1, (heads, dim))
    s["weight"], s["bias"] = _weights(case, gen)
    pos = torch.randint(0, 1 << 17, (n,), generator=gen, device="cuda", dtype=torch.int32)
    s["pos"] = torch.cat([pos, torch.full((case["pad"],), -1, dtype=torch.int32, device="cuda")])
    if own:
        s["sw"] = _context(1, 1)
        s["fmt"] = _head_format(case)
        shape = (n + case["pad"], heads, dim)
        if case["bits"] == 16:
            s["o"], s["scales"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), None
        else:
            s["o"] = torch.zeros(shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
            s["scales"] = torch.zeros((*shape[:2], dim // BLOCK), dtype=torch.uint8, device="cuda")
    return s


def _prepare_keys(case, gen):
    _, _, req, pos, H = _tokens(case)
    R, dim, bits = case["R"], case["dim"], case["bits"]
    n = len(req)
    s = {"case": case, "req": _int32(req), "pos": _int32(pos), "H": H}
    s["freqs"] = _frequencies(case["rope"]) if case["rope"] else None
    s["x"] = _normal((n, dim + 32), gen, 3.0)[:, :dim]
    s["weight"], s["bias"] = _weights(case, gen)
    if own:
        import hierarchical_memory_amd as hm
        s["sw"], s["fmt"], s["key"] = _context(R, H), _head_format(case), _key_format(case)
        s["cache"] = s["sw"].key_cache(s["key"])
        codes, s["scales"] = hm.key_parts(s["sw"].cfg, s["key"], s["cache"])
    else:
        # a row behind the last takes the tokens that are not there, so that no size depends on the data
        s["codes"] = torch.zeros((R * H + 1, dim * bits // 8), dtype=torch.uint8, device="cuda")
        s["rows"] = torch.zeros((R * H + 1, dim // BLOCK), dtype=torch.uint8, device="cuda")
        codes, s["scales"] = s["codes"][:-1].view(R, H, -1), s["rows"][:-1].view(R, H, -1)
    # (4-bit values have no type of their own: what they stand for comes back in bf16)
    s["stored"] = codes.view(torch.float8_e4m3fn) if bits == 8 else None
    s["values"] = torch.zeros((n, dim), dtype=torch.bfloat16, device="cuda") if bits == 4 else None
    return s


def _prepare_score(case, gen):
    new, old, req, pos, H = _tokens(case)
    R, dim, heads, bits = (case[x] for x in ("R", "dim", "heads", "bits"))
    n = len(req)
    s = {"case": case, "req": _int32(req), "pos": _int32(pos), "H": H}
    s["q"], s["q_scales"] = _quantised(torch.randn((n, heads, dim), generator=gen, device="cuda"), 8)
    s["q"] = s["q"].view(torch.float8_e4m3fn)
    s["weights"] = torch.randn((n, heads), generator=gen, device="cuda") * (heads * dim) ** -0.5
    codes = torch.empty((R, H, dim * bits // 8), dtype=torch.uint8, device="cuda")
    scales = torch.empty((R, H, dim // BLOCK), dtype=torch.uint8, device="cuda")
    for r in range(0, R, 32):
        size = (min(32, R - r), H, dim)
        codes[r:r + 32], scales[r:r + 32] = _quantised(torch.randn(size, generator=gen, device="cuda"), bits)
    if own:
        import hierarchical_memory_amd as hm
        s["sw"], s["key"] = _context(R, H), _key_format(case)
        s["cache"] = s["sw"].key_cache(s["key"])
        mine = hm.key_parts(s["sw"].cfg, s["key"], s["cache"])
        mine[0].copy_(codes)
        mine[1].copy_(scales)
        s["scores"] = torch.zeros((n, -(-H // 4) * 4), dtype=torch.float32, device="cuda")
    else:
        s["codes"], s["scales"] = codes, scales
        # the batch as [R, longest] tokens, those behind a request's last one repeating another, and where each token is
        first, most = [sum(new[:r]) for r in range(R)], case["longest"]
        s["padded"] = torch.tensor([[min(f + i, n - 1) for i in range(most)] for f in first], device="cuda")
        s["packed"] = torch.tensor([r * most + i for r, m in enumerate(new) for i in range(m)], device="cuda")
    return s


def _prepare_select(case, gen):
    rows, L, k = case["rows"], case["length"], case["k"]
    s = {"case": case}
    x = torch.randn((rows, -(-L // 4) * 4), generator=gen, device="cuda") * 0.3 + 0.5
    s["scores"] = x.to(torch.bfloat16).float() if case["ties"] else x
    s["pos"] = _int32([m - 1 for m in _even(case["least"], L, rows)])  # (-1: a row without a key)
    if own:
        s["sw"] = _context(rows, L, k)
        s["topk"] = torch.empty((rows, k), dtype=torch.int32, device="cuda")
        s["work"] = s["sw"].select_work(rows, x.shape[1])
    return s


def prepare(case, seed):
    gen = _generator(seed)
    return {"queries": _prepare_queries, "keys": _prepare_keys, "score": _prepare_score, "select": _prepare_select}[
        case["op"]](case, gen)


def run(s):
    op = s["case"]["op"]
    if op == "queries":
        return _own_queries(s) if own else _queries(s)
    if op == "keys":
        return _own_keys(s) if own else _keys(s)
    if op == "score":
        return _own_score(s) if own else _score(s)
    return _own_select(s) if own else _select(s)


# --- the framework's calls

def _own_queries(s):
    import hierarchical_memory_amd as hm
    hm.hs_norm_rotate(s["sw"].ctx, s["fmt"], s["x"], s["weight"], s["bias"], s["freqs"], s["pos"], s["o"],
                      scales=s["scales"])
    return _rounded(s["o"], s["scales"])


def _own_keys(s):
    import hierarchical_memory_amd as hm
    hm.hs_store_keys(s["sw"].ctx, s["fmt"], s["key"], s["x"], s["weight"], s["bias"], s["freqs"], s["req"], s["pos"],
                     s["cache"], values=s["values"])
    return _stored(s)


def _own_score(s):
    import hierarchical_memory_amd as hm
    hm.hs_score_keys(s["sw"].ctx, s["key"], s["cache"], s["q"], s["q_scales"], s["weights"], s["req"], s["pos"],
                     s["scores"])
    return {"scores": s["scores"]}


def _own_select(s):
    import hierarchical_memory_amd as hm
    hm.hs_select(s["sw"].ctx, s["scores"], s["pos"], s["topk"], recent=s["case"]["recent"], work=s["work"])
    return {"topk": s["topk"]}


def _rounded(o, scales):
    return {"o": o} if scales is None else {"o": o, "scales": scales.view(torch.float8_e8m0fnu)}


def _stored(s):
    """What a store leaves: the cache's values and scales as the numbers that they are."""
    got = {"scales": s["scales"].view(torch.float8_e8m0fnu)}
    return got | ({"values": s["values"]} if s["stored"] is None else {"stored": s["stored"]})


# --- plain forms

def _normed(x, case, weight, bias):
    if case["norm"] == "rms":
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    if case["norm"] == "layer":
        x = x - x.mean(-1, keepdim=True)
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float() + bias.float()
    return x


def _rotated(y, case, pos, freqs):
    """The pairs of y's rotated part [n, heads, at .. at + rope) turned by pos * freqs (angles in 64 bits)."""
    at, rope = case["at"], case["rope"]
    if not rope:
        return y
    turn = (pos.double()[:, None] * freqs)[:, None]
    c, sn = torch.cos(turn).to(y.dtype), torch.sin(turn).to(y.dtype)
    x = y[..., at:at + rope]
    a, b = (x[..., :rope // 2], x[..., rope // 2:]) if case["halves"] else (x[..., 0::2], x[..., 1::2])
    u, v = a * c - b * sn, a * sn + b * c
    z = torch.cat([u, v], -1) if case["halves"] else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([y[..., :at], z, y[..., at + rope:]], -1)


def _queries(s):
    case = s["case"]
    y = _rotated(_normed(s["x"].float(), case, s["weight"], s["bias"]), case, s["pos"], s["freqs"])
    there = (s["pos"] >= 0)[:, None, None]
    if case["bits"] == 16:
        return _rounded((y * there).to(torch.bfloat16), None)
    o, scales = _quantised(y, 8)
    return _rounded((o * there).view(torch.float8_e4m3fn), scales * there)


def _keys(s):
    case = s["case"]
    y = _rotated(_normed(s["x"].float()[:, None], case, s["weight"], s["bias"]), case, s["pos"], s["freqs"])[:, 0]
    codes, scales = _quantised(y, case["bits"])
    there = s["pos"] >= 0
    row = torch.where(there, s["req"].long() * s["H"] + s["pos"].long(), case["R"] * s["H"])
    s["codes"][row], s["rows"][row] = codes, scales
    if case["bits"] == 4:
        s["values"] = (_values(codes, scales, 4, torch.float32) * there[:, None]).to(torch.bfloat16)
    return _stored(s)


def _score(s):
    case, H = s["case"], s["H"]
    R, heads, most = case["R"], case["heads"], case["longest"]
    keys = _values(s["codes"], s["scales"], case["bits"], torch.float32)
    q = _values(s["q"].view(torch.uint8), s["q_scales"], 8, torch.float32)[s["padded"]]  # [R, most, heads, dim]
    dots = torch.bmm(q.flatten(1, 2), keys.transpose(1, 2).contiguous()).clamp_(min=0.0)  # [R, most * heads, H]
    scores = (dots.view(R * most, heads, H) * s["weights"][s["padded"].flatten()].unsqueeze(-1)).sum(1)[s["packed"]]
    x = torch.arange(-(-H // 4) * 4, device="cuda")
    scores = torch.nn.functional.pad(scores, (0, x.numel() - H))
    return {"scores": torch.where(x <= s["pos"][:, None], scores, 0.0)}


def _select(s):
    case = s["case"]
    k, recent = case["k"], case["recent"]
    x = torch.arange(s["scores"].shape[1], device="cuda")
    last = s["pos"].long()[:, None]
    score = torch.where(x > last - recent, math.inf, s["scores"])
    score = torch.where((x <= last) & (score == score), score, -math.inf)
    best, order = torch.sort(score, dim=1, descending=True, stable=True)
    best, order = best[:, :k], order[:, :k]
    ids = torch.where(best > -math.inf, order, x.numel()).sort(1).values
    ids = torch.nn.functional.pad(ids, (0, k - ids.shape[1]), value=x.numel())
    return {"topk": torch.where(ids < x.numel(), ids, -1).to(torch.int32)}


# --- the least work

def work(case):
    op = case["op"]
    if op == "queries":
        rows, dim = case["n"] * case["heads"], case["dim"]
        out = 2 * dim if case["bits"] == 16 else dim + dim // BLOCK
        return {"bytes": rows * (2 * dim + out) + 4 * case["n"], "flops": rows * (8 * dim + 6 * case["rope"])}
    if op == "select":
        keys = sum(_even(case["least"], case["length"], case["rows"]))
        return {"bytes": 4 * keys + 4 * case["rows"] * (case["k"] + 1), "flops": max(1, 2 * keys)}
    new, old, _, _, _ = _tokens(case)
    n, dim = sum(new), case["dim"]
    key = dim * case["bits"] // 8 + dim // BLOCK
    if op == "keys":
        return {"bytes": n * (2 * dim + key + 8 + (2 * dim if case["bits"] == 4 else 0)), "flops": n * 14 * dim}
    heads = case["heads"]
    pairs = sum(m * o + m * (m + 1) // 2 for m, o in zip(new, old))
    return {"bytes": sum(m + o for m, o in zip(new, old)) * key + 4 * pairs
            + n * (heads * (dim + dim // BLOCK + 4) + 8), "flops": pairs * heads * (2 * dim + 3)}


# --- the definitions in 64 bits

def exact(case, seed):
    op = case["op"]
    if op == "select":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "score":
        return _exact_score(s)
    return _exact_queries(s) if op == "queries" else _exact_keys(s)


def _turned(s, x):
    """Normed and rotated heads, unrounded, from x [n, heads, dim]."""
    case = s["case"]
    at, rope = case["at"], case["rope"]
    x = x.double()
    if case["norm"] == "rms":
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / case["dim"] + EPS) * s["weight"].double()
    elif case["norm"] == "layer":
        mean = x.sum(-1, keepdim=True) / case["dim"]
        var = ((x - mean) ** 2).sum(-1, keepdim=True) / case["dim"]
        x = (x - mean) / torch.sqrt(var + EPS) * s["weight"].double() + s["bias"].double()
    if not rope:
        return x
    angle = (s["pos"].double()[:, None] * s["freqs"])[:, None]
    z = torch.polar(torch.ones_like(angle), angle)
    part = x[..., at:at + rope]
    if case["halves"]:
        w = torch.complex(part[..., :rope // 2].contiguous(), part[..., rope // 2:].contiguous()) * z
        part = torch.cat([w.real, w.imag], -1)
    else:
        part = torch.view_as_real(torch.view_as_complex(part.unflatten(-1, (-1, 2)).contiguous()) * z).flatten(-2)
    return torch.cat([x[..., :at], part, x[..., at + rope:]], -1)


def _scale_of(y, largest):
    top = y.abs().reshape(*y.shape[:-1], -1, BLOCK).amax(-1)
    return 2.0 ** torch.ceil(torch.log2(top / largest)).clamp(min=-100)


def _exact_queries(s):
    """Unrounded values: bf16 and 8-bit outputs are compared with the numbers that they round."""
    y, there = _turned(s, s["x"]), (s["pos"] >= 0)[:, None, None]
    if s["case"]["bits"] == 16:
        return {"o": y * there}
    scale = _scale_of(y, 448.0)
    o = y / scale.repeat_interleave(BLOCK, -1)
    # (rows of tokens that are not there: zero bytes, whose scale stands for 2^-127)
    return {"o": o * there, "scales": torch.where(there, scale, 2.0 ** -127)}


def _exact_keys(s):
    case = s["case"]
    y, there = _turned(s, s["x"][:, None])[:, 0], s["pos"] >= 0
    scale = _scale_of(y, 448.0 if case["bits"] == 8 else 6.0)
    r, x = s["req"][there].long(), s["pos"][there].long()
    scales = torch.full((case["R"], s["H"], scale.shape[1]), 2.0 ** -127, dtype=torch.float64, device="cuda")
    scales[r, x] = scale[there]
    v = y / scale.repeat_interleave(BLOCK, -1)
    if case["bits"] == 8:
        stored = torch.zeros((case["R"], s["H"], case["dim"]), dtype=torch.float64, device="cuda")
        stored[r, x] = v[there]
        return {"scales": scales, "stored": stored}
    grid = torch.tensor(GRID, dtype=torch.float64, device="cuda")
    middle = (grid[1:] + grid[:-1]) / 2
    code = torch.bucketize(v.abs(), middle)  # (half way: the lower one, which has to be of even number)
    code = code + ((code % 2 == 1) & (v.abs() == middle[code.clamp(max=6)])).long()
    v = torch.sign(v) * grid[code]
    return {"scales": scales, "values": v * scale.repeat_interleave(BLOCK, -1) * there[:, None]}


def _exact_score(s):
    case, H = s["case"], s["H"]
    scores = torch.zeros((s["pos"].numel(), -(-H // 4) * 4), dtype=torch.float64, device="cuda")
    if own:
        import hierarchical_memory_amd as hm
        codes, scales = hm.key_parts(s["sw"].cfg, s["key"], s["cache"])
    else:
        codes, scales = s["codes"], s["scales"]
    q = _values(s["q"].view(torch.uint8), s["q_scales"], 8, torch.float64)
    t = 0
    for r, m in enumerate(_tokens(case)[0]):
        key = _values(codes[r], scales[r], case["bits"], torch.float64).T.contiguous()
        for i in range(0, m, 64):
            j = min(m, i + 64)
            dots = torch.relu(q[t + i:t + j].flatten(0, 1) @ key).unflatten(0, (j - i, -1))
            scores[t + i:t + j, :H] = (s["weights"][t + i:t + j].double().unsqueeze(-1) * dots).sum(1)
        t += m
    x = torch.arange(scores.shape[1], device="cuda")
    return {"scores": scores.masked_fill(x > s["pos"][:, None], 0.0)}
