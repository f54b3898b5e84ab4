"""Cases and plain forms of the latent-attention operators around the swap-in path.

Four operators, in the order in which a serving program calls them:

  map     every new token of a ragged batch: its request, its position, its row of the device tail
  store   the new tokens' latent rows: root-mean-square norm, rotation, and (8-bit rows) block scales, into the tail
  attend  one decode step's attention (absorbed form) over the selected rows, read in place through the slots that a
          resolve returned, or from the gathered rows of a trial
  prompt  the prompt's causal attention (expanded form) over ragged sequences

``run`` computes a case with elementary torch operations, or (``own``) with the framework's kernels; ``exact`` computes
it from the definitions in 64 bits.
"""
import math

import torch

own = False

BLOCK = 32       # values of an 8-bit row under one scale
EPS = 1e-6
THETA = 10000.0  # base of the rotation's frequencies


def listed():
    return [
        # one request with a 256-row selection: what a single user's step costs, all latency
        dict(name="attend_1req_k256_h16", op="attend", R=1, k=256, B=512, T=0, heads=16, latent=512, rope=64, bits=16,
             pad=0.0, empty=0, gathered=False),
        # a moderate batch, the heads of one GPU of eight
        dict(name="attend_32req_k2048_h16", op="attend", R=32, k=2048, B=4096, T=0, heads=16, latent=512, rope=64,
             bits=16, pad=0.0, empty=0, gathered=False),
        # high concurrency with every head on this GPU: the largest step
        dict(name="attend_256req_k2048_h128", op="attend", R=256, k=2048, B=4096, T=0, heads=128, latent=512, rope=64,
             bits=16, pad=0.0, empty=0, gathered=False),
        # rows of the hot buffer and of a device tail, held in 8 bits, some of the selection padding
        dict(name="attend_64req_tail_h64_8bit", op="attend", R=64, k=2048, B=4096, T=8192, heads=64, latent=512,
             rope=64, bits=8, pad=0.03, empty=0, gathered=False),
        # a retryable step: the gathered rows of a trial, sizes off every tile, requests without a row
        dict(name="attend_7req_k999_h20_trial", op="attend", R=7, k=999, B=1500, T=33, heads=20, latent=256, rope=32,
             bits=16, pad=0.2, empty=2, gathered=True),
        # a batch of short prompts of uneven lengths
        dict(name="prompt_8req_short_h16", op="prompt", R=8, shortest=1, longest=300, past=0, heads=16, nope=128,
             rope=64, value=128, latent=512, causal=True),
        # one long prompt, the heads of one GPU of eight
        dict(name="prompt_1req_8192_h16", op="prompt", R=1, shortest=8192, longest=8192, past=0, heads=16, nope=128,
             rope=64, value=128, latent=512, causal=True),
        # chunks of 512 tokens behind a context of up to 16384, with the larger head
        dict(name="prompt_4req_chunk512_h8", op="prompt", R=4, shortest=512, longest=512, past=15872, heads=8,
             nope=192, rope=64, value=256, latent=512, causal=True),
        # one new token for each of 256 requests, held in 8 bits: what every decode step begins with
        dict(name="store_256req_decode_8bit", op="store", R=256, shortest=1, longest=1, T=64, latent=512, rope=64,
             bits=8, past=2000, halves=False, pad=0),
        # prompts of uneven lengths into the device tail, bf16 rows
        dict(name="store_8req_prompt", op="store", R=8, shortest=2000, longest=8192, T=8192, latent=512, rope=64,
             bits=16, past=0, halves=True, pad=100),
        # the map of one decode step
        dict(name="map_256req_decode", op="map", R=256, shortest=1, longest=1, T=8192, past=32768, pad=0),
        # a large ragged batch, padded to a fixed length as a captured graph needs it
        dict(name="map_4096req_ragged", op="map", R=4096, shortest=0, longest=511, T=512, past=0, pad=5000),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "prompt", "prompt", "store", "map"])
    if op == "attend":
        heads = rng.choice([1, 8, 16, 16, 20, 32, 64, 100, 128])
        latent, rope = rng.choice([(512, 64), (512, 64), (512, 64), (256, 64), (256, 32)])
        k = _spread(rng, 1, 2048)
        R = _spread(rng, 1, max(1, min(256, (256 * 2048 * 128) // (k * max(heads, 32)))))
        return dict(op=op, R=R, k=k, B=k + _spread(rng, 1, 2048), T=rng.choice([0, 0, _spread(rng, 1, 1024)]),
                    heads=heads, latent=latent, rope=rope, bits=rng.choice([8, 16]),
                    pad=rng.choice([0.0, round(rng.uniform(0.0, 0.5), 3)]), empty=rng.choice([0, 0, (R + 3) // 4]),
                    gathered=rng.random() < 0.25)
    if op == "prompt":
        nope, value = rng.choice([(128, 128), (128, 128), (64, 64), (192, 256)])
        longest = _spread(rng, 1, 4096)
        past = rng.choice([0, 0, _spread(rng, 1, 8192)])
        heads = rng.choice([1, 4, 8, 16, 20])
        most = min(16 * 4096 * 8192 // (longest * (longest + past) * heads), 400_000 // ((longest + past) * heads))
        return dict(op=op, R=_spread(rng, 1, max(1, min(64, most))), shortest=_spread(rng, 1, longest),
                    longest=longest, past=past, heads=heads, nope=nope, rope=rng.choice([64, 64, 32]), value=value,
                    latent=512, causal=rng.random() < 0.8)
    if op == "store":
        longest = _spread(rng, 1, 4096)
        R = _spread(rng, 1, max(1, min(256, (1 << 15) // longest)))
        latent, rope = rng.choice([(512, 64), (512, 64), (256, 64), (256, 32), (512, 32)])
        # (the context's pinned host pool, R x positions x row, stays below 300 MB)
        past = _spread(rng, 1, max(1, min(1 << 17, 300_000_000 // (R * 2 * (latent + rope)) - longest)))
        return dict(op=op, R=R, shortest=_spread(rng, 1, longest), longest=longest, T=longest + _spread(rng, 1, 100),
                    latent=latent, rope=rope, bits=rng.choice([8, 16]), past=past,
                    halves=rng.random() < 0.5, pad=rng.choice([0, _spread(rng, 1, 200)]))
    R = _spread(rng, 1, 4096)
    return dict(op=op, R=R, shortest=rng.choice([0, 1]), longest=_spread(rng, 1, 256),
                T=rng.choice([0, 300, _spread(rng, 256, 8192)]), past=_spread(rng, 1, min(1 << 17, (1 << 24) // R)),
                pad=rng.choice([0, _spread(rng, 1, 2000)]))


def _lengths(case):
    """The requests' new tokens, the same for every seed (a case's work does not go by its seed): spread evenly
    between the shortest and the longest, out of order."""
    R, lo, hi = case["R"], case["shortest"], case["longest"]
    even = [hi if R == 1 else lo + (hi - lo) * i // (R - 1) for i in range(R)]
    step = next(s for s in range(R // 2 + 1, R + 2) if math.gcd(s, R) == 1)
    return [even[i * step % R] for i in range(R)]


def _row_bytes(latent, rope, bits):
    """bf16 rows: [latent | rope] in bf16. 8-bit rows: the latent's values in e4m3, one power-of-two scale (e8m0) for
    each block of 32, filled up to 16 bytes, then the rope part in bf16."""
    return 2 * (latent + rope) if bits == 16 else latent + 16 * -(-latent // (16 * BLOCK)) + 2 * rope


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, gen, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(torch.bfloat16)


def _scale_exponents(y):
    """For each block of 32 values in the last dimension, the least e with every value at most 448 * 2^e (448 is the
    largest e4m3 value, 0.875 * 2^9), and -100 at least."""
    top = y.abs().unflatten(-1, (-1, BLOCK)).amax(-1)
    m, e = torch.frexp(top)
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(top > 0, e, torch.full_like(e, -100)).clamp(min=-100)


def _pack8(y, rope):
    """8-bit rows of the latent parts y (float32) and the rope parts (bf16)."""
    e = _scale_exponents(y)
    scaled = torch.ldexp(y.unflatten(-1, (-1, BLOCK)), -e.unsqueeze(-1)).flatten(-2)
    fill = torch.zeros(*y.shape[:-1], -e.shape[-1] % 16, dtype=torch.uint8, device=y.device)
    return torch.cat([scaled.to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8), fill,
                      rope.contiguous().view(torch.uint8)], -1)


def _parts(rows, latent, rope):
    """The parts of 8-bit rows [..., bytes] as views: e4m3 values, e8m0 scales, rope values."""
    return (rows[..., :latent].view(torch.float8_e4m3fn),
            rows[..., latent:latent + latent // BLOCK].view(torch.float8_e8m0fnu),
            rows[..., rows.shape[-1] - 2 * rope:].view(torch.bfloat16))


def _values(rows, case, dtype):
    """The latent and rope values that rows (bytes) stand for."""
    latent, rope = case["latent"], case["rope"]
    if case["bits"] == 16:
        return rows.view(torch.bfloat16).to(dtype)
    q, s, r = rows[..., :latent], rows[..., latent:latent + latent // BLOCK], rows[..., rows.shape[-1] - 2 * rope:]
    v = q.contiguous().view(torch.float8_e4m3fn).to(dtype).unflatten(-1, (-1, BLOCK))
    v = v * torch.exp2(s.to(dtype) - 127).unsqueeze(-1)
    return torch.cat([v.flatten(-2), r.contiguous().view(torch.bfloat16).to(dtype)], -1)


def _context(case, host_rows, row_bytes):
    """The handle that a program keeps, with its device buffers. The plain form has buffers of the same shapes."""
    import hierarchical_memory_amd as hm
    B = case.get("B", 1)
    return hm.SwapIn(hm.config(case["R"], case.get("k", 1), B, 0.0, row_bytes, host_rows, case.get("T", 0)))


def _frequencies(rope):
    i = torch.arange(rope // 2, dtype=torch.float64, device="cuda")
    return THETA ** (-2.0 * i / rope)


def _prepare_attend(case, gen):
    R, k, B, T, heads = (case[n] for n in ("R", "k", "B", "T", "heads"))
    latent, rope = case["latent"], case["rope"]
    rb = _row_bytes(latent, rope, case["bits"])
    s = {"case": case, "scale": 192 ** -0.5}

    def rows(n):  # rows as a store leaves them: a normed latent part and a rotated part
        if case["bits"] == 16:
            return _normal((R, n, latent + rope), gen).view(torch.uint8)
        y = torch.randn((R, n, latent), generator=gen, device="cuda")
        return _pack8(y, _normal((R, n, rope), gen))

    # the selection as a resolve answers it: slots in the order of the ids, -1 where there was padding
    out = torch.rand((R, B + T), generator=gen, device="cuda").argsort(1)[:, :k].to(torch.int32)
    out[torch.rand((R, k), generator=gen, device="cuda") < case["pad"]] = -1
    if case["empty"]:
        out[torch.randperm(R, generator=gen, device="cuda")[:case["empty"]]] = -1
    s["out"] = out.contiguous()
    s["q"] = _normal((R, heads, latent + rope), gen, 0.9)
    s["gather"] = None
    if case["gathered"]:
        s["gather"] = rows(k) * (out >= 0).unsqueeze(-1)
        s["hot"] = s["tail"] = None
    else:
        s["hot"], s["tail"] = rows(B), rows(T) if T else None
    if own:
        import hierarchical_memory_amd as hm
        s["fmt"] = hm.row_format(latent, rope, hm.HS_ROW_BF16 if case["bits"] == 16 else hm.HS_ROW_MXFP8)
        s["sw"] = _context(case, 1, rb)
        if not case["gathered"]:
            s["sw"].hot.copy_(s["hot"])
            if T:
                s["sw"].tail.copy_(s["tail"])
        s["o"] = torch.empty((R, heads, latent), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((R, heads), dtype=torch.float32, device="cuda")
        s["work"] = s["sw"].attend_work(s["fmt"], heads)
    return s


def _prepare_prompt(case, gen):
    R, heads, nope, rope, value = (case[n] for n in ("R", "heads", "nope", "rope", "value"))
    new = torch.tensor(_lengths(case), dtype=torch.int32)
    old = torch.tensor([case["past"] * (i + 1) // R for i in range(R)], dtype=torch.int32)

    def ends(n):
        return torch.cat([torch.zeros(1, dtype=torch.int32), n.cumsum(0).to(torch.int32)]).cuda()

    s = {"case": case, "scale": (nope + rope) ** -0.5, "cu_q": ends(new), "cu_k": ends(new + old)}
    N, M = int(new.sum()), int((new + old).sum())
    s["q"] = _normal((N, heads, nope + rope), gen, 1.5)
    s["kv"] = _normal((M, heads, nope + value), gen)  # each head's [key | value], as one product with the weights gives it
    s["latent"] = _normal((M, case["latent"] + rope), gen)
    if own:
        s["sw"] = _context(case, 1, 16)
        s["o"] = torch.empty((N, heads, value), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((N, heads), dtype=torch.float32, device="cuda")
    return s


def _prepare_tokens(case, gen):
    """The lengths of a map or a store: each request has some tokens already, its tail window ends T tokens further on
    than the oldest token that it holds."""
    R, T = case["R"], case["T"]
    new = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    old = torch.randint(0, case["past"] + 1, (R,), generator=gen, device="cuda", dtype=torch.int32)
    first = (old + new - T).clamp(min=0).to(torch.int32) if T else None
    return new, old, first, sum(_lengths(case)) + case["pad"], case["past"] + case["longest"]


def _prepare_map(case, gen):
    new, old, first, N, H = _prepare_tokens(case, gen)
    if first is not None:  # half of the requests have begun to move tokens out of the tail's front
        first += torch.randint(0, 2, first.shape, generator=gen, device="cuda", dtype=torch.int32)
    s = {"case": case, "new": new, "old": old, "first": first, "N": N, "H": H, "B": 1}
    if own:
        s["sw"] = _context(case, H, 16)
        s["map"] = s["sw"].map_buffers(N)
        s["status"] = torch.empty((case["R"],), dtype=torch.int32, device="cuda")
    return s


def _prepare_store(case, gen):
    R, T, latent, rope = (case[n] for n in ("R", "T", "latent", "rope"))
    new, old, first, N, H = _prepare_tokens(case, gen)
    req, pos, slot = _map(new, old, first, N, 1, T, H)[1:4]
    s = {"case": case, "req": req, "pos": pos, "slot": slot, "freqs": _frequencies(rope)}
    s["x"] = _normal((N, latent + rope), gen, 3.0)
    s["weight"] = (1 + 0.1 * torch.randn((latent,), generator=gen, device="cuda")).to(torch.bfloat16)
    rb = _row_bytes(latent, rope, case["bits"])
    if own:
        import hierarchical_memory_amd as hm
        s["fmt"] = hm.row_format(latent, rope, hm.HS_ROW_BF16 if case["bits"] == 16 else hm.HS_ROW_MXFP8)
        s["sw"] = _context(case, H, rb)
        s["tail"] = s["sw"].tail
        s["latent"] = torch.zeros((N, latent + rope), dtype=torch.bfloat16, device="cuda")
    else:
        # a row behind the tail's takes the tokens that are not there, so that no size depends on the data
        s["rows"] = torch.zeros((R * T + 1, rb), dtype=torch.uint8, device="cuda")
        s["tail"] = s["rows"][:-1].view(R, T, rb)
    return s


def prepare(case, seed):
    gen = _generator(seed)
    return {"attend": _prepare_attend, "prompt": _prepare_prompt, "store": _prepare_store, "map": _prepare_map}[
        case["op"]](case, gen)


def run(s):
    op = s["case"]["op"]
    if op == "attend":
        return _own_attend(s) if own else _attend(s)
    if op == "prompt":
        return _own_prompt(s) if own else _prompt(s)
    if op == "store":
        return _own_store(s) if own else _store(s)
    if own:
        return _own_map(s)
    cu, req, pos, slot, status = _map(s["new"], s["old"], s["first"], s["N"], s["B"], s["case"]["T"], s["H"])
    return {"cu": cu, "req": req, "pos": pos, "slot": slot, "status": status}


# --- the framework's calls

def _own_attend(s):
    import hierarchical_memory_amd as hm
    hm.hs_attend(s["sw"].ctx, s["fmt"], s["q"], s["scale"], s["out"], s["o"], s["lse"], gather=s["gather"],
                 work=s["work"])
    return {"o": s["o"], "lse": s["lse"]}


def _own_prompt(s):
    import hierarchical_memory_amd as hm
    case = s["case"]
    hm.hs_attend_prompt(s["sw"].ctx, s["q"], s["kv"], s["latent"][:, case["latent"]:], s["cu_q"], s["cu_k"],
                        s["scale"], s["o"], s["lse"], causal=case["causal"])
    return {"o": s["o"], "lse": s["lse"]}


def _own_store(s):
    import hierarchical_memory_amd as hm
    style = hm.HS_ROPE_HALVES if s["case"]["halves"] else hm.HS_ROPE_PAIRS
    hm.hs_store_rows(s["sw"].ctx, s["fmt"], s["x"], s["weight"], EPS, s["freqs"], s["req"], s["pos"], s["slot"],
                     latent=s["latent"], rope_style=style)
    return _stored(s, s["latent"])


def _own_map(s):
    import hierarchical_memory_amd as hm
    cu, req, pos, slot = s["map"]
    hm.hs_map_tokens(s["sw"].ctx, s["new"], s["old"], s["first"], cu, req, pos, slot, status=s["status"])
    return {"cu": cu, "req": req, "pos": pos, "slot": slot, "status": s["status"]}


def _stored(s, latent):
    """What a store leaves: the bf16 latent rows, and the tail's rows as the numbers that they hold."""
    case, tail = s["case"], s["tail"]
    if case["bits"] == 16:
        return {"latent": latent, "tail": tail.view(torch.bfloat16)}
    values, scales, rope = _parts(tail, case["latent"], case["rope"])
    return {"latent": latent, "values": values, "scales": scales, "rope": rope}


# --- plain forms

def _rows_of(s):
    """The selected rows' bytes, [R, k, bytes]; a row that is not there is any row (its score is masked)."""
    if s["gather"] is not None:
        return s["gather"]
    out, B = s["out"].long(), s["case"]["B"]
    r = torch.arange(out.shape[0], device="cuda")[:, None]
    hot = s["hot"][r, out.clamp(0, B - 1)]
    if s["tail"] is None:
        return hot
    return torch.where((out >= B).unsqueeze(-1), s["tail"][r, (out - B).clamp(min=0)], hot)


def _attend(s):
    case = s["case"]
    kv = _values(_rows_of(s), case, torch.float32)
    there = (s["out"] >= 0).unsqueeze(1)
    score = torch.bmm(s["q"].float(), kv.transpose(1, 2).contiguous()) * s["scale"]
    score = score.masked_fill(~there, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    o = torch.bmm(p / total.masked_fill(total == 0, 1.0), kv[..., :case["latent"]].contiguous())
    return {"o": o.to(torch.bfloat16), "lse": (top + torch.log(total)).squeeze(-1)}


def _padded(x, at, there):
    """[R, L, ...] of the packed x: row `at` where there is one, zeros elsewhere."""
    return x[at.clamp(max=max(0, x.shape[0] - 1))].float() * there.reshape(*there.shape, *[1] * (x.dim() - 1))


def _prompt(s):
    case = s["case"]
    nope, latent = case["nope"], case["latent"]
    q0, k0 = s["cu_q"].long(), s["cu_k"].long()
    nq, nk = q0.diff(), k0.diff()
    i = torch.arange(case["longest"], device="cuda")
    j = torch.arange(case["longest"] + case["past"], device="cuda")
    there_q, there_k = i < nq[:, None], j < nk[:, None]
    q = _padded(s["q"], q0[:-1, None] + i, there_q).transpose(1, 2)                  # [R, heads, Lq, nope + rope]
    kv = _padded(s["kv"], k0[:-1, None] + j, there_k).transpose(1, 2)                # [R, heads, Lk, nope + value]
    rope = _padded(s["latent"][:, latent:], k0[:-1, None] + j, there_k).unsqueeze(1)  # [R, 1, Lk, rope]
    score = torch.matmul(q[..., :nope], kv[..., :nope].transpose(2, 3))
    score += torch.matmul(q[..., nope:], rope.transpose(2, 3))
    score *= s["scale"]
    seen = there_k[:, None, :].expand(-1, i.numel(), -1)
    if case["causal"]:
        seen = seen & (j[None, None, :] <= (nk - nq)[:, None, None] + i[None, :, None])
    score.masked_fill_(~seen.unsqueeze(1), -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp_(score.sub_(top.masked_fill(top == -math.inf, 0.0)))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, kv[..., nope:]) / total.masked_fill(total == 0, 1.0)
    lse = (top + torch.log(total)).squeeze(-1)
    return {"o": o.transpose(1, 2)[there_q].to(torch.bfloat16), "lse": lse.transpose(1, 2)[there_q]}


def _map(new, old, first, N, B, T, H):
    """Token j of request r has position old[r] + j. It goes into row (position mod T) of the tail where the window
    [first, first + T) holds it, and to the host pool (slot -1) before the window."""
    R = new.numel()
    cu = torch.zeros(R + 1, dtype=torch.int64, device=new.device)
    cu[1:] = new.long().cumsum(0)
    cu = cu.clamp(max=N)
    t = torch.arange(N, device=new.device)
    there = t < cu[-1]
    r = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=R - 1)
    x = old.long()[r] + t - cu[r]
    slot = torch.full_like(x, -1)
    if first is not None:
        f = first.long()[r]
        slot = torch.where((x >= f) & (x < f + T), B + x % T, slot)
        bad = (x >= H) | (x >= f + T)
    else:
        bad = x >= H
    bad &= there
    status = torch.zeros(R, dtype=torch.int32, device=new.device).index_add_(0, r, bad.to(torch.int32)).clamp(max=1)
    gone = ~there | bad
    return (cu.to(torch.int32), torch.where(there, r, -1).to(torch.int32), torch.where(gone, -1, x).to(torch.int32),
            torch.where(gone, -1, slot).to(torch.int32), status)


def _rotated(x, pos, freqs, halves, dtype):
    """The pairs of x's last dimension turned by pos * freqs (angles in 64 bits)."""
    turn = pos.double()[:, None] * freqs
    c, sn = torch.cos(turn).to(dtype), torch.sin(turn).to(dtype)
    a, b = (x[:, :x.shape[1] // 2], x[:, x.shape[1] // 2:]) if halves else (x[:, 0::2], x[:, 1::2])
    u, v = a * c - b * sn, a * sn + b * c
    return torch.cat([u, v], 1) if halves else torch.stack([u, v], 2).flatten(1)


def _store(s):
    case = s["case"]
    n = case["latent"]
    there = s["pos"] >= 0
    x = s["x"].float()
    y = x[:, :n] * torch.rsqrt(x[:, :n].square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    r = _rotated(x[:, n:], s["pos"], s["freqs"], case["halves"], torch.float32).to(torch.bfloat16)
    latent = torch.cat([y.to(torch.bfloat16), r], 1)
    rows = latent.view(torch.uint8) if case["bits"] == 16 else _pack8(y, r)
    spare = s["rows"].shape[0] - 1
    s["rows"][torch.where(s["slot"] >= 0, s["req"].long() * case["T"] + s["slot"].long() - 1, spare)] = rows
    return _stored(s, torch.where(there[:, None], latent, torch.zeros_like(latent)))


# --- the least work

def work(case):
    op, R = case["op"], case["R"]
    if op == "attend":
        heads, latent, rope = case["heads"], case["latent"], case["rope"]
        rows = (R - case["empty"]) * case["k"] * (1.0 - case["pad"])
        return {"bytes": rows * _row_bytes(latent, rope, case["bits"]) + 4 * R * case["k"]
                + R * heads * (2 * (latent + rope) + 2 * latent + 4), "flops": 2 * rows * heads * (2 * latent + rope)}
    new = _lengths(case)
    N = sum(new)
    if op == "prompt":
        heads, nope, rope, value = case["heads"], case["nope"], case["rope"], case["value"]
        old = [case["past"] * (i + 1) // R for i in range(R)]
        pairs = sum(n * o + (n * (n + 1) // 2 if case["causal"] else n * n) for n, o in zip(new, old))
        M = N + sum(old)
        return {"bytes": 2 * M * (heads * (nope + value) + rope) + N * heads * (2 * (nope + rope) + 2 * value + 4),
                "flops": 2 * pairs * heads * (nope + rope + value)}
    if op == "store":
        latent, rope = case["latent"], case["rope"]
        return {"bytes": N * (4 * (latent + rope) + _row_bytes(latent, rope, case["bits"]) + 12),
                "flops": N * (5 * latent + 6 * rope)}
    return {"bytes": 4 * (2 * R + (R if case["T"] else 0) + R + 1 + R) + 12 * (N + case["pad"]),
            "flops": 4 * (N + case["pad"])}


# --- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attend":
        return _exact_attend(s)
    if op == "prompt":
        return _exact_prompt(s)
    if op == "store":
        return _exact_store(s)
    return None  # a map's outputs are whole numbers


def _softmax_of(score, v):
    """The weighted values and the logarithm of the sum for scores [n, keys] and values [keys, m]."""
    if score.shape[1] == 0:
        return score.new_zeros(score.shape[0], v.shape[1]), score.new_full((score.shape[0],), -math.inf)
    lse = torch.logsumexp(score, 1)
    return torch.exp(score - lse[:, None]) @ v, lse


def _exact_attend(s):
    case = s["case"]
    o, lse = [], []
    for r in range(case["R"]):
        out = s["out"][r]
        if s["gather"] is not None:
            rows = s["gather"][r][out >= 0]
        else:
            every = s["hot"][r] if s["tail"] is None else torch.cat([s["hot"][r], s["tail"][r]])
            rows = every[out[out >= 0].long()]
        kv = _values(rows, case, torch.float64)
        a, b = _softmax_of(s["q"][r].double() @ kv.T.contiguous() * s["scale"], kv[:, :case["latent"]].contiguous())
        o.append(a)
        lse.append(b)
    return {"o": torch.stack(o), "lse": torch.stack(lse)}


def _exact_prompt(s):
    case = s["case"]
    nope = case["nope"]
    cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
    o = torch.zeros((cu_q[-1], case["heads"], case["value"]), dtype=torch.float64, device="cuda")
    lse = torch.zeros((cu_q[-1], case["heads"]), dtype=torch.float64, device="cuda")
    for q0, q1, k0, k1 in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        rope = s["latent"][k0:k1, case["latent"]:].double()
        for h in range(case["heads"]):
            kv = s["kv"][k0:k1, h].double()
            key = torch.cat([kv[:, :nope], rope], 1).T.contiguous()
            value = kv[:, nope:].contiguous()
            for a in range(q0, q1, 2048):
                b = min(q1, a + 2048)
                score = s["q"][a:b, h].double() @ key * s["scale"]
                if case["causal"]:
                    last = torch.arange(a - q1, b - q1, device="cuda") + (k1 - k0)
                    score.masked_fill_(torch.arange(k1 - k0, device="cuda") > last[:, None], -math.inf)
                o[a:b, h], lse[a:b, h] = _softmax_of(score, value)
    return {"o": o, "lse": lse}


def _exact_store(s):
    """Unrounded values: bf16 and 8-bit outputs are compared with the numbers that they round."""
    case, tail = s["case"], s["tail"]
    n, rope, T = case["latent"], case["rope"], case["T"]
    N = s["x"].shape[0]
    x = s["x"].double()
    y = x[:, :n] / torch.sqrt((x[:, :n] ** 2).sum(1, keepdim=True) / n + EPS) * s["weight"].double()
    angle = s["pos"].double()[:, None] * s["freqs"]
    z = torch.polar(torch.ones_like(angle), angle)
    if case["halves"]:
        w = torch.complex(x[:, n:n + rope // 2], x[:, n + rope // 2:]) * z
        turned = torch.cat([w.real, w.imag], 1)
    else:
        turned = torch.view_as_real(torch.view_as_complex(x[:, n:].reshape(N, -1, 2).contiguous()) * z).reshape(N, rope)
    there = s["pos"] >= 0
    r, row = s["req"][there].long(), s["slot"][there].long() - 1

    def in_tail(v):
        full = torch.zeros((case["R"], T, v.shape[1]), dtype=torch.float64, device="cuda")
        full[r, row] = v[there]
        return full

    latent = torch.cat([y, turned], 1) * there[:, None]
    if case["bits"] == 16:
        return {"latent": latent, "tail": in_tail(latent)}
    top = y.abs().reshape(N, -1, BLOCK).amax(2)
    scale = 2.0 ** torch.ceil(torch.log2(top / 448)).clamp(min=-100)
    values = (y.reshape(N, -1, BLOCK) / scale[:, :, None]).reshape(N, n)
    # rows that no token has: zero bytes, whose scale stands for 2^-127
    scales = in_tail(scale)
    scales[scales == 0] = 2.0 ** -127
    return {"latent": latent, "values": in_tail(values), "scales": scales, "rope": in_tail(turned)}
