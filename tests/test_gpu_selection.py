"""The operators that make a selection on the GPU (heads, key cache, index scores, top-k), against the plain 64-bit models of
tests/selection_ref.py. Bounds count the roundings that the header states; whole numbers are equal."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import hierarchical_memory_amd  # noqa: F401  (raises if the HIP library is missing)
    yield
    torch.cuda.synchronize()


import hierarchical_memory_amd as hm  # noqa: E402
from tests import selection_ref as ref  # noqa: E402

NORMS = {"none": hm.HS_NORM_NONE, "rms": hm.HS_NORM_RMS, "layer": hm.HS_NORM_LAYER}


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _context(R=1, H=8, k=1):
    return hm.SwapIn(hm.config(R, k, k, 0.0, 16, H, 0))


def _cu(t):
    return None if t is None else t.cuda()


def _head_inputs(seed, n, heads, dim, rope, norm, freqs=True, wide=0, std=2.0):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(n, heads * dim + wide, generator=gen) * std).bfloat16()[:, :heads * dim].unflatten(1, (heads, dim))
    w = (1 + 0.2 * torch.randn(dim, generator=gen)).bfloat16() if norm != "none" else None
    b = (0.3 * torch.randn(dim, generator=gen)).bfloat16() if norm == "layer" else None
    f = 10000.0 ** (-2.0 * torch.arange(rope // 2, dtype=torch.float64) / max(rope, 1)) if freqs and rope else None
    pos = torch.randint(0, 1 << 17, (n,), generator=gen, dtype=torch.int32)
    return x, w, b, f, pos


def _run_heads(x, w, b, f, pos, fmt, bits, sw=None):
    """hs_norm_rotate's outputs for x on the GPU: bf16, or (values, scales); outputs are filled with a pattern first."""
    sw = sw or _context()
    x = x.cuda() if not x.is_cuda else x
    n, heads, dim = x.shape
    if bits == 16:
        o = torch.full((n, heads, dim), 77.0, dtype=torch.bfloat16, device="cuda")
        hm.hs_norm_rotate(sw.ctx, fmt, x, _cu(w), _cu(b), _cu(f), _cu(pos), o)
        return o.cpu()
    o = torch.full((n, heads, dim), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((n, heads, dim // 32), 0xA5, dtype=torch.uint8, device="cuda")
    hm.hs_norm_rotate(sw.ctx, fmt, x, _cu(w), _cu(b), _cu(f), _cu(pos), o.view(torch.float8_e4m3fn), scales=s)
    return o.cpu(), s.cpu()


def _check_bf16(got, y, err, what):
    off = (got.double() - y).abs()
    bound = y.abs() * ref.BF16 * 1.001 + err * 1.01 + 1e-40
    assert (off <= bound).all(), f"{what}: worst {float((off / bound).max()):.3g} times the bound"


# ---- heads

HEADS = [(dim, rope, at, norm, halves, bits)
         for i, (dim, rope, at) in enumerate([(32, 32, 0), (64, 64, 0), (64, 32, 32), (96, 32, 64), (128, 64, 0), (128, 64, 64),
                                              (128, 16, 8), (160, 64, 96), (192, 64, 128), (256, 256, 0), (256, 64, 192),
                                              (224, 0, 0)])
         for norm in ("none", "rms", "layer") for halves in (False, True) for bits in (16, 8)
         if (i + len(norm) + halves + bits // 8) % 2 == 0 or dim in (96, 128)]


@pytest.mark.parametrize("dim,rope,at,norm,halves,bits", HEADS)
def test_heads(dim, rope, at, norm, halves, bits):
    n, heads = 23, 5
    x, w, b, f, pos = _head_inputs(dim + rope, n, heads, dim, rope, norm, wide=24)
    pos[3] = -1
    pos[7], pos[8] = 0, 2 ** 31 - 1
    fmt = hm.head_format(dim, rope, at, int(halves), NORMS[norm], 1e-5)
    wide = torch.zeros(n, heads * dim + 24, dtype=torch.bfloat16, device="cuda")  # heads of a wider projection
    xs = wide[:, 8:8 + heads * dim].unflatten(1, (heads, dim))
    xs.copy_(x)
    got = _run_heads(xs, w, b, f, pos, fmt, bits)
    y, err = ref.head(x.double(), norm, w, b, 1e-5, pos, f, at, rope, halves)
    there = pos >= 0
    if bits == 16:
        assert (got[3] == 77).all()
        _check_bf16(got[there], y[there], err[there], "o")
        if norm == "none":  # what is not rotated passes through
            same = torch.ones(dim, dtype=torch.bool)
            same[at:at + rope] = False
            assert torch.equal(got[there][..., same], x[there][..., same])
        return
    o, s = got
    assert (o[3] == 0x5A).all() and (s[3] == 0xA5).all()
    ref.check_quantised(o[there].view(torch.float8_e4m3fn), s[there], y[there], err[there], 8, "o")


@pytest.mark.parametrize("n,heads,dim", [(1, 1, 128), (1, 64, 128), (3, 512, 32), (300, 1, 64), (2, 7, 256), (5000, 16, 192),
                                         (70001, 1, 32), (17, 33, 160)])
@pytest.mark.parametrize("bits", [8, 16])
def test_heads_sizes(n, heads, dim, bits):
    """Every head of every token, one to many: against the same heads computed by themselves (bit for bit), a few of them
    against the model."""
    rope = min(64, dim)
    x, w, b, f, pos = _head_inputs(n, n, heads, dim, rope, "rms")
    fmt = hm.head_format(dim, rope, dim - rope, hm.HS_ROPE_HALVES, hm.HS_NORM_RMS, 1e-6)
    got = _run_heads(x, w, b, f, pos, fmt, bits)
    pick = sorted({0, n // 3, n // 2, n - 1})
    y, err = ref.head(x[pick].double(), "rms", w, b, 1e-6, pos[pick], f, dim - rope, rope, True)
    if bits == 16:
        _check_bf16(got[pick], y, err, "o")
    else:
        ref.check_quantised(got[0][pick].view(torch.float8_e4m3fn), got[1][pick], y, err, 8, "o")
    h = heads - 1
    alone = _run_heads(x[:, h:h + 1].contiguous(), w, b, f, pos, fmt, bits)
    for g, m in zip(got if bits == 8 else (got,), alone if bits == 8 else (alone,)):
        assert torch.equal(g[:, h:h + 1].view(torch.uint8), m.view(torch.uint8))


TURNS = [(dim, rope, at, heads) for dim, rope, at, heads in [
    (128, 128, 0, 3), (192, 192, 0, 1), (192, 128, 64, 5), (256, 192, 64, 2), (256, 256, 0, 1), (224, 128, 32, 70),
    (64, 48, 16, 1), (96, 16, 72, 9), (96, 80, 8, 1), (128, 32, 40, 1), (128, 32, 96, 33), (256, 240, 16, 1), (160, 64, 8, 4),
    (32, 16, 16, 300)]]


@pytest.mark.parametrize("dim,rope,at,heads", TURNS)
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("bits", [8, 16])
def test_heads_turns(dim, rope, at, heads, halves, bits):
    """Rotated parts of every width and place, for one token, a few, and more than a workgroup's."""
    for n in (1, 3, 150):
        x, w, b, f, pos = _head_inputs(dim + rope + n, n, heads, dim, rope, "layer")
        got = _run_heads(x, w, b, f, pos, hm.head_format(dim, rope, at, int(halves), hm.HS_NORM_LAYER, 1e-6), bits)
        y, err = ref.head(x.double(), "layer", w, b, 1e-6, pos, f, at, rope, halves)
        if bits == 16:
            _check_bf16(got, y, err, f"n {n}")
        else:
            ref.check_quantised(got[0].view(torch.float8_e4m3fn), got[1], y, err, 8, f"n {n}")


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("dim,rope,heads", [(256, 256, 1), (256, 240, 1), (256, 256, 2)])
def test_heads_many_turns(dim, rope, heads, halves, bits):
    """Single heads turned whole, for more tokens than leave a workgroup few of them (their turns are its largest share of LDS):
    as in small calls bit for bit, some of them against the model."""
    n = 40_003
    x, w, b, f, pos = _head_inputs(22, n, heads, dim, rope, "layer")
    fmt = hm.head_format(dim, rope, 0, int(halves), hm.HS_NORM_LAYER, 1e-6)
    got = _run_heads(x, w, b, f, pos, fmt, bits)
    got = got if bits == 8 else (got,)
    for t in (0, 20_000, n - 500):
        few = _run_heads(x[t:t + 500], w, b, f, pos[t:t + 500], fmt, bits)
        for g, m in zip(got, few if bits == 8 else (few,)):
            assert torch.equal(g[t:t + 500].view(torch.uint8), m.view(torch.uint8))
    pick = [0, 31, 32, 63, 64, n // 2, n - 2, n - 1]
    y, err = ref.head(x[pick].double(), "layer", w, b, 1e-6, pos[pick], f, 0, rope, halves)
    if bits == 16:
        _check_bf16(got[0][pick], y, err, "o")
    else:
        ref.check_quantised(got[0][pick].view(torch.float8_e4m3fn), got[1][pick], y, err, 8, "o")


def test_heads_past_one_pass():
    """More heads than workgroups take in one pass, values past 4 GiB."""
    n, heads, dim = 1_700_000, 40, 32
    x = torch.zeros(n, heads, dim, dtype=torch.bfloat16, device="cuda")
    pick = [0, 1, n // 2, n - 2, n - 1]
    some, w, _, f, _ = _head_inputs(14, len(pick), heads, dim, 32, "rms")
    x[pick] = some.cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    sw = _context()
    for mode in (0, 1):
        o = torch.zeros(n, heads, dim, dtype=torch.uint8, device="cuda")
        s = torch.zeros(n, heads, 1, dtype=torch.uint8, device="cuda")
        hm.hs_norm_rotate(sw.ctx, hm.head_format(dim, 32, 0, mode, hm.HS_NORM_RMS, 1e-6), x, w.cuda(), None, f.cuda(), pos,
                          o.view(torch.float8_e4m3fn), scales=s)
        y, err = ref.head(some.double(), "rms", w, None, 1e-6, torch.tensor(pick), f, 0, 32, bool(mode))
        ref.check_quantised(o[pick].cpu().view(torch.float8_e4m3fn), s[pick].cpu(), y, err, 8, "o")
        o[pick] = 0  # (the rest are zeros of either sign: a zero times a negative cosine is -0)
        assert int(o.bitwise_and_(0x7F).count_nonzero()) == 0 and int((s == 27).sum()) >= (n - len(pick)) * heads


def test_heads_strides():
    """Tokens and heads of any strides, transposed ones and the columns of a wider row, in and out; a call in place."""
    n, heads, dim = 19, 6, 64
    x, w, b, f, pos = _head_inputs(1, n, heads, dim, 64, "rms")
    fmt = hm.head_format(dim, 64, 0, 0, hm.HS_NORM_RMS, 1e-6)
    want = _run_heads(x, w, b, f, pos, fmt, 16)
    sw = _context()
    args = (_cu(w), _cu(b), _cu(f), _cu(pos))
    by_head = x.cuda().transpose(0, 1).contiguous().transpose(0, 1)      # [heads][n][dim] in memory
    o = torch.zeros(heads, n, dim, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    hm.hs_norm_rotate(sw.ctx, fmt, by_head, *args, o)
    assert torch.equal(o.cpu(), want)
    wide = torch.full((n, heads, 512 + 64), 5.0, dtype=torch.bfloat16, device="cuda")  # the rope columns of absorbed queries
    hm.hs_norm_rotate(sw.ctx, fmt, x.cuda(), *args, wide[:, :, 512:])
    assert torch.equal(wide[:, :, 512:].cpu(), want) and (wide[:, :, :512] == 5).all()
    wide[:, :, 512:] = x.cuda()
    hm.hs_norm_rotate(sw.ctx, fmt, wide[:, :, 512:], *args, wide[:, :, 512:])
    assert torch.equal(wide[:, :, 512:].cpu(), want) and (wide[:, :, :512] == 5).all()
    one = x[:, :1].cuda().expand(n, heads, dim)                         # a head that all share
    hm.hs_norm_rotate(sw.ctx, fmt, one, *args, o)
    assert torch.equal(o.cpu(), want[:, :1].expand(n, heads, dim))
    for bad in (x.cuda()[:, :, ::2], wide[:, :, 4:68]):
        with pytest.raises((ValueError, hm.HiSparseError)):
            hm.hs_norm_rotate(sw.ctx, hm.head_format(bad.shape[2]), bad, None, None, None, None, torch.empty_like(bad))


def test_heads_without_positions():
    x, w, _, _, _ = _head_inputs(2, 9, 4, 128, 0, "rms")
    got = _run_heads(x, w, None, None, None, hm.head_format(128, 64, 0, 0, hm.HS_NORM_RMS, 0.0), 16)
    y, err = ref.head(x.double(), "rms", w, None, 0.0, None, None, 0, 64, False)
    _check_bf16(got, y, err, "o")
    sw, x = _context(), x.cuda()
    f = torch.ones(32, dtype=torch.float64, device="cuda")
    with pytest.raises(hm.HiSparseError, match="pos"):
        hm.hs_norm_rotate(sw.ctx, hm.head_format(128, 64), x, None, None, f, None, torch.empty_like(x))
    hm.hs_norm_rotate(sw.ctx, hm.head_format(128, 64), x[:0], None, None, f, None, x[:0])


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("scale", [2.0 ** -130, 2.0 ** -60, 2.0 ** 62, 2.0 ** 120])
def test_heads_magnitudes(norm, scale):
    """Values whose squares 32 bits lose."""
    x, w, b, f, pos = _head_inputs(3, 6, 3, 128, 64, norm)
    x = (x.double() * scale).bfloat16()
    fmt = hm.head_format(128, 64, 0, 1, NORMS[norm], 0.0)
    y, err = ref.head(x.double(), norm, w, b, 0.0, pos, f, 0, 64, True)
    _check_bf16(_run_heads(x, w, b, f, pos, fmt, 16), y, err + 1e-38, "o")


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("scale", [2.0 ** 20, 2.0 ** 53, 2.0 ** 62])
def test_heads_largest_eps(norm, scale):
    """An eps that the mean of the squares lifts past 32 bits."""
    x, w, b, f, pos = _head_inputs(21, 6, 3, 128, 64, norm)
    x = (x.double() * scale).bfloat16()
    eps = torch.finfo(torch.float32).max
    y, err = ref.head(x.double(), norm, w, None, eps, pos, f, 0, 64, True)
    got = _run_heads(x, w, None, f, pos, hm.head_format(128, 64, 0, 1, NORMS[norm], eps), 16)
    _check_bf16(got, y, err, "o")


@pytest.mark.parametrize("bits", [8, 16])
def test_heads_rows_of_zeros(bits):
    x, w, b, f, pos = _head_inputs(4, 5, 2, 96, 32, "layer")
    x[2] = 0
    got = _run_heads(x, w, None, f, pos, hm.head_format(96, 32, 64, 1, hm.HS_NORM_LAYER, 1e-6), bits)
    if bits == 16:
        assert (got[2] == 0).all()
    else:
        assert (got[0][2] & 0x7F == 0).all() and (got[1][2] == 27).all()


def test_heads_exact_rounding():
    """bf16 inputs that pass without arithmetic: e4m3 values and scales bit for bit, ties and the largest values among them."""
    gen = torch.Generator().manual_seed(5)
    x = (torch.randn(64, 4, 128, generator=gen) * torch.exp2(torch.randint(-90, 90, (64, 4, 1), generator=gen).float())).bfloat16()
    x[0, 0, :32] = torch.tensor([448.0] + [i + 0.5 for i in range(31)])        # ties at several steps
    x[0, 0, 32:64] = torch.tensor([450.0] + [17.0] * 31)                       # just past the largest value
    x[0, 0, 64:96] = torch.tensor([2.0 ** -126] * 32)                          # below the least scale
    x[0, 0, 96:] = 0
    x[0, 1, :32] = torch.tensor([3.3e38] + [1e38] * 31)
    o, s = _run_heads(x, None, None, None, None, hm.head_format(128), 8)
    code, scale = ref.quantise(x.double(), 8)
    assert torch.equal(s, scale) and torch.equal(o, code)


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_heads_not_numbers(value):
    """A block that holds one becomes NaN, and no other."""
    x, _, _, _, _ = _head_inputs(6, 4, 3, 128, 0, "none")
    clean = _run_heads(x, None, None, None, None, hm.head_format(128), 8)
    x[1, 2, 40] = value
    o, s = _run_heads(x, None, None, None, None, hm.head_format(128), 8)
    assert s[1, 2, 1] == 255 and (o[1, 2, 32:64] & 0x7F == 0x7F).all()
    s[1, 2, 1], o[1, 2, 32:64] = clean[1][1, 2, 1], clean[0][1, 2, 32:64]
    assert torch.equal(s, clean[1]) and torch.equal(o, clean[0])
    w = torch.ones(128, dtype=torch.bfloat16)
    y = _run_heads(x, w, None, None, None, hm.head_format(128, norm=hm.HS_NORM_RMS, eps=1e-6), 16)
    assert torch.isnan(y[1, 2]).any() and torch.isfinite(y[0]).all() and torch.isfinite(y[1, :2]).all()


@pytest.mark.parametrize("dim", range(32, 257, 32))
@pytest.mark.parametrize("bits", [8, 16])
def test_layer_norm_of_equal_values(dim, bits):
    """A row of equal values is its own mean: zeros, and the bias behind them, whatever the value and the number of them."""
    v = torch.arange(0x3F80, 0x4000, dtype=torch.int16).view(torch.bfloat16).double()  # every mantissa
    x = torch.cat([v * s for s in (1.0, 512.0, -2.0 ** -9, 2.0 ** 60)]).bfloat16()[:, None, None].expand(-1, 3, dim).contiguous()
    b = (torch.arange(dim) % 7 - 3.0).bfloat16()
    for bias in (None, b):
        fmt = hm.head_format(dim, norm=hm.HS_NORM_LAYER, eps=1e-6)
        got = _run_heads(x, None, bias, None, None, fmt, bits)
        want = torch.zeros(dim) if bias is None else b.float()
        if bits == 16:
            assert torch.equal(got.float(), want.expand(got.shape))
        else:
            assert torch.equal(ref.decode(*got, 8).float(), want.expand(got[0].shape))


@pytest.mark.parametrize("dim", [32, 96, 128, 160, 192, 224, 256])
def test_layer_norm_of_nearly_equal_values(dim):
    """Few values of a row one or two steps of bf16 off the others. The sum is exact in 32 bits (multiples of a step, no more
    than 258 * 256 of them), values less their mean are too but for one rounding, and what is left are the roundings of the norm
    itself: no share for the mean's."""
    gen = torch.Generator().manual_seed(dim)
    n = 400
    m = 128 + torch.arange(n) % 127                                     # the mantissa, steps
    steps = m[:, None, None] + (torch.rand(n, 2, dim, generator=gen) < 3 / dim) * torch.randint(1, 3, (n, 2, dim), generator=gen)
    steps = steps.clamp(max=255)
    x = (steps * 2.0 ** torch.tensor([2, -6])[torch.arange(n) % 2][:, None, None]).bfloat16()
    for eps in (1e-6, 0.0):
        got = _run_heads(x, None, None, None, None, hm.head_format(dim, norm=hm.HS_NORM_LAYER, eps=eps), 16)
        v = x.double()
        there = (steps.amax(-1) > steps.amin(-1)) if eps == 0 else torch.ones(n, 2, dtype=torch.bool)  # (0 / 0)
        eps = float(torch.tensor(eps))  # as 32 bits hold it
        c = v - v.mean(-1, keepdim=True)
        y = c / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
        _check_bf16(got[there], y[there], (y.abs() * (dim + 24) * ref.F32)[there], f"eps {eps}")


# ---- key cache

STORES = [(dim, bits, rope, norm, halves) for dim in (64, 128) for bits in (4, 8) for rope in (0, 32, 64)
          for norm, halves in (("layer", False), ("rms", True), ("none", True))]


@pytest.mark.parametrize("dim,bits,rope,norm,halves", STORES)
def test_store_keys(dim, bits, rope, norm, halves):
    """Keys into their positions, skipped and refused tokens; what no token names stays as it was."""
    n, R, H = 41, 5, 61
    x, w, b, f, _ = _head_inputs(dim + bits, n, 1, dim, rope, norm, wide=32)
    sw = _context(R, H)
    key = hm.key_format(dim, hm.HS_KEY_MXFP8 if bits == 8 else hm.HS_KEY_MXFP4)
    cache = torch.full((hm.hs_key_bytes(sw.cfg, key),), 0xA5, dtype=torch.uint8, device="cuda")
    req = torch.arange(n, dtype=torch.int32) % R
    pos = torch.arange(n, dtype=torch.int32) + 3
    pos[20] = H - 1
    req[30], pos[31] = -1, -1          # skipped
    req[32], pos[33] = R, H            # refused
    status = torch.zeros(R, dtype=torch.int32, device="cuda")
    values = torch.full((n, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    wide = torch.zeros(n, dim + 32, dtype=torch.bfloat16, device="cuda")
    wide[:, 16:16 + dim] = x[:, 0].cuda()
    hm.hs_store_keys(sw.ctx, hm.head_format(dim, rope, 0, int(halves), NORMS[norm], 1e-5), key, wide[:, 16:16 + dim], _cu(w),
                     _cu(b), _cu(f), req.cuda(), pos.cuda(), cache, values=values, status=status)
    codes, scales = (v.cpu() for v in hm.key_parts(sw.cfg, key, cache))
    y, err = ref.head(x.double(), norm, w, b, 1e-5, pos, f, 0, rope, halves)
    there = (req >= 0) & (req < R) & (pos >= 0) & (pos < H)
    r, p = req[there].long(), pos[there].long()
    got = ref.decode(codes[r, p], scales[r, p], bits)
    plain = ref.decode(codes[r, p], torch.full_like(scales[r, p], 127), bits)
    ref.check_quantised(plain, scales[r, p], y[there][:, 0], err[there][:, 0], bits, "key")
    assert torch.equal(values[there.cuda()].cpu().double(), got)
    assert (values[~there.cuda()] == 7).all()
    rest = torch.ones(R, H, dtype=torch.bool)
    rest[r, p] = False
    assert (codes[rest] == 0xA5).all() and (scales[rest] == 0xA5).all()
    assert status.tolist() == [int(i == 33 % R) for i in range(R)]
    end = codes.numel()
    assert (cache[end:-(-end // 256) * 256] == 0xA5).all()


@pytest.mark.parametrize("bits", [4, 8])
def test_store_keys_exact_rounding(bits):
    """Inputs that pass without arithmetic: codes and scales bit for bit, ties among them."""
    gen = torch.Generator().manual_seed(8)
    n, dim = 300, 128
    x = (torch.randn(n, dim, generator=gen) * torch.exp2(torch.randint(-20, 20, (n, 1), generator=gen).float())).bfloat16()
    x[0, :32] = torch.tensor([6.0] + [0.25 * (i - 15) for i in range(31)])
    x[0, 32:64] = torch.tensor([6.03125] + [1.0] * 31)
    x[0, 64:96] = -0.0
    x[1, :32] = torch.tensor([-3.0] + [0.125 * i for i in range(31)])
    sw = _context(1, n)
    key = hm.key_format(dim, hm.HS_KEY_MXFP8 if bits == 8 else hm.HS_KEY_MXFP4)
    cache = sw.key_cache(key)
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    hm.hs_store_keys(sw.ctx, hm.head_format(dim), key, x.cuda(), None, None, None, torch.zeros_like(at), at, cache)
    codes, scales = (v.cpu()[0] for v in hm.key_parts(sw.cfg, key, cache))
    want, scale = ref.quantise(x.double(), bits)
    assert torch.equal(scales, scale)
    assert torch.equal(codes, want)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_store_keys_not_numbers(bits, value):
    sw = _context(1, 4)
    key = hm.key_format(128, hm.HS_KEY_MXFP8 if bits == 8 else hm.HS_KEY_MXFP4)
    cache = sw.key_cache(key)
    x = torch.ones(2, 128, dtype=torch.bfloat16, device="cuda")
    x[1, 70] = value
    values = torch.zeros_like(x)
    hm.hs_store_keys(sw.ctx, hm.head_format(128), key, x, None, None, None, _ints([0, 0]), _ints([0, 1]), cache, values=values)
    _, scales = hm.key_parts(sw.cfg, key, cache)
    assert scales[0, 1].tolist()[2] == 255 and (scales[0, :2].flatten() == 255).sum() == 1
    assert torch.isnan(values[1, 64:96]).all() and torch.isfinite(values[0]).all() and (values[1, :64] == 1).all()


# ---- scores

def _fill_cache(sw, key, gen):
    """Random keys of normal size in the whole cache: (codes, scales) on the CPU."""
    R, H = sw.R, sw.H
    bits = 8 if key.type == hm.HS_KEY_MXFP8 else 4
    y = torch.randn(R, H, key.dim, generator=gen)
    e = torch.randint(120, 132, (R, H, key.dim // 32), generator=gen, dtype=torch.uint8)
    if bits == 8:
        codes = (y * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        c = torch.randint(0, 16, (R, H, key.dim), generator=gen, dtype=torch.uint8)
        codes = c[..., 0::2] | (c[..., 1::2] << 4)
    cache = sw.key_cache(key)
    parts = hm.key_parts(sw.cfg, key, cache)
    parts[0].copy_(codes)
    parts[1].copy_(e)
    return cache, codes, e, bits


def _queries(n, heads, dim, gen):
    q = (torch.randn(n, heads, dim, generator=gen) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    e = torch.randint(118, 130, (n, heads, dim // 32), generator=gen, dtype=torch.uint8)
    return q, e, torch.randn(n, heads, generator=gen)


def _check_scores(sw, key, cache, codes, e, bits, q, qe, w, req, pos, what=""):
    n = q.shape[0]
    scores = torch.full((n, sw.H + 5), 77.0, device="cuda")
    hm.hs_score_keys(sw.ctx, key, cache, q.cuda(), qe.cuda(), w.cuda(), _ints(req), _ints(pos), scores)
    got = scores.cpu()
    qd = ref.decode(q.view(torch.uint8), qe, 8)
    keys = {}
    for t, (r, p) in enumerate(zip(req, pos)):
        if not (0 <= r < sw.R and 0 <= p < sw.H):
            assert (got[t] == 77).all(), f"{what} token {t}: a skipped row was written"
            continue
        if r not in keys:
            keys[r] = ref.decode(codes[r], e[r], bits)
        s, bound = ref.score(qd[t], w[t].double(), keys[r][:p + 1])
        off = (got[t, :p + 1].double() - s).abs()
        assert (off <= bound).all(), f"{what} token {t}: worst {float((off / bound).max()):.3g} times the bound"
        assert (got[t, p + 1:] == 77).all(), f"{what} token {t}: written behind its position"
    return got


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("heads", [1, 7, 16, 17, 32, 33, 50, 64])
def test_scores(dim, bits, heads):
    """Decode tokens with contexts that end everywhere in a tile, tokens of one request side by side, skipped tokens."""
    gen = torch.Generator().manual_seed(heads)
    sw = _context(6, 523)
    key = hm.key_format(dim, hm.HS_KEY_MXFP8 if bits == 8 else hm.HS_KEY_MXFP4)
    cache, codes, e, _ = _fill_cache(sw, key, gen)
    req = [0, 1, 2, 3, 4, 5, 0, 0, 0, 3, -1, 6, 2, 2, 5, 5, 5, 5, 5, 5, 5, 1, 1]
    pos = [0, 522, 31, 32, 63, 64, 65, 66, 67, 255, 5, 5, -1, 523, 127, 128, 129, 130, 131, 132, 256, 300, 200]
    q, qe, w = _queries(len(req), heads, dim, gen)
    _check_scores(sw, key, cache, codes, e, bits, q, qe, w, req, pos)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("R,H,heads,new,old", [
    (1, 4096, 16, [1], [4095]), (3, 3000, 32, [1, 1, 1], [2999, 0, 1500]), (2, 2100, 32, [130, 70], [1800, 5]),
    (5, 700, 20, [3, 0, 9, 1, 33], [600, 10, 0, 699, 100]), (1, 9000, 64, [2], [8900]), (1, 300, 8, [300], [0]),
    (64, 130, 16, [1] * 64, list(range(64, 128)))])
def test_scores_batches(R, H, heads, new, old, bits):
    """Ragged batches through the map: decode steps, drafts, chunks and whole prompts."""
    gen = torch.Generator().manual_seed(R + H)
    sw = _context(R, H)
    key = hm.key_format(128, hm.HS_KEY_MXFP8 if bits == 8 else hm.HS_KEY_MXFP4)
    cache, codes, e, _ = _fill_cache(sw, key, gen)
    n = sum(new) + 3
    cu, req, pos, slot = sw.map_buffers(n)
    hm.hs_map_tokens(sw.ctx, _ints(new), _ints(old), None, cu, req, pos, slot)
    q, qe, w = _queries(n, heads, 128, gen)
    _check_scores(sw, key, cache, codes, e, bits, q, qe, w, req.tolist(), pos.tolist())


@pytest.mark.parametrize("bits", [4, 8])
def test_scores_ranges(bits):
    """Keys and queries of very small and large scales, weights of zero, and scores that are all zero."""
    gen = torch.Generator().manual_seed(3)
    sw = _context(2, 300)
    key = hm.key_format(128, hm.HS_KEY_MXFP8 if bits == 8 else hm.HS_KEY_MXFP4)
    cache, codes, e, _ = _fill_cache(sw, key, gen)
    e = torch.randint(27, 200, e.shape, generator=gen, dtype=torch.uint8)
    hm.key_parts(sw.cfg, key, cache)[1].copy_(e)
    q, qe, w = _queries(4, 20, 128, gen)
    qe[0], qe[1], qe[2] = 60, 27, 165
    w[3] = 0
    _check_scores(sw, key, cache, codes, e, bits, q, qe, w, [0, 1, 0, 1], [299, 299, 298, 250])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dim,heads", [(128, 20), (64, 3), (64, 40)])
@pytest.mark.parametrize("copies", [1, 2])
def test_scores_every_scale(bits, dim, heads, copies):
    """Every scale byte but NaN's, 0 to 254: request b's keys have b, its queries 254 - b, and values that this keeps within
    2^-126 and 2^128, where bf16 holds them exactly. One token for each request, and two (in groups)."""
    gen = torch.Generator().manual_seed(heads + bits)
    R, H = 255, 8
    sw = _context(R, H)
    key = hm.key_format(dim, hm.HS_KEY_MXFP8 if bits == 8 else hm.HS_KEY_MXFP4)

    def codes_of(byte, count, kind):
        grid = ref.grid_of(kind)
        size = grid * 2.0 ** (byte - 127)
        fine = ((size == 0) | ((size >= 2.0 ** -126) & (size < 2.0 ** 128))).nonzero()[:, 0]
        code = fine[torch.randint(len(fine), (count,), generator=gen)]
        return (code + torch.randint(2, (count,), generator=gen) * (128 if kind == 8 else 8)).to(torch.uint8)

    c = torch.stack([codes_of(b, H * dim, bits).view(H, dim) for b in range(R)])
    codes = c if bits == 8 else c[..., 0::2] | (c[..., 1::2] << 4)
    e = torch.arange(R, dtype=torch.uint8)[:, None, None].expand(R, H, dim // 32).contiguous()
    cache = sw.key_cache(key)
    parts = hm.key_parts(sw.cfg, key, cache)
    parts[0].copy_(codes)
    parts[1].copy_(e)
    req = [b for b in range(R) for _ in range(copies)]
    q = torch.stack([codes_of(254 - b, heads * dim, 8).view(heads, dim) for b in req]).view(torch.float8_e4m3fn)
    qe = (254 - torch.tensor(req)).to(torch.uint8)[:, None, None].expand(-1, heads, dim // 32).contiguous()
    w = torch.randn(len(req), heads, generator=gen)
    _check_scores(sw, key, cache, codes, e, bits, q, qe, w, req, [H - 1 - i % 3 for i in range(len(req))])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("heads", [1, 16, 64])
def test_scores_not_numbers(bits, heads):
    """A NaN key makes its own scores NaN and no others; one behind a token's position, of another request, or in a NaN query
    of another token reaches nothing."""
    gen = torch.Generator().manual_seed(4)
    sw = _context(2, 200)
    key = hm.key_format(128, hm.HS_KEY_MXFP8 if bits == 8 else hm.HS_KEY_MXFP4)
    cache, codes, e, _ = _fill_cache(sw, key, gen)
    q, qe, w = _queries(3, heads, 128, gen)
    req, pos = [0, 0, 1], [100, 199, 150]
    clean = _check_scores(sw, key, cache, codes, e, bits, q, qe, w, req, pos)
    parts = hm.key_parts(sw.cfg, key, cache)
    bad = [(0, 40), (0, 101), (0, 150), (1, 151), (1, 60)]
    for r, x in bad:
        parts[1][r, x, 2] = 255
    if bits == 8:
        parts[1][1, 60] = e[1, 60].cuda()
        parts[0][1, 60, 5] = 0x7F
    scores = torch.full((3, 200), 77.0, device="cuda")
    hm.hs_score_keys(sw.ctx, key, cache, q.cuda(), qe.cuda(), w.cuda(), _ints(req), _ints(pos), scores)
    want = clean[:, :200].clone()
    want[0, 40] = want[1, 40] = want[1, 101] = want[1, 150] = want[2, 60] = math.nan
    assert torch.equal(torch.isnan(scores.cpu()), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(scores.cpu(), 5.0), torch.nan_to_num(want, 5.0))
    parts[0].copy_(codes)
    parts[1].copy_(e)
    qe[1, 0, 3] = 255
    hm.hs_score_keys(sw.ctx, key, cache, q.cuda(), qe.cuda(), w.cuda(), _ints(req), _ints(pos), scores)
    assert torch.isnan(scores[1]).all() and torch.equal(scores.cpu()[[0, 2]], clean[[0, 2], :200])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_stored_not_numbers_score_as_such(bits, dim, value):
    """A key stored with a NaN or an infinity, whatever its other values (zeros among them), makes its scores NaN, whatever the
    queries, and is never selected; its neighbours are scored and selected as without it."""
    gen = torch.Generator().manual_seed(dim + bits)
    n, heads, k = 40, 5, 8
    sw = _context(1, n, k)
    key = hm.key_format(dim, hm.HS_KEY_MXFP8 if bits == 8 else hm.HS_KEY_MXFP4)
    x = torch.randn(n, dim, generator=gen).bfloat16()
    bad = {3: 0, 17: dim // 2, 31: dim - 1, 39: 33}
    x[17] = 0
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    q = torch.randn(3, heads, dim, generator=gen).bfloat16()
    q[2] = 0
    q8 = torch.zeros(3, heads, dim, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    qs = torch.zeros(3, heads, dim // 32, dtype=torch.uint8, device="cuda")
    hm.hs_norm_rotate(sw.ctx, hm.head_format(dim), q.cuda(), None, None, None, None, q8, scales=qs)
    w = torch.ones(3, heads, device="cuda")
    got = []
    for with_them in (False, True):
        if with_them:
            for r, i in bad.items():
                x[r, i] = value
        cache = sw.key_cache(key)
        hm.hs_store_keys(sw.ctx, hm.head_format(dim), key, x.cuda(), None, None, None, torch.zeros_like(at), at, cache)
        scores = torch.full((3, n), 77.0, device="cuda")
        hm.hs_score_keys(sw.ctx, key, cache, q8, qs, w, _ints([0] * 3), _ints([n - 1] * 3), scores)
        ids = torch.zeros(3, k, dtype=torch.int32, device="cuda")
        hm.hs_select(sw.ctx, scores, _ints([n - 1] * 3), ids)
        got.append((scores.cpu(), ids.cpu()))
    (clean, _), (scores, ids) = got
    rows = list(bad)
    assert torch.isnan(scores[:, rows]).all()
    rest = [i for i in range(n) if i not in bad]
    assert torch.equal(scores[:, rest], clean[:, rest])
    for t in range(3):
        assert ids[t].tolist() == ref.select(scores[t], k, 0) and not set(ids[t].tolist()) & set(rows)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("heads", [16, 40])
def test_scores_many_tokens(bits, heads):
    """More tokens than are shared out evenly, alone in their groups (a token for each of many requests) and in groups of a
    request, with skipped ones among them."""
    gen = torch.Generator().manual_seed(heads)
    for R, n in ((5000, 5000), (3, 9000)):
        sw = _context(R, 90)
        key = hm.key_format(64, hm.HS_KEY_MXFP8 if bits == 8 else hm.HS_KEY_MXFP4)
        cache, codes, e, _ = _fill_cache(sw, key, gen)
        q, qe, w = _queries(n, heads, 64, gen)
        req = (torch.arange(n) * R // n).int()
        pos = (torch.arange(n) * 7919 % 90).int()
        req[::97], pos[::89] = -1, -1
        scores = torch.full((n, 90), 77.0, device="cuda")
        hm.hs_score_keys(sw.ctx, key, cache, q.cuda(), qe.cuda(), w.cuda(), req.cuda(), pos.cuda(), scores)
        there = (req >= 0) & (pos >= 0)
        assert (scores.cpu()[~there] == 77).all()
        qd, keys = ref.decode(q.view(torch.uint8), qe, 8), ref.decode(codes, e, bits)[req.clamp(min=0).long()]
        dots = torch.relu(qd @ keys.transpose(1, 2))
        want = (w.double().unsqueeze(-1) * dots).sum(1)
        size = (w.double().abs().unsqueeze(-1) * (qd.abs() @ keys.abs().transpose(1, 2))).sum(1)
        seen = there[:, None] & (torch.arange(90) <= pos[:, None])
        off = (scores.cpu().double() - want).abs()
        assert (off <= size * (64 + heads + 4) * ref.F32 * 1.01 + 1e-37)[seen].all()
        assert (scores.cpu()[there[:, None] & ~seen] == 77).all()


def test_scores_short_contexts_of_long_caches():
    """A cache of many positions of which few are filled, garbage (NaN bytes among it) behind them."""
    gen = torch.Generator().manual_seed(6)
    sw = _context(3, 200_000)
    key = hm.key_format(128, hm.HS_KEY_MXFP8)
    cache = torch.full((hm.hs_key_bytes(sw.cfg, key),), 0xFF, dtype=torch.uint8, device="cuda")
    codes = (torch.randn(3, 50, 128, generator=gen) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    e = torch.randint(120, 132, (3, 50, 4), generator=gen, dtype=torch.uint8)
    parts = hm.key_parts(sw.cfg, key, cache)
    parts[0][:, :50] = codes.cuda()
    parts[1][:, :50] = e.cuda()
    q, qe, w = _queries(4, 32, 128, gen)
    _check_scores(sw, key, cache, codes, e, 8, q, qe, w, [2, 0, 1, 2], [49, 0, 31, 12])


def test_scores_repeat():
    """Equal inputs give equal bits, alone and in a batch."""
    gen = torch.Generator().manual_seed(5)
    sw = _context(3, 5000)
    key = hm.key_format(128, hm.HS_KEY_MXFP4)
    cache, *_ = _fill_cache(sw, key, gen)
    q, qe, w = (v.cuda() for v in _queries(40, 32, 128, gen))
    req, pos = _ints([i // 14 for i in range(40)]), _ints([4000 + 7 * i for i in range(40)])
    a, b = (torch.zeros(40, 5000, device="cuda") for _ in range(2))
    for s in (a, b):
        hm.hs_score_keys(sw.ctx, key, cache, q, qe, w, req, pos, s)
    assert torch.equal(a, b)
    for t in (0, 13, 14, 39):
        one = torch.zeros(1, 5000, device="cuda")
        hm.hs_score_keys(sw.ctx, key, cache, q[t:t + 1], qe[t:t + 1], w[t:t + 1], req[t:t + 1], pos[t:t + 1], one)
        assert torch.equal(one[0], a[t])


# ---- select

def _check_select(scores, pos, k, recent=0, cu=None, R=None):
    """scores [n, columns] (CPU) through hs_select, against the model row by row."""
    n, columns = scores.shape
    rows = n if cu is None else R
    sw = _context(max(1, rows), 1, k)
    out = torch.full((rows + 1, k), 77, dtype=torch.int32, device="cuda")
    hm.hs_select(sw.ctx, scores.cuda(), _ints(pos), out[:rows], cu=None if cu is None else _ints(cu), recent=recent,
                 work=sw.select_work(rows, columns))
    got = out.cpu()
    assert (got[rows] == 77).all()
    for r in range(rows):
        t = r if cu is None else cu[r + 1] - 1 if cu[r + 1] > cu[r] and cu[r + 1] - 1 < n else -1
        m = 0 if t < 0 else max(0, min(pos[t] + 1, columns))
        want = ref.select(scores[t, :m] if m else torch.zeros(0), k, recent)
        assert got[r].tolist() == want, f"row {r} ({m} positions)"


LENGTHS = [1, 2, 3, 63, 64, 65, 255, 256, 1000, 1023, 1024, 1025, 4095, 4097, 9000]


@pytest.mark.parametrize("k", [1, 2, 63, 256, 2048, 5000])
@pytest.mark.parametrize("kind", ["normal", "ties", "wide"])
def test_select(k, kind):
    gen = torch.Generator().manual_seed(k)
    columns = 9000
    s = torch.randn(len(LENGTHS), columns, generator=gen)
    if kind == "ties":
        s = (s * 4).round() / 4
    elif kind == "wide":  # every exponent
        s = s * torch.exp2(torch.randint(-140, 120, s.shape, generator=gen).float())
    _check_select(s, [m - 1 for m in LENGTHS], k)
    _check_select(s, [m - 1 for m in LENGTHS], k, recent=min(k, 70))


SHAPES = {
    "equal": lambda m: torch.full((m,), 0.25),
    "zeros of both signs": lambda m: torch.where(torch.arange(m) % 3 == 0, -0.0, 0.0),
    "ascending": lambda m: torch.arange(m).float(),
    "descending": lambda m: -torch.arange(m).float(),
    "two values": lambda m: (torch.arange(m) % 5 == 4).float(),
    "one large": lambda m: torch.where(torch.arange(m) == m // 2, 3e38, 1e-3 * (torch.arange(m) % 97)),
    "one low": lambda m: torch.where(torch.arange(m) == m // 3, -3.4028234e38, torch.sin(torch.arange(m).float())),
    "subnormal": lambda m: (torch.arange(m) * 7919 % 4001).float() * 1e-45,
    "neighbours": lambda m: torch.tensor(1.0).view(torch.int32).add(torch.arange(m, dtype=torch.int32) * 31 % 2003).view(torch.float32),
    "powers": lambda m: torch.exp2((torch.arange(m) * 37 % 250 - 125).float()) * torch.where(torch.arange(m) % 2 == 0, 1.0, -1.0),
    "infinite": lambda m: torch.where(torch.arange(m) % 7 == 0, math.inf, torch.where(torch.arange(m) % 5 == 0, -math.inf, 1.0)),
    "masked": lambda m: torch.full((m,), -math.inf),
    "lowest": lambda m: torch.full((m,), torch.finfo(torch.float32).min),
    "no numbers": lambda m: torch.full((m,), math.nan),
    "some numbers": lambda m: torch.where(torch.arange(m) % 100 == 3, torch.arange(m).float(), math.nan),
    "mostly masked": lambda m: torch.where(torch.arange(m) % 50 == 0, torch.cos(torch.arange(m).float()), -math.inf),
}


@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("columns", [1024, 20000, 100000])
def test_select_distributions(name, columns):
    s = torch.stack([SHAPES[name](columns), SHAPES[name](columns).flip(0), torch.roll(SHAPES[name](columns), 333)])
    pos = [columns - 1, columns - 2, columns // 2]
    for k, recent in ((1, 0), (100, 0), (100, 100), (2048, 3)):
        _check_select(s, pos, k, recent)


@pytest.mark.parametrize("columns,rows", [(40960, 3), (65536, 2), (262144, 2), (1_000_000, 1), (1_000_004, 2)])
@pytest.mark.parametrize("k", [1, 2048, 5000])
def test_select_long(columns, rows, k):
    gen = torch.Generator().manual_seed(columns + k)
    s = torch.randn(rows, columns, generator=gen) * 0.3 + 0.5
    s[0] = s[0].bfloat16().float()
    _check_select(s, [columns - 1 - 777 * r for r in range(rows)], k, recent=1)


def test_select_lengths():
    """No position, fewer than k, positions past the columns, what lies behind a row's end."""
    gen = torch.Generator().manual_seed(9)
    s = torch.randn(8, 512, generator=gen)
    pos = [-1, 0, 5, 99, 511, 512, 2 ** 31 - 1, -2 ** 31]
    for t, p in enumerate(pos):
        s[t, max(0, p + 1):] = [math.inf, math.nan][t % 2]
    _check_select(s, pos, 100)
    _check_select(s, pos, 512, recent=512)
    _check_select(torch.zeros(0, 16), [], 4)
    _check_select(torch.zeros(3, 0), [0, 5, -1], 4)


def test_select_by_request():
    gen = torch.Generator().manual_seed(10)
    s = torch.randn(9, 256, generator=gen)
    pos = [5, 6, 7, 200, 30, -1, 255, 3, 4]
    _check_select(s, pos, 16, 2, cu=[0, 3, 3, 4, 6, 7, 7], R=6)
    _check_select(s, pos, 16, 0, cu=[0, 9, 12, 12], R=3)    # a request that ends past the tokens
    _check_select(s, pos, 16, 0, cu=[0, 0, 0, 0], R=3)
    _check_select(s, pos, 16, 0, cu=[0, 4, 2, 8], R=3)      # descending: not a batch's, no fault


def test_select_many_rows():
    """More rows than a launch takes, each of a few positions."""
    rows, columns, k = (1 << 21) + 5, 8, 2
    gen = torch.Generator().manual_seed(15)
    s = torch.randn(rows, columns, generator=gen)
    pos = (torch.arange(rows) % 9 - 1).int()
    sw = _context(1, 1, k)
    out = torch.full((rows, k), 77, dtype=torch.int32, device="cuda")
    hm.hs_select(sw.ctx, s.cuda(), pos.cuda(), out)
    masked = s.masked_fill(torch.arange(columns) > pos[:, None], -math.inf)
    best, order = masked.sort(dim=1, descending=True, stable=True)
    ids = torch.where(best[:, :k] > -math.inf, order[:, :k], columns).sort(dim=1).values
    assert torch.equal(out.cpu(), torch.where(ids < columns, ids, -1).int())


@pytest.mark.parametrize("columns,k", [(70_000, 2048), (300_000, 2048), (70_000, 5000), (500_000, 2048)])
def test_select_graph_of_long_rows(columns, k):
    """Rows in several launches, captured once and replayed over other scores and lengths."""
    rows = 2
    sw = _context(rows, 1, k)
    s = torch.zeros(rows, columns, device="cuda")
    pos, out = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.zeros(rows, k, dtype=torch.int32, device="cuda")
    work = sw.select_work(rows, columns)
    hm.hs_select(sw.ctx, s, pos, out, recent=3, work=work)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hm.hs_select(sw.ctx, s, pos, out, recent=3, work=work)
    gen = torch.Generator().manual_seed(16)
    for i in range(4):
        x = torch.randn(rows, columns, generator=gen)
        lengths = [columns - 1 - i, [0, 100, columns // 2, -1][i]]
        s.copy_(x)
        pos.copy_(torch.tensor(lengths, dtype=torch.int32))
        work.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        for r in range(rows):
            assert out[r].tolist() == ref.select(x[r, :lengths[r] + 1], k, 3), f"replay {i}, row {r}"


def _long_rows(kind, columns, gen):
    x = torch.randn(columns, generator=gen)
    at = torch.arange(columns)
    if kind == "up":
        return at.float()
    if kind == "down":
        return -at.float()
    if kind == "equal":
        return torch.full((columns,), -2.5)
    if kind == "two":
        return (x > 0).float()
    if kind == "few":  # fewer than are selected
        return torch.where(at % 1000 == 7, x, -math.inf)
    if kind == "nan":
        return torch.where(at % 3 == 0, math.nan, torch.where(at % 7 == 0, -math.inf, x))
    if kind == "infinite":
        return torch.where(at % 31 == 0, math.inf, x)
    if kind == "largest":
        return torch.where(at % 2 == 0, 1.0, -1.0) * torch.finfo(torch.float32).max
    if kind == "one part":
        return torch.where((at >= 40_000) & (at < 47_000), x + 9, x)
    if kind == "ties":
        return x.mul(4).round()
    if kind == "tiny":
        return x * 1e-39
    return x


@pytest.mark.parametrize("kind", ["up", "down", "equal", "two", "few", "nan", "infinite", "largest", "one part", "ties", "tiny",
                                  "normal"])
@pytest.mark.parametrize("columns,k,recent", [(1_000_000, 2048, 64), (420_000, 2048, 0), (210_004, 4096, 4096), (640_000, 1300, 1)])
def test_select_longest(kind, columns, k, recent):
    """Rows whose parts' best do not fit one workgroup, with scores that leave little or most of them to be joined."""
    gen = torch.Generator().manual_seed(columns + k)
    rows = 3
    s = torch.stack([_long_rows(kind, columns, gen) for _ in range(rows)])
    pos = [columns - 1, columns // 3, columns - 4097]
    sw = _context(rows, 1, k)
    out = torch.full((rows, k), 77, dtype=torch.int32, device="cuda")
    work = torch.full((hm.hs_select_work_bytes(sw.cfg, rows, columns) + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    hm.hs_select(sw.ctx, s.cuda(), _ints(pos), out, recent=recent, work=work[:-64])
    assert (work[-64:] == 0xFF).all()
    for r in range(rows):
        assert out[r].tolist() == ref.select(s[r, :pos[r] + 1], k, recent), f"row {r}"


def test_select_longest_empty_rows_and_batches():
    """Rows of no position, of one, of fewer than are selected, and requests' last tokens, in contexts of a million."""
    columns, k = 1_000_000, 2048
    gen = torch.Generator().manual_seed(17)
    s = torch.randn(6, columns, generator=gen)
    sw = _context(5, 1, k)
    dev, work = s.cuda(), sw.select_work(6, columns)
    for pos in ([-1, 0, 5, 2046, 2047, 2048], [16383, 16384, 49151, 49152, -1, 65535]):
        out = torch.full((6, k), 77, dtype=torch.int32, device="cuda")
        hm.hs_select(sw.ctx, dev, _ints(pos), out, recent=2, work=work)
        for r in range(6):
            assert out[r].tolist() == ref.select(s[r, :pos[r] + 1], k, 2), f"row {r}"
    cu, pos = _ints([0, 2, 2, 3, 6, 6]), [9, 700_000, 3, 8, 99, 999_999]
    out = torch.full((5, k), 77, dtype=torch.int32, device="cuda")
    hm.hs_select(sw.ctx, dev, _ints(pos), out, cu=cu, recent=2, work=work)
    for r, t in enumerate([1, None, 2, 5, None]):
        want = [-1] * k if t is None else ref.select(s[t, :pos[t] + 1], k, 2)
        assert out[r].tolist() == want, f"request {r}"


def test_select_more_parts_than_are_joined():
    columns, k = 17_000_000, 2048
    gen = torch.Generator().manual_seed(18)
    s = torch.randn(1, columns, generator=gen)
    sw = _context(1, 1, k)
    out = torch.full((1, k), 77, dtype=torch.int32, device="cuda")
    hm.hs_select(sw.ctx, s.cuda(), _ints([columns - 1]), out, recent=1, work=sw.select_work(1, columns))
    assert out[0].tolist() == ref.select(s[0], k, 1)


def test_select_two_streams():
    """Two calls at once, with a work buffer each."""
    columns, k = 1_000_000, 2048
    gen = torch.Generator().manual_seed(19)
    s = torch.randn(2, 1, columns, generator=gen)
    sw = _context(1, 1, k)
    dev, streams = s.cuda(), [torch.cuda.Stream(), torch.cuda.Stream()]
    out = torch.full((2, 1, k), 77, dtype=torch.int32, device="cuda")
    works = [sw.select_work(1, columns) for _ in range(2)]
    pos = _ints([columns - 1])
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            hm.hs_select(sw.ctx, dev[i], pos, out[i], recent=1, work=works[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert out[i, 0].tolist() == ref.select(s[i, 0], k, 1)


def test_select_random():
    import random
    rng = random.Random(11)
    for seed in range(30):
        gen = torch.Generator().manual_seed(seed)
        columns = 4 * rng.choice([1, 3, 17, 300, 3000, 11000, 20000])
        rows, k = rng.randint(1, 5), rng.choice([1, 3, 100, 777, 2048, 5000])
        s = torch.randn(rows, columns, generator=gen)
        if rng.random() < 0.5:
            s = (s * rng.choice([1, 8, 64])).round()
        s[torch.rand(s.shape, generator=gen) < rng.choice([0, 0.01, 0.9])] = rng.choice([math.nan, -math.inf, math.inf, 0.0])
        _check_select(s, [rng.randint(-1, columns + 3) for _ in range(rows)], k, rng.randint(0, min(k, 40)))


# ---- together

@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("graph", [False, True])
def test_decode_steps(bits, graph):
    """Prompts, then decode steps as a program makes them: queries, key store, scores, selection, swap-in and the fused gather;
    each step's selection is that of the model for the scores, the scores are the model's, and the gathered rows are the
    selected ones. With graph, a step is captured once and replayed."""
    gen = torch.Generator().manual_seed(bits)
    R, H, k, B, heads, dim, rope = 4, 640, 64, 96, 24, 128, 64
    sw = hm.SwapIn(hm.config(R, k, B, 0.0, 32, H, 0))
    pool = sw.host_pool()
    import numpy as np
    pool[:] = np.arange(R * H, dtype=np.uint32).view(np.uint8).reshape(R, H, 4).repeat(8, 2)[:, :, :32]
    key = hm.key_format(dim, hm.HS_KEY_MXFP8 if bits == 8 else hm.HS_KEY_MXFP4)
    cache = sw.key_cache(key)
    freqs = 10000.0 ** (-2.0 * torch.arange(rope // 2, dtype=torch.float64) / rope)
    w, b = (1 + 0.1 * torch.randn(dim, generator=gen)).bfloat16(), (0.1 * torch.randn(dim, generator=gen)).bfloat16()
    qf, kf = hm.head_format(dim, rope, 0, hm.HS_ROPE_PAIRS), hm.head_format(dim, rope, 0, hm.HS_ROPE_PAIRS, hm.HS_NORM_LAYER, 1e-6)
    length = torch.tensor([300, 0, 17, 600], dtype=torch.int32)
    status = torch.zeros(R, dtype=torch.int32, device="cuda")
    fd, wd, bd = freqs.cuda(), w.cuda(), b.cuda()

    def keys_of(new, old, x):
        n = int(sum(new))
        cu, req, pos, slot = sw.map_buffers(n)
        hm.hs_map_tokens(sw.ctx, _ints(new), _ints(old), None, cu, req, pos, slot, status)
        hm.hs_store_keys(sw.ctx, kf, key, x, wd, bd, fd, req, pos, cache, status=status)

    prompt = torch.randn(int(length.sum()), dim, generator=gen).bfloat16()
    keys_of(length.tolist(), [0] * R, prompt.cuda())
    # a decode step's buffers
    new, old = _ints([1] * R), length.cuda()
    cu, req, pos, slot = sw.map_buffers(R)
    xq = torch.zeros(R, heads, dim, dtype=torch.bfloat16, device="cuda")
    xk = torch.zeros(R, dim, dtype=torch.bfloat16, device="cuda")
    weights = torch.zeros(R, heads, device="cuda")
    q = torch.zeros(R, heads, dim, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    qs = torch.zeros(R, heads, dim // 32, dtype=torch.uint8, device="cuda")
    scores = torch.zeros(R, H, device="cuda")
    topk = torch.zeros(R, k, dtype=torch.int32, device="cuda")
    work = sw.select_work(R, H)
    out, miss, st, gathered = sw.outputs(gather=True)

    def step():
        hm.hs_map_tokens(sw.ctx, new, old, None, cu, req, pos, slot, status)
        hm.hs_norm_rotate(sw.ctx, qf, xq, None, None, fd, pos, q, scales=qs)
        hm.hs_store_keys(sw.ctx, kf, key, xk, wd, bd, fd, req, pos, cache)
        hm.hs_score_keys(sw.ctx, key, cache, q, qs, weights, req, pos, scores)
        hm.hs_select(sw.ctx, scores, pos, topk, cu=cu, recent=1, work=work)
        hm.hs_resolve(sw.ctx, topk, None, out, miss, st, gathered)

    replay = step
    if graph:
        step()  # (before the capture: the same step is made again by the first replay, from the same state)
        torch.cuda.synchronize()
        hm.hs_reset(sw.ctx)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        replay = g.replay
    for i in range(5):
        xq.copy_(torch.randn(R, heads, dim, generator=gen).bfloat16())
        xk.copy_(torch.randn(R, dim, generator=gen).bfloat16())
        weights.copy_(torch.randn(R, heads, generator=gen))
        if i == 3:
            new.copy_(torch.tensor([1, 0, 1, 1]))  # an idle request
        replay()
        torch.cuda.synchronize()
        codes, es = (v.cpu() for v in hm.key_parts(sw.cfg, key, cache))
        qd = ref.decode(q.view(torch.uint8), qs, 8)
        reqs, poss = req.tolist(), pos.tolist()
        for t, (r, p) in enumerate(zip(reqs, poss)):
            if r < 0:
                continue
            s, bound = ref.score(qd[t], weights[t].cpu().double(), ref.decode(codes[r, :p + 1], es[r, :p + 1], bits))
            assert ((scores[t, :p + 1].cpu().double() - s).abs() <= bound).all()
            y, err = ref.head(xq[t:t + 1].cpu().double(), "none", None, None, 0, torch.tensor([p]), freqs, 0, rope, False)
            ref.check_quantised(q[t].cpu(), qs[t].cpu(), y[0], err[0], 8, "q")
            want = ref.select(scores[t, :p + 1].cpu(), k, 1)
            assert topk[r].tolist() == want
            rows = np.ascontiguousarray(gathered[r].cpu().numpy()[:, ::8]).view(np.uint32)[:, 0]
            assert [int(v) for v, x in zip(rows, want) if x >= 0] == [r * H + x for x in want if x >= 0]
        if i == 3:
            assert (topk[1] == -1).all()
            new.fill_(1)
            old.sub_(torch.tensor([0, 1, 0, 0], dtype=torch.int32, device="cuda"))
        assert (st == 0).all()
        old.add_(1)


def test_streams():
    """Calls on a side stream, ordered by it alone, by handle and by current stream; the default stream by address 0."""
    gen = torch.Generator().manual_seed(12)
    sw = _context(2, 4096, 64)
    key = hm.key_format(128, hm.HS_KEY_MXFP8)
    cache, *_ = _fill_cache(sw, key, gen)
    q, qe, w = (v.cuda() for v in _queries(2, 16, 128, gen))
    req, pos = _ints([0, 1]), _ints([4095, 3000])
    want = torch.zeros(2, 4096, device="cuda")
    hm.hs_score_keys(sw.ctx, key, cache, q, qe, w, req, pos, want)
    ids = torch.zeros(2, 64, dtype=torch.int32, device="cuda")
    work = sw.select_work(2, 4096)
    hm.hs_select(sw.ctx, want, pos, ids, work=work)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0, None):
        s, t = torch.zeros_like(want), torch.zeros_like(ids)
        torch.cuda.synchronize()
        hm.hs_score_keys(sw.ctx, key, cache, q, qe, w, req, pos, s, stream=stream)
        hm.hs_select(sw.ctx, s, pos, t, work=work, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(s, want) and torch.equal(t, ids)


def test_offsets_past_32_bits():
    """A cache of more than 4 GiB and scores of more than 4 GiB."""
    R, H, dim = 36, 1_000_000, 128
    sw = _context(R, H, 2)
    key = hm.key_format(dim, hm.HS_KEY_MXFP8)
    cache = torch.empty(hm.hs_key_bytes(sw.cfg, key), dtype=torch.uint8, device="cuda")
    assert cache.numel() > 2 ** 32
    gen = torch.Generator().manual_seed(13)
    x = torch.randn(64, dim, generator=gen).bfloat16()
    at = torch.arange(64, dtype=torch.int32)
    pos = torch.cat([at[:32], at[32:] + (H - 64)])
    req = torch.full((64,), R - 1, dtype=torch.int32)
    values = torch.zeros(64, dim, dtype=torch.bfloat16, device="cuda")
    hm.hs_store_keys(sw.ctx, hm.head_format(dim), key, x.cuda(), None, None, None, req.cuda(), pos.cuda(), cache, values=values)
    parts = hm.key_parts(sw.cfg, key, cache)
    code, scale = ref.quantise(x.double(), 8)
    assert torch.equal(parts[0][R - 1, pos.long().cuda()].cpu(), code)
    assert torch.equal(parts[1][R - 1, pos.long().cuda()].cpu(), scale)
    n = 1100
    q, qe, w = _queries(n, 3, dim, gen)
    where = _ints([31] * (n - 1) + [H - 1])
    scores = torch.empty(n, H, device="cuda")
    hm.hs_score_keys(sw.ctx, key, cache, q.cuda(), qe.cuda(), w.cuda(), _ints([R - 1] * n), where, scores)
    qd, keys = ref.decode(q.view(torch.uint8), qe, 8), ref.decode(code, scale, 8)
    for t, cols in ((0, slice(0, 32)), (n - 2, slice(0, 32)), (n - 1, slice(0, 32)), (n - 1, slice(32, 64))):
        s, bound = ref.score(qd[t], w[t].double(), keys[cols])
        got = scores[t, pos[cols].long().cuda()].cpu().double()
        assert ((got - s).abs() <= bound).all()
    scores[n - 1] = 0.0
    scores[n - 1, H - 7] = 3.0
    scores[n - 1, 5] = 2.0
    ids = torch.zeros(n, 2, dtype=torch.int32, device="cuda")
    hm.hs_select(sw.ctx, scores, where, ids, work=sw.select_work(n, H))
    assert ids[n - 1].tolist() == [5, H - 7]


def test_refusals():
    """What the library itself refuses: strides, alignment, sizes, formats, work buffers."""
    sw = _context(2, 64, 4)
    ctx, lib = sw.ctx, hm.lib()
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16, device="cuda")
    flat = torch.zeros(100_000, dtype=torch.uint8, device="cuda")
    f8 = lambda *n: torch.zeros(n, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)  # noqa: E731
    ws, i2 = torch.zeros(2, 3, device="cuda"), _ints([0, 1])

    def refused(msg, call):
        with pytest.raises(hm.HiSparseError, match=msg) as e:
            call()
        assert e.value.code == hm.HS_E_INVALID

    for bad, msg in (((48,), "dim"), ((288,), "dim"), ((0,), "dim"), ((64, 24), "rope"), ((64, 80), "rope"), ((64, -16), "rope"),
                     ((64, 32, 4), "rope_at"), ((64, 32, 40), "rope_at"), ((64, 32, -8), "rope_at"), ((64, 32, 0, 2), "rope_style"),
                     ((64, 32, 0, 0, 3), "norm"), ((64, 32, 0, 0, 1, -1.0), "eps"), ((64, 32, 0, 0, 1, math.inf), "eps"),
                     ((64, 32, 0, 0, 1, math.nan), "eps")):
        y = torch.zeros(1, 1, max(bad[0], 0), dtype=torch.bfloat16, device="cuda")
        refused(msg, lambda: hm.hs_norm_rotate(ctx, hm.head_format(*bad), y, None, None, None, None, y))
    one = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    refused("weight", lambda: hm.hs_norm_rotate(ctx, hm.head_format(64), x, one, None, None, None, x))
    refused("bias", lambda: hm.hs_norm_rotate(ctx, hm.head_format(64, norm=1), x, one, one, None, None, x))
    odd = torch.zeros(65, dtype=torch.bfloat16, device="cuda")[1:]
    refused("aligned", lambda: hm.hs_norm_rotate(ctx, hm.head_format(64, norm=1), x, odd, None, None, None, x))
    wide = torch.zeros(2, 3, 68, dtype=torch.bfloat16, device="cuda")
    refused("strides", lambda: hm.hs_norm_rotate(ctx, hm.head_format(64), wide[..., :64], None, None, None, None, x))
    refused("strides", lambda: hm.hs_norm_rotate(ctx, hm.head_format(64), x, None, None, None, None, wide[..., :64]))
    refused("strides", lambda: hm.hs_norm_rotate(ctx, hm.head_format(64), x, None, None, None, None, x[:, :1].expand(2, 3, 64)))
    refused("aligned", lambda: hm.hs_norm_rotate(ctx, hm.head_format(64), x, None, None, None, None, f8(2, 3, 64),
                                                 scales=flat[1:13].view(2, 3, 2)))
    many = torch.zeros(1, 513, 64, dtype=torch.bfloat16, device="cuda")
    refused("heads", lambda: hm.hs_norm_rotate(ctx, hm.head_format(64), many, None, None, None, None, many))
    key = hm.key_format(64, hm.HS_KEY_MXFP8)
    rows = x[:, 0]
    refused("needs", lambda: hm.hs_store_keys(ctx, hm.head_format(64), key, rows, None, None, None, i2, i2, flat[:2 * 64 * 66 - 1]))
    refused("aligned", lambda: hm.hs_store_keys(ctx, hm.head_format(64), key, rows, None, None, None, i2, i2, flat[8:]))
    refused("dim", lambda: hm.hs_store_keys(ctx, hm.head_format(64), hm.key_format(128), rows, None, None, None, i2, i2, flat))
    refused("x_stride", lambda: hm.hs_store_keys(ctx, hm.head_format(64), key, wide[:, 0, :64].view(2, 64)[:, :64].as_strided(
        (2, 64), (68, 1)), None, None, None, i2, i2, flat))
    s = torch.zeros(2, 64, device="cuda")
    qs = torch.zeros(2, 3, 2, dtype=torch.uint8, device="cuda")
    refused("needs", lambda: hm.hs_score_keys(ctx, key, flat[:100], f8(2, 3, 64), qs, ws, i2, i2, s))
    refused("heads", lambda: hm.hs_score_keys(ctx, key, flat, f8(2, 65, 64), torch.zeros(2, 65, 2, dtype=torch.uint8, device="cuda"),
                                              torch.zeros(2, 65, device="cuda"), i2, i2, s))
    out = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    refused("recent", lambda: hm.hs_select(ctx, s, i2, out, recent=5))
    refused("recent", lambda: hm.hs_select(ctx, s, i2, out, recent=-1))
    refused("multiple of 4", lambda: hm.hs_select(ctx, torch.zeros(2, 63, device="cuda"), i2, out))
    refused("aligned", lambda: hm.hs_select(ctx, torch.zeros(200, device="cuda")[1:129].view(2, 64), i2, out))
    long = torch.zeros(2, 65536, device="cuda")
    refused("work buffer", lambda: hm.hs_select(ctx, long, i2, out))
    refused("work buffer", lambda: hm.hs_select(ctx, long, i2, out, work=flat[:hm.hs_select_work_bytes(sw.cfg, 2, 65536) - 1]))
    assert lib.hs_score_keys(ctx, None, None, 0, None, None, 1, None, None, None, 0, None, 64, None) == hm.HS_E_INVALID


def test_other_devices_and_contexts_are_refused():
    sw = _context(2, 64, 4)
    x = torch.zeros(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="GPU tensor"):
        hm.hs_norm_rotate(sw.ctx, hm.head_format(64), x, None, None, None, None, x.cpu())
    with pytest.raises(ValueError):
        hm.hs_norm_rotate(sw.ctx, hm.head_format(64), x.cpu(), None, None, None, None, x.cpu())
    sw2 = _context(1, 8)
    sw2.close()
    with pytest.raises(hm.HiSparseError):
        hm.hs_norm_rotate(None, hm.head_format(64), x, None, None, None, None, x)


def test_closed_context_is_refused():
    """Through a handle that was kept from before, by every call."""
    sw = _context(2, 64, 4)
    ctx = sw.ctx
    key = hm.key_format(64, hm.HS_KEY_MXFP8)
    cache, work = sw.key_cache(key), sw.select_work(2, 64)
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16, device="cuda")
    q, qs = torch.zeros(2, 3, 64, dtype=torch.uint8, device="cuda"), torch.zeros(2, 3, 2, dtype=torch.uint8, device="cuda")
    w, s, at = torch.zeros(2, 3, device="cuda"), torch.zeros(2, 64, device="cuda"), _ints([0, 1])
    out = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    sw.close()
    for call in (lambda: hm.hs_norm_rotate(ctx, hm.head_format(64), x, None, None, None, None, x),
                 lambda: hm.hs_store_keys(ctx, hm.head_format(64), key, x[:, 0], None, None, None, at, at, cache),
                 lambda: hm.hs_score_keys(ctx, key, cache, q.view(torch.float8_e4m3fn), qs, w, at, at, s),
                 lambda: hm.hs_select(ctx, s, at, out, work=work)):
        with pytest.raises(hm.HiSparseError, match="NULL") as e:
            call()
        assert e.value.code == hm.HS_E_INVALID
