"""The latent-attention operators at the ends of their ranges, on the GPU, against the plain 64-bit models of
tests/latent_ref.py."""
from __future__ import annotations

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
from tests import latent_ref as ref  # noqa: E402
from tests.test_gpu_latent import Attend, _check_row, _cu, _within  # noqa: E402


# ---- store

@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "8bit"])
@pytest.mark.parametrize("unit,eps", [(2.0 ** -133, 0.0), (2.0 ** -133, 2.0 ** -149), (2.0 ** 124, 0.0),
                                      (2.0 ** -50, 0.0), (2.0 ** 50, 1e-6)])
def test_store_norm_at_the_ends_of_bf16(unit, eps, mx):
    """Latent parts so small (bf16's least subnormals) that their root mean square has no inverse in 32 bits, and so large
    that their squares have no place there: rows of about one all the same. Bounds as for ordinary rows."""
    latent, rope, n, T = 512, 64, 6, 8
    sw = hm.SwapIn(hm.config(1, 1, 1, 0.0, ref.row_layout(latent, rope, mx)[2], 100, T))
    gen = torch.Generator().manual_seed(2)
    x = torch.randint(-12, 13, (n, latent + rope), generator=gen).double()
    x[1, 1:latent] = 0.0       # one value alone
    x[1, 0] = 1.0
    x[:, :latent] *= unit
    x = x.bfloat16()
    assert torch.equal(x[0, :latent].double() / unit, (x[0, :latent].double() / unit).round())
    w = (1 + 0.2 * torch.randn(latent, generator=gen)).bfloat16()
    lat = torch.zeros((n, latent + rope), dtype=torch.bfloat16, device="cuda")
    hm.hs_store_rows(sw.ctx, hm.row_format(latent, rope, int(mx)), x.cuda(), w.cuda(), eps, None,
                     torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda"),
                     (1 + torch.arange(n)).to(torch.int32).cuda(), lat)
    for t in range(n):
        _check_row(sw.tail[0, t].cpu(), lat[t].cpu(), x[t], w, eps, t, None, False, latent, rope, mx, f"token {t}")
    sw.close()


# ---- scores of any size

# Queries and keys of small whole numbers: every score is a whole number below 2^24 and so exact in 32 bits, times the power
# of two of its head. What is left is the rounding of a weight's exponent, relative to the exponent: under 40 nats of distance
# (weights below e^-40 are nothing), 40 * 8 half steps of 32 bits.
EXACT_SCORE_ERROR = 40 * 8 * ref.F32_HALF


# A far lse is the maximum times scale and log2 e, and back by ln 2: six roundings (both constants, three products, the sum of the
# logarithm), where attention_bounds counts four (an ordinary score's own error covers the others).
MORE_OF_LSE = 2 * ref.F32_HALF


def _nothing(keys):
    """What weights that end at zero may add: each is below 2^-126 of the largest (the least normal number), the largest is
    part of the sum, and values are 3 at most."""
    return keys * 3 * 2.0 ** -126


def _whole(shape, gen, most=3):
    return torch.randint(-most, most + 1, shape, generator=gen).to(torch.float32).bfloat16()


def _whole_rows(shape, latent, rope, mx, gen):
    v = _whole((*shape, latent + rope), gen)
    if not mx:
        return v.view(torch.uint8)
    s, at, _ = ref.row_layout(latent, rope, True)
    e4m3 = v[..., :latent].float().to(torch.float8_e4m3fn).view(torch.uint8)
    scales = torch.full((*shape, at - s), 127, dtype=torch.uint8)
    return torch.cat([e4m3, scales, v[..., latent:].contiguous().view(torch.uint8)], -1)


def _powers(heads, gen):
    """A power of two for each head, from scores of about one to 2^100, in no order."""
    return torch.exp2((100 * torch.arange(heads) // max(heads - 1, 1))[torch.randperm(heads, generator=gen)].double())


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "8bit"])
@pytest.mark.parametrize("R,k,heads,latent,rope", [(2, 40, 16, 512, 64), (1, 700, 100, 512, 64), (2, 300, 24, 256, 32),
                                                   (200, 90, 60, 512, 64), (180, 57, 128, 512, 64)])
def test_attend_scores_of_any_size(R, k, heads, latent, rope, mx, sign):
    """Heads whose scores reach from about one to 2^107: far ones take the row of the largest score (rows of one score share),
    near ones are as ever."""
    c = Attend(R, k, k + 5, 0, heads, latent, rope, mx, seed=50, pad=0.05)
    gen = torch.Generator().manual_seed(51)
    c.rows = _whole_rows((R, k + 5), latent, rope, mx, gen)
    c.sw.hot.copy_(c.rows)
    c.q = (_whole((R, heads, latent + rope), gen).double() * _powers(heads, gen)[:, None]).bfloat16()
    c.dev["q"] = c.q.cuda()
    c.scale = sign * 2.0 ** -7
    c.run()
    for r in {0, R // 2, R - 1}:
        rows = ref.unpack(c.rows[r][c.out[r][c.out[r] >= 0].long()], latent, rope, mx)
        # (weights over their own sum: beside 2^53 a logarithm would lose that equal scores share)
        s = c.q[r].double() @ rows.T * c.scale
        p, lse = torch.softmax(s, 1), torch.logsumexp(s, 1)
        o, pv = p @ rows[:, :latent], p @ rows[:, :latent].abs()
        bo, bl = ref.attention_bounds(o, lse, pv, torch.full((heads,), EXACT_SCORE_ERROR, dtype=torch.float64), rows.shape[0])
        _within(c.o[r], o, bo + _nothing(rows.shape[0]), f"request {r} o")
        _within(c.lse[r], lse, bl + MORE_OF_LSE * lse.abs(), f"request {r} lse")
    c.close()


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("nope,rope,value", [(64, 32, 64), (128, 64, 128), (192, 64, 256)])
@pytest.mark.parametrize("nq,nk,heads", [([40, 3], [40, 300], 8), ([1], [5000], 4), ([40, 3, 0], [2600, 1400, 900], 2),
                                         ([200], [200], 512), ([130], [4130], 64)])
def test_prompt_scores_of_any_size(nq, nk, heads, nope, rope, value, sign):
    gen = torch.Generator().manual_seed(52)
    sw = hm.SwapIn(hm.config(len(nq), 1, 1, 0.0, 16, 4, 0))
    N, M = sum(nq), sum(nk)
    q = (_whole((N, heads, nope + rope), gen).double() * _powers(heads, gen)[:, None]).bfloat16()
    kv, kr = _whole((M, heads, nope + value), gen), _whole((M, rope), gen)
    o = torch.full((N, heads, value), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((N, heads), 9.0, device="cuda")
    scale = sign * 2.0 ** -6
    cu_q, cu_k = _cu(nq), _cu(nk)
    hm.hs_attend_prompt(sw.ctx, q.cuda(), kv.cuda(), kr.cuda(), cu_q.cuda(), cu_k.cuda(), scale, o, lse)
    for r in range(len(nq)):
        a, b, c, d = int(cu_q[r]), int(cu_q[r + 1]), int(cu_k[r]), int(cu_k[r + 1])
        for h in range(0, heads, max(1, heads // 8)):
            n = d - c
            seen = torch.arange(n)[None, :] <= (n - (b - a)) + torch.arange(b - a)[:, None]
            s = q[a:b, h].double() @ torch.cat([kv[c:d, h, :nope], kr[c:d]], 1).double().T * scale
            s = s.masked_fill(~seen, -torch.inf)
            p, lse_want, v = torch.softmax(s, 1), torch.logsumexp(s, 1), kv[c:d, h, nope:].double()
            bo, bl = ref.attention_bounds(p @ v, lse_want, p @ v.abs(),
                                          torch.full((b - a,), EXACT_SCORE_ERROR, dtype=torch.float64), n)
            _within(o[a:b, h], p @ v, bo + _nothing(n), f"sequence {r} head {h} o")
            _within(lse[a:b, h], lse_want, bl + MORE_OF_LSE * lse_want.abs(), f"sequence {r} head {h} lse")
    sw.close()


# ---- scales

@pytest.mark.parametrize("scale", [0.0, -0.0, 2.0 ** -128, -2.0 ** -133, 2.0 ** -149])
@pytest.mark.parametrize("R,k,heads", [(2, 300, 24), (1, 700, 100), (180, 57, 128)])
def test_attend_scales_that_vanish(R, k, heads, scale):
    """A scale of zero beside scores near the largest number, and subnormal scales that such scores make matter."""
    c = Attend(R, k, k + 5, 0, heads, 512, 64, False, seed=53, pad=0.05)
    gen = torch.Generator().manual_seed(54)
    c.rows = (torch.randn(R, k + 5, 576, generator=gen) * 2.0 ** 58).bfloat16().view(torch.uint8)
    c.sw.hot.copy_(c.rows)
    c.q = (torch.randn(R, heads, 576, generator=gen) * 2.0 ** 60).bfloat16()
    c.dev["q"] = c.q.cuda()
    c.scale = scale
    c.run().check({0, R - 1})
    for refused in (2.0 ** 127, -2.0 ** 127):  # times log2 e past 32 bits
        c.scale = refused
        with pytest.raises(hm.HiSparseError, match="2\\^127"):
            c.run()
    c.close()


@pytest.mark.parametrize("scale", [0.0, -0.0, 2.0 ** -128, -2.0 ** -133, 2.0 ** -149])
@pytest.mark.parametrize("nq,nk,heads", [([40, 3], [40, 300], 8), ([3], [5000], 4), ([200], [200], 512)])
def test_prompt_scales_that_vanish(nq, nk, heads, scale):
    gen = torch.Generator().manual_seed(55)
    sw = hm.SwapIn(hm.config(len(nq), 1, 1, 0.0, 16, 4, 0))
    N, M = sum(nq), sum(nk)
    q = (torch.randn(N, heads, 192, generator=gen) * 2.0 ** 60).bfloat16()
    kv, kr = ((torch.randn(M, *s, generator=gen) * 2.0 ** 58).bfloat16() for s in ((heads, 256), (64,)))
    o = torch.full((N, heads, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((N, heads), 9.0, device="cuda")
    cu_q, cu_k = _cu(nq), _cu(nk)
    hm.hs_attend_prompt(sw.ctx, q.cuda(), kv.cuda(), kr.cuda(), cu_q.cuda(), cu_k.cuda(), scale, o, lse)
    for r in range(len(nq)):
        a, b, c, d = int(cu_q[r]), int(cu_q[r + 1]), int(cu_k[r]), int(cu_k[r + 1])
        for h in range(0, heads, max(1, heads // 8)):
            w = ref.prompt(q[a:b, h].double(), kv[c:d, h].double(), kr[c:d].double(), 128, scale, True)
            _within(o[a:b, h], w[0], w[2], f"sequence {r} head {h} o")
            _within(lse[a:b, h], w[1], w[3], f"sequence {r} head {h} lse")
    sw.close()


# ---- 8-bit rows

def _scaled_rows(R, n, latent, rope, byte, gen):
    """8-bit rows of every e4m3 number (both zeros, subnormals, 448), under one scale byte."""
    numbers = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8)
    s, at, _ = ref.row_layout(latent, rope, True)
    q = numbers[torch.randint(0, len(numbers), (R, n, latent), generator=gen)]
    scales = torch.full((R, n, at - s), byte, dtype=torch.uint8)
    r = torch.randn(R, n, rope, generator=gen).bfloat16().view(torch.uint8)
    return torch.cat([q, scales, r], -1)


@pytest.mark.parametrize("byte", [10, 27, 127, 198, 246])
@pytest.mark.parametrize("latent,rope", [(512, 64), (256, 32)])
@pytest.mark.parametrize("heads", [16, 64, 128])
def test_attend_scale_bytes_are_exact(byte, latent, rope, heads):
    """Attention over one row gives the row: every value of it exactly, at both ends of the range of scales."""
    R = 200 if heads > 16 else 3  # enough that a workgroup takes all heads
    c = Attend(R, 1, 2, 0, heads, latent, rope, True, seed=57)
    c.rows = _scaled_rows(R, 2, latent, rope, byte, torch.Generator().manual_seed(byte))
    c.sw.hot.copy_(c.rows)
    c.q.zero_()
    c.dev["q"] = c.q.cuda()
    c.run()
    rows = ref.unpack(c.rows, latent, rope, True)[torch.arange(R), c.out[:, 0].long(), :latent]
    assert torch.equal(c.o.cpu().double(), rows[:, None].expand(R, heads, latent))
    assert not c.lse.any()
    c.close()


@pytest.mark.parametrize("byte", [10, 198])
@pytest.mark.parametrize("R,k,heads", [(2, 300, 24), (1, 700, 100), (180, 57, 128)])
def test_attend_scale_bytes(byte, R, k, heads):
    """Many rows, whose values reach 2^-126 and 2^80."""
    c = Attend(R, k, k + 5, 0, heads, 512, 64, True, seed=58, pad=0.05)
    gen = torch.Generator().manual_seed(59)
    c.rows = _scaled_rows(R, k + 5, 512, 64, byte, gen)
    c.sw.hot.copy_(c.rows)
    c.q[..., :512] = (torch.randn(R, heads, 512, generator=gen) * 2.0 ** (127 - byte - 7)).bfloat16()
    c.dev["q"] = c.q.cuda()
    c.run().check({0, R - 1}).close()


# ---- streams

def test_prompt_work_buffer_on_the_default_stream_by_address(monkeypatch):
    """The default stream's address is 0: the work buffer is taken on it, not on a stream of torch's pool."""
    nq, nk, heads = [40, 3, 0], [2600, 1400, 900], 2
    assert hm.hs_attend_prompt_work_bytes(3, 43, 4900, heads, 128, 64, 128) > 0
    gen = torch.Generator().manual_seed(56)
    sw = hm.SwapIn(hm.config(3, 1, 1, 0.0, 16, 4, 0))
    q, kv, kr = (torch.randn(*s, generator=gen).bfloat16().cuda() for s in ((43, heads, 192), (4900, heads, 256), (4900, 64)))
    o = [torch.full((43, heads, 128), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cu_q, cu_k = _cu(nq).cuda(), _cu(nk).cuda()
    assert torch.cuda.default_stream().cuda_stream == 0
    taken, empty = [], torch.empty

    def watched(*a, **kw):
        taken.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **kw)

    hm.hs_attend_prompt(sw.ctx, q, kv, kr, cu_q, cu_k, 0.07, o[0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        monkeypatch.setattr(torch, "empty", watched)
        hm.hs_attend_prompt(sw.ctx, q, kv, kr, cu_q, cu_k, 0.07, o[1], stream=0)
        monkeypatch.setattr(torch, "empty", empty)
    torch.cuda.synchronize()
    assert taken == [0]
    assert torch.equal(o[0], o[1])
    sw.close()


# ---- boundaries that no batch has

class Guarded:
    """A tensor inside a larger allocation whose other bytes have to stay as they are."""
    PAD = 1 << 16

    def __init__(self, shape, dtype, fill):
        n = torch.Size(shape).numel() * torch.empty((), dtype=dtype).element_size()
        n += -n % 16
        self.whole = (torch.arange(n + 2 * self.PAD, device="cuda") % 251).to(torch.uint8)
        self.before = self.whole.clone()
        inner = torch.Size(shape).numel() * torch.empty((), dtype=dtype).element_size()
        self.t = self.whole[self.PAD:self.PAD + inner].view(dtype).view(shape)
        self.t.fill_(fill)
        self.inner = inner

    def kept(self):
        a, b = self.PAD, self.PAD + self.inner
        return torch.equal(self.whole[:a], self.before[:a]) and torch.equal(self.whole[b:], self.before[b:])


@pytest.mark.parametrize("nope,rope,value,n_q,n_k,heads", [(128, 64, 128, 66, 60, 2), (128, 64, 128, 60, 5000, 2),
                                                           (192, 32, 256, 60, 5000, 2), (64, 32, 64, 60, 3000, 1),
                                                           (128, 32, 128, 300, 300, 300)])
@pytest.mark.parametrize("fault", ["past the end", "below zero", "descending", "all of them"])
def test_prompt_bad_boundaries_write_only_their_tensors(fault, nope, rope, value, n_q, n_k, heads):
    """Starts out of range or descending: o, lse and the work buffer are written inside only, and where the starts of the
    queries, cut to the tensor, ascend, results are right."""
    big, least = 2**31 - 1, -2**31
    cu_q, cu_k, sound = {
        # (sound: the request whose rows no other names, and its rows and keys)
        "past the end": ([0, 20, 40, big], [0, 30, n_k // 2, big], (1, 20, 40, 30, n_k // 2)),
        "below zero": ([least, 25, 50, 50], [-7, 20, n_k, n_k], (1, 25, 50, 20, n_k)),
        "descending": ([0, 30, 10, 10], [0, n_k, 10, 10], None),
        "all of them": ([-3, big, 5, least], [least, big, least, big], None),
    }[fault]
    gen = torch.Generator().manual_seed(60)
    sw = hm.SwapIn(hm.config(3, 1, 1, 0.0, 16, 4, 0))
    q = torch.randn(n_q, heads, nope + rope, generator=gen).bfloat16()
    kv, kr = torch.randn(n_k, heads, nope + value, generator=gen).bfloat16(), torch.randn(n_k, rope, generator=gen).bfloat16()
    o, lse = Guarded((n_q, heads, value), torch.bfloat16, 9.0), Guarded((n_q, heads), torch.float32, 9.0)
    work = Guarded((hm.hs_attend_prompt_work_bytes(3, n_q, n_k, heads, nope, rope, value),), torch.uint8, 0xFF)
    args = (q.cuda(), kv.cuda(), kr.cuda(), torch.tensor(cu_q, dtype=torch.int32, device="cuda"),
            torch.tensor(cu_k, dtype=torch.int32, device="cuda"), 0.07)
    for causal in (True, False):
        o.t.fill_(9.0)
        lse.t.fill_(9.0)
        hm.hs_attend_prompt(sw.ctx, *args, o.t, lse.t, causal, work=work.t if work.t.numel() else None)
        torch.cuda.synchronize()
        assert o.kept() and lse.kept() and work.kept()
        if sound is None:
            continue
        r, a, b, c, d = sound
        for h in {0, heads - 1}:
            w = ref.prompt(q[a:b, h].double(), kv[c:d, h].double(), kr[c:d].double(), nope, 0.07, causal)
            _within(o.t[a:b, h], w[0], w[2], f"{fault} head {h} o")
            _within(lse.t[a:b, h], w[1], w[3], f"{fault} head {h} lse")
    sw.close()


# ---- large values

@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "8bit"])
@pytest.mark.parametrize("R,k,heads", [(1, 2048, 16), (200, 700, 60), (64, 1500, 128)])
def test_attend_large_values(R, k, heads, mx):
    """Latent values of 2^80 behind scores that rise by less than what moves the maximum (weights up to 2^16)."""
    c = Attend(R, k, k, 0, heads, 512, 64, mx, seed=61)
    gen = torch.Generator().manual_seed(62)
    c.out = torch.arange(k, dtype=torch.int32).repeat(R, 1)
    c.dev["out"] = c.out.cuda()
    v = torch.zeros(k, 576)
    v[:, :512] = torch.where(torch.rand(k, 512, generator=gen) < 0.5, -1.0, 1.0) * 2.0 ** 80
    v[:, 512] = (torch.arange(k) * 10.0 / k).bfloat16().float()
    if mx:
        s, at, _ = ref.row_layout(512, 64, True)
        row = torch.cat([(v[:, :512] * 2.0 ** -80).to(torch.float8_e4m3fn).view(torch.uint8),
                         torch.full((k, at - s), 207, dtype=torch.uint8), v[:, 512:].bfloat16().view(torch.uint8)], -1)
    else:
        row = v.bfloat16().view(torch.uint8)
    c.rows = row.repeat(R, 1, 1)
    c.sw.hot.copy_(c.rows)
    c.q.zero_()
    c.q[..., 512] = 1.0
    c.dev["q"] = c.q.cuda()
    c.scale = 1.0
    c.run().check({0, R - 1}).close()


@pytest.mark.parametrize("nope,value", [(64, 64), (128, 128), (192, 256)])
@pytest.mark.parametrize("nq,nk,heads", [([300], [300], 4), ([3], [5000], 4), ([200], [200], 512)])
def test_prompt_large_values(nq, nk, heads, nope, value):
    gen = torch.Generator().manual_seed(63)
    sw = hm.SwapIn(hm.config(1, 1, 1, 0.0, 16, 4, 0))
    N, M = nq[0], nk[0]
    q = torch.zeros(N, heads, nope + 32).bfloat16()
    q[..., nope] = 1.0
    kr = torch.zeros(M, 32)
    kr[:, 0] = torch.arange(M) * 10.0 / M
    kr = kr.bfloat16()
    kv = torch.zeros(M, heads, nope + value)
    kv[..., nope:] = torch.where(torch.rand(M, heads, value, generator=gen) < 0.5, -1.0, 1.0) * 2.0 ** 80
    kv = kv.bfloat16()
    o = torch.full((N, heads, value), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((N, heads), 9.0, device="cuda")
    hm.hs_attend_prompt(sw.ctx, q.cuda(), kv.cuda(), kr.cuda(), _cu(nq).cuda(), _cu(nk).cuda(), 1.0, o, lse)
    for h in {0, heads - 1}:
        w = ref.prompt(q[:, h].double(), kv[:, h].double(), kr.double(), nope, 1.0, True)
        _within(o[:, h], w[0], w[2], f"head {h} o")
        _within(lse[:, h], w[1], w[3], f"head {h} lse")
    sw.close()
