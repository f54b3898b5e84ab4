"""The latent-attention operators on the GPU, against the plain 64-bit models of tests/latent_ref.py. Bounds count
the roundings that the header states; whole numbers are equal."""
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
from tests import latent_ref as ref  # noqa: E402


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _within(got, want, bound, what):
    got, want = got.detach().double().cpu(), want.double()
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    off = (got - want).abs()
    bad = ~(off <= bound) & ~inf
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} out of bound, worst "
                           f"{float((off / bound.clamp(min=1e-300))[bad].max()):.3g} times")


# ---- map

MAPS = [  # (new, len, tail0, n, B, T, H)
    ([1], [0], [0], 1, 1, 4, 8),
    ([3, 0, 2], [5, 1, 0], [2, 0, 0], 5, 16, 8, 64),
    ([3, 0, 2], [5, 1, 0], None, 9, 16, 0, 64),            # padded, no tail
    ([0, 0, 0, 0], [1, 2, 3, 4], [0, 0, 0, 0], 6, 4, 3, 9),   # no token at all
    ([7, 9, 4], [0, 0, 0], [0, 0, 0], 11, 4, 16, 64),      # cut off inside a request
    ([5, 6], [0, 0], [0, 0], 5, 4, 16, 64),                # cut off at a request's end
    ([4, -3, 2], [0, 7, 1], [0, 0, 0], 8, 4, 16, 64),      # a negative count
    ([6, 6], [60, -2], [50, 0], 12, 4, 16, 64),            # past the host rows, before zero
    ([9, 9], [10, 10], [12, 3], 18, 4, 6, 64),             # before the window, and past its end
    ([2, 2], [2**31 - 2, 2**31 - 1], [0, 0], 4, 4, 8, 64), # positions at the end of 32 bits
    ([3, 3], [0, 4], [-5, 2**31 - 1], 6, 4, 7, 64),        # windows out of range
    ([2**31 - 1, 2**31 - 1, 1], [0, 0, 0], [0, 0, 0], 4100, 4, 5000, 5000),  # counts whose sum passes 32 bits
]


@pytest.mark.parametrize("new,length,tail0,n,B,T,H", MAPS, ids=range(len(MAPS)))
def test_map(new, length, tail0, n, B, T, H):
    _check_map(new, length, tail0, n, B, T, H)


@pytest.mark.parametrize("seed", range(6))
def test_map_random(seed):
    import random
    rng = random.Random(seed)
    R = [1, 37, 700, 2049, 5000, 9000][seed]
    T, H = rng.choice([0, 5, 300]), rng.randint(50, 400)
    new = [rng.choice([0, 0, 1, 1, rng.randint(0, 90)]) for _ in range(R)]
    if seed == 3:  # long runs without a token
        new = [0] * 2000 + [4000] + [0] * 48
    length = [rng.randint(0, H) for _ in range(R)]
    tail0 = [max(0, length[r] + new[r] - T + rng.randint(-3, 3)) for r in range(R)] if T else None
    _check_map(new, length, tail0, max(0, sum(new) + rng.choice([-5, 0, 0, 77])), 9, T, H)


def _check_map(new, length, tail0, n, B, T, H):
    R = len(new)
    sw = hm.SwapIn(hm.config(R, 1, B, 0.0, 16, H, T))
    cu, req, pos, slot = (torch.full((m + 3,), 77, dtype=torch.int32, device="cuda") for m in (R + 1, n, n, n))
    status = torch.full((R,), 77, dtype=torch.int32, device="cuda")
    hm.hs_map_tokens(sw.ctx, _ints(new), _ints(length), None if tail0 is None else _ints(tail0), cu[:R + 1], req[:n],
                     pos[:n], slot[:n], status)
    want = ref.map_tokens(new, length, tail0, n, B, T, H)
    for name, got, w in zip(("cu", "req", "pos", "slot", "status"), (cu, req, pos, slot, status), want):
        assert got[:len(w)].tolist() == w, name
        assert (got[len(w):] == 77).all(), name
    sw.close()


# ---- store

def _store_case(seed, latent, rope, mx, halves, freqs, stride, T, n=40, R=5, past=50):
    gen = torch.Generator().manual_seed(seed)
    sw = hm.SwapIn(hm.config(R, 2, 6, 0.0, ref.row_layout(latent, rope, mx)[2], past + n, T))
    wide = (torch.randn(n, stride, generator=gen) * 2).bfloat16()
    x = wide[:, 8:8 + latent + rope]
    w = (1 + 0.2 * torch.randn(latent, generator=gen)).bfloat16()
    f = 10000.0 ** (-2.0 * torch.arange(rope // 2, dtype=torch.float64) / rope) if freqs else None
    return gen, sw, wide, x, w, f


def _check_row(row, latent_row, x, w, eps, p, f, halves, latent, rope, mx, what):
    """row: bytes of one stored row (CPU) and its bf16 latent row, against the definition."""
    y, z = ref.store_values(x.double(), w.double(), eps, float(p), f, halves, latent)
    # 32-bit arithmetic before the rounding: the mean's sum, root, and products; the angle's rounding to 32 bits
    slack = (latent + 16) * ref.F32_HALF
    turn = 8 * ref.F32_HALF * x[latent:].double().abs().max()
    bz = z.abs() * ref.BF16_HALF * 1.001 + turn + 1e-38
    if f is None:
        bz = torch.zeros_like(z)
    want = torch.cat([y, z])
    bl = torch.cat([y.abs() * (ref.BF16_HALF + slack) * 1.001 + 1e-38, bz])
    _within(latent_row, want, bl, what + " latent")
    s, at, _ = ref.row_layout(latent, rope, mx)
    if not mx:
        assert torch.equal(row.view(torch.bfloat16), latent_row), what
        return
    assert torch.equal(row[at:].view(torch.bfloat16), latent_row[latent:]), what
    top = y.abs().reshape(-1, 32).amax(1)
    e = row[s:s + latent // 32].double() - 127
    scale = torch.exp2(e)
    # the least power of two that keeps the block within 448, but for the 32-bit rounding of its largest value
    assert (top <= 448 * scale * (1 + slack)).all() and (e >= -100).all(), what
    assert ((e == -100) | (top > 224 * scale * (1 - slack))).all(), what
    v = row[:latent].view(torch.float8_e4m3fn).double().reshape(-1, 32) * scale[:, None]
    y = y.reshape(-1, 32)
    _within(v, y, torch.maximum(y.abs() * (ref.E4M3_HALF + slack) * 1.001, scale[:, None] * 2.0 ** -10 * 1.001), what)
    assert (row[s + latent // 32:at] == 0).all(), what


STORES = [(latent, rope, mx, halves, freqs) for latent in (256, 512) for rope in (32, 64) for mx in (False, True)
          for halves, freqs in ((False, True), (True, True), (True, False))]


@pytest.mark.parametrize("latent,rope,mx,halves,freqs", STORES)
def test_store(latent, rope, mx, halves, freqs):
    """Rows into the tail ring and the host pool (and the hot slot of a token that has one), skipped and refused tokens,
    a wide projection's rows; what no token names stays as it was."""
    n, R, T, B, past = 40, 5, 7, 6, 50
    gen, sw, wide, x, w, f = _store_case(1, latent, rope, mx, halves, freqs, 8 + latent + rope + 24, T, n, R, past)
    H, rb = past + n, sw.rb
    req = torch.arange(n, dtype=torch.int32) % R
    pos = torch.arange(n, dtype=torch.int32) + 3
    slot = torch.where(torch.arange(n) < 25, B + pos % T, torch.full((n,), -1)).to(torch.int32)
    slot[:25] = torch.where(torch.arange(25) < 18, -1, slot[:25])  # the last of them keep distinct ring rows
    req[30], pos[31] = -1, -1                 # skipped
    req[32], pos[33], slot[34], slot[35] = R, H, B - 1, B + T  # refused
    sw.hot.fill_(0xA5)
    sw.tail.fill_(0xA5)
    pool = sw.host_pool()
    pool[:] = 0x5A
    sw.page.fill_(-1)
    sw.page[int(req[2]), int(pos[2])] = 4     # a hot slot holds token 2
    epoch0 = sw.epoch.clone()
    status = torch.zeros(R, dtype=torch.int32, device="cuda")
    lat = torch.full((n, latent + rope), 7.0, dtype=torch.bfloat16, device="cuda")
    hm.hs_store_rows(sw.ctx, hm.row_format(latent, rope, int(mx)), wide.cuda()[:, 8:8 + latent + rope], w.cuda(), 1e-5,
                     None if f is None else f.cuda(), req.cuda(), pos.cuda(), slot.cuda(), lat,
                     hm.HS_ROPE_HALVES if halves else hm.HS_ROPE_PAIRS, status)
    torch.cuda.synchronize()
    tail, hot, host, lat = sw.tail.cpu(), sw.hot.cpu(), torch.from_numpy(pool.copy()), lat.cpu()
    named = {"tail": set(), "host": set()}
    for t in range(n):
        if t in (30, 31, 32, 33, 34, 35):
            assert (lat[t] == 7).all()
            continue
        r, p, s = int(req[t]), int(pos[t]), int(slot[t])
        where, key = ("tail", (r, s - B)) if s >= 0 else ("host", (r, p))
        assert key not in named[where]
        named[where].add(key)
        row = (tail if s >= 0 else host)[key]
        _check_row(row, lat[t], x[t], w, 1e-5, p, f, halves, latent, rope, mx, f"token {t}")
    for name, buf, fill in (("tail", tail, 0xA5), ("host", host, 0x5A)):
        for i in range(buf.shape[0]):
            for j in range(buf.shape[1]):
                if (i, j) not in named[name]:
                    assert (buf[i, j] == fill).all(), (name, i, j)
    assert torch.equal(hot[int(req[2]), 4], host[int(req[2]), int(pos[2])])
    hot[int(req[2]), 4] = 0xA5
    assert (hot == 0xA5).all()
    want = torch.zeros(R, dtype=torch.int32)
    for t in (33, 34, 35):
        want[int(req[t])] = hm.HS_STATUS_BAD_ID
    assert torch.equal(status.cpu(), want)
    changed = {int(req[t]) for t in range(n) if int(slot[t]) == -1 and t not in (30, 31, 32, 33)}
    assert {r for r in range(R) if int(sw.epoch[r]) != int(epoch0[r])} == changed
    sw.close()


@pytest.mark.parametrize("mx", [False, True])
def test_store_far_positions(mx):
    """Angles of positions up to 200,000 (a rounded 32-bit angle would be off by hundredths)."""
    latent, rope, n, T = 256, 32, 64, 64
    past = 200_000
    gen, sw, wide, x, w, f = _store_case(3, latent, rope, mx, False, True, latent + rope + 8, T, n, 1, past)
    pos = torch.linspace(past - 20_000, past - 1, n).to(torch.int32)
    slot = (6 + torch.arange(n)).to(torch.int32)
    lat = torch.zeros((n, latent + rope), dtype=torch.bfloat16, device="cuda")
    hm.hs_store_rows(sw.ctx, hm.row_format(latent, rope, int(mx)), wide.cuda()[:, 8:8 + latent + rope], w.cuda(), 0.0,
                     f.cuda(), torch.zeros(n, dtype=torch.int32, device="cuda"), pos.cuda(), slot.cuda(), lat)
    for t in range(n):
        _check_row(sw.tail[0, t].cpu(), lat[t].cpu(), x[t], w, 0.0, int(pos[t]), f, False, latent, rope, mx, f"{t}")
    sw.close()


def test_store_extreme_values():
    """8-bit rows of zeros, of one value far above the rest, at the border between two scales, with NaN and infinity."""
    latent, rope, T, n = 512, 64, 8, 6
    sw = hm.SwapIn(hm.config(1, 1, 1, 0.0, 656, 100, T))
    x = torch.zeros(n, latent + rope, dtype=torch.bfloat16)
    x[1, 5] = 1.0                      # the rest of the block and row is zero
    x[2, :latent] = 1e-30
    x[2, 7] = 1e30
    x[3, :latent] = 448.0              # normed to 1 everywhere
    x[4, :latent], x[4, 9] = 1.0, float("nan")
    x[5, :latent], x[5, 9] = 1.0, float("inf")
    w = torch.ones(latent, dtype=torch.bfloat16)
    lat = torch.zeros((n, latent + rope), dtype=torch.bfloat16, device="cuda")
    hm.hs_store_rows(sw.ctx, hm.row_format(512, 64, hm.HS_ROW_MXFP8), x.cuda(), w.cuda(), 1e-6, None,
                     torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda"),
                     (1 + torch.arange(n)).to(torch.int32).cuda(), lat)
    got = ref.unpack(sw.tail[0, :n], latent, rope, True)
    assert (got[0] == 0).all()
    y1 = 1 / math.sqrt(1 / 512 + 1e-6)
    assert abs(float(got[1, 5]) - y1) <= y1 * ref.E4M3_HALF and (got[1, :5] == 0).all() and (got[1, 6:] == 0).all()
    assert abs(float(got[2, 7]) - math.sqrt(512)) <= math.sqrt(512) * ref.E4M3_HALF * 1.01
    assert (got[3, :latent] == 1).all()  # the norm's 32-bit error does not reach half a step of e4m3
    assert torch.isnan(got[4, :latent]).all()
    assert torch.isnan(got[5, 9]) and (got[5, 10:latent] == 0).all()
    sw.close()


def test_store_nothing():
    sw = hm.SwapIn(hm.config(1, 1, 1, 0.0, 1152, 10, 2))
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    hm.hs_store_rows(sw.ctx, hm.row_format(), torch.zeros(0, 576, dtype=torch.bfloat16, device="cuda"),
                     torch.ones(512, dtype=torch.bfloat16, device="cuda"), 1e-6, None, e, e, e)
    sw.close()


# ---- attend

class Attend:
    """A context whose hot and tail rows are random, a selection over them and its queries."""

    def __init__(self, R, k, B, T, heads, latent, rope, mx, seed=0, pad=0.0, empty=(), gathered=False, qstd=1.0):
        gen = torch.Generator().manual_seed(seed)
        self.latent, self.rope, self.mx, self.heads = latent, rope, mx, heads
        self.fmt = hm.row_format(latent, rope, int(mx))
        self.sw = hm.SwapIn(hm.config(R, k, B, 0.0, hm.hs_row_bytes(self.fmt), 4, T))
        self.rows = ref.random_rows((R, B + T), latent, rope, mx, gen)
        self.sw.hot.copy_(self.rows[:, :B])
        if T:
            self.sw.tail.copy_(self.rows[:, B:])
        self.out = torch.stack([torch.randperm(B + T, generator=gen)[:k] for _ in range(R)]).to(torch.int32)
        self.out[torch.rand(R, k, generator=gen) < pad] = -1
        for r in empty:
            self.out[r] = -1
        self.q = (torch.randn(R, heads, latent + rope, generator=gen) * qstd).bfloat16()
        self.gather = None
        if gathered:  # other rows than the context's, so that the place that was read shows
            self.gather = ref.random_rows((R, k), latent, rope, mx, gen)
        self.scale = (latent + rope) ** -0.5
        self.o = torch.full((R, heads, latent), 9.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((R, heads), 9.0, device="cuda")
        self.work = self.sw.attend_work(self.fmt, heads)
        if self.work is not None:
            self.work.fill_(0xFF)  # NaN everywhere: nothing in it may be read before it is written
        self.dev = {n: getattr(self, n).cuda() if getattr(self, n) is not None else None for n in ("q", "out", "gather")}

    def run(self, stream=None):
        hm.hs_attend(self.sw.ctx, self.fmt, self.dev["q"], self.scale, self.dev["out"], self.o, self.lse,
                     self.dev["gather"], self.work, stream)
        return self

    def want(self, r):
        n = self.rows.shape[1]
        there = (self.out[r] >= 0) & (self.out[r] < n)
        rows = self.gather[r][there] if self.gather is not None else self.rows[r][self.out[r][there].long()]
        rows = ref.unpack(rows, self.latent, self.rope, self.mx)
        return ref.attend(self.q[r].double(), rows, self.latent, self.scale)

    def check(self, requests=None):
        for r in range(self.out.shape[0]) if requests is None else requests:
            o, lse, bo, bl = self.want(r)
            _within(self.o[r], o, bo, f"request {r} o")
            _within(self.lse[r], lse, bl, f"request {r} lse")
        return self

    def close(self):
        self.sw.close()


ATTENDS = [  # (R, k, B, T, heads, pad, empty, gathered)
    (1, 1, 1, 0, 1, 0.0, (), False),
    (2, 2, 2, 1, 3, 0.0, (), False),
    (3, 31, 40, 0, 16, 0.0, (), False),
    (2, 33, 40, 9, 17, 0.2, (), True),
    (3, 64, 64, 0, 32, 0.0, (1,), False),
    (2, 65, 80, 16, 33, 0.5, (), False),
    (5, 129, 150, 0, 64, 0.1, (0, 4), True),
    (1, 700, 701, 50, 100, 0.03, (), False),
    (2, 257, 300, 33, 128, 0.0, (), False),
    (1, 90, 100, 0, 129, 0.1, (), False),
    (1, 40, 50, 4, 300, 0.1, (), False),
    (40, 300, 320, 10, 8, 0.9, (3, 39), False),
    (300, 17, 20, 3, 16, 0.3, (299,), False),
    (1, 2048, 2100, 0, 16, 0.0, (), False),
    # enough requests that a workgroup takes 64, or 128, heads; the last two with selections in parts
    (200, 65, 80, 16, 33, 0.5, (1,), False),
    (200, 90, 100, 0, 64, 0.1, (0, 199), True),
    (180, 57, 70, 5, 100, 0.2, (90,), False),
    (200, 33, 40, 0, 128, 0.0, (), False),
    (150, 65, 80, 9, 129, 0.3, (1,), False),
    (64, 1500, 1510, 7, 60, 0.05, (63,), False),
    (64, 1500, 1510, 0, 128, 0.02, (), False),
]


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "8bit"])
@pytest.mark.parametrize("latent,rope", [(512, 64), (512, 32), (256, 64), (256, 32)])
@pytest.mark.parametrize("R,k,B,T,heads,pad,empty,gathered", ATTENDS)
def test_attend(R, k, B, T, heads, pad, empty, gathered, latent, rope, mx):
    c = Attend(R, k, B, T, heads, latent, rope, mx, seed=k, pad=pad, empty=empty, gathered=gathered)
    c.run().check(range(R) if R <= 5 else {0, 1, R // 2, R - 1, *empty}).close()


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "8bit"])
@pytest.mark.parametrize("k,heads,latent,rope", [(2100, 16, 256, 32), (1100, 64, 512, 64), (1100, 128, 512, 64)])
def test_attend_whole_selections(k, heads, latent, rope, mx):
    """Enough requests that each selection stays in one part, longer than what is listed at a time."""
    c = Attend(256, k, k, 0, heads, latent, rope, mx, seed=heads, pad=0.02)
    assert c.work is None
    c.run().check({0, 100, 255}).close()


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "8bit"])
def test_attend_only_selected_rows_are_read(mx):
    """NaN and infinities in every row that is not selected, and indices outside the row space."""
    c = Attend(3, 70, 90, 20, 20, 512, 64, mx, seed=5, pad=0.1)
    c.out[0, :8] = torch.tensor([110, 111, 2**31 - 1, -2**31, -2, -1, 10**6, 110], dtype=torch.int32)
    c.dev["out"] = c.out.cuda()
    poison = torch.full((c.sw.rb,), 0xFF, dtype=torch.uint8)  # NaN as bf16, e4m3 and scale
    poison[:64] = torch.tensor([0x80, 0x7F] * 32, dtype=torch.uint8)  # infinity as bf16
    for r in range(3):
        used = set(c.out[r].tolist())
        for i in range(110):
            if i not in used:
                (c.sw.hot[r, i] if i < 90 else c.sw.tail[r, i - 90]).copy_(poison)
    c.run().check().close()


def test_attend_padding_of_a_gather_is_not_read():
    c = Attend(2, 50, 60, 0, 16, 512, 64, False, seed=6, pad=0.4, gathered=True)
    c.dev["gather"][(c.out < 0).cuda()] = 0xFF
    c.run().check().close()


def test_attend_nan_and_infinite_queries_stay_in_their_head():
    c = Attend(2, 100, 120, 0, 40, 512, 64, False, seed=7)
    c.dev["q"][0, 3] = float("nan")
    c.dev["q"][1, 39, 5] = float("inf")
    c.run()
    assert torch.isnan(c.o[0, 3]).all() and torch.isnan(c.lse[0, 3])
    assert torch.isnan(c.o[1, 39]).all()
    keep = torch.ones(40, dtype=torch.bool)
    for r, h in ((0, 3), (1, 39)):
        o, lse, bo, bl = c.want(r)
        m = keep.clone()
        m[h] = False
        _within(c.o[r][m.cuda()], o[m], bo[m], "o")
        _within(c.lse[r][m.cuda()], lse[m], bl[m], "lse")
    c.close()


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_attend_scales(scale):
    """Uniform weights, reversed scores, and scores so far apart that most weights vanish."""
    c = Attend(2, 300, 310, 0, 24, 256, 64, False, seed=8, pad=0.1)
    c.scale = scale
    c.run().check().close()


def test_attend_rising_scores():
    """Each row's score is above all before it (the running maximum moves at every tile)."""
    c = Attend(1, 400, 400, 0, 16, 512, 64, False, seed=9)
    up = torch.linspace(-3, 3, 400)
    rows = (torch.randn(400, 576, generator=torch.Generator().manual_seed(1)) * 0.1).bfloat16()
    rows[:, :8] = up[:, None].bfloat16()
    c.rows[0] = rows.view(torch.uint8)
    c.sw.hot.copy_(c.rows)
    c.out[0] = torch.arange(400)
    c.dev["out"] = c.out.cuda()
    c.q[:, :, :8] = 40.0
    c.dev["q"] = c.q.cuda()
    c.run().check().close()


def test_attend_the_same_row_twice_counts_twice():
    c = Attend(1, 64, 70, 0, 16, 512, 64, True, seed=10)
    c.out[0, 1:40] = c.out[0, 0]
    c.dev["out"] = c.out.cuda()
    c.run().check().close()


def test_attend_without_lse_and_equal_bits():
    c = Attend(3, 500, 600, 40, 48, 512, 64, False, seed=11, pad=0.05)
    c.run()
    o = c.o.clone()
    lse = c.lse.clone()
    for _ in range(5):
        c.o.fill_(0)
        c.run()
        assert torch.equal(c.o, o) and torch.equal(c.lse, lse)
    c.o.fill_(0)
    hm.hs_attend(c.sw.ctx, c.fmt, c.dev["q"], c.scale, c.dev["out"], c.o, work=c.work)
    assert torch.equal(c.o, o)
    c.close()


@pytest.mark.parametrize("R,B,T", [(210, 18000, 0), (1, 50, 4_000_000)], ids=["hot", "tail"])
def test_attend_rows_past_4_gib(R, B, T):
    """Rows beyond 32-bit byte offsets: of the whole hot buffer, and of one request's tail."""
    k = 40
    fmt = hm.row_format()
    sw = hm.SwapIn(hm.config(R, k, B, 0.0, 1152, 4, T))
    gen = torch.Generator().manual_seed(12)
    out = (B + T - 1 - 97 * torch.arange(k, dtype=torch.int32)).repeat(R, 1)
    rows = torch.randn(k, 576, generator=gen).bfloat16().view(torch.uint8)
    space = sw.tail if T else sw.hot
    some = {0, R - 2, R - 1} if R > 1 else {0}
    for r in some:
        space[r, out[r].long().cuda() - (B if T else 0)] = rows.cuda()
    q = torch.randn(R, 16, 576, generator=gen).bfloat16()
    o = torch.zeros(R, 16, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(R, 16, device="cuda")
    hm.hs_attend(sw.ctx, fmt, q.cuda(), 0.04, out.cuda(), o, lse, work=sw.attend_work(fmt, 16))
    for r in some:
        w, l, bo, bl = ref.attend(q[r].double(), ref.unpack(rows, 512, 64, False), 512, 0.04)
        _within(o[r], w, bo, f"request {r}")
        _within(lse[r], l, bl, f"request {r}")
    sw.close()


def test_attend_refusals():
    c = Attend(4, 2000, 2000, 0, 16, 512, 64, False, seed=13)
    need = hm.hs_attend_work_bytes(c.sw.cfg, c.fmt, 16)
    if need:
        with pytest.raises(hm.HiSparseError, match="work buffer"):
            hm.hs_attend(c.sw.ctx, c.fmt, c.dev["q"], 1.0, c.dev["out"], c.o)
        with pytest.raises(hm.HiSparseError, match="work buffer"):
            hm.hs_attend(c.sw.ctx, c.fmt, c.dev["q"], 1.0, c.dev["out"], c.o, work=c.work[:need - 16])
    with pytest.raises(hm.HiSparseError, match="finite"):
        hm.hs_attend(c.sw.ctx, c.fmt, c.dev["q"], float("nan"), c.dev["out"], c.o, work=c.work)
    with pytest.raises(hm.HiSparseError, match="656 bytes"):
        hm.hs_attend(c.sw.ctx, hm.row_format(512, 64, hm.HS_ROW_MXFP8), c.dev["q"], 1.0, c.dev["out"], c.o, work=c.work)
    buf = torch.zeros(4 * 16 * 576 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(hm.HiSparseError, match="aligned"):
        hm.hs_attend(c.sw.ctx, c.fmt, buf[4:4 + 4 * 16 * 576].view(4, 16, 576), 1.0, c.dev["out"], c.o, work=c.work)
    with pytest.raises(ValueError, match="contiguous"):
        hm.hs_attend(c.sw.ctx, c.fmt, c.dev["q"].transpose(0, 1).contiguous().transpose(0, 1), 1.0, c.dev["out"], c.o,
                     work=c.work)
    c.close()


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "8bit"])
def test_attend_streams_and_graphs(mx):
    """Two calls on two streams with a work buffer each, then both captured into graphs and replayed between eager
    calls; every result equals the first eager one."""
    cs = [Attend(3, 900, 1000, 20, 20 + 12 * i, 512, 64, mx, seed=20 + i, pad=0.1) for i in range(2)]
    want = []
    for c in cs:
        c.run().check()
        want.append((c.o.clone(), c.lse.clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        for c, s in zip(cs, streams):
            c.run(s)
    torch.cuda.synchronize()
    for c, w in zip(cs, want):
        assert torch.equal(c.o, w[0]) and torch.equal(c.lse, w[1])
    graphs = []
    for c in cs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for i in range(4):
        for c, g in zip(cs, graphs):
            c.o.fill_(3)
            g.replay()
        torch.cuda.synchronize()
        for c, w in zip(cs, want):
            assert torch.equal(c.o, w[0]) and torch.equal(c.lse, w[1]), i
            c.run()
            assert torch.equal(c.o, w[0])
    for c in cs:
        c.close()


# ---- prompt

def _cu(n):
    return torch.tensor([0] + list(n), dtype=torch.int64).cumsum(0).to(torch.int32)


def _prompt_case(nq, nk, heads, nope, rope, value, causal, seed=0, pad=3, qstd=1.0, latent=256, check=True, scale=None):
    gen = torch.Generator().manual_seed(seed)
    R, N, M = len(nq), sum(nq) + pad, sum(nk) + pad
    sw = hm.SwapIn(hm.config(R, 1, 1, 0.0, 16, 4, 0))
    q = (torch.randn(N, heads, nope + rope, generator=gen) * qstd).bfloat16()
    kv = torch.randn(M, heads, nope + value, generator=gen).bfloat16()
    rows = torch.randn(M, latent + rope, generator=gen).bfloat16()
    kv[sum(nk):], rows[sum(nk):] = float("nan"), float("nan")  # keys behind the last sequence
    o = torch.full((N, heads, value), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((N, heads), 9.0, device="cuda")
    scale = (nope + rope) ** -0.5 if scale is None else scale
    cu_q, cu_k = _cu(nq), _cu(nk)
    args = (q.cuda(), kv.cuda(), rows.cuda()[:, latent:], cu_q.cuda(), cu_k.cuda(), scale, o, lse, causal)
    hm.hs_attend_prompt(sw.ctx, *args)
    if check:
        for r in range(R):
            a, b, c, d = int(cu_q[r]), int(cu_q[r + 1]), int(cu_k[r]), int(cu_k[r + 1])
            for h in range(heads):
                w = ref.prompt(q[a:b, h].double(), kv[c:d, h].double(), rows[c:d, latent:].double(), nope, scale, causal)
                _within(o[a:b, h], w[0], w[2], f"sequence {r} head {h} o")
                _within(lse[a:b, h], w[1], w[3], f"sequence {r} head {h} lse")
        assert (o[sum(nq):] == 9).all() and (lse[sum(nq):] == 9).all()  # rows behind the last sequence
    return sw, args


DIMS = [(64, 32, 64), (64, 64, 64), (128, 32, 128), (128, 64, 128), (192, 32, 256), (192, 64, 256)]
PROMPTS = [  # (queries, keys, heads)
    ([1], [1], 1),
    ([3], [3], 2),
    ([31, 33], [31, 33], 1),
    ([64, 0, 65], [64, 0, 65], 2),
    ([127, 1, 129], [127, 1, 129], 1),
    ([5, 1, 40], [100, 300, 41], 3),      # chunks behind a context
    ([20, 7], [11, 0], 2),                # fewer keys than queries: the first queries see none
    ([0, 0, 260], [5, 0, 260], 1),
    ([0], [9], 1),
    ([300], [300], 5),
]


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("nope,rope,value", DIMS)
@pytest.mark.parametrize("nq,nk,heads", PROMPTS, ids=range(len(PROMPTS)))
def test_prompt(nq, nk, heads, nope, rope, value, causal):
    sw, _ = _prompt_case(nq, nk, heads, nope, rope, value, causal, seed=len(nq) + nope)
    sw.close()


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
def test_prompt_scales(scale, causal):
    """Uniform weights, reversed scores, and scores so far apart that most weights vanish and the maximum moves."""
    sw, _ = _prompt_case([150, 70], [150, 300], 2, 128, 64, 128, causal, seed=11, scale=scale)
    sw.close()


@pytest.mark.parametrize("heads", [8, 16])
def test_prompt_long(heads):
    sw, _ = _prompt_case([1500, 700], [1500, 1333], heads, 128, 64, 128, True, seed=4, qstd=2.0)
    sw.close()


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("rope", [32, 64])
@pytest.mark.parametrize("nq,nk,heads", [([200], [200], 512), ([257, 3], [300, 9], 300), ([130], [4130], 64),
                                         ([450, 540], [8400, 7000], 4)])
def test_prompt_many_queries(nq, nk, heads, rope, causal):
    """Enough of them for 256 queries to a workgroup, with 128 values; the keys of the last two in parts."""
    sw, _ = _prompt_case(nq, nk, heads, 128, rope, 128, causal, seed=heads)
    sw.close()


@pytest.mark.parametrize("nope,rope,value", DIMS)
@pytest.mark.parametrize("nq,nk,heads,causal", [([1], [5000], 1, True), ([40, 3, 0], [2600, 1400, 900], 2, True),
                                                ([7, 90], [4000, 10], 1, False), ([130], [3333], 4, True)])
def test_prompt_keys_in_parts(nq, nk, heads, causal, nope, rope, value):
    """Few queries over many keys: each tile's keys are cut into parts and joined, some of them without a key."""
    pad = 2
    assert hm.hs_attend_prompt_work_bytes(len(nq), sum(nq) + pad, sum(nk) + pad, heads, nope, rope, value) > 0
    sw, args = _prompt_case(nq, nk, heads, nope, rope, value, causal, seed=sum(nk), pad=pad)
    o, lse = args[6].clone(), args[7].clone()
    n = hm.hs_attend_prompt_work_bytes(len(nq), args[0].shape[0], args[1].shape[0], heads, nope, rope, value)
    work = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    for stream in (None, torch.cuda.Stream()):
        args[6].fill_(9)
        torch.cuda.synchronize()
        hm.hs_attend_prompt(sw.ctx, *args, work=work, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(args[6], o) and torch.equal(args[7], lse)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):  # the work buffer is taken on the call's stream
        args[6].fill_(9)
        torch.cuda.synchronize()
        hm.hs_attend_prompt(sw.ctx, *args, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(args[6], o)
    with pytest.raises(hm.HiSparseError, match="work buffer"):
        hm.hs_attend_prompt(sw.ctx, *args, work=work[:n - 16])
    sw.close()


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("nope,rope,value", DIMS)
@pytest.mark.parametrize("nq,nk,heads", [([70, 300], [70, 300], 2), ([5, 40], [300, 77], 2), ([30], [2600], 2),
                                         ([200], [200], 512), ([130], [4130], 64)])
def test_prompt_values_that_are_no_numbers(nq, nk, heads, nope, rope, value, causal):
    """An infinite value or a NaN reaches the queries that see its key, in its place, and nothing else."""
    sw, args = _prompt_case(nq, nk, heads, nope, rope, value, causal, seed=value, check=False)
    q, kv, rows, _, _, scale, o, lse, _ = args
    keys = []  # (sequence, key of it, head, place, what is there)
    for r in range(len(nq)):
        last = nk[r] - 1
        keys += [(r, last, 0, 1, math.nan), (r, last - 3, 1, value - 1, math.inf), (r, last - nq[r] // 2, 0, 5, -math.inf),
                 (r, max(last - nq[r] + 2, 0), 1, 37, math.nan)]
    starts = _cu(nk)
    clean = kv.cpu().double()
    for r, key, h, place, what in keys:
        kv[int(starts[r]) + key, h, nope + place] = what
        clean[int(starts[r]) + key, h, nope + place] = 0.0
    hm.hs_attend_prompt(sw.ctx, *args)
    for r in range(len(nq)):
        a, b, c, d = int(_cu(nq)[r]), int(_cu(nq)[r + 1]), int(starts[r]), int(starts[r + 1])
        for h in range(min(heads, 3)):
            w = ref.prompt(q[a:b, h].cpu().double(), clean[c:d, h], rows[c:d].cpu().double(), nope, scale, causal)
            got = o[a:b, h].clone()
            for rr, key, hh, place, _ in keys:
                if (rr, hh) == (r, h):
                    first = max(0, key - (nk[r] - nq[r])) if causal else 0
                    assert not got[first:, place].isfinite().any(), (r, h, key, place)
                    got[first:, place], w[0][first:, place] = 0.0, 0.0
            _within(got, w[0], w[2], f"sequence {r} head {h} o")
            _within(lse[a:b, h], w[1], w[3], f"sequence {r} head {h} lse")


@pytest.mark.parametrize("nq,nk", [([1, 40], [66000, 70]), ([90000, 40], [1, 70])], ids=["keys", "queries"])
def test_prompt_offsets_past_4_gib(nq, nk):
    heads, nope, rope, value = 128, 128, 64, 128
    sw = hm.SwapIn(hm.config(2, 1, 1, 0.0, 16, 4, 0))
    gen = torch.Generator().manual_seed(40)
    q = torch.zeros(sum(nq), heads, nope + rope, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(sum(nk), heads, nope + value, dtype=torch.bfloat16, device="cuda")
    kr = torch.zeros(sum(nk), rope, dtype=torch.bfloat16, device="cuda")
    o = torch.full((sum(nq), heads, value), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((sum(nq), heads), 9.0, device="cuda")
    assert max(q.numel(), kv.numel()) * 2 > 1 << 32
    last_q, last_kv, last_kr = (torch.randn(n, *x.shape[1:], generator=gen).bfloat16()
                                for n, x in ((nq[1], q), (nk[1], kv), (nk[1], kr)))
    q[nq[0]:], kv[nk[0]:], kr[nk[0]:] = last_q.cuda(), last_kv.cuda(), last_kr.cuda()
    hm.hs_attend_prompt(sw.ctx, q, kv, kr, _cu(nq).cuda(), _cu(nk).cuda(), 0.07, o, lse)
    for h in (0, 63, 127):
        w = ref.prompt(last_q[:, h].double(), last_kv[:, h].double(), last_kr.double(), nope, 0.07, True)
        _within(o[nq[0]:, h], w[0], w[2], f"head {h} o")
        _within(lse[nq[0]:, h], w[1], w[3], f"head {h} lse")
    assert not o[:nq[0]].any()  # no key, or keys of zeros
    sw.close()


def test_prompt_many_sequences():
    n = [(7 * i) % 23 for i in range(700)]
    sw, _ = _prompt_case(n, [m + i % 3 for i, m in enumerate(n)], 2, 64, 32, 64, True, seed=5)
    sw.close()


def test_prompt_bad_boundaries_stay_inside():
    """Boundaries out of range or descending: nothing outside the tensors is touched, and the rows that only a good
    sequence names (the first `alone`: the others lie in two sequences at once) are computed."""
    sw, args = _prompt_case([10, 20, 30], [10, 20, 30], 2, 128, 64, 128, True, seed=6, check=False)
    q, kv, rope, cu_q, cu_k, scale, o, lse, causal = args
    good_o, good_l = o.clone(), lse.clone()
    for alone, bad_q, bad_k in ((5, [0, 10, 5, 10**9], [0, 10, 5, 10**9]), (0, [0, 10, -7, 63], [0, 10, 2**31 - 1, -5]),
                                (10, [-3, 10, 30, 2**31 - 1], [-2**31, 10, 30, 60])):
        o.fill_(9)
        hm.hs_attend_prompt(sw.ctx, q, kv[:60], rope[:60], _ints(bad_q), _ints(bad_k), scale, o, lse, causal)
        torch.cuda.synchronize()
        assert torch.equal(o[:alone], good_o[:alone]) and torch.equal(lse[:alone], good_l[:alone])
    sw.close()


def test_prompt_nothing():
    for nq, nk in (([0, 0], [0, 0]), ([0, 0], [4, 5]), ([4, 2], [0, 0])):
        sw, _ = _prompt_case(nq, nk, 2, 128, 64, 128, True, pad=0)
        sw.close()


def test_prompt_graph_and_equal_bits():
    sw, args = _prompt_case([200, 90, 333], [300, 90, 333], 4, 128, 64, 128, True, seed=8)
    o, lse = args[6], args[7]
    n = 200 + 90 + 333  # the rows behind the last sequence hold what was there before the call
    want = o[:n].clone(), lse[:n].clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hm.hs_attend_prompt(sw.ctx, *args)
    for _ in range(3):
        o.fill_(1)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o[:n], want[0]) and torch.equal(lse[:n], want[1])
        hm.hs_attend_prompt(sw.ctx, *args)
        assert torch.equal(o[:n], want[0])
    sw.close()


def test_prompt_refusals():
    sw, args = _prompt_case([4], [4], 2, 128, 64, 128, True)
    q, kv, rope, cu_q, cu_k, scale, o, lse, causal = args
    with pytest.raises(hm.HiSparseError, match="finite"):
        hm.hs_attend_prompt(sw.ctx, q, kv, rope, cu_q, cu_k, float("inf"), o, lse)
    with pytest.raises(hm.HiSparseError, match="rope must be"):
        hm.hs_attend_prompt(sw.ctx, q[..., :144].contiguous(), kv, rope[:, :16], cu_q, cu_k, scale, o, lse)
    with pytest.raises(hm.HiSparseError, match="nope, value"):
        hm.hs_attend_prompt(sw.ctx, q, kv[..., :192].contiguous(), rope, cu_q, cu_k, scale, o[..., :64].contiguous(), lse)
    odd = torch.zeros(kv.shape[0], 64 + 5, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(hm.HiSparseError, match="rope_stride"):
        hm.hs_attend_prompt(sw.ctx, q, kv, odd[:, :64], cu_q, cu_k, scale, o, lse)
    with pytest.raises(ValueError, match="contiguous"):
        hm.hs_attend_prompt(sw.ctx, q[..., ::1].transpose(0, 1).contiguous().transpose(0, 1), kv, rope, cu_q, cu_k, scale,
                            o, lse)
    sw.close()


# ---- together

@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "8bit"])
def test_prompt_and_decode_steps_together(mx):
    """A prompt's tokens are mapped, stored (the older ones in the host pool, the last ones in the device tail) and
    attended over; then decode steps store one token each, resolve a selection (misses fetched from the pool), and
    attend over it through the slots, and through a trial's gathered rows. The model holds every token's row as stored."""
    R, k, B, T, H, heads, latent, rope = 3, 24, 32, 16, 120, 5, 512, 64
    nope = value = 128
    fmt = hm.row_format(latent, rope, int(mx))
    gen = torch.Generator().manual_seed(30)
    sw = hm.SwapIn(hm.config(R, k, B, 0.0, hm.hs_row_bytes(fmt), H, T))
    w = (1 + 0.1 * torch.randn(latent, generator=gen)).bfloat16().cuda()
    f = (10000.0 ** (-2.0 * torch.arange(rope // 2, dtype=torch.float64) / rope)).cuda()
    lens = [50, 9, 70]
    N = sum(lens) + 6
    new, length = _ints(lens), _ints([0] * R)
    tail0 = _ints([max(0, n - T + 4) for n in lens])
    cu, req, pos, slot = sw.map_buffers(N)
    status = torch.zeros(R, dtype=torch.int32, device="cuda")
    hm.hs_map_tokens(sw.ctx, new, length, tail0, cu, req, pos, slot, status)
    x = torch.randn(N, latent + rope, generator=gen).bfloat16().cuda()
    lat = torch.zeros(N, latent + rope, dtype=torch.bfloat16, device="cuda")
    hm.hs_store_rows(sw.ctx, fmt, x, w, 1e-6, f, req, pos, slot, lat, status=status)
    assert status.tolist() == [0] * R and cu.tolist() == _cu(lens).tolist()
    # the prompt's attention: keys and values expanded from the latent rows
    up = (torch.randn(latent, heads * (nope + value), generator=gen) * latent ** -0.5).bfloat16().cuda()
    kv = (lat[:, :latent] @ up).view(N, heads, nope + value)
    q = torch.randn(N, heads, nope + rope, generator=gen).bfloat16().cuda()
    o = torch.zeros(N, heads, value, dtype=torch.bfloat16, device="cuda")
    hm.hs_attend_prompt(sw.ctx, q, kv, lat[:, latent:], cu, cu, 0.07, o)
    for r in range(R):
        a, b = int(cu[r]), int(cu[r + 1])
        for h in range(heads):
            want = ref.prompt(q[a:b, h].double().cpu(), kv[a:b, h].double().cpu(), lat[a:b, latent:].double().cpu(),
                              nope, 0.07, True)
            _within(o[a:b, h], want[0], want[2], f"prompt {r} {h}")
    # every token's row as it was stored, by request and position
    torch.cuda.synchronize()
    pool = torch.from_numpy(sw.host_pool())

    def stored(r, p):
        return (sw.tail[r, p % T].cpu() if p >= int(tail0[r]) else pool[r, p].clone())

    out, miss, status, gathered = sw.outputs(gather=True)
    qd = torch.zeros(R, heads, latent + rope, dtype=torch.bfloat16, device="cuda")
    od = torch.zeros(R, heads, latent, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(R, heads, device="cuda")
    work = sw.attend_work(fmt, heads)
    trial = sw.trial_buffer()
    length = new.clone()
    one = _ints([1] * R)
    buffers = sw.map_buffers(R)
    for step in range(6):
        # the window moves on where the new token would pass its end
        move = ((length + 1 - T) > tail0).to(torch.int32) * 3
        hm.hs_advance_tail(sw.ctx, tail0, move)
        hm.hs_map_tokens(sw.ctx, one, length, tail0, *buffers, status)
        xd = torch.randn(R, latent + rope, generator=gen).bfloat16().cuda()
        hm.hs_store_rows(sw.ctx, fmt, xd, w, 1e-6, f, *buffers[1:], status=status)
        length += one
        ids = torch.full((R, k), -1, dtype=torch.int32)
        for r in range(R):
            n = int(length[r])
            pick = torch.randperm(n - 1, generator=gen)[:k - 1].tolist() + [n - 1]
            ids[r, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
        qd.copy_(torch.randn(R, heads, latent + rope, generator=gen))
        topk = ids.cuda()
        if step % 2:
            hm.hs_trial(sw.ctx, topk, tail0, out, miss, status, gathered, trial)
            hm.hs_attend(sw.ctx, fmt, qd, 0.05, out, od, lse, gather=gathered, work=work)
            hm.hs_commit(sw.ctx, trial, gathered)
        else:
            hm.hs_resolve(sw.ctx, topk, tail0, out, miss, status)
            hm.hs_attend(sw.ctx, fmt, qd, 0.05, out, od, lse, work=work)
        torch.cuda.synchronize()
        assert status.tolist() == [0] * R
        for r in range(R):
            rows = torch.stack([stored(r, p) for p in ids[r].tolist() if p >= 0])
            want = ref.attend(qd[r].double().cpu(), ref.unpack(rows, latent, rope, mx), latent, 0.05)
            _within(od[r], want[0], want[2], f"step {step} request {r}")
            _within(lse[r], want[1], want[3], f"step {step} request {r}")
    sw.close()


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "8bit"])
def test_captured_steps(mx):
    """A decode step (map, store, selection, attention) captured once and replayed as its inputs move on, between eager
    steps of another context with the same inputs, on a stream of their own: equal bits in everything written."""
    R, k, B, T, H, heads, latent, rope = 5, 40, 64, 48, 200, 20, 512, 64
    fmt = hm.row_format(latent, rope, int(mx))
    gen = torch.Generator().manual_seed(31)
    w = (1 + 0.1 * torch.randn(latent, generator=gen)).bfloat16().cuda()
    f = (10000.0 ** (-2.0 * torch.arange(rope // 2, dtype=torch.float64) / rope)).cuda()
    n = 2 * R  # room for two tokens of each request; some steps have fewer

    class Steps:
        def __init__(self):
            self.sw = sw = hm.SwapIn(hm.config(R, k, B, 0.0, hm.hs_row_bytes(fmt), H, T))
            self.new, self.length, self.tail0 = _ints([0] * R), _ints([0] * R), _ints([0] * R)
            self.map, self.status = sw.map_buffers(n), torch.zeros(R, dtype=torch.int32, device="cuda")
            self.x = torch.zeros(n, latent + rope, dtype=torch.bfloat16, device="cuda")
            self.lat = torch.zeros_like(self.x)
            self.topk = torch.full((R, k), -1, dtype=torch.int32, device="cuda")
            self.out, self.miss, self.resolved = sw.outputs()[:3]
            self.q = torch.zeros(R, heads, latent + rope, dtype=torch.bfloat16, device="cuda")
            self.o = torch.zeros(R, heads, latent, dtype=torch.bfloat16, device="cuda")
            self.lse = torch.zeros(R, heads, device="cuda")
            self.work = sw.attend_work(fmt, heads)

        def run(self, stream=None):
            hm.hs_map_tokens(self.sw.ctx, self.new, self.length, self.tail0, *self.map, self.status, stream=stream)
            hm.hs_store_rows(self.sw.ctx, fmt, self.x, w, 1e-6, f, *self.map[1:], self.lat, status=self.status,
                             stream=stream)
            hm.hs_resolve(self.sw.ctx, self.topk, self.tail0, self.out, self.miss, self.resolved, stream=stream)
            hm.hs_attend(self.sw.ctx, fmt, self.q, 0.05, self.out, self.o, self.lse, work=self.work, stream=stream)

        def written(self):
            return [*self.map, self.status, self.lat, self.out, self.resolved, self.o, self.lse, self.sw.tail]

    eager, captured = Steps(), Steps()
    side = torch.cuda.Stream()
    for c in (eager, captured):
        c.sw.tail.zero_()
    captured.run()  # (nothing: no token, no selection)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured.run()
    length = [0] * R
    for step in range(8):
        new = [(step + r) % 3 for r in range(R)]
        x, q = torch.randn(n, latent + rope, generator=gen), torch.randn(R, heads, latent + rope, generator=gen)
        topk = torch.full((R, k), -1, dtype=torch.int32)
        for r in range(R):
            pick = torch.randperm(length[r] + new[r], generator=gen)[:k].to(torch.int32)
            topk[r, :len(pick)] = pick
        for c in (eager, captured):
            c.new.copy_(_ints(new)), c.length.copy_(_ints(length)), c.topk.copy_(topk)
            c.x.copy_(x), c.q.copy_(q)
            c.lat.fill_(9)
        torch.cuda.synchronize()
        eager.run(side)
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(eager.written(), captured.written())):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), (step, i)
        total = sum(new)
        assert eager.map[0].tolist()[-1] == total and eager.status.tolist() == [0] * R
        assert (eager.lat[total:] == 9).all()  # rows of no token
        length = [a + b for a, b in zip(length, new)]
    assert eager.o.abs().sum() > 0
    eager.sw.close(), captured.sw.close()
