"""The operators that make a selection without a GPU: sizes, and every refusal that is decided on the host."""
import ctypes

import pytest
import torch

import hierarchical_memory_amd as hm


def test_key_bytes():
    cfg = hm.config(3, 8, 16, 0.0, 1152, 100, 4)
    assert hm.hs_key_bytes(cfg, hm.key_format(128, hm.HS_KEY_MXFP8)) == 3 * 100 * 128 + 3 * 100 * 4
    assert hm.hs_key_bytes(cfg, hm.key_format(128, hm.HS_KEY_MXFP4)) == -(-3 * 100 * 64 // 256) * 256 + 3 * 100 * 4
    assert hm.hs_key_bytes(cfg, hm.key_format(64, hm.HS_KEY_MXFP4)) == -(-3 * 100 * 32 // 256) * 256 + 3 * 100 * 2
    big = hm.config(256, 2048, 4096, 0.0, 1152, 40960, 0)
    assert hm.hs_key_bytes(big, hm.key_format(128, hm.HS_KEY_MXFP8)) == 256 * 40960 * 132
    for dim, kind, msg in ((32, 0, "dim"), (256, 0, "dim"), (-64, 0, "dim"), (128, 2, "type"), (128, -1, "type")):
        with pytest.raises(hm.HiSparseError, match=msg):
            hm.hs_key_bytes(cfg, hm.key_format(dim, kind))
    assert hm.lib().hs_key_bytes(None, None, None) == hm.HS_E_INVALID


def test_key_parts():
    cfg = hm.config(3, 8, 16, 0.0, 1152, 100, 4)
    for dim in (64, 128):
        for kind in (hm.HS_KEY_MXFP8, hm.HS_KEY_MXFP4):
            key = hm.key_format(dim, kind)
            cache = torch.zeros(hm.hs_key_bytes(cfg, key), dtype=torch.uint8)
            values, scales = hm.key_parts(cfg, key, cache)
            assert values.shape == (3, 100, dim if kind == hm.HS_KEY_MXFP8 else dim // 2) and scales.shape == (3, 100, dim // 32)
            scales[2, 99, -1] = 7
            assert cache[-1] == 7 and scales.storage_offset() % 256 == 0


def test_select_work_bytes():
    cfg = hm.config(3, 8, 16, 0.0, 1152, 100, 4)
    for rows, columns in ((0, 0), (1, 100), (3, 1_000_000), (256, 40960), (1, 1 << 31)):
        assert hm.hs_select_work_bytes(cfg, rows, columns) % 16 == 0
    for rows, columns in ((-1, 4), (1, -4), (1, (1 << 31) + 4), ((1 << 30) + 1, 4)):
        with pytest.raises(hm.HiSparseError):
            hm.hs_select_work_bytes(cfg, rows, columns)


def test_null_contexts():
    lib = hm.lib()
    assert lib.hs_norm_rotate(None, None, None, 0, 0, 1, None, None, None, None, 0, None, 0, 0, None, None) == hm.HS_E_INVALID
    assert lib.hs_store_keys(None, None, None, None, 0, None, None, None, None, None, 0, None, 0, None, None,
                             None) == hm.HS_E_INVALID
    assert lib.hs_score_keys(None, None, None, 0, None, None, 1, None, None, None, 0, None, 0, None) == hm.HS_E_INVALID
    assert lib.hs_select(None, None, 0, None, None, 0, 0, None, None, 0, None) == hm.HS_E_INVALID
    assert "NULL" in hm.hs_last_error()


@pytest.fixture()
def fake_ctx():
    cfg = hm.config(3, 8, 16, 0.0, 1152, 100, 4)
    key = 0x5EED2000
    hm.hisparse._register(key, cfg, hm.hs_required_sizes(cfg))
    yield ctypes.c_void_p(key)
    hm.hisparse._CTX_SIZES.pop(key, None)


def _refused(call, good, bad):
    """call(**good) gets as far as the check that its tensors are on the GPU; every change of bad is refused by itself."""
    with pytest.raises(ValueError, match="GPU tensor"):
        call(**good)
    for name, value, msg in bad:
        with pytest.raises(ValueError, match=msg):
            call(**{**good, name: value})


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def test_norm_rotate_arguments(fake_ctx):
    fmt = hm.head_format(128, 64, 0, 0, hm.HS_NORM_LAYER, 1e-6)
    good = dict(x=_bf(5, 4, 128), weight=_bf(128), bias=_bf(128), freqs=torch.zeros(32, dtype=torch.float64), pos=_i32(5),
                o=_bf(5, 4, 128))
    bad = [("x", None, "x must not be None"), ("x", _i32(5, 4, 128), "x must be"), ("x", _bf(5, 128), "x must have shape"),
           ("x", _bf(5, 4, 64), "x must have shape"), ("x", _bf(5, 4, 256)[:, :, ::2], "contiguous heads"),
           ("weight", _bf(64), "weight must have shape"), ("weight", torch.zeros(128), "weight must be"),
           ("bias", _bf(129), "bias must have shape"), ("freqs", torch.zeros(32), "freqs must be"),
           ("freqs", torch.zeros(64, dtype=torch.float64), "freqs must have shape"), ("pos", _i32(4), "pos must have shape"),
           ("pos", torch.zeros(5), "pos must be"), ("o", None, "o must not be None"), ("o", _bf(5, 3, 128), "o must have shape"),
           ("o", torch.zeros(5, 4, 128), "o must be")]
    _refused(lambda **a: hm.hs_norm_rotate(fake_ctx, fmt, **a), good, bad)
    eight = {**good, "o": _u8(5, 4, 128).view(torch.float8_e4m3fn), "scales": _u8(5, 4, 4)}
    _refused(lambda **a: hm.hs_norm_rotate(fake_ctx, fmt, **a), eight,
             [("scales", _u8(5, 4, 2), "scales must have shape"), ("scales", _i32(5, 4, 4), "scales must be"),
              ("o", _bf(5, 4, 128), "o must be")])


def test_store_keys_arguments(fake_ctx):
    fmt, key = hm.head_format(128, 64, 0, 0, hm.HS_NORM_LAYER, 1e-6), hm.key_format(128, hm.HS_KEY_MXFP4)
    good = dict(x=_bf(5, 128), weight=_bf(128), bias=_bf(128), freqs=torch.zeros(32, dtype=torch.float64), req=_i32(5),
                pos=_i32(5), keys=_u8(100000), values=_bf(5, 128), status=_i32(3))
    bad = [("x", None, "x must not be None"), ("x", _bf(5, 64), "x must have shape"), ("x", torch.zeros(5, 128), "x must be"),
           ("x", _bf(5, 256)[:, ::2], "contiguous rows"), ("weight", _bf(5), "weight"), ("bias", _bf(5), "bias"),
           ("freqs", _bf(32), "freqs"), ("req", _i32(4), "req must have shape"), ("pos", None, "pos must not be None"),
           ("pos", torch.zeros(5), "pos must be"), ("keys", None, "keys must not be None"), ("values", _bf(4, 128), "values"),
           ("status", _i32(2), "status")]
    _refused(lambda **a: hm.hs_store_keys(fake_ctx, fmt, key, **a), good, bad)


def test_score_keys_arguments(fake_ctx):
    key = hm.key_format(128, hm.HS_KEY_MXFP8)
    good = dict(keys=_u8(100000), q=_u8(5, 4, 128).view(torch.float8_e4m3fn), q_scales=_u8(5, 4, 4), weights=torch.zeros(5, 4),
                req=_i32(5), pos=_i32(5), scores=torch.zeros(5, 100))
    bad = [("keys", None, "keys must not be None"), ("q", None, "q must not be None"), ("q", _u8(5, 4, 128), "q must be"),
           ("q", _u8(5, 4, 64), "q must have shape"), ("q", _u8(20, 128), "q must have shape"),
           ("q_scales", _u8(5, 4, 2), "q_scales must have shape"), ("weights", torch.zeros(5, 3), "weights must have shape"),
           ("weights", _bf(5, 4), "weights must be"), ("req", _i32(6), "req"), ("pos", _i32(5).long(), "pos"),
           ("scores", None, "scores must not be None"), ("scores", torch.zeros(5, 99), "scores must have shape"),
           ("scores", torch.zeros(4, 100), "scores must have shape"), ("scores", torch.zeros(100, 5).T, "contiguous rows"),
           ("scores", torch.zeros(5, 100, dtype=torch.float64), "scores must be"),
           ("scores", torch.zeros(1, 100).expand(5, 100), "contiguous rows")]
    _refused(lambda **a: hm.hs_score_keys(fake_ctx, key, **a), good, bad)


def test_select_arguments(fake_ctx):
    good = dict(scores=torch.zeros(5, 100), pos=_i32(5), topk=_i32(5, 8))
    bad = [("scores", None, "scores must not be None"), ("scores", torch.zeros(100), "scores must have shape"),
           ("scores", _bf(5, 100), "scores must be"), ("scores", torch.zeros(100, 5).T, "contiguous rows"),
           ("scores", torch.zeros(5, 200)[:, :100], "elements apart"), ("pos", _i32(4), "pos has"),
           ("pos", None, "pos must not be None"), ("topk", _i32(4, 8), "topk has"), ("topk", torch.zeros(5, 8), "topk must be"),
           ("cu", _i32(3), "cu has")]
    _refused(lambda **a: hm.hs_select(fake_ctx, **a), good, bad)
    _refused(lambda **a: hm.hs_select(fake_ctx, **a), {**good, "cu": _i32(4), "topk": _i32(3, 8)},
             [("topk", _i32(2, 8), "topk has")])


@pytest.mark.parametrize("n", [(1 << 30) + 1, 1 << 31, (1 << 32) + 4])
def test_lengths_past_the_limit(fake_ctx, n):
    """Refused by the tensors' shapes, also where 32 bits of a length would be one in range."""
    meta = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device="meta")  # noqa: E731
    bf, i32, f32, f8 = torch.bfloat16, torch.int32, torch.float32, torch.float8_e4m3fn
    fmt, key = hm.head_format(64), hm.key_format(64, hm.HS_KEY_MXFP8)
    at, cache = meta(n, dtype=i32), _u8(100_000)
    most = "at most 1073741824"
    for shape in ((n, 1, 64), (2, n, 64)):
        with pytest.raises(ValueError, match=most):
            hm.hs_norm_rotate(fake_ctx, fmt, _bf(1, 1, 64).expand(shape), None, None, None, at, meta(*shape, dtype=bf))
        with pytest.raises(ValueError, match=most):
            hm.hs_score_keys(fake_ctx, key, cache, meta(*shape, dtype=f8), meta(*shape[:2], 2, dtype=torch.uint8),
                             meta(*shape[:2], dtype=f32), at[:shape[0]], at[:shape[0]], meta(shape[0], 100, dtype=f32))
    with pytest.raises(ValueError, match=most):
        hm.hs_store_keys(fake_ctx, fmt, key, meta(n, 64, dtype=bf), None, None, None, at, at, cache)
    for cu in (None, _i32(4)):
        with pytest.raises(ValueError, match=most):
            hm.hs_select(fake_ctx, meta(n, 4, dtype=f32), at, meta(n, 8, dtype=i32), cu=cu)


def test_numbers_past_32_bits(fake_ctx):
    cfg = hm.config(3, 8, 16, 0.0, 1152, 100, 4)
    for rows, columns in (((1 << 32) + 4, 100), (-(1 << 32), 100), (4, (1 << 64) + 100)):
        with pytest.raises(ValueError, match="rows must be in"):
            hm.hs_select_work_bytes(cfg, rows, columns)
    for recent in (1 << 32, -(1 << 32), (1 << 32) + 3):
        with pytest.raises(ValueError, match="recent must be in"):
            hm.hs_select(fake_ctx, torch.zeros(5, 100), _i32(5), _i32(5, 8), recent=recent)


def test_destroyed_handle_is_none(monkeypatch):
    """The handle itself ends with its context, so that a copy of it reaches the library as NULL."""
    seen = []

    class Library:
        hs_destroy = staticmethod(lambda ctx: seen.append(ctx.value))

    ctx = ctypes.c_void_p(0x5EED3000)
    copy = ctx
    monkeypatch.setattr(hm.hisparse, "lib", lambda: Library)
    for _ in range(2):
        hm.hs_destroy(ctx)
    assert seen == [0x5EED3000] and not copy.value


def test_formats_past_32_bits():
    for name in ("dim", "rope", "rope_at", "rope_style", "norm"):
        for v in ((1 << 32) + 32, -(1 << 32), 1 << 31):
            with pytest.raises(ValueError, match=f"{name} must be a number of 32 bits"):
                hm.head_format(**{"dim": 64, name: v})
    for name in ("dim", "key_type"):
        with pytest.raises(ValueError, match=f"{name} must be a number of 32 bits"):
            hm.key_format(**{name: 1 << 32})
    assert hm.head_format(-(1 << 31)).dim == -(1 << 31)  # (of 32 bits: the library's to refuse)
