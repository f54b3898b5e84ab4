"""The latent-attention operators without a GPU: formats, sizes, and every refusal that is decided on the host."""
import ctypes

import pytest
import torch

import hierarchical_memory_amd as hm
from tests.latent_ref import row_layout


@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("rope", [32, 64])
def test_row_bytes(latent, rope):
    assert hm.hs_row_bytes(hm.row_format(latent, rope, hm.HS_ROW_BF16)) == 2 * (latent + rope)
    n = hm.hs_row_bytes(hm.row_format(latent, rope, hm.HS_ROW_MXFP8))
    assert n == row_layout(latent, rope, True)[2] and n % 16 == 0


def test_row_bytes_of_the_workloads():
    assert hm.hs_row_bytes(hm.row_format()) == 1152
    assert hm.hs_row_bytes(hm.row_format(512, 64, hm.HS_ROW_MXFP8)) == 656


@pytest.mark.parametrize("fmt,msg", [((128, 64, 0), "latent"), ((0, 64, 0), "latent"), ((512, 16, 0), "rope"),
                                     ((512, -64, 0), "rope"), ((512, 64, 2), "type"), ((512, 64, -1), "type")])
def test_formats_refused(fmt, msg):
    with pytest.raises(hm.HiSparseError) as e:
        hm.hs_row_bytes(hm.row_format(*fmt))
    assert e.value.code == hm.HS_E_INVALID and msg in str(e.value)
    with pytest.raises(hm.HiSparseError):
        hm.hs_attend_work_bytes(hm.config(2, 8, 16, 2.0, 1152), hm.row_format(*fmt), 16)


def test_work_bytes():
    fmt = hm.row_format()
    for R, k, heads in ((1, 1, 1), (1, 256, 16), (32, 2048, 16), (256, 2048, 128), (3, 4096, 512), (65535, 8, 16)):
        n = hm.hs_attend_work_bytes(hm.config(R, k, k, 2.0, 1152), fmt, heads)
        assert n >= 0 and n % 16 == 0, (R, k, heads, n)
    for heads in (0, -1, 513):
        with pytest.raises(hm.HiSparseError, match="heads"):
            hm.hs_attend_work_bytes(hm.config(2, 8, 16, 2.0, 1152), fmt, heads)
    with pytest.raises(hm.HiSparseError, match="1152 bytes"):
        hm.hs_attend_work_bytes(hm.config(2, 8, 16, 2.0, 656), fmt, 16)
    assert hm.lib().hs_attend_work_bytes(None, None, 1, None) == hm.HS_E_INVALID


def test_prompt_work_bytes():
    for R, n_q, n_k, heads, dims in ((1, 0, 0, 1, (64, 32, 64)), (4, 512, 16384, 8, (192, 64, 256)),
                                     (8, 8192, 8192, 16, (128, 64, 128)), (1, 1, 1 << 30, 1, (128, 64, 128))):
        n = hm.hs_attend_prompt_work_bytes(R, n_q, n_k, heads, *dims)
        assert n >= 0 and n % 16 == 0
    for bad, msg in (((0, 1, 1, 1, 128, 64, 128), "num_requests"), ((1, -1, 1, 1, 128, 64, 128), "n_q"),
                     ((1, 1, -1, 1, 128, 64, 128), "n_k"), ((1, (1 << 30) + 1, 1, 1, 128, 64, 128), "n_q"),
                     ((1, 1, 1, 0, 128, 64, 128), "heads"), ((1, 1, 1, 1, 128, 48, 128), "rope"),
                     ((1, 1, 1, 1, 128, 64, 64), "nope, value")):
        with pytest.raises(hm.HiSparseError, match=msg):
            hm.hs_attend_prompt_work_bytes(*bad)


def test_null_contexts():
    lib = hm.lib()
    assert lib.hs_row_bytes(None, None) == hm.HS_E_INVALID
    assert lib.hs_map_tokens(None, None, None, None, 0, None, None, None, None, None, None) == hm.HS_E_INVALID
    assert lib.hs_store_rows(None, None, None, 0, None, 0.0, None, 0, None, None, None, 0, None, None,
                             None) == hm.HS_E_INVALID
    assert lib.hs_attend(None, None, None, 1, 1.0, None, None, None, None, None, 0, None) == hm.HS_E_INVALID
    assert lib.hs_attend_prompt(None, None, None, None, 0, None, None, 0, 0, 1, 128, 64, 128, 1.0, 1, None, None,
                                None, 0, None) == hm.HS_E_INVALID
    assert "NULL" in hm.hs_last_error()


@pytest.fixture()
def fake_ctx():
    cfg = hm.config(3, 8, 16, 0.0, 1152, 100, 4)
    key = 0x5EED1000
    hm.hisparse._register(key, cfg, hm.hs_required_sizes(cfg))
    yield ctypes.c_void_p(key)
    hm.hisparse._CTX_SIZES.pop(key, None)


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_map_arguments(fake_ctx):
    good = dict(new=_i32(3), length=_i32(3), tail0=_i32(3), cu=_i32(4), req=_i32(9), pos=_i32(9), slot=_i32(9))
    for kw, msg in ((dict(new=None), "new must not be None"), (dict(new=_i32(2)), "new has 2"),
                    (dict(length=torch.zeros(3, dtype=torch.int64)), "length must be a torch.int32"),
                    (dict(cu=_i32(3)), "cu has 3"), (dict(pos=_i32(8)), "one length"),
                    (dict(status=_i32(1)), "status has 1"), (dict(), "GPU tensor")):
        with pytest.raises(ValueError, match=msg):
            hm.hs_map_tokens(fake_ctx, **dict(good, **kw))


@pytest.mark.parametrize("n", [(1 << 30) + 1, 1 << 31, (1 << 32) + 5])
def test_map_length_past_the_limit(fake_ctx, n):
    """Refused by the tensors' length, also where 32 bits of it would be a length in range."""
    far = torch.empty(n, dtype=torch.int32, device="meta")
    with pytest.raises(ValueError, match="at most 1073741824"):
        hm.hs_map_tokens(fake_ctx, _i32(3), _i32(3), _i32(3), _i32(4), far, far, far)


def test_store_arguments(fake_ctx):
    good = dict(fmt=hm.row_format(), x=_bf(5, 576), weight=_bf(512), eps=1e-6, freqs=torch.zeros(32, dtype=torch.float64),
                req=_i32(5), pos=_i32(5), slot=_i32(5), latent=_bf(5, 576))
    for kw, msg in ((dict(x=_bf(5, 575)), "x must have shape"), (dict(x=torch.zeros(5, 576)), "x must be a torch.bfloat16"),
                    (dict(x=_bf(576, 5).T), "contiguous rows"), (dict(x=None), "x must not be None"),
                    (dict(weight=_bf(511)), "weight must have shape"), (dict(), "GPU tensor")):
        with pytest.raises(ValueError, match=msg):
            hm.hs_store_rows(fake_ctx, **dict(good, **kw))


def test_attend_arguments(fake_ctx):
    good = dict(fmt=hm.row_format(), q=_bf(3, 16, 576), scale=0.1, out=_i32(3, 8), o=_bf(3, 16, 512),
                lse=torch.zeros(3, 16))
    for kw, msg in ((dict(q=_bf(2, 16, 576)), "q must have shape"), (dict(q=_bf(3, 16, 512)), "q must have shape"),
                    (dict(q=None), "q must not be None"), (dict(o=_bf(3, 15, 512)), "o must have shape"),
                    (dict(o=torch.zeros(3, 16, 512)), "o must be a torch.bfloat16"),
                    (dict(lse=torch.zeros(3, 15)), "lse must have shape"), (dict(out=_i32(3, 7)), "out has 21"),
                    (dict(gather=torch.zeros(100, dtype=torch.uint8)), "gather has 100 bytes"), (dict(), "GPU tensor")):
        with pytest.raises(ValueError, match=msg):
            hm.hs_attend(fake_ctx, **dict(good, **kw))


def test_prompt_arguments(fake_ctx):
    good = dict(q=_bf(7, 4, 192), kv=_bf(9, 4, 256), rope=_bf(9, 576)[:, 512:], cu_q=_i32(4), cu_k=_i32(4), scale=0.1,
                o=_bf(7, 4, 128), lse=torch.zeros(7, 4))
    for kw, msg in ((dict(q=_bf(7, 192)), "q must have shape"), (dict(kv=_bf(9, 5, 256)), "kv must have shape"),
                    (dict(rope=_bf(8, 64)), "rope must have shape"), (dict(rope=_bf(64, 9).T), "contiguous rows"),
                    (dict(o=_bf(7, 4, 129)), "kv must hold"), (dict(lse=torch.zeros(7, 5)), "lse must have"),
                    (dict(), "GPU tensor")):
        with pytest.raises(ValueError, match=msg):
            hm.hs_attend_prompt(fake_ctx, **dict(good, **kw))


def test_stream_of_an_address(monkeypatch):
    """A work buffer is taken on the stream that the kernels run on: address 0 is the default stream."""
    class External:
        def __init__(self, address):
            assert address, "torch takes a null address for none given"
            self.cuda_stream = address

    default = object()
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: default)
    assert hm.hisparse._torch_stream(0) is default
    assert hm.hisparse._torch_stream(0x1000).cuda_stream == 0x1000
    assert hm.hisparse._torch_stream(None) is None
    assert hm.hisparse._torch_stream(default) is default
