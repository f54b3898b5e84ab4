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
from tests.test_gpu_latent import _check_row  # noqa: E402


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
