"""What a result keeps allocated."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K", [(16, 7168), (1024, 1024), (1025, 1024), (4096, 7168), (70000, 128)])
@pytest.mark.parametrize("transposed,want_amax", [(False, False), (True, True)])
def test_rstd_does_not_keep_the_scales(hq, M, K, transposed, want_amax):
    """A training step keeps rstd for its backward pass: 4 bytes a row, with at most 64 KB of what lies beside it."""
    g = torch.Generator(device="cuda").manual_seed(M)
    x, w = torch.randn((M, K), generator=g, device="cuda").bfloat16(), torch.ones(K, dtype=torch.bfloat16, device="cuda")
    layout = hq.HQ_SCALE_TRANSPOSED if transposed else hq.HQ_SCALE_ROWMAJOR
    want = hq.add_rmsnorm_fp8_k128(x, w, scale_layout=layout)
    out = hq.add_rmsnorm_fp8_k128(x, w, scale_layout=layout, want_rstd=True, want_amax=want_amax)
    assert torch.equal(out["codes"], want["codes"]) and torch.equal(out["scales"], want["scales"])
    for name in ("rstd", "amax") if want_amax else ("rstd",):
        t = out[name]
        assert t.untyped_storage().nbytes() <= t.nbytes + 65536 + 4 * M
    assert out["rstd"].untyped_storage().nbytes() <= 4 * M + 65536
    rstd = (x.double().square().mean(-1) + 1e-6).rsqrt()
    # the row's sum (a chain of at most K / 32 + 40 additions, halved by the root) and four roundings
    assert bool(((out["rstd"].double() - rstd).abs() <= (K / 64 + 24) * 2.0 ** -24 * rstd).all())
    if want_amax:
        assert bool((out["amax"] * (1 / 448) <= out["scales"] * 1.0001).all()) and out["amax"].shape == out["scales"].shape
