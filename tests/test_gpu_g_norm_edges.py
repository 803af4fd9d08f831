"""The norms of rows at the ends of fp32's range: what the header says of squares and sums that do not fit, and that other
rows are not touched by it."""
import pytest
import torch

from mixture_experts_layer_rmsnorm_gb300 import binding
from test_gpu_8_grouped import BF16, FP32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("h", [64, 136, 520, 1408, 4096, 16384])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_rows_whose_squares_or_sums_do_not_fit(kind, dtype, h):
    gen = torch.Generator(device="cuda").manual_seed(h)
    x = torch.randn((20, h), generator=gen, device="cuda").to(dtype)
    w = torch.randn(h, generator=gen, device="cuda").to(dtype)
    b = torch.randn(h, generator=gen, device="cuda").to(dtype) if kind == "layer" else None
    norm = binding.RowNorm(h, kind, dtype, eps=1e-6)
    clean = norm.forward(x, w, b, stats=True)
    huge, beyond = x.clone(), x.clone()
    huge[3] *= 1e25   # squares do not fit fp32, their sum's root would
    beyond[3] = 2e38  # nor does the layer norm's sum
    others = torch.arange(20, device="cuda") != 3
    for at, rows in (("huge", huge), ("beyond", beyond)):
        got = norm.forward(rows, w, b, stats=True)
        for g, c in zip(got, clean):
            assert torch.equal(g[others], c[others])
        if at == "huge" or kind == "rms":
            assert got[1][3] == 0.0
            assert torch.equal(got[0][3], b if kind == "layer" else torch.zeros_like(w))
        else:
            assert torch.isnan(got[0][3]).all() and torch.isnan(got[1][3])


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_rows_whose_squares_vanish(kind):
    x = torch.full((3, 256), 1e-30, device="cuda")
    x[1], x[2, ::2] = 1.0, -1e-30
    x[1, ::2] = -1.0
    y, r = binding.RowNorm(256, kind, FP32, eps=0.0).forward(x, stats=True)[:2]
    assert torch.all(y[1].abs() == 1.0) and r[1] == 1.0
    assert r[0] == float("inf") and r[2] == float("inf")
    y, r = binding.RowNorm(256, kind, FP32, eps=1e-6).forward(x, stats=True)[:2]
    assert torch.all(y[::2].abs() <= 1e-26) and torch.isfinite(r).all()
