"""The norms of rows and their gradients against their formulas in 64 bits.

Tolerances, u = 2^-24.  A row's sums: a thread adds 8 values one after the other and at most 8 sums of 8, 5 further additions
join the threads of a warp and at most 16 the warps: 37, say 48 roundings at most, each u relative to the sum of magnitudes.
Squares are fused; the variance, its root and the quotient add 5 u.  So r is within 30 u (half of 48, and 5, rounded up) relative.
The layer norm's m is within 49 u of mean|x|, but what it misses is taken out of n again, up to 49 u of mean|x - m|.
  y: n = (x - m) r: 30 u of |n|, the subtractions 2 u of |x - m| + u |m| r (m is kept in two parts whose sum is m to 49 u
     of mean|x - m| + u |m - part|), the product and the addition 2 u; then the output's rounding.
  gradient: with the same r and m as the formula: e, n: 3 u; mean(e), mean(e n): 48 + 4 u of the mean magnitudes; dx adds 4 u.
  dweight, dbias: the sum over `rows` values: 4 u a term, and as many additions as there are rows in one thread's walk, the
     CTA's row groups and the partial sums: each joins rows that no other did, so (4 + rows) u of the sum of magnitudes
     bounds them all.
"""
import pytest
import torch

from mixture_experts_layer_rmsnorm_gb300 import binding
from test_gpu_8_grouped import BF16, FP16, FP32, half_step

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
NAN, INF = float("nan"), float("inf")


def tiny(dtype):
    return 2.0 ** -25 if dtype == FP16 else 2.0 ** -130


def within(got, want, lim):
    lim = lim + half_step(got.dtype) * (want.abs() + lim) + tiny(got.dtype)
    worst = ((got.double() - want).abs() - lim).max().item() if got.numel() else 0.0
    assert worst <= 0, f"error above its bound by {worst:.3e}"


class Case:
    def __init__(self, kind, rows, h, dtype, wtype, pad=0, offset=0.0, eps=1e-5, weight=True):
        gen = torch.Generator(device="cuda").manual_seed(rows + h)

        def rand(*shape):
            return torch.randn(shape, generator=gen, device="cuda")

        self.layer, self.eps, self.rows, self.h = kind == "layer", eps, rows, h
        self.x = (rand(rows, h + pad) * 1.5 + offset).to(dtype)[:, :h]
        self.dy = (rand(rows, h + pad) * 0.3).to(dtype)[:, :h]
        self.w = (1 + 0.2 * rand(h)).to(wtype) if weight else None
        self.b = (0.2 * rand(h)).to(wtype) if self.layer and weight else None
        self.norm = binding.RowNorm(h, kind, dtype, wtype, eps)
        self.pad, self.dtype, self.wtype = pad, dtype, wtype

    def formula(self):
        x = self.x.double()
        m = x.mean(1, keepdim=True) if self.layer else torch.zeros_like(x[:, :1])
        r = 1 / torch.sqrt((x - m).square().mean(1, keepdim=True) + self.eps)
        return x, m, r

    def weights(self):
        one = torch.ones(self.h, dtype=torch.float64, device="cuda")
        return one if self.w is None else self.w.double(), 0 * one if self.b is None else self.b.double()


CASES = {
    "one": ("rms", 1, 8, BF16, BF16),
    "one_layer": ("layer", 1, 8, FP32, FP32),
    "lanes8": ("layer", 77, 56, FP16, FP32, 8),
    "lanes16": ("rms", 1001, 128, BF16, BF16),
    "lanes16_layer": ("layer", 33, 72, FP32, FP32, 16),
    "lanes32": ("layer", 515, 248, BF16, FP32),
    "warp": ("rms", 95, 264, FP16, FP16, 24),
    "warp_layer": ("layer", 4097, 1024, BF16, BF16),
    "warp_fp32": ("layer", 9, 1016, FP32, FP32),
    "cta": ("rms", 700, 1032, BF16, FP32, 8),
    "cta_layer": ("layer", 333, 1408, FP16, FP16),
    "cta_4096": ("rms", 2050, 4096, BF16, BF16),
    "cta_layer_2056": ("layer", 130, 2056, FP32, FP32, 8),
    "cta_layer_4096": ("layer", 611, 4096, BF16, FP32),
    "cta_7168": ("layer", 401, 7168, BF16, FP32),
    "cta_8192_fp32": ("rms", 161, 8192, FP32, FP32),
    "cta_wide": ("layer", 323, 8200, FP16, FP16, 16),
    "cta_widest": ("rms", 7, 16384, BF16, BF16),
    "cta_widest_fp32": ("layer", 5, 16384, FP32, FP32),
    "no_weight": ("layer", 50, 640, BF16, BF16, 0, 0.0, 1e-5, False),
    "no_weight_rms": ("rms", 21, 2048, FP32, FP32, 0, 0.0, 0.0, False),
    "far": ("layer", 200, 512, FP32, FP32, 0, 3000.0),
    "far_wide": ("layer", 60, 5120, FP32, FP32, 0, -20000.0),
}


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    c = Case(*CASES[name])
    x, m, r = c.formula()
    w, b = c.weights()
    full = torch.full((c.rows, c.h + c.pad), 7.0, dtype=c.dtype, device="cuda")
    out = c.norm.forward(c.x, c.w, c.b, y=full[:, :c.h], stats=True)
    assert torch.all(full[:, c.h:] == 7.0)
    y, rstd = out[0], out[1]
    d = (x - m).abs()
    n = d * r
    miss = 50 * U * d.mean(1, keepdim=True) + 3 * U * d + U * U * 50 * m.abs()
    if c.layer:
        within(out[2], m[:, 0], U * m[:, 0].abs() + 50 * U * d.mean(1))
    within(rstd, r[:, 0], 30 * U * r[:, 0])
    within(y, (x - m) * r * w + b, w.abs() * (32 * U * n + miss * r) + 2 * U * (n * w.abs() + b.abs()))
    assert torch.equal(c.norm.forward(c.x, c.w, c.b), y)
    same = c.x.clone(memory_format=torch.preserve_format)
    assert torch.equal(c.norm.forward(same, c.w, c.b, y=same), y)


@pytest.mark.parametrize("name", CASES)
def test_gradient(name):
    c = Case(*CASES[name])
    _, rstd, *mean = c.norm.forward(c.x, c.w, c.b, stats=True)
    mean = mean[0] if mean else None
    x, dy, r = c.x.double(), c.dy.double(), rstd.double()[:, None]
    m = mean.double()[:, None] if c.layer else torch.zeros_like(r)
    w, _ = c.weights()
    n, e = (x - m) * r, dy * w
    c1 = (e * n).mean(1, keepdim=True)
    c0 = e.mean(1, keepdim=True) if c.layer else torch.zeros_like(c1)
    dx = r * (e - c0 - n * c1)
    lim1 = 52 * U * (e * n).abs().mean(1, keepdim=True)
    lim0 = 50 * U * e.abs().mean(1, keepdim=True) if c.layer else 0.0 * c1
    lim = r * (lim0 + n.abs() * (lim1 + 4 * U * c1.abs()) + 4 * U * (e.abs() + c0.abs()))
    got = c.norm.grad(c.dy, c.x, c.w, rstd, mean, dtype=FP32)
    within(got[0], dx, lim)
    within(got[1], (dy * n).sum(0), (4 + c.rows) * U * (dy * n).abs().sum(0))
    if c.layer:
        within(got[2], dy.sum(0), c.rows * U * dy.abs().sum(0))
    # again, into the caller's, and over dy: the same bits
    full = torch.full((c.rows, c.h + c.pad), 7.0, dtype=c.dtype, device="cuda")
    rounded = c.norm.grad(c.dy, c.x, c.w, rstd, mean, dx=full[:, :c.h])
    assert torch.equal(rounded[0], got[0]) and torch.all(full[:, c.h:] == 7.0)
    for a, b in zip(rounded[1:], got[1:]):
        assert a.dtype == c.wtype and torch.equal(a, b.to(c.wtype))
    start = [torch.randn(c.h, device="cuda") for _ in got[1:]]
    sums = [s.clone() for s in start]
    dys = c.dy.clone(memory_format=torch.preserve_format)
    c.norm.grad(dys, c.x, c.w, rstd, mean, dx=dys, dweight=sums[0], dbias=sums[1] if c.layer else None, accumulate=True)
    assert torch.equal(dys, got[0])
    assert all(torch.equal(s, a + b) for s, a, b in zip(sums, start, got[1:]))


@pytest.mark.parametrize("kind,h", [("rms", 64), ("layer", 1040)])
def test_gradient_against_differences(kind, h):
    """The slope of sum(dy y) along a direction, from the kernel's own forward in fp32: the difference's error is some
    2^-24 sqrt(rows h) of the sum of magnitudes over the step, and the third derivative's share, step^2."""
    c = Case(kind, 12, h, FP32, FP32)
    gen = torch.Generator(device="cuda").manual_seed(1)
    vx, vw, vb = (torch.randn(t.shape, generator=gen, device="cuda") for t in (c.x, c.w, c.w))
    step = 2.0 ** -7

    def loss(s):
        y = c.norm.forward(c.x + s * step * vx, c.w + s * step * vw, c.b + s * step * vb if c.layer else None)
        return (c.dy.double() * y.double()).sum()

    slope = (loss(1) - loss(-1)) / (2 * step)
    _, rstd, *mean = c.norm.forward(c.x, c.w, c.b, stats=True)
    got = c.norm.grad(c.dy, c.x, c.w, rstd, *mean)
    want = sum((g.double() * v.double()).sum() for g, v in zip(got, (vx, vw, vb)))
    size = (c.dy.abs() * 4).sum().double()
    assert (slope - want).abs() <= size * (2.0 ** -23 / step + step ** 2)


def test_many_rows_and_offsets_beyond_32_bits():
    """2^22 rows 1032 elements apart: offsets of up to 2^32 elements; the last rows are right, and the sums whole."""
    rows, h, ld = 2 ** 22 + 3, 128, 1032
    x = torch.zeros((rows, ld), dtype=BF16, device="cuda")[:, :h]
    gen = torch.Generator(device="cuda").manual_seed(2)
    x.copy_(torch.randn((rows, h), generator=gen, device="cuda"))
    norm = binding.RowNorm(h, "rms", BF16, FP32)
    w = torch.ones(h, device="cuda")
    y, rstd = norm.forward(x, w, stats=True)
    tail = x[-1000:].double()
    r = 1 / torch.sqrt(tail.square().mean(1, keepdim=True) + 1e-6)
    within(y[-1000:], tail * r, 36 * U * (tail * r).abs())
    dx, dw = norm.grad(y, x, w, rstd)
    want, size = 0, 0
    for part in range(0, rows, 2 ** 19):
        at = slice(part, part + 2 ** 19)
        t = y[at].double() * x[at].double() * rstd[at].double()[:, None]
        want, size = want + t.sum(0), size + t.abs().sum(0)
    # a thread adds rows / (16 x 456) of them one after the other, at least 456 CTAs of 16 rows; 16 rows meet in the CTA,
    # then the sums of at most 1280 CTAs: 40 one after the other, and 32 of those
    within(dw, want, (4 + rows / 16 / 456 + 16 + 40 + 32) * U * size)
    n = tail * rstd[-1000:].double()[:, None]
    e = y[-1000:].double()
    within(dx[-1000:], rstd[-1000:].double()[:, None] * (e - n * (e * n).mean(1, keepdim=True)),
           60 * U * rstd[-1000:].double()[:, None] * (e.abs() + n.abs() * (e * n).abs().mean(1, keepdim=True)))


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("h", [64, 2048])
def test_rows_without_spread_and_rows_that_are_no_numbers(kind, h):
    x = torch.randn((6, h), device="cuda")
    clean = x.clone()
    x[1], x[2], x[3, 5], x[4, 6] = 0.0, 3.0, NAN, INF
    norm = binding.RowNorm(h, kind, FP32, eps=1e-4)
    w = torch.ones(h, device="cuda")
    out, ref = norm.forward(x, w, stats=True), norm.forward(clean, w)
    y = out[0]
    assert torch.equal(y[0], ref[0]) and torch.equal(y[5], ref[5])
    assert torch.all(y[1] == 0.0) and torch.isnan(y[3]).all()
    if kind == "layer":
        assert torch.all(y[2] == 0.0) and torch.isnan(y[4]).all()
    else:
        assert torch.isnan(y[4, 6]) and torch.all(y[4, :6] == 0.0)
    dy = torch.randn((6, h), device="cuda")
    dx = norm.grad(dy, x, w, *out[1:])[0]
    assert torch.isnan(dx[3]).all() and torch.isfinite(dx[[0, 1, 2, 5]]).all()


def test_no_rows():
    for kind in ("rms", "layer"):
        norm = binding.RowNorm(64, kind, BF16, FP32)
        x, w = torch.empty((0, 64), dtype=BF16, device="cuda"), torch.ones(64, device="cuda")
        out = norm.forward(x, w, stats=True)
        got = norm.grad(x, x, w, *out[1:])
        assert got[0].shape == (0, 64) and all(torch.all(g == 0.0) for g in got[1:])
        kept = [torch.full((64,), 3.0, device="cuda") for _ in got[1:]]
        norm.grad(x, x, w, *out[1:], dweight=kept[0], dbias=kept[1] if kind == "layer" else None, accumulate=True)
        assert all(torch.all(k == 3.0) for k in kept)


def test_replays_from_a_graph_on_new_rows():
    c = Case("layer", 300, 1024, BF16, FP32)
    y, dx = torch.empty_like(c.x), torch.empty_like(c.x)
    dw, db = torch.zeros(1024, device="cuda"), torch.zeros(1024, device="cuda")

    def step():
        _, rstd, mean = c.norm.forward(c.x, c.w, c.b, y=y, stats=True)
        c.norm.grad(c.dy, c.x, c.w, rstd, mean, dx=dx, dweight=dw, dbias=db)

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    c.x.mul_(-0.5).add_(0.25)
    c.dy.add_(0.125)
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in (y, dx, dw, db)]
    step()
    assert all(torch.equal(a, b) for a, b in zip(replayed, (y, dx, dw, db)))


def test_objects_refuse_what_does_not_fit():
    norm = binding.RowNorm(64, "rms", BF16)
    x = torch.ones((4, 64), dtype=BF16, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    y, rstd = norm.forward(x, w, stats=True)
    with pytest.raises(ValueError):
        binding.RowNorm(64, "batch", BF16)
    for h in (12, 16392, 0):
        with pytest.raises(binding.MoeError):
            binding.RowNorm(h, "rms", BF16)
    with pytest.raises(binding.MoeError):
        binding.RowNorm(64, "rms", BF16, FP16)
    with pytest.raises(TypeError):
        norm.forward(x.float(), w)
    with pytest.raises(ValueError):
        norm.forward(x, w[:32])
    with pytest.raises(binding.MoeError):
        norm.forward(x, w, bias=w)  # the rms norm has none
    with pytest.raises(ValueError):
        norm.grad(y, x, w, rstd, accumulate=True)
    with pytest.raises(binding.MoeError):
        norm.grad(y, x, w, rstd, dweight=w.clone(), accumulate=True)  # 16 bits
    with pytest.raises(binding.MoeError):
        binding.RowNorm(64, "layer", BF16).grad(y, x, w, rstd)  # no mean
    with pytest.raises(binding.MoeError):
        norm.forward(torch.ones((4, 72), dtype=BF16, device="cuda")[:, 4:68], w)  # not on a 16-byte border
