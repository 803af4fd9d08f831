"""The 8-bit products where their scales leave the range of ordinary numbers, and where each tile plan's units end, against
64 bits.

Tolerance as for ordinary scales: a block's sum meets the two scales with one fp32 rounding before the multiply-add, whether
the scales meet first or the sum meets one of them.  What lies below fp32's normal range costs half a subnormal step a
block more, and in the output half a subnormal step of its type (2^-134 for bf16).  So
|err| <= eps/2 |y| + (132 + (blocks + 257) / 2) 2^-23 S + blocks 2^-149 + tiny.
"""
import pytest
import torch

from mixture_experts_layer_rmsnorm_gb300 import binding
from test_gpu_8_grouped import BF16, FP16, FP32, Lists, half_step
from test_gpu_a_fp8 import define, e4m3_table, same_bits, values_of

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def plan_of(rows, groups):
    """The rule by which the library chooses a tile plan for an 8-bit product, restated."""
    mean = -(-rows // groups)
    if mean <= 16:
        return "small"
    return "pairs" if 12 * -(-mean // 256) <= 7 * -(-mean // 128) else "single"


PLANS = {"small": [5, 0, 20, 7], "single": [60, 1, 129, 33], "pairs": [255, 1, 300, 212]}


def check(got, xv, wv, blocks):
    """got [rows, F] against xv [rows, R] times wv [R, F]."""
    want, s = xv @ wv, xv.abs() @ wv.abs()
    tiny = 2.0 ** -25 if got.dtype == FP16 else 2.0 ** -134
    lim = half_step(got.dtype) * want.abs() + (132 + (blocks + 257) / 2) * 2.0 ** -23 * s + blocks * 2.0 ** -149 + tiny
    assert torch.isfinite(got).all()
    worst = ((got.double() - want).abs() - lim).max().item() if got.numel() else 0.0
    assert worst <= 0, f"error above its bound by {worst:.3e}"


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("plan", PLANS)
def test_scales_whose_product_is_no_fp32_number(plan, dgrad):
    """Codes and scales of a caller's own, the reduction's first block under weight scales of 2^60, the others 2^-70."""
    gen = torch.Generator(device="cuda").manual_seed(21)
    lists = Lists(PLANS[plan])
    assert plan_of(lists.rows, lists.groups) == plan
    rows, r, f, g = lists.rows, 528, 272, lists.groups
    blocks, kind = -(-r // 128), torch.arange(rows, device="cuda") % 5

    def pick(*shape):
        return torch.randint(0x70, 0x7F, shape, generator=gen, device="cuda", dtype=torch.uint8)

    def mantissa(*shape):
        return 1 + torch.rand(shape, generator=gen, device="cuda")

    # large codes, of one sign along the reduction, so that a block's sums are large ...
    xc, wc = pick(rows, r), pick(g, f, r)
    wc |= (torch.randint(0, 2, (g, f, 1), generator=gen, device="cuda") * 128).to(torch.uint8)
    # ... but in the first block, where rows and weights meet in one place at most, by the smallest codes
    xc[:, :128], wc[:, :, :128] = 0, 0
    xc[kind < 2, :64], wc[:, :, 64:128] = 0x77, 0x77
    xc[:, 5], wc[:, :, 5] = 0, 1
    xc[kind == 1, 5] = 1
    sx = mantissa(rows, blocks)
    for k, e in enumerate((70, 70, -74, -82, 70)):  # (then factors of 1, 1, 2^-144, 2^-152 and 1)
        sx[kind == k] *= 2.0 ** e
    sx[kind < 2, 0] *= 2.0 ** 10  # (2^140)
    sw = mantissa(g, -(-f // 128), blocks)
    sw[:, :, 0] *= 2.0 ** 60
    sw[:, :, 1:] *= 2.0 ** -70

    def value(codes, scales, height):
        table = e4m3_table()
        table = torch.cat([table, table.new_zeros(1), -table, table.new_zeros(1)])
        s = scales.double().repeat_interleave(128, -1)[..., :codes.shape[-1]]
        if height > 1:
            s = s.repeat_interleave(height, -2)[..., :codes.shape[-2], :]
        return table[codes.long()] * s

    assert torch.isfinite(sx).all() and torch.isfinite(sw).all()
    xv, wv = value(xc, sx, 1), value(wc, sw, 128)
    r8 = binding.Fp8Rows(r).quantize(torch.zeros((rows, r), dtype=BF16, device="cuda"))
    r8.codes[:rows * r].view(rows, r).copy_(xc)
    r8.scales[:rows, :blocks].copy_(sx)
    if dgrad:
        y = binding.Fp8Weights(wc.transpose(1, 2).contiguous(), sw.transpose(1, 2).contiguous()).dgrad(r8, lists.offsets)
    else:
        y = binding.Fp8Weights(wc, sw).forward(r8, lists.offsets)
    for i, (a, b) in enumerate(lists.spans):
        for k in range(5):
            mine = kind[a:b] == k
            check(y[a:b][mine], xv[a:b][mine], wv[i].T, blocks)
    assert torch.all(y[kind >= 2] != 0)


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("plan", PLANS)
def test_largest_magnitudes_that_do_not_meet(plan, dgrad):
    """Rows and weights with one element of 2^75 each, at different places of a block: its sum is zero."""
    gen = torch.Generator(device="cuda").manual_seed(22)
    lists = Lists(PLANS[plan])
    x = torch.randn((lists.rows, 400), generator=gen, device="cuda")
    w = torch.randn((lists.groups, 272, 400), generator=gen, device="cuda") * 0.05
    x[::3, 5] = 2.0 ** 75
    w[:, 3, 7] = 2.0 ** 75
    if dgrad:
        w = w.transpose(1, 2).contiguous()
    r8, w8 = binding.Fp8Rows(400).quantize(x), binding.Fp8Weights.quantize(w)
    y = w8.dgrad(r8, lists.offsets) if dgrad else w8.forward(r8, lists.offsets)
    xv, wv = values_of(r8, w8)
    for i, (a, b) in enumerate(lists.spans):
        for outlier in (True, False):
            mine = (torch.arange(a, b, device="cuda") % 3 == 0) == outlier
            for at in (slice(0, 128), slice(128, 272)):
                check(y[a:b, at][mine], xv[a:b][mine], (wv[i] if dgrad else wv[i].T)[:, at], 4)


@pytest.mark.parametrize("plan", PLANS)
def test_rows_do_not_depend_on_their_neighbours_scales(plan):
    """A row under scales whose products are no fp32 numbers leaves the bits of the others as they are."""
    gen = torch.Generator(device="cuda").manual_seed(23)
    lists = Lists(PLANS[plan])
    x = torch.randn((lists.rows, 400), generator=gen, device="cuda")
    w8 = binding.Fp8Weights.quantize(torch.randn((lists.groups, 272, 400), generator=gen, device="cuda") * 2.0 ** -60)
    clean = w8.forward(binding.Fp8Rows(400).quantize(x), lists.offsets)
    odd = torch.arange(lists.rows, device="cuda") % 7 == 3
    x[odd] *= 2.0 ** -75
    y = w8.forward(binding.Fp8Rows(400).quantize(x), lists.offsets)
    assert torch.equal(y[~odd], clean[~odd])


# counts, N, K, type, gap, tail, pad, and the plan that the case is for: groups of one row, chunk edges of 128 and 256 rows, a
# pair whose odd CTA has no row, lists with gaps, more groups than the kernels hold in shared memory
PLAN_CASES = {
    "pairs_edges": ([1, 2, 255, 256, 257, 511, 0, 513], 528, 336, BF16, 0, 0, 0, "pairs"),
    "pairs_fp16_gap": ([129, 0, 600, 400, 31, 1], 1424, 656, FP16, 7, 9, 24, "pairs"),
    "pairs_deep": ([400, 512, 385], 400, 4112, BF16, 0, 3, 0, "pairs"),
    "pairs_skewed": ([900, 1, 0, 2, 40], 256, 128, FP16, 1, 0, 8, "pairs"),
    "pairs_many_groups": ([1 + (i * 37) % 401 for i in range(160)], 144, 80, BF16, 0, 0, 0, "pairs"),
    "single_edges": ([1, 127, 128, 129, 0, 2, 33, 65], 528, 336, BF16, 0, 0, 0, "single"),
    "single_above_256": ([1, 255, 256, 257, 300, 513], 272, 528, FP16, 0, 5, 0, "single"),
    "single_many_groups": ([1 + (i * 37) % 67 for i in range(300)], 144, 80, BF16, 0, 0, 0, "single"),
    "small_edges": ([1, 16, 17, 32, 33, 0, 2, 1], 528, 336, BF16, 0, 0, 0, "small"),
}


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("name", PLAN_CASES)
def test_the_edges_of_every_plan(name, dgrad):
    counts, n, k, dtype, gap, tail, pad, plan = PLAN_CASES[name]
    gen = torch.Generator(device="cuda").manual_seed(len(name))
    lists = Lists(counts, gap, tail)
    assert plan_of(lists.rows, lists.groups) == plan
    x = lists.matrix(gen, n if dgrad else k, dtype, 0, 0.25)
    x.mul_(torch.exp2(torch.randint(-3, 4, (lists.rows, 1), generator=gen, device="cuda")).to(dtype))
    w8 = binding.Fp8Weights.quantize(torch.randn((lists.groups, n, k), generator=gen, device="cuda") * 0.05)
    r8 = binding.Fp8Rows(x.shape[1], lists.rows).quantize(x)
    y = lists.blank(k if dgrad else n, dtype, pad)
    if dgrad:
        w8.dgrad(r8, lists.offsets, lists.counts, dx=y)
    else:
        w8.forward(r8, lists.offsets, lists.counts, y=y)
    assert w8.device_status()[0] == binding.MOE_OK
    xv, wv = values_of(r8, w8)
    for g, (a, b) in enumerate(lists.spans):
        check(y[a:b], xv[a:b], wv[g] if dgrad else wv[g].T, -(-x.shape[1] // 128))
    assert torch.all(y[lists.free] == 7.0)


@pytest.mark.parametrize("plan", PLANS)
def test_nan_stays_in_its_row_and_its_block_of_weights_of_the_input_gradient(plan):
    gen = torch.Generator(device="cuda").manual_seed(24)
    lists = Lists(PLANS[plan])
    dy = torch.randn((lists.rows, 272), generator=gen, device="cuda")
    w = torch.randn((lists.groups, 272, 384), generator=gen, device="cuda")

    def dgrad():
        return binding.Fp8Weights.quantize(w).dgrad(binding.Fp8Rows(272).quantize(dy), lists.offsets)

    clean = dgrad()
    bad, (a, b) = lists.spans[2][0], lists.spans[0]
    dy[bad, 200], w[0, 5, 130] = NAN, -INF
    dx = dgrad()
    assert torch.isnan(dx[bad]).all() and torch.isnan(dx[a:b, 128:256]).all()
    keep = torch.ones_like(dx, dtype=torch.bool)
    keep[bad], keep[a:b, 128:256] = False, False
    assert torch.equal(dx[keep], clean[keep])


def test_every_plan_on_weights_behind_2_to_the_32_elements():
    """The last group's weights, with as many rows behind its list as bring the mean to each plan."""
    groups, n, k, count = 65, 8192, 8192, 307  # (every ninth row is checked)
    gen = torch.Generator(device="cuda").manual_seed(25)
    w = torch.zeros((groups, n, k), dtype=BF16, device="cuda")
    w[-1] = (torch.randn((n, k), generator=gen, device="cuda") * 0.02).to(BF16)
    w8 = binding.Fp8Weights.quantize(w)
    wv = define(w[-1:], 128)[2][0]
    off = torch.tensor([0] * groups + [count], dtype=torch.int32, device="cuda")
    for mean, plan in ((10, "small"), (40, "single"), (200, "pairs")):
        rows = groups * mean
        assert plan_of(rows, groups) == plan
        x = torch.randn((rows, k), generator=gen, device="cuda").to(BF16)
        xv = define(x[:count:9], 1)[2]
        for out, product, width, m in ((torch.full((rows, n), 7.0, dtype=BF16, device="cuda"), w8.forward, k, wv.T),
                                       (torch.full((rows, k), 7.0, dtype=BF16, device="cuda"), w8.dgrad, n, wv)):
            product(binding.Fp8Rows(width, rows).quantize(x), off, None, out)
            check(out[:count:9], xv, m, 64)
            assert torch.all((out[:count] != 7.0).any(1))
            assert torch.all(out[count:] == 7.0)
        assert w8.device_status()[0] == binding.MOE_OK


def test_more_rows_than_a_grid_holds():
    """2,097,190 rows: the quantizer's CTAs walk on to a second tile, the way back to a fourth."""
    rows, k = 65535 * 32 + 70, 16
    gen = torch.Generator(device="cuda").manual_seed(26)
    x = torch.randn((rows, k), generator=gen, device="cuda").to(BF16)
    r8 = binding.Fp8Rows(k, rows).quantize(x)
    for part in (slice(0, 40), slice(65535 * 32 - 20, rows)):
        codes, scales, values = define(x[part], 1)
        assert torch.equal(r8.codes[:rows * k].view(rows, k)[part], codes)
        assert same_bits(r8.scales[:rows, :1][part].contiguous(), scales)
    half = binding.Fp8Rows(k, rows // 2)
    for part in (slice(0, rows // 2), slice(rows // 2, rows)):
        assert torch.equal(half.quantize(x[part]).codes[:rows // 2 * k].view(-1, k), r8.codes[:rows * k].view(rows, k)[part])
        assert torch.equal(half.dequantize(dtype=FP32), r8.dequantize(dtype=FP32)[part])
