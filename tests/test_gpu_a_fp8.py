"""Rows and matrices in 8 bits, and their grouped products, against their definitions in 64 bits.

Codes and scales are compared bit for bit: s = fl(amax / 448), code = E4M3(fl(x / s)), fl one fp32 rounding.

Tolerance of the products.  Two E4M3 values multiply exactly.  Within a block of 128 the tensor core adds four times 32
products to an fp32 accumulator and may cut each of the 33 terms after the last bit of the largest, which is at most the
block's sum of magnitudes: 4 * 33 units of 2^-23 of it.  Blocks are then added in fp32, rounded to nearest (2^-24 each,
relative to the sum S of all magnitudes, as is the product of two scales), and at most 256 partial sums.  The output is
rounded once: half a step, or half a subnormal step (2^-25 for fp16).  So
|err| <= eps/2 |y| + (132 + (blocks + 257) / 2) 2^-23 S + 2^-25.
"""
import pytest
import torch

from mixture_experts_layer_rmsnorm_gb300 import binding
from test_gpu_8_grouped import BF16, FP16, FP32, Lists, half_step

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def e4m3_table():
    """The 127 magnitudes of E4M3 by their codes."""
    v = []
    for c in range(127):
        e, m = c >> 3, c & 7
        v.append((8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def blocks_of(m, height):
    """[blocks, ...] of m [..., rows, K]: the index tuples of every block of `height` x 128."""
    rows, k = m.shape[-2:]
    for r in range(0, rows, height):
        for c in range(0, k, 128):
            yield r // height, c // 128, (..., slice(r, r + height), slice(c, c + 128))


def define(m, height):
    """Codes (uint8), scales [..., ceil(rows / height), ceil(K / 128)] and values (64 bits) of m [..., rows, K]."""
    table = e4m3_table()
    mids = (table[1:] + table[:-1]) / 2
    x = m.double()
    rows, k = m.shape[-2:]
    codes = torch.zeros(m.shape, dtype=torch.uint8, device="cuda")
    scales = torch.zeros((*m.shape[:-2], -(-rows // height), -(-k // 128)), device="cuda")
    values = torch.zeros_like(x)
    for br, bc, at in blocks_of(m, height):
        part = x[at]
        bad = ~torch.isfinite(part).all(-1).all(-1)
        top = part.abs().amax((-2, -1))
        s = (top / 448).float()
        s = torch.where(s > 0, s, torch.ones_like(s))
        s = torch.where(bad, torch.full_like(s, NAN), s)
        q = (part / s.double()[..., None, None]).float().double()
        a = torch.nan_to_num(q.abs()).clamp(max=448.0)
        lo = torch.searchsorted(mids, a, right=False)  # magnitudes at a border go down ...
        tie = (lo < 126) & (a == mids[lo.clamp(max=125)]) & (lo % 2 == 1)
        c = lo + tie  # ... unless the lower code is odd
        c = torch.where(bad[..., None, None], torch.zeros_like(c), c)
        neg = torch.signbit(part) & ~bad[..., None, None]
        codes[at] = (c + 128 * neg).to(torch.uint8)
        scales[..., br, bc] = s
        values[at] = torch.where(neg, -table[c], table[c]) * s.double()[..., None, None]
    return codes, scales, values


def same_bits(got, want):
    return torch.equal(got.view(torch.int32) if got.dtype == FP32 else got,
                       want.view(torch.int32) if want.dtype == FP32 else want)


def spread(gen, shape, dtype):
    """Values of many magnitudes, with quotients that meet the codes' borders."""
    x = torch.randn(shape, generator=gen, device="cuda") * torch.exp(2 * torch.randn(shape, generator=gen, device="cuda"))
    x.view(-1)[::7] = torch.randint(-15, 16, x.view(-1)[::7].shape, generator=gen, device="cuda") * 0.25
    return x.to(dtype)


@pytest.mark.parametrize("rows,k,dtype,pad", [(1, 16, BF16, 0), (3, 128, FP16, 8), (33, 144, FP32, 0), (70, 4112, BF16, 16),
                                              (257, 1024, FP32, 24), (31, 496, FP16, 0), (600, 7168, BF16, 0)])
def test_rows_to_8_bits_and_back(rows, k, dtype, pad):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = spread(gen, (rows, k + pad), dtype)[:, :k]
    x[rows // 2, :16] = 0.0
    x[rows // 2, 3] = -0.0
    r8 = binding.Fp8Rows(k, max_rows=rows + 5)
    assert r8.quantize(x) is r8 and r8.rows == rows
    codes, scales, values = define(x, 1)
    assert torch.equal(r8.codes[:rows * k].view(rows, k), codes)
    assert same_bits(r8.scales[:rows, :scales.shape[1]].contiguous(), scales)
    for out in (BF16, FP16, FP32):
        y = torch.full((rows, k + pad), 7.0, dtype=out, device="cuda")
        assert r8.dequantize(y[:, :k]).data_ptr() == y.data_ptr()
        err = (y[:, :k].double() - values).abs()
        fits = values.abs() < 65000 if out == FP16 else torch.ones_like(values, dtype=torch.bool)
        # the product of code and scale is rounded to fp32, then to the output's type
        lim = values.abs() * (2.0 ** -24 + (half_step(out) if out != FP32 else 0.0) * (1 + 2.0 ** -24))
        lim = lim + (2.0 ** -25 if out == FP16 else 2.0 ** -134 if out == BF16 else 2.0 ** -150)
        assert (err <= lim)[fits].all()
        assert torch.all(y[:, k:] == 7.0)


@pytest.mark.parametrize("g,n,k,dtype", [(1, 16, 16, BF16), (3, 128, 256, FP16), (2, 272, 400, FP32), (5, 112, 1040, BF16)])
def test_matrices_to_8_bits_and_back(g, n, k, dtype):
    gen = torch.Generator(device="cuda").manual_seed(n)
    w = spread(gen, (g, n, k), dtype)
    w[0, :16, :16] = 0.0
    w8 = binding.Fp8Weights.quantize(w)
    codes, scales, values = define(w, 128)
    assert torch.equal(w8.codes, codes) and same_bits(w8.scales, scales)
    assert torch.equal(w8.dequantize(FP32).double(), (values.float()).double())


def test_quotients_next_to_every_border():
    """Codes are decided by x / s rounded to fp32, which the kernel works out from one reciprocal.  Divisors whose
    significand is all ones (which the method's theorem excepts), next to a power of two, and others; dividends at up to four
    steps of fp32 from every border between two codes, and at the borders."""
    gen = torch.Generator().manual_seed(5)
    ones = [(2 - 2.0 ** -23) * 2.0 ** e for e in (-60, -9, 0, 3, 50)]
    others = [1.0, 1 + 2.0 ** -23, 1 - 2.0 ** -24, 4 / 3, *(1 + torch.rand(150, generator=gen)).tolist()]
    table = e4m3_table().cpu()
    mids = (table[1:] + table[:-1]) / 2
    rows = []
    for s in ones + others:
        s = torch.tensor(s, dtype=torch.float32)
        for k in range(-2, 3):  # the largest magnitude that gives this scale
            top = (448 * s.double()).float()
            top = (top.view(torch.int32) + k).view(torch.float32)
            if (top.double() / 448).float() == s:
                break
        else:
            continue
        near = (mids * s.double()).float()
        for k in range(-4, 5):
            row = (near.view(torch.int32) + k).view(torch.float32)
            rows.append(torch.cat([top[None], torch.where(torch.arange(126) % 2 == 1, -row, row), torch.zeros(1)]))
    x = torch.stack(rows).cuda()
    assert x.shape[0] > 9 * 100
    codes, scales, _ = define(x, 1)
    r8 = binding.Fp8Rows(128, max_rows=x.shape[0]).quantize(x)
    assert same_bits(r8.scales[:x.shape[0], :1].contiguous(), scales)
    assert torch.equal(r8.codes[:x.numel()].view(x.shape), codes)


def test_extreme_blocks():
    """Blocks of zeros, of subnormal numbers, near the largest, with a NaN or an infinity."""
    x = torch.zeros((6, 384), device="cuda")
    x[0, :128] = torch.linspace(-1, 1, 128, device="cuda") * 3e38
    x[0, 128:256] = torch.linspace(-1, 1, 128, device="cuda") * 1e-37
    x[0, 256:] = torch.linspace(-1, 1, 128, device="cuda") * 1e-42
    x[1, 5], x[1, 130], x[2, 260] = NAN, INF, -INF
    x[3, 7] = 2.0 ** -149  # (s is 0 in fp32: 1, and the code 0)
    x[4, 100:300] = 448.0
    r8 = binding.Fp8Rows(384, max_rows=6).quantize(x)
    codes, scales, values = define(x, 1)
    assert torch.equal(r8.codes.view(6, 384), codes)
    got = r8.scales[:, :3]
    assert torch.equal(torch.isnan(got), torch.isnan(scales)) and same_bits(got[~torch.isnan(got)], scales[~torch.isnan(scales)])
    y = r8.dequantize(dtype=FP32)
    assert torch.isnan(y[1, :256]).all() and torch.isnan(y[2, 256:]).all() and torch.isfinite(y[2, :256]).all()
    w = torch.cat([x, x.new_zeros((250, 384))]).view(1, 256, 384)
    w8 = binding.Fp8Weights.quantize(w)
    assert torch.isnan(w8.scales[0, 0]).all() and torch.all(w8.scales[0, 1] == 1.0)


# counts, N, K, type, gap, tail, pad: every tile plan, single rows, empty groups, chunk edges (16, 32, 128, 256), sizes that
# are no multiple of a tile or a block, strided outputs, more groups than the shared-memory table holds
CASES = {
    "one": ([1], 16, 16, BF16, 0, 0, 0),
    "row_of_many": ([1], 1008, 4112, FP16, 0, 3, 0),
    "small_edges": ([0, 1, 15, 16, 17, 31, 32, 33, 0, 1, 1, 0], 272, 208, BF16, 0, 0, 8),
    "small_stream_k": ([3, 0, 5, 8, 0, 1, 2, 7], 1024, 2048, BF16, 3, 5, 0),
    "small_fp16_gap": ([9, 12, 0, 0, 31, 2, 1], 400, 1040, FP16, 5, 1, 16),
    "large_edges": ([255, 256, 257, 0, 1, 300, 511, 513], 528, 336, BF16, 0, 0, 0),
    "large_fp16": ([100, 0, 700, 33], 1424, 640, FP16, 7, 9, 24),
    "large_skewed": ([1500, 1, 0, 2, 40], 256, 128, BF16, 1, 0, 0),
    "large_deep": ([250, 190, 70, 130], 384, 4096, BF16, 0, 0, 0),
    "single_edges": ([300, 0, 2, 129, 128, 127, 1, 60, 0, 33], 528, 336, BF16, 0, 0, 0),
    "single_fp16_deep": ([90, 20, 0, 64, 97], 400, 2064, FP16, 3, 1, 8),
    "many_groups": ([(7 * i) % 5 for i in range(300)], 144, 80, BF16, 0, 2, 0),
    "most_groups": ([(i * i) % 61 for i in range(1024)], 64, 64, FP16, 0, 0, 0),
    "some_rows": ([20, 40, 0, 17, 24, 21, 19], 272, 208, BF16, 0, 3, 0),
    "no_rows_at_all": ([0, 0, 0], 128, 64, BF16, 0, 4, 0),
}


def make(name, dgrad=False):
    counts, n, k, dtype, gap, tail, pad = CASES[name]
    gen = torch.Generator(device="cuda").manual_seed(len(name))
    lists = Lists(counts, gap, tail)
    x = lists.matrix(gen, n if dgrad else k, dtype, 0, 0.25 if dgrad else 1.0)
    # (rows of very different magnitudes: their scales are not alike)
    x.mul_(torch.exp2(torch.randint(-3, 4, (lists.rows, 1), generator=gen, device="cuda")).to(dtype))
    w = torch.randn((lists.groups, n, k), generator=gen, device="cuda") * 0.05
    return lists, binding.Fp8Rows(x.shape[1], lists.rows).quantize(x), binding.Fp8Weights.quantize(w), dtype, pad


def check(got, xv, wv, r):
    """got [rows, F] against xv [rows, R] times wv [R, F]."""
    want, s = xv @ wv, xv.abs() @ wv.abs()
    lim = half_step(got.dtype) * want.abs() + (132 + (-(-r // 128) + 257) / 2) * 2.0 ** -23 * s + 2.0 ** -25
    worst = ((got.double() - want).abs() - lim).max().item() if got.numel() else 0.0
    assert worst <= 0, f"error above its bound by {worst:.3e}"


def values_of(rows8, weights8):
    return rows8.dequantize(dtype=FP32).double(), weights8.dequantize(FP32).double()


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    lists, r8, w8, dtype, pad = make(name)
    y = lists.blank(w8.N, dtype, pad)
    assert w8.forward(r8, lists.offsets, lists.counts, y=y) is y
    assert w8.device_status()[0] == binding.MOE_OK
    xv, wv = values_of(r8, w8)
    for g, (a, b) in enumerate(lists.spans):
        check(y[a:b], xv[a:b], wv[g].T, w8.K)
    assert torch.all(y[lists.free] == 7.0)


@pytest.mark.parametrize("name", CASES)
def test_input_gradient(name):
    lists, r8, w8, dtype, pad = make(name, dgrad=True)
    dx = lists.blank(w8.K, dtype, pad)
    assert w8.dgrad(r8, lists.offsets, lists.counts, dx=dx) is dx
    assert w8.device_status()[0] == binding.MOE_OK
    xv, wv = values_of(r8, w8)
    for g, (a, b) in enumerate(lists.spans):
        check(dx[a:b], xv[a:b], wv[g], w8.N)
    assert torch.all(dx[lists.free] == 7.0)


@pytest.mark.parametrize("rows", [6, 99, 399])
def test_equal_groups_without_lists(rows):
    gen = torch.Generator(device="cuda").manual_seed(3)
    w8 = binding.Fp8Weights.quantize(torch.randn((3, 144, 272), generator=gen, device="cuda"))
    x8 = binding.Fp8Rows(272).quantize(torch.randn((rows, 272), generator=gen, device="cuda"))
    d8 = binding.Fp8Rows(144).quantize(torch.randn((rows, 144), generator=gen, device="cuda"))
    y, dx = w8.forward(x8, dtype=FP16), w8.dgrad(d8)
    (xv, wv), (dv, _) = values_of(x8, w8), values_of(d8, w8)
    n = rows // 3
    for g in range(3):
        at = slice(g * n, g * n + n)
        check(y[at], xv[at], wv[g].T, 272)
        check(dx[at], dv[at], wv[g], 144)


@pytest.mark.parametrize("counts", [[3, 2, 4], [40, 21, 64], [300, 150, 200]])
def test_nan_stays_in_its_row_and_its_block_of_weights(counts):
    lists = Lists(counts)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((lists.rows, 384), generator=gen, device="cuda")
    w = torch.randn((3, 272, 384), generator=gen, device="cuda")
    clean = binding.Fp8Weights.quantize(w).forward(binding.Fp8Rows(384).quantize(x), lists.offsets)
    bad = lists.spans[1][0]
    x[bad, 300], w[2, 130, 5] = INF, NAN
    y = binding.Fp8Weights.quantize(w).forward(binding.Fp8Rows(384).quantize(x), lists.offsets)
    a, b = lists.spans[2]
    assert torch.isnan(y[bad]).all() and torch.isnan(y[a:b, 128:256]).all()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[bad], keep[a:b, 128:256] = False, False
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("offsets,counts,group", [([0, 10, 8, 30], None, 1), ([-1, 10, 20, 30], None, 0),
                                                  ([0, 10, 20, 41], None, 2), ([0, 10, 20, 30], [10, 11, 3], 1)])
def test_bad_lists_write_nothing_and_are_reported(offsets, counts, group):
    w8 = binding.Fp8Weights.quantize(torch.ones((3, 64, 64), device="cuda"))
    x8 = binding.Fp8Rows(64).quantize(torch.ones((40, 64), device="cuda"))
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    out = torch.full((40, 64), 7.0, dtype=BF16, device="cuda")
    for call in (lambda: w8.forward(x8, off, cnt, y=out), lambda: w8.dgrad(x8, off, cnt, dx=out)):
        call()
        st, detail = w8.device_status()
        assert st == binding.MOE_ERR_DEVICE and detail[1] == 9 and detail[2] == group
        assert torch.all(out == 7.0)
    good = torch.tensor([0, 10, 20, 30], dtype=torch.int32, device="cuda")
    w8.forward(x8, good, y=out)  # the next call clears the error
    assert w8.device_status()[0] == binding.MOE_OK and torch.all(out[:30] == 64.0)


@pytest.mark.parametrize("counts", [[5, 0, 9, 2], [100, 0, 90, 64], [300, 0, 190, 264]])
def test_calls_repeat_bit_for_bit_and_replay_from_a_graph_on_new_rows_and_lists(counts):
    lists = Lists(counts)
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn((lists.rows, 1024), generator=gen, device="cuda").to(BF16)
    dy = torch.randn((lists.rows, 512), generator=gen, device="cuda").to(BF16)
    w8 = binding.Fp8Weights.quantize(torch.randn((4, 512, 1024), generator=gen, device="cuda"))
    x8, d8 = binding.Fp8Rows(1024, lists.rows), binding.Fp8Rows(512, lists.rows)
    off, y, dx = lists.offsets.clone(), torch.zeros_like(dy), torch.zeros_like(x)

    def step():
        w8.forward(x8.quantize(x), off, y=y)
        w8.dgrad(d8.quantize(dy), off, dx=dx)

    step()
    first = [t.clone() for t in (y, dx)]
    step()
    assert all(torch.equal(a, b) for a, b in zip(first, (y, dx)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    n = lists.rows
    off.copy_(torch.tensor([0, 0, n - 4, n, n], dtype=torch.int32))
    x.mul_(-0.75)
    dy.add_(0.25)
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in (y, dx)]
    step()
    assert all(torch.equal(a, b) for a, b in zip(replayed, (y, dx)))
    assert not torch.equal(y, first[0])


def test_updated_weights_in_their_buffers():
    """An optimizer's step between two replays: the graph's product reads the new weights."""
    gen = torch.Generator(device="cuda").manual_seed(12)
    w = torch.randn((3, 144, 272), generator=gen, device="cuda")
    w8, r8 = binding.Fp8Weights.quantize(w), binding.Fp8Rows(272, 40)
    x, off = torch.randn((40, 272), generator=gen, device="cuda").to(BF16), torch.tensor([0, 9, 9, 40], dtype=torch.int32, device="cuda")
    y = w8.forward(r8.quantize(x), off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        w8.update(w)
        w8.forward(r8.quantize(x), off, y=y)
    w.mul_(-1.5).add_(0.01)
    graph.replay()
    fresh = binding.Fp8Weights.quantize(w)
    assert torch.equal(y, fresh.forward(r8, off))
    w.add_(0.25)
    kept = w8.codes.data_ptr()
    assert w8.update(w.to(BF16)) is w8 and w8.codes.data_ptr() == kept
    codes, scales, _ = define(w.to(BF16), 128)
    assert torch.equal(w8.codes, codes) and same_bits(w8.scales, scales)
    with pytest.raises(ValueError):
        w8.update(w[:2])
    with pytest.raises(ValueError):
        w8.update(w.transpose(1, 2).contiguous().transpose(1, 2))


def test_more_rows_get_larger_buffers_and_a_refused_call_keeps_them():
    r8 = binding.Fp8Rows(64, max_rows=4)
    x = torch.randn((9, 64), device="cuda")
    first = r8.quantize(x[:4]).codes
    assert r8.quantize(x).codes is not first and r8.max_rows >= 9
    assert torch.equal(r8.dequantize(dtype=FP32)[:4], binding.Fp8Rows(64).quantize(x[:4]).dequantize(dtype=FP32))
    with pytest.raises(TypeError):
        r8.quantize(x.double())
    assert r8.rows == 9


def test_objects_refuse_what_does_not_fit():
    w8 = binding.Fp8Weights.quantize(torch.ones((2, 32, 64), device="cuda"))
    x8 = binding.Fp8Rows(64).quantize(torch.ones((4, 64), device="cuda"))
    with pytest.raises(ValueError):
        w8.dgrad(x8)  # rows of K, not N
    with pytest.raises(binding.MoeError):
        w8.forward(binding.Fp8Rows(64).quantize(torch.ones((3, 64), device="cuda")))  # 3 rows, 2 equal groups
    with pytest.raises(binding.MoeError):
        binding.Fp8Rows(24)
    with pytest.raises(ValueError):
        binding.Fp8Weights(w8.codes, w8.scales[:1])
    with pytest.raises(TypeError):
        w8.forward(x8, y=torch.empty((4, 32), dtype=torch.int32, device="cuda"))
    with pytest.raises(binding.MoeError):
        w8.forward(x8, dtype=FP32)
    y = w8.forward(binding.Fp8Rows(64).quantize(torch.ones((0, 64), device="cuda")))
    assert y.shape == (0, 32) and w8.device_status()[0] == binding.MOE_OK


def test_rows_and_weights_behind_2_to_the_32_elements():
    """Sources, codes, weights and results whose offsets pass 32 bits: the last rows, and the last group's product."""
    rows, k, n = 2 ** 19 + 40, 8208, 144
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.zeros((rows, k), dtype=BF16, device="cuda")
    x[-70:] = torch.randn((70, k), generator=gen, device="cuda").to(BF16)
    r8 = binding.Fp8Rows(k, rows).quantize(x)
    codes, scales, values = define(x[-70:], 1)
    assert torch.equal(r8.codes[:rows * k].view(rows, k)[-70:], codes)
    assert same_bits(r8.scales[rows - 70:rows, :scales.shape[1]].contiguous(), scales)
    out = torch.full((rows, 8216), 7.0, dtype=BF16, device="cuda")
    r8.dequantize(out[:, :k])
    assert ((out[-70:, :k].double() - values).abs() <= values.abs() * (2.0 ** -8 * (1 + 2.0 ** -24) + 2.0 ** -24)).all()
    assert torch.all(out[0, :k] == 0.0) and torch.all(out[-70:, k:] == 7.0)
    w = (torch.randn((1, n, k), generator=gen, device="cuda") * 0.02).to(BF16)
    w8 = binding.Fp8Weights.quantize(w)
    wv = define(w, 128)[2][0]
    y = w8.forward(r8, y=out[:, -n:])
    check(y[-70:], values, wv.T, k)
    assert torch.all(y[:-70] == 0.0)
    del x, r8, out, y
    groups, n, k = 65, 8192, 8192
    w = torch.zeros((groups, n, k), dtype=BF16, device="cuda")
    w[-1] = (torch.randn((n, k), generator=gen, device="cuda") * 0.02).to(BF16)
    w8 = binding.Fp8Weights.quantize(w)
    wv = define(w[-1:], 128)[2][0]
    assert torch.all(w8.codes[-2] == 0)
    for count in (3, 40, 300):
        x = torch.randn((count, k), generator=gen, device="cuda").to(BF16)
        off = torch.tensor([0] * groups + [count], dtype=torch.int32, device="cuda")
        y = w8.forward(binding.Fp8Rows(k, count).quantize(x), off)
        xv = define(x, 1)[2]
        check(y, xv, wv.T, k)
        check(w8.dgrad(binding.Fp8Rows(n, count).quantize(x), off), xv, wv, n)
    back = w8.dequantize(BF16)
    assert torch.all(back[:-1] == 0.0) and torch.equal(back[-1], wv.float().to(BF16))
