"""Rows in 4 bits and their grouped product, against the formats' definitions.

The quantizer and its inverse are whole-number decisions and single roundings of
fp32 steps that numpy repeats (IEEE division and products): codes and scales are equal,
the values differ by no more than their one rounding.  The product of two E2M1
codes and two block scales is exact in fp32 (2 + 2 bits; NVFP4 4 + 4 more); sums
as in the 16-bit grouped products: a step of K = 64 cuts at most 65 terms after
the last bit of the largest, 65 * 2^-23 S per 64 terms with S = sum |a||b|, one
rounding per stream-K partial sum, three for NVFP4's fp32 scales (their product,
its product with the sum), and half a step of the output.
"""
import numpy as np
import pytest
import torch

from mixture_experts_layer_rmsnorm_gb300 import binding

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
BLOCK = {"mx": 32, "nv": 16}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float32)
E4M3 = np.array([(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)) for e in range(16) for m in range(8)][:127],
                np.float32)


def nearest(table, v):
    """Index of the nearest table entry, ties to the even index, the last beyond it (values >= 0)."""
    hi = np.clip(np.searchsorted(table, v), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = v.astype(np.float64) - table[lo], table[hi].astype(np.float64) - v
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def quantise(x, fmt, per_group):
    """Codes, scale bytes and (nv) fp32 scales of one group's rows, step by step in fp32; x: float32 [rows, K]."""
    rows, k = x.shape
    b = x.reshape(rows, k // BLOCK[fmt], BLOCK[fmt])
    amax = np.abs(b).max(2)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        if fmt == "mx":
            e = np.where(amax > 0, np.frexp(amax)[1] - 3, -127).clip(-127, 127)
            s, g = (e + 127).astype(np.uint8), None
            q = np.ldexp(b.astype(np.float64), -e[..., None])
        else:
            top = np.full(rows, amax.max(initial=0.0), np.float32) if per_group else amax.max(1)
            g = np.where(top > 0, top / np.float32(2688), np.float32(1)).astype(np.float32)
            u = amax / (np.float32(6) * g)[:, None]
            s = np.where(np.isnan(u), 0, nearest(E4M3, np.minimum(np.nan_to_num(u, posinf=448), 448))).astype(np.uint8)
            d = (E4M3[s] * g[:, None]).astype(np.float32)[..., None]
            q = np.where(d > 0, b / d, np.float32(0))
    c = nearest(E2M1, np.abs(q)).astype(np.uint8) | (np.signbit(q).astype(np.uint8) << 3)
    return c.reshape(rows, k), s, g


def values(c, s, g, fmt):
    """What codes stand for, in 64 bits."""
    v = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7].astype(np.float64)
    f = np.ldexp(1.0, s.astype(int) - 127) if fmt == "mx" else E4M3[s].astype(np.float64) * g[:, None].astype(np.float64)
    return v * np.repeat(f, BLOCK[fmt], axis=1)


class Lists:
    def __init__(self, counts, gap=0, tail=0, equal=False):
        off = np.concatenate([[0], np.cumsum([c + gap for c in counts])])
        self.spans = [(int(o), int(o + c)) for o, c in zip(off, counts)]
        self.rows, self.groups, self.equal = int(off[-1]) + tail, len(counts), equal
        self.offsets = None if equal else torch.tensor(off, dtype=torch.int32, device="cuda")
        self.counts = torch.tensor(counts, dtype=torch.int32, device="cuda") if gap else None
        self.free = np.ones(self.rows, bool)
        for a, b in self.spans:
            self.free[a:b] = False

    def tile_row(self, g):
        if self.equal:
            return g * (-(-(self.rows // self.groups) // 128))
        return self.spans[g][0] // 128 + g


def unpack(codes, rows, k):
    p = codes[:rows * k // 2].cpu().numpy().reshape(rows, k // 2)
    return np.stack([p & 15, p >> 4], axis=2).reshape(rows, k)


def scale_of(scales, lists, g, n, k, fmt):
    """The scale bytes [n, blocks] of group g from the tiles; bytes of blocks past K in whole chunks must be zero."""
    blocks, chunks = k // BLOCK[fmt], -(-k // (4 * BLOCK[fmt]))
    tiles = -(-n // 128)
    t0 = lists.tile_row(g)
    raw = scales.cpu().numpy()[t0 * chunks * 512:(t0 + tiles) * chunks * 512].reshape(tiles, chunks, 32, 4, 4)
    flat = raw.transpose(0, 3, 2, 1, 4).reshape(tiles * 128, chunks * 4)[:n]
    assert not flat[:, blocks:].any()
    return flat[:, :blocks]


def hard_rows(rng, rows, k, dtype):
    """Values over many binades, zeros, signed zeros, exact ties of every code, the type's extremes."""
    x = rng.standard_normal((rows, k)) * np.exp2(rng.integers(-6, 7, (rows, k // 16)).repeat(16, axis=1))
    x[rng.random((rows, k)) < 0.05] = 0.0
    x = torch.tensor(x).to(dtype)
    ties = torch.tensor([6.0, 0.25, -0.25, 0.75, 1.25, -1.75, 2.5, 3.5, 5.0, -5.0, 0.0, -0.0, 4.0, 1.0, 0.5, -6.0])
    x[0, :16] = ties.to(dtype)
    if k >= 64:
        x[0, 32:64] = 0.0
        x[-1, :16] = torch.finfo(dtype).tiny
        x[-1, 16:32] = torch.finfo(dtype).smallest_normal * 8
    if k >= 96:  # a block of subnormals alone
        x[-1, 64:96] = torch.arange(32).to(dtype) * (torch.finfo(dtype).smallest_normal / 32)
    if rows > 2:
        x[1] = 0.0
    return x


CASES = {
    "one_block": ([1], 32, 0, 0, False),
    "lists": ([0, 5, 130, 1, 0, 128, 127], 352, 0, 0, False),
    "gaps": ([33, 0, 256, 3], 1024, 13, 7, False),
    "equal": ([72, 72, 72], 160, 0, 0, True),
    "wide": ([3, 2], 8224, 0, 0, False),
    "wider_than_held": ([2, 0, 1], 20512, 5, 1, False),
    "many_groups": ([i % 4 for i in range(700)], 96, 1, 0, False),
}


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=str)
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("name", CASES)
def test_quantise_and_back(name, fmt, dtype):
    counts, k, gap, tail, equal = CASES[name]
    lists = Lists(counts, gap, tail, equal)
    rng = np.random.default_rng(len(name))
    x = torch.full((lists.rows, k), float("nan"), dtype=dtype)
    for a, b in lists.spans:
        if b > a:
            x[a:b] = hard_rows(rng, b - a, k, dtype)
    wide = torch.zeros((lists.rows, k + 16), dtype=dtype, device="cuda")
    wide[:, :k] = x.cuda()
    r4 = binding.Fp4Rows(fmt, k, lists.groups, lists.rows)
    r4.codes.fill_(0xAA)
    r4.quantize(wide[:, :k], lists.offsets, lists.counts)
    codes = unpack(r4.codes, lists.rows, k)
    assert (codes[lists.free] == 0xA).all()  # rows of no group are left alone
    back = {}
    for out in (BF16, FP16, FP32):
        y = torch.full((lists.rows, k + 8), 7.0, dtype=out, device="cuda")[:, :k]
        r4.dequantize(lists.offsets, lists.counts, y=y)
        back[out] = y
        assert (y.cpu()[lists.free] == 7.0).all()
    for g, (a, b) in enumerate(lists.spans):
        if a == b:
            continue
        c, s, gs = quantise(x[a:b].float().numpy(), fmt, False)
        assert np.array_equal(scale_of(r4.scales, lists, g, b - a, k, fmt), s)
        if fmt == "nv":
            assert np.array_equal(r4.gscale[a:b].cpu().numpy(), gs)
            zero = np.repeat(E4M3[s] * gs[:, None] == 0, 16, axis=1)
            c = np.where(zero, 0, c)
        assert np.array_equal(codes[a:b], c)
        want = torch.tensor(values(c, s, gs, fmt))
        for out, y in back.items():
            got = y[a:b].cpu().double()
            over = want.abs() > torch.finfo(out).max  # beyond the type: infinity
            tiny = torch.finfo(out).smallest_normal * torch.finfo(out).eps / 2
            # (code * s) * g in fp32, then the type: two roundings for 16 bits, one for 32
            rel = torch.finfo(out).eps / 2 + (2.0 ** -24 if out != FP32 else 0.0)
            assert ((got - want).abs() <= want.abs() * rel * (1 + 2.0 ** -20) + tiny)[~over].all()
            assert (got[over].abs() >= torch.finfo(out).max).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_weights_with_one_scale_per_matrix(fmt):
    rng = np.random.default_rng(2)
    w = torch.stack([hard_rows(rng, 200, 288, BF16) * 2.0 ** i for i in (0, -3, 5)]).to(BF16)
    w[2] = 0.0
    w4 = binding.Fp4Weights.quantize(w.cuda(), fmt)
    lists = Lists([200] * 3, equal=True)
    codes = unpack(w4.codes.view(-1), 600, 288).reshape(3, 200, 288)
    for g in range(3):
        c, s, gs = quantise(w[g].float().numpy(), fmt, True)
        assert np.array_equal(scale_of(w4.scales, lists, g, 200, 288, fmt), s)
        if fmt == "nv":
            assert w4.gscale[g].item() == gs[0]
            c = np.where(np.repeat(E4M3[s] * gs[:, None] == 0, 16, axis=1), 0, c)
        assert np.array_equal(codes[g], c)
        want = values(c, s, gs, fmt)
        assert np.abs(w4.dequantize(FP32)[g].cpu().double().numpy() - want).max() <= 2.0 ** -24 * np.abs(want).max()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_division_near_the_borders_of_codes(fmt):
    """Rows whose quotients lie on and next to the borders between codes, at many scales."""
    rng = np.random.default_rng(9)
    k = 4096
    x = np.empty((64, k), np.float32)
    for r in range(64):
        big = np.float32(rng.uniform(1, 2) * 2.0 ** rng.integers(-20, 20))
        x[r] = big
        g = np.float32(big / np.float32(2688))
        d = np.float32(448) * g if fmt == "nv" else np.float32(2.0 ** (np.frexp(big)[1] - 3))
        border = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)[rng.integers(0, 7, k)]
        at = (border * d).astype(np.float32)
        for _ in range(3):
            at = np.where(rng.random(k) < 0.5, np.nextafter(at, np.float32(np.inf)), np.nextafter(at, np.float32(0)))
        x[r] = at * np.where(rng.random(k) < 0.5, -1, 1)
        x[r, ::BLOCK[fmt]] = big
    r4 = binding.Fp4Rows(fmt, k, 1, 64).quantize(torch.tensor(x).cuda())
    c, s, gs = quantise(x, fmt, False)
    assert np.array_equal(unpack(r4.codes, 64, k), c)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_nan_and_infinity_become_nan(fmt):
    x = torch.ones((3, 64), device="cuda")
    x[1, 5], x[2, 40] = float("nan"), float("-inf")
    y = binding.Fp4Rows(fmt, 64, 1, 3).quantize(x).dequantize(dtype=FP32)
    assert torch.equal(y[0], x[0])
    if fmt == "nv":
        assert torch.isnan(y[1:]).all()
    else:
        assert torch.isnan(y[1, :32]).all() and torch.isnan(y[2, 32:]).all()
        assert torch.equal(y[1, 32:], x[1, 32:]) and torch.equal(y[2, :32], x[2, :32])


GEMMS = {
    # counts, N, K, gap, tail, equal
    "one": ([1], 8, 32, 0, 0, False),
    "small": ([0, 1, 15, 16, 17, 31, 32, 33, 0, 2], 264, 544, 0, 0, False),
    "small_stream_k": ([3, 0, 9, 12], 1032, 4096, 5, 3, False),
    "small_deep_group": ([300] + [0] * 30, 136, 320, 0, 0, False),
    "some_rows": ([20, 40, 0, 17, 24, 21, 19], 264, 544, 0, 0, False),
    "some_rows_whole_wave": ([19 + i % 5 for i in range(76)], 72, 2080, 0, 3, False),
    "large": ([255, 256, 257, 0, 1, 129, 511], 520, 288, 0, 0, False),
    "large_gap": ([100, 700, 0, 33], 776, 1152, 9, 40, False),
    "large_k64": ([300, 20], 256, 64, 0, 0, False),
    "equal": ([130, 130, 130], 384, 416, 0, 0, True),
    "many_groups": ([(5 * i) % 7 for i in range(300)], 72, 96, 0, 2, False),
}


@pytest.mark.parametrize("out", [BF16, FP16], ids=str)
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("name", GEMMS)
def test_product(name, fmt, out):
    counts, n, k, gap, tail, equal = GEMMS[name]
    lists = Lists(counts, gap, tail, equal)
    gen = torch.Generator(device="cuda").manual_seed(len(name))
    x = torch.randn((lists.rows, k), generator=gen, device="cuda").to(BF16)
    # the binade changes from block to block: a scale in the wrong place shows
    x *= torch.exp2(torch.randint(-3, 4, (lists.rows, k // 16), generator=gen, device="cuda")).repeat_interleave(16, 1).to(BF16)
    x[torch.tensor(lists.free, device="cuda")] = float("nan")
    w = (torch.randn((lists.groups, n, k), generator=gen, device="cuda") * 0.05).to(BF16)
    w *= torch.exp2(torch.randint(-3, 4, (lists.groups, n, k // 16), generator=gen, device="cuda")).repeat_interleave(16, 2).to(BF16)
    r4 = binding.Fp4Rows(fmt, k, lists.groups, lists.rows)
    r4.codes.fill_(0x77)
    r4.scales.fill_(0xFF)  # what the quantizer leaves alone may hold anything
    r4.quantize(x, lists.offsets, lists.counts)
    w4 = binding.Fp4Weights.quantize(w, fmt)
    y = torch.full((lists.rows, n + 8), 7.0, dtype=out, device="cuda")[:, :n]
    w4.forward(r4, lists.offsets, lists.counts, y=y)
    assert w4.device_status()[0] == binding.MOE_OK
    xv = r4.dequantize(lists.offsets, lists.counts, dtype=FP32).double()
    wv = w4.dequantize(FP32).double()
    for g, (a, b) in enumerate(lists.spans):
        if a == b:
            continue
        want, s = xv[a:b] @ wv[g].T, xv[a:b].abs() @ wv[g].abs().T
        # (the dequantized values carry one fp32 rounding each: 2 * 2^-24 S)
        lim = (torch.finfo(out).eps / 2 * want.abs() + (65 / 64 * (k + 64) + 256 + 8) * 2.0 ** -23 * s + 2.0 ** -25)
        err = (y[a:b].double() - want).abs()
        assert (err <= lim).all(), f"{(err - lim).max().item():.3e} above the bound"
    assert (y.cpu()[lists.free] == 7.0).all()
    again = y.clone()
    w4.forward(r4, lists.offsets, lists.counts, y=y)
    assert torch.equal(again, y)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_nan_rows_stay_rows_and_bad_lists_write_nothing(fmt):
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((50, 128), generator=gen, device="cuda").to(BF16)
    w = torch.randn((2, 136, 128), generator=gen, device="cuda").to(BF16)
    off = torch.tensor([0, 20, 50], dtype=torch.int32, device="cuda")
    w4 = binding.Fp4Weights.quantize(w, fmt)
    clean = w4.forward(binding.Fp4Rows(fmt, 128, 2).quantize(x, off), off)
    x[21, 100] = float("nan")
    r4 = binding.Fp4Rows(fmt, 128, 2).quantize(x, off)
    y = w4.forward(r4, off)
    keep = torch.arange(50, device="cuda") != 21
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[21]).all()
    bad = torch.tensor([0, 60, 50], dtype=torch.int32, device="cuda")
    binding.Fp4Rows(fmt, 128, 2).quantize(x, bad)  # in bounds whatever the lists say
    y.fill_(7.0)
    w4.forward(r4, bad, y=y)
    st, detail = w4.device_status()
    assert st == binding.MOE_ERR_DEVICE and detail[1] == 9 and (y == 7.0).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_replay_from_a_graph_on_new_rows_and_lists(fmt):
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((40, 256), generator=gen, device="cuda").to(BF16)
    w4 = binding.Fp4Weights.quantize(torch.randn((3, 200, 256), generator=gen, device="cuda").to(BF16), fmt)
    off = torch.tensor([0, 9, 9, 40], dtype=torch.int32, device="cuda")
    r4, y = binding.Fp4Rows(fmt, 256, 3, 40), torch.zeros((40, 200), dtype=BF16, device="cuda")

    def step():
        w4.forward(r4.quantize(x, off), off, y=y)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(torch.randn((40, 256), generator=gen, device="cuda"))
    off.copy_(torch.tensor([0, 1, 30, 40], dtype=torch.int32))
    graph.replay()
    replayed = y.clone()
    step()
    assert torch.equal(replayed, y)


def test_group_scales_over_listed_groups_and_fp16_rows():
    """One NVFP4 scale per listed group through the C entry point: empty groups get 1, rows of no group take no part."""
    lists = Lists([3, 0, 40], gap=2, tail=1)
    k = 96
    rng = np.random.default_rng(5)
    x = torch.full((lists.rows, k), float("inf"), dtype=FP16)
    for a, b in lists.spans:
        if b > a:
            x[a:b] = hard_rows(rng, b - a, k, FP16)
    xd = x.cuda()
    s = binding.fp4_shape(binding.MOE_FORMAT_NVFP4, 3, lists.rows, k)
    _, (n_codes, n_scales) = binding.moe_fp4_sizes(s)
    codes, scales = (torch.zeros(n, dtype=torch.uint8, device="cuda") for n in (n_codes, n_scales))
    gscale = torch.zeros(3, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    args = (lists.offsets.data_ptr(), lists.counts.data_ptr())
    assert binding.moe_fp4_quantize(s, binding.MOE_TYPE_FP16, xd.data_ptr(), k, *args, codes.data_ptr(), scales.data_ptr(),
                                    gscale.data_ptr(), binding.MOE_SCALE_PER_GROUP, stream) == binding.MOE_OK
    y = torch.zeros((lists.rows, k), device="cuda")
    assert binding.moe_fp4_dequantize(s, codes.data_ptr(), scales.data_ptr(), gscale.data_ptr(),
                                      binding.MOE_SCALE_PER_GROUP, *args, binding.MOE_TYPE_FP32, y.data_ptr(), k,
                                      stream) == binding.MOE_OK
    assert gscale[1].item() == 1.0
    for g, (a, b) in enumerate(lists.spans):
        if b > a:
            c, sc, gs = quantise(x[a:b].float().numpy(), "nv", True)
            assert gscale[g].item() == gs[0]
            c = np.where(np.repeat(E4M3[sc] * gs[:, None] == 0, 16, axis=1), 0, c)
            assert np.array_equal(unpack(codes, lists.rows, k)[a:b], c)
            want = values(c, sc, gs, "nv")
            assert np.abs(y[a:b].cpu().double().numpy() - want).max() <= 2.0 ** -24 * np.abs(want).max()


def test_rows_are_as_the_layers_weight_quantizer_makes_them():
    """w2 of the layer and the same matrix as groups of rows: the same codes and scale bytes (K a multiple of 128)."""
    E, H, I = 3, 256, 384
    gen = torch.Generator(device="cuda").manual_seed(2)
    w2 = (torch.randn((E, H, I), generator=gen, device="cuda") * 0.02).to(BF16)
    w13 = (torch.randn((E, 2 * I, H), generator=gen, device="cuda") * 0.02).to(BF16)
    layer = binding.MoeLayer(torch.ones(H, dtype=BF16, device="cuda"), torch.zeros((E, H), device="cuda"), w13, w2, 1)
    layer.quantize_mxfp4()
    layer.quantize_nvfp4()
    mx, nv = binding.Fp4Weights.quantize(w2, "mx"), binding.Fp4Weights.quantize(w2, "nv")
    assert torch.equal(mx.codes.view(-1), layer.w2_codes4) and torch.equal(nv.codes.view(-1), layer.w2_codes_nv)
    n = layer.w2_scales4.numel()
    assert torch.equal(mx.scales[:n], layer.w2_scales4) and torch.equal(nv.gscale, layer.w2_gscale_nv)
    n = layer.w2_scales_nv.numel()
    assert torch.equal(nv.scales[:n], layer.w2_scales_nv)


@pytest.mark.parametrize("counts", [[5, 0, 7], [300, 20, 0]], ids=["few", "many"])
@pytest.mark.parametrize("ex,ew", [(-63, -60), (-80, -38), (-113, 43), (66, 63), (113, -100), (83, 80)])
def test_scales_whose_product_leaves_the_range(ex, ew, counts):
    """NVFP4's two fp32 scales may multiply to less or more than fp32 holds where the results do not.  Inputs shifted by
    powers of two (normal ones: 2^-113 times randn's values above 2^-13; smaller ones have the code 0) have the same
    codes and block scales, and every scale and rounding of the product shifts with them: equal results, but for a
    step of the subnormal ones (half for each of the two roundings)."""
    n, k = 72, 128
    lists = Lists(counts)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, w = (torch.randn(s, generator=gen, device="cuda").to(BF16) for s in ((lists.rows, k), (3, n, k)))
    x[0] = 0.0
    x[1, :64], x[1, 64:], w[:, 0, :64], w[:, 0, 64:] = 0.0, 1.0, 1.0, 0.0  # a sum of zeros

    def run(a, b):
        return binding.Fp4Weights.quantize(b, "nv").forward(binding.Fp4Rows("nv", k, 3).quantize(a, lists.offsets),
                                                            lists.offsets)

    want = run(x, w).double() * 2.0 ** (ex + ew)
    got = run((x.float() * 2.0 ** ex).to(BF16), (w.float() * 2.0 ** ew).to(BF16)).double()
    top = torch.finfo(BF16).max
    assert (got[0] == 0).all() and got[1, 0] == 0
    inside, over = want.abs() <= top, want.abs() > top * (1 + 2.0 ** -8)
    assert ((got - want).abs()[inside] <= 2.0 ** -133).all()
    assert torch.isinf(got[over]).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_a_captured_graph_outlives_larger_buffers(fmt):
    """The buffers a graph was captured with are nobody else's after the object has grown."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn((100, 256), generator=gen, device="cuda").to(BF16)
    w4 = binding.Fp4Weights.quantize(torch.randn((2, 64, 256), generator=gen, device="cuda").to(BF16), fmt)
    off = torch.tensor([0, 40, 100], dtype=torch.int32, device="cuda")
    r4, y = binding.Fp4Rows(fmt, 256, 2, 100), torch.zeros((100, 64), dtype=BF16, device="cuda")
    w4.forward(r4.quantize(x, off), off, y=y)
    want = y.clone()
    held = {t.data_ptr(): t.numel() for t in (r4.codes, r4.scales)}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.forward(r4.quantize(x, off), off, y=y)
    more = torch.randn((1000, 256), generator=gen, device="cuda").to(BF16)
    off_more = torch.tensor([0, 900, 1000], dtype=torch.int32, device="cuda")
    w4.forward(r4.quantize(more, off_more), off_more)
    others = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in held.values() for _ in range(8)]
    assert not any(t.data_ptr() in held for t in others)
    y.zero_()
    graph.replay()
    assert torch.equal(y, want) and not any(t.any() for t in others)


def test_rows_and_product_take_the_same_kind_of_lists():
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    x, w = torch.ones((6, 64), dtype=BF16, device="cuda"), torch.ones((2, 8, 64), dtype=BF16, device="cuda")
    w4 = binding.Fp4Weights.quantize(w, "nv")
    listed, equal = (binding.Fp4Rows("nv", 64, 2).quantize(x, o) for o in (off, None))
    assert (w4.forward(listed, off) == 64).all() and (w4.forward(equal) == 64).all()
    for bad in (lambda: w4.forward(listed), lambda: w4.forward(equal, off), lambda: listed.dequantize(),
                lambda: equal.dequantize(off)):
        with pytest.raises(ValueError):
            bad()


def test_a_product_without_rows_reports_nothing_of_earlier_calls():
    x, w = torch.ones((6, 64), dtype=BF16, device="cuda"), torch.ones((2, 8, 64), dtype=BF16, device="cuda")
    bad = torch.tensor([0, 9, 6], dtype=torch.int32, device="cuda")
    w4 = binding.Fp4Weights.quantize(w, "mx")
    w4.workspace.fill_(0xFF)
    assert w4.device_status()[0] == binding.MOE_OK
    w4.forward(binding.Fp4Rows("mx", 64, 2).quantize(x, bad), bad)
    assert w4.device_status()[0] == binding.MOE_ERR_DEVICE
    assert w4.forward(binding.Fp4Rows("mx", 64, 2).quantize(x[:0], bad), bad).shape == (0, 8)
    assert w4.device_status()[0] == binding.MOE_OK


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_equal_groups_filled_in_part(fmt):
    """counts without offsets: the rows behind a group's count are skipped, their NaN reach nothing."""
    gen = torch.Generator(device="cuda").manual_seed(10)
    x = torch.randn((4 * 150, 96), generator=gen, device="cuda").to(BF16)
    w4 = binding.Fp4Weights.quantize(torch.randn((4, 72, 96), generator=gen, device="cuda").to(BF16), fmt)
    full = w4.forward(binding.Fp4Rows(fmt, 96, 4).quantize(x))
    cnt = torch.tensor([150, 0, 1, 131], dtype=torch.int32, device="cuda")
    on = (torch.arange(150, device="cuda")[None, :] < cnt[:, None]).reshape(-1)
    x[~on] = float("nan")
    y = torch.full((600, 72), 7.0, dtype=BF16, device="cuda")
    w4.forward(binding.Fp4Rows(fmt, 96, 4).quantize(x, None, cnt), None, cnt, y=y)
    assert w4.device_status()[0] == binding.MOE_OK
    assert torch.equal(y[on], full[on]) and (y[~on] == 7.0).all()


def test_weights_quantized_in_a_graph():
    """The group maxima (a memset, three kernels) replayed on new weights."""
    gen = torch.Generator(device="cuda").manual_seed(12)
    w = torch.randn((3, 72, 160), generator=gen, device="cuda").to(BF16)
    binding.Fp4Weights.quantize(w, "nv")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = binding.Fp4Weights.quantize(w, "nv")
    w.copy_(torch.randn(w.shape, generator=gen, device="cuda") * 3)
    graph.replay()
    eager = binding.Fp4Weights.quantize(w, "nv")
    assert torch.equal(captured.codes, eager.codes) and torch.equal(captured.gscale, eager.gscale)
    assert torch.equal(captured.dequantize(), eager.dequantize())


@pytest.mark.parametrize("offsets", [[0, 60, 50], [40, 20, 50], [-5, 10, 50], [0, 10, 1 << 30], [0, 0, 0], [60, 70, 80]])
@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_rows_in_wrong_lists_stay_in_bounds(fmt, offsets):
    """Whatever the lists say, only the call's own buffers are written (guards around them), and no scale is read elsewhere."""
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    x = torch.randn((50, 128), device="cuda").to(BF16)
    r4 = binding.Fp4Rows(fmt, 128, 2, 50)
    guarded = {}
    for name in ("codes", "scales") + (("gscale",) if fmt == "nv" else ()):
        t = getattr(r4, name)
        wide = torch.full((t.numel() + 64,), 99, dtype=t.dtype, device="cuda")
        guarded[name] = wide
        setattr(r4, name, wide[32:-32])
    r4.quantize(x, off)
    y = torch.full((52, 128), 7.0, dtype=BF16, device="cuda")
    r4.dequantize(off, y=y[1:-1])
    assert all((t[:32] == 99).all() and (t[-32:] == 99).all() for t in guarded.values())
    assert (y[0] == 7.0).all() and (y[-1] == 7.0).all()


def test_a_refused_quantize_leaves_the_rows_before():
    x = torch.randn((10, 64), device="cuda").to(BF16)
    r4 = binding.Fp4Rows("nv", 64, 1, 10).quantize(x)
    want = r4.dequantize()
    with pytest.raises(TypeError):
        r4.quantize(torch.zeros((500, 64), device="cuda").double())
    assert torch.equal(r4.dequantize(), want)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_larger_buffers_hold_no_rows_yet(fmt):
    """Buffers that grew hold none of the rows quantized before: they are forgotten, not read from new memory."""
    x = torch.ones((10, 64), dtype=BF16, device="cuda")
    r4 = binding.Fp4Rows(fmt, 64, 1, 10).quantize(x)
    r4.ensure_capacity(10)
    assert r4.rows == 10 and (r4.dequantize() == 1).all()
    r4.ensure_capacity(1000)
    assert r4.rows == 0 and r4.dequantize().shape == (0, 64)
    w4 = binding.Fp4Weights.quantize(torch.ones((1, 8, 64), dtype=BF16, device="cuda"), fmt)
    assert w4.forward(r4).shape == (0, 8) and (w4.forward(r4.quantize(x)) == 64).all()


def test_an_allocation_that_fails_leaves_the_rows_before(monkeypatch):
    x = torch.ones((10, 64), dtype=BF16, device="cuda")
    r4 = binding.Fp4Rows("nv", 64, 1, 10).quantize(x)
    big, real = torch.ones((1000, 64), dtype=BF16, device="cuda"), torch.empty
    for fail_at in range(3):  # codes, scales, gscale
        left = [fail_at]

        def empty(*args, **kw):
            if left[0] == 0:
                raise MemoryError
            left[0] -= 1
            return real(*args, **kw)

        monkeypatch.setattr(torch, "empty", empty)
        with pytest.raises(MemoryError):
            r4.quantize(big)
        monkeypatch.undo()
        assert r4.rows == 10 and (r4.dequantize() == 1).all()


def test_quotients_by_divisors_of_ones_alone():
    """Divisors with the significand 0x7FFFFF, which the correction's theorem excepts: the codes and scales are still those
    of the rounded quotients.  amax 0x40BFFFFF gives g = amax / 2688, scale 448 and d = RN(448 g) = 1 - 2^-24 (or d 2^k), so
    x = 0.25 lies just above a border (0.25 / d rounds to 0.25 + 2^-25, code 1, not the tie's 0)."""
    amax = np.array([0x40BFFFFF], np.uint32).view(np.float32)[0]
    assert (np.float32(448) * (amax / np.float32(2688))).view(np.uint32) == 0x3F7FFFFF
    x = np.zeros((8, 64), np.float32)
    x[:, ::16] = amax
    near = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    x[:, 1:8], x[:, 8:15] = near, -near
    x[1, 1:8], x[2, 1:8] = np.nextafter(near, np.float32(0)), np.nextafter(near, np.float32(9))
    x[3:] *= np.exp2(np.array([-40, -7, 1, 9, 40], np.float32))[:, None]
    r4 = binding.Fp4Rows("nv", 64, 1, 8).quantize(torch.tensor(x).cuda())
    c, s, _ = quantise(x, "nv", False)
    assert (s == 126).all() and c[0, 1] == 1 and c[1, 1] == 0  # 126: 448
    assert np.array_equal(unpack(r4.codes, 8, 64), c)
    # the scale's own quotient, amax of a block / (6 g): 6 g of ones alone, blocks next to every border of E4M3
    top = np.array([0x3FDFFFFF], np.uint32).view(np.float32)[0]
    six_g = np.float32(6) * (top / np.float32(2688))
    assert six_g.view(np.uint32) & 0x7FFFFF == 0x7FFFFF
    border = ((E4M3[1:] + E4M3[:-1]) / np.float32(2) * six_g).astype(np.float32)
    x = np.zeros((3, 128 * 16), np.float32)
    x[:, 0] = top
    x[:, 16:127 * 16:16] = border, np.nextafter(border, np.float32(0)), np.nextafter(border, np.float32(np.inf))
    r4 = binding.Fp4Rows("nv", 2048, 1, 3).quantize(torch.tensor(x).cuda())
    c, s, _ = quantise(x, "nv", False)
    assert np.array_equal(scale_of(r4.scales, Lists([3]), 0, 3, 2048, "nv"), s)
    assert np.array_equal(unpack(r4.codes, 3, 2048), c)


def hard_matrix(rows, k, dtype, hard, seed):
    """Rows of many binades made on the GPU, those of ``hard`` from hard_rows."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, k), generator=gen, device="cuda")
    x *= torch.exp2(torch.randint(-6, 7, (rows, k // 16), generator=gen, device="cuda").float()).repeat_interleave(16, 1)
    x = x.to(dtype)
    x[torch.tensor(hard, device="cuda")] = hard_rows(np.random.default_rng(seed), len(hard), k, dtype).cuda()
    return x


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=str)
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("rows,k", [(2500, 2048), (2500, 4128), (1500, 4096), (1500, 8224), (700, 8192), (700, 16416),
                                    (40, 32800)])
def test_rows_of_every_number_of_threads(rows, k, fmt, dtype):
    """32, 64, 128 and 256 threads a row (fewer where there are more rows), their vectors held at once or in several
    rounds: codes, scales and values of rows in every part, the first, the last and those at tile edges among them."""
    lists = Lists([rows // 2 + 1, 0, rows // 8, rows - rows // 2 - 1 - rows // 8 - 3], tail=3)
    at = sorted({min(a + d, b - 1) for a, b in lists.spans if b > a for d in (0, 1, 31, 32, 127, 128, 129, 10 ** 6)}
                | set(range(5, rows - 3, max(1, rows // 11))))
    x = hard_matrix(rows, k, dtype, at[::2], len(at))
    r4 = binding.Fp4Rows(fmt, k, 4, rows).quantize(x, lists.offsets)
    c, s, gs = quantise(x[torch.tensor(at, device="cuda")].float().cpu().numpy(), fmt, False)
    raw = unpack(r4.codes, rows, k)[at]
    if fmt == "nv":
        assert np.array_equal(r4.gscale[torch.tensor(at, device="cuda")].cpu().numpy(), gs)
        c = np.where(np.repeat(E4M3[s] * gs[:, None] == 0, 16, axis=1), 0, c)
    assert np.array_equal(raw, c)
    for g, (a, b) in enumerate(lists.spans):
        mine = [i for i, p in enumerate(at) if a <= p < b]
        if mine:
            assert np.array_equal(scale_of(r4.scales, lists, g, b - a, k, fmt)[[at[i] - a for i in mine]], s[mine])
    want = torch.tensor(values(c, s, gs, fmt))
    for out in (BF16, FP16, FP32):
        got = r4.dequantize(lists.offsets, dtype=out)[torch.tensor(at, device="cuda")].cpu().double()
        over = want.abs() > torch.finfo(out).max
        tiny = torch.finfo(out).smallest_normal * torch.finfo(out).eps / 2
        # (the roundings of test_quantise_and_back)
        rel = torch.finfo(out).eps / 2 + (2.0 ** -24 if out != FP32 else 0.0)
        assert ((got - want).abs() <= want.abs() * rel * (1 + 2.0 ** -20) + tiny)[~over].all()
        assert (got[over].abs() >= torch.finfo(out).max).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("groups,n,k", [(2, 1304, 4128), (3, 400, 8224), (5, 136, 16416)])
def test_large_weights(groups, n, k, fmt):
    """Matrices whose rows take 32, 64 and 128 threads in several rounds, one NVFP4 scale each."""
    w = torch.stack([hard_matrix(n, k, BF16, [0, 1, n // 2, n - 1], g) * 2.0 ** (3 * g - 4) for g in range(groups)]).to(BF16)
    w4 = binding.Fp4Weights.quantize(w, fmt)
    lists, back = Lists([n] * groups, equal=True), w4.dequantize(FP32)
    codes = unpack(w4.codes.view(-1), groups * n, k).reshape(groups, n, k)
    for g in range(groups):
        top = int(w[g].abs().amax(1).argmax())  # (its row sets the matrix's scale)
        at = sorted({0, 1, 31, 32, 127, 128, n // 2, n // 2 + 1, n - 2, n - 1, top})
        c, s, gs = quantise(w[g][torch.tensor(at, device="cuda")].float().cpu().numpy(), fmt, True)
        assert np.array_equal(scale_of(w4.scales, lists, g, n, k, fmt)[at], s)
        if fmt == "nv":
            assert w4.gscale[g].item() == gs[0]
            c = np.where(np.repeat(E4M3[s] * gs[:, None] == 0, 16, axis=1), 0, c)
        assert np.array_equal(codes[g][at], c)
        want = values(c, s, gs, fmt)
        got = back[g][torch.tensor(at, device="cuda")].cpu().double().numpy()
        assert (np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -150).all()
