"""The grouped products and their gradients, and SwiGLU, against their definitions in 64 bits.

Tolerances.  A product of two 16-bit operands is exact in fp32 (bf16: 16 bits,
fp16: 22 bits).  One tensor-core step adds 16 products to the fp32 accumulator
and may cut each of the 17 terms after the last bit of the largest, which is at
most S = sum |a||b|: an error of 17 ulps of S, 17 * 2^-23 S, per 16 terms of the
reduction, R * 2^-23 * 17/16 * S in all (R rounded up to whole steps); stream-K
adds one fp32 rounding for each of at most 256 partial sums.  The output is
rounded once: half a step, eps/2 relative, or half a subnormal step (2^-25 for
fp16).  So |err| <= eps/2 |y| + (17/16 (R + 16) + 256) 2^-23 S + 2^-25.
"""
import numpy as np
import pytest
import torch

from mixture_experts_layer_rmsnorm_gb300 import binding

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def bound(want, s, r, dtype):
    return half_step(dtype) * want.abs() + (17 / 16 * (r + 16) + 256) * 2.0 ** -23 * s + 2.0 ** -25


def check(got, want, s, r):
    err = (got.double() - want).abs()
    lim = bound(want, s, r, got.dtype)
    worst = (err - lim).max().item() if err.numel() else 0.0
    assert worst <= 0, f"error above its bound by {worst:.3e} (largest error {err.max().item():.3e})"


class Lists:
    """Groups of the given counts; gap: rows left free behind every group (they hold NaN); tail: rows behind the last."""

    def __init__(self, counts, gap=0, tail=0):
        held = [c + gap for c in counts]
        off = np.concatenate([[0], np.cumsum(held)])
        self.spans = [(int(o), int(o + c)) for o, c in zip(off, counts)]
        self.offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        self.counts = torch.tensor(counts, dtype=torch.int32, device="cuda") if gap else None
        self.rows = int(off[-1]) + tail
        self.groups = len(counts)
        self.free = torch.ones(self.rows, dtype=torch.bool, device="cuda")
        for a, b in self.spans:
            self.free[a:b] = False

    def matrix(self, gen, width, dtype, pad=0, scale=1.0):
        full = torch.randn((self.rows, width + pad), generator=gen, device="cuda").mul_(scale).to(dtype)
        full[self.free] = float("nan")
        return full[:, :width]

    def blank(self, width, dtype, pad=0):
        return torch.full((self.rows, width + pad), 7.0, dtype=dtype, device="cuda")[:, :width]


# counts, N, K, dtype, gap, tail, pad: every tile plan, single rows, empty groups, chunk edges (32, 256), sizes that are no
# multiple of a tile, strided matrices, more groups than the shared-memory table holds
CASES = {
    "one": ([1], 8, 8, BF16, 0, 0, 0),
    "row_of_many": ([1], 1000, 4104, FP16, 0, 3, 0),
    "small_edges": ([0, 1, 15, 16, 17, 31, 32, 33, 0, 1, 1, 0], 264, 200, BF16, 0, 0, 8),
    "small_stream_k": ([3, 0, 5, 8, 0, 1, 2, 7], 1024, 2048, BF16, 3, 5, 0),
    "small_fp16_gap": ([9, 12, 0, 0, 31, 2, 1], 392, 1032, FP16, 5, 1, 16),
    "large_edges": ([255, 256, 257, 0, 1, 300, 511, 513], 520, 328, BF16, 0, 0, 0),
    "large_fp16": ([100, 0, 700, 33], 1416, 640, FP16, 7, 9, 24),
    "large_skewed": ([1500, 1, 0, 2, 40], 256, 128, BF16, 1, 0, 0),
    "many_groups": ([(7 * i) % 5 for i in range(300)], 136, 72, BF16, 0, 2, 0),
    "most_groups": ([(i * i) % 41 for i in range(1024)], 64, 64, FP16, 0, 0, 0),
    "long_groups": ([2500, 0, 769, 768, 1537], 264, 136, BF16, 0, 1, 0),
    "some_rows": ([20, 40, 0, 17, 24, 21, 19], 264, 200, BF16, 0, 3, 0),
    "some_rows_whole_wave": ([19 + i % 5 for i in range(76)], 256, 72, FP16, 0, 0, 8),
    "no_rows_at_all": ([0, 0, 0], 128, 64, BF16, 0, 4, 0),
}


def make(name):
    counts, n, k, dtype, gap, tail, pad = CASES[name]
    gen = torch.Generator(device="cuda").manual_seed(len(name))
    lists = Lists(counts, gap, tail)
    x = lists.matrix(gen, k, dtype, pad)
    dy = lists.matrix(gen, n, dtype, pad, 0.25)
    w = (torch.randn((lists.groups, n, k), generator=gen, device="cuda") * 0.05).to(dtype)
    return lists, x, dy, w, binding.GroupedProducts(lists.groups, n, k, dtype), pad


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    lists, x, _, w, gp, pad = make(name)
    y = lists.blank(gp.N, x.dtype, pad)
    assert gp.forward(x, w, lists.offsets, lists.counts, y=y) is y
    assert gp.device_status()[0] == binding.MOE_OK
    for g, (a, b) in enumerate(lists.spans):
        xd, wd = x[a:b].double(), w[g].double()
        check(y[a:b], xd @ wd.T, xd.abs() @ wd.abs().T, gp.K)
    assert torch.all(y[lists.free] == 7.0)


@pytest.mark.parametrize("name", CASES)
def test_input_gradient(name):
    lists, _, dy, w, gp, pad = make(name)
    dx = lists.blank(gp.K, dy.dtype, pad)
    gp.dgrad(dy, w, lists.offsets, lists.counts, dx=dx)
    assert gp.device_status()[0] == binding.MOE_OK
    for g, (a, b) in enumerate(lists.spans):
        dd, wd = dy[a:b].double(), w[g].double()
        check(dx[a:b], dd @ wd, dd.abs() @ wd.abs(), gp.N)
    assert torch.all(dx[lists.free] == 7.0)


@pytest.mark.parametrize("out", ["same", "fp32", "accumulate"])
@pytest.mark.parametrize("name", CASES)
def test_weight_gradient(name, out):
    lists, x, dy, w, gp, pad = make(name)
    if out == "accumulate":
        start = torch.randn(w.shape, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
        dw = start.clone()
        gp.wgrad(dy, x, lists.offsets, lists.counts, dw=dw, accumulate=True)
    else:
        dw = gp.wgrad(dy, x, lists.offsets, lists.counts, dtype=FP32 if out == "fp32" else None)
    assert gp.device_status()[0] == binding.MOE_OK
    for g, (a, b) in enumerate(lists.spans):
        dd, xd = dy[a:b].double(), x[a:b].double()
        want, s = dd.T @ xd, dd.abs().T @ xd.abs()
        if out == "accumulate":  # one fp32 addition more
            want, s = want + start[g].double(), s + start[g].abs().double()
        # into fp32 at most 768 rows are accumulated by the tensor core, then added in fp32 (one of the 256 roundings each)
        check(dw[g], want, s, b - a if out == "same" else min(b - a, 768))


def test_long_sums_into_fp32_keep_their_precision():
    """The tensor core cuts towards zero once a step: unsplit, 16384 rows of one sign lose some 1e-4.  Split, a segment of
    768 rows takes 48 steps, each cutting less than a unit in the last place of the accumulator, 2^-23 of it, by its own
    sum and, on average over the 16 products' random bits below it, half a unit for each product: 48 (1 + 16 / 2) 2^-23
    = 5.2e-5 of the sum at most, and the segments' own additions 22 2^-24."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    x = torch.rand((16384, 136), generator=gen, device="cuda").to(BF16)
    dy = torch.rand((16384, 264), generator=gen, device="cuda").to(BF16)
    gp = binding.GroupedProducts(1, 264, 136, BF16)
    want = dy.double().T @ x.double()
    rel = ((gp.wgrad(dy, x, dtype=FP32)[0].double() - want) / want).abs().max().item()
    assert rel <= 48 * 9 * 2.0 ** -23 + 22 * 2.0 ** -24, rel


def test_equal_groups_without_lists():
    gen = torch.Generator(device="cuda").manual_seed(3)
    gp = binding.GroupedProducts(3, 136, 264, BF16)
    x = torch.randn((3 * 35, 264), generator=gen, device="cuda").to(BF16)
    dy = torch.randn((3 * 35, 136), generator=gen, device="cuda").to(BF16)
    w = (torch.randn((3, 136, 264), generator=gen, device="cuda") * 0.05).to(BF16)
    y, dx, dw = gp.forward(x, w), gp.dgrad(dy, w), gp.wgrad(dy, x, dtype=FP32)
    xd, dd, wd = x.double().view(3, 35, -1), dy.double().view(3, 35, -1), w.double()
    check(y.view(3, 35, -1), xd @ wd.mT, xd.abs() @ wd.abs().mT, 264)
    check(dx.view(3, 35, -1), dd @ wd, dd.abs() @ wd.abs(), 136)
    check(dw, dd.mT @ xd, dd.abs().mT @ xd.abs(), 35)


def test_nan_and_inf_stay_in_their_row_and_group():
    lists = Lists([40, 21, 64])
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, dy = lists.matrix(gen, 192, BF16), lists.matrix(gen, 136, BF16)
    w = (torch.randn((3, 136, 192), generator=gen, device="cuda") * 0.05).to(BF16)
    gp = binding.GroupedProducts(3, 136, 192, BF16)
    clean = [t.clone() for t in (gp.forward(x, w, lists.offsets), gp.dgrad(dy, w, lists.offsets),
                                 gp.wgrad(dy, x, lists.offsets))]
    x[40, 3], x[60, 5], dy[60, 7], dy[40, 1] = float("nan"), float("inf"), float("nan"), float("-inf")
    y, dx, dw = gp.forward(x, w, lists.offsets), gp.dgrad(dy, w, lists.offsets), gp.wgrad(dy, x, lists.offsets)
    for got, ref in ((y, clean[0]), (dx, clean[1])):
        hit = torch.zeros(lists.rows, dtype=torch.bool, device="cuda")
        hit[[40, 60]] = True
        assert torch.equal(got[~hit], ref[~hit])
        assert not torch.isfinite(got[hit]).any()
    assert torch.equal(dw[0], clean[2][0]) and torch.equal(dw[2], clean[2][2])
    assert torch.isnan(dw[1, :, 3]).all() and torch.isnan(dw[1, 7]).all()


@pytest.mark.parametrize("offsets,counts,group", [
    ([0, 10, 8, 30], None, 1),            # decreasing
    ([-1, 10, 20, 30], None, 0),          # negative
    ([0, 10, 20, 41], None, 2),           # behind the last row
    ([0, 10, 20, 30], [10, 11, 3], 1),    # into the next group
    ([0, 10, 20, 30], [10, 10, -1], 2),   # a negative count
])
def test_bad_lists_write_nothing_and_are_reported(offsets, counts, group):
    gp = binding.GroupedProducts(3, 64, 64, BF16)
    x = torch.ones((40, 64), dtype=BF16, device="cuda")
    w = torch.ones((3, 64, 64), dtype=BF16, device="cuda")
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    outs = [torch.full((40, 64), 7.0, dtype=BF16, device="cuda") for _ in range(2)] + [torch.full_like(w, 7.0)]
    for call, out in ((lambda o: gp.forward(x, w, off, cnt, y=o), outs[0]),
                      (lambda o: gp.dgrad(x, w, off, cnt, dx=o), outs[1]),
                      (lambda o: gp.wgrad(x, x, off, cnt, dw=o), outs[2])):
        call(out)
        st, detail = gp.device_status()
        assert st == binding.MOE_ERR_DEVICE and detail[1] == 9 and detail[2] == group
        assert torch.all(out == 7.0)
    good = torch.tensor([0, 10, 20, 30], dtype=torch.int32, device="cuda")
    gp.forward(x, w, good, y=outs[0])  # the next call clears the error
    assert gp.device_status()[0] == binding.MOE_OK and torch.all(outs[0][:30] == 64.0)


def test_calls_repeat_bit_for_bit_and_replay_from_a_graph_on_new_lists():
    lists = Lists([5, 0, 9, 2])
    gen = torch.Generator(device="cuda").manual_seed(6)
    x, dy = lists.matrix(gen, 1024, BF16), lists.matrix(gen, 512, BF16)
    w = (torch.randn((4, 512, 1024), generator=gen, device="cuda") * 0.05).to(BF16)
    gp = binding.GroupedProducts(4, 512, 1024, BF16)
    off = lists.offsets.clone()
    y, dx = torch.zeros_like(dy), torch.zeros_like(x)
    dw = torch.zeros(w.shape, device="cuda")

    def step():
        gp.forward(x, w, off, y=y)
        gp.dgrad(dy, w, off, dx=dx)
        gp.wgrad(dy, x, off, dw=dw)

    step()
    first = [t.clone() for t in (y, dx, dw)]
    step()
    assert all(torch.equal(a, b) for a, b in zip(first, (y, dx, dw)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    off.copy_(torch.tensor([0, 0, 12, 16, 16], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in (y, dx, dw)]
    step()
    assert all(torch.equal(a, b) for a, b in zip(replayed, (y, dx, dw)))
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(replayed, (y, dx, dw)))


# ------------------------------------------------------------------ SwiGLU


@pytest.mark.parametrize("rows,i,dtype,pad", [(1, 8, BF16, 0), (7, 136, FP16, 8), (301, 1408, BF16, 16),
                                              (64, 4096, FP16, 0), (5000, 24, BF16, 0)])
def test_swiglu_and_its_gradient(rows, i, dtype, pad):
    """fp32 inside.  exp(-|g|) is 2 ulps + |g| 2^-24 (its scaled argument is rounded), the quotient 2, each of at most six
    further operations half: relative errors below (|g| + 16) 2^-23 of the terms, then one rounding of the output.  Below
    fp32's smallest normal number the intermediate e may be cut: an absolute 2^-126 times the other factors."""
    gen = torch.Generator(device="cuda").manual_seed(rows)
    h = (torch.randn((rows, 2 * i + pad), generator=gen, device="cuda") * 3).to(dtype)[:, :2 * i]
    edge = torch.tensor([0.0, -0.0, 40.0, -40.0, 88.0, -88.0, 300.0, -300.0], device="cuda").to(dtype)
    h[0, :8] = edge
    da = torch.randn((rows, i), generator=gen, device="cuda").to(dtype)
    g, u, d = h[:, :i].double(), h[:, i:].double(), da.double()
    s, t = torch.special.expit(g), torch.special.expit(-g)
    rel = (g.abs() + 16) * 2.0 ** -23
    tiny = 2.0 ** -126 * 400 * (u.abs() + 1) * (d.abs() + 1) + 2.0 ** -25 * (dtype == FP16) + 2.0 ** -134

    def within(got, want, size):
        err = (got.double() - want).abs()
        lim = half_step(dtype) * (want.abs() + rel * size) + rel * size + tiny
        assert (err <= lim).all(), f"largest error {err.max().item():.3e}"

    within(binding.swiglu(h), g * s * u, (g * s * u).abs())
    for dh in (binding.swiglu_grad(h, da), binding.swiglu_grad(h.clone(), da)):
        within(dh[:, :i], d * u * s * (1 + g * t), (d * u).abs() * s * (1 + g.abs() * t))
        within(dh[:, i:], d * g * s, (d * g * s).abs())
    inplace = h.clone()
    assert torch.equal(binding.swiglu_grad(inplace, da, dh=inplace), dh)


def test_swiglu_keeps_nan_and_infinities():
    h = torch.tensor([[float("nan"), 1.0, float("inf"), 2.0, float("-inf"), 0.0, 1.0, 1.0] + [1.0] * 8], device="cuda")
    h[0, 9] = float("nan")
    a = binding.swiglu(h.to(BF16)).float()[0]
    assert torch.isnan(a[0]) and torch.isnan(a[1]) and a[2] == float("inf") and torch.isnan(a[4])
    assert torch.isfinite(a[[3, 5, 6, 7]]).all()


# ------------------------------------------------------------------ a training step of the experts


def test_training_step_of_the_experts():
    """Gate/up product, SwiGLU, down product, and every gradient, over the router's own lists (16-row padding, counts);
    against 64 bits with each stored tensor rounded as the chain rounds it, and the loss's slope against differences."""
    T, H, I, E, top_k = 50, 256, 192, 6, 2
    gen = torch.Generator(device="cuda").manual_seed(8)
    xs = torch.randn((T, H), generator=gen, device="cuda").to(BF16)
    g_norm = torch.ones(H, dtype=BF16, device="cuda")
    w_router = torch.randn((E, H), generator=gen, device="cuda") * 0.02
    w13 = (torch.randn((E, 2 * I, H), generator=gen, device="cuda") * 0.05).to(BF16)
    w2 = (torch.randn((E, H, I), generator=gen, device="cuda") * 0.05).to(BF16)
    layer = binding.MoeLayer(g_norm, w_router, w13, w2, top_k, max_tokens=T)
    layer.forward(xs)
    h = layer.view_tensor(T, "h", BF16, (T, H)).clone()
    counts = layer.view_tensor(T, "counts", torch.int32, (E,)).clone()
    offsets = layer.view_tensor(T, "offsets", torch.int32, (E + 1,)).clone()
    p_max = layer.views(T).P_max
    ids = layer.view_tensor(T, "sorted_ids", torch.int32, (p_max,)).clone()
    rows = torch.cat([torch.arange(o, o + c) for o, c in zip(offsets.tolist(), counts.tolist())]).cuda()
    x = torch.full((p_max, H), float("nan"), dtype=BF16, device="cuda")
    x[rows] = h[(ids[rows] // top_k).long()]

    up, down = binding.GroupedProducts(E, 2 * I, H, BF16), binding.GroupedProducts(E, H, I, BF16)
    hid = up.forward(x, w13, offsets, counts, y=torch.zeros((p_max, 2 * I), dtype=BF16, device="cuda"))
    act = binding.swiglu(hid)
    y = down.forward(act, w2, offsets, counts, y=torch.zeros((p_max, H), dtype=BF16, device="cuda"))
    # the layer computes the same rows
    out_rows = layer.view_tensor(T, "out_rows", BF16, (p_max, H))
    ref = out_rows[rows].double()
    assert (y[rows].double() - ref).norm() <= 2 * half_step(BF16) * ref.norm()

    dy = torch.randn((p_max, H), generator=gen, device="cuda").to(BF16)
    dact = down.dgrad(dy, w2, offsets, counts, dx=torch.zeros((p_max, I), dtype=BF16, device="cuda"))
    dw2 = down.wgrad(dy, act, offsets, counts, dtype=FP32)
    dhid = binding.swiglu_grad(hid, dact)
    dx = up.dgrad(dhid, w13, offsets, counts, dx=torch.zeros((p_max, H), dtype=BF16, device="cuda"))
    dw13 = up.wgrad(dhid, x, offsets, counts, dtype=FP32)

    group = torch.repeat_interleave(torch.arange(E, device="cuda"), counts.long())
    leaf = [t.double().requires_grad_() for t in (x[rows], w13, w2)]

    def loss(xd, w13d, w2d):
        hd = torch.einsum("ph,pnh->pn", xd, w13d[group])
        ad = torch.nn.functional.silu(hd[:, :I]) * hd[:, I:]
        return (torch.einsum("pi,phi->ph", ad, w2d[group]) * dy[rows].double()).sum()

    loss(*leaf).backward()
    # five roundings to bf16 at most lie between the inputs and a gradient (hid, act or dact, dhid, the output), each at
    # most half a step of its tensor's norm; a product passes relative norms on with a factor of order one (here < 2)
    for got, want in ((dx[rows], leaf[0].grad), (dw13, leaf[1].grad), (dw2, leaf[2].grad)):
        rel = ((got.double() - want).norm() / want.norm()).item()
        assert rel <= 5 * 2 * half_step(BF16), rel
    # differences: the loss along the gradient's own direction
    with torch.no_grad():
        for at, got in ((0, dx[rows]), (1, dw13), (2, dw2)):
            step = got.double() / got.double().norm()
            args = [t.detach() for t in leaf]
            eps = 1e-4
            plus, minus = list(args), list(args)
            plus[at], minus[at] = args[at] + eps * step, args[at] - eps * step
            slope = ((loss(*plus) - loss(*minus)) / (2 * eps)).item()
            assert abs(slope - got.double().norm().item()) <= 5 * 2 * half_step(BF16) * abs(slope) + 1e-5


@pytest.mark.parametrize("counts", [[513, 512, 1, 1024, 31, 1023, 545], [96, 480, 130, 290, 272, 33], [2000, 17, 17, 17, 17],
                                    [64 + 32 * (i % 15) for i in range(90)]], ids=lambda c: f"{len(c)}_groups")
@pytest.mark.parametrize("op", ["forward", "dgrad"])
def test_units_of_every_width_follow_one_another(op, counts):
    """Units of 32 to 512 rows in one call: shared memory and TMEM are handed on between units of different sizes,
    over several units per CTA pair."""
    lists = Lists(counts)
    gen = torch.Generator(device="cuda").manual_seed(len(counts))
    n, k = (2560, 320) if op == "forward" else (320, 2560)
    gp = binding.GroupedProducts(lists.groups, n, k, BF16)
    w = (torch.randn((lists.groups, n, k), generator=gen, device="cuda") * 0.05).to(BF16)
    a = lists.matrix(gen, k if op == "forward" else n, BF16)
    out = gp.forward(a, w, lists.offsets) if op == "forward" else gp.dgrad(a, w, lists.offsets)
    assert gp.device_status()[0] == binding.MOE_OK
    for g, (lo, hi) in enumerate(lists.spans):
        ad, wd = a[lo:hi].double(), w[g].double().T if op == "forward" else w[g].double()
        check(out[lo:hi], ad @ wd, ad.abs() @ wd.abs(), 320)


def test_two_host_threads_on_their_own_streams():
    """Objects, workspaces and streams of their own, calls at once: the bits of calls alone.  (The host side's
    once-per-device configuration and the shape an object keeps are shared state.)"""
    import threading

    def work(seed):
        lists = Lists([9 * seed, 0, 300, 17 + seed])
        gen = torch.Generator(device="cuda").manual_seed(seed)
        x, dy = lists.matrix(gen, 512, BF16), lists.matrix(gen, 384, BF16)
        w = (torch.randn((4, 384, 512), generator=gen, device="cuda") * 0.05).to(BF16)
        few = Lists([1, 0, 2, 1])
        xf = few.matrix(gen, 512, BF16)
        return lists, x, dy, w, few, xf

    def run(gp, lists, x, dy, w, few, xf):
        r4 = binding.Fp4Rows("nv", 512, 4).quantize(x, lists.offsets)
        return [gp.forward(x, w, lists.offsets), gp.dgrad(dy, w, lists.offsets), gp.wgrad(dy, x, lists.offsets, dtype=FP32),
                gp.forward(xf, w, few.offsets), binding.swiglu(x), r4.dequantize(lists.offsets),
                binding.Fp4Weights.quantize(w, "mx").forward(binding.Fp4Rows("mx", 512, 4).quantize(x, lists.offsets),
                                                             lists.offsets)]

    data = [work(1), work(2)]
    alone = [run(binding.GroupedProducts(4, 384, 512, BF16), *d) for d in data]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def thread(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                gp = binding.GroupedProducts(4, 384, 512, BF16)
                for _ in range(20):
                    out = run(gp, *data[i])
                torch.cuda.current_stream().synchronize()
                got[i] = out
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors, errors
    for a, b in zip(alone, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_the_objects_refuse_wrong_tensors():
    gp = binding.GroupedProducts(2, 64, 128, BF16)
    x, w = torch.zeros((6, 128), dtype=BF16, device="cuda"), torch.zeros((2, 64, 128), dtype=BF16, device="cuda")
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    gp.forward(x, w, off)
    for bad in (lambda: gp.forward(x.cpu(), w, off), lambda: gp.forward(x[:, :64], w, off),
                lambda: gp.forward(x.t().contiguous().t(), w, off), lambda: gp.forward(x, w[:1], off),
                lambda: gp.forward(x, w, off[:2]), lambda: gp.forward(x, w, off, y=torch.zeros((6, 64), device="cuda").cpu()),
                lambda: gp.wgrad(x[:, :64], x, off, accumulate=True), lambda: gp.wgrad(x[:5, :64], x, off)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: gp.forward(x.half(), w, off), lambda: gp.forward(x, w, off.long()), lambda: binding.swiglu(x.double())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(binding.MoeError):
        gp.forward(x[:5], w)  # no lists, and 5 rows do not make 2 equal groups
    with pytest.raises(binding.MoeError):
        gp.wgrad(x[:, :64], x, off, dw=torch.zeros((2, 64, 128), dtype=BF16, device="cuda"), accumulate=True)


def test_swiglu_refuses_an_odd_width():
    h, a = torch.zeros((4, 17), dtype=BF16, device="cuda"), torch.zeros((4, 8), dtype=BF16, device="cuda")
    for bad in (lambda: binding.swiglu(h), lambda: binding.swiglu_grad(h, a)):
        with pytest.raises(ValueError):
            bad()


def test_calls_without_rows_report_nothing_of_earlier_calls():
    gp = binding.GroupedProducts(2, 8, 64, BF16)
    gp.workspace.fill_(0xFF)
    assert gp.device_status()[0] == binding.MOE_OK  # no call yet
    x, w = torch.ones((6, 64), dtype=BF16, device="cuda"), torch.ones((2, 8, 64), dtype=BF16, device="cuda")
    dy, dw = torch.ones((6, 8), dtype=BF16, device="cuda"), torch.ones((2, 8, 64), device="cuda")
    bad = torch.tensor([0, 9, 6], dtype=torch.int32, device="cuda")
    empty = (lambda: gp.forward(x[:0], w, bad), lambda: gp.dgrad(dy[:0], w, bad),
             lambda: gp.wgrad(dy[:0], x[:0], dw=dw, accumulate=True))
    for call in empty:
        gp.forward(x, w, bad)
        assert gp.device_status()[0] == binding.MOE_ERR_DEVICE
        call()
        assert gp.device_status()[0] == binding.MOE_OK
    assert (dw == 1).all()


@pytest.mark.parametrize("rows_per_group", [12, 200], ids=["few", "many"])
def test_equal_groups_filled_in_part(rows_per_group):
    """counts without offsets: group g holds the first counts[g] of its rows / groups rows."""
    counts = [rows_per_group, 0, 1, rows_per_group // 2]
    gen = torch.Generator(device="cuda").manual_seed(8)
    rows, n, k = 4 * rows_per_group, 136, 200
    x, dy = (torch.full((rows, c), float("nan"), dtype=BF16, device="cuda") for c in (k, n))
    w = (torch.randn((4, n, k), generator=gen, device="cuda") * 0.05).to(BF16)
    free = torch.ones(rows, dtype=torch.bool, device="cuda")
    spans = [(g * rows_per_group, g * rows_per_group + c) for g, c in enumerate(counts)]
    for a, b in spans:
        x[a:b] = torch.randn((b - a, k), generator=gen, device="cuda").to(BF16)
        dy[a:b] = torch.randn((b - a, n), generator=gen, device="cuda").to(BF16)
        free[a:b] = False
    gp, cnt = binding.GroupedProducts(4, n, k, BF16), torch.tensor(counts, dtype=torch.int32, device="cuda")
    y, dx = (torch.full((rows, c), 7.0, dtype=BF16, device="cuda") for c in (n, k))
    gp.forward(x, w, None, cnt, y=y)
    gp.dgrad(dy, w, None, cnt, dx=dx)
    dw = gp.wgrad(dy, x, None, cnt, dtype=FP32)
    assert gp.device_status()[0] == binding.MOE_OK and (y[free] == 7.0).all() and (dx[free] == 7.0).all()
    for g, (a, b) in enumerate(spans):
        xd, dd, wd = x[a:b].double(), dy[a:b].double(), w[g].double()
        check(y[a:b], xd @ wd.T, xd.abs() @ wd.abs().T, k)
        check(dx[a:b], dd @ wd, dd.abs() @ wd.abs(), n)
        check(dw[g], dd.T @ xd, dd.abs().T @ xd.abs(), b - a)
    gp.forward(x, w, None, cnt + (torch.arange(4, device="cuda") == 2).int() * rows_per_group, y=y)  # one row too many
    status, detail = gp.device_status()
    assert status == binding.MOE_ERR_DEVICE and detail[2] == 2


def test_rows_behind_2_to_the_32_elements():
    """Matrices whose last rows start more than 2^32 elements behind the first."""
    rows, ld, n, k = 66000, 65600, 72, 64
    x = torch.empty(rows * ld, dtype=BF16, device="cuda").view(rows, ld)[:, :k]
    gen = torch.Generator(device="cuda").manual_seed(9)
    x.copy_(torch.randn((rows, k), generator=gen, device="cuda"))
    packed = x.contiguous()
    off = torch.tensor([0, 7, 65700, rows], dtype=torch.int32, device="cuda")
    w = (torch.randn((3, n, k), generator=gen, device="cuda") * 0.05).to(BF16)
    gp = binding.GroupedProducts(3, n, k, BF16)
    y = gp.forward(x, w, off)
    assert torch.equal(y, gp.forward(packed, w, off))
    assert torch.equal(gp.wgrad(y, x, off, dtype=FP32), gp.wgrad(y, packed, off, dtype=FP32))
    assert torch.equal(binding.swiglu(x), binding.swiglu(packed))
    for fmt in ("mx", "nv"):
        a, b = (binding.Fp4Rows(fmt, k, 3).quantize(t, off) for t in (x, packed))
        assert torch.equal(a.codes, b.codes)
        values = b.dequantize(off)
        a.dequantize(off, y=x)
        assert torch.equal(x, values)
        x.copy_(packed)
    want = gp.dgrad(y, w, off)
    assert torch.equal(gp.dgrad(y, w, off, dx=x), want)
    x.copy_(packed)
    act = torch.ones((rows, k // 2), dtype=BF16, device="cuda")
    want = binding.swiglu_grad(packed, act)
    assert torch.equal(binding.swiglu_grad(x, act, dh=x), want)  # in place


@pytest.mark.parametrize("op", ["forward", "dgrad"])
@pytest.mark.parametrize("rows,n,k", [(8, 152, 5168), (1, 2096, 200), (3, 72, 8), (32, 128, 640), (9, 5168, 136)])
def test_few_blocks_are_shared_by_few_workers(op, rows, n, k):
    """Products with fewer K-blocks than SMs, of one group among empty ones: parts of several K-blocks, joined."""
    lists = Lists([0, rows, 0])
    gen = torch.Generator(device="cuda").manual_seed(rows)
    w = (torch.randn((3, n, k), generator=gen, device="cuda") * 0.05).to(BF16)
    gp = binding.GroupedProducts(3, n, k, BF16)
    wd = w[1].double()
    if op == "forward":
        x = lists.matrix(gen, k, BF16)
        y = gp.forward(x, w, lists.offsets)
        check(y, x.double() @ wd.T, x.double().abs() @ wd.abs().T, k)
    else:
        x = lists.matrix(gen, n, BF16)
        y = gp.dgrad(x, w, lists.offsets)
        check(y, x.double() @ wd, x.double().abs() @ wd.abs(), n)
    assert gp.device_status()[0] == binding.MOE_OK


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=str)
def test_long_sums_into_16_bits_keep_their_precision(dtype):
    """2^19 rows of one sign: accumulated whole, the tensor core's cuts take some 3e-3 of the sum, most of half a bf16 step and six
    half fp16 steps.  A segment of 3840 rows takes 240 steps of 9 2^-23 (as above: 2.6e-4), the 137 segments' additions 2^-24
    each, and the output is rounded once."""
    gen = torch.Generator(device="cuda").manual_seed(13)
    rows = 1 << 19
    x = torch.rand((rows, 136), generator=gen, device="cuda").to(dtype)
    dy = torch.rand((rows, 264), generator=gen, device="cuda").mul_(0.125).to(dtype)  # (sums of 16384: fp16 holds them)
    lists = [None, torch.tensor([0, rows - 3840 * 5 + 1, rows], dtype=torch.int32, device="cuda")]
    for offsets in lists:
        groups = 1 if offsets is None else 2
        spans = [(0, rows)] if offsets is None else [(0, rows - 3840 * 5 + 1), (rows - 3840 * 5 + 1, rows)]
        dw = binding.GroupedProducts(groups, 264, 136, dtype).wgrad(dy, x, offsets)
        for g, (a, b) in enumerate(spans):
            want = dy[a:b].double().T @ x[a:b].double()
            rel = ((dw[g].double() - want) / want).abs().max().item()
            assert rel <= half_step(dtype) + 240 * 9 * 2.0 ** -23 + 137 * 2.0 ** -24, rel


def test_status_of_an_object_whose_calls_never_ran():
    """A refused first call and a captured one that is not replayed leave no status: what the workspace's memory held
    before (here an error of another object's) is not theirs."""
    x, w = torch.ones((6, 64), dtype=BF16, device="cuda"), torch.ones((2, 8, 64), dtype=BF16, device="cuda")
    bad = torch.tensor([0, 9, 6], dtype=torch.int32, device="cuda")

    def used():  # an object on memory that holds an error word
        gp = binding.GroupedProducts(2, 8, 64, BF16)
        gp.forward(x, w, bad)
        assert gp.device_status()[0] == binding.MOE_ERR_DEVICE
        place = gp.workspace.data_ptr()
        del gp
        gp = binding.GroupedProducts(2, 8, 64, BF16)
        assert gp.workspace.data_ptr() == place  # (the allocator hands the block on)
        return gp

    gp = used()
    with pytest.raises(binding.MoeError):
        gp.forward(x[:5], w)  # five rows do not make two equal groups
    assert gp.device_status() == (binding.MOE_OK, [0] * 4)
    gp, y = used(), torch.zeros((6, 8), dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gp.forward(x, w, bad, y=y)
    assert gp.device_status() == (binding.MOE_OK, [0] * 4)
    graph.replay()
    assert gp.device_status()[0] == binding.MOE_ERR_DEVICE


def test_objects_may_go_while_their_work_is_queued_on_another_stream():
    """Their memory is nobody else's until the stream that uses it has come past."""
    gen = torch.Generator(device="cuda").manual_seed(14)
    x = torch.randn((40, 64), generator=gen, device="cuda").to(BF16)
    w = torch.randn((2, 72, 64), generator=gen, device="cuda").to(BF16)
    off = torch.tensor([0, 9, 40], dtype=torch.int32, device="cuda")
    want = binding.GroupedProducts(2, 72, 64, BF16).forward(x, w, off)
    want4 = binding.Fp4Weights.quantize(w, "nv").forward(binding.Fp4Rows("nv", 64, 2, 40).quantize(x, off), off)
    gp, r4, w4 = binding.GroupedProducts(2, 72, 64, BF16), binding.Fp4Rows("nv", 64, 2, 40), binding.Fp4Weights.quantize(w, "nv")
    buffers = [gp.workspace, r4.codes, r4.scales, r4.gscale, w4.workspace, w4.codes, w4.scales, w4.gscale]
    places, sizes = {t.data_ptr() for t in buffers}, [t.numel() * t.element_size() for t in buffers]
    del buffers
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1_000_000_000)  # (some 0.5 s)
        y, y4 = gp.forward(x, w, off), w4.forward(r4.quantize(x, off), off)
    del gp, r4, w4
    others = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    assert not side.query() and not places & {t.data_ptr() for t in others}
    side.synchronize()
    assert torch.equal(y, want) and torch.equal(y4, want4)


@pytest.mark.parametrize("op", ["forward", "dgrad", "mx", "nv"])
def test_many_short_units_pass_through_the_pairs(op):
    """Units of one or two K-blocks, some 25 a CTA pair: each slot of the ring that hands them out is written again soon
    after its last reader.  Every row of every call comes from its own unit, and calls repeat bit for bit."""
    groups, rows_each = 500, 40
    n, k = (1024, 64) if op != "dgrad" else (64, 1024)
    lists = Lists([rows_each + (7 * i) % 25 for i in range(groups)])
    gen = torch.Generator(device="cuda").manual_seed(15)
    w = (torch.randn((groups, n, k), generator=gen, device="cuda") * 0.1).to(BF16)
    a = lists.matrix(gen, k if op != "dgrad" else n, BF16)
    if op in ("mx", "nv"):
        r4, w4 = binding.Fp4Rows(op, k, groups, lists.rows).quantize(a, lists.offsets), binding.Fp4Weights.quantize(w, op)
        of, call = w4, lambda: w4.forward(r4, lists.offsets)
        ad, wd = r4.dequantize(lists.offsets, dtype=FP32).double(), w4.dequantize(FP32).double()
    else:
        of = binding.GroupedProducts(groups, n, k, BF16)
        call = (lambda: of.forward(a, w, lists.offsets)) if op == "forward" else lambda: of.dgrad(a, w, lists.offsets)
        ad, wd = a.double(), w.double()
    if op == "dgrad":
        wd = wd.mT.contiguous()
    out = call()
    assert of.device_status()[0] == binding.MOE_OK
    want = torch.empty((lists.rows, wd.shape[1]), dtype=torch.float64, device="cuda")
    s = torch.empty_like(want)
    for g, (lo, hi) in enumerate(lists.spans):
        want[lo:hi], s[lo:hi] = ad[lo:hi] @ wd[g].T, ad[lo:hi].abs() @ wd[g].abs().T
    check(out, want, s, 128)  # (the 4-bit values and steps: 65 / 64 (64 + 64) + 264 2^-23 S, below 17 / 16 (128 + 16) + 256)
    for _ in range(20):
        assert torch.equal(call(), out)


def test_a_c_call_without_rows_leaves_the_status():
    x, w = torch.ones((6, 64), dtype=BF16, device="cuda"), torch.ones((2, 8, 64), dtype=BF16, device="cuda")
    bad = torch.tensor([0, 9, 6], dtype=torch.int32, device="cuda")
    gp = binding.GroupedProducts(2, 8, 64, BF16)
    gp.forward(x, w, bad)
    stream = torch.cuda.current_stream().cuda_stream
    args = (None, 64, w.data_ptr(), bad.data_ptr(), None, None, 8, gp.workspace.data_ptr(), gp.workspace.numel(), stream)
    assert binding.moe_grouped_gemm(gp.shape(0), *args) == binding.MOE_OK
    assert gp.device_status()[0] == binding.MOE_ERR_DEVICE


@pytest.mark.parametrize("out", ["same", "fp32", "accumulate"])
@pytest.mark.parametrize("groups,n,k,dtype", [(300, 520, 776, BF16), (900, 136, 264, FP16), (60, 1032, 1544, FP16)])
def test_weight_gradient_of_many_tiles(groups, n, k, dtype, out):
    """Dozens of tiles for each CTA pair, nearly every one of another group (other tensor maps), empty groups and rests of
    every length among them."""
    lists = Lists([(37 * i) % 150 if i % 5 else 0 for i in range(groups)], gap=1)
    gen = torch.Generator(device="cuda").manual_seed(groups)
    x, dy = lists.matrix(gen, k, dtype), lists.matrix(gen, n, dtype, scale=0.25)
    gp = binding.GroupedProducts(groups, n, k, dtype)
    start = torch.full((groups, n, k), 0.5, device="cuda") if out == "accumulate" else None
    for _ in range(2):
        if out == "accumulate":
            dw = gp.wgrad(dy, x, lists.offsets, lists.counts, dw=start.clone(), accumulate=True)
        else:
            dw = gp.wgrad(dy, x, lists.offsets, lists.counts, dtype=FP32 if out == "fp32" else None)
        assert gp.device_status()[0] == binding.MOE_OK
        for g, (a, b) in enumerate(lists.spans):
            dd, xd = dy[a:b].double(), x[a:b].double()
            want, s = dd.T @ xd, dd.abs().T @ xd.abs()
            if out == "accumulate":
                want, s = want + 0.5, s + 0.5
            check(dw[g], want, s, b - a)


def test_a_long_sum_into_16_bits_captured_first():
    """The workspace's growth inside a capture, replayed on new rows and called beside it."""
    gen = torch.Generator(device="cuda").manual_seed(16)
    x, dy = (torch.randn((9000, c), generator=gen, device="cuda").to(BF16) for c in (72, 136))
    gp = binding.GroupedProducts(1, 136, 72, BF16)
    gp.wgrad(dy[:100], x[:100])
    dw = torch.zeros((1, 136, 72), dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gp.wgrad(dy, x, dw=dw)
    eager = gp.wgrad(dy, x)
    graph.replay()
    assert gp.device_status()[0] == binding.MOE_OK and torch.equal(dw, eager)
    x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
    graph.replay()
    assert torch.equal(dw, gp.wgrad(dy, x))
    dd, xd = dy.double(), x.double()
    check(dw[0], dd.T @ xd, dd.abs().T @ xd.abs(), 3840)
