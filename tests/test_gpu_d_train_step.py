"""A training step of the experts with its operators together: norm of the rows, both products in 8 bits forward and for
the inputs' gradients, SwiGLU, the weights' gradients in 16 bits, the norm's gradient, the norm of all gradients and
clipping.  Each stage against 64 bits on the operands that the step hands it (what is rounded to 8 bits between two
stages is compared as codes, so no error is carried along), the whole captured and replayed, and on two streams at once.

Tolerances: those of the operators' own tests, on operands of this step.
"""
import threading

import pytest
import torch

from mixture_experts_layer_rmsnorm_gb300 import binding
from test_gpu_8_grouped import BF16, FP32, check, half_step
from test_gpu_a_fp8 import define

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


class Step:
    """The experts of one layer, [groups, 2I, H] and [groups, H, I], on rows that are sorted by expert."""

    def __init__(self, counts, hidden, inter, seed=0, dtype=BF16, max_norm=0.5):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def rand(*shape, scale=1.0):
            return torch.randn(shape, generator=gen, device="cuda") * scale

        self.counts, self.h, self.i, self.rows, self.dtype, self.max_norm = counts, hidden, inter, sum(counts), dtype, max_norm
        g = len(counts)
        self.offsets = torch.tensor([sum(counts[:k]) for k in range(g + 1)], dtype=torch.int32, device="cuda")
        self.x, self.dy = rand(self.rows, hidden).to(dtype), rand(self.rows, hidden, scale=0.1).to(dtype)
        self.gain = 1 + rand(hidden, scale=0.1)
        self.w13 = rand(g, 2 * inter, hidden, scale=hidden ** -0.5).to(dtype)
        self.w2 = rand(g, hidden, inter, scale=inter ** -0.5).to(dtype)
        self.norm = binding.RowNorm(hidden, "rms", dtype, FP32)
        self.w13_8, self.w2_8 = binding.Fp8Weights.quantize(self.w13), binding.Fp8Weights.quantize(self.w2)
        self.rows8 = {name: binding.Fp8Rows(width, self.rows) for name, width in
                      (("x", hidden), ("act", inter), ("dy", hidden), ("dh", 2 * inter))}
        self.up, self.down = binding.GroupedProducts(g, 2 * inter, hidden, dtype), binding.GroupedProducts(g, hidden, inter, dtype)
        self.grads = [torch.zeros(s, device="cuda") for s in ((g, 2 * inter, hidden), (g, hidden, inter), (hidden,))]
        self.clipped = [torch.zeros_like(t, dtype=dtype) for t in self.grads]
        self.gradients = binding.Gradients(self.grads, self.clipped)
        # what the step returns, in the caller's buffers
        self.y, self.dx = torch.empty_like(self.x), torch.empty_like(self.x)
        self.total = torch.zeros((), device="cuda")

    def run(self):
        off, s = self.offsets, {}
        s["xn"], s["rstd"] = self.norm.forward(self.x, self.gain, stats=True)
        s["h"] = self.w13_8.forward(self.rows8["x"].quantize(s["xn"]), off)
        s["act"] = binding.swiglu(s["h"])
        self.w2_8.forward(self.rows8["act"].quantize(s["act"]), off, y=self.y)
        s["dact"] = self.w2_8.dgrad(self.rows8["dy"].quantize(self.dy), off)
        self.down.wgrad(self.dy, s["act"], off, dw=self.grads[1])
        s["dh"] = binding.swiglu_grad(s["h"], s["dact"])
        s["dxn"] = self.w13_8.dgrad(self.rows8["dh"].quantize(s["dh"]), off)
        self.up.wgrad(s["dh"], s["xn"], off, dw=self.grads[0])
        self.norm.grad(s["dxn"], self.x, self.gain, s["rstd"], dx=self.dx, dweight=self.grads[2])
        self.total.copy_(self.gradients.clip(self.max_norm))
        return s

    def results(self):
        return [self.y, self.dx, self.total, *self.grads, *self.clipped]

    def spans(self):
        a = 0
        for g, n in enumerate(self.counts):
            yield g, slice(a, a + n)
            a += n


def near(got, want, lim):
    lim = lim + half_step(got.dtype) * (want.abs() + lim)
    worst = ((got.double() - want).abs() - lim).max().item() if got.numel() else 0.0
    assert worst <= 0, f"error above its bound by {worst:.3e}"


def check_product(st, got, rows, weights, transposed):
    """An 8-bit product on what ``rows`` and ``weights`` (16 bits) stand for in 8 bits."""
    xv, wv = define(rows, 1)[2], define(weights, 128)[2]
    terms = weights.shape[1 if transposed else 2]
    for g, at in st.spans():
        w = wv[g] if transposed else wv[g].T
        near(got[at], xv[at] @ w, (132 + (-(-terms // 128) + 257) / 2) * 2.0 ** -23 * (xv[at].abs() @ w.abs()))


@pytest.mark.parametrize("counts,hidden,inter", [
    ([3, 0, 1, 7, 16], 256, 144),          # few rows a group, one without
    ([130, 40, 0, 97], 400, 128),          # a group of more than a tile; blocks that end inside 128
    ([300, 511, 256], 512, 272),           # pairs of tiles
])
def test_each_stage_of_a_step(counts, hidden, inter):
    st = Step(counts, hidden, inter)
    s = st.run()
    x, gain = st.x.double(), st.gain.double()
    r = 1 / torch.sqrt(x.square().mean(1, keepdim=True) + st.norm.eps)
    near(s["rstd"], r[:, 0], 30 * U * r[:, 0])
    near(s["xn"], x * r * gain, 34 * U * (x * r * gain).abs())
    check_product(st, s["h"], s["xn"], st.w13, False)
    gate, up = s["h"].double().chunk(2, 1)
    sig, rest = torch.special.expit(gate), torch.special.expit(-gate)
    rel = (gate.abs() + 16) * 2.0 ** -23
    near(s["act"], gate * sig * up, rel * (gate * sig * up).abs() + 2.0 ** -126)
    check_product(st, st.y, s["act"], st.w2, False)
    check_product(st, s["dact"], st.dy, st.w2, True)
    da = s["dact"].double()
    near(s["dh"][:, :inter], da * up * sig * (1 + gate * rest), rel * (da * up).abs() * sig * (1 + gate.abs() * rest) + 2.0 ** -126)
    near(s["dh"][:, inter:], da * gate * sig, rel * (da * gate * sig).abs() + 2.0 ** -126)
    check_product(st, s["dxn"], s["dh"], st.w13, True)
    for got, dy, xs in ((st.grads[0], s["dh"], s["xn"]), (st.grads[1], st.dy, s["act"])):
        for g, at in st.spans():
            d, v = dy[at].double(), xs[at].double()
            check(got[g], d.T @ v, d.abs().T @ v.abs(), min(d.shape[0], 768))
    n, e = x * s["rstd"].double()[:, None], s["dxn"].double() * gain
    rs = s["rstd"].double()[:, None]
    c1 = (e * n).mean(1, keepdim=True)
    near(st.dx, rs * (e - n * c1), rs * (n.abs() * 56 * U * (e * n).abs().mean(1, keepdim=True) + 4 * U * e.abs()))
    terms = s["dxn"].double() * n
    near(st.grads[2], terms.sum(0), (4 + st.rows) * U * terms.abs().sum(0))
    total = sum(t.double().square().sum() for t in st.grads).sqrt()
    near(st.total, total, 33 * U * total)
    f = min(1.0, st.max_norm / (total.item() + 1e-6))
    assert f < 1.0
    for got, t in zip(st.clipped, st.grads):
        near(got, t.double() * f, 36 * U * (t.double() * f).abs() + 2.0 ** -133)


@pytest.mark.parametrize("counts", [[3, 0, 9], [70, 128, 5], [256, 300, 12]])
def test_the_input_gradient_is_the_forward_product_transposed(counts):
    """<dy, x w^T> = <dy w, x> for the values that the codes stand for; what lies between is each output's rounding and
    its accumulation, as bounded above."""
    st = Step(counts, 272, 144)
    x, dy, w = define(st.x, 1)[2], define(st.x[:, :144].contiguous(), 1)[2], define(st.w13[:, :144], 128)[2]
    w8 = binding.Fp8Weights.quantize(st.w13[:, :144].contiguous())
    y = w8.forward(st.rows8["x"].quantize(st.x), st.offsets)
    dx = w8.dgrad(binding.Fp8Rows(144, st.rows).quantize(st.x[:, :144]), st.offsets)
    one, other, lim = 0.0, 0.0, 0.0
    for g, at in st.spans():
        one, other = one + (dy[at] * y[at].double()).sum(), other + (dx[at].double() * x[at]).sum()
        size = (dy[at].abs() * (x[at].abs() @ w[g].abs().T)).sum()
        lim = lim + 2 * (132 + 130) * 2.0 ** -23 * size
        lim = lim + half_step(BF16) * ((dy[at] * y[at].double()).abs().sum() + (dx[at].double() * x[at]).abs().sum()) * 1.01
    assert (one - other).abs() <= lim


def test_a_step_repeats_bit_for_bit_and_replays_on_new_rows_and_lists():
    st = Step([30, 1, 0, 201, 24], 384, 160)
    st.run()
    first = [t.clone() for t in st.results()]
    st.run()
    assert all(torch.equal(a, b) for a, b in zip(first, st.results()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        st.run()
    gen = torch.Generator(device="cuda").manual_seed(9)
    st.x.copy_(torch.randn(st.x.shape, generator=gen, device="cuda"))
    st.dy.copy_(torch.randn(st.dy.shape, generator=gen, device="cuda"))
    st.offsets.copy_(torch.tensor([0, 0, 100, 130, 131, 256], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in st.results()]
    assert not torch.equal(replayed[0], first[0])
    st.run()
    assert all(torch.equal(a, b) for a, b in zip(replayed, st.results()))


def test_two_steps_on_their_own_streams_and_host_threads():
    shapes = [([64, 3, 90], 256, 128), ([5, 0, 2, 9, 1, 1], 512, 144)]
    alone = []
    for k, shape in enumerate(shapes):
        st = Step(*shape, seed=k)
        st.run()
        alone.append([t.clone() for t in st.results()])
    steps = [Step(*shape, seed=k) for k, shape in enumerate(shapes)]
    torch.cuda.synchronize()
    failures = []

    def work(st):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    st.run()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # (an assertion of its own thread)
            failures.append(e)

    threads = [threading.Thread(target=work, args=(st,)) for st in steps]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures
    for st, want in zip(steps, alone):
        assert all(torch.equal(a, b) for a, b in zip(st.results(), want))


def test_padded_rows_behind_the_last_list_stay_out():
    """Rows that belong to no expert hold NaN: no product, gradient of a weight or row of a group sees them."""
    st = Step([17, 40, 3], 256, 128)
    st.run()
    want = [t.clone() for t in st.grads[:2]] + [st.y.clone()]
    padded = Step([17, 40, 3, 9], 256, 128)
    off = torch.cat([st.offsets, st.offsets[-1:]])  # the last expert has no row, nine rows have no expert
    padded.offsets.copy_(off)
    for a, b in ((padded.w13_8, st.w13_8), (padded.w2_8, st.w2_8)):
        a.codes[:3].copy_(b.codes)
        a.scales[:3].copy_(b.scales)
    padded.x[:60].copy_(st.x), padded.dy[:60].copy_(st.dy), padded.gain.copy_(st.gain)
    padded.x[60:], padded.dy[60:] = float("nan"), float("nan")
    padded.y.fill_(7.0)
    padded.run()
    assert torch.equal(padded.y[:60], want[2]) and torch.all(padded.y[60:] == 7.0)
    for got, ref in zip(padded.grads[:2], want):
        assert torch.equal(got[:3], ref) and torch.all(got[3] == 0.0)
