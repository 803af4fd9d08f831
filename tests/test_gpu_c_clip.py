"""The norm of many tensors and their clipping against the formulas in 64 bits.

u = 2^-24.  Squares of up to 64 elements are added in fp32: 64 roundings of u relative at most, halved by the root; the
norm is rounded to fp32: 33 u.  The factor is rounded once more, and each product: 36 u, then the output's type.
"""
import math

import pytest
import torch

from mixture_experts_layer_rmsnorm_gb300 import binding
from test_gpu_8_grouped import BF16, FP16, FP32, half_step

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6
NAN, INF = float("nan"), float("inf")


def make(sizes, types, scale=1.0, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=gen, device="cuda") * scale).to(t) for n, t in zip(sizes, types)]


def norm_of(tensors):
    return math.sqrt(math.fsum(float(t.double().square().sum()) for t in tensors))


def check_clipped(tensors, out, norm, max_norm, eps=EPS):
    f = min(1.0, max_norm / (norm + eps))
    for t, o in zip(tensors, out):
        want = t.double() * f
        lim = want.abs() * (36 * U + half_step(o.dtype)) * (1 + U) + (2.0 ** -25 if o.dtype == FP16 else 2.0 ** -133)
        assert ((o.double() - want).abs() <= lim).all()


SETS = {
    "one_number": ([1], [FP32]),
    "one_chunk": ([16384], [BF16]),
    "a_chunk_and_a_number": ([16385, 0, 3], [FP32, FP32, FP16]),
    "few": ([5, 70000, 1, 16383, 8, 200001], [BF16, FP16, FP32, FP32, BF16, BF16]),
    "thirty_three": ([i * i * 37 for i in range(33)], [(BF16, FP16, FP32)[i % 3] for i in range(33)]),
    "a_small_table": ([1 + (i * 131) % 700 for i in range(300)], [(BF16, FP32)[i % 2] for i in range(300)]),
    "one_more": ([1 + (i * 131) % 700 for i in range(301)], [(FP32, FP16)[i % 2] for i in range(301)]),
    "more_than_a_launch": ([1 + (i * 7919) % 3000 for i in range(2001)], [(FP32, BF16)[i % 2] for i in range(2001)]),
    "large": ([30000000, 1, 20000003], [FP32, BF16, BF16]),
}


@pytest.mark.parametrize("name", SETS)
def test_norm_and_clip(name):
    sizes, types = SETS[name]
    g = make(sizes, types, 0.02)
    want = norm_of(g)
    kept = [t.clone() for t in g]
    grads = binding.Gradients(g)
    norm = grads.norm()
    assert norm.shape == () and abs(norm.item() - want) <= 33 * U * want
    assert torch.equal(grads.norm(), norm)
    # below the limit: untouched
    assert torch.equal(grads.clip(want * 2), norm)
    assert all(torch.equal(a, b) for a, b in zip(g, kept))
    # above: apart, into any type, then in place
    for out_type in (BF16, FP16, FP32):
        out = [torch.empty_like(t, dtype=out_type) for t in g]
        assert torch.equal(binding.Gradients(g, out).clip(want / 3), norm)
        check_clipped(kept, out, want, want / 3)
        assert all(torch.equal(a, b) for a, b in zip(g, kept))
        binding.Gradients(g, out).clip(want * 2)  # a factor of 1 copies
        assert all(torch.equal(o, t.to(out_type)) for o, t in zip(out, g))
    grads.clip(want / 3)
    check_clipped(kept, g, want, want / 3)


def test_tensors_off_16_byte_borders():
    base = [torch.randn(50011, device="cuda").to(t) for t in (BF16, FP16, FP32)]
    g = [b[i + 1:i + 1 + n] for i, (b, n) in enumerate(zip(base, (40001, 7, 50000)))]
    kept = [b.clone() for b in base]
    want = norm_of(g)
    norm = binding.Gradients(g).clip(want / 2)
    assert abs(norm.item() - want) <= 33 * U * want
    check_clipped([k[i + 1:i + 1 + t.numel()] for i, (k, t) in enumerate(zip(kept, g))], g, want, want / 2)
    for i, (b, k, t) in enumerate(zip(base, kept, g)):
        assert torch.equal(b[:i + 1], k[:i + 1]) and torch.equal(b[i + 1 + t.numel():], k[i + 1 + t.numel():])


@pytest.mark.parametrize("values,types", [
    ([3e38, -2e38, 1e30], [FP32, BF16, FP32]),       # squares beyond fp32
    ([1e-30, 2e-38, -3e-28], [FP32, BF16, BF16]),    # squares below it
    ([1e30, 1e-30, 1.0], [FP32, FP32, FP16]),
    ([2.0 ** -24, 65504.0, -2.0 ** -20], [FP16, FP16, FP16]),
])
def test_elements_of_extreme_sizes(values, types):
    g = [torch.full((n,), v, dtype=t, device="cuda") for v, t, n in zip(values, types, (1001, 17, 16400))]
    want = norm_of(g)
    norm = binding.Gradients(g).norm().item()
    assert norm == INF if want > 3.4028235e38 else abs(norm - want) <= 33 * U * want + 2.0 ** -150


def test_zeros_and_no_tensors():
    g = [torch.zeros(40000, dtype=BF16, device="cuda"), torch.zeros(0, device="cuda")]
    assert binding.Gradients(g).clip(1.0).item() == 0.0 and torch.all(g[0] == 0.0)
    assert binding.Gradients([]).clip(1.0).item() == 0.0
    one = [torch.ones(4, device="cuda")]
    binding.Gradients(one).clip(0.0)
    assert torch.all(one[0] == 0.0)


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_a_norm_that_is_no_number_clips_nothing(bad):
    g = make([100, 50000], [FP32, BF16])
    g[1][33333] = bad
    kept = [t.clone() for t in g]
    norm = binding.Gradients(g).clip(0.5)
    assert torch.isnan(norm) if bad != bad else norm == INF
    assert all(torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)) for a, b in zip(g, kept))


def test_a_norm_of_these_and_others():
    g = make([1000, 300], [FP32, BF16])
    kept = [t.clone() for t in g]
    total = torch.tensor(500.0, device="cuda")
    assert binding.Gradients(g).clip(5.0, norm=total) is total
    check_clipped(kept, g, 500.0, 5.0)


@pytest.mark.parametrize("n", [1, 20, 1300, 3500])
def test_calls_follow_one_another_without_a_pause(n):
    """Each call reads what the one before wrote, in place; a call of many tensors is several launches, whose later ones
    begin beside the first."""
    sizes = [1 + (i * 7919) % 20000 for i in range(n)]
    flat = torch.randn(sum(sizes), generator=torch.Generator(device="cuda").manual_seed(n), device="cuda")
    start, src = flat.clone(), flat * 3

    def run(pause):
        flat.copy_(src)
        flat.mul_(1 / 3)
        grads = binding.Gradients(list(flat.split(sizes)))
        norms = []
        for k in range(8):
            norms.append(grads.clip(first * 0.7 ** (k + 1)) if k % 2 else grads.clip(first * 0.7 ** (k + 1), norm=grads.norm()))
            if pause:
                torch.cuda.synchronize()
        return torch.stack(norms), flat.clone()

    first = norm_of([start])
    norms, out = run(False)
    paused, same = run(True)
    assert torch.equal(norms, paused) and torch.equal(out, same)
    for k, norm in enumerate(norms.tolist()):  # each clipping leaves 36 u, and the source's two roundings
        want = first * 0.7 ** k
        assert abs(norm - want) <= (36 * k + 33 + 4) * U * want + EPS * k


@pytest.mark.parametrize("sizes", [[7], [100000, 33, 5], [777] * 1500, [33] * 3500])
def test_replays_from_a_graph_on_new_gradients(sizes):
    g = make(sizes, [FP32] * len(sizes))
    out = [torch.empty_like(t) for t in g]
    grads = binding.Gradients(g, out)
    grads.clip(1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        norm = grads.clip(1.0)
    for t in g:
        t.mul_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    first = [t.clone() for t in out]
    want = norm_of(g)
    assert abs(norm.item() - want) <= 33 * U * want
    assert torch.equal(grads.clip(1.0), norm) and all(torch.equal(a, b) for a, b in zip(first, out))


def test_tensors_of_more_than_2_to_the_32_elements():
    n = 2 ** 32 + 12345
    g = torch.full((n,), 2.0 ** -10, dtype=BF16, device="cuda")
    g[-1] = 3.0
    want = math.sqrt((n - 1) * 2.0 ** -20 + 9.0)
    norm = binding.Gradients([g]).clip(want / 2)
    assert abs(norm.item() - want) <= 33 * U * want
    f = (want / 2) / (want + EPS)
    assert abs(g[-1].item() - 3.0 * f) <= 3.0 * f * (36 * U + 2.0 ** -8)
    assert (g[:-1].float() == torch.tensor(2.0 ** -10 * f).to(BF16).float().item()).all()


def test_objects_refuse_what_does_not_fit():
    t = torch.ones(8, device="cuda")
    with pytest.raises(ValueError):
        binding.Gradients([t], [t, t])
    with pytest.raises(ValueError):
        binding.Gradients([t], [torch.ones(7, device="cuda")])
    with pytest.raises(TypeError):
        binding.Gradients([t.double()])
    with pytest.raises(ValueError):
        binding.Gradients([torch.ones((4, 4), device="cuda").t()])
    with pytest.raises(ValueError):
        binding.Gradients([t, t.cpu()])
    pair, half = torch.ones(16, device="cuda"), torch.ones(16, dtype=BF16, device="cuda")
    for tensors, out in (([t, t], None), ([pair[:9], pair[8:]], None), ([pair[:8], pair[8:]], [pair[8:], pair[:8]]),
                         ([pair[:4], pair[4:8]], [pair[8:12], pair[10:14]]), ([half[:8]], [half[4:12]])):
        with pytest.raises(ValueError):
            binding.Gradients(tensors, out)
    binding.Gradients([pair[:8], pair[8:]]).clip(1.0)  # side by side
    binding.Gradients([pair, pair], [t.new_empty(16), t.new_empty(16)]).clip(1.0)  # read twice, written apart
    for max_norm, eps in ((-1.0, 0.0), (NAN, 0.0), (1.0, -1e-6), (1.0, INF)):
        with pytest.raises(binding.MoeError):
            binding.Gradients([t]).clip(max_norm, eps)
    with pytest.raises(ValueError):
        binding.Gradients([t]).clip(1.0, norm=t)
