"""Clipping at the ends of fp32's range, against the formula in 64 bits; tolerances as for ordinary numbers."""
import math

import pytest
import torch

from mixture_experts_layer_rmsnorm_gb300 import binding
from test_gpu_8_grouped import BF16, FP32
from test_gpu_c_clip import INF, U, check_clipped, norm_of

pytestmark = pytest.mark.gpu


def large(sizes, values, types):
    """Tensors of the sizes, filled with the values (from 1 to 2 times, by place) and of the types, in turn."""
    return [(torch.linspace(1, 2, n, device="cuda") * values[i % len(values)]).to(types[i % len(types)])
            for i, n in enumerate(sizes)]


@pytest.mark.parametrize("max_norm", [1.0, 1e-3, 1e-6, 1e-30])
@pytest.mark.parametrize("out", [None, BF16, FP32])
def test_factors_below_fp32s_normal_numbers(max_norm, out):
    """Norms that are fp32 numbers, and factors down to 2^-226: the results lie inside fp32's range."""
    g = large([1001, 17, 20000, 3], [4e36, -4e35, 4e30], [FP32, BF16])
    kept, want = [t.clone() for t in g], norm_of(g)
    assert want < 3e38 and max_norm / want < 2.0 ** -126
    into = g if out is None else [torch.empty_like(t, dtype=out) for t in g]
    norm = binding.Gradients(g, None if out is None else into).clip(max_norm)
    assert abs(norm.item() - want) <= 33 * U * want
    check_clipped(kept, into, want, max_norm)
    g = [t.clone() for t in kept]  # and by a norm already known
    binding.Gradients(g).clip(max_norm, norm=norm)
    check_clipped(kept, g, want, max_norm)


@pytest.mark.parametrize("n", [1, 20, 400, 1300, 3500])
def test_finite_gradients_whose_norm_passes_fp32(n):
    """The norm as an fp32 number is infinity, but the tensors are clipped by its value."""
    sizes = [1001] + [1 + (i * 7919) % 300 for i in range(n - 1)]
    g = large(sizes, [1.5e38, -1e37, 1e20], [FP32, BF16, FP32])
    kept, want = [t.clone() for t in g], norm_of(g)
    assert want > 3.5e38
    for max_norm in (1.0, 1e37):
        for out_type in (BF16, FP32):
            out = [torch.empty_like(t, dtype=out_type) for t in g]
            assert binding.Gradients(g, out).clip(max_norm).item() == INF
            check_clipped(kept, out, want, max_norm)
    grads = binding.Gradients(g)
    assert grads.clip(math.inf).item() == INF and all(torch.equal(a, b) for a, b in zip(g, kept))
    # (a norm that was rounded to fp32 before says no more than that it is infinite)
    assert grads.clip(1.0, norm=grads.norm()).item() == INF and all(torch.equal(a, b) for a, b in zip(g, kept))
    assert grads.clip(1.0).item() == INF
    check_clipped(kept, g, want, 1.0)


def test_a_finite_norm_beyond_fp32_replays_from_a_graph():
    g = large([5000, 33], [1.5e38, 1e38], [FP32, BF16])
    out = [torch.empty_like(t) for t in g]
    grads = binding.Gradients(g, out)
    grads.clip(2.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        norm = grads.clip(2.0)
    for t in g:
        t.mul_(0.75)
    graph.replay()
    torch.cuda.synchronize()
    assert norm.item() == INF
    check_clipped(g, out, norm_of(g), 2.0)
    g[0][77] = INF  # no number: nothing is clipped
    graph.replay()
    torch.cuda.synchronize()
    assert norm.item() == INF and all(torch.equal(a, b) for a, b in zip(g, out))
