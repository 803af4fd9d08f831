"""The grouped products and SwiGLU refuse bad arguments on the host, before anything is enqueued (no GPU needed)."""
import pytest

from mixture_experts_layer_rmsnorm_gb300 import binding

OK, INV, UNS, WS = (binding.MOE_OK, binding.MOE_ERR_INVALID_ARG, binding.MOE_ERR_UNSUPPORTED,
                    binding.MOE_ERR_WORKSPACE)
A = 0x10000  # an aligned address that no refused call reads
BIG = 1 << 40


@pytest.mark.parametrize("groups,n,k,rows,type_,want", [
    (1, 8, 8, 0, 0, OK), (1024, 1 << 20, 1 << 20, (1 << 31) - 512, 1, OK),
    (0, 8, 8, 1, 0, INV), (1, 0, 8, 1, 0, INV), (1, 8, -8, 1, 0, INV), (1, 8, 8, -1, 0, INV),
    (1, 8, 8, 1, 2, INV), (1, 8, 8, 1, 3, INV),
    (1025, 8, 8, 1, 0, UNS), (1, 12, 8, 1, 0, UNS), (1, 8, 7, 1, 0, UNS), (1, (1 << 20) + 8, 8, 1, 0, UNS),
    (1, 8, 8, 1 << 31, 0, UNS),
])
def test_shapes(groups, n, k, rows, type_, want):
    st, size = binding.moe_grouped_workspace_size(binding.grouped_shape(groups, n, k, rows, type_))
    assert st == want and (size > 0) == (want == OK)


def call(fn, **over):
    a = dict(groups=4, N=64, K=128, rows=20, type=0, a=A, lda=128, b=A, off=A, cnt=None, out=A, ldo=64, ws=A, ws_bytes=BIG)
    a.update(over)
    s = binding.grouped_shape(a["groups"], a["N"], a["K"], a["rows"], a["type"])
    return fn(s, a["a"], a["lda"], a["b"], a["off"], a["cnt"], a["out"], a["ldo"], a["ws"], a["ws_bytes"], None)


BAD = [
    (dict(a=None), INV), (dict(b=None), INV), (dict(out=None), INV), (dict(ws=None), INV),
    (dict(a=A + 8), INV), (dict(b=A + 2), INV), (dict(out=A + 4), INV), (dict(ws=A + 64), INV), (dict(off=A + 2), INV),
    (dict(cnt=A + 1), INV), (dict(rows=21, off=None), INV), (dict(ws_bytes=1024), WS), (dict(type=2), INV),
    (dict(rows=-1), INV), (dict(groups=0), INV), (dict(N=60), UNS), (dict(K=1), UNS),
]


@pytest.mark.parametrize("over,want", BAD + [(dict(lda=120), INV), (dict(ldo=56), INV), (dict(lda=132), UNS),
                                             (dict(ldo=68), UNS)])
def test_forward_refuses(over, want):
    assert call(binding.moe_grouped_gemm, **over) == want


@pytest.mark.parametrize("over,want", BAD + [(dict(lda=56), INV), (dict(ldo=120), INV), (dict(lda=68), UNS),
                                             (dict(ldo=132), UNS)])
def test_input_gradient_refuses(over, want):
    assert call(binding.moe_grouped_gemm_dgrad, **{"lda": 64, "ldo": 128, **over}) == want


@pytest.mark.parametrize("over,want", [
    (dict(dy=None), INV), (dict(x=None), INV), (dict(dw=None), INV), (dict(dw=A + 8), INV), (dict(lddy=56), INV),
    (dict(ldx=120), INV), (dict(ldx=133), UNS), (dict(dw_type=1), INV), (dict(dw_type=3), INV), (dict(accumulate=1), INV),
    (dict(ws_bytes=0), WS), (dict(off=None, rows=21), INV),
])
def test_weight_gradient_refuses(over, want):
    a = dict(rows=20, dy=A, lddy=64, x=A, ldx=128, off=A, dw=A, dw_type=0, accumulate=0, ws_bytes=BIG)
    a.update(over)
    s = binding.grouped_shape(4, 64, 128, a["rows"])
    assert binding.moe_grouped_gemm_wgrad(s, a["dy"], a["lddy"], a["x"], a["ldx"], a["off"], None, a["dw"], a["dw_type"],
                                          a["accumulate"], A, a["ws_bytes"], None) == want


def test_no_rows_is_a_no_op():
    assert call(binding.moe_grouped_gemm, rows=0, a=None, out=None) == OK
    assert call(binding.moe_grouped_gemm_dgrad, rows=0, a=None, out=None, lda=64, ldo=128) == OK
    s = binding.grouped_shape(4, 64, 128, 0)
    assert binding.moe_grouped_gemm_wgrad(s, None, 64, None, 128, A, None, A, 2, 1, A, BIG, None) == OK
    assert binding.moe_swiglu(0, 0, 64, None, 128, None, 64, None) == OK
    assert binding.moe_swiglu_grad(1, 0, 64, None, 128, None, 64, None, 128, None) == OK


@pytest.mark.parametrize("type_,rows,i,h,ldh,act,ldact,want", [
    (2, 4, 64, A, 128, A, 64, INV), (0, -1, 64, A, 128, A, 64, INV), (0, 4, 0, A, 128, A, 64, INV),
    (0, 4, 60, A, 128, A, 64, UNS), (0, 4, 64, A, 120, A, 64, INV), (0, 4, 64, A, 132, A, 64, UNS),
    (0, 4, 64, None, 128, A, 64, INV), (0, 4, 64, A, 128, A + 2, 64, INV), (0, 4, 64, A, 128, A, 56, INV),
    (0, 1 << 31, 64, A, 128, A, 64, UNS), (0, 1 << 30, 64, A, 128, A, 64, UNS),
])
def test_swiglu_refuses(type_, rows, i, h, ldh, act, ldact, want):
    assert binding.moe_swiglu(type_, rows, i, h, ldh, act, ldact, None) == want
    if ldact == 64 and act == A:
        assert binding.moe_swiglu_grad(type_, rows, i, h, ldh, act, 64, A, 128, None) == want


@pytest.mark.parametrize("fmt,groups,rows,k,want", [
    (0, 1, 1, 32, OK), (1, 1024, 1 << 20, 1 << 20, OK), (2, 1, 1, 32, INV), (0, 0, 1, 32, INV), (0, 1, -1, 32, INV),
    (0, 1, 1, 0, INV), (1, 1, 1, 16, UNS), (0, 1, 1, 48, UNS), (0, 1025, 1, 32, UNS), (0, 1, 1 << 31, 32, UNS),
    (0, 1, 1, (1 << 20) + 32, UNS),
])
def test_fp4_sizes(fmt, groups, rows, k, want):
    st, (codes, scales) = binding.moe_fp4_sizes(binding.fp4_shape(fmt, groups, rows, k))
    assert st == want
    if want == OK:
        chunk = 128 if fmt == 0 else 64
        assert codes == rows * k // 2 and scales == (rows // 128 + groups) * -(-k // chunk) * 512


FP4_BAD = [(dict(src=None), INV), (dict(src=A + 8), INV), (dict(ld=60), INV), (dict(ld=68), UNS), (dict(type=3), INV),
           (dict(codes=None), INV), (dict(codes=A + 8), INV), (dict(scales=None), INV), (dict(scales=A + 4), INV),
           (dict(gscale=None), INV), (dict(gscale=A + 2), INV), (dict(per=2), INV), (dict(off=None), INV),
           (dict(off=A + 2), INV), (dict(K=48), UNS), (dict(format=5), INV)]


@pytest.mark.parametrize("over,want", FP4_BAD)
def test_fp4_rows_refuse(over, want):
    a = dict(format=1, groups=2, rows=7, K=64, type=0, src=A, ld=64, off=A, cnt=None, codes=A, scales=A, gscale=A, per=0)
    a.update(over)
    s = binding.fp4_shape(a["format"], a["groups"], a["rows"], a["K"])
    assert binding.moe_fp4_quantize(s, a["type"], a["src"], a["ld"], a["off"], a["cnt"], a["codes"], a["scales"],
                                    a["gscale"], a["per"], None) == want
    assert binding.moe_fp4_dequantize(s, a["codes"], a["scales"], a["gscale"], a["per"], a["off"], a["cnt"], a["type"],
                                      a["src"], a["ld"], None) == want


@pytest.mark.parametrize("over,want", [
    (dict(xc=None), INV), (dict(xs=A + 8), INV), (dict(xg=None), INV), (dict(wc=A + 8), INV), (dict(ws=None), INV),
    (dict(wg=None), INV), (dict(off=None), INV), (dict(y=None), INV), (dict(ldy=56), INV), (dict(ldy=70), UNS),
    (dict(space=A + 16), INV), (dict(space_bytes=64), WS), (dict(K=48), UNS), (dict(N=60), UNS), (dict(format=2), INV),
    (dict(type=2), INV), (dict(rows=0, xc=None, xs=None, xg=None, y=None), OK),
])
def test_fp4_product_refuses(over, want):
    a = dict(format=1, groups=2, rows=7, N=64, K=64, type=0, xc=A, xs=A, xg=A, wc=A, ws=A, wg=A, off=A, y=A, ldy=64,
             space=A, space_bytes=BIG)
    a.update(over)
    s = binding.grouped_shape(a["groups"], a["N"], a["K"], a["rows"], a["type"])
    assert binding.moe_fp4_gemm(s, a["format"], a["xc"], a["xs"], a["xg"], a["wc"], a["ws"], a["wg"], a["off"], None,
                                a["y"], a["ldy"], a["space"], a["space_bytes"], None) == want


def test_swiglu_gradient_in_place_has_one_stride():
    assert binding.moe_swiglu_grad(0, 4, 64, A, 128, 2 * A, 64, A, 136, None) == INV


def test_weight_gradient_into_16_bits_of_too_many_rows():
    for rows, want in (((1 << 26) + 1, UNS), (1 << 26, WS)):  # (the second is refused for its workspace alone)
        s = binding.grouped_shape(4, 64, 128, rows)
        ws = 64 if want == WS else BIG
        assert binding.moe_grouped_gemm_wgrad(s, A, 64, A, 128, A, None, A, 0, 0, A, ws, None) == want


def test_weight_gradient_into_16_bits_of_long_groups_wants_its_larger_workspace():
    sizes = [binding.moe_grouped_workspace_size(binding.grouped_shape(4, 64, 128, rows))[1] for rows in (0, 3840, 3841)]
    assert sizes[0] == sizes[1] < sizes[2]
    s = binding.grouped_shape(4, 64, 128, 3841)
    assert binding.moe_grouped_gemm_wgrad(s, A, 64, A, 128, A, None, A, 0, 0, A, sizes[2] - 1, None) == WS


def test_tensors_on_the_cpu_are_refused():
    import torch
    bf16, w = torch.bfloat16, torch.zeros((2, 64, 128), dtype=torch.bfloat16)
    h, act = torch.zeros((4, 128), dtype=bf16), torch.zeros((4, 64), dtype=bf16)
    gp, r4 = binding.GroupedProducts(2, 64, 128, bf16, device="cpu"), binding.Fp4Rows("nv", 128, 2, 4, device="cpu")
    for call in (lambda: binding.swiglu(h), lambda: binding.swiglu_grad(h, act), lambda: gp.forward(h, w),
                 lambda: gp.dgrad(act, w), lambda: gp.wgrad(act, h), lambda: r4.quantize(h),
                 lambda: binding.Fp4Weights.quantize(w, "mx")):
        with pytest.raises(ValueError, match="not on a CUDA device"):
            call()
    assert gp.device_status() == (OK, [0] * 4) and r4.rows == 0
