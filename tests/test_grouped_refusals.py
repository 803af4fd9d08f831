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
