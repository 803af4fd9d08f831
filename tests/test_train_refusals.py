"""The 8-bit rows and products, the norms of rows and the clipping refuse bad arguments on the host, before anything is
enqueued (no GPU needed)."""
import pytest

from mixture_experts_layer_rmsnorm_gb300 import binding

OK, INV, UNS, WS = (binding.MOE_OK, binding.MOE_ERR_INVALID_ARG, binding.MOE_ERR_UNSUPPORTED,
                    binding.MOE_ERR_WORKSPACE)
A = 0x10000  # an aligned address that no refused call reads
BIG = 1 << 40
NAN, INF = float("nan"), float("inf")
ROW, GROUP, BLOCK = binding.MOE_SCALE_PER_ROW, binding.MOE_SCALE_PER_GROUP, binding.MOE_SCALE_PER_BLOCK


@pytest.mark.parametrize("per,groups,rows,k,want", [
    (ROW, 0, 0, 16, OK), (ROW, 7, (1 << 31) - 512, 1 << 20, OK), (BLOCK, 3, 3 * 200, 400, OK), (BLOCK, 1024, 0, 16, OK),
    (GROUP, 1, 4, 16, INV), (3, 1, 4, 16, INV), (ROW, 1, -1, 16, INV), (ROW, 1, 4, 0, INV), (BLOCK, 0, 4, 16, INV),
    (BLOCK, 3, 4, 16, INV), (ROW, 1, 4, 24, UNS), (ROW, 1, 4, (1 << 20) + 16, UNS), (ROW, 1, 1 << 31, 16, UNS),
    (BLOCK, 1025, 1025, 16, UNS), (BLOCK, 1, (1 << 31) - 512, 1 << 20, UNS),
])
def test_fp8_shapes(per, groups, rows, k, want):
    st, (codes, scales) = binding.moe_fp8_sizes(binding.fp8_shape(per, groups, rows, k))
    assert st == want
    if want == OK:
        assert codes == rows * k
        blocks = -(-k // 128)
        assert scales == 4 * ((blocks + 3) // 4 * 4 * rows if per == ROW else blocks * groups * -(-(rows // groups) // 128))


QUANT = [
    (dict(src=None), INV), (dict(src=A + 8), INV), (dict(codes=None), INV), (dict(codes=A + 8), INV),
    (dict(scales=None), INV), (dict(scales=A + 8), INV), (dict(lds=0), INV), (dict(lds=6), UNS), (dict(ld=120), INV), (dict(ld=132), UNS),
    (dict(type=3), INV), (dict(K=120), UNS), (dict(rows=-1), INV),
]


@pytest.mark.parametrize("over,want", QUANT)
def test_fp8_rows_refuse(over, want):
    a = dict(rows=20, K=128, type=0, src=A, ld=128, codes=A, scales=A, lds=4)
    a.update(over)
    s = binding.fp8_shape(ROW, 1, a["rows"], a["K"])
    assert binding.moe_fp8_quantize(s, a["type"], a["src"], a["ld"], a["codes"], a["scales"], a["lds"], None) == want
    assert binding.moe_fp8_dequantize(s, a["codes"], a["scales"], a["lds"], a["type"], a["src"], a["ld"], None) == want


def call(fn, **over):
    a = dict(groups=4, N=64, K=128, rows=20, type=0, a=A, s=A, lds=4, w=A, ws_=A, off=A, cnt=None, out=A, ldo=64, ws=A,
             ws_bytes=BIG)
    a.update(over)
    s = binding.grouped_shape(a["groups"], a["N"], a["K"], a["rows"], a["type"])
    return fn(s, a["a"], a["s"], a["lds"], a["w"], a["ws_"], a["off"], a["cnt"], a["out"], a["ldo"], a["ws"],
              a["ws_bytes"], None)


@pytest.mark.parametrize("over,want", [
    (dict(a=None), INV), (dict(a=A + 8), INV), (dict(s=None), INV), (dict(s=A + 4), INV), (dict(lds=0), INV), (dict(lds=5), UNS),
    (dict(w=None), INV), (dict(w=A + 8), INV), (dict(ws_=None), INV), (dict(ws_=A + 8), INV), (dict(out=None), INV),
    (dict(out=A + 8), INV), (dict(off=A + 2), INV), (dict(cnt=A + 1), INV), (dict(rows=21, off=None), INV),
    (dict(ws=None), INV), (dict(ws=A + 64), INV), (dict(ws_bytes=1024), WS), (dict(type=2), INV), (dict(groups=0), INV),
    (dict(N=56), UNS), (dict(K=72), UNS), (dict(rows=0, a=None, s=None, out=None), OK),
])
def test_fp8_products_refuse(over, want):
    assert call(binding.moe_fp8_gemm, **{"ldo": 1024, **over}) == want
    assert call(binding.moe_fp8_gemm_dgrad, **{"ldo": 1024, **over}) == want


def test_fp8_products_want_their_own_widths():
    assert call(binding.moe_fp8_gemm, ldo=56) == INV and call(binding.moe_fp8_gemm, ldo=68) == UNS
    assert call(binding.moe_fp8_gemm_dgrad, ldo=120) == INV and call(binding.moe_fp8_gemm_dgrad, ldo=132) == UNS


@pytest.mark.parametrize("kind,type_,wtype,h,rows,eps,want", [
    (0, 0, 0, 8, 0, 0.0, OK), (1, 2, 2, 16384, (1 << 31) - 512, 1e-5, OK), (1, 1, 2, 64, 3, 1.0, OK),
    (2, 0, 0, 8, 1, 0.0, INV), (0, 3, 3, 8, 1, 0.0, INV), (0, 0, 1, 8, 1, 0.0, INV), (0, 2, 0, 8, 1, 0.0, INV),
    (0, 0, 0, 0, 1, 0.0, INV), (0, 0, 0, 8, -1, 0.0, INV), (0, 0, 0, 8, 1, -1e-6, INV), (0, 0, 0, 8, 1, NAN, INV),
    (0, 0, 0, 8, 1, INF, INV), (0, 0, 0, 12, 1, 0.0, UNS), (0, 0, 0, 16392, 1, 0.0, UNS), (0, 0, 0, 8, 1 << 31, 0.0, UNS),
])
def test_norm_shapes(kind, type_, wtype, h, rows, eps, want):
    st, n = binding.moe_norm_grad_workspace_size(binding.norm_shape(kind, type_, wtype, h, rows, eps))
    assert st == want and (n > 0) == (want == OK)


def norm(**over):
    a = dict(kind=1, rows=4, x=A, ldx=64, w=A, b=A, y=A + 4096, ldy=64, mean=A, rstd=A)
    a.update(over)
    s = binding.norm_shape(a["kind"], 0, 2, 64, a["rows"], 1e-6)
    return binding.moe_norm(s, a["x"], a["ldx"], a["w"], a["b"], a["y"], a["ldy"], a["mean"], a["rstd"], None)


@pytest.mark.parametrize("over,want", [
    (dict(x=None), INV), (dict(x=A + 8), INV), (dict(ldx=56), INV), (dict(ldx=68), UNS), (dict(y=None), INV),
    (dict(y=A + 4), INV), (dict(ldy=56), INV), (dict(ldy=70), UNS), (dict(w=A + 8), INV), (dict(b=A + 4), INV),
    (dict(mean=A + 2), INV), (dict(rstd=A + 1), INV), (dict(y=A, ldy=72), INV), (dict(kind=0), INV),
    (dict(kind=0, b=None), INV), (dict(rows=0, x=None, y=None), OK),
])
def test_norm_refuses(over, want):
    assert norm(**over) == want


def grad(**over):
    a = dict(kind=1, rows=4, dy=A, lddy=64, x=A, ldx=64, w=A, mean=A, rstd=A, dx=A + 4096, lddx=64, dw=A, db=A, type=2,
             acc=0, ws=A, ws_bytes=BIG)
    a.update(over)
    s = binding.norm_shape(a["kind"], 0, 0, 64, a["rows"], 1e-6)
    return binding.moe_norm_grad(s, a["dy"], a["lddy"], a["x"], a["ldx"], a["w"], a["mean"], a["rstd"], a["dx"],
                                 a["lddx"], a["dw"], a["db"], a["type"], a["acc"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("over,want", [
    (dict(dy=None), INV), (dict(dy=A + 8), INV), (dict(lddy=56), INV), (dict(lddy=68), UNS), (dict(x=None), INV),
    (dict(ldx=60), INV), (dict(dx=None), INV), (dict(dx=A + 2), INV), (dict(lddx=68), UNS), (dict(w=A + 8), INV),
    (dict(mean=None), INV), (dict(rstd=None), INV), (dict(dw=A + 8), INV), (dict(db=A + 4), INV), (dict(type=1), INV),
    (dict(type=0, acc=1), INV), (dict(ws=None), INV), (dict(ws=A + 128), INV), (dict(ws_bytes=64), WS),
    (dict(dx=A, lddx=72), INV), (dict(kind=0), INV), (dict(kind=0, db=None), INV),
    (dict(rows=0, dy=None, x=None, dx=None, mean=None, rstd=None, acc=1), OK),
    (dict(rows=0, dy=None, x=None, dx=None, mean=None, rstd=None, dw=None, db=None, ws=None, ws_bytes=0), OK),
])
def test_norm_gradient_refuses(over, want):
    assert grad(**over) == want


def tensors(**over):
    a = dict(data=A, out=A, n=5, type=2, out_type=2)
    a.update(over)
    return binding.grad_tensors([(A, A, 3, 0, 0), (a["data"], a["out"], a["n"], a["type"], a["out_type"])])


@pytest.mark.parametrize("over,want", [
    (dict(data=None), INV), (dict(data=A + 2), INV), (dict(n=-1), INV), (dict(type=3), INV), (dict(n=(1 << 40) + 1), UNS),
])
def test_gradient_norm_and_clipping_refuse_tensors(over, want):
    t = tensors(**over)
    assert binding.moe_grad_norm(t, 2, A, A, BIG, None) == want
    assert binding.moe_grad_clip(t, 2, A, 1.0, 0.0, None) == want
    assert binding.moe_grad_norm_clip(t, 2, 1.0, 0.0, A, A, BIG, None) == want


@pytest.mark.parametrize("over", [dict(out=None), dict(out=A + 2), dict(out_type=3), dict(out_type=0)])
def test_clipping_refuses_outputs(over):
    assert binding.moe_grad_clip(tensors(**over), 2, A, 1.0, 0.0, None) == INV
    assert binding.moe_grad_norm_clip(tensors(**over), 2, 1.0, 0.0, A, A, BIG, None) == INV


def test_gradient_norm_and_clipping_refuse_the_rest():
    t = tensors()
    assert binding.moe_grad_norm_workspace_size(-1)[0] == INV
    need = binding.moe_grad_norm_workspace_size(2)[1]
    assert binding.moe_grad_norm_workspace_size(3201)[1] == 3 * need
    assert binding.moe_grad_norm(t, -1, A, A, BIG, None) == INV
    assert binding.moe_grad_norm(None, 2, A, A, BIG, None) == INV
    assert binding.moe_grad_norm(t, 2, None, A, BIG, None) == INV
    assert binding.moe_grad_norm(t, 2, A + 2, A, BIG, None) == INV
    assert binding.moe_grad_norm(t, 2, A, None, BIG, None) == INV
    assert binding.moe_grad_norm(t, 2, A, A + 8, BIG, None) == INV
    assert binding.moe_grad_norm(t, 2, A, A, need - 1, None) == WS
    for norm_, max_norm, eps in ((None, 1.0, 0.0), (A + 2, 1.0, 0.0), (A, -1.0, 0.0), (A, NAN, 0.0), (A, 1.0, -1.0),
                                 (A, 1.0, INF), (A, 1.0, NAN)):
        assert binding.moe_grad_clip(t, 2, norm_, max_norm, eps, None) == INV
        assert binding.moe_grad_norm_clip(t, 2, max_norm, eps, norm_, A, BIG, None) == INV
    assert binding.moe_grad_norm_clip(t, 2, 1.0, 0.0, A, None, BIG, None) == INV
    assert binding.moe_grad_norm_clip(t, 2, 1.0, 0.0, A, A + 8, BIG, None) == INV
    assert binding.moe_grad_norm_clip(t, 2, 1.0, 0.0, A, A, need - 1, None) == WS
    assert binding.moe_grad_clip(None, 0, A, 1.0, 0.0, None) == OK
    assert binding.moe_grad_clip(tensors(n=0, data=None, out=None), 0, A, 1.0, 0.0, None) == OK


def test_objects_refuse_tensors_on_the_cpu():
    torch = pytest.importorskip("torch")
    x = torch.ones((4, 64))
    norm_ = binding.RowNorm(64, "rms", torch.float32, device="cpu")
    with pytest.raises(ValueError):
        norm_.forward(x)
    with pytest.raises(ValueError):
        binding.Fp8Rows(64, device="cpu").quantize(x)
    with pytest.raises(ValueError):
        binding.Fp8Weights.quantize(x.view(1, 4, 64))
    with pytest.raises(ValueError):
        binding.Gradients([x]).norm()
