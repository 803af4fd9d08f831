"""A training step of the experts in 8 bits: what is measured, on which inputs, and the operators' plain forms.

  fp8          weights to 8 bits and back to the values that the codes stand for
  fp8_forward  rows to 8 bits, times weights kept in 8 bits: y[p, :] = x[p, :] w_g^T for the rows p of group (expert) g
  fp8_dgrad    the same for the input gradient: dx[p, :] = dy[p, :] w_g, with the same weights
  norm         y = (x - m) r weight + bias for every row, with m its mean and r = 1 / sqrt(mean((x - m)^2) + eps)
               ("layer"), or m = 0 and no bias ("rms"); m and r are kept for the gradient
  norm_grad    dx, dweight, dbias from dy
  clip         the norm of all elements of many tensors, and the tensors times min(1, max_norm / (norm + eps))

8 bits: 128 elements of a row (weights: a block of 128 x 128) share an fp32 scale s = largest magnitude / 448 (1 where that
is zero); an element is the E4M3 value nearest to x / s, ties to the even code; each division is one fp32 operation.
Groups: group g holds the rows offsets[g] .. offsets[g] + counts[g], any number of them; w is [groups, N, K].
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
BLOCK = 128
CLIP_EPS = 1e-6


# ------------------------------------------------------------------ cases


def _product(op, rows, groups, active, n, k, type_="bf16", skew=0.0, padded=False):
    return {"op": op, "rows": rows, "groups": groups, "active": active, "N": n, "K": k, "type": type_, "skew": skew,
            "padded": padded}


def _norm(op, kind, rows, h, type_="bf16", weight="bf16", eps=1e-6):
    return {"op": op, "kind": kind, "rows": rows, "H": h, "type": type_, "weight": weight, "eps": eps}


def _clip(tensors, elements, types, out, clipped):
    return {"op": "clip", "tensors": tensors, "elements": elements, "types": types, "out": out, "clipped": clipped}


def listed():
    cases = {
        # one token through its 8 experts' gate/up weights of the decode layer: 8 weight matrices streamed once
        "fp8_forward_one_token": _product("fp8_forward", 8, 64, 8, 8192, 4096),
        # the down product of a prompt of 4096 tokens, top 8 of 64
        "fp8_forward_prompt": _product("fp8_forward", 32768, 64, 64, 4096, 4096),
        # a training step of 1024 tokens over 256 small experts: 32 rows an expert, every expert's weight read
        "fp8_dgrad_fine_grained": _product("fp8_dgrad", 8192, 256, 256, 4096, 7168),
        # uneven experts, some without a row, odd row counts, fp16, lists padded to 16 rows as the router makes them
        "fp8_dgrad_uneven_fp16": _product("fp8_dgrad", 4091, 128, 101, 2816, 4096, "fp16", 0.5, True),
        # the down weights of the decode layer's experts to 8 bits and back to bf16 (training on rounded weights)
        "fp8_weights": {"op": "fp8", "groups": 64, "N": 4096, "K": 4096, "type": "bf16", "out": "bf16"},
        # the norm before the experts: a prompt of 4096 tokens of the fine-grained layer
        "norm_rms_prompt": _norm("norm", "rms", 4096, 7168),
        # the smallest layer of the tests, with a layer norm in fp32: what a call costs when there is little to do
        "norm_layer_tiny_fp32": _norm("norm", "layer", 4, 128, "fp32", "fp32", 1e-5),
        # its gradient in a training step of 16384 tokens, gains kept in fp32
        "norm_grad_rms_step": _norm("norm_grad", "rms", 16384, 4096, "bf16", "fp32"),
        # the norm of every head of Q and K: 4096 tokens, 40 heads of 128
        "norm_grad_rms_heads": _norm("norm_grad", "rms", 163840, 128),
        # an odd number of rows at the uneven layer's width, layer norm in fp16
        "norm_grad_layer_uneven_fp16": _norm("norm_grad", "layer", 6141, 1408, "fp16", "fp16", 1e-5),
        # the down weights' gradients of 64 experts, summed in fp32, clipped into bf16 for the optimizer
        "clip_experts": _clip(2, 64 * 4096 * 4096, "fp32", "bf16", True),
        # everything else of a model: gains, biases, routers, 1200 tensors of any size and type; below the limit
        "clip_many_small": _clip(1200, 30000000, "mixed", "", False),
    }
    return [dict(c, name=name) for name, c in cases.items()]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fp8", "fp8_forward", "fp8_dgrad", "fp8_forward", "fp8_dgrad", "norm", "norm_grad", "norm_grad",
                     "clip"])
    if op == "clip":
        tensors = _log(rng, 1, 1500)
        return _clip(tensors, max(tensors, _log(rng, 1000, 64 * 4096 * 4096)),
                     rng.choice(["bf16", "fp16", "fp32", "mixed"]), rng.choice(["", "bf16", "fp32"]),
                     rng.random() < 0.6)
    type_ = rng.choice(["bf16", "fp16"])
    if op in ("norm", "norm_grad"):
        h = 8 * _log(rng, 2, 2048)
        type_ = rng.choice([type_, type_, "fp32"])
        rows = _log(rng, 1, 200000)
        return _norm(op, rng.choice(["rms", "layer"]), max(1, min(rows, 16384 * 4096 // h)), h, type_,
                     rng.choice([type_, "fp32"]), rng.choice([1e-5, 1e-6]))
    while True:
        groups = _log(rng, 1, 256)
        n, k = 16 * _log(rng, 8, 512), 16 * _log(rng, 8, 512)
        if groups * n * k > 64 * 4096 * 4096:
            continue
        if op == "fp8":
            return {"op": op, "groups": groups, "N": n, "K": k, "type": rng.choice([type_, "fp32"]),
                    "out": rng.choice(["bf16", "fp16"])}
        rows = _log(rng, 1, 32768)
        skew = rng.choice([0.0, 0.0, 0.5])
        active = max(1, min(groups, rows, int(round(groups * rng.uniform(0.5, 1.0)))))
        if rows > 768 * active or rows * n * k * (4 if skew else 1) > 32768 * 4096 * 4096:
            continue
        return _product(op, rows, groups, active, n, k, type_, skew, rng.random() < 0.5)


def work(case):
    op = case["op"]
    if op == "clip":
        size = {"bf16": 2, "fp16": 2, "fp32": 4, "mixed": 8 / 3}
        n, read = case["elements"], size[case["types"]]
        written = case["clipped"] or case["out"]
        return {"bytes": int(n * (read + (size[case["out"] or case["types"]] if written else 0))), "flops": 3 * n}
    if op in ("norm", "norm_grad"):
        n, size = case["rows"] * case["H"], BYTES[case["type"]]
        return {"bytes": n * size * (2 if op == "norm" else 3) + 2 * case["H"] * BYTES[case["weight"]],
                "flops": n * (6 if op == "norm" else 14)}
    n, k = case["N"], case["K"]
    if op == "fp8":
        return {"bytes": case["groups"] * n * k * (BYTES[case["type"]] + BYTES[case["out"]]),
                "flops": 4 * case["groups"] * n * k}
    return {"bytes": case["active"] * n * k + case["rows"] * (n + k) * 2, "flops": 2 * case["rows"] * n * k}


# ------------------------------------------------------------------ inputs


def _groups(case, seed):
    """Offsets and counts (host lists) of the case's groups, and the buffers' rows."""
    rng = np.random.default_rng([seed, 7])
    g, a, rows = case["groups"], case["active"], case["rows"]
    counts = np.zeros(g, np.int64)
    p = (1.0 + np.arange(a)) ** -case["skew"]
    counts[rng.permutation(g)[:a]] = 1 + rng.multinomial(rows - a, p / p.sum())
    held = (counts + 15) // 16 * 16 if case["padded"] else counts
    offsets = np.concatenate([[0], np.cumsum(held)])
    return offsets, counts, rows + 15 * g if case["padded"] else rows


def _normal(gen, shape, std, type_):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(TYPES[type_])


def _sizes(case):
    """Elements of each tensor: spread over their logarithm, `elements` in all; and their types."""
    t, total = case["tensors"], case["elements"]
    rng = np.random.default_rng([t, total])
    if t <= 4:
        sizes = np.full(t, total // t)
    else:
        sizes = np.exp(rng.uniform(0, math.log(1000), t))
        sizes = np.maximum(1, (sizes / sizes.sum() * total).astype(np.int64))
        sizes[: t // 8] = np.minimum(sizes[: t // 8], 1 + np.arange(t // 8) % 37)  # (biases and single numbers)
    sizes[-1] += max(0, total - int(sizes.sum()))
    names = ["bf16", "fp16", "fp32"] if case["types"] == "mixed" else [case["types"]]
    return [int(s) for s in sizes], [names[i] for i in rng.integers(0, len(names), t)]


def _buffers(sizes, types, out):
    """A zeroed buffer for each type of `types`, of the type `out` says, and the tensors in them."""
    at, used = [], {}
    for n, t in zip(sizes, types):
        at.append(used.get(t, 0))
        used[t] = at[-1] + (n + 7) // 8 * 8
    into = dict(zip(types, out))
    buffers = {t: torch.zeros(used[t], dtype=TYPES[into[t]], device="cuda") for t in sorted(used)}
    return list(buffers.values()), [buffers[t][a:a + n] for n, t, a in zip(sizes, types, at)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st, op = {"case": case}, case["op"]
    if own:
        from mixture_experts_layer_rmsnorm_gb300 import binding
    if op == "clip":
        sizes, types = _sizes(case)
        # the gradients lie one behind the other in a buffer for each type, on 16-byte borders
        scales = 1e-3 * torch.exp(torch.randn(len(sizes), generator=gen, device="cuda"))
        st["buffers"], st["grads"] = _buffers(sizes, types, types)
        for i, g in enumerate(st["grads"]):
            g.copy_(torch.randn(g.shape, generator=gen, device="cuda").mul_(scales[i]))
        norm = math.sqrt(math.fsum(float(torch.dot(g.float(), g.float())) for g in st["grads"][-64:]))
        st["max_norm"] = norm * (0.3 if case["clipped"] else 100.0 * len(sizes))
        # where the clipped gradients go: their own place, or (a pass leaves them for the next one) other buffers
        if case["out"] or case["clipped"]:
            st["out_buffers"], st["out"] = _buffers(sizes, types, [case["out"] or t for t in types])
        else:
            st["out_buffers"], st["out"] = st["buffers"], st["grads"]
        if own:
            st["gradients"] = binding.Gradients(st["grads"], None if st["out"] is st["grads"] else st["out"])
        return st
    if op in ("norm", "norm_grad"):
        rows, h, type_, weight = case["rows"], case["H"], case["type"], case["weight"]
        st["x"] = _normal(gen, (rows, h), 1.5, type_)
        if case["kind"] == "layer":
            st["x"] += 0.5
        st["weight"] = (1 + 0.1 * torch.randn(h, generator=gen, device="cuda")).to(TYPES[weight])
        st["bias"] = _normal(gen, (h,), 0.1, weight) if case["kind"] == "layer" else None
        if op == "norm_grad":
            st["dy"] = _normal(gen, (rows, h), 0.1, type_)
            x = st["x"].float()  # what the forward pass kept
            m = x.mean(1) if case["kind"] == "layer" else torch.zeros(rows, device="cuda")
            st["mean"] = m if case["kind"] == "layer" else None
            st["rstd"] = torch.rsqrt((x - m[:, None]).square().mean(1) + case["eps"])
        if own:
            st["norm"] = binding.RowNorm(h, case["kind"], TYPES[type_], TYPES[weight], case["eps"])
        return st
    g, n, k, type_ = case["groups"], case["N"], case["K"], case["type"]
    w = _normal(gen, (g, n, k), 0.02, type_)
    if op == "fp8":
        st["w"] = w
        if own:
            st["binding"] = binding
        return st
    offsets, counts, held = _groups(case, seed)
    st["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    st["counts"] = torch.tensor(counts, dtype=torch.int32, device="cuda") if case["padded"] else None
    # for the plain forms: a [groups, longest list] table of rows, `held` where a list is shorter
    most = int(counts.max())
    idx = np.minimum(offsets[:-1, None] + np.arange(most)[None], held)
    idx[np.arange(most)[None] >= counts[:, None]] = held
    st["table"] = torch.tensor(idx, device="cuda")
    st["rows"] = torch.tensor(np.concatenate([np.arange(o, o + c) for o, c in zip(offsets, counts)]), device="cuda")
    # weights kept in 8 bits: codes [groups, N, K], scales [groups, N / 128, K / 128]
    st["w_codes"], st["w_scales"] = _quantise(w, True)
    del w
    into, from_ = (k, n) if op == "fp8_dgrad" else (n, k)
    st["x"] = _normal(gen, (held, from_), 0.1 if op == "fp8_dgrad" else 1.0, type_)
    # the caller's output buffer: rows between the lists stay as they are
    st["y"] = torch.zeros((held, into), dtype=TYPES[type_], device="cuda")
    if own:
        st["rows8"] = binding.Fp8Rows(from_, max_rows=held)
        st["weights8"] = binding.Fp8Weights(st["w_codes"], st["w_scales"])
    return st


# ------------------------------------------------------------------ plain forms


def _blocks(m, square):
    """m [..., rows, K] cut into blocks of 128 elements of a row (or 128 x 128), zeros past its ends:
    [..., rows / 128, 128, K / 128, 128], or [..., rows, 1, K / 128, 128]."""
    rows, k = m.shape[-2:]
    height = BLOCK if square else 1
    m = torch.nn.functional.pad(m, (0, -k % BLOCK, 0, -rows % height))
    return m.view(*m.shape[:-2], m.shape[-2] // height, height, m.shape[-1] // BLOCK, BLOCK)


def _whole(b, rows, k):
    m = b.reshape(*b.shape[:-4], b.shape[-4] * b.shape[-3], b.shape[-2] * b.shape[-1])
    return m[..., :rows, :k]


def _quantise(m, square=False):
    """E4M3 codes of m [..., rows, K] (a byte each) and the scales [..., rows / 128 (or rows), K / 128]."""
    rows, k = m.shape[-2:]
    b = _blocks(m.float(), square)
    top = b.abs().amax((-3, -1))
    s = top / torch.full_like(top, 448.0)  # (a true division)
    s = torch.where(s > 0, s, torch.ones_like(s))
    codes = (b / s[..., :, None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return _whole(codes.view(torch.uint8), rows, k).contiguous(), s


def _values(codes, scales, square=False):
    """The fp32 values of codes [..., rows, K]."""
    rows, k = codes.shape[-2:]
    b = _blocks(codes, square).view(torch.float8_e4m3fn).float()
    return _whole(b * scales[..., :, None, :, None], rows, k)


def _lists(t, table):
    """[groups, longest list, width] in fp32, zeros behind each list's end."""
    return torch.cat([t, t.new_zeros((1, t.shape[1]))])[table]


def _back(lists, table, rows, into):
    """Rows of the lists to their places in `into`."""
    flat = torch.zeros((into.shape[0] + 1, into.shape[1]), dtype=torch.float32, device=into.device)
    flat[table] = lists
    into[rows] = flat[rows].to(into.dtype)
    return into


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        if op == "clip":
            norm = st["gradients"].clip(st["max_norm"], CLIP_EPS)
            return [norm] + st["out_buffers"]
        if op == "norm":
            return st["norm"].forward(st["x"], st["weight"], st["bias"], stats=True)
        if op == "norm_grad":
            return st["norm"].grad(st["dy"], st["x"], st["weight"], st["rstd"], st["mean"])
        if op == "fp8":
            return st["binding"].Fp8Weights.quantize(st["w"]).dequantize(TYPES[case["out"]])
        product = st["weights8"].forward if op == "fp8_forward" else st["weights8"].dgrad
        return product(st["rows8"].quantize(st["x"]), st["offsets"], st["counts"], st["y"])

    if op == "clip":
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        for g in st["grads"]:
            total += g.float().square().sum(dtype=torch.float64)
        norm = total.sqrt()
        factor = (st["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0).float()
        for g, o in zip(st["grads"], st["out"]):
            o.copy_(g.float() * factor)
        return [norm.float()] + st["out_buffers"]
    if op in ("norm", "norm_grad"):
        x, weight = st["x"].float(), st["weight"].float()
        if op == "norm":
            m = x.mean(1, keepdim=True) if case["kind"] == "layer" else torch.zeros_like(x[:, :1])
            d = x - m
            r = 1.0 / torch.sqrt(d.square().mean(1, keepdim=True) + case["eps"])
            y = d * r * weight
            if st["bias"] is not None:
                y = y + st["bias"].float()
            y = y.to(st["x"].dtype)
            return (y, r[:, 0], m[:, 0]) if case["kind"] == "layer" else (y, r[:, 0])
        dy, r = st["dy"].float(), st["rstd"][:, None]
        layer = case["kind"] == "layer"
        n = (x - st["mean"][:, None]) * r if layer else x * r
        dn = dy * weight
        dx = dn - n * (dn * n).mean(1, keepdim=True)
        if layer:
            dx = dx - dn.mean(1, keepdim=True)
        dx, dweight = (dx * r).to(st["x"].dtype), (dy * n).sum(0).to(st["weight"].dtype)
        return (dx, dweight, dy.sum(0).to(st["weight"].dtype)) if layer else (dx, dweight)
    if op == "fp8":
        return _values(*_quantise(st["w"], True), True).to(TYPES[case["out"]])
    x = _lists(_values(*_quantise(st["x"])), st["table"])
    w = _values(st["w_codes"], st["w_scales"], True)
    y = torch.bmm(x, w.transpose(1, 2) if op == "fp8_forward" else w)
    return _back(y, st["table"], st["rows"], st["y"])


# ------------------------------------------------------------------ from the definitions, in 64 bits


def _f32(t):
    return t.float().double()


def _exact_fp8(m, height):
    """What the matrix m is rounded to, in 64 bits; the divisions are rounded to fp32 as the definition says."""
    m = m.double()
    out = torch.empty_like(m)
    for c in range(0, m.shape[1], 128):
        part = m[:, c:c + 128]
        top = part.abs().amax(1)
        if height > 1:
            top = torch.cat([t.amax().expand(t.numel()) for t in top.split(height)])
        s = _f32(top / 448)
        s = torch.where(s > 0, s, torch.ones_like(s))[:, None]
        q = _f32(part / s)
        a = q.abs()
        step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
        out[:, c:c + 128] = torch.copysign((torch.round(a / step) * step).clamp(max=448.0), q) * s
    return out


def exact(case, seed):
    op = case["op"]
    if op in ("fp8_forward", "fp8_dgrad") and 2 * case["rows"] * case["N"] * case["K"] > 4e12:
        return None  # (long in 64 bits)
    st = prepare(case, seed)
    if op == "clip":
        squares = 0.0
        for g in st["grads"]:
            for part in g.split(2 ** 27):
                squares += float(part.double().pow(2).sum())
        norm = math.sqrt(squares)
        factor = min(1.0, st["max_norm"] / (norm + CLIP_EPS))
        # (between the tensors there are zeros)
        return [torch.tensor(norm, dtype=torch.float64, device="cuda")] + [b.double().mul_(factor) for b in st["buffers"]]
    if op in ("norm", "norm_grad"):
        x, weight = st["x"].double(), st["weight"].double()
        h, layer = case["H"], case["kind"] == "layer"
        if op == "norm":
            m = x.sum(1) / h if layer else torch.zeros(case["rows"], dtype=torch.float64, device="cuda")
            r = ((x - m[:, None]).pow(2).sum(1) / h + case["eps"]).pow(-0.5)
            y = torch.einsum("rh,r,h->rh", x - m[:, None], r, weight)
            if layer:
                return y + st["bias"].double(), r, m
            return y, r
        dy, r = st["dy"].double(), st["rstd"].double()
        n = (x - st["mean"].double()[:, None] if layer else x) * r[:, None]
        dn = dy * weight
        dx = r[:, None] * (dn - n * (torch.einsum("rh,rh->r", dn, n) / h)[:, None]
                           - ((dn.sum(1) / h)[:, None] if layer else 0.0))
        dweight = torch.einsum("rh,rh->h", dy, n)
        return (dx, dweight, dy.sum(0)) if layer else (dx, dweight)
    g, n, k = case["groups"], case["N"], case["K"]
    if op == "fp8":
        return torch.stack([_exact_fp8(st["w"][i], 128) for i in range(g)]) if g * n * k <= 2 ** 30 else None
    offsets, counts, held = _groups(case, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w = _normal(gen, (g, n, k), 0.02, case["type"])
    out = torch.zeros(st["y"].shape, dtype=torch.float64, device="cuda")
    for i in range(g):
        if counts[i]:
            r = slice(int(offsets[i]), int(offsets[i] + counts[i]))
            wi = _exact_fp8(w[i], 128)
            out[r] = _exact_fp8(st["x"][r], 1) @ (wi.T if op == "fp8_forward" else wi)
    return out
