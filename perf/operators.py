"""The experts' products as separate operators: what is measured, on which inputs, and their plain forms.

Rows of x (and of y, dy) belong to groups (experts): group g holds the rows offsets[g] .. offsets[g] + counts[g], any
number of them, none included; w is [groups, N, K].

  forward    y[p, :]  = x[p, :] w_g^T
  dgrad      dx[p, :] = dy[p, :] w_g
  wgrad      dw_g     = sum over the group's rows of dy[p, :]^T x[p, :]         (zeros for an empty group)
  swiglu     a = silu(gate) * up for rows [gate | up]; its gradient: d[gate | up] from da
  fp4        4-bit round trip: rows to E2M1 codes with block scales, and back to the values the codes stand for
  fp4_gemm   rows quantised to 4 bits, times weights kept in 4 bits, grouped like `forward`

MXFP4: blocks of 32 along K share 2^E, E = floor(log2(largest magnitude)) - 2 (-127 for a block of zeros).  NVFP4:
blocks of 16 share an E4M3 scale s = E4M3(largest magnitude / (6 g)) under one fp32 scale g = largest magnitude of the
row (of the matrix, for weights) / 2688 (1 for zeros); each of these steps, and x / (s g), is one fp32 operation.  Codes:
the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with ties to the even code.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases


def _products(op, name, rows, groups, active, n, k, type_="bf16", out="", skew=0.0, padded=False, fmt=""):
    c = {"op": op, "name": name, "rows": rows, "groups": groups, "active": active, "N": n, "K": k, "type": type_,
         "out": out or type_, "skew": skew, "padded": padded, "fmt": fmt}
    if not name:
        del c["name"]
    return c


def listed():
    return [
        # one token through its 8 experts' gate/up weights of the decode layer: 8 weight matrices streamed once
        _products("forward", "forward_one_token", 8, 64, 8, 8192, 4096),
        # a prompt of 4096 tokens, top 8 of 64, gate/up
        _products("forward", "forward_prompt", 32768, 64, 64, 8192, 4096),
        # a training step of 1024 tokens over 256 small experts: 32 rows an expert, every expert's weight read
        _products("dgrad", "dgrad_fine_grained", 8192, 256, 256, 4096, 7168),
        # uneven experts, some of them without a row, odd row counts, fp16, lists padded to 16 rows as the router makes them
        _products("dgrad", "dgrad_uneven_fp16", 4091, 128, 101, 2816, 4096, "fp16", skew=0.5, padded=True),
        # the weight gradient of the prompt's down product, kept in fp32 for the optimizer
        _products("wgrad", "wgrad_prompt", 32768, 64, 64, 4096, 4096, out="fp32"),
        # the smallest layer of the tests: what a call costs when there is next to nothing to compute
        _products("wgrad", "wgrad_tiny", 21, 8, 6, 512, 128),
        # the prompt's activation, and the gradient at the uneven layer's width (odd rows, fp16)
        {"op": "swiglu", "name": "swiglu_prompt", "rows": 32768, "I": 4096, "type": "bf16"},
        {"op": "swiglu_grad", "name": "swiglu_grad_uneven_fp16", "rows": 6141, "I": 1408, "type": "fp16"},
        # a weight matrix of every expert of the decode layer to MXFP4 and back to bf16 (training on rounded weights)
        _products("fp4", "fp4_mx_weights", 64 * 4096, 64, 64, 0, 4096, fmt="mx"),
        # token rows of the fine-grained layer to NVFP4 and back to fp32
        _products("fp4", "fp4_nv_tokens", 1021, 256, 241, 0, 7168, out="fp32", fmt="nv", skew=0.5),
        # the prompt's down product with weights and tokens in NVFP4
        _products("fp4_gemm", "fp4_gemm_nv_prompt", 32768, 64, 64, 4096, 4096, fmt="nv"),
        # eight decoded tokens through MXFP4 gate/up weights
        _products("fp4_gemm", "fp4_gemm_mx_step", 64, 64, 41, 8192, 4096, fmt="mx"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "dgrad", "wgrad", "swiglu", "swiglu_grad", "fp4", "fp4_gemm"])
    type_ = rng.choice(["bf16", "fp16"])
    if op in ("swiglu", "swiglu_grad"):
        i = 8 * _log(rng, 16, 1024)
        return {"op": op, "rows": max(1, min(_log(rng, 1, 40000), 32768 * 4096 // i)), "I": i, "type": type_}
    while True:
        groups = _log(rng, 1, 256)
        rows = _log(rng, 1, 32768)
        step = 32 if op in ("fp4", "fp4_gemm") else 8
        n, k = 8 * _log(rng, 16, 1024), step * _log(rng, 128 // step, 8192 // step)
        skew = rng.choice([0.0, 0.0, 0.5])
        active = max(1, min(groups, rows, int(round(groups * rng.uniform(0.5, 1.0)))))
        if rows > 768 * active or groups * n * k > 64 * 4096 * 8192:
            continue
        if rows * n * k * (4 if skew else 1) > 32768 * 4096 * 8192:
            continue
        fmt = rng.choice(["mx", "nv"]) if step == 32 else ""
        out = rng.choice([type_, "fp32"]) if op in ("wgrad", "fp4") else type_
        return _products(op, "", rows, groups, active, 0 if op == "fp4" else n, k, type_, out, skew,
                         rng.random() < 0.5, fmt)


def work(case):
    op, r, size = case["op"], case["rows"], {"bf16": 2, "fp16": 2, "fp32": 4}
    if op == "swiglu":
        return {"bytes": r * 3 * case["I"] * 2, "flops": r * case["I"] * 5}
    if op == "swiglu_grad":
        return {"bytes": r * 5 * case["I"] * 2, "flops": r * case["I"] * 12}
    n, k, active = case["N"], case["K"], case["active"]
    if op == "fp4":
        return {"bytes": r * k * (2 + size[case["out"]]), "flops": r * k * 4}
    flops = 2 * r * n * k
    if op == "wgrad":
        return {"bytes": r * (n + k) * 2 + case["groups"] * n * k * size[case["out"]], "flops": flops}
    if op == "fp4_gemm":
        w = active * n * k // 2 + active * n * k // (32 if case["fmt"] == "mx" else 16)
        return {"bytes": w + r * (k + n) * 2, "flops": flops}
    return {"bytes": active * n * k * 2 + r * (n + k) * 2, "flops": flops}


# ------------------------------------------------------------------ inputs


def _groups(case, seed):
    """Offsets and counts (host lists) of the case's groups, and the buffers' rows."""
    rng = np.random.default_rng([seed, 7])
    g, a, rows = case["groups"], case["active"], case["rows"]
    counts = np.zeros(g, np.int64)
    if case["op"] == "fp4" and a == g and rows % g == 0 and not case["skew"]:
        counts[:] = rows // g  # matrices of equal height
    else:
        p = (1.0 + np.arange(a)) ** -case["skew"]
        counts[rng.permutation(g)[:a]] = 1 + rng.multinomial(rows - a, p / p.sum())
    held = (counts + 15) // 16 * 16 if case["padded"] else counts
    offsets = np.concatenate([[0], np.cumsum(held)])
    return offsets, counts, rows + 15 * g if case["padded"] else rows


def _normal(gen, shape, std, type_):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(TYPES[type_])


def _tile_scales(s):
    """Scale bytes [matrices, rows, blocks] in the layout of the 4-bit tensor cores: 512-byte tiles of 128 rows x 4
    blocks, byte r * 16 + 4 * j + b for row 32 j + r and block b of the tile."""
    m, r, b = s.shape
    t, c = -(-r // 128), -(-b // 4)
    full = torch.zeros((m, t * 128, c * 4), dtype=torch.uint8, device=s.device)
    full[:, :r, :b] = s
    return full.view(m, t, 4, 32, c, 4).permute(0, 1, 4, 3, 2, 5).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    if case["op"] in ("swiglu", "swiglu_grad"):
        st["h"] = _normal(gen, (case["rows"], 2 * case["I"]), 1.5, case["type"])
        if case["op"] == "swiglu_grad":
            st["da"] = _normal(gen, (case["rows"], case["I"]), 0.1, case["type"])
        if own:
            from mixture_experts_layer_rmsnorm_gb300 import binding
            st["binding"] = binding
        return st
    offsets, counts, held = _groups(case, seed)
    n, k, g, op, type_ = case["N"], case["K"], case["groups"], case["op"], case["type"]
    st["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    st["counts"] = torch.tensor(counts, dtype=torch.int32, device="cuda") if case["padded"] else None
    # for the plain forms: a [groups, longest list] table of rows, `held` where a list is shorter
    most = int(counts.max())
    idx = np.minimum(offsets[:-1, None] + np.arange(most)[None], held)
    idx[np.arange(most)[None] >= counts[:, None]] = held
    st["table"] = torch.tensor(idx, device="cuda")
    st["rows"] = torch.tensor(np.concatenate([np.arange(o, o + c) for o, c in zip(offsets, counts)]), device="cuda")
    if op in ("forward", "wgrad", "fp4", "fp4_gemm"):
        st["x"] = _normal(gen, (held, k), 1.0, type_)
    if op in ("dgrad", "wgrad"):
        st["dy"] = _normal(gen, (held, n), 0.1, type_)
    if op in ("forward", "dgrad", "fp4_gemm"):
        w = _normal(gen, (g, n, k), 0.02, type_)
        if op == "fp4_gemm":  # kept in 4 bits: packed codes, scales as rows and as tiles, scale of each matrix
            codes, scales, gscale = _quantise(w.view(g * n, k), case["fmt"], g)
            st["w_codes"] = (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous()
            st["w_scales"] = scales
            st["w_gscale"] = gscale
            st["w_tiles"] = _tile_scales(scales.view(g, n, -1))
        else:
            st["w"] = w
    # the caller's output buffers: rows between the lists stay as they are
    if op in ("forward", "fp4_gemm"):
        st["y"] = torch.zeros((held, n), dtype=TYPES[type_], device="cuda")
    if op == "dgrad":
        st["dx"] = torch.zeros((held, k), dtype=TYPES[type_], device="cuda")
    if op == "fp4":
        st["y"] = torch.zeros((held, k), dtype=TYPES[case["out"]], device="cuda")
    if op == "wgrad":
        st["dw"] = torch.empty((g, n, k), dtype=TYPES[case["out"]], device="cuda")
    if own:
        from mixture_experts_layer_rmsnorm_gb300 import binding
        if op in ("forward", "dgrad", "wgrad"):
            st["products"] = binding.GroupedProducts(g, n, k, TYPES[type_], max_rows=held)
        elif op == "fp4":
            st["rows4"] = binding.Fp4Rows(case["fmt"], k, g, max_rows=held)
        else:
            st["rows4"] = binding.Fp4Rows(case["fmt"], k, g, max_rows=held)
            st["weights4"] = binding.Fp4Weights(case["fmt"], st["w_codes"].view(g, n, k // 2), st["w_tiles"],
                                                st["w_gscale"])
    return st


# ------------------------------------------------------------------ plain forms


def _quantise(x, fmt, matrices=0):
    """Codes [rows, K] (one a byte, the sign in bit 3), scale bytes [rows, blocks] and, for NVFP4, the fp32 scales (one a
    row, or one for each of `matrices` equal parts)."""
    x = x.float()
    rows, k = x.shape
    block = 32 if fmt == "mx" else 16
    b = x.view(rows, k // block, block)
    amax = b.abs().amax(2)
    if fmt == "mx":
        e = torch.where(amax > 0, (torch.frexp(amax)[1] - 3).clamp(-127, 127), -127)
        scales, g = (e + 127).to(torch.uint8), None
        q = torch.ldexp(b, -e[..., None])
    else:
        top = amax.view(matrices, -1).amax(1) if matrices else amax.amax(1)
        g = torch.where(top > 0, top / torch.full_like(top, 2688.0), torch.ones_like(top))  # (a true division)
        gr = g.repeat_interleave(rows // matrices)[:, None] if matrices else g[:, None]
        s8 = (amax / (6.0 * gr)).clamp(max=448.0).to(torch.float8_e4m3fn)
        scales = s8.view(torch.uint8)
        d = (s8.float() * gr)[..., None]
        q = torch.where(d > 0, b / d, torch.zeros_like(b))
    m = q.abs()
    codes = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    codes = codes | (torch.signbit(b).to(torch.uint8) << 3)
    return codes.view(rows, k), scales, g


def _values(codes, scales, gscale, fmt):
    """The fp32 values of codes [rows, K]; gscale: fp32, broadcast over the rows, or None."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    rows, k = codes.shape
    block = 32 if fmt == "mx" else 16
    v = table[codes.int()].view(rows, k // block, block)
    if fmt == "mx":
        return torch.ldexp(v, (scales.int() - 127)[..., None]).view(rows, k)
    return (v * scales.view(torch.float8_e4m3fn).float()[..., None]).view(rows, k) * gscale[:, None]


def _lists(t, table):
    """[groups, longest list, width] in fp32, zeros behind each list's end."""
    return torch.cat([t.float(), t.new_zeros((1, t.shape[1])).float()])[table]


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
        if op == "swiglu":
            return st["binding"].swiglu(st["h"])
        if op == "swiglu_grad":
            return st["binding"].swiglu_grad(st["h"], st["da"])
        if op == "forward":
            return st["products"].forward(st["x"], st["w"], st["offsets"], st["counts"], y=st["y"])
        if op == "dgrad":
            return st["products"].dgrad(st["dy"], st["w"], st["offsets"], st["counts"], dx=st["dx"])
        if op == "wgrad":
            return st["products"].wgrad(st["dy"], st["x"], st["offsets"], st["counts"], dw=st["dw"])
        st["rows4"].quantize(st["x"], st["offsets"], st["counts"])
        if op == "fp4":
            return st["rows4"].dequantize(st["offsets"], st["counts"], y=st["y"])
        return st["weights4"].forward(st["rows4"], st["offsets"], st["counts"], y=st["y"])

    if op in ("swiglu", "swiglu_grad"):
        gate, up = st["h"].float().chunk(2, dim=1)
        s = 1.0 / (1.0 + torch.exp(-gate))
        if op == "swiglu":
            return (gate * s * up).to(st["h"].dtype)
        da = st["da"].float()
        dh = torch.cat([da * up * s * (1.0 + gate * (1.0 - s)), da * gate * s], dim=1)
        return dh.to(st["h"].dtype)
    if op == "forward":
        y = torch.bmm(_lists(st["x"], st["table"]), st["w"].float().transpose(1, 2))
        return _back(y, st["table"], st["rows"], st["y"])
    if op == "dgrad":
        dx = torch.bmm(_lists(st["dy"], st["table"]), st["w"].float())
        return _back(dx, st["table"], st["rows"], st["dx"])
    if op == "wgrad":
        dw = torch.bmm(_lists(st["dy"], st["table"]).transpose(1, 2), _lists(st["x"], st["table"]))
        st["dw"].copy_(dw)
        return st["dw"]
    xq = _values(*_quantise(st["x"], case["fmt"]), case["fmt"])
    if op == "fp4":
        st["y"][st["rows"]] = xq[st["rows"]].to(st["y"].dtype)
        return st["y"]
    g, n, k = case["groups"], case["N"], case["K"]
    packed = st["w_codes"]
    codes = torch.stack([packed & 15, packed >> 4], dim=2).view(g * n, k)
    gw = None if st["w_gscale"] is None else st["w_gscale"].repeat_interleave(n)
    w = _values(codes, st["w_scales"], gw, case["fmt"]).view(g, n, k)
    y = torch.bmm(_lists(xq, st["table"]), w.transpose(1, 2))
    return _back(y, st["table"], st["rows"], st["y"])


# ------------------------------------------------------------------ from the definitions, in 64 bits


def _f32(t):
    return t.float().double()


def _exact_fp4(x, fmt, matrices):
    """What x is rounded to, in 64 bits; the fp32 steps of the NVFP4 definition are rounded where it rounds."""
    x = x.double()
    block = 32 if fmt == "mx" else 16
    b = x.reshape(x.shape[0], -1, block)
    top = b.abs().amax(2, keepdim=True)
    if fmt == "mx":
        log = torch.floor(torch.log2(top.clamp(min=1e-300)))
        log = torch.where(torch.exp2(log) > top, log - 1, log)
        log = torch.where(torch.exp2(log + 1) <= top, log + 1, log)
        unit = torch.exp2(torch.where(top > 0, (log - 2).clamp(-127, 127), torch.full_like(log, -127)))
        q = b / unit
    else:
        whole = top.reshape(matrices or x.shape[0], -1).amax(1)
        g = torch.where(whole > 0, _f32(whole / 2688), torch.ones_like(whole))
        g = g.repeat_interleave(x.shape[0] // g.numel()).reshape(-1, 1, 1)
        s = _f32(top / _f32(6 * g)).clamp(max=448)
        step = torch.exp2(torch.floor(torch.log2(s.clamp(min=2.0 ** -6))) - 3)
        s = torch.round(s / step) * step
        d = _f32(s * g)
        q = torch.where(d > 0, _f32(b / torch.where(d > 0, d, torch.ones_like(d))), torch.zeros_like(b))
        unit = s * g
    m = q.abs()
    step = torch.exp2(torch.floor(torch.log2(m.clamp(1.0, 6.0))) - 1)
    m = torch.minimum(torch.round(m / step) * step, torch.full_like(m, 6.0))
    return (torch.copysign(m, b) * unit).reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("swiglu", "swiglu_grad"):
        h = st["h"].double()
        i = case["I"]
        gate, up = h[:, :i], h[:, i:]
        s = torch.special.expit(gate)
        if op == "swiglu":
            return gate * s * up
        da = st["da"].double()
        return torch.hstack([da * up * (s + gate * s * (1 - s)), da * gate * s])
    offsets, counts, held = _groups(case, seed)
    g, n, k = case["groups"], case["N"], case["K"]
    if op == "fp4":
        y = torch.zeros((held, k), dtype=torch.float64, device="cuda")
        for i in range(g):
            if counts[i]:
                r = slice(int(offsets[i]), int(offsets[i] + counts[i]))
                y[r] = _exact_fp4(st["x"][r], case["fmt"], 0)
        return y
    if op == "fp4_gemm":
        gen = torch.Generator(device="cuda").manual_seed(seed)
        x = _normal(gen, (held, k), 1.0, case["type"])
        w = _normal(gen, (g, n, k), 0.02, case["type"])
    if op == "wgrad":
        out = torch.zeros((g, n, k), dtype=torch.float64, device="cuda")
    else:
        out = torch.zeros((held, k if op == "dgrad" else n), dtype=torch.float64, device="cuda")
    for i in range(g):
        if not counts[i]:
            continue
        r = slice(int(offsets[i]), int(offsets[i] + counts[i]))
        if op == "forward":
            out[r] = st["x"][r].double() @ st["w"][i].double().T
        elif op == "dgrad":
            out[r] = st["dy"][r].double() @ st["w"][i].double()
        elif op == "wgrad":
            out[i] = st["dy"][r].double().T @ st["x"][r].double()
        else:
            out[r] = _exact_fp4(x[r], case["fmt"], 0) @ _exact_fp4(w[i], case["fmt"], 1).T
    return out
