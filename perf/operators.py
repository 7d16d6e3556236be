"""Workloads of the GEMMs with a fused epilogue and of the GEMMs grouped by expert.

Two operators, each on NVFP4 (e2m1 codes, e4m3 scales per 16) and MXFP8 (e4m3 elements, e8m0 scales per 32):

  dense    D = act(alpha * row_scale[m] * A B^T + bias[n]) + residual[m, n]
  grouped  the same without a residual for each expert e on its rows offsets[e] <= m < offsets[e + 1] of A, with
           weights B[e], alpha[e] and bias[e]; rows outside every expert stay as they were in the output

`gated`: the weight's rows alternate between a gate and an up projection, D[m, j] = act(y[m, 2j]) * y[m, 2j + 1].
Every operand is what a quantizer leaves: packed codes and scale bytes in 128x4 tiles.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------------------- the cases
def _dense(name, kind, m, n, k, activation=None, gated=False, bias=False, residual=False, per_row=False, out="bfloat16"):
    return {"name": name, "op": "dense", "kind": kind, "m": m, "n": n, "k": k, "activation": activation or "none",
            "gated": gated, "bias": bias, "residual": residual, "per_row": per_row, "out": out}


def _grouped(name, kind, experts, active, m, n, k, activation=None, gated=False, bias=False, per_row=False, tail=0,
             out="bfloat16"):
    return {"name": name, "op": "grouped", "kind": kind, "experts": experts, "active": active, "m": m, "n": n, "k": k,
            "activation": activation or "none", "gated": gated, "bias": bias, "per_row": per_row, "tail": tail, "out": out}


def listed():
    return [
        # one token through the 14B feed-forward layer's first linear, bias and GELU fused: the smallest call
        _dense("dense_fp4_in_m1", "nvfp4", 1, 13824, 5120, "gelu_tanh", bias=True, per_row=True),
        # a small decoding batch through its second linear, added onto the residual stream
        _dense("dense_fp4_out_m16", "nvfp4", 16, 5120, 13824, bias=True, residual=True, per_row=True),
        # an odd prompt length through a gated first linear
        _dense("dense_fp4_gated_m1013", "nvfp4", 1013, 13824, 5120, "silu", gated=True, per_row=True),
        # the whole sequence of a video through the feed-forward layer: first and second linear, the largest calls
        _dense("dense_fp4_in_m32760", "nvfp4", 32760, 13824, 5120, "gelu_tanh", bias=True),
        _dense("dense_fp4_out_m32760", "nvfp4", 32760, 5120, 13824, bias=True, residual=True),
        # an attention output projection in 8 bits onto a residual stream held in 32 bits
        _dense("dense_fp8_m4100_f32", "mxfp8", 4100, 5120, 5120, bias=True, residual=True, out="float32"),
        # 128 small experts, eight for each token: one token, a decoding batch, and a prompt's first and second product
        _grouped("experts_fp4_token", "nvfp4", 128, 8, 8, 1536, 2048, "silu", gated=True, per_row=True),
        _grouped("experts_fp4_batch64", "nvfp4", 128, 117, 512, 1536, 2048, "silu", gated=True, per_row=True),
        _grouped("experts_fp4_prompt_in", "nvfp4", 128, 128, 32768, 1536, 2048, "silu", gated=True, per_row=True),
        _grouped("experts_fp4_prompt_out", "nvfp4", 128, 128, 32768, 2048, 768, per_row=True),
        # eight large experts, two for each token, a prompt of 8190 tokens
        _grouped("experts_fp4_large", "nvfp4", 8, 8, 16380, 13824, 5120, "gelu_tanh", gated=True, bias=True),
        # 8-bit experts with a bias, some of them without a token, in a buffer with rows to spare
        _grouped("experts_fp8_m1501", "mxfp8", 16, 13, 1501, 2048, 1024, "gelu", bias=True, tail=35),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step) * step))


def draw(rng):
    kind = rng.choice(("nvfp4", "nvfp4", "mxfp8"))
    activation = rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu"))
    gated, bias, out = rng.random() < 0.3, rng.random() < 0.5, rng.choice(("bfloat16", "bfloat16", "float32"))
    per_row = kind == "nvfp4" and rng.random() < 0.5
    if rng.random() < 0.5:
        # every size from one row to the largest listed; K also where it ends inside a stage of the pipeline
        m, n, k = _log(rng, 1, 32760), _log(rng, 256, 13824, 16), _log(rng, 256, 13824, 32)
        while m * n * k > 32760 * 13824 * 5120:
            m = max(1, m // 2)
        return _dense("", kind, m, n, k, activation, gated, bias, rng.random() < 0.5, per_row, out)
    experts = _log(rng, 2, 256)
    n, k = _log(rng, 256, 13824, 16), _log(rng, 256, 5120, 32)
    while experts * n * k > 256 * 1536 * 2048:  # about the weights of the listed cases
        experts = max(2, experts // 2)
        if experts == 2:
            break
    m = _log(rng, 1, 32768)
    while m * n * k > 32760 * 13824 * 5120:
        m //= 2
    active = max(1, min(experts, m, round(experts * rng.uniform(0.3, 1.0))))
    return _grouped("", kind, experts, active, m, n, k, activation, gated, bias, per_row, rng.choice((0, 0, 1, 100)), out)


# --------------------------------------------------------------------------------------------------------- the inputs
def _tiles(s):
    """[B, rows, cols] scale bytes -> [B, bytes] in 128x4 tiles: 512 bytes for 128 rows x 4 columns, padding 0."""
    b, r, c = s.shape
    rb, cb = -(-r // 128), -(-c // 4)
    p = torch.zeros((b, rb * 128, cb * 4), dtype=torch.uint8, device=s.device)
    p[:, :r, :c] = s
    return p.view(b, rb, 4, 32, cb, 4).permute(0, 1, 4, 3, 2, 5).reshape(b, -1).contiguous()


def _quantized(gen, kind, shape, outliers):
    """Normal values, quantized along the last axis as a quantizer leaves them: (codes, tiled scales, decode scale).
    Some activations are fifty times the others, as a transformer's are."""
    b, r, k = shape
    group = 16 if kind == "nvfp4" else 32
    codes = torch.empty((b, r, k // 2 if kind == "nvfp4" else k), dtype=torch.uint8, device="cuda")
    scales = torch.empty((b, r, k // group), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // k)  # rows at a time, to bound the memory
    gs = 1.0 if outliers else 448.0
    edges = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), device="cuda")
    flat_c, flat_s = codes.view(b * r, -1), scales.view(b * r, -1)
    for i in range(0, b * r, step):
        x = torch.randn((min(step, b * r - i), k), generator=gen, device="cuda")
        if outliers:
            x[torch.rand(x.shape, generator=gen, device="cuda") < 1e-3] *= 50
        x = x.view(x.shape[0], -1, group)
        top = x.abs().amax(-1, keepdim=True)
        if kind == "nvfp4":
            s = (top * (gs / 6)).clamp(max=448).to(torch.float8_e4m3fn)
            x = x * (gs / s.float().clamp(min=2.0 ** -9))
            c = torch.bucketize(x.abs(), edges).to(torch.uint8) + (x < 0).to(torch.uint8) * 8
            c = c.view(c.shape[0], -1)
            flat_c[i:i + step] = c[:, 0::2] + c[:, 1::2] * 16
            flat_s[i:i + step] = s.view(torch.uint8).view(c.shape[0], -1)
        else:
            e = (top.log2().floor() - 8).clamp(-127, 127)
            x = (x * torch.exp2(-e)).clamp(-448, 448).to(torch.float8_e4m3fn)
            flat_c[i:i + step] = x.view(torch.uint8).view(x.shape[0], -1)
            flat_s[i:i + step] = (e + 127).to(torch.uint8).view(x.shape[0], -1)
    return codes, _tiles(scales), 1.0 / gs


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    kind, m, n, k = case["kind"], case["m"], case["n"], case["k"]
    grouped = case["op"] == "grouped"
    experts = case["experts"] if grouped else 1
    rows = m + case.get("tail", 0)
    a, sfa, _ = _quantized(gen, kind, (1, rows, k), True)
    b, sfb, inv = _quantized(gen, kind, (experts, n, k), False)
    s = {"case": case, "a": a[0], "sfa": sfa[0], "b": b, "sfb": sfb}
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    # products of a width-k sum come out near one, each expert's weights with a scale of their own
    unit = inv if kind == "nvfp4" else 1.0
    s["alpha"] = unit / math.sqrt(k) * (0.5 + torch.rand(experts, generator=gen, device="cuda"))
    s["row_scale"] = (0.5 + torch.rand(rows, generator=gen, device="cuda")) if case["per_row"] else None
    s["bias"] = (rand(experts, n) * 0.1).bfloat16() if case["bias"] else None
    dtype = getattr(torch, case["out"])
    cols = n // 2 if case["gated"] else n
    s["residual"] = rand(rows, cols).to(dtype) if case.get("residual") else None
    if grouped:
        # `active` experts have a token at least; the rest of the rows fall unevenly, as a router's do
        on = torch.randperm(experts, generator=gen, device="cuda")[:case["active"]]
        share = torch.rand(case["active"], generator=gen, device="cuda").clamp(min=1e-6) ** 1.5
        more = torch.multinomial(share, m - case["active"], replacement=True, generator=gen) if m > case["active"] \
            else torch.zeros(0, dtype=torch.long, device="cuda")
        count = torch.zeros(experts, dtype=torch.long, device="cuda")
        count[on] = 1 + torch.bincount(more, minlength=case["active"])
        s["offsets"] = torch.cat((count.new_zeros(1), count.cumsum(0))).int()
        s["out"] = torch.zeros((rows, cols), dtype=dtype, device="cuda") if case["tail"] else None
    else:
        s["b"], s["sfb"] = b[0], sfb[0]
    return s


# --------------------------------------------------------------------------------------------------------- the passes
def _values(kind, codes, tiles, rows, k):
    """The fp32 values of [rows, k] packed codes with tiled scales."""
    group = 16 if kind == "nvfp4" else 32
    c = k // group
    rb, cb = -(-rows // 128), -(-c // 4)
    s = tiles.view(rb, cb, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rb * 128, cb * 4)[:rows, :c]
    if kind == "nvfp4":
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
        v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).view(rows, c, group)
        s = s.contiguous().view(torch.float8_e4m3fn).float()
    else:
        v = codes.view(torch.float8_e4m3fn).float().view(rows, c, group)
        s = torch.exp2(s.float() - 127)
    return (v * s[:, :, None]).view(rows, k)


def _activated(y, name):
    if name == "relu":
        return y.clamp(min=0)
    if name == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    return y * torch.sigmoid(y) if name == "silu" else y


def _epilogue(case, acc, alpha, row_scale, bias):
    y = acc * alpha
    if row_scale is not None:
        y = y * row_scale[:, None]
    if bias is not None:
        y = y + bias.float()
    return _activated(y[:, 0::2], case["activation"]) * y[:, 1::2] if case["gated"] else _activated(y, case["activation"])


def _plain(s):
    case = s["case"]
    kind, n, k = case["kind"], case["n"], case["k"]
    a = _values(kind, s["a"], s["sfa"], s["a"].shape[0], k)
    dtype = getattr(torch, case["out"])
    if case["op"] == "dense":
        acc = a @ _values(kind, s["b"], s["sfb"], n, k).t()
        y = _epilogue(case, acc, s["alpha"], s["row_scale"], None if s["bias"] is None else s["bias"][0])
        return (y if s["residual"] is None else y + s["residual"].float()).to(dtype)
    out = s["out"] if s["out"] is not None else torch.empty((a.shape[0], n // 2 if case["gated"] else n), dtype=dtype,
                                                            device=a.device)
    edge = s["offsets"].tolist()
    for e in range(case["experts"]):
        i, j = edge[e], edge[e + 1]
        if i == j:
            continue
        acc = a[i:j] @ _values(kind, s["b"][e], s["sfb"][e], n, k).t()
        out[i:j] = _epilogue(case, acc, s["alpha"][e], None if s["row_scale"] is None else s["row_scale"][i:j],
                             None if s["bias"] is None else s["bias"][e]).to(dtype)
    return out


def run(state):
    if not own:
        return _plain(state)
    import block_scaled_precision_05_b200 as bsp
    s, case = state, state["case"]
    k, fp4 = case["k"], case["kind"] == "nvfp4"
    kw = {"alpha": s["alpha"], "bias": s["bias"], "out_dtype": getattr(torch, case["out"]),
          "activation": None if case["activation"] == "none" else case["activation"], "gated": case["gated"]}
    if fp4:
        kw["row_scale"] = s["row_scale"]
    a = (bsp.NVFP4Tensor if fp4 else bsp.MXFP8Tensor)(s["a"], s["sfa"], k)
    if case["op"] == "dense":
        b = (bsp.NVFP4Tensor if fp4 else bsp.MXFP8Tensor)(s["b"], s["sfb"], k)
        if s["bias"] is not None:
            kw["bias"] = s["bias"][0]
        return (bsp.nvfp4_gemm if fp4 else bsp.mxfp8_gemm)(a, b, residual=s["residual"], **kw)
    b = (bsp.NVFP4Experts if fp4 else bsp.MXFP8Experts)(s["b"], s["sfb"], k)
    return (bsp.nvfp4_grouped_gemm if fp4 else bsp.mxfp8_grouped_gemm)(a, b, s["offsets"], out=s["out"], **kw)


def work(case):
    """Each operand read once (of the experts, those with rows), the output written once."""
    m, n, k = case["m"], case["n"], case["k"]
    row = k / 2 + k / 16 if case["kind"] == "nvfp4" else k + k / 32
    experts = case["active"] if case["op"] == "grouped" else 1
    size = 4 if case["out"] == "float32" else 2
    cols = n // 2 if case["gated"] else n
    total = m * row + experts * n * row + m * cols * size + experts * 4
    total += 4 * m * case["per_row"] + 2 * n * experts * case["bias"] + m * cols * size * bool(case.get("residual"))
    total += 4 * (case["experts"] + 1) if case["op"] == "grouped" else 0
    return {"bytes": int(total), "flops": 2 * m * n * k}


# ------------------------------------------------------------------------------------------------------ the definition
def _decoded64(kind, codes, tiles, k):
    """Every element from its byte and its scale's byte, found by the tile map's formula, in 64 bits."""
    rows, dev = codes.shape[0], codes.device
    group = 16 if kind == "nvfp4" else 32
    r = torch.arange(rows, device=dev)[:, None]
    c = torch.arange(k // group, device=dev)[None, :]
    where = ((r // 128) * (-(-(k // group) // 4)) + c // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + c % 4
    byte = tiles[where].long()
    if kind == "nvfp4":
        def e4m3(t):
            e, f = (t >> 3) & 15, (t & 7).double()
            return torch.where(e > 0, (8 + f) * 2.0 ** (e.double() - 10), f * 2.0 ** -9)
        def e2m1(t):
            e, f = (t >> 1) & 3, (t & 1).double()
            return torch.where(e > 0, (2 + f) * 2.0 ** (e.double() - 2), f / 2) * (1 - 2 * (t >> 3).double())
        out = torch.empty((rows, k), dtype=torch.float64, device=dev)
        out[:, 0::2], out[:, 1::2] = e2m1(codes.int() & 15), e2m1(codes.int() >> 4)
        scale = e4m3(byte)
    else:
        t = codes.int()
        e, f = (t >> 3) & 15, (t & 7).double()
        out = torch.where(e > 0, (8 + f) * 2.0 ** (e.double() - 10), f * 2.0 ** -9) * (1 - 2 * (t >> 7).double())
        scale = 2.0 ** (byte.double() - 127)
    out.view(rows, -1, group).mul_(scale[:, :, None])
    return out


def _act64(x, name):
    if name == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if name == "gelu":
        return x * torch.special.erfc(-x / math.sqrt(2.0)) / 2
    if name == "gelu_tanh":
        return x / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
    return x / (1 + torch.exp(-x)) if name == "silu" else x


def exact(case, seed):
    s = prepare(case, seed)
    grouped = case["op"] == "grouped"
    edge = s["offsets"].tolist() if grouped else [0, case["m"]]
    rows = case["m"] + case.get("tail", 0)
    d = torch.zeros((rows, case["n"] // 2 if case["gated"] else case["n"]), dtype=torch.float64, device="cuda")
    a = _decoded64(case["kind"], s["a"], s["sfa"], case["k"])
    for e in range(len(edge) - 1):
        lo, hi = edge[e], edge[e + 1]
        if lo == hi:
            continue
        b = _decoded64(case["kind"], s["b"][e], s["sfb"][e], case["k"]) if grouped else \
            _decoded64(case["kind"], s["b"], s["sfb"], case["k"])
        y = torch.mm(a[lo:hi], b.T).mul_(s["alpha"][e].double())
        if s["row_scale"] is not None:
            y.mul_(s["row_scale"][lo:hi].double().unsqueeze(1))
        if s["bias"] is not None:
            y.add_(s["bias"][e].double())
        if case["gated"]:
            y = y.view(hi - lo, -1, 2)
            d[lo:hi] = _act64(y[..., 0], case["activation"]) * y[..., 1]
        else:
            d[lo:hi] = _act64(y, case["activation"])
    return d if s["residual"] is None else d + s["residual"].double()
