"""GEMMs with a fused epilogue and GEMMs grouped by expert against the
definition in 64 bits on the oracle's quantized operands.

Tolerance, derived per output (u32 = 2^-24, S = |alpha row_scale| sum |a b|):
  accumulation  every MMA step (K = 64 fp4, 32 fp8) aligns its products and adds them to the fp32 accumulator,
                off by at most 2^-22 of S each: (steps + 4) 2^-22 S; the scale and bias add 3 u32 (|y| + |bias|)
  activation    slope at most 1.13; its exponential's argument s (in powers of two) is off by 2 u32 |s|, the two
                hardware approximations by 2^-22 each, the fitted tail of gelu by 6e-7: (|s| + 6) 2^-22 + 6e-7 relative
                to act(y), which for gelu stands for |y| Q(|y|) <= |y|
  gate          |act| tol(up) + |up| tol(act);   residual and product: u32 each
  output        half a step: finfo.eps / 2 relative to the value, plus the smallest normal number
"""
import math

import numpy as np
import pytest
import torch

import block_scaled_precision_05_b200 as bsp
import oracle
from block_scaled_precision_05_b200 import _native as nat
from block_scaled_precision_05_b200 import api
from tests._gpu import DEV, down, up, up_bf16

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


def bf16_bits(rng, *shape, scale=1.0):
    return oracle.bf16_round(rng.standard_normal(shape) * scale).astype(np.uint16)


def bits64(b):
    return oracle.bf16_bits_to_f64(b)


class Operand:
    """[B, rows, K] random values quantized by the oracle: device codes and scales, and their values in 64 bits."""

    def __init__(self, rng, fp4, b, rows, K, scale=1.0):
        codes, sfs, dec = [], [], []
        for _ in range(b):
            x = bf16_bits(rng, rows, K, scale=scale)
            if fp4:
                c, s = oracle.nvfp4_quantize(x, 1.0)
                dec.append(oracle.nvfp4_dequantize(c, s, K))
            else:
                c, s = oracle.mxfp8_quantize(x)
                dec.append(oracle.mxfp8_dequantize(c, s, K))
            codes.append(c)
            sfs.append(np.asarray(s, dtype=np.uint8).reshape(-1))
        self.codes, self.sf = up(np.stack(codes)), up(np.stack(sfs))
        self.dec, self.K, self.fp4 = dec, K, fp4

    def tensor(self):
        return (bsp.NVFP4Tensor if self.fp4 else bsp.MXFP8Tensor)(self.codes[0], self.sf[0], self.K)

    def experts(self):
        return (bsp.NVFP4Experts if self.fp4 else bsp.MXFP8Experts)(self.codes, self.sf, self.K)


def act64(y, name):
    """(act(y), bound of its relative error) in 64 bits."""
    s = np.zeros_like(y)
    with np.errstate(over="ignore"):
        if name == "relu":
            a = np.maximum(y, 0)
        elif name == "gelu":
            a = y * np.vectorize(lambda v: 0.5 * math.erfc(-v / math.sqrt(2)))(y) if y.size else y
            s = 0.73 * y * y
        elif name == "gelu_tanh":
            s = np.abs(y) * (2.31 + 0.103 * y * y)
            a = y / (1 + np.exp(-2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
        elif name == "silu":
            s = 1.45 * np.abs(y)
            a = y / (1 + np.exp(-y))
        else:
            return y, 0.0
    return a, (np.minimum(s, 200) + 6) * 2.0 ** -22 + 6e-7


def reference(a, b, fp4, alpha, row_scale, bias, act, gated, residual, dtype):
    """(D, tolerance) in 64 bits for decoded operands a [M, K], b [N, K]."""
    K = a.shape[1]
    scale = np.float64(alpha) * (np.ones(a.shape[0]) if row_scale is None else row_scale.astype(np.float64))
    y = a @ b.T * scale[:, None]
    size = np.abs(a) @ np.abs(b).T * np.abs(scale)[:, None]
    bz = 0.0 if bias is None else bits64(bias)[None, :]
    y = y + bz
    tol = (K / (64 if fp4 else 32) + 4) * 2.0 ** -22 * size + 3 * U32 * (np.abs(y) + np.abs(bz))

    def activated(v, t):
        r, rel = act64(v, act)
        if act is None:
            return v, t
        # gelu for v > 0 is v - v Q: the relative error falls on v Q and the rounding on the result
        return r, 1.13 * t + rel * np.abs(r) + (2 * U32 + 6e-7) * np.abs(v) * (act == "gelu")

    if gated:
        g, tg = activated(y[:, 0::2], tol[:, 0::2])
        u, tu = y[:, 1::2], tol[:, 1::2]
        d = g * u
        tol = np.abs(g) * tu + np.abs(u) * tg + tg * tu + U32 * np.abs(d)
    else:
        d, tol = activated(y, tol)
    if residual is not None:
        d = d + residual
        tol = tol + U32 * np.abs(d)
    info = torch.finfo(dtype)
    return d, tol * (1 + info.eps) + info.eps / 2 * np.abs(d) + info.tiny


def check(got, ref, tol, what=""):
    g = got.double().cpu().numpy()
    assert g.shape == ref.shape
    bad = ~(np.abs(g - ref) <= tol)
    if bad.any():
        i = tuple(int(v) for v in np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())}/{bad.size} out of tolerance, first {i}: got {g[i]}, "
                             f"want {ref[i]} +- {tol[i]}; rows {sorted(set(np.argwhere(bad)[:, 0].tolist()))[:8]}, "
                             f"columns {sorted(set(np.argwhere(bad)[:, 1].tolist()))[:8]}")


def dense(rng, fp4, M, N, K, act=None, gated=False, bias=False, residual=False, row=False, dtype=torch.bfloat16,
          ld=None, in_place=False):
    A, B = Operand(rng, fp4, 1, M, K), Operand(rng, fp4, 1, N, K, 0.5)
    alpha = np.float32(1.3 / math.sqrt(K))
    rs = (0.5 + rng.random(M)).astype(np.float32) if row else None
    bz = bf16_bits(rng, N, scale=0.3) if bias else None
    cols = N // 2 if gated else N
    wide = torch.zeros((M, ld or cols), dtype=dtype, device=DEV)
    wide.fill_(7.0)
    out = wide[:, :cols]
    res = res64 = None
    if residual:
        res = (out if in_place else torch.empty((M, ld or cols), dtype=dtype, device=DEV)[:, :cols])
        res.copy_(torch.from_numpy(rng.standard_normal((M, cols))).to(dtype))
        res64 = res.double().cpu().numpy()
    kw = dict(alpha=up(np.array([alpha])), bias=None if bz is None else up_bf16(bz), out=out, out_dtype=dtype,
              activation=act, gated=gated, residual=res)
    if fp4:
        kw["row_scale"] = None if rs is None else up(rs)
    got = (bsp.nvfp4_gemm if fp4 else bsp.mxfp8_gemm)(A.tensor(), B.tensor(), **kw)
    assert bsp.device_status() == 0
    assert got.data_ptr() == out.data_ptr()
    ref, tol = reference(A.dec[0], B.dec[0], fp4, alpha, rs, bz, act, gated, res64, dtype)
    check(got, ref, tol, f"M={M} N={N} K={K}")
    if ld:
        assert bool((wide[:, cols:] == 7.0).all()), "columns past D were written"


# every token-tile width (1 row to several tiles), weights that end inside a panel, K inside a stage and over the ring
DENSE = [
    (True, 1, 8, 32, "silu", False, False, False, False, torch.bfloat16),
    (True, 1, 16, 64, "silu", True, True, True, True, torch.bfloat16),
    (True, 5, 136, 96, "gelu", False, True, False, True, torch.float32),
    (True, 16, 256, 256, None, False, True, True, False, torch.bfloat16),
    (True, 17, 264, 288, "relu", False, True, True, True, torch.float32),
    (True, 33, 128, 2048, "gelu_tanh", True, False, False, True, torch.bfloat16),
    (True, 48, 400, 512, "gelu", True, True, True, False, torch.float32),
    (True, 64, 640, 1536, "gelu_tanh", False, True, True, True, torch.bfloat16),
    (True, 65, 264, 1056, "silu", False, False, True, True, torch.bfloat16),
    (True, 97, 256, 256, "silu", True, True, False, False, torch.float32),
    (True, 130, 520, 512, "gelu", False, True, True, True, torch.bfloat16),
    (True, 256, 384, 1024, "gelu_tanh", True, True, True, True, torch.bfloat16),
    (True, 257, 8, 64, None, False, False, True, False, torch.float32),
    (True, 300, 272, 2048, "relu", True, True, False, True, torch.bfloat16),
    (True, 777, 1000, 352, "gelu", False, True, True, True, torch.float32),
    (False, 1, 16, 32, "gelu", True, True, True, False, torch.float32),
    (False, 13, 136, 160, "silu", False, True, False, False, torch.bfloat16),
    (False, 64, 256, 1056, "gelu_tanh", False, True, True, False, torch.bfloat16),
    (False, 100, 272, 512, None, True, True, False, False, torch.float32),
    (False, 258, 264, 1024, "relu", False, False, True, False, torch.bfloat16),
    (False, 600, 512, 224, "gelu", False, True, True, False, torch.float32),
]


@pytest.mark.parametrize("fp4,M,N,K,act,gated,bias,residual,row,dtype", DENSE)
def test_dense(fp4, M, N, K, act, gated, bias, residual, row, dtype):
    dense(np.random.default_rng(M * 7919 + N), fp4, M, N, K, act, gated, bias, residual, row, dtype)


@pytest.mark.parametrize("M", [7, 64, 200])
@pytest.mark.parametrize("in_place", [False, True])
def test_dense_strided_output_and_residual(M, in_place):
    dense(np.random.default_rng(M), True, M, 272, 256, "gelu_tanh", False, True, True, True, ld=304, in_place=in_place)
    dense(np.random.default_rng(M), False, M, 272, 256, "silu", True, True, True, False, torch.float32, ld=200,
          in_place=in_place)


@pytest.mark.parametrize("M", list(range(16, 257, 16)) + [2, 31, 95, 129, 161, 225])
def test_every_tile_width(M):
    """The MMA's N takes every multiple of its granularity, in both forms."""
    dense(np.random.default_rng(M), True, M, 256, 512, None, False, False, True)
    dense(np.random.default_rng(M), False, M, 128, 256, None, False, False, True)


# --------------------------------------------------------------------------- grouped
def grouped(rng, fp4, counts, N, K, act=None, gated=False, bias=False, row=False, dtype=torch.bfloat16, head=0, tail=0):
    E, M = len(counts), head + sum(counts) + tail
    A, B = Operand(rng, fp4, 1, M, K), Operand(rng, fp4, E, N, K, 0.5)
    alpha = ((0.5 + rng.random(E)) * 1.3 / math.sqrt(K)).astype(np.float32)
    rs = (0.5 + rng.random(M)).astype(np.float32) if row else None
    bz = bf16_bits(rng, E, N, scale=0.3) if bias else None
    off = head + np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    cols = N // 2 if gated else N
    out = torch.full((M, cols), 7.0, dtype=dtype, device=DEV)
    kw = dict(alpha=up(alpha), bias=None if bz is None else up_bf16(bz), out=out, out_dtype=dtype, activation=act,
              gated=gated)
    if fp4:
        kw["row_scale"] = None if rs is None else up(rs)
    got = (bsp.nvfp4_grouped_gemm if fp4 else bsp.mxfp8_grouped_gemm)(A.tensor(), B.experts(), up(off.astype(np.int32)),
                                                                      **kw)
    assert bsp.device_status() == 0
    for e in range(E):
        i, j = off[e], off[e + 1]
        if i < j:
            ref, tol = reference(A.dec[0][i:j], B.dec[e], fp4, alpha[e], None if rs is None else rs[i:j],
                                 None if bz is None else bz[e], act, gated, None, dtype)
            check(got[i:j], ref, tol, f"expert {e} rows {i}..{j}")
    rest = torch.cat((got[:head], got[M - tail:] if tail else got[:0]))
    assert bool((rest == 7.0).all()), "rows outside every expert were written"
    return got


GROUPED = [
    # few rows per expert: the 64-token form
    (True, [1], 16, 32, "silu", True, False, False, torch.bfloat16, 0, 0),
    (True, [1, 0, 2, 0, 0, 5], 136, 64, "gelu", False, True, True, torch.float32, 0, 3),
    (True, [0, 31, 64, 65, 1, 0, 16, 17, 130, 3], 272, 288, "silu", True, True, True, torch.bfloat16, 5, 9),
    (True, [3] * 40, 128, 512, "gelu_tanh", False, True, True, torch.bfloat16, 0, 0),
    (True, [127, 1, 1, 127, 0, 33, 95], 264, 1056, None, False, False, True, torch.float32, 1, 1),
    # many rows per expert: CTA pairs, starts at every offset within a 32-row line and a 128-row band
    (True, [1, 255, 256, 257, 31, 33, 700], 264, 320, "silu", False, True, True, torch.bfloat16, 0, 0),
    (True, [300, 0, 95, 161, 513], 272, 2048, "silu", True, True, True, torch.bfloat16, 33, 40),
    (True, [90, 91, 92, 93, 94], 400, 96, "gelu_tanh", True, False, False, torch.float32, 7, 0),
    (True, [600], 520, 512, "relu", False, True, False, torch.bfloat16, 64, 64),
    (False, [2, 0, 1, 7], 24, 32, "gelu", False, True, False, torch.bfloat16, 0, 1),
    (False, [20, 64, 1, 100, 3], 272, 480, "silu", True, True, False, torch.float32, 3, 0),
    (False, [130, 257, 0, 333, 80], 264, 1024, "gelu", False, True, False, torch.bfloat16, 97, 5),
]


@pytest.mark.parametrize("fp4,counts,N,K,act,gated,bias,row,dtype,head,tail", GROUPED)
def test_grouped(fp4, counts, N, K, act, gated, bias, row, dtype, head, tail):
    grouped(np.random.default_rng(sum(counts) + N), fp4, counts, N, K, act, gated, bias, row, dtype, head, tail)


@pytest.mark.parametrize("head", [0, 1, 31, 32, 63, 64, 96, 100, 127])
def test_grouped_scale_shift(head):
    """An expert's first row at every word and line of a scale band, for both formats and forms."""
    for fp4 in (True, False):
        grouped(np.random.default_rng(head), fp4, [40, 7], 128, 256, head=head, tail=1)
        grouped(np.random.default_rng(head), fp4, [250, 131], 256, 256, head=head, tail=1)


def test_grouped_many_experts():
    rng = np.random.default_rng(5)
    counts = rng.integers(0, 4, size=512).tolist()
    grouped(rng, True, counts, 32, 64, "silu", True, True, True)


def test_grouped_without_rows():
    rng = np.random.default_rng(6)
    grouped(rng, True, [0, 0, 0], 128, 64, head=4, tail=3)
    A = bsp.NVFP4Tensor(torch.empty((0, 32), dtype=torch.uint8, device=DEV), torch.empty(0, dtype=torch.uint8, device=DEV), 64)
    B = Operand(rng, True, 2, 16, 64).experts()
    assert bsp.nvfp4_grouped_gemm(A, B, torch.zeros(3, dtype=torch.int32, device=DEV)).shape == (0, 16)


def test_grouped_offsets_out_of_order():
    """Offsets outside [0, M] are clamped, one below an earlier one counts as that one."""
    rng = np.random.default_rng(8)
    M, N, K = 200, 64, 64
    A, B = Operand(rng, True, 1, M, K), Operand(rng, True, 5, N, K)
    run = lambda o: bsp.nvfp4_grouped_gemm(A.tensor(), B.experts(), up(np.array(o, np.int32)),  # noqa: E731
                                           out=torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV))
    got = run([-9, 30, 10, 150, 120, 10 ** 9])
    want = run([0, 30, 30, 150, 150, 200])
    assert bsp.device_status() == 0
    assert torch.equal(got, want)


def test_one_expert_is_the_dense_gemm():
    """Same operands, one expert with every row: the same bits as the dense call, and as the plain GEMM within the
    accumulation's freedom (none of it observed: both sum the same MMA steps in the same order)."""
    rng = np.random.default_rng(9)
    for M in (20, 300):
        A, B = Operand(rng, True, 1, M, 512), Operand(rng, True, 1, 272, 512)
        alpha = torch.tensor([0.05], device=DEV)
        off = torch.tensor([0, M], dtype=torch.int32, device=DEV)
        g = bsp.nvfp4_grouped_gemm(A.tensor(), B.experts(), off, alpha, activation="silu")
        d = bsp.nvfp4_gemm(A.tensor(), B.tensor(), alpha, activation="silu")
        assert torch.equal(g, d)


def test_repeated_launches_give_the_same_bits():
    rng = np.random.default_rng(10)
    A, B = Operand(rng, True, 1, 900, 768), Operand(rng, True, 6, 272, 768)
    off = torch.tensor([0, 3, 300, 300, 557, 600, 900], dtype=torch.int32, device=DEV)
    first = bsp.nvfp4_grouped_gemm(A.tensor(), B.experts(), off, activation="gelu", gated=True)
    for _ in range(50):
        assert torch.equal(first, bsp.nvfp4_grouped_gemm(A.tensor(), B.experts(), off, activation="gelu", gated=True))
    assert bsp.device_status() == 0


# --------------------------------------------------------------------------- as a user has them
def test_linear_layers_take_the_epilogue():
    """NVFP4Linear / MXFP8Linear with activation, gate and residual equal their parts put together from plain calls:
    the fused result lies within the roundings of the unfused one (one bf16 rounding of y, of act(y) and of the sum)."""
    torch.manual_seed(0)
    w1, w3 = (torch.randn(256, 128, device=DEV).bfloat16() * 0.1 for _ in range(2))
    b = torch.randn(512, device=DEV).bfloat16()
    x = torch.randn(3, 50, 128, device=DEV).bfloat16()
    res = torch.randn(3, 50, 256, device=DEV).bfloat16()
    for make in (lambda: bsp.NVFP4Linear(bsp.interleave_gated(w1, w3), b, per_token=True),
                 lambda: bsp.NVFP4Linear(bsp.interleave_gated(w1, w3), b),
                 lambda: bsp.MXFP8Linear(bsp.interleave_gated(w1, w3), b)):
        lin = make()
        got = lin(x, activation="silu", gated=True, residual=res)
        assert got.shape == (3, 50, 256)
        y = lin(x, out_dtype=torch.float32).double()
        want = torch.nn.functional.silu(y[..., 0::2]) * y[..., 1::2] + res.double()
        assert bool(((got.double() - want).abs() <= 2 ** -8 * want.abs() + 1e-4).all())


def check_layer(layer, x, edge, got, act, gated):
    """One grouped layer's output against the definition on the operands it quantizes its tokens and weights to."""
    fp4 = isinstance(layer, bsp.NVFP4GroupedLinear)
    K, w = layer.in_features, layer.weight
    if fp4:
        xq = layer.quantize_input(x)
        a = oracle.nvfp4_dequantize(down(xq.codes), down(xq.sf), K)
        alpha, rs = down(layer.alpha), down(xq.row_inv_gs) if layer.per_token else None
        dec = lambda e: oracle.nvfp4_dequantize(down(w.codes[e]), down(w.sf[e]), K)  # noqa: E731
    else:
        xq = bsp.mxfp8_quantize(x)
        a = oracle.mxfp8_dequantize(down(xq.q), down(xq.sf), K)
        alpha, rs = np.ones(layer.experts, np.float32), None
        dec = lambda e: oracle.mxfp8_dequantize(down(w.q[e]), down(w.sf[e]), K)  # noqa: E731
    for e in range(layer.experts):
        i, j = edge[e], edge[e + 1]
        if i < j:
            ref, tol = reference(a[i:j], dec(e), fp4, alpha[e], None if rs is None else rs[i:j], None, act, gated, None,
                                 got.dtype)
            check(got[i:j], ref, tol, f"expert {e}")


def test_expert_feed_forward_chain():
    """Tokens through both products of a mixture's experts (quantize, gated product, quantize, product), captured in a
    graph and replayed on new tokens and another routing."""
    torch.manual_seed(1)
    E, T, K, F = 8, 96, 256, 192
    w1, w3 = (torch.randn(E, F, K, device=DEV).bfloat16() / 16 for _ in range(2))
    w2 = torch.randn(E, K, F, device=DEV).bfloat16() / 14
    for mx in (False, True):
        if mx:
            up_, down_ = bsp.MXFP8GroupedLinear(bsp.interleave_gated(w1, w3), activation="silu", gated=True), bsp.MXFP8GroupedLinear(w2)
        else:
            up_ = bsp.NVFP4GroupedLinear(bsp.interleave_gated(w1, w3), per_token=True, activation="silu", gated=True)
            down_ = bsp.NVFP4GroupedLinear(w2, per_token=True)
        x = torch.empty(T, K, device=DEV, dtype=torch.bfloat16)
        off = torch.empty(E + 1, dtype=torch.int32, device=DEV)

        def fill(seed):
            g = torch.Generator(DEV).manual_seed(seed)
            x.copy_(torch.randn(T, K, generator=g, device=DEV))
            ids = torch.randint(0, E, (T,), generator=g, device=DEV)
            off.copy_(torch.cat((off.new_zeros(1), torch.bincount(ids, minlength=E).cumsum(0).int())))

        def layer():
            return down_(up_(x, off), off)

        fill(0)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer()
        for seed in (1, 2):
            fill(seed)
            graph.replay()
            eager = layer()
            torch.cuda.synchronize()
            assert bsp.device_status() == 0
            assert torch.equal(out, eager)
            h = up_(x, off)
            for layer_, tokens, got, act, gated in ((up_, x, h, "silu", True), (down_, h, eager, None, False)):
                check_layer(layer_, tokens, off.tolist(), got, act, gated)


def test_on_a_side_stream():
    rng = np.random.default_rng(12)
    A, B = Operand(rng, True, 1, 300, 256), Operand(rng, True, 4, 128, 256)
    off = torch.tensor([0, 10, 200, 200, 300], dtype=torch.int32, device=DEV)
    want = bsp.nvfp4_grouped_gemm(A.tensor(), B.experts(), off)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            outs.append([bsp.nvfp4_grouped_gemm(A.tensor(), B.experts(), off) for _ in range(5)])
    torch.cuda.synchronize()
    assert all(torch.equal(want, o) for group in outs for o in group)
    assert bsp.device_status() == 0


# --------------------------------------------------------------------------- refusals
def test_refusals():
    rng = np.random.default_rng(13)
    A, B = Operand(rng, True, 1, 32, 64), Operand(rng, True, 2, 32, 64)
    a, e, b = A.tensor(), B.experts(), bsp.NVFP4Tensor(B.codes[0], B.sf[0], 64)
    off = torch.tensor([0, 3, 32], dtype=torch.int32, device=DEV)
    res = torch.zeros(32, 32, dtype=torch.bfloat16, device=DEV)
    wide = torch.zeros(32, 40, dtype=torch.bfloat16, device=DEV)
    ones = torch.ones(3, device=DEV)
    bad = [
        lambda: bsp.nvfp4_gemm(a, b, activation="tanh"),
        lambda: bsp.nvfp4_gemm(a, b, residual=res.float()),
        lambda: bsp.nvfp4_gemm(a, b, residual=res[:, :16]),
        lambda: bsp.nvfp4_gemm(a, b, residual=res[:16]),
        lambda: bsp.nvfp4_gemm(a, b, residual=res.cpu()),
        lambda: bsp.nvfp4_gemm(a, b, residual=wide[:, 8:], out=wide[:, :32]),
        lambda: bsp.nvfp4_gemm(a, b, gated=True, out=res),
        lambda: bsp.nvfp4_gemm(a, b, row_scale=ones, activation="relu"),
        lambda: bsp.nvfp4_gemm(bsp.NVFP4Tensor(a.codes, a.sf, 64, sf_layout="8x4"), b, activation="relu"),
        lambda: bsp.nvfp4_gemm(bsp.NVFP4Tensor(a.codes, a.sf[:100], 64), b, activation="relu"),
        lambda: bsp.nvfp4_gemm(bsp.NVFP4Tensor(a.codes[:, :16], a.sf, 64), b, activation="relu"),
        lambda: bsp.nvfp4_grouped_gemm(a, e, off[:2]),
        lambda: bsp.nvfp4_grouped_gemm(a, e, off.long()),
        lambda: bsp.nvfp4_grouped_gemm(a, e, off.cpu()),
        lambda: bsp.nvfp4_grouped_gemm(a, e, None),
        lambda: bsp.nvfp4_grouped_gemm(a, e, off, alpha=ones),
        lambda: bsp.nvfp4_grouped_gemm(a, e, off, bias=res[0]),
        lambda: bsp.nvfp4_grouped_gemm(a, e, off, out=res[:16]),
        lambda: bsp.nvfp4_grouped_gemm(a, bsp.NVFP4Experts(e.codes, e.sf[:1], 64), off),
        lambda: bsp.nvfp4_grouped_gemm(a, bsp.NVFP4Experts(e.codes, e.sf, 96), off),
        lambda: bsp.nvfp4_quantize_experts(torch.zeros(2, 8, 48, device=DEV)),
        lambda: bsp.nvfp4_quantize_experts(torch.zeros(8, 64, device=DEV)),
        lambda: bsp.nvfp4_quantize_experts(torch.zeros(nat.BSP_MAX_EXPERTS + 1, 8, 32, device=DEV)),
        lambda: bsp.interleave_gated(torch.zeros(4, 8), torch.zeros(5, 8)),
        lambda: bsp.NVFP4GroupedLinear(torch.zeros(2, 8, 64, device=DEV), activation="swish"),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            raise AssertionError(f"call {i} was not refused")
    with pytest.raises(api.nat.BSPError):  # 24 gated columns would leave rows of D off their 16-byte boundary
        bsp.nvfp4_gemm(a, bsp.NVFP4Tensor(B.codes[0][:24].contiguous(), B.sf[0], 64), gated=True)
    assert bsp.device_status() == 0
    assert down(res).any() == False  # noqa: E712


# --------------------------------------------------------------------------- what callers do besides
def test_operands_on_one_row_with_any_stride():
    """A single row has no stride: out and residual from a broadcast or a slice."""
    rng = np.random.default_rng(20)
    A, B = Operand(rng, True, 1, 1, 64), Operand(rng, True, 1, 32, 64)
    want = bsp.nvfp4_gemm(A.tensor(), B.tensor(), activation="silu", residual=torch.ones(1, 32, dtype=torch.bfloat16, device=DEV))
    res = torch.ones(40, dtype=torch.bfloat16, device=DEV)[:32].expand(1, 32)
    out = torch.empty(33, 8, 40, dtype=torch.bfloat16, device=DEV)[5, 3, :32].as_strided((1, 32), (7, 1))
    assert torch.equal(want, bsp.nvfp4_gemm(A.tensor(), B.tensor(), activation="silu", residual=res, out=out))


@pytest.mark.parametrize("M", [16, 100, 300])
def test_infinite_and_nan_inputs_stay_in_their_rows(M):
    """alpha, row scales, bias and residual that are infinite or NaN reach only the outputs that the formula gives them;
    padding rows and columns hold nothing that leaks."""
    rng = np.random.default_rng(M)
    A, B = Operand(rng, True, 1, M, 128), Operand(rng, True, 1, 264, 128)
    rs = torch.ones(M, device=DEV)
    rs[3], rs[M - 1] = float("inf"), float("nan")
    bias = torch.zeros(264, dtype=torch.bfloat16, device=DEV)
    bias[5] = float("nan")
    res = torch.zeros(M, 264, dtype=torch.bfloat16, device=DEV)
    res[7, 9] = float("-inf")
    got = bsp.nvfp4_gemm(A.tensor(), B.tensor(), None, rs, bias, activation="relu", residual=res)
    plain = bsp.nvfp4_gemm(A.tensor(), B.tensor(), None, rs, bias, out_dtype=torch.float32)
    # torch's clamp keeps NaN as the kernel does
    want = plain.clamp(min=0) + res.float()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.isinf(got), torch.isinf(want))
    clean = torch.isfinite(want)
    assert int((~clean).sum()) == int(torch.isnan(want).sum()) + int(torch.isinf(want).sum()) > 264
    assert bool(((got.float() - want)[clean].abs() <= 2 ** -8 * want[clean].abs() + 1e-4).all())


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_activation_tails(act):
    """y far out on both sides, through the bias: relative accuracy down to each form's clamp, and the limits."""
    vals = torch.tensor([-1e30, -1000, -60, -39, -20, -13, -9, -6.9, -5, -3, -1, -0.1, -1e-3, 0, 1e-3, 0.1, 1, 3, 5, 9, 20, 60, 1000,
                         1e30], dtype=torch.float64)
    rng = np.random.default_rng(21)
    A, B = Operand(rng, True, 1, 2, 32), Operand(rng, True, 1, 24, 32)
    zero = torch.zeros(1, device=DEV)
    bias = vals.to(torch.bfloat16).to(DEV)
    got = bsp.nvfp4_gemm(A.tensor(), B.tensor(), zero, None, bias, out_dtype=torch.float32, activation=act)[0].double().cpu().numpy()
    y = bias.double().cpu().numpy()
    want, rel = act64(y, act)
    # below the clamp (silu -40, gelu_tanh -7) the value stays at the clamp's: 1.7e-16, 2.3e-15; gelu underflows past 13
    floor = {"silu": 2e-16, "gelu_tanh": 3e-15, "gelu": 1e-37}[act]
    tol = rel * np.abs(want) + 2 * U32 * np.maximum(y, 0) + 6e-7 * np.maximum(y, 0) * (act == "gelu") + floor
    assert np.all(np.abs(got - want) <= tol), list(zip(y, got, want))


def test_two_graphs_at_once():
    """Two captured graphs of the same layer replayed on two streams at a time: nothing is shared between launches."""
    rng = np.random.default_rng(22)
    A, B = Operand(rng, True, 1, 64, 4608), Operand(rng, True, 1, 256, 4608)  # split over a cluster
    C, D = Operand(rng, True, 1, 700, 256), Operand(rng, True, 5, 256, 256)
    off = torch.tensor([0, 100, 100, 350, 699, 700], dtype=torch.int32, device=DEV)
    run = lambda: (bsp.nvfp4_gemm(A.tensor(), B.tensor(), activation="gelu"),  # noqa: E731
                   bsp.nvfp4_grouped_gemm(C.tensor(), D.experts(), off, activation="silu"))
    want = run()
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for _ in streams:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run())
        graphs.append(g)
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(w, o) for pair in outs for w, o in zip(want, pair))
    assert bsp.device_status() == 0


@pytest.mark.parametrize("M,N,K", [(5, 256, 8192), (40, 136, 13824), (128, 128, 4352), (1, 640, 9216)])
def test_split_over_a_cluster(M, N, K):
    """K shared by the CTAs of a cluster (few weight panels, long K): against the definition, and the same bits again."""
    dense(np.random.default_rng(K), True, M, N, K, "silu", False, True, True, True)
    dense(np.random.default_rng(K), False, M, N, K // 2, None, N % 16 == 0, True, False, False, torch.float32)
    rng = np.random.default_rng(M)
    A, B = Operand(rng, True, 1, M, K), Operand(rng, True, 1, N, K)
    first = bsp.nvfp4_gemm(A.tensor(), B.tensor(), activation="relu")
    for _ in range(30):
        assert torch.equal(first, bsp.nvfp4_gemm(A.tensor(), B.tensor(), activation="relu"))


def test_more_tiles_than_a_block_lists():
    """A CTA's tiles past the ones it looks up first: many tiles of one small panel, dense and grouped."""
    rng = np.random.default_rng(23)
    A, B = Operand(rng, False, 1, 40000, 32), Operand(rng, False, 1, 512, 32)
    alpha = torch.tensor([0.1], device=DEV)
    got = bsp.mxfp8_gemm(A.tensor(), B.tensor(), alpha, activation="relu")
    want = bsp.mxfp8_gemm(A.tensor(), B.tensor(), alpha, out_dtype=torch.float32).clamp(min=0)
    assert bool(((got.float() - want).abs() <= 2 ** -8 * want + 1e-5).all())
    counts = rng.integers(0, 40, size=512)
    E, M = Operand(rng, False, 512, 2560, 32), int(counts.sum())
    off = torch.from_numpy(np.concatenate(([0], np.cumsum(counts))).astype(np.int32)).to(DEV)
    X = Operand(rng, False, 1, M, 32)
    got = bsp.mxfp8_grouped_gemm(X.tensor(), E.experts(), off)
    for e in (0, 1, 255, 300, 510, 511):
        i, j = int(off[e]), int(off[e + 1])
        if i < j:
            ref, tol = reference(X.dec[0][i:j], E.dec[e], False, 1.0, None, None, None, False, None, torch.bfloat16)
            check(got[i:j], ref, tol, f"expert {e}")
    assert bsp.device_status() == 0


def test_overlapping_residuals_are_refused():
    """A residual may be the output itself or share no element with it: halves of one wide matrix, rows apart."""
    rng = np.random.default_rng(24)
    A, B = Operand(rng, True, 1, 4, 64).tensor(), Operand(rng, True, 1, 8, 64).tensor()
    buf = torch.zeros(128, dtype=torch.bfloat16, device=DEV)
    m = lambda off, ld: torch.as_strided(buf, (4, 8), (ld, 1), off)  # noqa: E731
    run = lambda out, res: bsp.nvfp4_gemm(A, B, out=out, residual=res)  # noqa: E731
    for out, res in ((m(0, 16), m(8, 16)), (m(8, 16), m(0, 16)), (m(0, 8), m(32, 8)), (m(0, 16), m(0, 16)), (m(0, 24), m(8, 24)),
                     (m(0, 24), m(16, 24)), (m(8, 16), m(16, 16))):
        buf.zero_()
        want = bsp.nvfp4_gemm(A, B, activation=None, residual=torch.zeros(4, 8, dtype=torch.bfloat16, device=DEV))
        assert torch.equal(run(out, res), want)
    for out, res in ((m(0, 8), m(24, 8)), (m(0, 8), m(16, 16)), (m(0, 16), m(0, 8)), (m(0, 16), m(0, 24))):
        with pytest.raises(ValueError, match="overlap"):
            run(out, res)


@pytest.mark.parametrize("M", [1, 40, 300, 1500])
def test_dependent_launches_back_to_back(M):
    """Each launch adds onto the output of the one before (residual in place), and every second one reads what a plain
    GEMM and a quantizer just wrote: the same bits whether or not the host waits in between, eager and from a graph."""
    rng = np.random.default_rng(M)
    A, B = Operand(rng, True, 1, M, 512), Operand(rng, True, 1, 512, 512)
    alpha = torch.tensor([0.02], device=DEV)
    one = torch.ones(1, device=DEV)
    a, b = A.tensor(), B.tensor()

    def chain(wait):
        x = torch.zeros(M, 512, dtype=torch.bfloat16, device=DEV)
        q = a
        for _ in range(6):
            bsp.nvfp4_gemm(q, b, alpha, activation="silu", residual=x, out=x)
            wait()
            bsp.nvfp4_gemm(q, b, alpha, activation="relu", residual=x, out=x)
            wait()
            y = bsp.nvfp4_gemm(q, b, alpha, out_dtype=torch.bfloat16)
            wait()
            x2 = bsp.nvfp4_gemm(q, b, alpha, activation="gelu", residual=y)
            wait()
            q = bsp.nvfp4_quantize(x2, one)
            wait()
        return x

    want = chain(torch.cuda.synchronize)
    for _ in range(5):
        assert torch.equal(want, chain(lambda: None))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(lambda: None)
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, got)
    assert bsp.device_status() == 0


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", [None, "relu", "gelu", "gelu_tanh", "silu"])
def test_nan_stays_in_its_column(act, gated):
    """One column that is NaN or infinite (through the bias) changes no bit of any other, though two share a reciprocal."""
    rng = np.random.default_rng(33)
    A, B = Operand(rng, True, 1, 40, 128), Operand(rng, True, 1, 256, 128)
    plain = torch.zeros(256, dtype=torch.bfloat16, device=DEV)
    want = bsp.nvfp4_gemm(A.tensor(), B.tensor(), None, None, plain, activation=act, gated=gated)
    assert bool(torch.isfinite(want).all())
    for col in (0, 21, 138, 255):
        for value in ("nan", "inf", "-inf"):
            bias = plain.clone()
            bias[col] = float(value)
            got = bsp.nvfp4_gemm(A.tensor(), B.tensor(), None, None, bias, activation=act, gated=gated)
            at = col // 2 if gated else col
            others = torch.arange(want.shape[1], device=DEV) != at
            assert torch.equal(got[:, others], want[:, others]), (col, value)
            assert value != "nan" or bool(torch.isnan(got[:, at]).all())
