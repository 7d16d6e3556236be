"""Fused and grouped GEMMs, host side (no GPU): refusals of the C ABI before any device call, the binding's checks that
need no device, and the order of a gated pair's rows."""
import os
import re

import pytest
import torch

import block_scaled_precision_05_b200 as bsp
from block_scaled_precision_05_b200 import _native as nat
from block_scaled_precision_05_b200 import api

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "bsp.h")
P, ODD, BYTE = 0x10000, 0x10008, 0x10001  # never dereferenced: validation fails first


def call(fp4, **kw):
    d = dict(A=P, sfA=P, B=P, sfB=P, offsets=0, E=1, M=4, N=32, K=64, alpha=0, row_scale=0, bias=0, act=0, gated=0, residual=0,
             ld_res=0, D=P, dtype=0, ld=None)
    d.update(kw)
    if d["ld"] is None:
        d["ld"] = d["N"] // 2 if d["gated"] else d["N"]
    fn = nat.lib().nvfp4_gemm_fused if fp4 else nat.lib().mxfp8_gemm_fused
    return fn(nat.pack_fused_desc(*d.values()), None)


def fused(fp4=True, **kw):
    return call(fp4, **kw)


def grouped(fp4=True, **kw):
    return call(fp4, **{"offsets": P, "E": 2, **kw})


BAD = [dict(K=48), dict(K=0), dict(M=-1), dict(N=-8), dict(N=12), dict(N=24, gated=1), dict(act=5), dict(act=-1),
       dict(gated=2), dict(dtype=2), dict(ld=16), dict(D=0), dict(M=1 << 31), dict(N=1 << 31)]
MISALIGNED = [dict(D=ODD), dict(ld=36), dict(bias=ODD), dict(alpha=BYTE)]


@pytest.mark.parametrize("fp4", [True, False])
def test_c_abi_refuses(fp4):
    for bad in BAD + [dict(A=0), dict(sfA=0), dict(B=0), dict(sfB=0), dict(residual=P, ld_res=16), dict(E=2), dict(E=0)]:
        assert fused(fp4, **bad) == nat.BSP_ERR_INVALID_ARG, bad
    for bad in MISALIGNED + [dict(A=ODD), dict(sfB=ODD), dict(residual=ODD, ld_res=32), dict(residual=P, ld_res=36)]:
        assert fused(fp4, **bad) == nat.BSP_ERR_ALIGNMENT, bad
    for bad in BAD + [dict(offsets=0), dict(E=0), dict(E=-1), dict(E=nat.BSP_MAX_EXPERTS + 1), dict(residual=P, ld_res=32)]:
        assert grouped(fp4, **bad) == nat.BSP_ERR_INVALID_ARG, bad
    for bad in MISALIGNED + [dict(offsets=BYTE)]:
        assert grouped(fp4, **bad) == nat.BSP_ERR_ALIGNMENT, bad
    if fp4:
        assert fused(row_scale=BYTE) == nat.BSP_ERR_ALIGNMENT and grouped(row_scale=BYTE) == nat.BSP_ERR_ALIGNMENT
    else:
        assert fused(False, row_scale=P) == nat.BSP_ERR_INVALID_ARG  # MXFP8 has none
    assert (nat.lib().nvfp4_gemm_fused if fp4 else nat.lib().mxfp8_gemm_fused)(None, None) == nat.BSP_ERR_INVALID_ARG


@pytest.mark.parametrize("fp4", [True, False])
def test_empty_is_a_no_op(fp4):
    assert fused(fp4, M=0) == nat.BSP_OK and fused(fp4, N=0) == nat.BSP_OK
    assert grouped(fp4, M=0) == nat.BSP_OK and grouped(fp4, N=0) == nat.BSP_OK


def test_descriptor_layout():
    """The packed bytes are the header's struct: nineteen 8-byte fields in declaration order."""
    src = open(HEADER).read()
    body = re.search(r"typedef struct \{([^}]*)\} bsp_fused_gemm_desc;", src).group(1)
    body = re.sub(r"/\*.*?\*/", "", body)
    names = [n.strip(" *") for line in body.split(";") for n in re.sub(r"^\s*(const )?\w+ ", "", line.strip()).split(",")
             if n.strip(" *")]
    assert names == ["A", "sfA", "B", "sfB", "offsets", "E", "M", "N", "K", "alpha", "row_scale", "bias", "activation",
                     "gated", "residual", "ld_residual", "D", "d_dtype", "ld_d"]
    assert re.findall(r"\b(int|float|uint32_t|int32_t)\s+\w+[,;]", body) == []  # by value: int64_t only
    assert len(nat.pack_fused_desc(*range(19))) == 19 * 8


def test_header_constants():
    src = open(HEADER).read()
    assert f"#define BSP_MAX_EXPERTS {nat.BSP_MAX_EXPERTS}" in src
    for name in ("NONE", "RELU", "GELU", "GELU_TANH", "SILU"):
        assert f"BSP_ACT_{name} = {getattr(nat, 'BSP_ACT_' + name)}" in src
    assert api.ACTIVATIONS == {None: 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


def test_cpu_tensors_are_refused():
    a = bsp.NVFP4Tensor(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 64)
    b = bsp.NVFP4Tensor(torch.zeros(32, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 64)
    e = bsp.NVFP4Experts(torch.zeros(2, 32, 32, dtype=torch.uint8), torch.zeros(2, 512, dtype=torch.uint8), 64)
    m = bsp.MXFP8Tensor(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 64)
    n = bsp.MXFP8Experts(torch.zeros(2, 32, 64, dtype=torch.uint8), torch.zeros(2, 512, dtype=torch.uint8), 64)
    off = torch.zeros(3, dtype=torch.int32)
    w = torch.zeros(2, 32, 64, dtype=torch.bfloat16)
    for call in (lambda: bsp.nvfp4_gemm(a, b, activation="silu"), lambda: bsp.nvfp4_grouped_gemm(a, e, off),
                 lambda: bsp.mxfp8_grouped_gemm(m, n, off), lambda: bsp.nvfp4_quantize_experts(w),
                 lambda: bsp.mxfp8_quantize_experts(w), lambda: bsp.NVFP4GroupedLinear(w), lambda: bsp.MXFP8GroupedLinear(w)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_operands_that_contradict_their_sizes():
    good = dict(codes=torch.zeros(4, 32, dtype=torch.uint8), sf=torch.zeros(512, dtype=torch.uint8), K=64)
    b = bsp.NVFP4Tensor(torch.zeros(32, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 64)
    for change in (dict(K=128), dict(codes=torch.zeros(4, 16, dtype=torch.uint8)), dict(codes=torch.zeros(4, 32)),
                   dict(codes=torch.zeros(4, 64, dtype=torch.uint8)[:, ::2]), dict(sf=torch.zeros(511, dtype=torch.uint8)),
                   dict(sf=torch.zeros(512)), dict(sf_layout="8x4")):
        with pytest.raises(ValueError):
            bsp.nvfp4_gemm(bsp.NVFP4Tensor(**{**good, **change}), b, activation="relu")
    with pytest.raises(ValueError, match="activation"):
        bsp.nvfp4_gemm(bsp.NVFP4Tensor(**good), b, activation="swish")
    e = bsp.NVFP4Experts(torch.zeros(2, 32, 32, dtype=torch.uint8), torch.zeros(2, 512, dtype=torch.uint8), 64)
    for off in (None, torch.zeros(2, dtype=torch.int32), torch.zeros(3), torch.zeros(3, dtype=torch.int64),
                torch.zeros(6, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError, match="offsets"):
            bsp.nvfp4_grouped_gemm(bsp.NVFP4Tensor(**good), e, off)
    big = bsp.NVFP4Experts(torch.zeros(nat.BSP_MAX_EXPERTS + 1, 8, 32, dtype=torch.uint8), torch.zeros(1, dtype=torch.uint8), 64)
    with pytest.raises(ValueError, match="experts"):
        bsp.nvfp4_grouped_gemm(bsp.NVFP4Tensor(**good), big, torch.zeros(2, dtype=torch.int32))


def test_interleave_gated():
    g, u = torch.arange(6).view(3, 2), torch.arange(6).view(3, 2) + 10
    w = bsp.interleave_gated(g, u)
    assert w.shape == (6, 2) and torch.equal(w[0::2], g) and torch.equal(w[1::2], u)
    w = bsp.interleave_gated(g[None].expand(4, 3, 2), u[None].expand(4, 3, 2))
    assert w.shape == (4, 6, 2) and torch.equal(w[3, 1::2], u)
    b = bsp.interleave_gated(g[:, 0], u[:, 0], dim=-1)
    assert b.tolist() == [0, 10, 2, 12, 4, 14]
    with pytest.raises(ValueError):
        bsp.interleave_gated(g, u[:2])


def test_grouped_layer_refuses_row_scales_it_would_leave_out():
    """A layer with one activation scale has no use for the row scales of a per-token input: its result would lack them."""
    layer = bsp.NVFP4GroupedLinear.__new__(bsp.NVFP4GroupedLinear)
    layer.weight = bsp.NVFP4Experts(torch.zeros(2, 32, 32, dtype=torch.uint8), torch.zeros(2, 512, dtype=torch.uint8), 64)
    layer.per_token, layer.activation, layer.gated, layer.alpha, layer.bias = False, None, False, torch.ones(2), None
    off = torch.tensor([0, 1, 4], dtype=torch.int32)
    xq = bsp.NVFP4Tensor(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 64, torch.ones(4), torch.ones(4))
    with pytest.raises(ValueError, match="each row"):
        layer(None, off, pre_quantized=xq)
    layer.per_token = True
    with pytest.raises(ValueError, match="CUDA"):  # taken as far as the binding's refusal of CPU tensors
        layer(None, off, pre_quantized=xq)


class _Elsewhere:
    """Stands for a tensor on cuda:1 while cuda:0 is current: what the quantizers ask of one, over CPU memory."""

    def __init__(self, t, dtype=None):
        self.t, self.dtype, self.is_cuda, self.device = t, dtype or t.dtype, True, torch.device("cuda", 1)
        self.shape = t.shape

    def reshape(self, *s):
        return _Elsewhere(self.t.reshape(*s), self.dtype)

    def stride(self, i):
        return self.t.stride(i)

    def data_ptr(self):
        return self.t.data_ptr()

    def is_floating_point(self):
        return True


def test_a_grouped_layers_tokens_on_another_device(monkeypatch):
    """The layers quantize their tokens on the tokens' device and its stream, where the product runs too, not on the
    current device."""
    calls = []
    current = [0]

    class Device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            self.was, current[0] = current[0], self.d.index

        def __exit__(self, *e):
            current[0] = self.was

    class Lib:
        def __getattr__(self, name):
            return (lambda *a: calls.append((name, current[0], a[-1])) or 0) if "quantize" in name else (lambda *a: 512)

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 100 + d, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(nat, "lib", lambda: Lib())
    x = _Elsewhere(torch.zeros(4, 64, dtype=torch.bfloat16))
    buf = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    api.nvfp4_quantize(x, _Elsewhere(torch.ones(1)), out=api.NVFP4Tensor(buf(4, 32), buf(512), 64))
    api.mxfp8_quantize(x, out=api.MXFP8Tensor(buf(4, 64), buf(512), 64))
    assert calls == [("nvfp4_quantize_ex", 1, 101), ("mxfp8_quantize", 1, 101)] and current == [0]


def test_plan_of_the_sizes():
    """The form a call takes, at both sides of each border of the rules (148 SMs)."""
    import ctypes

    def plan(mxfp8, E, M, N, K, sms=148):
        out = (ctypes.c_int32 * 3)()
        assert nat.lib().bsp_debug_fused_plan(mxfp8, int(E > 0), max(E, 1), M, N, K, sms, ctypes.addressof(out)) == nat.BSP_OK
        return tuple(out)

    pair = (2, 256, 1)
    # dense: pairs once the 128 x 128 tiles exceed one wave, three waves up to 8 steps of 128 bytes
    assert plan(0, 0, 128, 148 * 128, 2080) == (1, 128, 1) and plan(0, 0, 128, 148 * 128 + 8, 2080) == pair
    assert plan(0, 0, 1, 148 * 128 + 8, 2080) == pair and plan(0, 0, 1, 148 * 128 + 8, 2048)[0] == 1
    assert plan(0, 0, 128, 444 * 128, 2048) == (1, 128, 1) and plan(0, 0, 129, 222 * 128 + 8, 2048) == pair
    assert plan(1, 0, 128, 148 * 128 + 8, 1056) == pair and plan(1, 0, 128, 148 * 128 + 8, 1024) == (1, 128, 1)
    # token tiles of single CTAs
    assert [plan(0, 0, m, 1024, 2080)[1] for m in (1, 32, 33, 64, 65, 128, 500)] == [32, 32, 64, 64, 128, 128, 128]
    assert plan(0, 0, 256, 1536, 1536) == (1, 32, 1) and plan(0, 0, 512, 1536, 1536) == (1, 64, 1)
    # split K: 16 steps a CTA at least, 4 CTAs at most, no more than the SMs hold
    assert [plan(0, 0, 1, 1024, 256 * s)[2] for s in (31, 32, 47, 48, 63, 64, 200)] == [1, 2, 2, 3, 3, 4, 4]
    assert [plan(0, 0, 1, 128 * p, 256 * 64)[2] for p in (37, 38, 49, 50, 74, 75)] == [4, 3, 3, 2, 2, 1]
    # experts: pairs above a mean of 64 rows (160 up to 4 steps) and about 3.5 waves; never split
    assert plan(0, 4, 256, 128 * 200, 1312) == (1, 128, 1) and plan(0, 4, 257, 128 * 200, 1312) == pair
    assert plan(0, 4, 640, 128 * 200, 1024) == (1, 128, 1) and plan(0, 4, 641, 128 * 200, 1024) == pair
    assert plan(0, 8, 1152, 128 * 39, 1312) == (1, 128, 1) and plan(0, 8, 1152, 128 * 40, 1312) == pair
    assert [plan(0, 4, 4 * m, 1024, 16384)[1:] for m in (1, 8, 9, 24, 25, 64)] == [(32, 1), (32, 1), (64, 1), (64, 1), (128, 1), (128, 1)]
    plan_of = nat.lib().bsp_debug_fused_plan
    buf = ctypes.addressof((ctypes.c_int32 * 3)())
    for bad in ((0, 0, 1, 0, 8, 32, 148, buf), (0, 0, 1, 1, 0, 32, 148, buf), (0, 0, 1, 1, 8, 48, 148, buf),
                (0, 0, 0, 1, 8, 32, 148, buf), (0, 0, 1, 1, 8, 32, 0, buf), (0, 0, 1, 1, 8, 32, 148, None)):
        assert plan_of(*bad) == nat.BSP_ERR_INVALID_ARG
