"""Stacked experts' weights and the grouped layers against the oracle: every expert's codes, scales and global scale bit for
bit, and the layers' outputs against the definition on operands that the oracle alone quantized."""
import numpy as np
import pytest
import torch

import block_scaled_precision_05_b200 as bsp
import oracle
from block_scaled_precision_05_b200 import api
from tests._gpu import down, up, up_bf16
from tests.test_gpu_fused_gemm import bf16_bits, check, reference

pytestmark = pytest.mark.gpu

# experts of different sizes: their scales differ, so that one taken for another shows; the last is all zeros
STD = (0.02, 3.0, 0.3, 0.0)


def stacked(rng, N, K, f16=False):
    """(device weights [E, N, K], their 16-bit patterns)."""
    w = np.stack([rng.standard_normal((N, K)).astype(np.float32) * s for s in STD])
    if f16:
        h = w.astype(np.float16)
        return up(h), h.view(np.uint16)
    bits = np.stack([oracle.bf16_round(x).astype(np.uint16) for x in w])
    return up_bf16(bits), bits


def oracle_expert(bits, f16, fmax):
    gs = oracle.nvfp4_global_scale(oracle.amax_f16(bits) if f16 else oracle.amax_bf16(bits), fmax)
    return (gs, *oracle.nvfp4_quantize(bits, gs, fmt="f16" if f16 else "bf16"))


@pytest.mark.parametrize("N,K", [(8, 32), (40, 96), (136, 64), (264, 1056)])
@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("fmax", [api.FP8_FP4_MAX, api.FP8_FP4_MAX_4OVER6])
def test_nvfp4_experts_are_the_oracles(N, K, f16, fmax):
    w, bits = stacked(np.random.default_rng(N + K), N, K, f16)
    for form in (w, w.transpose(1, 2).contiguous().transpose(1, 2)):  # the same weights in another order of strides
        q, gs, inv = bsp.nvfp4_quantize_experts(form, fmax)
        assert (q.experts, q.rows, q.K) == (len(STD), N, K) and gs.shape == inv.shape == (len(STD),)
        for e in range(len(STD)):
            g, codes, sf = oracle_expert(bits[e], f16, fmax)
            assert np.array_equal(down(q.codes[e]), codes), e
            assert np.array_equal(down(q.sf[e]).reshape(-1), np.asarray(sf, np.uint8).reshape(-1)), e
            assert down(gs)[e] == np.float32(g) and down(inv)[e] == np.float32(1) / np.float32(g), e
    assert bsp.device_status() == 0


@pytest.mark.parametrize("N,K", [(8, 32), (40, 96), (264, 1056)])
def test_mxfp8_experts_are_the_oracles(N, K):
    w, bits = stacked(np.random.default_rng(N + K), N, K)
    for form in (w, w.transpose(1, 2).contiguous().transpose(1, 2)):
        q = bsp.mxfp8_quantize_experts(form)
        assert (q.experts, q.rows, q.K) == (len(STD), N, K)
        for e in range(len(STD)):
            codes, sf = oracle.mxfp8_quantize(bits[e])
            assert np.array_equal(down(q.q[e]), codes), e
            assert np.array_equal(down(q.sf[e]).reshape(-1), np.asarray(sf, np.uint8).reshape(-1)), e
    assert bsp.device_status() == 0


COUNTS = (17, 0, 70, 5)
OFF = np.concatenate(([0], np.cumsum(COUNTS))).astype(np.int32)


def expected(e, a, dec, alpha, rs, bias, act, gated, dtype, fp4):
    i, j = OFF[e], OFF[e + 1]
    return reference(a[i:j], dec, fp4, alpha, None if rs is None else rs[i:j], None if bias is None else bias[e], act, gated,
                     None, dtype)


@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("act,gated", [(None, False), ("silu", True)])
def test_nvfp4_layer_from_the_oracles_operands(per_token, f16, four, act, gated):
    """Weights and tokens in both input types, bias, 4over6 scales, one activation scale or one a token; x, its quantized
    form and an output of the caller's give the same bits."""
    rng = np.random.default_rng(1)
    N, K, M = 48, 96, int(OFF[-1]) + 3
    w, bits = stacked(rng, N, K, f16)
    fmt = "f16" if f16 else "bf16"
    x = rng.standard_normal((M, K)).astype(np.float32)
    xb = x.astype(np.float16).view(np.uint16) if f16 else oracle.bf16_round(x).astype(np.uint16)
    xt = up(xb.view(np.float16)) if f16 else up_bf16(xb)
    bias = bf16_bits(rng, len(STD), N, scale=0.3)
    layer = bsp.NVFP4GroupedLinear(w, up_bf16(bias), per_token, four, act, gated)
    off = up(OFF)
    got = layer(xt, off)
    f32 = layer(xt, off, out_dtype=torch.float32)
    out = torch.full_like(got, 7.0)
    assert layer(None, off, pre_quantized=layer.quantize_input(xt), out=out) is out
    assert bsp.device_status() == 0
    assert torch.equal(out[:OFF[-1]], got[:OFF[-1]]) and bool((out[OFF[-1]:] == 7.0).all())
    if per_token:
        gs, rs = oracle.row_global_scales(xb, fmt)
        codes, sf = oracle.nvfp4_quantize(xb, gs, per_row=True, fmt=fmt)
    else:
        codes, sf = oracle.nvfp4_quantize(xb, 1.0, fmt=fmt)
        rs = None
    a = oracle.nvfp4_dequantize(codes, sf, K)
    for e in range(len(STD)):
        if COUNTS[e]:
            g, c, s = oracle_expert(bits[e], f16, api.FP8_FP4_MAX_4OVER6 if four else api.FP8_FP4_MAX)
            for y in (got, f32):
                ref, tol = expected(e, a, oracle.nvfp4_dequantize(c, s, K), np.float32(1) / np.float32(g), rs, bias, act, gated,
                                    y.dtype, True)
                check(y[OFF[e]:OFF[e + 1]], ref, tol, f"expert {e}")


@pytest.mark.parametrize("act,gated", [(None, False), ("gelu_tanh", True)])
def test_mxfp8_layer_from_the_oracles_operands(act, gated):
    rng = np.random.default_rng(2)
    N, K, M = 48, 96, int(OFF[-1]) + 3
    w, bits = stacked(rng, N, K)
    xb, bias = bf16_bits(rng, M, K), bf16_bits(rng, len(STD), N, scale=0.3)
    layer = bsp.MXFP8GroupedLinear(w, up_bf16(bias), act, gated)
    off = up(OFF)
    got = layer(up_bf16(xb), off)
    out = torch.full_like(got, 7.0)
    assert layer(None, off, pre_quantized=bsp.mxfp8_quantize(up_bf16(xb)), out=out) is out
    assert bsp.device_status() == 0
    assert torch.equal(out[:OFF[-1]], got[:OFF[-1]]) and bool((out[OFF[-1]:] == 7.0).all())
    c, s = oracle.mxfp8_quantize(xb)
    a = oracle.mxfp8_dequantize(c, s, K)
    for e in range(len(STD)):
        if COUNTS[e]:
            ref, tol = expected(e, a, oracle.mxfp8_dequantize(*oracle.mxfp8_quantize(bits[e]), K), 1.0, None, bias, act, gated,
                                got.dtype, False)
            check(got[OFF[e]:OFF[e + 1]], ref, tol, f"expert {e}")
