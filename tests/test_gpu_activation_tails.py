"""The activations of the fused epilogues over their whole tails, in fp32 and through a gate, against their formulas in 64 bits.

Tolerance, relative to act(y): (|s| + 6) 2^-22 for the approximated exponential 2^s and reciprocal, 6e-7 for the fitted tail of
gelu, and u32 = 2^-24 for each rounding; the tail ends where 2^s drops below the smallest normal number, 2^-126: what is lost
there is at most |y| 2^-126 < 1.1e-36 (s = -126 at y = -87.4 for silu, -10.2 for gelu_tanh, -13.3 for gelu)."""
import numpy as np
import pytest
import torch

import block_scaled_precision_05_b200 as bsp
from tests._gpu import DEV
from tests.test_gpu_fused_gemm import Operand, act64

pytestmark = pytest.mark.gpu

U32, END = 2.0 ** -24, 1.1e-36


def operands(n):
    rng = np.random.default_rng(0)
    return Operand(rng, True, 1, 2, 32).tensor(), Operand(rng, True, 1, n, 32).tensor(), torch.zeros(1, device=DEV)


def values():
    """Every bf16 number of magnitude 2^-6 to 2^7 of either sign, and far ones: y itself, through the bias (alpha is 0)."""
    mag = torch.arange(0x3C80, 0x4300, dtype=torch.int16).view(torch.bfloat16)
    far = torch.tensor([0.0, 1e-30, 200.0, 1e4, 1e19, 3e38, float("inf")], dtype=torch.bfloat16)
    y = torch.cat((mag, far))
    y = torch.cat((y, -y))
    return y[: y.numel() // 8 * 8].to(DEV)


def expected(y, act):
    with np.errstate(invalid="ignore", over="ignore"):
        want, rel = act64(y, act)
    want = np.where(y == -np.inf, 0.0, np.where(y == np.inf, np.inf, want))  # the limits
    with np.errstate(invalid="ignore"):
        tol = np.where(np.isfinite(want), rel * np.abs(want), 0.0) + END
        if act == "gelu":  # for y > 0 the relative error falls on y Q(y) and the rounding on the result
            tol = tol + np.where((y > 0) & np.isfinite(y), (2 * U32 + 6e-7) * y, 0.0)
        return want, tol + np.where(np.isfinite(want), 2 * U32 * np.abs(want), 0.0)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_tails(act):
    bias = values()
    A, B, zero = operands(bias.numel())
    got = bsp.nvfp4_gemm(A, B, zero, None, bias, out_dtype=torch.float32, activation=act)
    assert bsp.device_status() == 0
    got, y = got.double().cpu().numpy(), bias.double().cpu().numpy()
    want, tol = expected(y, act)
    inf = ~np.isfinite(want)
    assert np.array_equal(got[:, inf], np.broadcast_to(want[inf], got[:, inf].shape))
    bad = ~(np.abs(got - want) <= tol)[:, ~inf]
    assert not bad.any(), [(y[~inf][j], got[0, ~inf][j], want[~inf][j]) for j in np.argwhere(bad[0])[:8, 0]]


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_tails_through_a_gate(act):
    """act(y) times 2^60: the tail of the gate in bf16, where what a bound of y would leave of it shows."""
    gate = values()
    gate = gate[torch.isfinite(gate) & (gate.abs() < 1e4)]
    gate = gate[: gate.numel() // 8 * 8]
    up = torch.full_like(gate, 2.0 ** 60)
    bias = bsp.interleave_gated(gate, up, dim=-1)
    A, B, zero = operands(bias.numel())
    got = bsp.nvfp4_gemm(A, B, zero, None, bias, activation=act, gated=True)
    assert bsp.device_status() == 0
    y = gate.double().cpu().numpy()
    want, tol = expected(y, act)
    want, tol = want * 2.0 ** 60, tol * 2.0 ** 60
    err = np.abs(got.double().cpu().numpy() - want)
    bad = ~(err <= tol + 2.0 ** -8 * (np.abs(want) + tol))
    assert not bad.any(), [(y[j], float(got[0, j]), want[j]) for j in np.argwhere(bad[0])[:8, 0]]
