"""The forms that the fused and grouped GEMMs choose by their sizes: CTA pairs, and K split over a cluster.  Each test states
the form that its sizes take and fails if a later rule takes another.  Definition and tolerance as in
tests/test_gpu_fused_gemm.py."""
import ctypes
import functools
import math

import numpy as np
import pytest
import torch

import block_scaled_precision_05_b200 as bsp
from block_scaled_precision_05_b200 import _native as nat
from tests._gpu import DEV, up, up_bf16
from tests.test_gpu_fused_gemm import Operand, bf16_bits, check, reference

pytestmark = pytest.mark.gpu


def plan(fp4, M, N, K, E=0):
    """(CTAs per tile, token tile, CTAs sharing K) of a dense (E = 0) or grouped call on this device."""
    out = (ctypes.c_int32 * 3)()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert nat.lib().bsp_debug_fused_plan(int(not fp4), int(E > 0), max(E, 1), M, N, K, sms, ctypes.addressof(out)) == nat.BSP_OK
    return tuple(out)


@functools.lru_cache(maxsize=3)
def weights(fp4, E, N, K):
    return Operand(np.random.default_rng(N + K), fp4, E, N, K, 0.5)


def dense(fp4, M, N, K, act=None, gated=False, bias=False, residual=False, row=False, dtype=torch.bfloat16, ld=None,
          in_place=False, want=None):
    assert plan(fp4, M, N, K) == want
    rng = np.random.default_rng(M * 7919 + N)
    A, B = Operand(rng, fp4, 1, M, K), weights(fp4, 1, N, K)
    alpha = np.float32(1.3 / math.sqrt(K))
    rs = (0.5 + rng.random(M)).astype(np.float32) if row else None
    bz = bf16_bits(rng, N, scale=0.3) if bias else None
    cols = N // 2 if gated else N
    wide = torch.full((M, ld or cols), 7.0, dtype=dtype, device=DEV)
    out, res, res64 = wide[:, :cols], None, None
    if residual:
        res = out if in_place else torch.empty((M, ld or cols), dtype=dtype, device=DEV)[:, :cols]
        res.copy_(torch.from_numpy(rng.standard_normal((M, cols))).to(dtype))
        res64 = res.double().cpu().numpy()
    kw = dict(alpha=up(np.array([alpha])), bias=None if bz is None else up_bf16(bz), out=out, out_dtype=dtype, activation=act,
              gated=gated, residual=res)
    if fp4:
        kw["row_scale"] = None if rs is None else up(rs)
    assert act is not None or gated or residual  # else the plain GEMM runs
    (bsp.nvfp4_gemm if fp4 else bsp.mxfp8_gemm)(A.tensor(), B.tensor(), **kw)
    assert bsp.device_status() == 0
    ref, tol = reference(A.dec[0], B.dec[0], fp4, alpha, rs, bz, act, gated, res64, dtype)
    check(out, ref, tol, f"M={M} N={N} K={K}")
    assert bool((wide[:, cols:] == 7.0).all()), "columns past D were written"


def grouped(fp4, counts, N, K, act=None, gated=False, bias=False, row=False, dtype=torch.bfloat16, head=0, tail=0, want=None):
    E, M = len(counts), head + sum(counts) + tail
    assert plan(fp4, M, N, K, E) == want
    rng = np.random.default_rng(M + N)
    A, B = Operand(rng, fp4, 1, M, K), weights(fp4, E, N, K)
    alpha = ((0.5 + rng.random(E)) * 1.3 / math.sqrt(K)).astype(np.float32)
    rs = (0.5 + rng.random(M)).astype(np.float32) if row else None
    bz = bf16_bits(rng, E, N, scale=0.3) if bias else None
    off = (head + np.concatenate(([0], np.cumsum(counts)))).astype(np.int32)
    out = torch.full((M, N // 2 if gated else N), 7.0, dtype=dtype, device=DEV)
    kw = dict(alpha=up(alpha), bias=None if bz is None else up_bf16(bz), out=out, out_dtype=dtype, activation=act, gated=gated)
    if fp4:
        kw["row_scale"] = None if rs is None else up(rs)
    (bsp.nvfp4_grouped_gemm if fp4 else bsp.mxfp8_grouped_gemm)(A.tensor(), B.experts(), up(off), **kw)
    assert bsp.device_status() == 0
    for e in range(E):
        i, j = off[e], off[e + 1]
        if i < j:
            ref, tol = reference(A.dec[0][i:j], B.dec[e], fp4, alpha[e], None if rs is None else rs[i:j],
                                 None if bz is None else bz[e], act, gated, None, dtype)
            check(out[i:j], ref, tol, f"expert {e} rows {i}..{j}")
    assert bool((torch.cat((out[:head], out[M - tail:] if tail else out[:0])) == 7.0).all()), "rows outside every expert were written"


# --------------------------------------------------------------------------- CTA pairs
PAIR = (2, 256, 1)
BF16, F32 = torch.bfloat16, torch.float32


# K steps of 128 bytes: 2 (one ring, part used), 9 (the ring of 5 wraps, the last step ends inside), 17; weights that end
# inside a panel, and inside a pair's first half
@pytest.mark.parametrize("fp4,M,N,K,act,gated,bias,residual,row,dtype", [
    (True, 600, 3840, 2080, "silu", True, True, True, True, BF16),
    (True, 777, 3728, 2080, "gelu_tanh", False, True, True, True, F32),
    (True, 600, 3840, 2080, None, False, False, True, False, BF16),
    (True, 1030, 2576, 4352, "relu", False, True, False, True, BF16),
    (True, 2000, 3600, 288, "gelu", False, True, False, True, F32),
    (True, 2000, 3600, 288, "silu", True, False, True, False, F32),
    (True, 1900, 3792, 512, "gelu_tanh", True, True, False, False, F32),
    (False, 600, 3840, 1056, "silu", True, True, True, False, F32),
    (False, 777, 3728, 1056, "gelu_tanh", False, True, True, False, BF16),
    (False, 1030, 2576, 2176, "gelu", False, True, False, False, F32),
    (False, 2000, 3600, 224, "relu", True, True, True, False, BF16),
])
def test_dense_in_pairs(fp4, M, N, K, act, gated, bias, residual, row, dtype):
    dense(fp4, M, N, K, act, gated, bias, residual, row, dtype, want=PAIR)


@pytest.mark.parametrize("M", [1, 16, 31, 32, 33, 64, 65, 96, 97, 128, 129, 160, 161, 192, 223, 224, 225, 256])
def test_every_pair_width(M):
    """Every token width of a pair's MMA (a multiple of 32), with a whole and a part-filled last box of D."""
    N = 18952 if M <= 128 else 9480  # one token tile: weight panels enough for the pair form
    dense(True, M, N, 2080, None, False, False, True, True, want=PAIR)
    dense(False, M, N, 1056, "relu", False, False, M % 2 == 0, False, F32, want=PAIR)


@pytest.mark.parametrize("in_place", [False, True])
def test_pairs_with_strided_output_and_residual(in_place):
    dense(True, 600, 3728, 2080, "gelu_tanh", False, True, True, True, ld=3760, in_place=in_place, want=PAIR)
    dense(False, 600, 3728, 1056, "silu", True, True, True, False, F32, ld=1880, in_place=in_place, want=PAIR)


@pytest.mark.parametrize("fp4,counts,N,K,act,gated,bias,row,dtype,head,tail", [
    (True, [31, 0, 257, 400, 512], 5264, 1312, "silu", True, True, True, BF16, 0, 0),
    (True, [31, 0, 257, 400, 512], 5264, 1312, "gelu", False, True, True, F32, 33, 40),
    (True, [1, 255, 256, 700], 5392, 1312, None, False, False, False, BF16, 64, 64),
    (True, [500, 0, 1000], 4880, 288, "gelu_tanh", True, True, False, F32, 7, 0),
    (False, [31, 0, 257, 400, 512], 5264, 672, "silu", True, True, False, F32, 97, 5),
    (False, [1, 255, 256, 700], 5520, 672, "relu", False, True, False, BF16, 0, 1),
    (False, [500, 0, 1000], 4880, 160, None, True, False, False, BF16, 3, 0),
])
def test_grouped_in_pairs(fp4, counts, N, K, act, gated, bias, row, dtype, head, tail):
    grouped(fp4, counts, N, K, act, gated, bias, row, dtype, head, tail, want=PAIR)


@pytest.mark.parametrize("head", [0, 1, 31, 32, 63, 64, 96, 100, 127])
def test_pairs_scale_shift(head):
    """An expert's first row at every word and line of a scale band, for tiles of two bands' words and of one."""
    grouped(True, [250, 131, 90, 300], 8080, 1312, head=head, tail=1, want=PAIR)
    grouped(False, [250, 131, 90, 300], 8080, 672, head=head, tail=1, want=PAIR)


@pytest.mark.parametrize("act", [None, "silu"])
def test_pairs_keep_nan_and_infinity_in_place(act):
    """Row scales, bias and residual that are infinite or NaN change no bit of any other row and column."""
    M, N, K = 600, 3840, 2080
    assert plan(True, M, N, K) == PAIR
    A, B = Operand(np.random.default_rng(1), True, 1, M, K).tensor(), weights(True, 1, N, K).tensor()
    rs, bias = torch.ones(M, device=DEV), torch.zeros(N, dtype=BF16, device=DEV)
    res = torch.zeros(M, N, dtype=BF16, device=DEV)
    want = bsp.nvfp4_gemm(A, B, None, rs, bias, activation=act, residual=res)
    assert bool(torch.isfinite(want).all())
    rs[3], rs[300], rs[M - 1] = float("inf"), float("nan"), float("-inf")
    bias[5], bias[N - 1] = float("nan"), float("inf")
    res[7, 9], res[290, 1000] = float("-inf"), float("nan")
    got = bsp.nvfp4_gemm(A, B, None, rs, bias, activation=act, residual=res)
    assert bsp.device_status() == 0
    hit = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    hit[[3, 300, M - 1]] = True
    hit[:, [5, N - 1]] = True
    hit[7, 9] = hit[290, 1000] = True
    assert torch.equal(got[~hit], want[~hit])
    assert bool(torch.isnan(got[300]).all()) and bool(torch.isnan(got[:, 5]).all()) and bool(torch.isnan(got[290, 1000]))
    assert float(got[7, 9]) == float("-inf")


def test_pairs_repeat_their_bits():
    M, N, K = 1200, 5264, 1312
    assert plan(True, M, N, K, 5) == PAIR
    A, B = Operand(np.random.default_rng(2), True, 1, M, K).tensor(), weights(True, 5, N, K).experts()
    off = torch.tensor([0, 31, 31, 288, 688, 1200], dtype=torch.int32, device=DEV)
    first = bsp.nvfp4_grouped_gemm(A, B, off, activation="gelu", gated=True)
    for _ in range(50):
        assert torch.equal(first, bsp.nvfp4_grouped_gemm(A, B, off, activation="gelu", gated=True))
    assert bsp.device_status() == 0


def test_pairs_one_expert_is_the_dense_gemm():
    M, N, K = 700, 13824, 2080
    assert plan(True, M, N, K) == plan(True, M, N, K, 1) == PAIR
    A, B = Operand(np.random.default_rng(3), True, 1, M, K), weights(True, 1, N, K)
    off = torch.tensor([0, M], dtype=torch.int32, device=DEV)
    alpha = torch.tensor([0.02], device=DEV)
    g = bsp.nvfp4_grouped_gemm(A.tensor(), B.experts(), off, alpha, activation="silu", gated=True)
    assert torch.equal(g, bsp.nvfp4_gemm(A.tensor(), B.tensor(), alpha, activation="silu", gated=True))


def test_pairs_launched_back_to_back():
    """Each launch adds onto the output of the one before in place, beside plain GEMMs and quantizers: the same bits whether
    or not the host waits in between, eager and from a graph."""
    M, N = 14300, 512
    assert plan(True, M, N, N) == PAIR
    a, b = Operand(np.random.default_rng(4), True, 1, M, N).tensor(), weights(True, 1, N, N).tensor()
    alpha, one = torch.tensor([0.02], device=DEV), torch.ones(1, device=DEV)

    def chain(wait):
        x, q = torch.zeros(M, N, dtype=BF16, device=DEV), a
        for _ in range(4):
            bsp.nvfp4_gemm(q, b, alpha, activation="silu", residual=x, out=x)
            wait()
            bsp.nvfp4_gemm(q, b, alpha, activation="relu", residual=x, out=x)
            wait()
            y = bsp.nvfp4_gemm(q, b, alpha)
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


# --------------------------------------------------------------------------- K split over a cluster
# 2, 3 and 4 CTAs; one box of D a warp (up to 64 rows) and two, one token tile and several
@pytest.mark.parametrize("fp4,M,N,K,want", [
    (True, 1, 136, 8192, (1, 32, 2)), (True, 40, 264, 12288, (1, 64, 3)), (True, 65, 136, 12288, (1, 128, 3)),
    (True, 97, 264, 16384, (1, 128, 4)), (True, 128, 520, 8192, (1, 128, 2)), (True, 200, 264, 16384, (1, 128, 4)),
    (True, 300, 136, 12320, (1, 128, 3)), (True, 17, 520, 16448, (1, 32, 4)),
    (False, 5, 264, 8192, (1, 32, 4)), (False, 65, 264, 8192, (1, 128, 4)), (False, 128, 136, 6176, (1, 128, 3)),
    (False, 200, 520, 4096, (1, 128, 2)), (False, 97, 4736, 8192, (1, 128, 4)),
])
def test_split_forms(fp4, M, N, K, want):
    """Against the definition with bias, residual and gate in both output types: the residual's next box is loaded past
    boxes that another CTA of the cluster finishes."""
    dense(fp4, M, N, K, "silu", False, True, True, fp4, BF16, want=want)
    dense(fp4, M, N, K, "gelu_tanh", False, True, True, fp4, F32, want=want)
    if N % 16 == 0:
        dense(fp4, M, N, K, "relu", True, False, True, False, BF16, want=want)
    dense(fp4, M, N, K, None, False, False, True, False, BF16, in_place=True, ld=N + 24, want=want)


@pytest.mark.parametrize("M,N,K,split", [(128, 136, 16384, 4), (200, 136, 12288, 3)])
def test_split_repeats_its_bits(M, N, K, split):
    assert plan(True, M, N, K) == (1, 128, split)
    A, B = Operand(np.random.default_rng(5), True, 1, M, K).tensor(), weights(True, 1, N, K).tensor()
    res = torch.randn(M, N, device=DEV).bfloat16()
    first = bsp.nvfp4_gemm(A, B, activation="relu", residual=res)
    for _ in range(30):
        assert torch.equal(first, bsp.nvfp4_gemm(A, B, activation="relu", residual=res))
    assert bsp.device_status() == 0


def test_two_graphs_of_split_and_paired_calls():
    """Two captured graphs of the same calls (one split over a cluster, one in pairs) replayed on two streams at a time."""
    assert plan(True, 64, 264, 16384) == (1, 64, 4) and plan(True, 1200, 5264, 1312, 5) == PAIR
    A, B = Operand(np.random.default_rng(6), True, 1, 64, 16384).tensor(), weights(True, 1, 264, 16384).tensor()
    C, D = Operand(np.random.default_rng(7), True, 1, 1200, 1312).tensor(), weights(True, 5, 5264, 1312).experts()
    off = torch.tensor([0, 31, 31, 288, 688, 1200], dtype=torch.int32, device=DEV)
    run = lambda: (bsp.nvfp4_gemm(A, B, activation="gelu"), bsp.nvfp4_grouped_gemm(C, D, off, activation="silu"))  # noqa: E731
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
