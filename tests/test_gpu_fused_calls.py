"""What a program meets around the fused and grouped GEMMs: errors of the allocation."""
import pytest
import torch

import block_scaled_precision_05_b200 as bsp

pytestmark = pytest.mark.gpu


def test_out_of_memory_is_torchs_own_error():
    """An output that does not fit raises torch.OutOfMemoryError, as the plain GEMM's does (a caller that catches it to free
    memory and try again), and nothing is launched."""
    M, N, K = 1 << 17, 8192, 32
    a = bsp.MXFP8Tensor(torch.zeros(M, K, dtype=torch.uint8, device="cuda"),
                        torch.full((bsp.mxfp8_sf_bytes(M, K),), 127, dtype=torch.uint8, device="cuda"), K)
    b = bsp.MXFP8Tensor(torch.zeros(N, K, dtype=torch.uint8, device="cuda"),
                        torch.full((bsp.mxfp8_sf_bytes(N, K),), 127, dtype=torch.uint8, device="cuda"), K)
    e = bsp.MXFP8Experts(b.q[None], b.sf[None], K)
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    torch.cuda.empty_cache()
    room = torch.cuda.memory_reserved() + (1 << 30)  # D takes 2 GiB
    torch.cuda.set_per_process_memory_fraction(room / torch.cuda.get_device_properties(0).total_memory)
    try:
        for call in (lambda: bsp.mxfp8_gemm(a, b), lambda: bsp.mxfp8_gemm(a, b, activation="relu"),
                     lambda: bsp.mxfp8_grouped_gemm(a, e, off)):
            with pytest.raises(torch.OutOfMemoryError):
                call()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert bsp.device_status() == 0
    assert not bool(bsp.mxfp8_gemm(a, b, activation="relu").any())


FIRST_CALLS = r"""
import sys
import threading
import torch
import block_scaled_precision_05_b200 as bsp

def make(seed):
    g = torch.Generator("cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    one = torch.ones(1, device="cuda")
    a, b = bsp.nvfp4_quantize(rand(600, 320), one), bsp.nvfp4_quantize(rand(512, 320), one)
    s, t = bsp.nvfp4_quantize(rand(9, 8192), one), bsp.nvfp4_quantize(rand(264, 8192), one)
    w, _, _ = bsp.nvfp4_quantize_experts(rand(3, 8976, 1312))
    x = bsp.nvfp4_quantize(rand(700, 1312), one)
    off = torch.tensor([0, 250, 381, 700], dtype=torch.int32, device="cuda")
    # single CTAs, K split over a cluster, CTA pairs
    return lambda: (bsp.nvfp4_gemm(a, b, activation="silu"), bsp.nvfp4_gemm(s, t, activation="gelu"),
                    bsp.nvfp4_grouped_gemm(x, w, off, activation="gelu_tanh"))

run = make(0)
torch.cuda.synchronize()
if sys.argv[1] == "captured":
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = run()
    graph.replay()
    outs = [first]
else:
    outs, start = [None] * 8, threading.Barrier(8)
    def work(i):
        start.wait()
        with torch.cuda.stream(torch.cuda.Stream()):
            outs[i] = run()
            torch.cuda.current_stream().synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
torch.cuda.synchronize()
want = run()
torch.cuda.synchronize()
assert bsp.device_status() == 0
for got in outs:
    assert all(torch.equal(g, w) for g, w in zip(got, want))
print("same bits")
"""


@pytest.mark.parametrize("how", ["captured", "threads"])
def test_a_process_whose_first_calls_are(how):
    """The first fused calls of a process inside a graph capture, and from eight threads at once."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS, how], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same bits" in r.stdout, r.stdout[-500:] + r.stderr[-3000:]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_outputs_past_32_bits(dtype):
    """D and a residual of more than 2^31 elements: rows at both ends and around the border, computed exactly (one 1.0 in each
    row of A picks a column of B out)."""
    N, K = 13824, 32
    M = 2 ** 31 // N + 300
    codes = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
    pick = torch.arange(M, device="cuda") % K
    codes[torch.arange(M, device="cuda"), pick] = 0x38  # 1.0
    ones = lambda rows: torch.full((bsp.mxfp8_sf_bytes(rows, K),), 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    g = torch.Generator("cuda").manual_seed(0)
    b = torch.randint(0, 0x50, (N, K), generator=g, device="cuda").to(torch.uint8)
    res = torch.empty((M, N), dtype=dtype, device="cuda")
    res[:] = (torch.arange(M, device="cuda") % 8).to(dtype)[:, None]
    out = bsp.mxfp8_gemm(bsp.MXFP8Tensor(codes, ones(M), K), bsp.MXFP8Tensor(b, ones(N), K), out_dtype=dtype, residual=res, out=res)
    assert bsp.device_status() == 0
    values = b.view(torch.float8_e4m3fn).double()
    edge = 2 ** 31 // N
    rows = torch.cat((torch.arange(0, 300), torch.arange(edge - 300, M))).to("cuda")
    want = values[:, pick[rows]].t() + (rows % 8).double()[:, None]
    assert torch.equal(out[rows], want.float().to(dtype))
