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
