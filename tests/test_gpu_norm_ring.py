"""The residual norm's form for many long rows, which walks them through shared memory."""
import ctypes

import pytest
import torch

import serving_kda_chunk_gb300 as kda

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


# a row length of each of its forms
@pytest.mark.parametrize("d,res", [(1032, BF16), (2048, BF16), (4096, F32), (8192, BF16), (16384, BF16)])
def test_a_refused_launch_leaves_no_error(d, res):
    rt = ctypes.CDLL("libcudart.so.13")
    x = torch.randn(1100, d, device="cuda").to(BF16)
    r, out = torch.zeros(1100, d, dtype=res, device="cuda"), torch.zeros_like(x)
    s = torch.cuda.Stream()
    call = lambda: kda.kda_residual_norm(x, r, out=out, stream=s)  # noqa: E731
    torch.cuda.synchronize()
    call()
    torch.cuda.synchronize()
    first = out.clone()
    out.zero_()
    h = ctypes.c_void_p(s.cuda_stream)
    torch.cuda.synchronize()
    assert rt.cudaStreamBeginCapture(h, 2) == 0  # relaxed
    assert rt.cudaStreamSynchronize(h) != 0      # not allowed while capturing: the capture is invalid now
    rt.cudaGetLastError()
    try:
        with pytest.raises(kda.KdaError):
            call()
        left = rt.cudaGetLastError()
    finally:
        graph = ctypes.c_void_p()
        rt.cudaStreamEndCapture(h, ctypes.byref(graph))
        rt.cudaGetLastError()
    assert left == 0
    torch.cuda.synchronize()
    assert (out == 0).all()
    call()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
