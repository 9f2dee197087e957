"""A launch that the CUDA runtime refuses comes back as KDA_ERR_CUDA and leaves no error behind for
whoever asks next.  The refusal is the host's: a stream whose capture was invalidated takes no launch."""
import ctypes

import pytest
import torch

import serving_kda_chunk_gb300 as kda

pytestmark = pytest.mark.gpu


def latent_decode(s, t):
    kda.kda_latent_decode(t["q"][..., :512], t["q"][..., 512:], t["cache"], t["table"], t["len"], t["out"], t["ws"], stream=s)


def latent_prefill(s, t):
    kda.kda_latent_prefill(t["q3"], t["k"], t["kr"], t["k"], t["cu"], t["cu"], t["o3"], stream=s)


def latent_append(s, t):
    kda.kda_latent_append(t["q"][:, 0], t["cache"], t["len"], stream=s)


def token_logprobs(s, t):
    kda.kda_token_logprobs(t["q"][:, 0], t["len"], t["lp"], stream=s)


@pytest.mark.parametrize("call", [latent_decode, latent_prefill, latent_append, token_logprobs])
def test_a_refused_launch_leaves_no_error(call):
    rt = ctypes.CDLL("libcudart.so.13")
    z = lambda *n, dtype=torch.bfloat16: torch.zeros(*n, dtype=dtype, device="cuda")  # noqa: E731
    i = torch.int32
    t = dict(q=z(2, 4, 576), cache=z(20, 64, 576), table=z(2, 10, dtype=i), len=z(2, dtype=i) + 500, out=z(2, 4, 512),
             ws=z(kda.kda_latent_decode_workspace_size(2, 1, 4), dtype=torch.uint8), q3=z(5, 2, 192), k=z(5, 2, 128),
             kr=z(5, 64), o3=z(5, 2, 128), lp=z(2, dtype=torch.float32), cu=torch.tensor([0, 5], dtype=i, device="cuda"))
    s = torch.cuda.Stream()
    call(s, t)
    torch.cuda.synchronize()
    h = ctypes.c_void_p(s.cuda_stream)
    assert rt.cudaStreamBeginCapture(h, 2) == 0  # relaxed
    assert rt.cudaStreamSynchronize(h) != 0      # not allowed while capturing: the capture is invalid now
    rt.cudaGetLastError()
    try:
        with pytest.raises(kda.KdaError):
            call(s, t)
        left = rt.cudaGetLastError()
    finally:
        graph = ctypes.c_void_p()
        rt.cudaStreamEndCapture(h, ctypes.byref(graph))
        rt.cudaGetLastError()
    assert left == 0
    call(s, t)
    torch.cuda.synchronize()
