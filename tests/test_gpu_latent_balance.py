"""Blocks of a latent prefill go to the pair of SMs that comes free first.  Eight heads of 8192 tokens are
128 blocks of falling length for 76 pairs: where pairs take their second block before they know how long the
first one is, some walk two long ones.  Timed against 16 heads (3.4 blocks a pair, which any order evens out):
0.54 of their time, and 0.72 when every pair asked for its next block at once."""
import pytest
import torch

from test_gpu_latent import SCALE

import serving_kda_chunk_gb300 as kda

pytestmark = pytest.mark.gpu


def best_ms(heads, tokens=8192):
    z = lambda *n: torch.randn(*n, device="cuda").bfloat16()  # noqa: E731
    q, kv, kr, out = z(tokens, heads, 192), z(tokens, heads, 256), z(tokens, 64), z(tokens, heads, 128)
    cu = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    times = []
    for _ in range(12):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        for _ in range(10):
            kda.kda_latent_prefill(q, kv[..., :128], kr, kv[..., 128:], cu, cu, out, scale=SCALE)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) / 10)
    return min(times)


def test_few_blocks_a_pair_are_taken_by_the_pair_that_is_free():
    few, many = best_ms(8), best_ms(16)
    print(f"[balance] 8 heads {few * 1e3:.1f} us, 16 heads {many * 1e3:.1f} us, ratio {few / many:.3f}")
    assert few <= 0.62 * many
