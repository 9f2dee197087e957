"""Host-side refusals: a scale that is not finite (a NaN would pass for a scale of 0), and the self-test's."""
import ctypes

import pytest

FAKE = 1 << 20  # 16-byte aligned, never dereferenced: checks fail first
OK, INVALID, UNSUPPORTED, BF16, F16 = 0, 1, 2, 0, 2


@pytest.fixture(scope="module")
def kda():
    import __graft_entry__

    __graft_entry__.build()
    import serving_kda_chunk_gb300 as kda

    return kda


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), float("-inf")])
def test_latent_calls_refuse_a_scale_that_is_not_finite(kda, scale):
    L = kda.lib()
    d = ctypes.byref(kda.RowsDesc(FAKE, 512, 512))
    size = L.kda_latent_decode_workspace_size(4, 2, 8)

    def decode(R):
        return L.kda_latent_decode(d, d, BF16, R, 2, None, 8, 512, 64, scale, FAKE, 8, 16, 16 * 576, FAKE, 4, FAKE, d,
                                   BF16, None, FAKE, size, None, None)

    def prefill(N):
        return L.kda_latent_prefill(d, d, FAKE, 64, d, BF16, FAKE, FAKE, N, 10, 10, 4, 128, 64, 128, scale, 0, d, BF16,
                                    None, None, None)

    assert decode(4) == INVALID and prefill(2) == INVALID
    assert decode(0) == OK and prefill(0) == OK  # nothing to do


def test_decode_self_test_refusals(kda):
    L = kda.lib()
    d = ctypes.byref(kda.RowsDesc(FAKE, 512, 512))

    def call(H=8, K=2, dt=BF16, block=0, load=0, table=FAKE):
        size = L.kda_latent_decode_workspace_size(4, K, H)
        return L.kda_selftest_latent_decode_give_up(d, d, dt, 4, K, None, H, 512, 64, 1.0, FAKE, 8, 16, 16 * 576, table,
                                                    4, FAKE, d, BF16, None, FAKE, size, None, None, block, load)

    assert call(block=-1) == INVALID and call(load=-1) == INVALID and call(table=None) == INVALID
    assert call(H=9) == UNSUPPORTED and call(dt=F16) == UNSUPPORTED


def test_prefill_self_test_refusals(kda):
    L = kda.lib()
    d = ctypes.byref(kda.RowsDesc(FAKE, 512, 512))

    def call(dt=BF16, block=0, tile=0, cu=FAKE):
        return L.kda_selftest_latent_prefill_give_up(d, d, FAKE, 64, d, dt, cu, FAKE, 2, 10, 10, 4, 128, 64, 128, 1.0, 0,
                                                     d, BF16, None, None, None, block, tile)

    assert call(block=-1) == INVALID and call(tile=-1) == INVALID and call(cu=None) == INVALID
    assert call(dt=F16) == UNSUPPORTED
