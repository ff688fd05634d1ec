"""Adapters' arguments at the edge of what they may be, on the CPU: nothing here touches the GPU."""
import ctypes

import pytest

FAKE = 0x10000  # 16-byte aligned, never dereferenced
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def nv():
    import bit_gemm_nvfp4_amd as m
    return m


@pytest.mark.parametrize("m, n, rank", [(1, 1 << 23, 256), (16, (1 << 28) + 5, 8), (40, 1 << 24, 256), (200, 1 << 25, 64)])
def test_an_adapters_up_matrix_may_pass_two_billion_elements(nv, m, n, rank):
    import torch
    if torch.cuda.is_available():
        pytest.skip("would be launched")
    from bit_gemm_nvfp4_amd.mx import CMXTensor
    k = 32
    w = CMXTensor(FAKE, FAKE, n, k)
    need = nv.lib.mxfp4_adapters_workspace_size(m, n, k, 2, rank, 0)
    assert need >= m * rank * 4 and n * rank >= 1 << 31

    def call(up):
        return nv.lib.mxfp4_gemm_adapters(P(FAKE), None, m, k, ctypes.byref(w), P(FAKE), 2, rank, P(FAKE), up, None, P(FAKE), 1, n,
                                          P(FAKE), need, None)
    assert call(None) == 1 and call(P(FAKE + 8)) == 3
    assert call(P(FAKE)) == 7  # no device; NVFP4_ERR_SHAPE before
