"""Workspace sizes of the linear with an adapter per row (CPU only): a larger
batch never needs less, so a workspace for the largest batch serves all."""

import ctypes
import os

import pytest

from bit_nf4_quantized_amd import api

ROWS = list(range(0, 2600)) + [m + d for m in (4096, 8192, 11008, 16384, 32768, 65536, 1 << 17, 1 << 20, 1 << 22)
                               for d in (-129, -128, -64, -1, 0)]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(api.LIB_PATH):
        from bit_nf4_quantized_amd import build
        build.build()
    return api.library()


@pytest.mark.parametrize("back", [0, 1])
@pytest.mark.parametrize("K,N,r,A", [(4096, 4096, 16, 4), (4096, 11008, 64, 16), (11008, 4096, 32, 300), (64, 8, 8, 1),
                                     (4096, 136, 256, 2), (256, 8192, 136, 4096), (28672, 8192, 64, 7), (1088, 264, 24, 40)])
def test_a_larger_batch_never_needs_less(lib, K, N, r, A, back):
    n, last = ctypes.c_size_t(), 0
    for M in ROWS:
        assert lib.qlora_linear_multi_workspace(M, K, N, r, A, back, ctypes.byref(n)) == api.QLORA_OK
        assert n.value >= last, (M, n.value, last)
        last = n.value


P = 4096   # a 16-byte aligned address that is never dereferenced


def test_operands_beyond_one_launch(lib):
    """Adapters whose laid-out factor would take 2^32 work-items or more are refused before anything is enqueued."""
    def call(back, M, K, N, r, A, dX=P):
        W = api.QNF4(N, K, P, P, P, P, 0, 0, None)
        if back:
            return lib.qlora_linear_multi_bwd(ctypes.byref(W), P, P, M, P, A, P, P, r, P, None, dX, P, P, 0, P, 0, None)
        return lib.qlora_linear_multi_fwd(ctypes.byref(W), P, M, P, A, P, P, r, P, P, None, P, 0, None)

    # 4096 adapters of [32768][256] are 2^35 values: 2^32 work-items of 8; the workspace of 0 bytes is checked later
    assert call(True, 5000, 32768, 64, 256, 4096) == api.QLORA_ERR_SHAPE
    assert call(True, 5000, 32768, 64, 256, 4096, dX=None) == api.QLORA_ERR_WORKSPACE
    assert call(True, 5000, 32768, 64, 256, 2048) == api.QLORA_ERR_WORKSPACE
    assert call(True, 1000, 32768, 64, 256, 4096) == api.QLORA_ERR_WORKSPACE          # 1000 rows: at most 1000 adapters
    assert call(False, 5000, 64, 1 << 17, 256, 4096) == api.QLORA_ERR_SHAPE            # 2^37 values, 16 a work-item
    assert call(False, 5000, 64, 1 << 15, 256, 4096) == api.QLORA_ERR_WORKSPACE
    assert call(False, 100, 64, 1 << 17, 256, 4096) == api.QLORA_ERR_WORKSPACE
