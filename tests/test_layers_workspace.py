"""What the workspace of the loss over the vocabulary holds (CPU only): the
probabilities of one piece of rows where a gradient is asked for, and none for
the loss alone."""

import ctypes
import os

import pytest

from bit_nf4_quantized_amd import api


@pytest.fixture(scope="module")
def size():
    if not os.path.exists(api.LIB_PATH):
        from bit_nf4_quantized_amd import build
        build.build()
    fn = api.library().qlora_head_workspace

    def size(M, K, V, dH, dW, dtype=0):
        n = ctypes.c_size_t()
        assert fn(M, K, V, dH, dW, dtype, ctypes.byref(n)) == api.QLORA_OK
        return n.value

    return size


def others(M, K, V):
    """The counted rows of H, 28 bytes per row and 8 per row and tile of 256 words, some rounding."""
    rows = (M + 255) // 256 * 256
    return 2 * M * K + 28 * rows + 8 * rows * ((V + 255) // 256) + 16 * 256


@pytest.mark.parametrize("M,K,V", [(1, 64, 5), (48, 4096, 32000), (8192, 4096, 32000), (4096, 4096, 128256), (300, 64, 1 << 22), (1 << 18, 64, 32001)])
def test_loss_alone_holds_no_probabilities(size, M, K, V):
    assert size(M, K, V, 0, 0) <= others(M, K, V)


@pytest.mark.parametrize("M,K,V", [(1, 64, 5), (8192, 4096, 32000), (300, 64, 1 << 22), (1 << 18, 64, 32001)])
def test_gradients_hold_one_piece(size, M, K, V):
    """Pieces of at most 2^29 / V rows and at least 256, so P takes 1 GiB at most, or 512 V bytes."""
    for dH, dW in ((1, 0), (0, 1), (1, 1)):
        ldp = (V + 63) // 64 * 64
        most = max((1 << 29) // ldp // 256 * 256, 256)
        piece = min((max(M, 1) + 255) // 256 * 256, most)
        p = 2 * piece * ldp
        assert p <= max(1 << 30, 512 * ldp)
        assert p <= size(M, K, V, dH, dW) - size(M, K, V, 0, 0) + 4096
        assert size(M, K, V, dH, dW) >= size(M, K, V, 0, 0)


def test_never_shrinks_without_gradients(size):
    rows = [*range(0, 600), *range(600, 40000, 777), 1 << 16, 1 << 18, 1 << 21]
    for K, V in ((64, 5), (1024, 32001), (64, 1 << 22)):
        for dH, dW in ((0, 0), (1, 0), (0, 1)):
            sizes = [size(M, K, V, dH, dW) for M in rows]
            assert sizes == sorted(sizes), (K, V, dH, dW)
