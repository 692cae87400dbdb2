"""Values that are not finite in the 8 bits that the layer operators keep: a
block of 64 that holds an infinity or NaN stands for 64 NaN, other blocks hold
what they hold without it, and the backward pass from kept values is not finite
where the one that computes them again is not."""

import numpy as np
import pytest

from gpu_util import require_gpu
from test_gpu_layers import Gated, bf16, dev

pytestmark = pytest.mark.gpu

BLOCK = 64


@pytest.fixture(scope="module")
def api():
    return require_gpu()


def check_blocks(api, got, ref, bad, shape):
    """`bad`: truth values per element; a block with one is NaN, the others are ref's bit for bit."""
    import torch

    blocks = bad.reshape(-1, BLOCK).any(1)
    codes, absmax = got
    out = api.qlora_int8_dequantize(codes, absmax).reshape(-1, BLOCK)
    assert torch.isnan(out[blocks]).all()
    assert (codes.reshape(-1, BLOCK)[blocks] == 0).all() and not torch.isfinite(absmax[blocks]).any()
    assert (codes.reshape(-1, BLOCK)[~blocks] == ref[0].reshape(-1, BLOCK)[~blocks]).all()
    assert (absmax[~blocks] == ref[1][~blocks]).all()


VALUES = [float("nan"), float("inf"), float("-inf")]


@pytest.mark.parametrize("value", VALUES)
@pytest.mark.parametrize("K", [64, 256, 4160])
@pytest.mark.parametrize("f32", [False, True])
def test_norm_kept(api, value, K, f32):
    """A weight that is not finite, and a row of x with one value that is not."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(9, K, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.ones(K, device="cuda")
    ref = api.qlora_norm_fwd(x, w, want_int8=True)
    for at in (0, 7, K // 2 + 13, K - 1):
        w2 = w.clone()
        w2[at] = value
        o = api.qlora_norm_fwd(x, w2, want_int8=True)
        bad = torch.zeros(9, K, dtype=torch.bool, device="cuda")
        bad[:, at] = True
        assert (torch.isfinite(o.y) == ~bad).all()
        check_blocks(api, o.int8, ref.int8, bad, x.shape)
    x2 = x.clone()
    x2[4, K // 2] = value
    o = api.qlora_norm_fwd(x2, w, want_int8=True)
    y = api.qlora_int8_dequantize(*o.int8).reshape(9, K)
    nan = torch.isnan(y[4]).reshape(-1, BLOCK)
    if np.isnan(value):                            # the whole row; an infinity leaves zeros beside it
        assert nan.all()
    else:
        assert nan[K // 2 // BLOCK].all() and nan.sum() == BLOCK
    rest = torch.arange(9, device="cuda") != 4
    assert (y[rest] == api.qlora_int8_dequantize(*ref.int8).reshape(9, K)[rest]).all()


@pytest.mark.parametrize("value", VALUES)
@pytest.mark.parametrize("M", [1, 20, 150])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_kept(api, value, M, kind):
    """One feature of gate's and one of up's adapter that are not finite."""
    import torch

    K, F, r = 128, 192, 16
    c = Gated(api, M, K, F, r, kind=kind)
    ref = c.fwd(want_T=True, want_int8=True)
    c.L2d[0, 3, 70] = value
    c.L2d[1, 5, 130] = value
    o = c.fwd(want_T=True, want_int8=True)
    for k, (got, was, at) in enumerate(((o.gate8, ref.gate8, 70), (o.up8, ref.up8, 130))):
        bad = torch.zeros(M, F, dtype=torch.bool, device="cuda")
        bad[:, at] = True
        check_blocks(api, got, was, bad, (M, F))
    again = c.bwd(T=o.T)
    kept = c.bwd(T=o.T, gate8=o.gate8, up8=o.up8)
    for a, b in zip(again, kept):
        assert not torch.isfinite(b[~torch.isfinite(a)]).any()
    assert torch.isnan(kept[0]).all() and torch.isnan(kept[2][0, :, 64:128]).all() and torch.isfinite(kept[2][:, :, :64]).all()


def test_one_row_kept(api):
    """A NaN in one row of X reaches the kept values and dX of that row alone."""
    import torch

    for M in (3, 40, 200):
        c = Gated(api, M, 128, 192, 16)
        ref = c.fwd(want_T=True, want_int8=True)
        dX = c.bwd(T=ref.T, gate8=ref.gate8, up8=ref.up8)[0]
        c.Xd[M // 2, 5] = float("nan")
        o = c.fwd(want_T=True, want_int8=True)
        bad = torch.zeros(M, 192, dtype=torch.bool, device="cuda")
        bad[M // 2] = True
        for got, was in ((o.gate8, ref.gate8), (o.up8, ref.up8)):
            check_blocks(api, got, was, bad, (M, 192))
        got = c.bwd(T=o.T, gate8=o.gate8, up8=o.up8)[0]
        rest = torch.arange(M, device="cuda") != M // 2
        assert (got[rest] == dX[rest]).all() and torch.isnan(got[M // 2]).all()


def test_finite_blocks_are_the_codec(api):
    """y from a bf16 norm of unit weight against the codec on the same fp32 values, zeros and tiny values among them."""
    import torch

    x = dev(bf16(np.random.default_rng(3).standard_normal((40, 128)).astype(np.float32)))
    x[3] = 0.0
    x[4, :64] = 0.0
    x[5, 64:] = 1e-38
    w = torch.ones(128, device="cuda")
    w[64:] = 2.0 ** -100
    o = api.qlora_norm_fwd(x, w, want_int8=True)
    y = x.float() * o.rstd[:, None] * w               # each product rounded once, as in the kernel
    codes, absmax = api.qlora_int8_quantize(y)
    assert (codes == o.int8[0]).all() and (absmax == o.int8[1]).all()
