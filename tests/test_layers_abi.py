"""Host-side checks of the entry points of include/qlora_layers.h (CPU only):
the library exports what the header declares, reports sizes that grow with
their arguments, and rejects bad arguments before anything is enqueued."""

import ctypes
import os
import re

import pytest

from bit_nf4_quantized_amd import api

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qlora_layers.h")
P = 4096   # a 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(api.LIB_PATH):
        from bit_nf4_quantized_amd import build
        build.build()
    return api.library()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_ ]*[\s\*]+(qlora_[a-z0-9_]+)\s*\(", text, flags=re.M)))
    assert sorted(api.LAYER_EXPORTS) == names
    for n in names:
        assert hasattr(lib, n), n


def nf4(rows=128, cols=64, codes=P, **kw):
    q = api.QNF4(rows, cols, codes, P, P, P, 0, 0, None)
    for k, v in kw.items():
        setattr(q, k, v)
    return q


def int8(codes=P, absmax=P):
    return ctypes.byref(api.QInt8Values(codes, absmax))


def size(fn, *args):
    n = ctypes.c_size_t()
    assert fn(*args, ctypes.byref(n)) == api.QLORA_OK, args
    return n.value


BIG = 1 << 40


def test_gated_workspace(lib):
    w = lib.qlora_gated_workspace
    n = ctypes.c_size_t()
    sizes = [size(w, M, 4096, 11008, 64, 1) for M in (0, 1, 129, 4096, 1 << 21)]
    assert sizes == sorted(sizes) and sizes[0] >= 2 * 11008 * 4096 * 2
    assert size(w, 128, 4096, 11008, 64, 0) < size(w, 129, 4096, 11008, 64, 0)
    for args in ((-1, 64, 64, 8), (1, 63, 64, 8), (1, 64, 65, 8), (1, 0, 64, 8), ((1 << 21) + 1, 64, 64, 8),
                 (1, 1 << 22, 64, 8), (1, 64, 1 << 22, 8)):
        assert w(*args, 0, ctypes.byref(n)) == api.QLORA_ERR_SHAPE, args
    for r in (0, 4, 12, 264):
        assert w(1, 64, 64, r, 0, ctypes.byref(n)) == api.QLORA_ERR_ARG
    assert w(1, 64, 64, 8, 0, None) == api.QLORA_ERR_ARG


def test_gated_fwd_refusals(lib):
    def call(gate=nf4(), up=nf4(), X=P, M=4, L1=P, L2=P, r=8, scale=1.0, act=0, A=P, T=None, g8=None, u8=None, ws=P,
             wsb=BIG):
        return lib.qlora_gated_fwd(gate and ctypes.byref(gate), up and ctypes.byref(up), X, M, L1, L2, r, scale, act, A, T,
                                   g8, u8, ws, wsb, None)

    E = api
    assert call(M=0) == E.QLORA_OK and call(M=0, X=None, A=None, ws=None, wsb=0) == E.QLORA_OK
    for bad in (dict(gate=None), dict(up=None), dict(X=None), dict(A=None), dict(L1=None), dict(L2=None), dict(r=12),
                dict(r=0), dict(scale=float("nan")), dict(act=2), dict(act=-1), dict(g8=int8()), dict(u8=int8()),
                dict(g8=int8(), u8=int8(None)), dict(g8=int8(P, None), u8=int8()), dict(gate=nf4(qtype=9)),
                dict(up=nf4(no_dq=1))):
        assert call(**bad) == E.QLORA_ERR_ARG, bad
    for bad in (dict(M=-1), dict(M=(1 << 21) + 1), dict(up=nf4(rows=136)), dict(up=nf4(cols=128)),
                dict(gate=nf4(rows=100), up=nf4(rows=100)), dict(gate=nf4(cols=72), up=nf4(cols=72)),
                dict(gate=nf4(rows=72), up=nf4(rows=72), g8=int8(), u8=int8())):
        assert call(**bad) == E.QLORA_ERR_SHAPE, bad
    for bad in (dict(X=P + 8), dict(A=P + 4), dict(L1=P + 2), dict(L2=P + 2), dict(T=P + 2), dict(ws=P + 4),
                dict(gate=nf4(codes=P + 4)), dict(g8=int8(P + 4), u8=int8()), dict(g8=int8(), u8=int8(P, P + 2))):
        assert call(**bad) == E.QLORA_ERR_ALIGN, bad
    need = size(lib.qlora_gated_workspace, 4, 64, 128, 8, 0)
    assert call(ws=None) == E.QLORA_ERR_WORKSPACE and call(wsb=need - 1) == E.QLORA_ERR_WORKSPACE


def test_gated_bwd_refusals(lib):
    def call(gate=nf4(), up=nf4(), X=P, X8=None, dA=P, M=4, L1=P, L2=P, r=8, scale=1.0, act=0, T=None, g8=None, u8=None,
             dX=P, dL1=P, dL2=P, gd=0, ws=P, wsb=BIG):
        return lib.qlora_gated_bwd(ctypes.byref(gate), ctypes.byref(up), X, X8, dA, M, L1, L2, r, scale, act, T, g8, u8, dX,
                                   dL1, dL2, gd, ws, wsb, None)

    E = api
    for bad in (dict(X=None), dict(X8=int8()), dict(dA=None), dict(dL1=None), dict(dL2=None), dict(gd=2), dict(act=3),
                dict(X=None, X8=int8(None)), dict(g8=int8()), dict(scale=float("inf"))):
        assert call(**bad) == E.QLORA_ERR_ARG, bad
    assert call(gate=nf4(rows=72), up=nf4(rows=72), g8=int8(), u8=int8()) == E.QLORA_ERR_SHAPE
    assert call(M=(1 << 21) + 1) == E.QLORA_ERR_SHAPE
    for bad in (dict(X=P + 8), dict(dA=P + 8), dict(dX=P + 8), dict(dL1=P + 8), dict(dL2=P + 8), dict(T=P + 8),
                dict(X=None, X8=int8(P + 8)), dict(ws=P + 8)):
        assert call(**bad) == E.QLORA_ERR_ALIGN, bad
    need = size(lib.qlora_gated_workspace, 4, 64, 128, 8, 1)
    assert call(ws=None) == E.QLORA_ERR_WORKSPACE and call(wsb=need - 1) == E.QLORA_ERR_WORKSPACE


def test_linear_bwd_int8_refusals(lib):
    def call(W=nf4(), X8=int8(), dY=P, M=4, L1=P, L2=P, r=8, scale=1.0, T=None, dX=P, dL1=P, dL2=P, gd=0, ws=P, wsb=BIG):
        return lib.qlora_linear_bwd_int8(ctypes.byref(W), X8, dY, M, L1, L2, r, scale, T, dX, dL1, dL2, gd, ws, wsb, None)

    E = api
    for bad in (dict(X8=None), dict(X8=int8(None)), dict(X8=int8(P, None)), dict(dY=None), dict(L1=None), dict(dL2=None),
                dict(gd=5), dict(r=4), dict(scale=float("nan"))):
        assert call(**bad) == E.QLORA_ERR_ARG, bad
    for bad in (dict(M=-1), dict(M=(1 << 21) + 1), dict(W=nf4(cols=96)), dict(W=nf4(rows=100))):
        assert call(**bad) == E.QLORA_ERR_SHAPE, bad
    for bad in (dict(X8=int8(P + 1)), dict(X8=int8(P, P + 1)), dict(dY=P + 2), dict(dX=P + 2), dict(dL1=P + 2),
                dict(T=P + 2), dict(ws=P + 2)):
        assert call(**bad) == E.QLORA_ERR_ALIGN, bad
    need = size(lib.qlora_linear_bwd_int8_workspace, 4, 64, 128, 8)
    assert need >= 128 * 64 * 2 + 4 * 64 * 2            # the dequantised weight and X
    assert call(ws=None) == E.QLORA_ERR_WORKSPACE and call(wsb=need - 1) == E.QLORA_ERR_WORKSPACE


def test_norm_refusals(lib):
    E = api

    def fwd(x=P, xd=1, res=P, sd=0, w=P, wd=1, M=4, K=64, eps=1e-6, y=P, y8=None, h=P, rstd=P):
        return lib.qlora_norm_fwd(x, xd, res, sd, w, wd, M, K, eps, y, y8, h, rstd, None)

    assert fwd(M=0) == E.QLORA_OK
    for bad in (dict(x=None), dict(h=None), dict(res=None), dict(xd=2), dict(sd=2), dict(wd=7), dict(eps=-1.0),
                dict(eps=float("nan")), dict(y8=int8(None))):
        assert fwd(**bad) == E.QLORA_ERR_ARG, bad
    for bad in (dict(M=-1), dict(M=(1 << 21) + 1), dict(K=0), dict(K=12), dict(K=16392), dict(K=72, y8=int8())):
        assert fwd(**bad) == E.QLORA_ERR_SHAPE, bad
    for bad in (dict(x=P + 4), dict(res=P + 4), dict(w=P + 4), dict(y=P + 4), dict(h=P + 4), dict(rstd=P + 2),
                dict(y8=int8(P + 4))):
        assert fwd(**bad) == E.QLORA_ERR_ALIGN, bad

    def bwd(dy=P, h=P, sd=0, rstd=P, w=P, wd=1, dres=None, M=4, K=64, dh=P, dx=None, dw=P, ws=P, wsb=BIG):
        return lib.qlora_norm_bwd(dy, h, sd, rstd, w, wd, dres, M, K, dh, dx, dw, ws, wsb, None)

    for bad in (dict(dy=None), dict(h=None), dict(rstd=None), dict(dh=None), dict(sd=3), dict(wd=3)):
        assert bwd(**bad) == E.QLORA_ERR_ARG, bad
    assert bwd(K=20) == E.QLORA_ERR_SHAPE and bwd(M=-1) == E.QLORA_ERR_SHAPE
    for bad in (dict(dy=P + 4), dict(dh=P + 8), dict(dres=P + 8), dict(dx=P + 8), dict(dw=P + 2), dict(ws=P + 8)):
        assert bwd(**bad) == E.QLORA_ERR_ALIGN, bad
    need = size(lib.qlora_norm_workspace, 4, 64)
    assert bwd(ws=None) == E.QLORA_ERR_WORKSPACE and bwd(wsb=need - 1) == E.QLORA_ERR_WORKSPACE


def test_head_refusals(lib):
    E = api

    def call(H=P, W=P, labels=P, weights=None, M=4, K=64, V=100, div=0.0, gs=1.0, loss=P, nll=P, dH=P, dW=None, gd=0, ws=P,
             wsb=BIG):
        return lib.qlora_head_loss(H, W, labels, weights, M, K, V, div, gs, loss, nll, dH, dW, gd, ws, wsb, None)

    for bad in (dict(H=None), dict(W=None), dict(labels=None), dict(loss=None), dict(nll=None), dict(div=-1.0),
                dict(div=float("inf")), dict(gs=float("nan")), dict(gd=2)):
        assert call(**bad) == E.QLORA_ERR_ARG, bad
    for bad in (dict(M=-1), dict(M=(1 << 21) + 1), dict(K=96), dict(K=0), dict(K=1 << 23), dict(V=0), dict(V=(1 << 22) + 1)):
        assert call(**bad) == E.QLORA_ERR_SHAPE, bad
    for bad in (dict(H=P + 8), dict(W=P + 8), dict(labels=P + 4), dict(weights=P + 2), dict(loss=P + 2), dict(nll=P + 2),
                dict(dH=P + 8), dict(dW=P + 8), dict(ws=P + 8)):
        assert call(**bad) == E.QLORA_ERR_ALIGN, bad
    need = size(lib.qlora_head_workspace, 4, 64, 100, 1, 0, 0)
    assert call(ws=None) == E.QLORA_ERR_WORKSPACE and call(wsb=need - 1) == E.QLORA_ERR_WORKSPACE
    # with the head's gradient in bf16 over several pieces of rows there is an fp32 sum too
    assert size(lib.qlora_head_workspace, 1 << 16, 64, 128256, 1, 1, 1) > size(lib.qlora_head_workspace, 1 << 16, 64, 128256, 1, 0, 1)
    # the probabilities of one piece of rows, however many rows there are
    assert size(lib.qlora_head_workspace, 1 << 20, 64, 128256, 1, 0, 0) < (2 << 30) + (1 << 20) * 200


def test_workspaces_of_no_rows(lib):
    assert size(lib.qlora_head_workspace, 0, 64, 100, 1, 1, 1) > 0
    for backward in (0, 1):
        assert size(lib.qlora_gated_workspace, 0, 64, 128, 8, backward) > 0
    assert size(lib.qlora_linear_bwd_int8_workspace, 0, 64, 128, 8) > 0
    assert size(lib.qlora_norm_workspace, 0, 64) > 0


def test_workspaces_never_shrink(lib):
    """One of the largest batch's size serves smaller batches."""
    rows = [*range(0, 400), *range(400, 17000, 83), 1 << 15, 40000, 1 << 16, 1 << 18, 1 << 21]
    for K, F, r in ((64, 8, 8), (64, 8, 72), (1024, 64, 64), (4096, 11008, 16), (4096, 11008, 136)):
        for backward in (0, 1):
            sizes = [size(lib.qlora_gated_workspace, M, K, F, r, backward) for M in rows]
            assert sizes == sorted(sizes), (K, F, r, backward)
        sizes = [size(lib.qlora_linear_bwd_int8_workspace, M, K, F, r) for M in rows]
        assert sizes == sorted(sizes), (K, F, r)
        sizes = [size(lib.qlora_head_workspace, M, K, F, 1, 1, 0) for M in rows]
        assert sizes == sorted(sizes), (K, F)
        sizes = [size(lib.qlora_norm_workspace, M, K) for M in rows]
        assert sizes == sorted(sizes), K
