"""Host-side checks of the entry points of include/qlora_adapters.h (CPU only):
the library exports what the header declares, reports the sizes the layouts
imply, and rejects bad arguments before anything is enqueued."""

import ctypes
import os
import re

import pytest

from bit_nf4_quantized_amd import api
from oracle import optim_batch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qlora_adapters.h")
P = 4096   # a 16-byte aligned address that is never dereferenced


def declared_functions():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_ ]*[\s\*]+(qlora_[a-z0-9_]+)\s*\(", text, flags=re.M)
    return sorted(set(names))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(api.LIB_PATH):
        from bit_nf4_quantized_amd import build
        build.build()
    return api.library()


def test_exports_every_declared_symbol(lib):
    names = declared_functions()
    assert sorted(api.ADAPTER_EXPORTS) == names
    for n in names:
        assert hasattr(lib, n), n


def ptrs(*a):
    return (ctypes.c_void_p * max(len(a), 1))(*a)


def sizes(*a):
    return (ctypes.c_int64 * max(len(a), 1))(*a)


def test_adam_state_numel(lib):
    total = ctypes.c_int64(-1)
    for numel in ([], [0], [1], [256], [257, 0, 3], [10 ** 9 + 1] * 5):
        assert lib.qlora_adam_state_numel(len(numel), sizes(*numel), ctypes.byref(total)) == api.QLORA_OK
        assert total.value == optim_batch.offsets(numel)[-1]
    assert lib.qlora_adam_state_numel(-1, sizes(1), ctypes.byref(total)) == api.QLORA_ERR_ARG
    assert lib.qlora_adam_state_numel(1, None, ctypes.byref(total)) == api.QLORA_ERR_ARG
    assert lib.qlora_adam_state_numel(1, sizes(1), None) == api.QLORA_ERR_ARG
    assert lib.qlora_adam_state_numel(1, sizes(-1), ctypes.byref(total)) == api.QLORA_ERR_SHAPE
    assert lib.qlora_adam_state_numel(1, sizes((1 << 40) + 1), ctypes.byref(total)) == api.QLORA_ERR_SHAPE
    assert lib.qlora_adam_state_numel(2, sizes(1 << 40, 1 << 40), ctypes.byref(total)) == api.QLORA_ERR_SHAPE


def test_clip_grad_norm_batch_refusals(lib):
    def call(n=1, g=ptrs(P), dt=0, numel=sizes(8), mx=0.3, coef=P, norm=P, ws=P, wsb=8192):
        return lib.qlora_clip_grad_norm_batch(n, g, dt, numel, mx, coef, norm, ws, wsb, None)

    E = api
    assert call(n=-1) == E.QLORA_ERR_ARG
    assert call(g=None) == E.QLORA_ERR_ARG
    assert call(g=ptrs(None)) == E.QLORA_ERR_ARG
    assert call(dt=2) == E.QLORA_ERR_ARG
    assert call(numel=sizes(-8)) == E.QLORA_ERR_SHAPE
    assert call(mx=0.0) == E.QLORA_ERR_ARG
    assert call(mx=float("nan")) == E.QLORA_ERR_ARG
    assert call(coef=None, norm=None) == E.QLORA_ERR_ARG
    assert call(ws=None) == E.QLORA_ERR_WORKSPACE
    assert call(wsb=8191) == E.QLORA_ERR_WORKSPACE
    assert call(g=ptrs(P + 8)) == E.QLORA_ERR_ALIGN
    assert call(norm=P + 4) == E.QLORA_ERR_ALIGN
    assert call(coef=P + 2) == E.QLORA_ERR_ALIGN


def test_adamw_batch_refusals(lib):
    good_hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1)

    def call(n=1, th=ptrs(P), g=ptrs(P), dt=0, tb=None, numel=sizes(8), bits=8, m=P, v=P, ms=P, vs=P, coef=None, **hp):
        st = api.QAdamState(bits, m, v, ms, vs)
        h = api.AdamParams(**{**good_hp, **hp})
        return lib.qlora_adamw_batch(n, th, g, dt, tb, numel, ctypes.byref(st), ctypes.byref(h), coef, None)

    E = api
    assert call(n=0) == E.QLORA_OK
    assert call(numel=sizes(0), th=ptrs(None)) == E.QLORA_OK
    assert call(n=-1) == E.QLORA_ERR_ARG
    assert call(th=None) == E.QLORA_ERR_ARG
    assert call(th=ptrs(None)) == E.QLORA_ERR_ARG
    assert call(g=ptrs(None)) == E.QLORA_ERR_ARG
    assert call(tb=ptrs(None)) == E.QLORA_ERR_ARG
    assert call(dt=3) == E.QLORA_ERR_ARG
    assert call(bits=4) == E.QLORA_ERR_ARG
    assert call(m=None) == E.QLORA_ERR_ARG
    assert call(ms=None) == E.QLORA_ERR_ARG
    assert call(numel=sizes(-1)) == E.QLORA_ERR_SHAPE
    for bad in (dict(step=0), dict(lr=-1.0), dict(lr=float("inf")), dict(beta1=1.0), dict(beta2=-0.1),
                dict(eps=-1.0), dict(weight_decay=float("nan"))):
        assert call(**bad) == E.QLORA_ERR_ARG, bad
    assert call(th=ptrs(P + 4)) == E.QLORA_ERR_ALIGN
    assert call(g=ptrs(P + 4)) == E.QLORA_ERR_ALIGN
    assert call(tb=ptrs(P + 2)) == E.QLORA_ERR_ALIGN
    assert call(v=P + 8) == E.QLORA_ERR_ALIGN
    assert call(vs=P + 2) == E.QLORA_ERR_ALIGN
    assert call(coef=P + 1) == E.QLORA_ERR_ALIGN
    assert lib.qlora_adamw_batch(1, ptrs(P), ptrs(P), 0, None, sizes(8), None, None, None, None) == E.QLORA_ERR_ARG


def test_preference_refusals(lib):
    n = ctypes.c_size_t()
    for pairs, T, V in ((0, 0, 1), (1, 1, 1), (3, 100, 32000), (1 << 20, 1, 7)):
        assert lib.qlora_preference_workspace(pairs, T, V, ctypes.byref(n)) == api.QLORA_OK
        assert n.value >= 8 * pairs * T + 8 * pairs
    for pairs, T, V in ((-1, 1, 1), (1, -1, 1), (1, 1, 0), ((1 << 20) + 1, 1, 1), (1 << 15, 1 << 15, 8), (1, 1, (1 << 30) + 1)):
        assert lib.qlora_preference_workspace(pairs, T, V, ctypes.byref(n)) == api.QLORA_ERR_SHAPE, (pairs, T, V)
    assert lib.qlora_preference_workspace(1, 1, 1, None) == api.QLORA_ERR_ARG

    def call(x=P, dt=0, pairs=1, T=2, V=8, ld=8, lab=P, ref=P, beta=0.1, eps=0.0, gs=1.0, loss=P, rew=P, lp=P,
             dx=2 * P, ldd=8, ws=P, wsb=1 << 20):
        return lib.qlora_preference_loss(x, dt, pairs, T, V, ld, lab, ref, beta, eps, gs, loss, rew, lp, dx, ldd, ws,
                                         wsb, None)

    E = api
    for bad in (dict(dt=5), dict(beta=float("inf")), dict(eps=-0.1), dict(eps=1.1), dict(eps=float("nan")),
                dict(gs=float("nan")), dict(x=None), dict(lab=None), dict(ref=None), dict(loss=None),
                dict(rew=None), dict(lp=None)):
        assert call(**bad) == E.QLORA_ERR_ARG, bad
    for bad in (dict(pairs=-1), dict(V=0), dict(ld=7), dict(ldd=7), dict(dx=P, ldd=9)):
        assert call(**bad) == E.QLORA_ERR_SHAPE, bad
    for bad in (dict(ws=None), dict(wsb=16)):
        assert call(**bad) == E.QLORA_ERR_WORKSPACE, bad
    for bad in (dict(x=P + 2), dict(dx=P + 1), dict(lab=P + 4), dict(ref=P + 2), dict(lp=P + 1), dict(ws=P + 8),
                dict(dt=1, x=P + 1)):
        assert call(**bad) == E.QLORA_ERR_ALIGN, bad


def multi_weight(N=264, K=256, codes=P, no_dq=0):
    return api.QNF4(N, K, codes, P, P, P, 0, no_dq, None)


def test_multi_workspace(lib):
    n, m = ctypes.c_size_t(), ctypes.c_size_t()
    ws = lambda *a: lib.qlora_linear_multi_workspace(*a, ctypes.byref(n))  # noqa: E731
    for M in (0, 1, 16, 100, 5000, 1 << 22):
        for back in (0, 1):
            assert ws(M, 256, 264, 72, 5, back) == api.QLORA_OK and n.value > 0
    assert lib.qlora_linear_multi_workspace(1, 256, 264, 8, 1, 0, None) == api.QLORA_ERR_ARG
    for bad in ((1, 256, 264, 8, 0, 0), (1, 256, 264, 8, 4097, 0), (1, 256, 264, 4, 1, 0), (1, 256, 264, 264, 1, 0)):
        assert ws(*bad) == api.QLORA_ERR_ARG, bad
    for bad in ((-1, 256, 264, 8, 1, 0), (1, 250, 264, 8, 1, 0), (1, 256, 262, 8, 1, 0), ((1 << 22) + 1, 256, 264, 8, 1, 0)):
        assert ws(*bad) == api.QLORA_ERR_SHAPE, bad
    # a larger batch never needs less
    last = 0
    for M in (1, 2, 16, 17, 128, 129, 1000, 10000):
        assert lib.qlora_linear_multi_workspace(M, 512, 512, 16, 7, 1, ctypes.byref(m)) == api.QLORA_OK
        assert m.value >= M * 16 and m.value >= last // 4
        last = m.value


@pytest.mark.parametrize("M", [1, 9, 100, 500])
def test_multi_forward_refusals(lib, M):
    def call(W=multi_weight(), X=P, M=M, ids=P, A=3, L1=P, L2=P, r=16, s=P, Y=P, T=None, ws=P, wsb=1 << 40):
        return lib.qlora_linear_multi_fwd(ctypes.byref(W), X, M, ids, A, L1, L2, r, s, Y, T, ws, wsb, None)

    E = api
    assert call(M=0) == E.QLORA_OK
    for bad in (dict(X=None), dict(ids=None), dict(A=0), dict(A=5000), dict(L1=None), dict(L2=None), dict(r=12),
                dict(r=264), dict(s=None), dict(Y=None), dict(W=multi_weight(codes=None))):
        assert call(**bad) == E.QLORA_ERR_ARG, bad
    for bad in (dict(M=-1), dict(M=(1 << 22) + 1), dict(W=multi_weight(K=250)), dict(W=multi_weight(N=260))):
        assert call(**bad) == E.QLORA_ERR_SHAPE, bad
    for bad in (dict(ws=None), dict(wsb=8)):
        assert call(**bad) == E.QLORA_ERR_WORKSPACE, bad
    for bad in (dict(X=P + 8), dict(ids=P + 2), dict(L1=P + 8), dict(L2=P + 4), dict(s=P + 1), dict(Y=P + 8),
                dict(T=P + 8), dict(ws=P + 8)):
        assert call(**bad) == E.QLORA_ERR_ALIGN, bad


def test_multi_backward_refusals(lib):
    def call(W=multi_weight(), X=P, dY=P, M=50, ids=P, A=3, L1=P, L2=P, r=16, s=P, T=None, dX=P, d1=P, d2=P, dt=0,
             ws=P, wsb=1 << 40):
        return lib.qlora_linear_multi_bwd(ctypes.byref(W), X, dY, M, ids, A, L1, L2, r, s, T, dX, d1, d2, dt, ws, wsb,
                                          None)

    E = api
    for bad in (dict(X=None), dict(dY=None), dict(ids=None), dict(A=0), dict(L1=None), dict(L2=None), dict(r=0),
                dict(s=None), dict(d1=None), dict(d2=None), dict(dt=7)):
        assert call(**bad) == E.QLORA_ERR_ARG, bad
    for bad in (dict(M=-1), dict(M=(1 << 22) + 1), dict(W=multi_weight(K=1 << 17, N=1 << 14))):
        assert call(**bad) == E.QLORA_ERR_SHAPE, bad
    for bad in (dict(ws=None), dict(wsb=8)):
        assert call(**bad) == E.QLORA_ERR_WORKSPACE, bad
    for bad in (dict(X=P + 8), dict(dY=P + 2), dict(T=P + 8), dict(dX=P + 8), dict(d1=P + 4), dict(d2=P + 8),
                dict(ws=P + 8)):
        assert call(**bad) == E.QLORA_ERR_ALIGN, bad
