"""GPU parity of the gated block, 8-bit activations in the backward pass, the
norm and the loss over the vocabulary against the float64 oracle
(oracle/layers.py).

Every output stays, element by element, within the bound that its roundings
give. With u = 2^-24, h = 2^-8 (half a bf16 step, relative) and a sum of n
products off by at most n u times the sum of their magnitudes:

 gated   E(T) = K u |X||L1|,  E(sT) = s E(T) + h |sT|  (s T is rounded to bf16)
         E(G) = K u |X||W| + E(sT)|L2| + r u |sT||L2|  (M <= 16: + 2 h |X||W|: a decode path may take q from
                fp16, which can move a weight to the neighbouring bf16)
         act and act': the function's own error (8 |z| + 16) u relative (exp of an argument z rounded to fp32,
                and a few operations), and |act'| <= 1.13, |act''| <= 1 times E(G)
         dG, dU: those of their factors, then h (rounded once as the operands of the products)
         dX, dL1, dL2: magnitudes of the operands times the operands' errors, plus the sums'; an input in 8 bits adds
                h |X| (rounded to bf16)
 norm    a sum of K squares: K u relative, so rstd K u / 2; the rest a few u
 head    E(S) = K u |H||W|; P = exp(S - S_y) is off by E(S) + E(S_y) + (2 |t| + 8) u relative, plus h (rounded to
         bf16); nll by the largest of these; dH and dW their magnitudes' sums, for dW + h (scaled rows of H)

plus half a step of a bf16 output. Values in 8 bits are off by half a step of
their block on top of the value's own bound.
"""

import numpy as np
import pytest

from gpu_util import gpu_quantize, require_gpu, say
from oracle import layers, linear, nf4

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def api():
    return require_gpu()


def bf16(x):
    return nf4.bf16_rne(np.ascontiguousarray(x, np.float32).reshape(-1)).reshape(x.shape)


def dev(bits_or_floats):
    import torch

    from bit_nf4_quantized_amd import api as a

    if bits_or_floats.dtype == np.uint16:
        return a.to_device_bf16(bits_or_floats)
    return torch.from_numpy(np.ascontiguousarray(bits_or_floats)).cuda()


def host(t):
    """float64 values of a device tensor, and whether it is bf16."""
    import torch

    return t.detach().double().cpu().numpy(), t.dtype == torch.bfloat16


def within(label, key, got, R, E):
    G, is16 = host(got)
    E = 1.01 * E + (1.01 * linear.bf16_half_ulp(np.abs(R) + E) if is16 else 2 * U * np.abs(R)) + 1e-30
    worst = float((np.abs(G - R) / E).max()) if R.size else 0.0
    say(f"  {label} {key}: {worst:.3f} of its bound")
    assert worst <= 1.0, (label, key, worst)


def within_int8(label, key, coded, R, E):
    """int8 values against R whose own bound is E."""
    codes, absmax = coded[0].cpu().numpy(), coded[1].cpu().numpy()
    b = np.abs(R).reshape(-1, 64).max(axis=1)
    eb = E.reshape(-1, 64).max(axis=1)
    assert (np.abs(absmax - b) <= eb + 2 * U * b + 1e-30).all(), (label, key)
    step = (b + eb) / 127.0
    off = np.abs(layers.int8_values(codes, absmax) - R.reshape(-1)).reshape(-1, 64)
    bound = 0.501 * step[:, None] + E.reshape(-1, 64) + eb[:, None] + 1e-30
    worst = float((off / bound).max()) if R.size else 0.0
    say(f"  {label} {key}: {worst:.3f} of its bound")
    assert worst <= 1.0, (label, key, worst)


def int8_of(api, x):
    """int8 values of a host matrix, on the device, and what they stand for."""
    c = api.qlora_int8_quantize(dev(np.asarray(x, np.float32)))
    return c, layers.int8_values(c[0].cpu().numpy(), c[1].cpu().numpy()).reshape(x.shape)


# ---- gated ------------------------------------------------------------------------------


class Gated:
    def __init__(self, api, M, K, F, r, seed=0, kind="silu", qtypes=("nf4", "nf4"), dq=(True, True), s=0.5):
        rng = np.random.default_rng(seed + 1000 * M + F)
        self.api, self.M, self.K, self.F, self.r, self.s, self.kind = api, M, K, F, r, s, kind
        self.q, self.W = [], []
        for qt, d in zip(qtypes, dq):
            q, _ = gpu_quantize(api, (rng.standard_normal((F, K)) / np.sqrt(K)).astype(np.float32), qtype=qt, double_quant=d)
            self.q.append(q)
            self.W.append(linear.widen(api.to_host_bits(api.qlora_dequantize(q))))
        self.X = bf16(rng.standard_normal((M, K)))
        self.L1 = bf16(rng.standard_normal((2, K, r)) / np.sqrt(K))
        self.L2 = bf16(rng.standard_normal((2, r, F)) * 0.5)
        self.dA = bf16(rng.standard_normal((M, F)))
        self.Xd, self.L1d, self.L2d, self.dAd = (dev(a) for a in (self.X, self.L1, self.L2, self.dA))

    def fwd(self, **kw):
        return self.api.qlora_gated_fwd(*self.q, self.Xd, self.L1d, self.L2d, self.s, act=self.kind, **kw)

    def bwd(self, X=None, **kw):
        return self.api.qlora_gated_bwd(*self.q, self.Xd if X is None else X, self.dAd, self.L1d, self.L2d, self.s,
                                        act=self.kind, **kw)

    def sums(self, X):
        """E(T), E(G), E(U) of the module's docstring."""
        aX, s = np.abs(X), abs(self.s)
        ET, E = [], []
        for k in range(2):
            L1, L2 = np.abs(linear.widen(self.L1[k])), np.abs(linear.widen(self.L2[k]))
            et = self.K * U * (aX @ L1)
            st = s * np.abs(X @ linear.widen(self.L1[k]))
            est = s * et + H * (st + s * et)
            base = aX @ np.abs(self.W[k]).T
            E.append((self.K * U + (2 * H if self.M <= 16 else 0.0)) * base + est @ L2 + self.r * U * ((st + est) @ L2))
            ET.append(et)
        return ET, E[0], E[1]


def act_errors(g, e, kind):
    """(act, act', E(act), E(act')) at g off by e."""
    a, d, z = layers.act(g, kind)
    f = (8 * np.abs(z) + 16) * U
    # sigmoid (1 - sigmoid) dz g: its factors are off by f each; where it is tiny its error is too
    return a, d, 1.13 * e + f * np.abs(a), 1.0 * e + f * (np.abs(d) + np.abs(d - 0.5) + 0.5)


SHAPES = [(1, 64, 8, 8), (1, 256, 136, 16), (2, 64, 72, 24), (16, 128, 64, 8), (17, 192, 200, 64), (33, 320, 128, 72),
          (100, 64, 16384, 8), (128, 64, 256, 8), (129, 64, 8, 8), (130, 128, 72, 16), (200, 256, 320, 136), (300, 64, 512, 64), (515, 192, 328, 40)]


@pytest.mark.parametrize("M,K,F,r", SHAPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_forward(api, M, K, F, r, kind):
    c = Gated(api, M, K, F, r, kind=kind)
    save = F % 64 == 0
    o = c.fwd(want_T=True, want_int8=save)
    X = linear.widen(c.X)
    A, G, Uv, T = layers.gated_fwd(c.X, *c.W, c.L1, c.L2, c.s, kind)
    ET, EG, EU = c.sums(X)
    label = f"gated fwd {M}x{K}x{F} r{r} {kind}"
    for k in range(2):
        within(label, f"T{k}", o.T[k], T[k], ET[k])
    a, _, Ea, _ = act_errors(G, EG, kind)
    within(label, "A", o.A, A, Ea * np.abs(Uv) + np.abs(a) * EU + Ea * EU + 2 * U * np.abs(A))
    if save:
        within_int8(label, "gate8", o.gate8, G, EG)
        within_int8(label, "up8", o.up8, Uv, EU)
        assert (c.fwd().A == o.A).all()            # keeping G and U does not change A


@pytest.mark.parametrize("K,F,r", [(256, 11272, 64), (4096, 2056, 24), (1024, 24, 8), (512, 8, 16), (8192, 520, 64)])
def test_gated_one_token(api, K, F, r):
    """Few features, uneven shares of them, and more than one round of workgroups holds."""
    c = Gated(api, 1, K, F, r)
    o = c.fwd(want_T=True)
    A, G, Uv, T = layers.gated_fwd(c.X, *c.W, c.L1, c.L2, c.s, c.kind)
    ET, EG, EU = c.sums(linear.widen(c.X))
    label = f"gated one token {K}x{F} r{r}"
    for k in range(2):
        within(label, f"T{k}", o.T[k], T[k], ET[k])
    a, _, Ea, _ = act_errors(G, EG, c.kind)
    within(label, "A", o.A, A, Ea * np.abs(Uv) + np.abs(a) * EU + Ea * EU + 2 * U * np.abs(A))


@pytest.mark.parametrize("M,K,F,r", SHAPES)
@pytest.mark.parametrize("keep", ["nothing", "T", "int8", "all8"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_backward(api, M, K, F, r, keep, kind):
    import torch

    if keep in ("int8", "all8") and F % 64:
        F = F // 64 * 64 + 64
    c = Gated(api, M, K, F, r, kind=kind, seed=7)
    X, kw, x_arg = linear.widen(c.X), {}, None
    ex = 0.0
    if keep == "all8":
        x_arg, X = int8_of(api, X)
        ex = H
    G, Uv, T = layers.gate_up(X, *c.W, c.L1, c.L2, c.s)
    if keep in ("int8", "all8"):
        (kw["gate8"], G), (kw["up8"], Uv) = int8_of(api, G), int8_of(api, Uv)
    if keep != "nothing":
        T = linear.widen(bf16(T))
        kw["T"] = dev(bf16(T))
    dX, dL1, dL2 = c.bwd(x_arg, grad_dtype=torch.float32 if M % 2 else torch.bfloat16, **kw)
    GU = (G, Uv) if keep in ("int8", "all8") else None
    RX, R1, R2, dG, dU = layers.gated_bwd(X, *c.W, c.L1, c.L2, c.s, kind, c.dA, GU)
    aX, s, dA = np.abs(X), abs(c.s), np.abs(linear.widen(c.dA))
    ET, EG, EU = c.sums(X)
    if GU is not None:
        EG, EU = 2 * U * np.abs(G), 2 * U * np.abs(Uv)
    a, d, Ea, Ed = act_errors(G, EG, kind)
    EdG = dA * (EU * np.abs(d) + np.abs(Uv) * Ed + EU * Ed) + 4 * U * np.abs(dG)
    EdU = dA * Ea + 2 * U * np.abs(dU)
    label = f"gated bwd {M}x{K}x{F} r{r} {kind} keep {keep}"
    EX = 0.0
    for k, (dY, e) in enumerate(((dG, EdG), (dU, EdU))):
        e = e + H * (np.abs(dY) + e)               # rounded to bf16 as an operand
        aY, L1, L2, W = np.abs(dY) + e, np.abs(linear.widen(c.L1[k])), np.abs(linear.widen(c.L2[k])), np.abs(c.W[k])
        sU = s * np.abs(dY @ linear.widen(c.L2[k]).T)
        EsU = s * (e @ L2.T + F * U * (aY @ L2.T))
        EsU = EsU + H * (sU + EsU)
        EX = EX + 2 * F * U * (aY @ W) + e @ W + EsU @ L1.T + r * U * ((sU + EsU) @ L1.T)
        within(label, f"dL1[{k}]", dL1[k], R1[k], aX.T @ EsU + (M * U + ex) * (aX.T @ (sU + EsU)))
        aT = np.abs(T[k])
        eT = np.zeros_like(aT) if keep != "nothing" else ET[k] + H * (aT + ET[k])
        if keep != "nothing":                      # dL2 of the given T, not of the oracle's X L1
            R2[k] = c.s * (T[k].T @ dY)
        within(label, f"dL2[{k}]", dL2[k], R2[k], s * (eT.T @ aY + aT.T @ e + M * U * (aT.T @ aY)))
    within(label, "dX", dX, RX, EX)
    got = c.bwd(x_arg, need_dX=False, grad_dtype=dL1.dtype, **kw)
    assert got[0] is None and (got[1] == dL1).all() and (got[2] == dL2).all()


@pytest.mark.parametrize("qtypes,dq", [(("nf4", "int4"), (True, True)), (("fp4_e2m1", "nf4"), (True, False)),
                                       (("int4", "fp4_e3m0"), (False, False))])
@pytest.mark.parametrize("M", [1, 20, 140])
def test_gated_data_types(api, qtypes, dq, M):
    c = Gated(api, M, 128, 192, 16, qtypes=qtypes, dq=dq, seed=3)
    A, G, Uv, _ = layers.gated_fwd(c.X, *c.W, c.L1, c.L2, c.s, "silu")
    _, EG, EU = c.sums(linear.widen(c.X))
    a, _, Ea, _ = act_errors(G, EG, "silu")
    within(f"gated {qtypes} M {M}", "A", c.fwd().A, A, Ea * np.abs(Uv) + np.abs(a) * EU + Ea * EU + 2 * U * np.abs(A))


def test_gated_large_arguments(api):
    """Gates far outside exp's range: act is 0 or g, its derivative 0 or 1."""
    import torch

    c = Gated(api, 4, 64, 64, 8)
    g = np.tile(np.array([-3e4, -200.0, -90.0, 90.0, 200.0, 3e4, 0.0, 1e-30], np.float32), (4, 8))
    g8, G = int8_of(api, g)
    u8, Uv = int8_of(api, np.ones((4, 64)))
    for kind in ("silu", "gelu"):
        c.kind = kind
        dX, dL1, dL2 = c.bwd(gate8=g8, up8=u8)
        RX = layers.gated_bwd(c.X, *c.W, c.L1, c.L2, c.s, kind, c.dA, (G, Uv))[0]
        assert torch.isfinite(dX).all() and torch.isfinite(dL1).all() and torch.isfinite(dL2).all()
        assert np.abs(host(dX)[0] - RX).max() <= 3e-2 * np.abs(RX).max()


@pytest.mark.parametrize("M", [3, 100, 300])
def test_gated_rows_are_apart(api, M):
    """A NaN or infinity in one row of X reaches no other row of A or dX."""
    import torch

    c = Gated(api, M, 128, 200, 16)
    A, dX = c.fwd().A, c.bwd()[0]
    c.Xd[M // 2, 5] = float("nan")
    c.Xd[M - 1, 7] = float("inf")
    A2, dX2 = c.fwd().A, c.bwd()[0]
    rest = torch.ones(M, dtype=torch.bool, device="cuda")
    rest[[M // 2, M - 1]] = False
    assert (A2[rest] == A[rest]).all() and (dX2[rest] == dX[rest]).all()
    assert torch.isnan(A2[M // 2]).all()


def test_gated_empty(api):
    import torch

    c = Gated(api, 4, 64, 64, 8)
    e = c.Xd[:0].contiguous()
    o = api.qlora_gated_fwd(*c.q, e, c.L1d, c.L2d, 1.0, want_T=True, want_int8=True)
    assert o.A.shape == (0, 64) and o.T.shape == (2, 0, 8) and o.gate8[0].numel() == 0
    for X in (e, (o.gate8[0], o.gate8[1])):
        dX, dL1, dL2 = api.qlora_gated_bwd(*c.q, X, c.dAd[:0].contiguous(), c.L1d, c.L2d, 1.0, grad_dtype=torch.bfloat16)
        assert dX.shape == (0, 64) and (dL1 == 0).all() and (dL2 == 0).all()


def test_gated_outputs_stay_inside(api):
    """Rows and features behind the last are left as they were."""
    import torch

    for M, F in ((1, 72), (20, 72), (130, 72)):
        c = Gated(api, M, 64, F, 8)
        buf = torch.full((M * F + 512,), 7.0, dtype=torch.bfloat16, device="cuda")
        c.fwd(A=buf[256:256 + M * F].view(M, F))
        assert (buf[:256] == 7).all() and (buf[256 + M * F:] == 7).all()
        buf = torch.full((M * 64 + 512,), 7.0, dtype=torch.bfloat16, device="cuda")
        c.bwd(dX=buf[256:256 + M * 64].view(M, 64))
        assert (buf[:256] == 7).all() and (buf[256 + M * 64:] == 7).all()


# ---- the linear's backward pass from 8 bits -----------------------------------------------------


@pytest.mark.parametrize("M,K,N,r", [(1, 64, 8, 8), (5, 128, 72, 16), (64, 256, 128, 64), (300, 192, 320, 72), (130, 64, 512, 24)])
def test_linear_bwd_int8(api, M, K, N, r):
    import torch

    rng = np.random.default_rng(M + N)
    q, _ = gpu_quantize(api, (rng.standard_normal((N, K)) / np.sqrt(K)).astype(np.float32))
    W = linear.widen(api.to_host_bits(api.qlora_dequantize(q)))
    L1, L2, dY = bf16(rng.standard_normal((K, r)) / np.sqrt(K)), bf16(rng.standard_normal((r, N))), bf16(rng.standard_normal((M, N)))
    L1d, L2d, dYd, s = dev(L1), dev(L2), dev(dY), 0.75
    X8, X = int8_of(api, rng.standard_normal((M, K)))
    T = bf16(X @ linear.widen(L1))
    aX, a1, a2, aY, aW = np.abs(X), *(np.abs(linear.widen(v)) for v in (L1, L2, dY)), np.abs(W)
    for t in (None, T):
        got = api.qlora_linear_bwd_int8(q, X8, dYd, L1d, L2d, s, T=None if t is None else dev(t))
        RX, R1, R2 = linear.linear_bwd(X, W, L1, L2, s, dY)
        if t is not None:
            R2 = s * (linear.widen(T).T @ linear.widen(dY))
        sU = s * np.abs(linear.widen(dY) @ linear.widen(L2).T)
        EsU = s * N * U * (aY @ a2.T)
        EsU = EsU + H * (sU + EsU)
        label = f"linear int8 {M}x{K}x{N} r{r} T {'given' if t is not None else 'computed'}"
        within(label, "dX", got[0], RX, 2 * N * U * (aY @ aW) + EsU @ a1.T + r * U * ((sU + EsU) @ a1.T)
               + (2 * H * (aY @ aW) if M <= 16 or N % 64 else 0.0))
        within(label, "dL1", got[1], R1, aX.T @ EsU + (M * U + H) * (aX.T @ (sU + EsU)))
        eT = np.zeros((M, r)) if t is not None else (K * U + H) * (aX @ a1) + H * np.abs(X @ linear.widen(L1))
        within(label, "dL2", got[2], R2, s * (eT.T @ aY + M * U * ((aX @ a1).T @ aY)))
        no = api.qlora_linear_bwd_int8(q, X8, dYd, L1d, L2d, s, T=None if t is None else dev(t), need_dX=False)
        assert no[0] is None and (no[1] == got[1]).all()
        again = api.qlora_linear_bwd_int8(q, X8, dYd, L1d, L2d, s, T=None if t is None else dev(t))
        assert all((a == b).all() for a, b in zip(got, again))
    b = torch.bfloat16
    d = api.qlora_linear_bwd_int8(q, X8, dYd, L1d, L2d, s, grad_dtype=b)
    assert d[1].dtype == b and d[2].dtype == b
    e = api.qlora_linear_bwd_int8(q, (X8[0][:0], X8[1][:0]), dYd[:0], L1d, L2d, s)
    assert e[0].shape == (0, K) and (e[1] == 0).all() and (e[2] == 0).all()


# ---- norm ---------------------------------------------------------------------------------------


@pytest.mark.parametrize("M,K", [(1, 8), (3, 64), (5, 72), (4, 1000), (7, 2048), (3, 2056), (300, 4096), (9, 6656), (2, 8192),
                                 (3, 8200), (2, 16384), (4099, 64)])
@pytest.mark.parametrize("x32,res,weight", [(False, "f32", "bf16"), (False, "bf16", "f32"), (True, None, "bf16"), (False, None, None)])
def test_norm(api, M, K, x32, res, weight):
    import torch

    rng = np.random.default_rng(K + M)
    make = lambda shape, f32: rng.standard_normal(shape).astype(np.float32) if f32 else bf16(rng.standard_normal(shape))  # noqa: E731
    x = make((M, K), x32)
    r = None if res is None else make((M, K), res == "f32")
    w = None if weight is None else make((K,), weight == "f32")
    eps = 1e-5
    t = lambda a: None if a is None else dev(a)  # noqa: E731
    save = K % 64 == 0
    o = api.qlora_norm_fwd(t(x), t(w), eps=eps, residual=t(r), want_int8=save)
    y, h, rstd = layers.norm_fwd(x, r, w, eps)
    label = f"norm {M}x{K} {x32} {res} {weight}"
    E = (K / 2 + 8) * U * np.abs(y) + (2 * U * np.abs(rstd[:, None] * h) * (1 if w is None else np.abs(linear.widen(w))))
    within(label, "y", o.y, y, E)
    within(label, "rstd", o.rstd, rstd, (K / 2 + 6) * U * rstd)
    within(label, "h", o.h, h, U * np.abs(h))
    if save:
        within_int8(label, "int8", o.int8, y, E)
        only = api.qlora_norm_fwd(t(x), t(w), eps=eps, residual=t(r), want_y=False, want_int8=True)
        assert only.y is None and (only.int8[0] == o.int8[0]).all() and (only.int8[1] == o.int8[1]).all()
    if r is not None:                              # in place on the residual stream
        stream = t(r)
        i = api.qlora_norm_fwd(t(x), t(w), eps=eps, residual=stream, h=stream)
        assert i.h is stream and (stream == o.h).all() and (i.y == o.y).all()
    # backward, from the rounded h and the fp32 rstd that the forward pass left
    hb, rb = host(o.h)[0], host(o.rstd)[0]
    dy = bf16(rng.standard_normal((M, K)))
    for dres in (None, rng.standard_normal((M, K)).astype(np.float32)):
        if dres is not None and o.h.dtype == torch.bfloat16:
            dres = bf16(dres)
        g = api.qlora_norm_bwd(t(dy), o.h, o.rstd, t(w), dres=t(dres), want_dx16=True)
        dh, dw = layers.norm_bwd(dy, hb, rb, w, dres)
        xh, wd = np.abs(hb) * rb[:, None], np.abs(linear.widen(dy)) * (1 if w is None else np.abs(linear.widen(w)))
        mean = (wd * xh).mean(axis=1, keepdims=True)
        Eh = rb[:, None] * (4 * U * wd + (K + 8) * U * xh * mean) + 2 * U * (np.abs(dh) + (0 if dres is None else np.abs(linear.widen(dres))))
        within(label, "dh", g.dh, dh, Eh)
        within(label, "dx16", g.dx16, dh, Eh)
        within(label, "dweight", g.dweight, dw, (M + 6) * U * (np.abs(linear.widen(dy)) * xh).sum(axis=0))
        no = api.qlora_norm_bwd(t(dy), o.h, o.rstd, t(w), dres=t(dres), need_dweight=False)
        assert no.dweight is None and no.dx16 is None and (no.dh == g.dh).all()
        if dres is not None:                       # in place
            d = t(dres)
            assert (api.qlora_norm_bwd(t(dy), o.h, o.rstd, t(w), dres=d, dh=d).dh == g.dh).all()


def test_norm_edges(api):
    import torch

    x = torch.zeros(5, 64, dtype=torch.bfloat16, device="cuda")
    o = api.qlora_norm_fwd(x, want_int8=True)
    assert (o.y == 0).all() and (o.int8[0] == 0).all() and torch.isfinite(o.rstd).all()
    x[1, 3], x[2, 5] = float("nan"), float("inf")
    x[3] = 2.0
    o = api.qlora_norm_fwd(x, want_int8=True)
    assert torch.isnan(o.y[1]).all() and (o.y[0] == 0).all() and (o.y[4] == 0).all() and (o.y[3] == 1).all()
    e = api.qlora_norm_fwd(x[:0], want_int8=True)
    g = api.qlora_norm_bwd(x[:0], e.h, e.rstd)
    assert e.y.shape == (0, 64) and g.dh.shape == (0, 64) and (g.dweight == 0).all()


# ---- loss over the vocabulary ----------------------------------------------------------------------


def head_case(M, K, V, seed=0, lift=1.0):
    rng = np.random.default_rng(seed + V + M)
    W = bf16(rng.standard_normal((V, K)) * (2.0 / np.sqrt(K)))
    labels = rng.integers(0, V, M)
    Hs = bf16(rng.standard_normal((M, K)) + lift * rng.random((M, 1)) * linear.widen(W)[labels])
    return Hs, W, labels.astype(np.int64), rng


def check_head(label, o, Hs, W, labels, weights=None, div=0.0, scale=1.0):
    M, K = Hs.shape
    V = W.shape[0]
    loss, nll, dH, dW, p, g = layers.head_loss(Hs, W, labels, weights, div, scale)
    h, w = linear.widen(Hs), linear.widen(W)
    on = (labels >= 0) & (labels < V)
    at = np.where(on, labels, 0)
    S, ES = h @ w.T, K * U * (np.abs(h) @ np.abs(w).T)
    sy = np.take_along_axis(S, at[:, None], 1)
    e = ES + np.take_along_axis(ES, at[:, None], 1) + (2 * np.abs(S - sy) + 8) * U       # relative, of each P
    q = p.copy()
    np.put_along_axis(q, at[:, None], 0.0, 1)
    rest = q.sum(axis=1, keepdims=True)                  # 1 - p_y
    el = (q * e).sum(axis=1, keepdims=True) / np.maximum(rest, 1e-300) + (V / 64 + 20) * U    # relative, of l
    q_all = q.copy()
    np.put_along_axis(q_all, at[:, None], rest, 1)
    e_all = e.copy()
    np.put_along_axis(e_all, at[:, None], el, 1)
    En = (rest * el)[:, 0] + 8 * U * (1 + np.abs(nll))
    En = np.where(on, En, 0.0)
    within(label, "nll", o.nll, nll, En)
    wt = np.where(on, 1.0 if weights is None else weights, 0.0) / (div or max(int(on.sum()), 1))
    within(label, "loss", o.loss, np.array([loss]), np.array([(np.abs(wt) * En).sum()]) + U * abs(loss))
    er = np.where(on[:, None], np.abs(g)[:, None] * q_all * (e_all + H + el * rest + 8 * U), 0.0)
    aq = np.where(on[:, None], np.abs(g)[:, None] * q_all, 0.0)
    if o.dH is not None:
        within(label, "dH", o.dH, dH, er @ np.abs(w) + V * U * (aq @ np.abs(w)))
        assert (host(o.dH)[0][~on] == 0).all()
    if o.dW is not None:
        within(label, "dW", o.dW, dW, (er + (H + M * U) * 1.01 * aq).T @ np.abs(h))
    assert (host(o.nll)[0][~on] == 0).all()


HEADS = [(1, 64, 1), (1, 64, 5), (2, 128, 64), (5, 64, 257), (48, 192, 1000), (130, 256, 1025), (300, 64, 3001), (257, 320, 515),
         (600, 128, 32001)]


@pytest.mark.parametrize("M,K,V", HEADS)
@pytest.mark.parametrize("dW", [None, "f32", "bf16"])
def test_head_loss(api, M, K, V, dW):
    import torch

    Hs, W, labels, rng = head_case(M, K, V)
    kw = dict(need_dW=dW is not None, grad_dtype=torch.bfloat16 if dW == "bf16" else torch.float32)
    label = f"head {M}x{K}x{V} dW {dW}"
    o = api.qlora_head_loss(dev(Hs), dev(W), dev(labels), **kw)
    check_head(label, o, Hs, W, labels)
    some = labels.copy()
    some[rng.random(M) < 0.4] = -100
    if M > 2:
        some[1], some[2] = V, -1
    weights = rng.random(M).astype(np.float32)
    o = api.qlora_head_loss(dev(Hs), dev(W), dev(some), weights=dev(weights), divisor=3.5, grad_scale=0.5, **kw)
    check_head(label + " some", o, Hs, W, some, weights, 3.5, 0.5)
    alone = api.qlora_head_loss(dev(Hs), dev(W), dev(some), weights=dev(weights), divisor=3.5, need_dH=False)
    assert alone.dH is None and alone.dW is None and (alone.nll == o.nll).all() and (alone.loss == o.loss).all()


@pytest.mark.parametrize("M,K,V,masked", [(2049, 64, 300, 0.0), (2500, 128, 700, 0.3), (3000, 64, 1000, 0.97), (2100, 128, 9000, 0.5),
                                          (4200, 64, 9000, 0.9)])
def test_head_many_rows(api, M, K, V, masked):
    """Rows counted by one workgroup; fewer counted rows than the grids are for, dH in slices planned from their number."""
    Hs, W, labels, rng = head_case(M, K, V)
    labels[rng.random(M) < masked] = -100
    o = api.qlora_head_loss(dev(Hs), dev(W), dev(labels), need_dW=True)
    check_head(f"head {M}x{K}x{V} masked {masked}", o, Hs, W, labels)


def test_head_no_counted_row(api):
    import torch

    Hs, W, labels, _ = head_case(70, 64, 300)
    labels[:] = -100
    Hd = dev(Hs)
    Hd[3] = float("nan")                              # not used
    o = api.qlora_head_loss(Hd, dev(W), dev(labels), need_dW=True)
    assert o.loss.item() == 0 and (o.nll == 0).all() and (o.dH == 0).all() and (o.dW == 0).all()
    e = api.qlora_head_loss(Hd[:0], dev(W), dev(labels)[:0], need_dW=True, grad_dtype=torch.bfloat16)
    assert e.loss.item() == 0 and e.dH.shape == (0, 64) and (e.dW == 0).all()


@pytest.mark.parametrize("gap", [30.0, 60.0, 200.0, 3000.0])
def test_head_labels_of_no_probability(api, gap):
    """Labels far below the largest logit, in all tiles or one: the tiles take their row's maximum out."""
    import torch

    Hs, W, labels, rng = head_case(140, 64, 1100, seed=5)
    h = linear.widen(Hs)
    h[:, 0] = 1.0
    w = linear.widen(W)
    w[:, 0] = 0.0
    w[300:310, 0] = gap                                # ten columns of the second tile far above the rest
    w[900, 0] = gap + 5.0
    Hs, W = bf16(h), bf16(w)
    labels = np.where((labels >= 300) & (labels < 310) | (labels == 900), 7, labels)
    labels[:5] = 305                                   # and labels among them
    labels[5] = 900
    o = api.qlora_head_loss(dev(Hs), dev(W), dev(labels), need_dW=True)
    assert all(torch.isfinite(t).all() for t in o)
    check_head(f"head gap {gap}", o, Hs, W, labels)


def test_head_confident_labels(api):
    """Labels of nearly all probability: the gradient p - 1 has no cancellation."""
    Hs, W, labels, _ = head_case(140, 64, 700, seed=6, lift=8.0)
    o = api.qlora_head_loss(dev(Hs), dev(W), dev(labels), need_dW=True)
    check_head("head confident", o, Hs, W, labels)


@pytest.mark.parametrize("M", [3, 200])
def test_head_rows_are_apart(api, M):
    """A NaN or infinity in one row of H reaches no other row of nll or dH."""
    import torch

    Hs, W, labels, _ = head_case(M, 128, 900)
    Hd, Wd, Ld = dev(Hs), dev(W), dev(labels)
    a = api.qlora_head_loss(Hd, Wd, Ld)
    Hd[1, 3], Hd[M - 1, 0] = float("nan"), float("inf")
    b = api.qlora_head_loss(Hd, Wd, Ld)
    rest = torch.ones(M, dtype=torch.bool, device="cuda")
    rest[[1, M - 1]] = False
    assert (a.nll[rest] == b.nll[rest]).all() and (a.dH[rest] == b.dH[rest]).all()
    assert torch.isnan(b.nll[1]) and torch.isnan(b.dH[1]).all() and torch.isnan(b.loss).all()


@pytest.mark.parametrize("dW", ["f32", "bf16"])
def test_head_pieces(api, dW):
    """More rows than one piece holds, some pieces without a counted row."""
    import torch

    M, K, V = 1100, 64, 1 << 20                       # pieces of 512 rows
    g = torch.Generator(device="cuda").manual_seed(1)
    Hd = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g)
    Wd = torch.empty(V, K, dtype=torch.bfloat16, device="cuda").normal_(0, 0.25, generator=g)
    Ld = torch.randint(0, V, (M,), device="cuda", generator=g)
    kw = dict(need_dW=True, grad_dtype=torch.bfloat16 if dW == "bf16" else torch.float32)
    for some in (Ld, torch.where(torch.arange(M, device="cuda") % 5 == 0, Ld, -100)):
        o = api.qlora_head_loss(Hd, Wd, some, **kw)
        on = some >= 0
        n = int(on.sum())
        h, w = Hd[on].double(), Wd.double()
        logp = torch.log_softmax(h @ w.T, 1)
        y = some[on]
        nll = -logp[torch.arange(n, device="cuda"), y]
        # logits off by K u |H||W| < 64 2^-24 30, twice, and the sums' roundings: 1e-4 is well above
        assert (o.nll[on].double() - nll).abs().max() < 1e-4 and (o.nll[~on] == 0).all()
        assert abs(o.loss.item() - nll.mean().item()) < 1e-4
        D = logp.exp_()
        D[torch.arange(n, device="cuda"), y] -= 1.0
        D /= n
        # every term is rounded to bf16 once as an operand (dW: both operands), outputs once: 2-norms within 2^-8 each
        dH = torch.zeros(M, K, dtype=torch.float64, device="cuda")
        dH[on] = D @ w
        assert (o.dH.double() - dH).norm() <= 2 * H * dH.norm()
        RW = D.T @ h
        assert (o.dW.double() - RW).norm() <= 3 * H * RW.norm()
        del logp, D, RW


# ---- offsets that pass 32 bits ---------------------------------------------------------------------


def rows_near(big, small, at, label):
    """Rows of a large call beside a small call on them: the same products, in sums of another order, so every rounding to
    bf16 (the adapters' operand, the outputs) may fall the other way: 2-norms within three of them."""
    d = (big[at:at + small.shape[0]].double() - small.double()).norm()
    assert d <= 3 * H * small.double().norm(), (label, at, float(d))


PLACES = (0, 131000, (1 << 18) - 300)


def normal(shape, seed, std=1.0, dtype=None):
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=dtype or torch.bfloat16, device="cuda").normal_(0, std, generator=g)


def test_gated_long(api):
    import torch

    M, K, F, r, s = 1 << 18, 64, 8256, 8, 0.5
    rng = np.random.default_rng(0)
    q = [gpu_quantize(api, (rng.standard_normal((F, K)) / 8).astype(np.float32))[0] for _ in range(2)]
    X, dA = normal((M, K), 1), normal((M, F), 2)
    L1, L2 = normal((2, K, r), 3, 0.125), normal((2, r, F), 4, 0.5)
    o = api.qlora_gated_fwd(*q, X, L1, L2, s, want_T=True, want_int8=True)
    for at in PLACES:
        m = slice(at, at + 300)
        t = api.qlora_gated_fwd(*q, X[m], L1, L2, s, want_T=True, want_int8=True)
        rows_near(o.A, t.A, at, "A")
        rows_near(o.T[1], t.T[1], at, "T")
        rows_near(o.up8[1].view(M, -1), t.up8[1].view(300, -1), at, "up8 absmax")
        # codes are off by one where G is rounded the other way
        assert (o.gate8[0].view(M, F)[m].int() - t.gate8[0].view(300, F).int()).abs().max() <= 1
    full = api.qlora_gated_bwd(*q, X, dA, L1, L2, s)
    kept = api.qlora_gated_bwd(*q, X, dA, L1, L2, s, T=o.T, gate8=o.gate8, up8=o.up8)
    sums = [[torch.zeros_like(full[i], dtype=torch.float64) for i in (1, 2)] for _ in range(2)]
    P = M // 8
    for m in range(0, M, P):
        g8, u8 = (tuple(v.view(M, -1)[m:m + P].reshape(-1) for v in w) for w in (o.gate8, o.up8))
        for k, part in enumerate((api.qlora_gated_bwd(*q, X[m:m + P], dA[m:m + P], L1, L2, s),
                                  api.qlora_gated_bwd(*q, X[m:m + P], dA[m:m + P], L1, L2, s, gate8=g8, up8=u8,
                                                      T=o.T[:, m:m + P].contiguous()))):
            rows_near((full, kept)[k][0], part[0], m, f"dX {k}")
            for i in range(2):
                sums[k][i] += part[1 + i].double()
    for k, got in enumerate((full, kept)):
        for i in range(2):
            assert (got[1 + i].double() - sums[k][i]).norm() <= 3 * H * sums[k][i].norm(), (k, i)
    del o, full, kept
    torch.cuda.empty_cache()


@pytest.mark.parametrize("K,N", [(64, 8200), (8256, 64)])
def test_linear_bwd_int8_long(api, K, N):
    import torch

    M, r, s = 1 << 18, 8, 0.5
    rng = np.random.default_rng(0)
    q, _ = gpu_quantize(api, (rng.standard_normal((N, K)) / np.sqrt(K)).astype(np.float32))
    X8 = api.qlora_int8_quantize(normal((M, K), 1))
    dY, L1, L2 = normal((M, N), 2), normal((K, r), 3, K ** -0.5), normal((r, N), 4)
    full = api.qlora_linear_bwd_int8(q, X8, dY, L1, L2, s)
    sums = [torch.zeros_like(full[i], dtype=torch.float64) for i in (1, 2)]
    P = M // 8
    for m in range(0, M, P):
        x8 = tuple(v.view(M, -1)[m:m + P].reshape(-1) for v in X8)
        part = api.qlora_linear_bwd_int8(q, x8, dY[m:m + P], L1, L2, s)
        rows_near(full[0], part[0], m, "dX")
        for i in range(2):
            sums[i] += part[1 + i].double()
    for i in range(2):
        assert (full[1 + i].double() - sums[i]).norm() <= 3 * H * sums[i].norm(), i
    del X8, dY, full
    torch.cuda.empty_cache()


def test_norm_long(api):
    """Rows do not depend on their number: the same bits."""
    import torch

    M, K = 1 << 18, 8256
    x, res, w = normal((M, K), 1), normal((M, K), 2, dtype=torch.float32), normal((K,), 3)
    o = api.qlora_norm_fwd(x, w, residual=res, want_int8=True)
    g = api.qlora_norm_bwd(x, o.h, o.rstd, w, dres=res, want_dx16=True)
    dw = torch.zeros(K, dtype=torch.float64, device="cuda")
    for at in PLACES:
        m = slice(at, at + 300)
        t = api.qlora_norm_fwd(x[m], w, residual=res[m], want_int8=True)
        b = api.qlora_norm_bwd(x[m], t.h, t.rstd, w, dres=res[m], want_dx16=True)
        for big, small in ((o.y, t.y), (o.h, t.h), (o.rstd, t.rstd), (o.int8[0].view(M, K), t.int8[0].view(300, K)),
                           (o.int8[1].view(M, -1), t.int8[1].view(300, -1)), (g.dh, b.dh), (g.dx16, b.dx16)):
            assert (big[m] == small).all()
    P = M // 8
    for m in range(0, M, P):
        dw += api.qlora_norm_bwd(x[m:m + P], o.h[m:m + P], o.rstd[m:m + P], w).dweight.double()
    # a thread adds M / 1024 products, then the groups' sums are added: (M / 1024 + 1024) u of the magnitudes, whose sum
    # is M E|dy||xh| < M against a result of about sqrt(M) per column
    assert (g.dweight.double() - dw).abs().max() <= (M / 1024 + 1024) * U * M
    del x, res, o, g
    torch.cuda.empty_cache()


def test_head_long_rows(api):
    import torch

    M, K, V = 1 << 18, 8256, 70
    Hd, Wd = normal((M, K), 1), normal((V, K), 2, 0.02)
    Ld = torch.randint(-20, V, (M,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    o = api.qlora_head_loss(Hd, Wd, Ld, divisor=1.0, need_dW=True)
    loss, dW = 0.0, torch.zeros(V, K, dtype=torch.float64, device="cuda")
    P = M // 8
    for m in range(0, M, P):
        t = api.qlora_head_loss(Hd[m:m + P], Wd, Ld[m:m + P], divisor=1.0, need_dW=True)
        rows_near(o.dH, t.dH, m, "dH")
        # logits in the same order; the statistics' too
        assert (o.nll[m:m + P] == t.nll).all()
        loss += t.loss.item()
        dW += t.dW.double()
    assert abs(o.loss.item() - loss) <= 8 * U * abs(loss)
    assert (o.dW.double() - dW).norm() <= 3 * H * dW.norm()
    del Hd, o
    torch.cuda.empty_cache()


def test_head_long_vocabulary(api):
    import torch

    M, K, V = 130, 4160, 1 << 19
    Hd, Wd = normal((M, K), 1), normal((V, K), 2, 0.02)
    Ld = torch.randint(0, V, (M,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    Ld[0], Ld[1] = V - 1, 0
    o = api.qlora_head_loss(Hd, Wd, Ld, need_dW=True)
    h, C = Hd.double(), 1 << 16
    S = torch.cat([h @ Wd[v:v + C].double().t().contiguous() for v in range(0, V, C)], 1)
    nll = torch.logsumexp(S, 1) - S[torch.arange(M), Ld]
    # logits off by K u |H||W| < 4160 2^-24 4160 0.016, taken loosely; their mean over the vocabulary by far less
    assert (o.nll.double() - nll).abs().max() < 1e-2
    D = torch.softmax(S, 1)
    D[torch.arange(M), Ld] -= 1.0
    D /= M
    dH = sum(D[:, v:v + C] @ Wd[v:v + C].double() for v in range(0, V, C))
    assert (o.dH.double() - dH).norm() <= 3 * H * dH.norm()
    for v in range(0, V, C):
        R = D[:, v:v + C].t().contiguous() @ h
        assert (o.dW[v:v + C].double() - R).norm() <= 3 * H * R.norm(), v
    del Wd, o, S, D
    torch.cuda.empty_cache()


# ---- as they are used ----------------------------------------------------------------------------


def test_same_bits_again(api):
    """Repeated calls, a caller's dirty workspace and another stream give the same bits."""
    import torch

    c = Gated(api, 150, 128, 192, 16)
    Hs, W, labels, _ = head_case(150, 128, 900)
    Hd, Wd, Ld = dev(Hs), dev(W), dev(labels)

    def all_of(fill=None, stream=None):
        ws = lambda n: None if fill is None else torch.full((n,), fill, dtype=torch.uint8, device="cuda")  # noqa: E731
        o = c.fwd(want_T=True, want_int8=True, workspace=ws(api.qlora_gated_workspace(150, 128, 192, 16)), stream=stream)
        b = c.bwd(T=o.T, gate8=o.gate8, up8=o.up8, workspace=ws(api.qlora_gated_workspace(150, 128, 192, 16, True)), stream=stream)
        b2 = c.bwd(workspace=ws(api.qlora_gated_workspace(150, 128, 192, 16, True)), stream=stream)
        n = api.qlora_norm_fwd(c.Xd, residual=c.Xd, want_int8=True, stream=stream)
        nb = api.qlora_norm_bwd(c.Xd, n.h, n.rstd, workspace=ws(api.qlora_norm_workspace(150, 128)), stream=stream)
        hl = api.qlora_head_loss(Hd, Wd, Ld, need_dW=True, stream=stream,
                                 workspace=ws(api.qlora_head_workspace(150, 128, 900, True, True)))
        torch.cuda.synchronize()
        return [o.A, o.T, *o.gate8, *o.up8, *b, *b2, n.y, n.h, n.rstd, *n.int8, nb.dh, nb.dweight, *hl]

    ref = all_of()
    for got in (all_of(), all_of(fill=255), all_of(fill=0x7F), all_of(stream=torch.cuda.Stream())):
        assert all((a == b).all() for a, b in zip(ref, got))


def test_a_workspace_of_more_rows(api):
    """One of the largest batch's size serves smaller ones, with the same bits."""
    import torch

    K, F, r, V, most = 128, 192, 16, 900, 700

    def ws(n):
        return torch.full((n,), 255, dtype=torch.uint8, device="cuda")

    w = [ws(api.qlora_gated_workspace(most, K, F, r)), ws(api.qlora_gated_workspace(most, K, F, r, True)),
         ws(api.qlora_linear_bwd_int8_workspace(most, K, F, r)), ws(api.qlora_norm_workspace(most, K)),
         ws(api.qlora_head_workspace(most, K, V, True, True))]
    for M in (1, 7, 128, 129, 400, 700):
        c = Gated(api, M, K, F, r)
        Hs, W, labels, _ = head_case(M, K, V)
        x8 = api.qlora_int8_quantize(c.Xd)
        rstd = torch.ones(M, device="cuda")
        ref, got = ([c.fwd(workspace=v[0]).A, *c.bwd(workspace=v[1]),
                     *api.qlora_linear_bwd_int8(c.q[0], x8, c.dAd, c.L1d[0].contiguous(), c.L2d[0].contiguous(), 0.5, workspace=v[2]),
                     api.qlora_norm_bwd(c.Xd, c.Xd, rstd, workspace=v[3]).dweight,
                     *api.qlora_head_loss(dev(Hs), dev(W), dev(labels), need_dW=True, workspace=v[4])] for v in ([None] * 5, w))
        assert all((a == b).all() for a, b in zip(ref, got)), M


def test_arguments_by_name_and_place(api):
    import torch

    x = normal((5, 64), 1)
    w, labels, other = normal((9, 64), 2), torch.tensor([1, 8, -1, 9, 0], device="cuda"), torch.cuda.Stream()
    a, b = api.qlora_norm_fwd(x), api.qlora_norm_fwd(x=x, weight=None)
    torch.cuda.synchronize()
    c = api.qlora_norm_fwd(x, None, 1e-6, None, True, False, None, None, None, other)
    d, e = api.qlora_head_loss(x, w, labels), api.qlora_head_loss(labels=labels, W=w, H=x, stream=other)
    torch.cuda.synchronize()
    assert (a.y == b.y).all() and (a.y == c.y).all() and (d.dH == e.dH).all() and (d.loss == e.loss).all()


@pytest.mark.parametrize("M", [1, 40, 200])
def test_training_step_in_a_graph(api, M):
    """Norm, gated block, down projection, norm and loss, forward and backward, captured once and replayed on new
    inputs with eager work between: the same bits as the eager calls."""
    import torch

    K, F, r, V, s = 128, 192, 16, 500, 0.5
    c = Gated(api, M, K, F, r)
    rng = np.random.default_rng(5)
    down, _ = gpu_quantize(api, (rng.standard_normal((K, F)) / np.sqrt(F)).astype(np.float32))
    D1, D2 = dev(bf16(rng.standard_normal((F, r)) / np.sqrt(F))), dev(bf16(rng.standard_normal((r, K)) * 0.1))
    Wd = dev(bf16(rng.standard_normal((V, K)) * 0.1))
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    stream = torch.empty(M, K, dtype=torch.float32, device="cuda")
    labels = torch.empty(M, dtype=torch.int64, device="cuda")

    def step():
        n1 = api.qlora_norm_fwd(x, residual=stream, want_int8=True)
        o = api.qlora_gated_fwd(*c.q, n1.y, c.L1d, c.L2d, s, want_T=True, want_int8=True)
        a8 = api.qlora_int8_quantize(o.A)
        Y, T = api.qlora_linear_fwd(down, o.A, D1, D2, s, want_T=True)
        n2 = api.qlora_norm_fwd(Y, residual=n1.h)
        loss = api.qlora_head_loss(n2.y, Wd, labels, need_dW=True)
        g2 = api.qlora_norm_bwd(loss.dH, n2.h, n2.rstd, want_dx16=True)
        dA, dD1, dD2 = api.qlora_linear_bwd_int8(down, a8, g2.dx16, D1, D2, s, T=T)
        dX, dL1, dL2 = api.qlora_gated_bwd(*c.q, n1.int8, dA, c.L1d, c.L2d, s, T=o.T, gate8=o.gate8, up8=o.up8)
        g1 = api.qlora_norm_bwd(dX, n1.h, n1.rstd, dres=g2.dh, want_dx16=True)
        return [loss.loss, loss.nll, loss.dW, dD1, dD2, dL1, dL2, g1.dh, g1.dx16, g1.dweight]

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.normal_(generator=g)
        stream.normal_(generator=g)
        labels.copy_(torch.randint(-50, V, (M,), device="cuda", generator=g))
        if seed == 2:
            labels.fill_(-100)

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2, 3, 4):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        ref = step()
        torch.cuda.synchronize()
        assert all((a == b).all() for a, b in zip(got, ref)), seed
        assert all(torch.isfinite(t).all() for t in got)


def test_binding_refusals(api):
    import torch

    c = Gated(api, 4, 64, 64, 8)
    x8 = api.qlora_int8_quantize(c.Xd)
    with pytest.raises(ValueError, match="shape"):
        c.fwd(A=torch.empty(4, 72, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        api.qlora_gated_fwd(*c.q, c.Xd.float(), c.L1d, c.L2d, 1.0)
    with pytest.raises(ValueError, match="device"):
        api.qlora_gated_fwd(*c.q, c.Xd.cpu(), c.L1d, c.L2d, 1.0)
    with pytest.raises(ValueError, match="act"):
        api.qlora_gated_fwd(*c.q, c.Xd, c.L1d, c.L2d, 1.0, act="relu")
    with pytest.raises(ValueError, match="contiguous"):
        api.qlora_gated_fwd(*c.q, c.Xd.t().contiguous().t(), c.L1d, c.L2d, 1.0)
    with pytest.raises(ValueError, match="together"):
        c.bwd(gate8=x8)
    with pytest.raises(ValueError, match="workspace"):
        c.fwd(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError, match="pair"):
        api.qlora_linear_bwd_int8(c.q[0], x8[0], c.dAd, c.L1d[0], c.L2d[0], 1.0)
    with pytest.raises(ValueError, match="shape"):
        api.qlora_linear_bwd_int8(c.q[0], (x8[0][:64], x8[1]), c.dAd, c.L1d[0], c.L2d[0], 1.0)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        api.qlora_norm_fwd(c.Xd.half())
    with pytest.raises(ValueError, match="multiple of 64"):
        api.qlora_norm_fwd(c.Xd[:, :40].contiguous(), want_int8=True)
    with pytest.raises(ValueError, match="residual"):
        api.qlora_norm_fwd(c.Xd, h=c.Xd)
    with pytest.raises(TypeError):
        api.qlora_head_loss(c.Xd, c.Xd, torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        api.qlora_head_loss(c.Xd, c.Xd[:, :32].contiguous(), torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(api.QLoRAError):
        api.qlora_head_loss(c.Xd, c.Xd, torch.zeros(4, dtype=torch.int64, device="cuda"), divisor=-1.0)
