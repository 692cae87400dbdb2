"""The layer operators' optional inputs, each with and without the others, against
the float64 oracle, and the bounds of tests/test_gpu_layers.py without the
allowance for a weight's neighbouring bf16 where no kernel needs it.

Only a single token of rank <= 64 with K a multiple of 256, both weights
double-quantised in one data type and nothing kept takes the code values from a
table in fp16 (off by 2^-11 of the value, so that the weight's rounding to bf16 may
fall to the neighbour: 2 h |X||W|). Everything else multiplies the fp32 code value
by its block constant and rounds once, which is the oracle's weight bit for bit.

An input in 8 bits is rounded to bf16 as an operand, one rounding of a value that
the codes give exactly, so the oracle takes the rounded values and no bound grows.
Given T, gate and up are independent of X here: what a call is given is what it
has to use.
"""

import numpy as np
import pytest

from gpu_util import gpu_quantize, require_gpu
from oracle import layers, linear
from test_gpu_layers import H, U, Gated, act_errors, bf16, check_head, dev, head_case, int8_of, within, within_int8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    return require_gpu()


def gate_up_errors(c, X, fp16_table=False):
    """(E(T), E(G), E(U)) of the bounds' derivation in test_gpu_layers.py."""
    aX, s = np.abs(X), abs(c.s)
    ET, E = [], []
    for k in range(2):
        L1, L2 = np.abs(linear.widen(c.L1[k])), np.abs(linear.widen(c.L2[k]))
        et = c.K * U * (aX @ L1)
        st = s * np.abs(X @ linear.widen(c.L1[k]))
        est = s * et + H * (st + s * et)
        base = aX @ np.abs(c.W[k]).T
        E.append((c.K * U + (2 * H if fp16_table else 0.0)) * base + est @ L2 + c.r * U * ((st + est) @ L2))
        ET.append(et)
    return ET, E[0], E[1]


@pytest.mark.parametrize("M,K,F,r", [(1, 256, 136, 72), (1, 320, 136, 16), (1, 256, 192, 16), (2, 64, 72, 24), (2, 256, 200, 64), (5, 512, 128, 8),
                                     (11, 192, 264, 40), (16, 128, 64, 8), (16, 256, 328, 136)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_forward_few_rows(api, M, K, F, r, kind):
    c = Gated(api, M, K, F, r, kind=kind, seed=11)
    save = F % 64 == 0
    o = c.fwd(want_T=True, want_int8=save)
    A, G, Uv, T = layers.gated_fwd(c.X, *c.W, c.L1, c.L2, c.s, kind)
    ET, EG, EU = gate_up_errors(c, linear.widen(c.X))
    label = f"gated fwd {M}x{K}x{F} r{r} {kind}"
    for k in range(2):
        within(label, f"T{k}", o.T[k], T[k], ET[k])
    a, _, Ea, _ = act_errors(G, EG, kind)
    within(label, "A", o.A, A, Ea * np.abs(Uv) + np.abs(a) * EU + Ea * EU + 2 * U * np.abs(A))
    if save:
        within_int8(label, "gate8", o.gate8, G, EG)
        within_int8(label, "up8", o.up8, Uv, EU)


@pytest.mark.parametrize("M,K,F,r", [(17, 576, 16384, 72), (40, 64, 22016, 256), (96, 1088, 1032, 256), (100, 576, 136, 136), (128, 512, 16384, 256),
                                     (128, 2048, 64, 256)])
def test_gated_forward_wide_adapters(api, M, K, F, r):
    """T's workgroups beside the base product's, where those fill the device and where they do not."""
    test_gated_forward_few_rows(api, M, K, F, r, "silu")


def test_gated_forward_longest_rows(api):
    """More of T's workgroups than a grid has layers for. Signs as X and L1 make T exact."""
    import torch

    M, K, F, r = 128, (1 << 22) - 64, 8, 256
    g = torch.Generator(device="cuda").manual_seed(0)

    def signs(*shape):
        return torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.int8).mul_(2).sub_(1).to(torch.bfloat16)

    w = api.qlora_quantize(torch.empty(F, K, device="cuda").normal_(0, 1, generator=g))
    X, L1, L2 = signs(M, K), signs(2, K, r), signs(2, r, F)
    ws = torch.full((api.qlora_gated_workspace(M, K, F, r),), 255, dtype=torch.uint8, device="cuda")
    o = api.qlora_gated_fwd(w, w, X, L1, L2, 2.0 ** -20, want_T=True, workspace=ws)
    for k in range(2):
        T = torch.zeros(M, r, device="cuda")
        for at in range(0, K, 1 << 18):               # whole numbers below 2^24: exact in every order
            T += X[:, at:at + (1 << 18)].float() @ L1[k, at:at + (1 << 18)].float()
        assert (o.T[k] == T.to(torch.bfloat16)).all()
    assert torch.isfinite(o.A).all()
    del w, X, L1, ws
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,K,F,r", [(1, 64, 8, 8), (5, 64, 72, 16), (20, 128, 192, 16), (33, 128, 200, 136), (140, 64, 328, 64), (150, 192, 256, 72)])
@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("given_t", [False, True])
def test_gated_backward_inputs(api, M, K, F, r, x8, kept, given_t):
    import torch

    if kept:
        F = (F + 63) // 64 * 64
    c = Gated(api, M, K, F, r, kind="gelu" if M % 2 else "silu", seed=13)
    rng = np.random.default_rng(M + F + r)
    X, kw, x_arg, GU = linear.widen(c.X), {}, None, None
    if x8:
        x_arg, X = int8_of(api, X)
        X = linear.widen(bf16(X))
    if kept:
        (kw["gate8"], G), (kw["up8"], Uv) = int8_of(api, 2 * rng.standard_normal((M, F))), int8_of(api, rng.standard_normal((M, F)))
        GU = (G, Uv)
    else:
        G, Uv = layers.gate_up(X, *c.W, c.L1, c.L2, c.s)[:2]
    if given_t:
        T = bf16(rng.standard_normal((2, M, r)))
        kw["T"] = dev(T)
        T = linear.widen(T)
    else:
        T = np.stack([X @ linear.widen(c.L1[k]) for k in range(2)])
    dX, dL1, dL2 = c.bwd(x_arg, grad_dtype=torch.bfloat16 if r % 16 else torch.float32, **kw)
    RX, R1, R2, dG, dU = layers.gated_bwd(X, *c.W, c.L1, c.L2, c.s, c.kind, c.dA, GU)
    aX, s, dA = np.abs(X), abs(c.s), np.abs(linear.widen(c.dA))
    ET, EG, EU = gate_up_errors(c, X)
    if kept:
        EG, EU = 2 * U * np.abs(G), 2 * U * np.abs(Uv)
    a, d, Ea, Ed = act_errors(G, EG, c.kind)
    EdG = dA * (EU * np.abs(d) + np.abs(Uv) * Ed + EU * Ed) + 4 * U * np.abs(dG)
    EdU = dA * Ea + 2 * U * np.abs(dU)
    label = f"gated bwd {M}x{K}x{F} r{r} {c.kind} X8 {x8} kept {kept} T {given_t}"
    EX = 0.0
    for k, (dY, e) in enumerate(((dG, EdG), (dU, EdU))):
        e = e + H * (np.abs(dY) + e)               # rounded to bf16 as an operand
        aY, L1, L2, W = np.abs(dY) + e, np.abs(linear.widen(c.L1[k])), np.abs(linear.widen(c.L2[k])), np.abs(c.W[k])
        sU = s * np.abs(dY @ linear.widen(c.L2[k]).T)
        EsU = s * (e @ L2.T + F * U * (aY @ L2.T))
        EsU = EsU + H * (sU + EsU)
        EX = EX + 2 * F * U * (aY @ W) + e @ W + EsU @ L1.T + r * U * ((sU + EsU) @ L1.T)
        within(label, f"dL1[{k}]", dL1[k], R1[k], aX.T @ EsU + M * U * (aX.T @ (sU + EsU)))
        aT = np.abs(T[k])
        eT = np.zeros_like(aT) if given_t else ET[k] + H * (aT + ET[k])
        within(label, f"dL2[{k}]", dL2[k], c.s * (T[k].T @ dY), s * (eT.T @ aY + aT.T @ e + M * U * ((aT + eT).T @ aY)))
    within(label, "dX", dX, RX, EX)


@pytest.mark.parametrize("M,K,N,r", [(1, 64, 8, 8), (2, 256, 64, 16), (5, 128, 72, 16), (16, 64, 200, 72), (40, 192, 136, 64), (130, 64, 264, 24),
                                     (150, 128, 328, 136)])
@pytest.mark.parametrize("given_t", [False, True])
def test_linear_bwd_int8_few_rows_ragged(api, M, K, N, r, given_t):
    rng = np.random.default_rng(M + N)
    q, _ = gpu_quantize(api, (rng.standard_normal((N, K)) / np.sqrt(K)).astype(np.float32))
    W = linear.widen(api.to_host_bits(api.qlora_dequantize(q)))
    L1, L2, dY = bf16(rng.standard_normal((K, r)) / np.sqrt(K)), bf16(rng.standard_normal((r, N))), bf16(rng.standard_normal((M, N)))
    s = 0.75
    X8, X = int8_of(api, rng.standard_normal((M, K)))
    X = linear.widen(bf16(X))
    T = bf16(rng.standard_normal((M, r)))
    got = api.qlora_linear_bwd_int8(q, X8, dev(dY), dev(L1), dev(L2), s, T=dev(T) if given_t else None)
    RX, R1, _ = linear.linear_bwd(X, W, L1, L2, s, dY)
    T = linear.widen(T) if given_t else X @ linear.widen(L1)
    aX, a1, a2, aY, aW, aT = np.abs(X), *(np.abs(linear.widen(v)) for v in (L1, L2, dY)), np.abs(W), np.abs(T)
    sU = s * np.abs(linear.widen(dY) @ linear.widen(L2).T)
    EsU = s * N * U * (aY @ a2.T)
    EsU = EsU + H * (sU + EsU)
    label = f"linear int8 {M}x{K}x{N} r{r} T {given_t}"
    within(label, "dX", got[0], RX, 2 * N * U * (aY @ aW) + EsU @ a1.T + r * U * ((sU + EsU) @ a1.T))
    within(label, "dL1", got[1], R1, aX.T @ EsU + M * U * (aX.T @ (sU + EsU)))
    eT = 0.0 * aT if given_t else K * U * (aX @ a1) + H * (aT + K * U * (aX @ a1))
    within(label, "dL2", got[2], s * (T.T @ linear.widen(dY)), s * (eT.T @ aY + M * U * ((aT + eT).T @ aY)))


@pytest.mark.parametrize("M,K,V", [(1, 64, 5), (48, 192, 1000), (300, 64, 3001), (2500, 64, 700)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_head_weight_gradient_alone(api, M, K, V, dtype):
    import torch

    Hs, W, labels, rng = head_case(M, K, V, seed=3)
    labels[rng.random(M) < 0.3] = -100
    kw = dict(need_dW=True, grad_dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    o = api.qlora_head_loss(dev(Hs), dev(W), dev(labels), need_dH=False, **kw)
    assert o.dH is None
    check_head(f"head {M}x{K}x{V} dW alone {dtype}", o, Hs, W, labels)
    both = api.qlora_head_loss(dev(Hs), dev(W), dev(labels), **kw)
    assert (both.dW == o.dW).all() and (both.nll == o.nll).all() and (both.loss == o.loss).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_head_pieces_without_a_gradient(api, dtype):
    """Several pieces of rows, dW without dH and the loss alone: the bits of the call with both gradients."""
    import torch

    M, K, V = 1100, 64, 1 << 20                       # pieces of 512 rows
    g = torch.Generator(device="cuda").manual_seed(2)
    Hd = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g)
    Wd = torch.empty(V, K, dtype=torch.bfloat16, device="cuda").normal_(0, 0.25, generator=g)
    Ld = torch.randint(0, V, (M,), device="cuda", generator=g)
    kw = dict(grad_dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    for some in (Ld, torch.where(torch.arange(M, device="cuda") % 3 == 0, Ld, -100)):
        both = api.qlora_head_loss(Hd, Wd, some, need_dW=True, **kw)
        dW = api.qlora_head_loss(Hd, Wd, some, need_dH=False, need_dW=True, **kw)
        alone = api.qlora_head_loss(Hd, Wd, some, need_dH=False)
        for o in (dW, alone):
            assert o.dH is None and (o.nll == both.nll).all() and (o.loss == both.loss).all()
        assert (dW.dW == both.dW).all()
        del both, dW, alone
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,K,V", [(3, 64, 5), (300, 128, 3001), (2500, 64, 700), (600, 64, 1 << 20)])
def test_head_alone_stays_in_its_workspace(api, M, K, V):
    """The loss alone, whose workspace has no room for probabilities: nothing behind it is written."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(M)
    Hd = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g)
    Wd = torch.empty(V, K, dtype=torch.bfloat16, device="cuda").normal_(0, 0.25, generator=g)
    Wd[V // 2] *= 64.0                                # a tile that takes its rows' maxima out
    Ld = torch.randint(-2, V, (M,), device="cuda", generator=g)
    full = api.qlora_head_loss(Hd, Wd, Ld)
    n = api.qlora_head_workspace(M, K, V, False, False)
    buf = torch.full((n + (1 << 22),), 0xA5, dtype=torch.uint8, device="cuda")
    o = api.qlora_head_loss(Hd, Wd, Ld, need_dH=False, workspace=buf[:n])
    assert (buf[n:] == 0xA5).all()
    assert (o.nll == full.nll).all() and (o.loss == full.loss).all() and torch.isfinite(o.loss).all()
