"""GPU parity of the optimiser step over many tensors (qlora_clip_grad_norm_batch,
qlora_adamw_batch) against the float64 oracle (oracle/optim.py,
oracle/optim_batch.py).

The norm is a float64 sum in another order: 1e-12 relative. The update is
fp32 with one rounding per operation in its written order: theta, the
moments, the codes and the scales must equal the numpy fp32 evaluation
(tests/adam_fp32.py) bit for bit, and with fp32 state stay within the bounds
propagated from the roundings around the float64 trajectory. An 8-bit state
stays within half an E4M3 step (2^-4 of the value, 2^-10 of 448 / top below
the normal range, a whole 2^-9 for a root kept from 0) of the exact moments of
the values it held before, plus that fp32 error.
"""

import ctypes

import numpy as np
import pytest

from adam_fp32 import U, adam_error_bounds, adam_step_fp32
from gpu_util import require_gpu, say
from oracle import nf4, optim, optim_batch

pytestmark = pytest.mark.gpu

HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
# one value, short and whole blocks and chunks of 4096, ragged ends, empty tensors, more than one launch's 64
SIZES = {
    "one": [1],
    "edges": [0, 1, 3, 4, 255, 256, 257, 0, 4095, 4096, 4097, 12289],
    "many": [17 * k % 700 + 1 for k in range(150)],
    "empties": [0] * 70 + [5],
    "launches": [17 * k % 700 + 1 for k in range(300)],                          # more than any launch's table
    "gaps": [0] * 70 + [5, 4096, 0] + [0] * 300 + [8192, 3, 0],
}


@pytest.fixture(scope="module")
def api():
    return require_gpu()


def draw(sizes, bf16, seed):
    rng = np.random.default_rng(seed)
    theta = [(0.02 * rng.standard_normal(n)).astype(np.float32) for n in sizes]
    grads = [(0.1 * rng.standard_normal(n) * np.exp(2 * rng.standard_normal(n))).astype(np.float32) for n in sizes]
    if bf16:
        grads = [nf4.bf16_bits_to_f32(nf4.bf16_rne(g)).astype(np.float32) for g in grads]
    return theta, grads


def on_gpu(arrays, bf16=False):
    import torch

    ts = [torch.from_numpy(a.copy()).cuda() for a in arrays]
    return [t.to(torch.bfloat16) for t in ts] if bf16 else ts


@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("bf16", [False, True])
def test_norm(api, sizes, bf16):
    say(f"clip batch {sizes} bf16={bf16}")
    _, grads = draw(SIZES[sizes], bf16, 1)
    dev = on_gpu(grads, bf16)
    for max_norm in (0.3, 1e9, float("inf")):
        coef, norm = api.qlora_clip_grad_norm_batch(dev, max_norm)
        c, n = optim_batch.clip(grads, max_norm)
        assert norm.item() == pytest.approx(n, rel=1e-12, abs=0.0)
        assert coef.item() == pytest.approx(c, rel=2 ** -23)
        again = api.qlora_clip_grad_norm_batch(dev, max_norm)
        assert again[0].item() == coef.item() and again[1].item() == norm.item()


def test_norm_of_nothing(api):
    coef, norm = api.qlora_clip_grad_norm_batch([], 0.3)
    assert coef.item() == 1.0 and norm.item() == 0.0


@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("paged", [False, True])
def test_steps_bit_for_bit(api, sizes, bf16, bits, paged):
    import torch

    say(f"adamw batch {sizes} bf16={bf16} bits={bits} paged={paged}")
    numel = SIZES[sizes]
    theta, _ = draw(numel, bf16, 2)
    dev = on_gpu(theta)
    copies = [torch.full_like(t, 7.0, dtype=torch.bfloat16) for t in dev]
    state = api.AdamWState.zeros(dev, bits=bits, pin_memory=paged)
    at = optim_batch.offsets(numel)
    held = [tuple(np.zeros(n, np.float32) for _ in "mv") for n in numel]
    for t in range(1, 4):
        _, grads = draw(numel, bf16, 10 * t)
        if t == 2:
            for g in grads:
                g[::3] = 0.0                     # gradients that vanish
        gdev = on_gpu(grads, bf16)
        coef = torch.tensor([0.37], device="cuda") if t != 3 else None
        api.qlora_adamw_batch(dev, gdev, state, t, coef=coef, thetas_bf16=copies if t != 2 else None, **HP)
        torch.cuda.synchronize()
        m_all, v_all = state.m.cpu(), state.v.cpu()
        if bits == 8:
            m_all, v_all = (x.view(torch.uint8).numpy() for x in (m_all, v_all))
            ms, vs = state.m_scale.cpu().numpy(), state.v_scale.cpu().numpy()
        else:
            m_all, v_all = m_all.numpy(), v_all.numpy()
        for k, n in enumerate(numel):
            if n == 0:
                continue
            m, v = held[k]
            theta[k], m, v = adam_step_fp32(theta[k], grads[k], m, v, t, HP["lr"], HP["beta1"], HP["beta2"],
                                            HP["eps"], HP["weight_decay"], 0.37 if coef is not None else 1.0)
            sl = slice(at[k], at[k] + n)
            np.testing.assert_array_equal(dev[k].cpu().numpy().view(np.uint32), theta[k].view(np.uint32))
            if t != 2:
                np.testing.assert_array_equal(api.to_host_bits(copies[k]), nf4.bf16_rne(theta[k]))
            if bits == 32:
                np.testing.assert_array_equal(m_all[sl].view(np.uint32), m.view(np.uint32))
                np.testing.assert_array_equal(v_all[sl].view(np.uint32), v.view(np.uint32))
            else:
                r = np.sqrt(v)
                sp = slice(at[k], at[k + 1])
                bs = slice(at[k] // 256, at[k + 1] // 256)
                for x, keep, codes, scales in ((m, False, m_all, ms), (r, True, v_all, vs)):
                    c, s = optim_batch.encode(x, keep)
                    # +0 and -0 are one value
                    same = (codes[sp] & 0x7F == 0) & (c & 0x7F == 0)
                    np.testing.assert_array_equal(np.where(same, 0, codes[sp]), np.where(same, 0, c))
                    np.testing.assert_array_equal(scales[bs].view(np.uint32), s.view(np.uint32))
                    # within half a step of what was encoded
                    got = optim_batch.decode(codes[sp], scales[bs])[:n].astype(np.float64)
                    top = np.repeat(s.astype(np.float64), 256)[:n]
                    least = (2.0 ** -9 if keep else 2.0 ** -10) * top
                    assert (np.abs(got - x) <= np.maximum(2.0 ** -4 * np.abs(x), least) * (1 + 8 * U) + 1e-44).all()
                    if keep:
                        assert ((got > 0) | (x == 0) | (top == 0)).all()
                m = optim_batch.decode(*(optim_batch.encode(m, False)))[:n]
                root = optim_batch.decode(*(optim_batch.encode(r, True)))[:n]
                v = root * root
            held[k] = (m, v)


@pytest.mark.parametrize("wd", [0.0, 0.1])
def test_steps_within_the_float64_bounds(api, wd):
    import torch

    numel = [1000, 37, 5000]
    theta, _ = draw(numel, False, 3)
    dev = on_gpu(theta)
    state = api.AdamWState.zeros(dev, bits=32)
    steps, coefs = [], []
    for t in range(1, 5):
        _, grads = draw(numel, False, 30 + t)
        gdev = on_gpu(grads)
        coef, _ = api.qlora_clip_grad_norm_batch(gdev, 0.3)
        api.qlora_adamw_batch(dev, gdev, state, t, **{**HP, "weight_decay": wd}, coef=coef)
        steps.append(np.concatenate(grads))
        coefs.append(optim.clip_coef(steps[-1], 0.3))
    torch.cuda.synchronize()
    th, m, v, eth, em, ev = adam_error_bounds(np.concatenate(theta), steps, coefs, HP["lr"], HP["beta1"], HP["beta2"],
                                              HP["eps"], wd)
    at = optim_batch.offsets(numel)
    take = lambda x: np.concatenate([x.cpu().numpy()[o:o + n] for o, n in zip(at, numel)])  # noqa: E731
    assert (np.abs(np.concatenate([t.cpu().numpy() for t in dev]) - th) <= eth).all()
    assert (np.abs(take(state.m) - m) <= em).all()
    assert (np.abs(take(state.v) - v) <= ev).all()


def test_codes_of_extreme_blocks(api):
    """Blocks of zeros, of values near the largest and the smallest fp32, and of 17 binades at once."""
    import torch

    n = 6 * 256
    m = np.zeros((6, 256), np.float32)
    m[1] = 1e38 * np.linspace(-1, 1, 256, dtype=np.float32)
    m[2] = 2.0 ** -99
    m[3] = 2.0 ** -101                                        # below the threshold: zeros
    m[4] = np.float32(2.0) ** -np.arange(256, dtype=np.float32) * 0.5
    m[5, 7] = 1.0
    # with beta1 = 0 and coef 1 the new m is the gradient, and sqrt(v) its magnitude up to rounding
    th = on_gpu([np.zeros(n, np.float32)])
    g = on_gpu([np.clip(m, -1e15, 1e15).reshape(-1)])
    state = api.AdamWState.zeros(th, bits=8)
    api.qlora_adamw_batch(th, g, state, 1, lr=0.0, beta1=0.0, beta2=0.0)
    x = g[0].cpu().numpy()
    for name, val, keep in (("m", x, False), ("v", np.sqrt(x * x), True)):
        codes = getattr(state, name).cpu().view(torch.uint8).numpy()
        scale = getattr(state, name + "_scale").cpu().numpy()
        c, s = optim_batch.encode(val, keep)
        same = (codes & 0x7F == 0) & (c & 0x7F == 0)
        np.testing.assert_array_equal(np.where(same, 0, codes), np.where(same, 0, c))
        np.testing.assert_array_equal(scale.view(np.uint32), s.view(np.uint32))


def test_another_stream(api):
    import torch

    theta, grads = draw([5000, 333], False, 5)
    ref, dev = on_gpu(theta), on_gpu(theta)
    g = on_gpu(grads)
    a, b = api.AdamWState.zeros(ref), api.AdamWState.zeros(dev)
    c, _ = api.qlora_clip_grad_norm_batch(g, 0.3)
    api.qlora_adamw_batch(ref, g, a, 1, coef=c, **HP)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    c, _ = api.qlora_clip_grad_norm_batch(g, 0.3, stream=s)
    api.qlora_adamw_batch(dev, g, b, 1, coef=c, stream=s, **HP)
    s.synchronize()
    for x, y in zip(ref, dev):
        assert torch.equal(x, y)
    assert torch.equal(a.m.view(torch.uint8), b.m.view(torch.uint8))


def test_graph_replays(api):
    """Captured once and replayed with eager work between: every replay steps like an eager call."""
    import torch

    theta, grads = draw([5000, 333, 1], False, 6)
    eager, dev, g = on_gpu(theta), on_gpu(theta), on_gpu(grads)
    a, b = api.AdamWState.zeros(eager), api.AdamWState.zeros(dev)
    coef, norm = torch.empty(1, device="cuda"), torch.empty(1, dtype=torch.float64, device="cuda")
    ws = torch.empty(api.QLORA_CLIP_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")

    def step(th, st):
        api.qlora_clip_grad_norm_batch(g, 0.3, coef=coef, norm=norm, workspace=ws)
        api.qlora_adamw_batch(th, g, st, 3, coef=coef, **HP)

    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        step(dev, b)
    for k in range(4):
        step(eager, a)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(eager, dev):
            assert torch.equal(x, y), k
        g[0].mul_(0.5)


def test_refusals(api):
    import torch

    th = on_gpu([np.zeros(300, np.float32)])
    g = on_gpu([np.zeros(300, np.float32)])
    st = api.AdamWState.zeros(th)
    with pytest.raises(ValueError):
        api.qlora_adamw_batch(th, g + g, st, 1, 1e-3)
    with pytest.raises(ValueError):
        api.qlora_adamw_batch(on_gpu([np.zeros(301, np.float32)]), on_gpu([np.zeros(301, np.float32)]), st, 1, 1e-3)
    with pytest.raises(TypeError):
        api.qlora_adamw_batch(th, [g[0].half()], st, 1, 1e-3)
    with pytest.raises(TypeError):
        api.qlora_adamw_batch([th[0].double()], g, st, 1, 1e-3)
    with pytest.raises(ValueError):
        api.qlora_adamw_batch(th, [torch.zeros(600, device="cuda")[::2]], st, 1, 1e-3)
    with pytest.raises(ValueError):
        api.qlora_adamw_batch(th, [g[0].cpu()], st, 1, 1e-3)
    for bad in (dict(step=0), dict(lr=-1.0), dict(beta1=1.0), dict(lr=float("nan"))):
        with pytest.raises(api.QLoRAError):
            api.qlora_adamw_batch(th, g, st, **{"step": 1, "lr": 1e-3, **bad})
    with pytest.raises(api.QLoRAError):          # not 16-byte aligned
        api.qlora_adamw_batch([torch.zeros(301, device="cuda")[1:]], g, st, 1, 1e-3)
    with pytest.raises(ValueError):
        api.AdamWState.zeros(th, bits=4)
    with pytest.raises(api.QLoRAError):
        api.qlora_clip_grad_norm_batch(g, 0.0)
    with pytest.raises(ValueError):              # pageable host memory
        api.qlora_adamw_batch(th, g, api.AdamWState.zeros(th, device="cpu"), 1, 1e-3)
    assert (th[0] == 0).all()
