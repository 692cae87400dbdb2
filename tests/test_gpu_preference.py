"""GPU parity of qlora_preference_loss against the float64 oracle (oracle/preference.py).

Bounds, with u = 2^-24: a thread sums at most V / 256 + 16 exponentials in
fp32, the joins add 16 more roundings, and each exponent x log2(e) - max
carries a rounding of numbers up to 2 log2(e) max|x| < 3 max|x| (twice: the
product's constant and the fused sum), so a row's sum is off by at most
    rho = u (V / 256 + 48 + 8 max|x|)     relative,
lp by rho + 2 u |lp|, a reward by beta times the sum of its lp's errors + u, the
loss by the mean of its pairs' reward errors + 2 u, a weight by beta / (4 P) of
the h error + 2 u, and a gradient element w (onehot - q) by |w| q 2 rho, the
weight's error and the rounding of its type (u, or 2^-8 in bf16: half an ulp is
2^-9 of the binade's top); one smallest fp32 step covers underflow.
"""

import numpy as np
import pytest

from gpu_util import require_gpu, say
from oracle import nf4
from oracle import preference as oracle

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def api():
    return require_gpu()


def draw(pairs, T, V, bf16, seed, std=2.0, mask=0.4):
    rng = np.random.default_rng(seed)
    S = 2 * pairs
    x = (std * rng.standard_normal((S, T, V))).astype(np.float32)
    labels = rng.integers(0, V, (S, T))
    np.put_along_axis(x, labels[..., None], np.take_along_axis(x, labels[..., None], 2) + np.float32(3.0), 2)
    if bf16:
        x = nf4.bf16_bits_to_f32(nf4.bf16_rne(x.reshape(-1))).astype(np.float32).reshape(x.shape)
    labels = np.where(rng.random((S, T)) < mask, rng.choice([-100, -1, V, V + 5, -(1 << 40), 1 << 40], (S, T)), labels)
    ref = (-3.0 + rng.standard_normal((S, T))).astype(np.float32)
    return x, labels.astype(np.int64), ref


def device(x, labels, ref, bf16, pad=0, shift=0):
    """Device tensors; rows `pad` elements apart beyond V, the first `shift` elements into its allocation."""
    import torch

    S, T, V = x.shape
    dt = torch.bfloat16 if bf16 else torch.float32
    flat = torch.full((S * T * (V + pad) + shift,), 50.0, dtype=dt, device="cuda")   # the gaps are not to be read
    t = flat[shift:].view(S, T, V + pad)[:, :, :V]
    t.copy_(torch.from_numpy(x))
    return t, torch.from_numpy(labels).cuda(), torch.from_numpy(ref).cuda()


def check(out, x, labels, ref, beta, eps, bf16, scale=1.0, label=""):
    loss, rewards, lp, grad, w, q = oracle.preference(x, labels, ref, beta, eps, scale)
    S, T, V = x.shape
    P = S // 2
    on = (labels >= 0) & (labels < V)
    finite = np.where(np.isfinite(x), np.abs(x), 0.0)
    rho = U * (V / 256 + 48 + 8 * (finite.max(axis=2) if V and S * T else np.zeros((S, T))))
    e_lp = np.where(on, rho + 2 * U * np.abs(lp), 0.0)
    g_lp = out.logps.cpu().numpy().astype(np.float64)
    assert (np.abs(g_lp - lp) <= e_lp).all(), (label, np.abs(g_lp - lp).max())
    e_r = np.abs(beta) * e_lp.sum(axis=1) + 2 * U * np.abs(rewards) + 1e-30
    g_r = out.rewards.cpu().numpy().astype(np.float64)
    assert (np.abs(g_r - rewards) <= e_r).all(), (label, np.abs(g_r - rewards).max())
    e_h = e_r[:P] + e_r[P:]
    assert abs(out.loss.item() - loss) <= (e_h.mean() if P else 0.0) + 2 * U * abs(loss), (label, out.loss.item(), loss)
    if out.dlogits is None:
        return
    e_w = np.tile(np.abs(scale * beta) / max(P, 1) * e_h / 4, 2) + 4 * U * np.abs(w)
    g = out.dlogits.float().cpu().numpy().astype(np.float64)
    assert not np.isnan(g).any()
    hot = np.zeros_like(q)
    np.put_along_axis(hot, np.where(on, labels, 0)[..., None], 1.0, 2)
    tol = np.abs(w)[:, None, None] * q * 2 * rho[..., None] + e_w[:, None, None] * np.abs(hot - q)
    tol = tol * 1.01 + np.abs(grad) * (2.0 ** -8 if bf16 else 4 * U) + 2.0 ** -133
    tol = np.where(on[..., None], tol, 0.0)
    assert (np.abs(g - grad) <= tol).all(), (label, np.abs(g - grad).max())


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("pairs,T,V", [(1, 1, 1), (1, 1, 2), (2, 5, 7), (1, 3, 8), (3, 4, 255), (2, 17, 1000),
                                       (1, 2, 4099), (2, 3, 32001), (1, 2, 70001), (17, 65, 33)])
@pytest.mark.parametrize("eps", [0.0, 0.2])
def test_loss_and_gradient(api, pairs, T, V, bf16, eps):
    say(f"preference pairs={pairs} T={T} V={V} bf16={bf16} eps={eps}")
    x, labels, ref = draw(pairs, T, V, bf16, 7 * V + T)
    a, b, c = device(x, labels, ref, bf16)
    keep = a.clone()
    out = api.qlora_preference_loss(a, b, c, 0.1, label_smoothing=eps)
    check(out, x, labels, ref, 0.1, eps, bf16)
    assert (a == keep).all()
    again = api.qlora_preference_loss(a, b, c, 0.1, label_smoothing=eps)
    for p, q in zip(out, again):
        assert (p == q).all()
    only = api.qlora_preference_loss(a, b, c, 0.1, label_smoothing=eps, need_grad=False)
    assert only.dlogits is None and (only.logps == out.logps).all() and only.loss.item() == out.loss.item()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V,pad,shift", [(1000, 3, 0), (1001, 0, 1), (999, 1, 5), (64, 8, 3), (5, 2, 1), (40003, 5, 2)])
def test_strides_and_alignment(api, V, pad, shift, bf16):
    """Rows at any stride and element alignment, a gradient aligned otherwise, and the gradient in place."""
    import torch

    say(f"preference V={V} pad={pad} shift={shift} bf16={bf16}")
    x, labels, ref = draw(2, 6, V, bf16, V)
    a, b, c = device(x, labels, ref, bf16, pad, shift)
    check(api.qlora_preference_loss(a, b, c, 0.3), x, labels, ref, 0.3, 0.0, bf16)
    flat = torch.full((2 * 2 * 6 * (V + 4) + 3,), 9.0, dtype=a.dtype, device="cuda")
    d = flat[3:].view(4, 6, V + 4)[:, :, :V]
    check(api.qlora_preference_loss(a, b, c, 0.3, dlogits=d), x, labels, ref, 0.3, 0.0, bf16)
    assert (flat[3:].view(4, 6, V + 4)[:, :, V:] == 9.0).all() and (flat[:3] == 9.0).all()
    gaps = a.as_strided((24, pad), (V + pad, 1), a.storage_offset() + V) if pad else None
    out = api.qlora_preference_loss(a, b, c, 0.3, dlogits=a)
    check(out, x, labels, ref, 0.3, 0.0, bf16, label="in place")
    assert gaps is None or (gaps[:-1] == 50.0).all()


def test_nothing_counts(api):
    """Masked sequences, masked pairs, no positions, no pairs."""
    import torch

    x, labels, ref = draw(3, 8, 500, False, 3, mask=0.0)
    labels[1] = -100            # the preferred sequence of pair 1
    labels[2] = labels[5] = -1  # both of pair 2
    x[2] = np.nan               # logits that do not count are not used
    ref[2, 3] = np.nan
    a, b, c = device(x, labels, ref, False)
    out = api.qlora_preference_loss(a, b, c, 0.1)
    xs = np.where(np.isnan(x), 0.0, x)
    check(out, xs, labels, np.where(np.isnan(ref), 0.0, ref), 0.1, 0.0, False)
    assert out.rewards[1].item() == 0.0 and (out.dlogits[1] == 0).all() and (out.dlogits[2] == 0).all()
    out = api.qlora_preference_loss(a[:, :0].contiguous(), b[:, :0].contiguous(), c[:, :0].contiguous(), 0.1)
    assert out.loss.item() == pytest.approx(np.log(2.0), rel=2 * U) and (out.rewards == 0).all()
    out = api.qlora_preference_loss(a[:0], b[:0], c[:0], 0.1)
    assert out.loss.item() == 0.0 and out.dlogits.numel() == 0
    torch.cuda.synchronize()


@pytest.mark.parametrize("bf16", [False, True])
def test_extreme_logits(api, bf16):
    """-inf entries (tokens that are ruled out), the type's lowest value, and large magnitudes."""
    x, labels, ref = draw(2, 4, 3000, bf16, 11, mask=0.0)
    low = -3.3895313892515355e38 if bf16 else np.finfo(np.float32).min
    rng = np.random.default_rng(5)
    gone = rng.random(x.shape) < 0.5
    np.put_along_axis(gone, labels[..., None], False, 2)
    x[0] = np.where(gone[0], -np.inf, x[0])
    x[1] = np.where(gone[1], low, x[1])
    x[2, 0, :2000] = -np.inf                # whole pieces of a row
    x[2, 0, labels[2, 0]] = 1.0
    x[3] = np.float32(64.0) * np.sign(x[3])
    a, b, c = device(x, labels, ref, bf16)
    xs = np.where(x == np.float32(low), -np.inf, x)     # either way no probability
    check(api.qlora_preference_loss(a, b, c, 0.1), xs, labels, ref, 0.1, 0.0, bf16)


def test_scale_and_sign(api):
    x, labels, ref = draw(2, 9, 777, False, 21)
    a, b, c = device(x, labels, ref, False)
    check(api.qlora_preference_loss(a, b, c, 0.5, grad_scale=-0.25), x, labels, ref, 0.5, 0.0, False, scale=-0.25)
    check(api.qlora_preference_loss(a, b, c, 20.0), x, labels, ref, 20.0, 0.0, False)     # saturated pairs


def test_gradient_against_differences(api):
    """The kernel's gradient against central differences of the float64 loss."""
    x, labels, ref = draw(2, 3, 11, False, 31)
    a, b, c = device(x, labels, ref, False)
    g = api.qlora_preference_loss(a, b, c, 0.7, label_smoothing=0.1).dlogits.cpu().numpy().astype(np.float64)
    h = 1e-5
    num = np.zeros(x.shape)
    for i in np.ndindex(*x.shape):
        up, down = x.astype(np.float64), x.astype(np.float64)
        up[i] += h
        down[i] -= h
        num[i] = (oracle.preference(up, labels, ref, 0.7, 0.1)[0] - oracle.preference(down, labels, ref, 0.7, 0.1)[0]) / (2 * h)
    # differences: h^2 / 6 of a third derivative below 1, and 2^-52 of a loss below 4 over h; the kernel: fp32
    assert (np.abs(g - num) <= 1e-9 + 100 * U * np.abs(g).max()).all(), np.abs(g - num).max()


def test_stream_and_graph(api):
    import torch

    x, labels, ref = draw(2, 33, 2001, True, 41)
    a, b, c = device(x, labels, ref, True)
    want = api.qlora_preference_loss(a, b, c, 0.1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = api.qlora_preference_loss(a, b, c, 0.1, stream=s)
    s.synchronize()
    for p, q in zip(want, got):
        assert torch.equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = api.qlora_preference_loss(a, b, c, 0.1)
    for _ in range(4):
        a.mul_(0.75)
        want = api.qlora_preference_loss(a, b, c, 0.1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(want, got):
            assert torch.equal(p, q)


def test_refusals(api):
    import torch

    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    lab = z(2, 3, dt=torch.int64)
    with pytest.raises(ValueError):
        api.qlora_preference_loss(z(3, 3, 8), z(3, 3, dt=torch.int64), z(3, 3), 0.1)      # an odd sequence
    with pytest.raises(TypeError):
        api.qlora_preference_loss(z(2, 3, 8, dt=torch.float16), lab, z(2, 3), 0.1)
    with pytest.raises(TypeError):
        api.qlora_preference_loss(z(2, 3, 8), lab.int(), z(2, 3), 0.1)
    with pytest.raises(ValueError):
        api.qlora_preference_loss(z(2, 3, 8), lab, z(2, 4), 0.1)
    with pytest.raises(ValueError):
        api.qlora_preference_loss(z(2, 8, 3).transpose(1, 2), lab, z(2, 3), 0.1)
    with pytest.raises(ValueError):
        api.qlora_preference_loss(z(2, 3, 8), lab, z(2, 3), 0.1, dlogits=z(2, 3, 9))
    with pytest.raises(ValueError):
        api.qlora_preference_loss(z(2, 3, 8).cpu(), lab, z(2, 3), 0.1)
    with pytest.raises(api.QLoRAError):
        api.qlora_preference_loss(z(2, 3, 8), lab, z(2, 3), float("nan"))
    with pytest.raises(api.QLoRAError):
        api.qlora_preference_loss(z(2, 3, 8), lab, z(2, 3), 0.1, label_smoothing=1.5)
