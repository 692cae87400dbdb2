"""GPU tests of the many-adapter entry points where values are not finite and
where sizes pass a launch's reach.

An infinity or NaN of one adapter or of one row changes that adapter's rows, or
that row, alone: everything else keeps its bits. What it does change follows
the formula: an infinity times a finite nonzero number is an infinity of their
sign.
"""

import numpy as np
import pytest

from gpu_util import require_gpu, say
from test_gpu_multi import Case

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def api():
    return require_gpu()


def set_ids(c, ids):
    c.ids = np.asarray(ids, np.int32)
    c.d["ids"].copy_(c.d["ids"].new_tensor(c.ids.tolist()))


# ---- a single token -------------------------------------------------------------------

@pytest.mark.parametrize("K,N,r", [(512, 512, 64), (512, 264, 16), (320, 72, 8)])
@pytest.mark.parametrize("bare", [-1, 3])
@pytest.mark.parametrize("what", ["L1", "L2", "scale"])
def test_bare_token_beside_a_diverged_adapter(api, K, N, r, bare, what):
    """A token without an adapter is the base alone, whatever adapter 0 holds."""
    import torch

    say(f"multi bare token K={K} N={N} r={r} id={bare} {what}")
    c = Case(api, 1, K, N, r, 3, "one")
    set_ids(c, [bare])
    Y, T = c.fwd(want_T=True)
    assert torch.isfinite(Y).all() and (T == 0).all()
    for value in (INF, -INF, NAN):
        if what == "scale":
            c.d["scale"][:] = value
        else:
            c.d[what][0, ::3, ::5] = value
            c.d[what][2, ::3, ::5] = value
        Y2, T2 = c.fwd(want_T=True)
        assert torch.equal(Y2, Y) and (T2 == 0).all(), value


@pytest.mark.parametrize("M,K,N,r", [(1, 512, 512, 24), (1, 512, 512, 64), (1, 320, 72, 8), (7, 512, 264, 16),
                                     (16, 640, 264, 40), (60, 512, 264, 24), (200, 512, 264, 24), (300, 512, 264, 72)])
def test_an_infinity_of_the_last_rank(api, M, K, N, r):
    """Ranks past r add nothing: an infinity in the last rank is an infinity of the product's sign."""
    import torch

    say(f"multi last rank M={M} K={K} N={N} r={r}")
    c = Case(api, M, K, N, r, 2, "one")
    T = c.fwd(want_T=True)[1]
    assert (T[:, r - 1] != 0).all()
    c.d["L2"][1, r - 1, 5] = INF
    c.d["L2"][1, r - 1, 40] = -INF
    Y = c.fwd()[0].float()
    sign = torch.sign(T[:, r - 1].float())
    assert torch.equal(Y[:, 5], sign * INF) and torch.equal(Y[:, 40], sign * -INF)


@pytest.mark.parametrize("r", [8, 24, 64])
def test_an_infinity_of_the_last_rank_of_one_adapter(api, r):
    """The same for the single-adapter linear's token."""
    import torch

    c = Case(api, 1, 512, 512, r, 1, "one")
    L1, L2 = c.d["L1"][0], c.d["L2"][0]
    T = api.qlora_linear_fwd(c.q, c.d["X"], L1, L2, 0.5, want_T=True)[1]
    L2[r - 1, 5] = INF
    Y = api.qlora_linear_fwd(c.q, c.d["X"], L1, L2, 0.5)[0]
    assert torch.equal(Y[:, 5].float(), torch.sign(T[:, r - 1].float()) * INF)


# ---- adapters without rows ----------------------------------------------------------------

@pytest.mark.parametrize("M,r,A", [(5, 16, 4), (300, 24, 5), (2500, 64, 3)])
@pytest.mark.parametrize("value", [INF, -INF, NAN, -2.0])
def test_gradients_of_an_idle_adapter(api, M, r, A, value):
    """Zeros, whatever its scale and factors hold."""
    import torch

    say(f"multi idle adapter M={M} r={r} A={A} scale={value}")
    c = Case(api, M, 256, 264, r, A, "rows")
    set_ids(c, np.where(c.ids == 1, 0, c.ids))
    want = c.bwd()
    c.d["scale"][1] = value
    c.d["L1"][1, :, 0] = value
    c.d["L2"][1, 0] = value
    for dt in (torch.float32, torch.bfloat16):
        got = c.bwd(grad_dtype=dt)
        assert torch.equal(got[0], want[0])
        for g, w in zip(got[1:], want[1:]):
            assert torch.equal(g, w.to(dt))
            assert not g[1].view(torch.int16 if dt == torch.bfloat16 else torch.int32).any()


# ---- infinities of a row ---------------------------------------------------------------------

@pytest.mark.parametrize("M", [1, 7, 17, 60, 96, 128, 200])
@pytest.mark.parametrize("K", [320, 64, 512])
def test_an_infinity_in_a_bare_row(api, M, K):
    """Y[m][n] is an infinity with the weight's sign where only one x is infinite, and NaN where that weight is 0."""
    import torch

    say(f"multi infinity in a bare row M={M} K={K}")
    c = Case(api, M, K, 264, 16, 3, "rows")
    m = M // 2
    ids = c.ids.copy()
    ids[m] = -1
    set_ids(c, ids)
    Y = c.fwd()[0]
    W = api.qlora_dequantize(c.q).float()
    others = torch.arange(M, device="cuda") != m
    for k in (0, K // 2 + 3, K - 64, K - 33, K - 1):
        x = c.d["X"][m, k].clone()
        c.d["X"][m, k] = -INF
        Y2 = c.fwd()[0]
        c.d["X"][m, k] = x
        want = W[:, k] * -INF
        assert torch.equal(Y2[others], Y[others]), k
        assert torch.equal(Y2[m].float().nan_to_num(nan=7.0), want.nan_to_num(nan=7.0)), k


# ---- rows past a launch's reach ----------------------------------------------------------------

@pytest.mark.parametrize("T", [(1 << 23) - 1, 1 << 23, (1 << 23) + 3])
def test_preference_of_more_than_2_24_rows(api, T):
    """One pair of long sequences over a tiny vocabulary, against float64 sums on the device."""
    import torch

    U, V, beta = 2.0 ** -24, 3, 1e-3
    say(f"preference 2 x {T} rows of {V}")
    gen = torch.Generator("cuda").manual_seed(T)
    x = torch.randn(2, T, V, generator=gen, device="cuda")
    y = torch.randint(-1, V, (2, T), generator=gen, device="cuda")
    ref = -1.0 + 0.1 * torch.randn(2, T, generator=gen, device="cuda")
    out = api.qlora_preference_loss(x, y, ref, beta)
    only = api.qlora_preference_loss(x, y, ref, beta, need_grad=False)
    d = x.double()
    q = d.exp()
    total = q.sum(2, keepdim=True)
    on, at = y >= 0, y.clamp(min=0)[..., None]
    lp = torch.where(on, d.gather(2, at)[..., 0] - total[..., 0].log(), 0.0)
    q /= total
    rho = U * (V / 256 + 48 + 8 * x.abs().amax(2).double())      # as in test_gpu_preference.py
    e_lp = torch.where(on, rho + 2 * U * lp.abs(), 0.0)
    assert ((out.logps - lp).abs() <= e_lp).all()
    reward = beta * torch.where(on, lp - ref, 0.0).sum(1)
    e_r = beta * e_lp.sum(1) + 2 * U * reward.abs()
    assert ((out.rewards - reward).abs() <= e_r).all()
    h = reward[0] - reward[1]
    loss = torch.nn.functional.softplus(-h)
    assert (out.loss - loss).abs() <= e_r.sum() + 2 * U * loss
    w = -beta * torch.sigmoid(-h) * torch.tensor([1.0, -1.0], dtype=torch.float64, device="cuda")
    e_w = beta * e_r.sum() / 4 + 4 * U * w.abs()
    hot = torch.zeros_like(q).scatter_(2, at, 1.0)
    grad = torch.where(on[..., None], w[:, None, None] * (hot - q), 0.0)
    tol = w.abs()[:, None, None] * q * 2 * rho[..., None] + e_w[:, None, None] * (hot - q).abs()
    tol = tol * 1.01 + 4 * U * grad.abs() + 2.0 ** -133
    tol = torch.where(on[..., None], tol, 0.0)
    assert ((out.dlogits - grad).abs() <= tol).all()
    for a, b in zip(out[:3], only[:3]):
        assert torch.equal(a, b)


# ---- workspaces ------------------------------------------------------------------------------------

@pytest.mark.parametrize("M,K,N,r,A", [(1, 512, 512, 16, 3), (13, 512, 264, 16, 5), (33, 4096, 136, 16, 3), (128, 320, 1032, 72, 9),
                                       (129, 512, 264, 64, 4), (150, 4096, 264, 24, 40), (300, 256, 4096, 72, 3),
                                       (513, 512, 512, 16, 7), (2500, 256, 512, 64, 2)])
def test_nothing_beyond_the_workspace(api, M, K, N, r, A):
    """A workspace of the query's size for this batch or a larger one is enough, and nothing past the former is written."""
    import torch

    say(f"multi workspace M={M} K={K} N={N} r={r} A={A}")
    c = Case(api, M, K, N, r, A, "rows")
    for back, call in ((False, lambda **kw: c.fwd(want_T=True, **kw)), (True, c.bwd)):
        want = call()
        need = api.qlora_linear_multi_workspace(M, K, N, r, A, back)
        ws = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
        got = call(workspace=ws)
        assert (ws[need:] == 171).all()
        large = torch.empty(api.qlora_linear_multi_workspace(3 * M + 500, K, N, r, A, back), dtype=torch.uint8, device="cuda")
        for other in (got, call(workspace=ws[:need]), call(workspace=large)):
            for a, b in zip(other, want):
                assert torch.equal(a, b)
        with pytest.raises(ValueError):
            call(workspace=ws[:need - 1])


def test_refused_workspaces(api):
    """A workspace in host memory, or one whose values do not lie in a row, is refused before anything is enqueued."""
    import torch

    c = Case(api, 20, 256, 264, 16, 3, "rows")
    z = torch.zeros(2, 3, 8, device="cuda")
    lab = torch.zeros(2, 3, dtype=torch.int64, device="cuda")
    calls = [lambda ws: c.fwd(workspace=ws), lambda ws: c.bwd(workspace=ws),
             lambda ws: api.qlora_preference_loss(z, lab, z[:, :, 0].contiguous(), 0.1, workspace=ws),
             lambda ws: api.qlora_clip_grad_norm_batch([z], 1.0, workspace=ws)]
    n = 1 << 24
    for call in calls:
        for bad in (torch.empty(n, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(n),
                    torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2]):
            with pytest.raises(ValueError):
                call(bad)
        with pytest.raises(TypeError):
            call(n)
        call(torch.empty(n, dtype=torch.uint8, device="cuda"))
        call(torch.empty(n // 4, device="cuda"))
    torch.cuda.synchronize()


# ---- one adapter or one row beside the others -----------------------------------------------------

def diverged(c, what, a):
    """Infinities and NaN in parts of adapter a."""
    if what == "scale":
        c.d["scale"][a] = NAN
    else:
        t = c.d[what][a]
        t[t.shape[0] // 2, 3] = INF
        t[0, t.shape[1] - 1] = -INF
        t[t.shape[0] - 1, 0] = NAN


def mixed_ids(M, A, skip=None):
    """Every adapter but `skip`, and rows without one (or -1 alone)."""
    pool = [-1] + [a for a in range(A) if a != skip] + [A]
    return [pool[i % len(pool)] for i in range(M)] if M > 1 else [pool[1]]


SIZES = [(1, 512, 512, 64), (1, 320, 264, 16), (6, 512, 264, 16), (16, 512, 512, 64), (13, 640, 264, 24), (33, 512, 264, 16),
         (128, 320, 264, 72), (200, 512, 264, 8), (300, 512, 264, 64), (150, 4096, 264, 16), (150, 256, 4096, 16),
         (700, 256, 264, 72)]


@pytest.mark.parametrize("M,K,N,r", SIZES)
@pytest.mark.parametrize("bad", [0, 2])
@pytest.mark.parametrize("what", ["L1", "L2", "scale"])
def test_a_diverged_adapter_stays_alone(api, M, K, N, r, bad, what):
    """Outputs and gradients of the others' rows and of the others keep their bits, beside its rows or without any."""
    import torch

    say(f"multi alone M={M} K={K} N={N} r={r} adapter {bad} {what}")
    for idle in (False, True):
        c = Case(api, M, K, N, r, 4, "rows")
        set_ids(c, mixed_ids(M, 4, bad if idle or M == 1 else None))
        Y, T = c.fwd(want_T=True)
        back = c.bwd()
        diverged(c, what, bad)
        Y2, T2 = c.fwd(want_T=True)
        back2 = c.bwd()
        back3 = c.bwd(T=T2)
        other = c.d["ids"] != bad
        assert other.any()
        assert torch.equal(Y2[other], Y[other]) and torch.equal(T2[other], T[other])
        for b in (back2, back3):
            assert torch.equal(b[0][other], back[0][other])
            for a in range(4):
                if a != bad or idle:
                    assert torch.equal(b[1][a], back[1][a]) and torch.equal(b[2][a], back[2][a]), a


@pytest.mark.parametrize("M,K,N,r", [s for s in SIZES if s[0] > 1])
@pytest.mark.parametrize("value", [INF, NAN])
def test_a_row_that_is_not_finite_stays_alone(api, M, K, N, r, value):
    import torch

    say(f"multi row alone M={M} K={K} N={N} r={r} {value}")
    c = Case(api, M, K, N, r, 4, "rows")
    set_ids(c, mixed_ids(M, 4))
    Y, T = c.fwd(want_T=True)
    back = c.bwd()
    for m in (0, 1, M - 1):              # a row without an adapter, one of adapter 0, the last one
        a = int(c.ids[m])
        other = torch.arange(M, device="cuda") != m
        x, dy = c.d["X"][m].clone(), c.d["dY"][m].clone()
        c.d["X"][m, [0, K // 2, K - 1]] = value
        c.d["dY"][m, [1, N // 2, N - 1]] = value
        Y2, T2 = c.fwd(want_T=True)
        b = c.bwd()
        c.d["X"][m], c.d["dY"][m] = x, dy
        assert torch.equal(Y2[other], Y[other]) and torch.equal(T2[other], T[other])
        assert torch.equal(b[0][other], back[0][other])
        for k in range(4):
            if k != a:
                assert torch.equal(b[1][k], back[1][k]) and torch.equal(b[2][k], back[2][k]), (m, k)


def test_norm_of_gradients_with_nan(api):
    """As the flat call: norm NaN, coef 1; an infinity gives norm inf and coef 0."""
    import torch

    for value, coef in ((NAN, 1.0), (INF, 0.0)):
        g = torch.ones(300, device="cuda")
        g[7] = value
        flat, both = api.qlora_clip_grad_norm(g, 0.3), api.qlora_clip_grad_norm_batch([g, g.clone()], 0.3)
        for c, n in (flat, both):
            assert c.item() == coef and str(n.item()) == str(value)
