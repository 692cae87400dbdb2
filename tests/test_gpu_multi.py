"""GPU parity of the linear with an adapter per row (qlora_linear_multi_fwd / _bwd)
against the float64 oracle (oracle/multi.py).

Two bars. Y, T and dX meet the single linear's: max |G - R| / RMS(R) <= 2e-2
after taking out the bf16 output's own rounding. Every output also stays, element
by element, within the bound that its roundings give: with u = 2^-24, h = 2^-8
(half a bf16 ulp, relative: 8 significand bits) and a sum of n products off by at most n u times
the sum of their magnitudes,
    E(T)   = K u |X| |L1|,     E(sT) = s E(T) + h |sT|     (s T is rounded to bf16)
    E(Y)   = K u |X| |W| + E(sT) |L2| + r u |sT| |L2|      (M <= 16: + 2 h |X| |W|: the
             GEMV takes q from fp16, which can move a weight to the neighbouring bf16)
    E(sU)  = s N u |dY| |L2| + h |sU|,  E(dX) = N u |dY| |W| + E(sU) |L1| + r u |sU| |L1|
    E(dL1) = X^T E(sU) + n u |X| |sU|,  E(dL2) = s (E(T) + h |T|)^T |dY| + n u |sT| |dY|
(products of matrices of magnitudes) and half an ulp of a bf16 output. An RMS
over gradients that are mostly zeros (adapters without rows) is no measure of
the others' roundings, so dL1 and dL2 have the second bar alone.

The adapters are drawn so large that their term matches the base's: a row that
took another adapter fails at once. Exact identities: a row's result does not
depend on the others' order, rows without an adapter equal the layer with L2 =
0, adapters without rows get zero gradients, repeated calls give the same bits.
"""

import numpy as np
import pytest

from gpu_util import check_output, gpu_quantize, require_gpu, say
from oracle import linear, multi, nf4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    return require_gpu()


def bf16(x):
    return nf4.bf16_rne(np.ascontiguousarray(x, np.float32).reshape(-1)).reshape(x.shape)


def ids_of(kind, M, A, rng):
    if kind == "runs":
        cuts = np.sort(rng.integers(0, M + 1, 2 * A))
        return np.repeat(rng.integers(-1, A, len(cuts) + 1), np.diff(np.concatenate([[0], cuts, [M]])))
    if kind == "rows":
        return rng.integers(-1, A, M)
    if kind == "none":
        return rng.choice([-1, A, A + 7, -2 ** 31, 2 ** 31 - 1], M)
    if kind == "one":
        return np.full(M, A - 1)
    if kind == "few":                    # most adapters have no rows
        return np.where(rng.random(M) < 0.5, A // 2, -1)
    raise ValueError(kind)


U, H = 2.0 ** -24, 2.0 ** -8


def within(label, key, G, R, E):
    """|G - R| <= E (+ half a bf16 ulp for a bf16 output), element by element."""
    bits = np.asarray(G).dtype == np.uint16
    G = linear.widen(G)
    E = 1.01 * E + (1.01 * linear.bf16_half_ulp(np.abs(R) + E) if bits else U * np.abs(R)) + 1e-30
    worst = float((np.abs(G - R) / E).max()) if R.size else 0.0
    say(f"  {label} {key}: {worst:.3f} of its bound")
    assert worst <= 1.0, (label, key, worst)


class Bounds:
    """The bounds of the module's docstring for one case."""

    def __init__(self, c, T):
        X, W, L1, L2, dY = (np.abs(linear.widen(a)) for a in (c.X, c.W, c.L1, c.L2, c.dY))
        M, K, N, r = c.M, c.K, c.N, c.r
        s = np.abs(c.scale.astype(np.float64))
        self.T, self.Y = np.zeros((M, r)), (K * U + (2 * H if M <= 16 else 0.0)) * (X @ W.T)
        self.dX = N * U * (dY @ W)
        self.dL1, self.dL2 = np.zeros(L1.shape), np.zeros(L2.shape)
        for a, at in enumerate(multi.rows_of(c.ids, c.A)):
            t, n = np.abs(T[at]), len(at)
            self.T[at] = K * U * (X[at] @ L1[a])
            est = s[a] * (self.T[at] + H * t)
            self.Y[at] += est @ L2[a] + r * U * s[a] * (t @ L2[a])
            mag = s[a] * (dY[at] @ L2[a].T)
            u = s[a] * np.abs(linear.widen(c.dY)[at] @ linear.widen(c.L2)[a].T)
            esu = N * U * mag + H * u
            self.dX[at] += esu @ L1[a].T + r * U * (u @ L1[a].T)
            self.dL1[a] = X[at].T @ esu + n * U * (X[at].T @ u)
            self.dL2[a] = est.T @ dY[at] + n * U * s[a] * (t.T @ dY[at])


class Case:
    def __init__(self, api, M, K, N, r, A, kind, qtype="nf4", dq=True, seed=None):
        import torch

        rng = np.random.default_rng(seed if seed is not None else M * 7 + K + N + r + A)
        self.api, self.M, self.K, self.N, self.r, self.A = api, M, K, N, r, A
        W = (0.02 * rng.standard_normal((N, K))).astype(np.float32)
        self.q, _ = gpu_quantize(api, W, qtype=qtype, double_quant=dq)
        self.W = api.to_host_bits(api.qlora_dequantize(self.q))
        self.X = bf16(rng.standard_normal((M, K)))
        self.dY = bf16(rng.standard_normal((M, N)))
        self.L1 = bf16(rng.standard_normal((A, K, r)) / np.sqrt(K))
        self.L2 = bf16(rng.standard_normal((A, r, N)) * 0.02 * np.sqrt(K / r))
        self.scale = rng.choice([0.25, 0.5, 1.0, 2.0], A).astype(np.float32)
        self.ids = ids_of(kind, M, A, rng).astype(np.int32)
        d = api.to_device_bf16
        self.d = dict(X=d(self.X), L1=d(self.L1), L2=d(self.L2), dY=d(self.dY), ids=torch.from_numpy(self.ids).cuda(),
                      scale=torch.from_numpy(self.scale).cuda())

    def fwd(self, **kw):
        d = self.d
        return self.api.qlora_linear_multi_fwd(self.q, d["X"], d["ids"], d["L1"], d["L2"], d["scale"], **kw)

    def bwd(self, **kw):
        d = self.d
        return self.api.qlora_linear_multi_bwd(self.q, d["X"], d["dY"], d["ids"], d["L1"], d["L2"], d["scale"], **kw)

    def check_fwd(self, label):
        Y, T = self.fwd(want_T=True)
        Yr, Tr = multi.multi_fwd(self.X, self.W, self.ids, self.L1, self.L2, self.scale)
        check_output(label, "Y", self.api.to_host_bits(Y), Yr)
        check_output(label, "T", self.api.to_host_bits(T), Tr)
        self.bounds = Bounds(self, Tr)
        within(label, "Y", self.api.to_host_bits(Y), Yr, self.bounds.Y)
        within(label, "T", self.api.to_host_bits(T), Tr, self.bounds.T)
        bare = (self.ids < 0) | (self.ids >= self.A)
        assert (self.api.to_host_bits(T)[bare] == 0).all()
        assert (self.api.to_host_bits(self.fwd()[0]) == self.api.to_host_bits(Y)).all()
        return T

    def check_bwd(self, label, T):
        import torch

        ref = dict(zip(("dX", "dL1", "dL2"), multi.multi_bwd(self.X, self.W, self.ids, self.L1, self.L2, self.scale, self.dY)))
        first = self.bwd(T=T)
        for how, out in (("T kept", first), ("T again", self.bwd())):
            check_output(label + " " + how, "dX", self.api.to_host_bits(out[0]), ref["dX"])
            within(label + " " + how, "dX", self.api.to_host_bits(out[0]), ref["dX"], self.bounds.dX)
            within(label + " " + how, "dL1", out[1].cpu().numpy(), ref["dL1"], self.bounds.dL1)
            within(label + " " + how, "dL2", out[2].cpu().numpy(), ref["dL2"], self.bounds.dL2)
            empty = [a for a in range(self.A) if not (self.ids == a).any()]
            assert (out[1][empty] == 0).all() and (out[2][empty] == 0).all()
        for a, b in zip(first, self.bwd(T=T)):
            assert torch.equal(a, b)
        none, d1, d2 = self.bwd(T=T, need_dX=False)
        assert none is None and torch.equal(d1, first[1]) and torch.equal(d2, first[2])
        b = self.bwd(T=T, grad_dtype=torch.bfloat16)
        assert torch.equal(b[1], first[1].bfloat16()) and torch.equal(b[2], first[2].bfloat16())


# M, K, N, r, A, kind
FWD = [
    (1, 512, 512, 64, 3, "one"),           # one token
    (1, 512, 512, 16, 3, "none"),
    (1, 320, 72, 8, 1, "one"),             # one token, a shape beyond the single-token kernel
    (2, 512, 520, 64, 5, "rows"),
    (3, 256, 40, 8, 2, "rows"),
    (4, 64 * 41, 200, 64, 4, "rows"),      # odd number of 64-blocks
    (7, 512, 264, 256, 3, "rows"),         # the largest rank
    (13, 1024, 512, 16, 32, "rows"),       # more adapters than rows
    (16, 640, 1032, 64, 16, "rows"),
    (16, 640, 1032, 32, 2, "runs"),
    (16, 512, 16, 24, 40, "few"),
    (9, 512, 512, 72, 9, "none"),
    (17, 256, 264, 8, 4, "rows"),
    (33, 448, 136, 40, 7, "runs"),
    (96, 512, 1040, 16, 24, "rows"),
    (100, 320, 200, 136, 3, "few"),
    (128, 256, 264, 64, 128, "rows"),
    (128, 512, 512, 16, 1, "one"),
    (64, 512, 512, 16, 5, "none"),
    (129, 256, 264, 64, 5, "rows"),
    (200, 320, 136, 16, 6, "runs"),
    (300, 512, 600, 200, 40, "rows"),
    (391, 1024, 768, 32, 4, "runs"),
    (700, 256, 264, 8, 70, "rows"),        # more segments than lanes in a wave
    (1000, 512, 520, 64, 300, "rows"),
    (513, 256, 512, 64, 2, "few"),
    (600, 256, 264, 16, 4, "none"),
    (1030, 256, 4160, 16, 3, "one"),
    (320, 256, 264, 8, 45, "rows"),        # eight segments to a group, several groups to a tile
    (300, 256, 136, 16, 3, "rows"),        # a group that is not full
    (260, 128, 264, 24, 33, "rows"),
]


@pytest.mark.parametrize("M,K,N,r,A,kind", FWD)
def test_forward(api, M, K, N, r, A, kind):
    label = f"multi fwd M={M} K={K} N={N} r={r} A={A} {kind}"
    say(label)
    Case(api, M, K, N, r, A, kind).check_fwd(label)


BWD = [
    (1, 320, 72, 8, 2, "one"),
    (5, 256, 264, 24, 8, "rows"),
    (64, 512, 512, 64, 3, "runs"),
    (130, 448, 328, 256, 2, "rows"),       # the largest rank, N not a multiple of 64
    (200, 320, 136, 16, 6, "runs"),
    (391, 512, 768, 32, 4, "runs"),
    (700, 256, 264, 8, 70, "rows"),
    (300, 256, 512, 72, 5, "none"),
    (2500, 256, 512, 64, 2, "few"),        # a segment of several pieces, and adapters without rows
    (4200, 320, 256, 16, 3, "one"),
    (1000, 512, 520, 64, 300, "rows"),
    (320, 256, 264, 8, 45, "rows"),
    (300, 192, 136, 24, 7, "rows"),
    (260, 128, 192, 32, 33, "few"),
]


@pytest.mark.parametrize("M,K,N,r,A,kind", BWD)
def test_backward(api, M, K, N, r, A, kind):
    label = f"multi bwd M={M} K={K} N={N} r={r} A={A} {kind}"
    say(label)
    c = Case(api, M, K, N, r, A, kind)
    c.check_bwd(label, c.check_fwd(label))


# a few rows per adapter: pieces that end inside an MFMA step, one and two stages of rows, groups of small ranks
FEW = [(2, 8, 2), (15, 8, 9), (16, 64, 1), (17, 64, 1), (31, 16, 5), (33, 64, 33), (63, 24, 2), (65, 64, 1), (88, 8, 44),
       (127, 32, 1), (128, 16, 128), (129, 64, 1), (190, 40, 1)]


@pytest.mark.parametrize("M,r,A", FEW)
def test_backward_of_few_rows(api, M, r, A):
    label = f"multi bwd of few rows M={M} r={r} A={A}"
    say(label)
    c = Case(api, M, 320, 264, r, A, "rows" if A > 1 else "one")
    c.check_bwd(label, c.check_fwd(label))


@pytest.mark.parametrize("M,K", [(20, 4096), (30, 1088), (50, 2048), (17, 640)])
def test_many_slices(api, M, K):
    """Narrow weights: the base product of up to 128 rows in many slices of the reduction."""
    label = f"multi fwd many slices M={M} K={K}"
    say(label)
    Case(api, M, K, 136, 16, 3, "rows").check_fwd(label)


@pytest.mark.parametrize("qtype,dq", [("nf4", False), ("int4", True), ("fp4_e2m1", False)])
@pytest.mark.parametrize("M", [1, 6, 50, 200])
def test_other_weight_formats(api, M, qtype, dq):
    label = f"multi {qtype} dq={dq} M={M}"
    say(label)
    c = Case(api, M, 512, 264, 16, 4, "rows", qtype=qtype, dq=dq)
    T = c.check_fwd(label)
    if M == 200:
        c.check_bwd(label, T)


@pytest.mark.parametrize("M", [5, 16, 60, 128, 300])
def test_order_of_rows(api, M):
    """Permuted rows give permuted results, bit for bit."""
    import torch

    say(f"multi order M={M}")
    c = Case(api, M, 512, 264, 24, 6, "rows")
    Y, T = c.fwd(want_T=True)
    dX = c.bwd(T=T)[0]
    p = torch.from_numpy(np.random.default_rng(1).permutation(M)).cuda()
    for k in ("X", "ids", "dY"):
        c.d[k] = c.d[k][p].contiguous()
    Y2, T2 = c.fwd(want_T=True)
    assert torch.equal(Y2, Y[p]) and torch.equal(T2, T[p])
    assert torch.equal(c.bwd(T=T2)[0], dX[p])


@pytest.mark.parametrize("M,r,A", [(150, 24, 40), (300, 72, 3), (260, 8, 130)])
def test_order_of_rows_in_slices(api, M, r, A):
    """The same where the reduction is cut into slices, against the oracle too."""
    import torch

    label = f"multi order in slices M={M} r={r} A={A}"
    say(label)
    c = Case(api, M, 4096, 264, r, A, "rows")
    c.check_fwd(label)
    Y = c.fwd()[0]
    p = torch.from_numpy(np.random.default_rng(2).permutation(M)).cuda()
    for k in ("X", "ids"):
        c.d[k] = c.d[k][p].contiguous()
    assert torch.equal(c.fwd()[0], Y[p])


@pytest.mark.parametrize("M,r,A", [(150, 24, 40), (200, 72, 3), (330, 8, 130)])
def test_backward_in_slices(api, M, r, A):
    label = f"multi bwd in slices M={M} r={r} A={A}"
    say(label)
    c = Case(api, M, 256, 4096, r, A, "rows")
    c.check_bwd(label, c.check_fwd(label))


@pytest.mark.parametrize("M", [1, 7, 16, 40, 128, 200])
def test_rows_without_an_adapter(api, M):
    """They equal the layer whose second factor is zero, whatever the other rows do."""
    import torch

    say(f"multi bare M={M}")
    c = Case(api, M, 512, 264, 16, 3, "rows")
    if M == 1:
        c.d["ids"][:] = -1
    Y = c.fwd()[0]
    bare = (c.d["ids"] < 0) | (c.d["ids"] >= 3)
    assert bare.any()
    c.d["L2"].zero_()
    assert torch.equal(c.fwd()[0][bare], Y[bare])


@pytest.mark.parametrize("M,K,r", [(1, 512, 16), (7, 512, 16), (16, 512, 64), (13, 640, 24), (60, 512, 16), (128, 320, 72),
                                   (200, 512, 8), (300, 512, 64), (150, 4096, 16), (700, 256, 72)])
def test_an_adapter_that_diverged(api, M, K, r):
    """Infinities and NaN of one adapter's second factor reach its own rows alone, and there their own columns."""
    import torch

    say(f"multi diverged M={M} K={K} r={r}")
    c = Case(api, M, K, 264, r, 4, "rows")
    c.d["ids"][0] = 1
    Y = c.fwd()[0]
    c.d["L2"][1, 3, 5] = float("inf")
    c.d["L2"][1, 2, 9] = float("nan")
    c.d["L2"][1, 0, 200] = float("-inf")
    Y2 = c.fwd()[0]
    own = c.d["ids"] == 1
    assert torch.equal(Y2[~own], Y[~own])
    hit = torch.zeros(264, dtype=torch.bool, device="cuda")
    hit[[5, 9, 200]] = True
    assert torch.equal(Y2[:, ~hit], Y[:, ~hit])
    assert not torch.isfinite(Y2[own][:, hit]).any() and torch.isnan(Y2[own][:, 9]).all()


@pytest.mark.parametrize("M,N,r", [(5, 264, 16), (200, 264, 64), (300, 512, 8), (150, 4096, 16), (150, 4096, 64), (700, 256, 72)])
def test_an_adapter_that_diverged_backward(api, M, N, r):
    import torch

    say(f"multi diverged bwd M={M} N={N} r={r}")
    c = Case(api, M, 320, N, r, 4, "rows")
    c.d["ids"][0] = 1
    T = c.fwd(want_T=True)[1]
    dX = c.bwd(T=T)[0]
    c.d["L1"][1, 6, 3] = float("inf")
    c.d["L1"][1, 70, 2] = float("nan")
    dX2 = c.bwd(T=T)[0]
    own = c.d["ids"] == 1
    assert torch.equal(dX2[~own], dX[~own])
    hit = torch.zeros(320, dtype=torch.bool, device="cuda")
    hit[[6, 70]] = True
    assert torch.equal(dX2[:, ~hit], dX[:, ~hit])
    assert not torch.isfinite(dX2[own][:, hit]).any() and torch.isnan(dX2[own][:, 70]).all()


def test_no_rows(api):
    import torch

    c = Case(api, 0, 256, 264, 16, 3, "rows")
    Y, T = c.fwd(want_T=True)
    assert Y.shape == (0, 264) and T.shape == (0, 16)
    dX, dL1, dL2 = c.bwd()
    assert dX.shape == (0, 256) and (dL1 == 0).all() and (dL2 == 0).all()
    torch.cuda.synchronize()


@pytest.mark.parametrize("M", [1, 9, 50, 300])
def test_stream_and_graph(api, M):
    """On another stream, and replayed from a graph with eager work between."""
    import torch

    c = Case(api, M, 512, 264, 16, 5, "rows")
    s = torch.cuda.Stream()
    want, T = c.fwd(want_T=True)
    back = c.bwd(T=T)
    torch.cuda.synchronize()
    got = c.fwd(stream=s)[0]
    got_back = c.bwd(T=T, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    for a, b in zip(got_back, back):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        Yg, Tg = c.fwd(want_T=True)
        Bg = c.bwd(T=Tg)
    for k in range(4):
        c.d["ids"].copy_(torch.roll(c.d["ids"], 1))          # other groups than at the capture
        want, T = c.fwd(want_T=True)
        back = c.bwd(T=T)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Yg, want) and torch.equal(Tg, T), k
        for a, b in zip(Bg, back):
            assert torch.equal(a, b), k


def test_rows_beyond_32_bit_offsets(api):
    """Rows that span more than 4 GB: the dense GEMM's variant with 64-bit addresses."""
    import torch

    M, K, N, r, A = 540000, 4096, 64, 8, 3
    say(f"multi M={M} K={K}: {M * K * 2 / 2 ** 30:.1f} GiB of rows")
    c = Case(api, 300, K, N, r, A, "rows")
    X = c.d["X"].repeat(M // 300, 1)
    ids = c.d["ids"].repeat(M // 300)
    Y = api.qlora_linear_multi_fwd(c.q, X, ids, c.d["L1"], c.d["L2"], c.d["scale"])[0]
    blocks = Y.view(M // 300, 300, N)
    assert torch.equal(blocks, blocks[:1].expand(M // 300, 300, N))     # the same 300 rows over and over
    Yr, Tr = multi.multi_fwd(c.X, c.W, c.ids, c.L1, c.L2, c.scale)
    within("rows beyond 4 GB", "Y", api.to_host_bits(blocks[0]), Yr, Bounds(c, Tr).Y)


def test_refusals(api):
    import torch

    c = Case(api, 20, 256, 264, 16, 3, "rows")
    d = c.d
    call = lambda **kw: api.qlora_linear_multi_fwd(c.q, **{**dict(X=d["X"], row_adapter=d["ids"], L1=d["L1"], L2=d["L2"],  # noqa: E731
                                                                  scale=d["scale"]), **kw})
    with pytest.raises(TypeError):
        call(row_adapter=d["ids"].long())
    with pytest.raises(ValueError):
        call(row_adapter=d["ids"][:-1])
    with pytest.raises(ValueError):
        call(X=d["X"][:, :-64])
    with pytest.raises(TypeError):
        call(X=d["X"].float())
    with pytest.raises(ValueError):
        call(L2=d["L2"][:2])
    with pytest.raises(ValueError):
        call(scale=d["scale"][:2])
    with pytest.raises(ValueError):
        call(X=torch.cat([d["X"], d["X"]], 1)[:, :256])
    with pytest.raises(api.QLoRAError):
        call(L1=d["L1"][:, :, :4].contiguous(), L2=d["L2"][:, :4].contiguous())
    with pytest.raises(api.QLoRAError):
        call(L1=d["L1"][:0], L2=d["L2"][:0], scale=d["scale"][:0])
    with pytest.raises(ValueError):
        call(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        c.bwd(grad_dtype=torch.float16)
    with pytest.raises(ValueError):
        c.bwd(T=torch.zeros(20, 8, dtype=torch.bfloat16, device="cuda"))
