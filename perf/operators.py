"""The operators around many adapters on one quantised base, as a user runs them.

One frozen NF4 weight serves rows of several adapters at once (and rows of
none: a reference model), forward and backward; a preference loss gives the
gradient of the logits; the optimiser clips and steps all adapter tensors in
one call. ``own`` selects the library's entry points or the plain form of
elementary torch operations.
"""

import math
import random
import statistics

import numpy as np
import torch

own = False

BLOCK, GROUP = 64, 256      # weights per absmax constant, constants per second-level scale
STATE_BLOCK = 256           # optimiser-state values per scale
SCALES = (0.25, 1.0, 2.0)   # LoRA scales (alpha / r) the adapters are drawn with


def listed():
    return [
        # one token of one request among 8 resident adapters: the latency of a decode step's largest linear
        dict(name="linear-token", op="linear_fwd", M=1, K=4096, N=11008, r=64, A=8, runs=False, bare=0.0),
        # a decode step of 13 requests, each with its own small adapter, some on the bare base
        dict(name="linear-decode", op="linear_fwd", M=13, K=11008, N=4096, r=16, A=32, runs=False, bare=0.15),
        # a batched decode step of 96 requests over 24 adapters
        dict(name="linear-batch", op="linear_fwd", M=96, K=4096, N=11008, r=16, A=24, runs=False, bare=0.1),
        # prompts of 12 adapters' requests and of the reference model (rows without an adapter), one after another
        dict(name="linear-prefill", op="linear_fwd", M=4096, K=4096, N=11008, r=64, A=12, runs=True, bare=0.2),
        # training: a short ragged batch of 4 adapters on a square projection
        dict(name="linear-bwd-short", op="linear_bwd", M=391, K=4096, N=4096, r=32, A=4, runs=True, bare=0.0, keep=False),
        # training: 8192 tokens of 16 adapters on the widest linear
        dict(name="linear-bwd", op="linear_bwd", M=8192, K=4096, N=11008, r=64, A=16, runs=True, bare=0.1, keep=True),
        # two short preference pairs: the latency of the loss
        dict(name="preference-short", op="preference", pairs=2, T=64, V=32000, f32=False, eps=0.0, spans=3),
        # fp32 logits over an odd vocabulary (one token added): rows that start unaligned
        dict(name="preference-odd", op="preference", pairs=4, T=333, V=32001, f32=True, eps=0.1, spans=5),
        # eight long pairs
        dict(name="preference-long", op="preference", pairs=8, T=1024, V=32000, f32=False, eps=0.0, spans=7),
        # the adapters of one layer's linears, rank 8, fp32 state: the latency of a step
        dict(name="adamw-layer", op="adamw", layers=1, hidden=4096, ffn=11008, r=8, bits=32, g32=True),
        # many tensors of odd sizes, 8-bit state, bf16 gradients
        dict(name="adamw-ragged", op="adamw", tensors=150, mean=40000, shapes=11, bits=8, g32=False),
        # every adapter of a 32-layer model, rank 64: 448 tensors, 160 M parameters, 8-bit state
        dict(name="adamw-model", op="adamw", layers=32, hidden=4096, ffn=11008, r=64, bits=8, g32=True),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def draw(rng):
    while True:
        case = _draw(rng)
        if 3072 not in case.values():   # a width that no configuration here has
            return case


def _draw(rng):
    op = rng.choice(("linear_fwd", "linear_fwd", "linear_bwd", "preference", "adamw"))
    if op.startswith("linear"):
        K = 64 * round(_log(rng, 16, 172))
        N = 8 * round(_log(rng, 128, 1376))
        if op == "linear_bwd" and rng.random() < 0.7:
            N = max(64, N // 64 * 64)
        M = round(_log(rng, 1, 4096) if op == "linear_fwd" else _log(rng, 48, 8192))
        M = max(1, min(M, int(8192 * 4096 * 11008 / (K * N))))
        case = dict(op=op, M=M, K=K, N=N, r=8 * round(_log(rng, 1, 16)), A=round(_log(rng, 1, 48)),
                    runs=rng.random() < 0.5, bare=round(rng.choice((0.0, 0.1, 0.5)), 2))
        if op == "linear_bwd":
            case["keep"] = rng.random() < 0.5
        return case
    if op == "preference":
        V = round(_log(rng, 4000, 64000))
        if rng.random() < 0.5:
            V = V // 8 * 8
        f32 = rng.random() < 0.4
        pairs = round(_log(rng, 1, 12))
        T = max(1, min(round(_log(rng, 16, 2048)), int(8 * 1024 * 32000 / (pairs * V)) // (2 if f32 else 1)))
        return dict(op=op, pairs=pairs, T=T, V=V, f32=f32, eps=rng.choice((0.0, 0.1)), spans=rng.randrange(1 << 20))
    mean = _log(rng, 300, 1e6)
    return dict(op=op, tensors=max(1, min(round(_log(rng, 1, 300)), int(5e7 / mean))), mean=round(mean),
                shapes=rng.randrange(1 << 20), bits=rng.choice((8, 8, 32)), g32=rng.random() < 0.5)


# ---- what the cases are made of -------------------------------------------------------

def _sizes(c):
    """Elements of each adapter tensor of an optimiser case."""
    if "layers" in c:
        h, f, r = c["hidden"], c["ffn"], c["r"]
        one = [n * r for k, o in ((h, h),) * 4 + ((h, f),) * 2 + ((f, h),) for n in (k, o)]
        return one * c["layers"]
    rng = random.Random(c["shapes"])
    return [max(1, round(c["mean"] * math.exp(rng.uniform(-1.5, 0.8)))) for _ in range(c["tensors"])]


def _spans(c):
    """(prompt, end) of each sequence: positions [prompt, end) count; a pair shares its prompt."""
    rng = random.Random(c["spans"])
    T = c["T"]
    prompts = [rng.randrange(0, max(1, T // 3)) for _ in range(c["pairs"])]
    return [(p, max(min(p + 1, T), T - rng.randrange(0, max(1, T // 3)))) for p in prompts + prompts]


def _row_adapters(c, rng):
    """Adapter of each row, -1 for none: whole requests one after another, or any order."""
    M, A = c["M"], c["A"]
    pick = lambda: -1 if rng.random() < c["bare"] else rng.randrange(A)  # noqa: E731
    if not c["runs"]:
        return [pick() for _ in range(M)]
    cuts = sorted(rng.randrange(M) for _ in range(2 * A))
    return [a for lo, hi in zip([0] + cuts, cuts + [M]) for a in [pick()] * (hi - lo)]


def _codebook():
    """The 16 NF4 values: midpoints of normal quantiles, negative side from 15 values, positive from 17."""
    inv = statistics.NormalDist().inv_cdf

    def half(c):
        v = [0.5 * (inv(i / (c + 2)) + inv((i + 1) / (c + 2))) for i in range(1, c + 1)]
        v[c // 2] = 0.0
        return v

    a, b = half(15), half(17)
    return [x / -a[0] for x in a[:7]] + [0.0] + [x / b[16] for x in b[9:]]


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    rng = random.Random(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device=dev).normal_(0.0, std, generator=g)

    s = dict(case=dict(c))
    if c["op"].startswith("linear"):
        M, K, N, r, A = c["M"], c["K"], c["N"], c["r"], c["A"]
        nb = -(-N * K // BLOCK)
        ng = -(-nb // GROUP)
        s["codes"] = torch.randint(0, 256, (N * K // 2,), generator=g, device=dev, dtype=torch.uint8)
        s["absmax8"] = (normal(nb, dtype=torch.float32).clamp(-3.9, 3.9) * 112.0).to(torch.float8_e4m3fn).view(torch.uint8)
        s["scale2"] = 7e-5 * (1.0 + 0.1 * torch.rand(ng, generator=g, device=dev))
        s["mean"] = torch.full((1,), 0.048, device=dev)
        s["book"] = torch.tensor(_codebook(), dtype=torch.float32, device=dev)
        s["X"] = normal(M, K)
        s["L1"] = normal(A, K, r, std=K ** -0.5)
        s["L2"] = normal(A, r, N, std=0.05)
        s["scale"] = torch.tensor([rng.choice(SCALES) for _ in range(A)], device=dev)
        s["ids"] = torch.tensor(_row_adapters(c, rng), dtype=torch.int32, device=dev)
        if c["op"] == "linear_bwd":
            s["dY"] = normal(M, N, std=0.1)
            s["T"] = _down(s["X"].float(), s["L1"].float(), s["ids"]).to(torch.bfloat16) if c["keep"] else None
    elif c["op"] == "preference":
        S, T, V = 2 * c["pairs"], c["T"], c["V"]
        dtype = torch.float32 if c["f32"] else torch.bfloat16
        s["logits"] = normal(S, T, V, std=2.0, dtype=dtype)
        labels = torch.randint(0, V, (S, T), generator=g, device=dev)
        # the language model puts weight on its labels
        s["logits"].scatter_add_(2, labels[..., None], torch.full((S, T, 1), 5.0, dtype=dtype, device=dev))
        pos = torch.arange(T, device=dev)
        lo, hi = (torch.tensor(v, device=dev)[:, None] for v in zip(*_spans(c)))
        s["labels"] = torch.where((pos >= lo) & (pos < hi), labels, -100)
        lp = torch.stack([x.float().gather(1, y[:, None])[:, 0] - x.float().logsumexp(1) for x, y in zip(s["logits"], labels)])
        # some training in, both sequences of a pair have lost weight against the reference
        s["ref"] = lp + 0.05 + normal(S, T, std=0.3, dtype=torch.float32)
        s["beta"], s["eps"] = 0.1, c["eps"]
    else:
        sizes = _sizes(c)
        at = [0]
        for n in sizes:
            at.append(at[-1] + -(-n // STATE_BLOCK) * STATE_BLOCK)
        n = at[-1]
        # the tensors lie in one allocation, each from a multiple of the state block
        cut = lambda flat: [flat[o:o + k] for o, k in zip(at, sizes)]  # noqa: E731
        s["theta"], s["theta16"] = normal(n, std=0.02, dtype=torch.float32), torch.zeros(n, dtype=torch.bfloat16, device=dev)
        grad = normal(n, std=0.01, dtype=torch.float32)
        inside = torch.zeros(n, dtype=torch.bool, device=dev)
        for o, k in zip(at, sizes):
            inside[o:o + k] = True
        # heavy-tailed magnitudes: coordinates and blocks that see much larger gradients than others
        grad.mul_(torch.empty_like(grad).log_normal_(0.0, 1.5, generator=g))
        zero = ~inside
        grad[zero] = 0
        s["theta"][zero] = 0
        s["grad"] = grad if c["g32"] else grad.to(torch.bfloat16)
        m, root = 0.3 * grad + normal(n, std=0.003, dtype=torch.float32), grad.abs() * torch.empty_like(grad).log_normal_(0.0, 0.3, generator=g)
        m[zero] = 0
        if c["bits"] == 8:
            s["m"], s["m_scale"] = _encode(m, False)
            s["v"], s["v_scale"] = _encode(root, True)
        else:
            s["m"], s["v"], s["m_scale"], s["v_scale"] = m, root * root, None, None
        s["sizes"] = sizes
        s["thetas"], s["thetas16"], s["grads"] = cut(s["theta"]), cut(s["theta16"]), cut(s["grad"])
        s["inside"] = inside
        s["max_norm"], s["step"], s["lr"], s["wd"] = 0.3, 20, 1e-3, 0.01
        # the step's constants in 32 bits, on the device
        b1, b2 = float(np.float32(0.9)), float(np.float32(0.999))
        s["b"] = (b1, b2, float(np.float32(1.0 - b1)), float(np.float32(1.0 - b2)))
        s["bc"] = torch.tensor([1.0 - b1 ** s["step"], 1.0 - b2 ** s["step"]], dtype=torch.float32, device=dev)
    return s


# ---- plain forms --------------------------------------------------------------------------

def _weight(s):
    """The dequantised weight [N][K] in bf16's values: bf16(q[code] * (e4m3(c8) * scale2 + mean))."""
    c = s["case"]
    codes = torch.stack((s["codes"] & 15, s["codes"] >> 4), 1).reshape(-1, BLOCK).long()
    sc = s["scale2"].repeat_interleave(GROUP)[:s["absmax8"].numel()]
    a = s["absmax8"].view(torch.float8_e4m3fn).float() * sc + s["mean"]
    return (s["book"][codes] * a[:, None]).to(torch.bfloat16).float().reshape(c["N"], c["K"])


def _one_hot(ids, A):
    """[M][A]: 1 where the row has the adapter; rows of no adapter are 0."""
    return (ids[:, None] == torch.arange(A, device=ids.device, dtype=ids.dtype)).to(torch.float32)


def _down(X, L1, ids):
    """T[m] = X[m] L1[ids[m]], 0 for rows without an adapter."""
    A, K, r = L1.shape
    every = (X @ L1.permute(1, 0, 2).reshape(K, A * r)).reshape(-1, A, r)
    return (every * _one_hot(ids, A).to(X.dtype)[:, :, None]).sum(1)


def _linear_fwd(s):
    X, L1, L2 = s["X"].float(), s["L1"].float(), s["L2"].float()
    A, r, N = L2.shape
    wide = _one_hot(s["ids"], A)[:, :, None] * (_down(X, L1, s["ids"])[:, None, :] * s["scale"][:, None])
    return (X @ _weight(s).t() + wide.reshape(-1, A * r) @ L2.reshape(A * r, N)).to(torch.bfloat16)


def _linear_bwd(s):
    X, dY, L1, L2 = s["X"].float(), s["dY"].float(), s["L1"].float(), s["L2"].float()
    A, r, N = L2.shape
    K = X.shape[1]
    on = _one_hot(s["ids"], A)[:, :, None]
    T = s["T"].float() if s["T"] is not None else _down(X, L1, s["ids"])
    wide_l2, wide_l1 = L2.reshape(A * r, N), L1.permute(0, 2, 1).reshape(A * r, K)
    dU = ((dY @ wide_l2.t()).reshape(-1, A, r) * on * s["scale"][:, None]).reshape(-1, A * r)
    sT = (T[:, None, :] * on * s["scale"][:, None]).reshape(-1, A * r)
    dX = dY @ _weight(s) + dU @ wide_l1
    dL1 = (dU.t() @ X).reshape(A, r, K).permute(0, 2, 1)
    dL2 = (sT.t() @ dY).reshape(A, r, N)
    return dX.to(torch.bfloat16), dL1.to(torch.bfloat16).contiguous(), dL2.to(torch.bfloat16)


def _preference(s):
    x, labels = s["logits"].float(), s["labels"]
    P = x.shape[0] // 2
    counts = (labels >= 0) & (labels < x.shape[2])
    y = torch.where(counts, labels, 0)[..., None]
    top = x.amax(2, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(2, keepdim=True)
    lp = torch.where(counts, (x.gather(2, y) - top - torch.log(total))[..., 0], 0.0)
    reward = s["beta"] * torch.where(counts, lp - s["ref"], 0.0).sum(1)
    h = reward[:P] - reward[P:]
    soft = lambda z: torch.clamp(-z, min=0.0) + torch.log1p(torch.exp(-z.abs()))  # noqa: E731  -log(sigmoid(z))
    loss = ((1.0 - s["eps"]) * soft(h) + s["eps"] * soft(-h)).mean()
    d = (s["beta"] / P) * (1.0 / (1.0 + torch.exp(h)) - s["eps"])   # -d loss / d logp of the preferred sequence
    w = torch.where(counts, torch.cat((-d, d))[:, None], 0.0)[..., None]
    grad = (-w / total) * e
    grad.scatter_add_(2, y, w)
    return loss.reshape(1), reward, lp, grad.to(s["logits"].dtype)


def _encode(v, keep):
    """E4M3 values and scales of blocks of 256; with ``keep`` no value but 0 becomes 0."""
    b = v.reshape(-1, STATE_BLOCK)
    top = b.abs().amax(1)
    top = torch.where(top < 2.0 ** -100, 0.0, top)
    inv = torch.where(top > 0, 448.0 / torch.where(top > 0, top, 1.0), 0.0)
    x = b * inv[:, None]
    if keep:
        x = torch.where(x > 0, torch.clamp(x, min=2.0 ** -9), x)
    return x.to(torch.float8_e4m3fn).reshape(-1), top / 448.0


def _decode(q, scale):
    return (q.float().reshape(-1, STATE_BLOCK) * scale[:, None]).reshape(-1)


def _adamw(s):
    b1, b2, o1, o2 = s["b"]
    g = s["grad"].float()
    norm = torch.sqrt((g * g).sum())
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    g = coef * g
    if s["case"]["bits"] == 8:
        m, root = _decode(s["m"], s["m_scale"]), _decode(s["v"], s["v_scale"])
        v = root * root
    else:
        m, v = s["m"], s["v"]
    m = b1 * m + o1 * g
    v = b2 * v + o2 * (g * g)
    upd = (m / s["bc"][0]) / (torch.sqrt(v / s["bc"][1]) + 1e-8)
    theta = s["theta"] - s["lr"] * (upd + s["wd"] * s["theta"])
    s["theta"].copy_(theta)
    s["theta16"].copy_(theta)
    if s["case"]["bits"] == 8:
        q, scale = _encode(m, False)
        s["m"].copy_(q)
        s["m_scale"].copy_(scale)
        q, scale = _encode(torch.sqrt(v), True)
        s["v"].copy_(q)
        s["v_scale"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return coef


def _state_out(s, coef):
    out = [coef.reshape(1), s["theta"], s["theta16"], s["m"], s["v"]]
    return out + [s["m_scale"], s["v_scale"]] if s["case"]["bits"] == 8 else out


# ---- one pass -------------------------------------------------------------------------------

def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        if op == "linear_fwd":
            return _linear_fwd(s)
        if op == "linear_bwd":
            return _linear_bwd(s)
        if op == "preference":
            return _preference(s)
        return _state_out(s, _adamw(s))

    from bit_nf4_quantized_amd import api

    if op.startswith("linear"):
        q = api.NF4Tensor(s["case"]["N"], s["case"]["K"], s["codes"], s["absmax8"], s["scale2"], s["mean"])
        if op == "linear_fwd":
            return api.qlora_linear_multi_fwd(q, s["X"], s["ids"], s["L1"], s["L2"], s["scale"])[0]
        return api.qlora_linear_multi_bwd(q, s["X"], s["dY"], s["ids"], s["L1"], s["L2"], s["scale"], T=s["T"],
                                          grad_dtype=torch.bfloat16)
    if op == "preference":
        o = api.qlora_preference_loss(s["logits"], s["labels"], s["ref"], s["beta"], label_smoothing=s["eps"])
        return o.loss, o.rewards, o.logps, o.dlogits
    adam = api.AdamWState(s["case"]["bits"], s["sizes"], s["m"], s["v"], s["m_scale"], s["v_scale"])
    coef, _ = api.qlora_clip_grad_norm_batch(s["grads"], s["max_norm"])
    api.qlora_adamw_batch(s["thetas"], s["grads"], adam, s["step"], s["lr"], 0.9, 0.999, 1e-8, s["wd"], coef=coef,
                          thetas_bf16=s["thetas16"])
    return _state_out(s, coef)


def work(case):
    """Bytes: each input once, each output once. Flops: the products (a loss: some 6 per logit; a step: some 20 per value)."""
    c = case
    if c["op"].startswith("linear"):
        M, K, N, r = c["M"], c["K"], c["N"], c["r"]
        w = N * K / 2 + N * K / BLOCK + 4 * N * K / (BLOCK * GROUP)
        # the adapters that rows can have; rows without one need none
        live = min(c["A"], M * (1.0 - c["bare"])) if not c["runs"] else c["A"] * (1.0 - c["bare"])
        rows = M * (1.0 - c["bare"])
        ad = live * r * (K + N) * 2
        if c["op"] == "linear_fwd":
            return dict(bytes=w + ad + 2.0 * M * (K + N) + 4 * M, flops=2.0 * M * N * K + 2.0 * rows * r * (K + N))
        return dict(bytes=w + 2 * ad + 2.0 * M * (K + N + K) + 4 * M + (2.0 * M * r if c["keep"] else 0.0),
                    flops=2.0 * M * N * K + 2.0 * rows * r * (2 * (K + N) + (0 if c["keep"] else K)))
    if c["op"] == "preference":
        S, T, V, e = 2 * c["pairs"], c["T"], c["V"], 4 if c["f32"] else 2
        counted = sum(hi - lo for lo, hi in _spans(c))
        return dict(bytes=float(counted * V * e + S * T * V * e + S * T * (8 + 4 + 4)), flops=6.0 * counted * V)
    n = sum(_sizes(c))
    state = 16 if c["bits"] == 32 else 4 + 16 / STATE_BLOCK
    return dict(bytes=n * (8.0 + (4 if c["g32"] else 2) + 2 + state), flops=20.0 * n)


# ---- in 64 bits, from the definitions ---------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c = case
    D = torch.float64
    if c["op"].startswith("linear"):
        M, K, N, r, A = c["M"], c["K"], c["N"], c["r"], c["A"]
        low, high = s["codes"] % 16, torch.div(s["codes"], 16, rounding_mode="floor")
        q = s["book"][torch.stack((low, high), 1).flatten().int()]
        groups = torch.arange(s["absmax8"].numel(), device=q.device) // GROUP
        a = s["absmax8"].view(torch.float8_e4m3fn).to(D) * s["scale2"].to(D)[groups]
        a = a.to(torch.float32) + s["mean"]              # the format's own roundings: the constant is an fp32,
        W = (q.view(-1, BLOCK) * a.view(-1, 1)).bfloat16().to(D).view(N, K)   # the weight a bf16
        X, L1, L2, sc = s["X"].to(D), s["L1"].to(D), s["L2"].to(D), s["scale"].to(D)
        rows = [(s["ids"] == k).nonzero().flatten() for k in range(A)]
        if c["op"] == "linear_fwd":
            Y = X.matmul(W.T)
            for k, at in enumerate(rows):
                Y[at] += sc[k] * X[at].matmul(L1[k]).matmul(L2[k])
            return Y
        dY = s["dY"].to(D)
        dX = dY.matmul(W)
        dL1, dL2 = torch.zeros_like(L1), torch.zeros_like(L2)
        for k, at in enumerate(rows):
            U = sc[k] * dY[at].matmul(L2[k].T)
            dX[at] += U.matmul(L1[k].T)
            dL1[k] = X[at].T.matmul(U)
            T = s["T"][at].to(D) if s["T"] is not None else X[at].matmul(L1[k])
            dL2[k] = sc[k] * T.T.matmul(dY[at])
        return dX, dL1, dL2
    if c["op"] == "preference":
        S, T, V = s["logits"].shape
        P = S // 2
        lp = torch.zeros(S, T, dtype=D, device=s["logits"].device)
        for i, (lo, hi) in enumerate(_spans(c)):
            full = torch.log_softmax(s["logits"][i, lo:hi].to(D), dim=1)
            lp[i, lo:hi] = full[torch.arange(hi - lo, device=full.device), s["labels"][i, lo:hi]]
        on = s["labels"] != -100
        reward = s["beta"] * ((lp - s["ref"].to(D)) * on).sum(dim=1)
        h = reward[:P] - reward[P:]
        loss = -((1 - s["eps"]) * torch.nn.functional.logsigmoid(h) + s["eps"] * torch.nn.functional.logsigmoid(-h))
        slope = (-(1 - s["eps"]) * torch.sigmoid(-h) + s["eps"] * torch.sigmoid(h)) / P   # d mean loss / d h
        grad = torch.zeros(S, T, V, dtype=D if S * T * V < 2 ** 28 else torch.float32, device=lp.device)
        for i, (lo, hi) in enumerate(_spans(c)):
            g = -torch.softmax(s["logits"][i, lo:hi].to(D), dim=1)
            g[torch.arange(hi - lo, device=g.device), s["labels"][i, lo:hi]] += 1.0
            grad[i, lo:hi] = (s["beta"] * slope[i % P] * (1.0 if i < P else -1.0)) * g
        return loss.mean().reshape(1), reward, lp, grad
    b1, b2 = s["b"][:2]
    g = s["grad"].to(D)
    coef = min(1.0, s["max_norm"] / (math.sqrt(float((g * g).sum())) + 1e-6))
    g *= coef
    per = lambda v: torch.repeat_interleave(v.to(D), STATE_BLOCK)  # noqa: E731
    if c["bits"] == 8:
        m, v = s["m"].to(D) * per(s["m_scale"]), (s["v"].to(D) * per(s["v_scale"])) ** 2
    else:
        m, v = s["m"].to(D), s["v"].to(D)
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + g * g * (1.0 - b2)
    step = (m / (1.0 - b1 ** s["step"])) / ((v / (1.0 - b2 ** s["step"])).sqrt() + 1e-8)
    theta = s["theta"].to(D) * (1.0 - s["lr"] * s["wd"]) - s["lr"] * step
    out = [torch.tensor([coef], dtype=D), theta, theta]
    if c["bits"] == 32:
        return out + [m, v]
    held = []
    for x, least in ((m, 0.0), (v.sqrt(), 2.0 ** -9)):
        x = x.view(-1, STATE_BLOCK)
        top = x.abs().max(dim=1, keepdim=True).values
        x = x * torch.where(top > 0, 448.0 / top, 0.0)
        quantum = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
        near = torch.round(x / quantum) * quantum
        held.append((torch.where(x > 0, near.clamp_min(least), near).flatten(), top.flatten() / 448.0))
    return out + [held[0][0], held[1][0], held[0][1], held[1][1]]
