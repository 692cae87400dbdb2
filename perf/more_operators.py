"""The rest of a layer's step beside its quantised linears, as a user runs it.

The gated feed-forward block over two NF4 bases with adapters, forward and
backward; activations kept in 8 bits and read by the backward passes; the norm
with the residual's addition; the loss over the vocabulary from hidden states,
without logits. ``own`` selects the library's entry points or the plain form of
elementary torch operations.
"""

import math
import random
import statistics

import torch

own = False

BLOCK, GROUP = 64, 256      # weights (and 8-bit activations) per absmax constant, constants per second-level scale
EPS = 1e-6                  # of the norm


def listed():
    return [
        # one token of a decode step: the latency of the block
        dict(name="gated-token", op="gated_fwd", M=1, K=4096, F=11008, r=64, act="silu", save=False),
        # a batched decode step of 96 requests
        dict(name="gated-batch", op="gated_fwd", M=96, K=4096, F=11008, r=16, act="silu", save=False),
        # training: 2048 tokens, gate and up kept in 8 bits for the backward pass
        dict(name="gated-train", op="gated_fwd", M=2048, K=4096, F=11008, r=64, act="silu", save=True),
        # a short ragged batch whose forward pass kept nothing: gate and up are computed again
        dict(name="gated-bwd-short", op="gated_bwd", M=391, K=4096, F=11008, r=32, act="gelu", save=False, keep=False, x8=False),
        # training: 8192 tokens, gate, up and the block's input kept in 8 bits
        dict(name="gated-bwd", op="gated_bwd", M=8192, K=4096, F=11008, r=64, act="silu", save=True, keep=True, x8=True),
        # a short batch of a square projection whose input was kept in 8 bits
        dict(name="linear-bwd-int8-short", op="linear_bwd", M=200, K=4096, N=4096, r=16, keep=False),
        # 8192 tokens of the widest linear, input in 8 bits
        dict(name="linear-bwd-int8", op="linear_bwd", M=8192, K=4096, N=11008, r=64, keep=True),
        # the norm before a projection on a float32 residual stream, with the projection's input in 8 bits
        dict(name="norm-train", op="norm_fwd", M=8192, K=4096, f32=True, res=True, save=True),
        # its backward pass for a ragged batch on a bf16 stream, with the weight's gradient
        dict(name="norm-bwd", op="norm_bwd", M=1001, K=6656, f32=False, res=True),
        # the loss of 48 tokens (a short answer after a long prompt): latency and one pass over the head
        dict(name="head-short", op="head", M=48, K=4096, V=32000, bare=0.0, weighted=False, dW=False),
        # a vocabulary with one token added, tokens with weights, and the head trained too
        dict(name="head-odd", op="head", M=777, K=4096, V=32001, bare=0.1, weighted=True, dW=True),
        # 8192 tokens, a quarter of them prompts that do not count
        dict(name="head-train", op="head", M=8192, K=4096, V=32000, bare=0.25, weighted=False, dW=False),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


MOST = 4.0 * 8192 * 4096 * 32000     # flops of the largest listed case


def draw(rng):
    op = rng.choice(("gated_fwd", "gated_fwd", "gated_bwd", "linear_bwd", "norm_fwd", "norm_bwd", "head", "head"))
    if op in ("gated_fwd", "gated_bwd"):
        K = 64 * round(_log(rng, 16, 104))
        F = 8 * round(_log(rng, 128, 2240))
        M = round(_log(rng, 1, 8192))
        act = rng.choice(("silu", "silu", "gelu"))
        save = rng.random() < 0.5
        if save:
            F = max(64, F // 64 * 64)
        c = dict(op=op, M=M, K=K, F=F, r=8 * round(_log(rng, 1, 16)), act=act, save=save)
        if op == "gated_bwd":
            c.update(M=max(24, M), keep=rng.random() < 0.5, x8=rng.random() < 0.5)
    elif op == "linear_bwd":
        c = dict(op=op, M=round(_log(rng, 24, 8192)), K=64 * round(_log(rng, 16, 104)), N=8 * round(_log(rng, 128, 2240)),
                 r=8 * round(_log(rng, 1, 16)), keep=rng.random() < 0.5)
    elif op == "head":
        c = dict(op=op, M=round(_log(rng, 1, 8192)), K=64 * round(_log(rng, 8, 104)), V=round(_log(rng, 1000, 131072)),
                 bare=rng.choice((0.0, 0.1, 0.6)), weighted=rng.random() < 0.4, dW=rng.random() < 0.3)
    else:
        c = dict(op=op, M=round(_log(rng, 1, 8192)), K=8 * round(_log(rng, 64, 1024)), f32=rng.random() < 0.5, res=rng.random() < 0.7)
        if op == "norm_fwd":
            c["save"] = rng.random() < 0.5
            if c["save"]:
                c["K"] = c["K"] // 64 * 64
    if work(c)["flops"] > MOST:
        c["M"] = max(1, int(c["M"] * MOST / work(c)["flops"]))
    return c


# ---- what the cases are made of -------------------------------------------------------

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

    def base(N, K):
        nb = -(-N * K // BLOCK)
        return dict(rows=N, cols=K,
                    codes=torch.randint(0, 256, (-(-N * K // 2),), generator=g, device=dev, dtype=torch.uint8),
                    absmax8=(normal(nb, dtype=torch.float32).clamp(-3.9, 3.9) * 112.0).to(torch.float8_e4m3fn).view(torch.uint8),
                    scale2=7e-5 * (1.0 + 0.1 * torch.rand(-(-nb // GROUP), generator=g, device=dev)),
                    mean=torch.full((1,), 0.048, device=dev))

    s = dict(case=dict(c), book=torch.tensor(_codebook(), dtype=torch.float32, device=dev))
    if c["op"].startswith("gated"):
        M, K, F, r = c["M"], c["K"], c["F"], c["r"]
        s["gate"], s["up"] = base(F, K), base(F, K)
        s["L1"], s["L2"] = normal(2, K, r, std=K ** -0.5), normal(2, r, F, std=0.05)
        s["scale"] = rng.choice((0.25, 1.0, 2.0))
        s["X"] = normal(M, K)
        if c["op"] == "gated_bwd":
            s["dA"] = normal(M, F, std=0.1)
            s["X8"] = s["G8"] = s["U8"] = s["T"] = None
            if c["x8"]:
                s["X8"] = _encode(s["X"].float())
                s["X"] = None
            x = s["X"].float() if s["X"] is not None else _decode(s["X8"]).reshape(M, K)
            if c["save"]:
                s["G8"], s["U8"] = (_encode(v) for v in _gate_up(s, x))
            if c["keep"]:
                s["T"] = torch.stack((x @ s["L1"][0].float(), x @ s["L1"][1].float())).to(torch.bfloat16)
    elif c["op"] == "linear_bwd":
        M, K, N, r = c["M"], c["K"], c["N"], c["r"]
        s["base"] = base(N, K)
        s["L1"], s["L2"] = normal(K, r, std=K ** -0.5), normal(r, N, std=0.05)
        s["scale"] = rng.choice((0.25, 1.0, 2.0))
        s["X8"] = _encode(normal(M, K, dtype=torch.float32))
        s["dY"] = normal(M, N, std=0.1)
        s["T"] = (_decode(s["X8"]).reshape(M, K) @ s["L1"].float()).to(torch.bfloat16) if c["keep"] else None
    elif c["op"].startswith("norm"):
        M, K = c["M"], c["K"]
        stream = torch.float32 if c["f32"] else torch.bfloat16
        # a residual stream grows with depth, with a few channels far above the others
        channels = torch.empty(K, device=dev).log_normal_(0.0, 0.6, generator=g)
        h = normal(M, K, std=3.0, dtype=torch.float32) * channels
        s["w"] = (1.0 + normal(K, std=0.2, dtype=torch.float32)).to(torch.bfloat16)
        if c["op"] == "norm_fwd":
            s["x"] = normal(M, K) if c["res"] else h.to(stream)
            s["res"] = h.to(stream) if c["res"] else None
        else:
            s["h"] = h.to(stream)
            s["rstd"] = torch.rsqrt((s["h"].float() ** 2).mean(1) + EPS)
            s["dy"] = normal(M, K, std=0.02)
            s["dres"] = normal(M, K, std=0.02, dtype=torch.float32).to(stream) if c["res"] else None
    else:
        M, K, V = c["M"], c["K"], c["V"]
        s["W"] = normal(V, K, std=2.0 * K ** -0.5)
        labels = torch.randint(0, V, (M,), generator=g, device=dev)
        # the model puts weight on its labels, on some more than on others
        lift = 2.5 * torch.rand(M, 1, generator=g, device=dev)
        s["H"] = (normal(M, K, dtype=torch.float32) + lift * s["W"][labels].float()).to(torch.bfloat16)
        bare = torch.rand(M, generator=g, device=dev) < c["bare"]
        s["labels"] = torch.where(bare, -100, labels)
        s["weights"] = (0.1 + torch.rand(M, generator=g, device=dev)) if c["weighted"] else None
    return s


# ---- plain forms --------------------------------------------------------------------------

def _weight(s, q):
    """The dequantised weight [rows][cols] in bf16's values: bf16(q[code] * (e4m3(c8) * scale2 + mean))."""
    codes = torch.stack((q["codes"] & 15, q["codes"] >> 4), 1).reshape(-1, BLOCK).long()
    sc = q["scale2"].repeat_interleave(GROUP)[:q["absmax8"].numel()]
    a = q["absmax8"].view(torch.float8_e4m3fn).float() * sc + q["mean"]
    return (s["book"][codes] * a[:, None]).to(torch.bfloat16).float().reshape(q["rows"], q["cols"])


def _encode(x):
    """int8 codes and absmax of blocks of 64: round(x * (127 / absmax))."""
    b = x.reshape(-1, BLOCK)
    top = b.abs().amax(1)
    inv = torch.where(top > 0, 127.0 / torch.where(top > 0, top, 1.0), 0.0)
    return torch.round(b * inv[:, None]).to(torch.int8).reshape(-1), top


def _decode(coded):
    codes, top = coded
    return (codes.float().reshape(-1, BLOCK) * (top / 127.0)[:, None]).reshape(-1)


def _gate_up(s, x):
    def one(q, L1, L2):
        return x @ _weight(s, q).t() + s["scale"] * ((x @ L1.float()) @ L2.float())

    return one(s["gate"], s["L1"][0], s["L2"][0]), one(s["up"], s["L1"][1], s["L2"][1])


def _act(g, kind):
    """act(g) and act'(g): g sigma(z), z = g for silu, sqrt(8 / pi) (g + 0.044715 g^3) for gelu's tanh form."""
    if kind == "silu":
        z, dz = g, 1.0
    else:
        a = math.sqrt(8.0 / math.pi)
        z, dz = a * (g + 0.044715 * g ** 3), a * (1.0 + 3.0 * 0.044715 * g * g)
    p = 1.0 / (1.0 + torch.exp(-z))
    return g * p, p + g * p * (1.0 - p) * dz


def _gated_fwd(s):
    c = s["case"]
    G, U = _gate_up(s, s["X"].float())
    A = (_act(G, c["act"])[0] * U).to(torch.bfloat16)
    if not c["save"]:
        return A
    return A, _decode(_encode(G)).to(torch.bfloat16), _decode(_encode(U)).to(torch.bfloat16)


def _gated_bwd(s):
    c = s["case"]
    M, K, F = c["M"], c["K"], c["F"]
    X = s["X"].float() if s["X"] is not None else _decode(s["X8"]).reshape(M, K)
    G, U = (_decode(s["G8"]).reshape(M, F), _decode(s["U8"]).reshape(M, F)) if c["save"] else _gate_up(s, X)
    dA = s["dA"].float()
    a, d = _act(G, c["act"])
    dX, dL1, dL2 = 0.0, [], []
    for k, (q, dY) in enumerate(((s["gate"], dA * U * d), (s["up"], dA * a))):
        L1, L2 = s["L1"][k].float(), s["L2"][k].float()
        T = s["T"][k].float() if s["T"] is not None else X @ L1
        V = s["scale"] * (dY @ L2.t())
        dX = dX + dY @ _weight(s, q) + V @ L1.t()
        dL1.append(X.t() @ V)
        dL2.append(s["scale"] * (T.t() @ dY))
    return dX.to(torch.bfloat16), torch.stack(dL1).to(torch.bfloat16), torch.stack(dL2).to(torch.bfloat16)


def _linear_bwd(s):
    c = s["case"]
    X, dY, L1, L2 = _decode(s["X8"]).reshape(c["M"], c["K"]), s["dY"].float(), s["L1"].float(), s["L2"].float()
    T = s["T"].float() if s["T"] is not None else X @ L1
    V = s["scale"] * (dY @ L2.t())
    dX = dY @ _weight(s, s["base"]) + V @ L1.t()
    return dX.to(torch.bfloat16), (X.t() @ V).to(torch.bfloat16), (s["scale"] * (T.t() @ dY)).to(torch.bfloat16)


def _norm_fwd(s):
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    rstd = torch.rsqrt((h * h).mean(1) + EPS)
    y = h * rstd[:, None] * s["w"].float()
    out = [y.to(torch.bfloat16), rstd]
    if s["res"] is not None:
        out.append(h.to(s["res"].dtype))
    if s["case"]["save"]:
        out.append(_decode(_encode(y)).to(torch.bfloat16))
    return out


def _norm_bwd(s):
    h, dy = s["h"].float(), s["dy"].float()
    xh = h * s["rstd"][:, None]
    wd = dy * s["w"].float()
    dh = s["rstd"][:, None] * (wd - xh * (wd * xh).mean(1, keepdim=True))
    if s["dres"] is not None:
        dh = dh + s["dres"].float()
    return dh.to(s["h"].dtype), (dy * xh).sum(0)


def _head(s):
    c = s["case"]
    H, W, y = s["H"].float(), s["W"].float(), s["labels"]
    on = (y >= 0) & (y < c["V"])
    at = torch.where(on, y, 0)[:, None]
    S = H @ W.t()
    top = S.amax(1, keepdim=True)
    e = torch.exp(S - top)
    total = e.sum(1, keepdim=True)
    nll = torch.where(on, (torch.log(total) + top - S.gather(1, at))[:, 0], 0.0)
    w = torch.where(on, s["weights"] if s["weights"] is not None else 1.0, 0.0) / on.sum().clamp(min=1)
    loss = (w * nll).sum().reshape(1)
    G = e.mul_((w[:, None] / total))
    G.scatter_add_(1, at, -w[:, None])
    out = [loss, nll, (G @ W).to(torch.bfloat16)]
    return out + [(G.t() @ H).to(torch.bfloat16)] if c["dW"] else out


# ---- one pass -------------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return dict(gated_fwd=_gated_fwd, gated_bwd=_gated_bwd, linear_bwd=_linear_bwd, norm_fwd=_norm_fwd,
                    norm_bwd=_norm_bwd, head=_head)[op](s)

    from bit_nf4_quantized_amd import api

    def base(q):
        return api.NF4Tensor(q["rows"], q["cols"], q["codes"], q["absmax8"], q["scale2"], q["mean"])

    def values(coded, *shape):
        return api.qlora_int8_dequantize(*coded, dtype=torch.bfloat16).view(*shape)

    if op == "gated_fwd":
        o = api.qlora_gated_fwd(base(s["gate"]), base(s["up"]), s["X"], s["L1"], s["L2"], s["scale"], act=c["act"],
                                want_int8=c["save"])
        return (o.A, values(o.gate8, -1), values(o.up8, -1)) if c["save"] else o.A
    if op == "gated_bwd":
        return api.qlora_gated_bwd(base(s["gate"]), base(s["up"]), s["X"] if s["X"] is not None else s["X8"], s["dA"],
                                   s["L1"], s["L2"], s["scale"], act=c["act"], T=s["T"], gate8=s["G8"], up8=s["U8"],
                                   grad_dtype=torch.bfloat16)
    if op == "linear_bwd":
        return api.qlora_linear_bwd_int8(base(s["base"]), s["X8"], s["dY"], s["L1"], s["L2"], s["scale"], T=s["T"],
                                         grad_dtype=torch.bfloat16)
    if op == "norm_fwd":
        o = api.qlora_norm_fwd(s["x"], s["w"], eps=EPS, residual=s["res"], want_int8=c["save"])
        out = [o.y, o.rstd]
        if s["res"] is not None:
            out.append(o.h)
        return out + [values(o.int8, -1)] if c["save"] else out
    if op == "norm_bwd":
        o = api.qlora_norm_bwd(s["dy"], s["h"], s["rstd"], s["w"], dres=s["dres"])
        return o.dh, o.dweight
    o = api.qlora_head_loss(s["H"], s["W"], s["labels"], weights=s["weights"], need_dW=c["dW"], grad_dtype=torch.bfloat16)
    return [o.loss, o.nll, o.dH] + ([o.dW] if c["dW"] else [])


def work(case):
    """Bytes: each input once, each output once. Flops: the products (the norm: some 10 per value)."""
    c = case
    base = lambda N, K: N * K / 2 + N * K / BLOCK + 4 * N * K / (BLOCK * GROUP)  # noqa: E731
    coded = 1.0 + 4.0 / BLOCK
    if c["op"].startswith("gated"):
        M, K, F, r = c["M"], c["K"], c["F"], c["r"]
        ad = 4.0 * r * (K + F)
        if c["op"] == "gated_fwd":
            return dict(bytes=2 * base(F, K) + ad + 2.0 * M * (K + F) + (2 * coded * M * F if c["save"] else 0.0),
                        flops=4.0 * M * K * F + 4.0 * M * r * (K + F))
        return dict(bytes=2 * base(F, K) + 2 * ad + (coded if c["x8"] else 2.0) * M * K + 2.0 * M * (F + K)
                    + (2 * coded * M * F if c["save"] else 0.0) + (4.0 * M * r if c["keep"] else 0.0),
                    flops=(4.0 if c["save"] else 8.0) * M * K * F + 4.0 * M * r * (2 * (K + F) + (0 if c["keep"] else K)
                                                                                + (0 if c["save"] else F)))
    if c["op"] == "linear_bwd":
        M, K, N, r = c["M"], c["K"], c["N"], c["r"]
        return dict(bytes=base(N, K) + 4.0 * r * (K + N) + coded * M * K + 2.0 * M * (N + K) + (2.0 * M * r if c["keep"] else 0.0),
                    flops=2.0 * M * N * K + 2.0 * M * r * (2 * (K + N) + (0 if c["keep"] else K)))
    if c["op"].startswith("norm"):
        n, e = float(c["M"]) * c["K"], 4 if c["f32"] else 2
        if c["op"] == "norm_fwd":
            return dict(bytes=n * ((2 + 2 * e if c["res"] else e) + 2 + (coded if c["save"] else 0)) + 4.0 * c["M"], flops=10.0 * n)
        return dict(bytes=n * (2 + 2 * e + (e if c["res"] else 0)) + 4.0 * c["M"] + 6.0 * c["K"], flops=10.0 * n)
    M, K, V = c["M"], c["K"], c["V"]
    rows = M * (1.0 - c["bare"])
    return dict(bytes=2.0 * V * K * (2 if c["dW"] else 1) + 2.0 * K * (rows + M) + 12.0 * M,
                flops=(6.0 if c["dW"] else 4.0) * rows * V * K)


# ---- in 64 bits, from the definitions ---------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c = case
    D = torch.float64

    def matrix(q):
        low, high = q["codes"] % 16, torch.div(q["codes"], 16, rounding_mode="floor")
        v = s["book"][torch.stack((low, high), 1).flatten().int()]
        groups = torch.arange(q["absmax8"].numel(), device=v.device) // GROUP
        a = q["absmax8"].view(torch.float8_e4m3fn).to(D) * q["scale2"].to(D)[groups]
        a = a.to(torch.float32) + q["mean"]              # the format's own roundings: the constant is an fp32,
        return (v.view(-1, BLOCK) * a.view(-1, 1)).bfloat16().to(D).view(q["rows"], q["cols"])   # the weight a bf16

    def held(x):
        """The values that 8 bits hold of x."""
        x = x.reshape(-1, BLOCK)
        top = x.abs().max(dim=1, keepdim=True).values
        step = torch.where(top > 0, top, 1.0) / 127.0
        return (torch.round(x / step) * step).flatten()

    def values(coded):
        return (coded[0].to(D).view(-1, BLOCK) * (coded[1].to(D) / 127.0).view(-1, 1)).flatten()

    def sigmoid_part(g):
        if c["act"] == "silu":
            return torch.sigmoid(g), torch.ones_like(g)
        k = math.sqrt(2.0 / math.pi)
        return 0.5 * (1.0 + torch.tanh(k * (g + 0.044715 * g.pow(3)))), 2.0 * k * (1.0 + 0.134145 * g.pow(2))

    if c["op"].startswith("gated"):
        M, K, F = c["M"], c["K"], c["F"]
        Wg, Wu = matrix(s["gate"]), matrix(s["up"])
        L1, L2, sc = s["L1"].to(D), s["L2"].to(D), s["scale"]
        X = s["X"].to(D) if s["X"] is not None else values(s["X8"]).view(M, K)
        if c["op"] == "gated_bwd" and c["save"]:
            G, U = values(s["G8"]).view(M, F), values(s["U8"]).view(M, F)
        else:
            G = X.matmul(Wg.T + sc * L1[0].matmul(L2[0]))
            U = X.matmul(Wu.T + sc * L1[1].matmul(L2[1]))
        p, dz = sigmoid_part(G)
        if c["op"] == "gated_fwd":
            return (G * p * U, held(G), held(U)) if c["save"] else G * p * U
        dA = s["dA"].to(D)
        dU = dA * (G * p)
        dG = dA * U * (p * (1.0 + G * (1.0 - p) * dz))
        dX = dG.matmul(Wg) + dU.matmul(Wu)
        d1, d2 = torch.empty_like(L1), torch.empty_like(L2)
        for k, dY in enumerate((dG, dU)):
            V = sc * dY.matmul(L2[k].T)
            dX += V.matmul(L1[k].T)
            d1[k] = X.T.matmul(V)
            T = s["T"][k].to(D) if s["T"] is not None else X.matmul(L1[k])
            d2[k] = sc * T.T.matmul(dY)
        return dX, d1, d2
    if c["op"] == "linear_bwd":
        X, dY, L1, L2, sc = values(s["X8"]).view(c["M"], c["K"]), s["dY"].to(D), s["L1"].to(D), s["L2"].to(D), s["scale"]
        V = sc * dY.matmul(L2.T)
        T = s["T"].to(D) if s["T"] is not None else X.matmul(L1)
        return dY.matmul(matrix(s["base"])) + V.matmul(L1.T), X.T.matmul(V), sc * T.T.matmul(dY)
    if c["op"] == "norm_fwd":
        h = s["x"].to(D) + (s["res"].to(D) if s["res"] is not None else 0.0)
        r = 1.0 / torch.sqrt(h.square().sum(dim=1) / c["K"] + EPS)
        y = s["w"].to(D) * (h * r.view(-1, 1))
        out = [y, r] + ([h] if s["res"] is not None else [])
        return out + [held(y)] if c["save"] else out
    if c["op"] == "norm_bwd":
        h, dy, w, r = s["h"].to(D), s["dy"].to(D), s["w"].to(D), s["rstd"].to(D).view(-1, 1)
        inner = (dy * w * h).sum(dim=1, keepdim=True) / c["K"]
        dh = r * dy * w - r.pow(3) * h * inner
        if s["dres"] is not None:
            dh = dh + s["dres"].to(D)
        return dh, (dy * h * r).sum(dim=0)
    H, W, y = s["H"].to(D), s["W"].to(D), s["labels"]
    rows = (y != -100).nonzero().flatten()
    logp = torch.log_softmax(H[rows].matmul(W.T), dim=1)
    nll = torch.zeros(c["M"], dtype=D, device=H.device)
    nll[rows] = -logp[torch.arange(rows.numel(), device=H.device), y[rows]]
    w = (s["weights"].to(D)[rows] if s["weights"] is not None else torch.ones_like(rows, dtype=D)) / max(1, rows.numel())
    G = logp.exp_()
    G[torch.arange(rows.numel(), device=H.device), y[rows]] -= 1.0
    G *= w.view(-1, 1)
    dH = torch.zeros_like(H)
    dH[rows] = G.matmul(W)
    out = [(w * nll[rows]).sum().reshape(1), nll, dH]
    return out + [G.T.matmul(H[rows])] if c["dW"] else out
