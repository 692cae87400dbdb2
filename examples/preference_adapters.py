"""Several adapters trained from preference pairs over one quantised base, then served together.

A frozen two-layer network (NF4 weights, random) gets one adapter per user.
User a prefers sequences of the tokens t = a (mod users); the rejected
sequence of a pair has tokens of the whole vocabulary. Every step is one batch
of all users' pairs and of the reference (the same rows with adapter id -1):

    linear forward (adapter or none per row) -> preference loss and the logits'
    gradient -> linear backward -> clipped AdamW step with 8-bit state

after which one batched decode loop serves a request of every user.

    python examples/preference_adapters.py --steps 60
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_nf4_quantized_amd import api  # noqa: E402


class Linear:
    """A frozen NF4 weight with one adapter per user: float32 masters and the bf16 copies that are computed with."""

    def __init__(self, out_features, in_features, users, rank, gen):
        W = torch.randn(out_features, in_features, generator=gen, device="cuda") / in_features**0.5
        self.base = api.qlora_quantize(W)
        L1 = torch.randn(users, in_features, rank, generator=gen, device="cuda") / in_features**0.5
        self.master = [L1, torch.zeros(users, rank, out_features, device="cuda")]
        self.half = [t.bfloat16() for t in self.master]
        self.scale = torch.full((users,), 2.0, device="cuda")

    def forward(self, X, user, want_T=False):
        return api.qlora_linear_multi_fwd(self.base, X, user, *self.half, self.scale, want_T=want_T)

    def backward(self, X, dY, user, T, need_dX):
        return api.qlora_linear_multi_bwd(self.base, X, dY, user, *self.half, self.scale, T=T, need_dX=need_dX,
                                          grad_dtype=torch.float32)


class Network:
    def __init__(self, users, vocab=1000, width=512, hidden=1408, rank=8, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.embed = torch.randn(vocab, width, generator=gen, device="cuda").bfloat16()
        self.up = Linear(hidden, width, users, rank, gen)
        self.head = Linear(vocab, hidden, users, rank, gen)
        self.vocab, self.users = vocab, users
        self.masters = self.up.master + self.head.master
        self.halves = self.up.half + self.head.half
        self.state = api.AdamWState.zeros(self.masters, bits=8)
        self.steps = 0

    def logits(self, tokens, user):
        H, _ = self.up.forward(self.embed[tokens], user)
        return self.head.forward(H.relu_(), user)[0]

    def train_step(self, tokens, labels, user, beta=0.2, lr=5e-3):
        """tokens, labels [2 pairs, T] (preferred sequences first), user [2 pairs]: the loss of the step."""
        S, T = tokens.shape
        own = user.repeat_interleave(T)
        both = torch.cat([own, torch.full_like(own, -1)])
        X = self.embed[tokens.flatten().repeat(2)]
        H, T1 = self.up.forward(X, both, want_T=True)
        H.relu_()
        Z, T2 = self.head.forward(H, both, want_T=True)
        n = S * T
        policy, reference = Z[:n].view(S, T, -1), Z[n:].view(S, T, -1)
        none = torch.zeros(S, T, device="cuda")
        ref = api.qlora_preference_loss(reference, labels, none, beta, need_grad=False).logps
        out = api.qlora_preference_loss(policy, labels, ref, beta)
        dZ = out.dlogits.view(n, -1)
        dH, *g2 = self.head.backward(H[:n], dZ, own, T2[:n], need_dX=True)
        _, *g1 = self.up.backward(X[:n], dH.mul_(H[:n] > 0), own, T1[:n], need_dX=False)
        grads = g1 + g2
        self.steps += 1
        coef, _ = api.qlora_clip_grad_norm_batch(grads, 1.0)
        api.qlora_adamw_batch(self.masters, grads, self.state, self.steps, lr, coef=coef, thetas_bf16=self.halves)
        return out.loss

    def decode(self, tokens, user, steps):
        """Greedy continuation of one token per request: [requests, steps]."""
        out = []
        for _ in range(steps):
            tokens = self.logits(tokens, user).argmax(1)
            out.append(tokens)
        return torch.stack(out, 1)


def draw_pairs(net, pairs, length, gen):
    """Preference pairs of random users: tokens, labels [2 pairs, length], user [2 pairs]."""
    user = torch.randint(0, net.users, (pairs,), generator=gen, device="cuda", dtype=torch.int32)
    own = torch.randint(0, net.vocab // net.users, (pairs, length + 1), generator=gen, device="cuda") * net.users
    own += user[:, None]
    any_ = torch.randint(0, net.vocab, (pairs, length + 1), generator=gen, device="cuda")
    any_[:, 0] = own[:, 0]                                          # the pair's common prompt
    seq = torch.cat([own, any_])
    labels = seq[:, 1:].clone()
    cut = torch.randint(length // 2, length + 1, (2 * pairs, 1), generator=gen, device="cuda")
    labels[torch.arange(length, device="cuda") >= cut] = -100       # sequences end at different places
    return seq[:, :-1].contiguous(), labels, user.repeat(2)


def run(steps=60, users=6, pairs=16, length=24, seed=0, say=print):
    """Trains, then decodes: (losses per step, share of decoded tokens that each user prefers)."""
    net = Network(users, seed=seed)
    gen = torch.Generator("cuda").manual_seed(seed + 1)
    losses = []
    for k in range(steps):
        losses.append(net.train_step(*draw_pairs(net, pairs, length, gen)))
        if k % 10 == 0 or k + 1 == steps:
            say(f"step {k:3d}  loss {losses[-1].item():.4f}")
    user = torch.arange(users, dtype=torch.int32, device="cuda")
    start = torch.randint(0, net.vocab, (users,), generator=gen, device="cuda")
    text = net.decode(start, user, 32)
    alone = torch.cat([net.decode(start[a:a + 1], user[a:a + 1], 32) for a in range(users)])   # a request at a time
    share = (text % users == user[:, None]).float().mean(1)
    solo = (alone % users == user[:, None]).float().mean(1)
    base = (net.decode(start, torch.full_like(user, -1), 32) % users == user[:, None]).float().mean(1)
    for a in range(users):
        say(f"user {a}: preferred tokens {share[a]:.2f} decoded in a batch, {solo[a]:.2f} alone, {base[a]:.2f} without an adapter")
    return [x.item() for x in losses], share.tolist(), solo.tolist()


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--users", type=int, default=6)
    p.add_argument("--pairs", type=int, default=16)
    p.add_argument("--length", type=int, default=24)
    p.add_argument("--seed", type=int, default=0)
    run(**vars(p.parse_args()))


if __name__ == "__main__":
    main()
