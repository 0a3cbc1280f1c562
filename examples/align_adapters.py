"""Preference or policy training of two adapters on one frozen attention block, from the library's operators alone.

    python examples/align_adapters.py                       # preference pairs
    python examples/align_adapters.py --loss policy         # sampled tokens with advantages

A packed batch (each sample starts on a 128-row tile, as the multi-adapter calls want it) goes through a frozen fused
Q/K/V projection and a frozen output projection, both with the adapters' branches, packed causal attention between
them, and a frozen head; then the loss with the gradient of its logits (in place), the backward of all of it, and one
AdamW step over every adapter matrix with 8-bit states.  Tokens and weights are random.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from lora_fine_tuning_gb300 import api  # noqa: E402

TILE = 128
Q_HEADS, KV_HEADS, HEAD_DIM, VOCAB, RANK, ALPHA, DROPOUT = 8, 2, 64, 4001, 16, 2.0, 0.05
HIDDEN = Q_HEADS * HEAD_DIM
QKV = (Q_HEADS + 2 * KV_HEADS) * HEAD_DIM
PROMPT = 20   # tokens of each sample that are given: the loss does not count them


class Block:
    """The frozen weights and the two adapters, one (A, B) for each of the two projections."""

    def __init__(self, n_adapters: int, gen: torch.Generator):
        def normal(rows, cols, size):
            return (torch.randn(rows, cols, device="cuda", generator=gen) * size).bfloat16()

        self.embed = normal(VOCAB, HIDDEN, 1.0)
        self.w_qkv, self.w_out = normal(HIDDEN, QKV, HIDDEN ** -0.5), normal(HIDDEN, HIDDEN, HIDDEN ** -0.5)
        self.head = normal(HIDDEN, VOCAB, HIDDEN ** -0.5)

        def adapters(n):
            return [api.Adapter(normal(HIDDEN, RANK, HIDDEN ** -0.5), torch.zeros(RANK, n, device="cuda").bfloat16(),
                                ALPHA, DROPOUT) for _ in range(n_adapters)]

        self.qkv, self.out = adapters(QKV), adapters(HIDDEN)
        for a in self.qkv + self.out:
            a.dA, a.dB = torch.empty_like(a.A), torch.empty_like(a.B)

    def parameters(self):
        for a in self.qkv + self.out:
            yield a.A, a.dA
            yield a.B, a.dB

    @staticmethod
    def heads(x):
        """Q, K and V as strided views of the fused projection's rows."""
        q, k, v = x.split([Q_HEADS * HEAD_DIM, KV_HEADS * HEAD_DIM, KV_HEADS * HEAD_DIM], dim=1)
        return (t.unflatten(1, (-1, HEAD_DIM)) for t in (q, k, v))

    def forward(self, tokens, segments, seqs, seed):
        x = self.embed[tokens]
        qkv, s_qkv, _ = api.multi_lora_fwd(x, self.w_qkv, self.qkv, segments, seed)
        o, lse = api.attn_fwd(*self.heads(qkv), seqs)
        y, s_out, _ = api.multi_lora_fwd(o.flatten(1), self.w_out, self.out, segments, seed + 1)
        return (x + y) @ self.head, (x, qkv, s_qkv, o, lse, s_out)

    def backward(self, dlogits, saved, segments, seqs, seed):
        x, qkv, s_qkv, o, lse, s_out = saved
        dy = dlogits @ self.head.T
        d_o = api.multi_lora_bwd(dy, o.flatten(1), self.w_out, self.out, segments, seed + 1, s_out)
        d_qkv = torch.empty_like(qkv)
        dq, dk, dv = self.heads(d_qkv)
        api.attn_bwd(d_o.view_as(o), *self.heads(qkv), o, lse, seqs, dQ=dq, dK=dk, dV=dv)
        api.multi_lora_bwd(d_qkv, x, self.w_qkv, self.qkv, segments, seed, s_qkv)


def batch(lengths, gen):
    """Samples on tiles of their own.  Returns (tokens, labels, [(first row, rows)], rows of the batch)."""
    places, row = [], 0
    for n in lengths:
        places.append((row, n))
        row += -(-n // TILE) * TILE
    tokens = torch.randint(0, VOCAB, (row,), device="cuda", generator=gen)
    labels = torch.full((row,), -1, dtype=torch.int64, device="cuda")
    for a, n in places:
        labels[a + PROMPT - 1:a + n - 1] = tokens[a + PROMPT:a + n]   # each row predicts the next token
    return tokens, labels, places, row


def train(loss="preference", steps=12, lr=2e-3, seed=0, verbose=False):
    """Returns the loss of each step."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    block = Block(2, gen)
    lengths = [190, 203, 77, 128, 140, 131, 300, 64]
    tokens, labels, places, rows = batch(lengths, gen)
    # samples 2i and 2i + 1 are a pair; the first half belongs to adapter 0, the second to adapter 1
    segments = [(a, -(-n // TILE) * TILE, 0 if i < len(lengths) // 2 else 1) for i, (a, n) in enumerate(places)]
    seqs = api.attn_seqs(places)
    pairs = api.pref_pairs([(c[0], r[0], c[1], r[1]) for c, r in zip(places[::2], places[1::2])])
    counted = labels >= 0
    advantages = torch.zeros(rows, device="cuda")
    for i, (a, n) in enumerate(places):
        advantages[a:a + n] = 1.0 if i % 2 == 0 else -1.0
    states = [api.adamw_tensor(p, g, bits=8, master=True) for p, g in block.parameters()]
    optimiser = api.adamw_tensors(states)

    # the adapters' B are zero: this is the frozen model, the reference of both losses
    zeros = torch.zeros(rows, device="cuda")
    logits, _ = block.forward(tokens, segments, seqs, seed)
    ref = api.policy_loss(logits, labels, zeros, advantages, want_grad=False)[1]
    old, losses = ref, []
    for step in range(1, steps + 1):
        logits, saved = block.forward(tokens, segments, seqs, 2 * step)
        if loss == "preference":
            value, logp, margins, dlogits = api.pref_loss(logits, labels, pairs, ref, beta=0.1, scale=1 / len(pairs),
                                                          dlogits=logits)
        else:
            value, logp, dlogits = api.policy_loss(logits, labels, old, advantages, ref, kl_coef=0.02,
                                                   scale=1 / int(counted.sum()), dlogits=logits)
            old = logp
        block.backward(dlogits, saved, segments, seqs, 2 * step)
        api.adamw_step(optimiser, lr=lr, weight_decay=0.01, step=step)
        losses.append(float(value))
        if verbose:
            shift = torch.where(advantages > 0, logp - ref, ref - logp)[counted].mean()
            print(f"step {step:3d}  loss {losses[-1]:+.4f}  preferred over the frozen model by {float(shift):+.4f} a token")
    assert all(math.isfinite(x) for x in losses)
    shift = torch.where(advantages > 0, logp - ref, ref - logp)[counted].mean()
    return losses, float(shift)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--loss", choices=("preference", "policy"), default="preference")
    ap.add_argument("--steps", type=int, default=12)
    ap.add_argument("--lr", type=float, default=2e-3)
    args = ap.parse_args()
    train(args.loss, args.steps, args.lr, verbose=True)
