"""Adapters on a small decoder, from the library's operators alone: trained with the inputs of norms and Q/K/V projections kept in 8 bits, then
generating into a cache of pages.

    python examples/decoder_layers.py                 # these inputs kept in 8 bits; Q, K, V and the attention's output in bf16
    python examples/decoder_layers.py --keep bf16     # all of them in bf16

Each layer: the stream's norm, a frozen fused Q/K/V projection with an adapter, rotary positions in place, causal attention over the packed
samples, a frozen output projection with an adapter, whose output joins the stream normed, gated and scaled, in one call with the
next layer's norm.  Tokens and weights are random.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from lora_fine_tuning_gb300 import api  # noqa: E402

LAYERS, Q_HEADS, KV_HEADS, HEAD_DIM, VOCAB, RANK, ALPHA = 2, 8, 2, 64, 2001, 16, 2.0
WIDTH, PAGE = Q_HEADS * HEAD_DIM, 16
QKV = (Q_HEADS + 2 * KV_HEADS) * HEAD_DIM
RES_SCALE, EPS = 0.7, 1e-5


class Layer:
    def __init__(self, normal):
        self.norm, self.post, self.gate = (normal(WIDTH, size=0.1, mean=1.0) for _ in range(3))
        self.qkv, self.out = normal(WIDTH, QKV, size=WIDTH ** -0.5), normal(WIDTH, WIDTH, size=WIDTH ** -0.5)
        self.adapters = [(normal(WIDTH, RANK, size=WIDTH ** -0.5), normal(RANK, n, size=0.02)) for n in (QKV, WIDTH)]
        self.grads = None

    def block(self):
        """What joins a layer's output to the stream."""
        return dict(post_w=self.post, gate=self.gate, res_scale=RES_SCALE, eps=EPS)


class Decoder:
    def __init__(self, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, size, mean=0.0):
            return (torch.randn(*shape, device="cuda", generator=gen) * size + mean).bfloat16()

        self.embed, self.head = normal(VOCAB, WIDTH, size=1.0), normal(WIDTH, VOCAB, size=WIDTH ** -0.5)
        self.layers = [Layer(normal) for _ in range(LAYERS)]
        self.last = normal(WIDTH, size=0.1, mean=1.0)
        self.rope = api.rope_table(HEAD_DIM, 10000.0)

    @staticmethod
    def heads(qkv):
        q, k, v = qkv.split([Q_HEADS * HEAD_DIM, KV_HEADS * HEAD_DIM, KV_HEADS * HEAD_DIM], dim=1)
        return tuple(t.unflatten(1, (-1, HEAD_DIM)) for t in (q, k, v))

    def norm_of(self, i):
        return self.layers[i].norm if i < LAYERS else self.last

    def forward(self, tokens, positions, seqs, seed, dropout, keep):
        """Logits, and what the backward needs: of each layer its input x, the stream h that x is the norm of, and its output y (in 8 bits with
        keep="8 bits"), and as they are Q, K, V, O (the output projection's input), the attention's statistics and the adapters' S."""
        rows, eight = len(tokens), keep == "8 bits"

        def room():
            return api.act8(rows, WIDTH) if eight else None

        h, saved = self.embed[tokens], []
        x8, h8 = room(), room()
        x, h = api.norm_fwd(h, self.norm_of(0), eps=EPS, x8=x8, h8=h8)
        for i, layer in enumerate(self.layers):
            (a1, b1), (a2, b2) = layer.adapters
            qkv, s1, _ = api.lora_fwd(x, layer.qkv, a1, b1, ALPHA, dropout, seed + 2 * i)
            q, k, v = self.heads(qkv)
            api.rope_fwd(q, k, positions, self.rope, Q_out=q, K_out=k)
            o, lse = api.attn_fwd(q, k, v, seqs)
            y, s2, _ = api.lora_fwd(o.flatten(1), layer.out, a2, b2, ALPHA, dropout, seed + 2 * i + 1)
            kept = dict(x=x8 if eight else x, h=h8 if eight else h, qkv=qkv, s1=s1, o=o, lse=lse, s2=s2)
            x8, h8, y8 = room(), room(), room()
            x, h = api.norm_fwd(h, self.norm_of(i + 1), y=y, x8=x8, h8=h8, y8=y8, **layer.block())
            saved.append(dict(kept, y=y8 if eight else y))
        return x @ self.head, (saved, h8 if eight else h)

    def backward(self, dlogits, state, positions, seqs, seed, dropout):
        saved, after = state
        dx, dh = dlogits @ self.head.T, None
        for i in reversed(range(LAYERS)):
            layer, k = self.layers[i], saved[i]
            (a1, b1), (a2, b2) = layer.adapters
            g = api.norm_bwd(dx, after, self.norm_of(i + 1), dh=dh, y=k["y"], want_weights=False, **layer.block())
            d_o, da2, db2 = api.lora_bwd(g.dy, k["o"].flatten(1), layer.out, a2, b2, k["s2"], ALPHA, dropout, seed + 2 * i + 1)
            d_qkv = torch.empty_like(k["qkv"])
            dq, dk, dv = self.heads(d_qkv)
            api.attn_bwd(d_o.view_as(k["o"]), *self.heads(k["qkv"]), k["o"], k["lse"], seqs, dQ=dq, dK=dk, dV=dv)
            api.rope_bwd(dq, dk, positions, self.rope, dQ_out=dq, dK_out=dk)
            dx, da1, db1 = api.lora_bwd(d_qkv, k["x"], layer.qkv, a1, b1, k["s1"], ALPHA, dropout, seed + 2 * i)
            new = (da1, db1, da2, db2)
            if layer.grads is None:
                layer.grads = new
            else:   # the optimiser keeps its tensors' addresses
                for old, t in zip(layer.grads, new):
                    old.copy_(t)
            after, dh = k["h"], g.dh

    def parameters(self):
        for layer in self.layers:
            yield from zip((t for pair in layer.adapters for t in pair), layer.grads)


class Cache:
    """K and V of every layer in pages of PAGE rows; a request's pages follow each other, so that attention reads them as they are."""

    def __init__(self, lengths):
        self.first, rows = [], 0
        for n in lengths:
            self.first.append(rows)
            rows += -(-n // PAGE) * PAGE
        self.k, self.v = ([torch.zeros(rows, KV_HEADS, HEAD_DIM, device="cuda").bfloat16() for _ in range(LAYERS)] for _ in range(2))


def step(model, cache, tokens, positions, slots, seqs):
    """Logits of some rows, whose keys and values go into the cache."""
    x, h = api.norm_fwd(model.embed[tokens], model.norm_of(0), eps=EPS)
    for i, layer in enumerate(model.layers):
        (a1, b1), (a2, b2) = layer.adapters
        q, k, v = model.heads(api.lora_fwd(x, layer.qkv, a1, b1, ALPHA, 0.0, 0)[0])
        q = api.rope_append(q, k, v, positions, slots, cache.k[i], cache.v[i], model.rope)
        o = api.attn_fwd(q, cache.k[i], cache.v[i], seqs)[0]
        y = api.lora_fwd(o.flatten(1), layer.out, a2, b2, ALPHA, 0.0, 0)[0]
        x, h = api.norm_fwd(h, model.norm_of(i + 1), y=y, **layer.block())
    return x @ model.head


def generate(model, prompts, new):
    """Greedy continuations of several prompts: the prompts' rows at once, then a row a prompt.  Returns (tokens, logits of each new row)."""
    lengths = [len(p) for p in prompts]
    cache = Cache([n + new for n in lengths])

    def index(values):
        return torch.tensor(values, device="cuda")

    rows = [sum(lengths[:i]) for i in range(len(prompts))]
    logits = step(model, cache, torch.cat(prompts), index([t for n in lengths for t in range(n)]),
                  index([f + t for f, n in zip(cache.first, lengths) for t in range(n)]),
                  [(r, n, f, n) for r, f, n in zip(rows, cache.first, lengths)])
    logits = logits[index([r + n - 1 for r, n in zip(rows, lengths)])]
    tokens, seen = [], []
    for i in range(new):
        seen.append(logits)
        tokens.append(logits.argmax(1))
        if i + 1 < new:
            at = [n + i for n in lengths]
            logits = step(model, cache, tokens[-1], index(at), index([f + t for f, t in zip(cache.first, at)]),
                          [(r, 1, f, t + 1) for r, (f, t) in enumerate(zip(cache.first, at))])
    return torch.stack(tokens, 1), torch.stack(seen, 1)


def packed(lengths, seed):
    """Samples one after another: (tokens, labels, positions, [(first row, rows)])."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    places = [(sum(lengths[:i]), n) for i, n in enumerate(lengths)]
    tokens = torch.randint(0, VOCAB, (sum(lengths),), device="cuda", generator=gen)
    labels = torch.full_like(tokens, -1)
    for a, n in places:
        labels[a:a + n - 1] = tokens[a + 1:a + n]
    return tokens, labels, torch.cat([torch.arange(n, device="cuda") for n in lengths]), places


def train(steps=8, keep="8 bits", lr=2e-3, seed=0, verbose=False):
    """Trains every adapter on the samples' own tokens.  Returns (model, losses)."""
    model = Decoder(seed)
    tokens, labels, positions, places = packed([190, 77, 131, 64], seed)
    seqs, rows = api.attn_seqs(places), len(tokens)
    zeros, ones, optimiser, losses = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda"), None, []
    for n in range(1, steps + 1):
        logits, saved = model.forward(tokens, positions, seqs, 100 * n, 0.05, keep)
        # the policy loss at a ratio of one with advantages of one has the gradient of the mean log probability
        old = api.policy_loss(logits, labels, zeros, ones, want_grad=False)[1]
        _, logp, dlogits = api.policy_loss(logits, labels, old, ones, scale=1 / int((labels >= 0).sum()), dlogits=logits)
        model.backward(dlogits, saved, positions, seqs, 100 * n, 0.05)
        if optimiser is None:
            optimiser = api.adamw_tensors([api.adamw_tensor(p, g, bits=8, master=True) for p, g in model.parameters()])
        api.adamw_step(optimiser, lr=lr, step=n)
        losses.append(float(-logp.sum() / (labels >= 0).sum()))
        if verbose:
            print(f"step {n:2d}  loss {losses[-1]:.4f}")
    return model, losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--keep", choices=("8 bits", "bf16"), default="8 bits")
    ap.add_argument("--steps", type=int, default=8)
    args = ap.parse_args()
    trained, _ = train(args.steps, args.keep, verbose=True)
    prompts = [packed([n], n)[0] for n in (20, 7)]
    print("continuations", generate(trained, prompts, 8)[0].tolist())
