"""Cases that measure the operators around the LoRA linear layer in one fine-tuning step.

Three operators, each with its plain form (elementary torch operations in 32 bits) and the library's calls:

  attention   causal softmax attention over packed sequences with grouped heads, forward ("fwd") or
              forward and backward ("train")
  preference  the paired log-ratio loss on the logits of chosen and rejected responses, with d(loss)/d(logits)
  policy      the clipped policy loss with a KL term on the logits of sampled responses, with d(loss)/d(logits)
  adamw       one AdamW step over all adapter tensors, states in 32 bits or in 8

`own` selects which of the two run() computes.
"""
import math
import random

import numpy as np
import torch

own = False

# k and n of the seven projections of the two decoder layers this repository benchmarks (8B and 70B sizes)
LAYER_8B = [(4096, 4096), (4096, 1024), (4096, 1024), (4096, 4096), (4096, 14336), (4096, 14336), (14336, 4096)]
LAYER_70B = [(8192, 8192), (8192, 1024), (8192, 1024), (8192, 8192), (8192, 28672), (8192, 28672), (28672, 8192)]
BLOCK = 256     # values that share a scale in the 8-bit optimiser states
E4M3_MAX = 448.0
TINY = 2.0 ** -100   # a block whose largest value is below this is held as zeros


def listed():
    return [
        # one short prompt through one small attention layer: latency
        dict(name="attn_fwd_77", op="attention", mode="fwd", seqs=1, q_len=77, k_len=77, spread=0.0, hq=8, hkv=2, d=64,
             layout="rows"),
        # one whole long prompt, the 8B layer's heads
        dict(name="attn_fwd_8192", op="attention", mode="fwd", seqs=1, q_len=8192, k_len=8192, spread=0.0, hq=32,
             hkv=8, d=128, layout="rows"),
        # short continuations (some of a single token) of long prompts, K and V head by head
        dict(name="attn_fwd_continue", op="attention", mode="fwd", seqs=24, q_len=9, k_len=3000, spread=0.8, hq=32,
             hkv=8, d=128, layout="heads"),
        # a packed batch of ragged samples, 8B heads, Q, K and V slices of one fused projection output
        dict(name="attn_train_packed", op="attention", mode="train", seqs=14, q_len=450, k_len=450, spread=0.5, hq=32,
             hkv=8, d=128, layout="fused"),
        # a large training batch with the 70B layer's heads
        dict(name="attn_train_4x4096", op="attention", mode="train", seqs=4, q_len=4096, k_len=4096, spread=0.0,
             hq=64, hkv=8, d=128, layout="rows"),
        # a few short pairs, small vocabulary
        dict(name="preference_small", op="preference", pairs=4, length=40, spread=0.4, vocab=32000, dtype="bf16"),
        # a full batch of pairs, large vocabulary
        dict(name="preference_large", op="preference", pairs=16, length=256, spread=0.3, vocab=128000, dtype="bf16"),
        # a few sampled tokens, fp32 logits with an odd vocabulary
        dict(name="policy_small_odd", op="policy", tokens=203, vocab=50021, dtype="fp32", kl=0.05),
        # a full batch of sampled tokens, large vocabulary
        dict(name="policy_large", op="policy", tokens=8192, vocab=128000, dtype="bf16", kl=0.02),
        # the adapters of a single decoder layer
        dict(name="adamw_layer_32bit", op="adamw", layers=1, size="8b", rank=16, bits=32, master=False, odd=0),
        # every adapter of a 32-layer model, states in 8 bits, and some odd-sized fp32 vectors
        dict(name="adamw_model_8bit", op="adamw", layers=32, size="8b", rank=16, bits=8, master=False, odd=32),
        # a large rank on a large model, 32-bit states and an fp32 copy of the weights
        dict(name="adamw_large_master", op="adamw", layers=20, size="70b", rank=64, bits=32, master=True, odd=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "preference", "policy", "adamw"])
    if op == "attention":
        mode = rng.choice(["fwd", "train"])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 7, 8])
        d = rng.choice([40, 64, 96, 128])
        rows = _log_int(rng, 64, 16384)                    # rows of the whole batch
        seqs = min(_log_int(rng, 1, 48), max(1, rows // 8))
        k_len = max(8, min(8192, rows // seqs + rng.randint(-5, 5)))
        q_len = k_len if mode == "train" or rng.random() < 0.6 else max(1, k_len // rng.choice([2, 9, 50]))
        case = dict(op=op, mode=mode, seqs=seqs, q_len=q_len, k_len=k_len, spread=rng.choice([0.0, 0.3, 0.8]), hq=hq,
                    hkv=hkv, d=d, layout=rng.choice(["rows", "heads", "fused"]))
        while _attention_scores(case) > 4.3e9 and case["seqs"] > 1:      # the scores of the largest listed case
            case["seqs"] = case["seqs"] * 2 // 3
        while _attention_scores(case) > 4.3e9:
            case.update(q_len=case["q_len"] * 2 // 3, k_len=case["k_len"] * 2 // 3)
        return case
    if op == "preference":
        vocab = _log_int(rng, 2000, 160000)
        tokens = min(_log_int(rng, 32, 8192), 8192 * 128000 // vocab)
        pairs = max(1, min(_log_int(rng, 1, 64), tokens // 8))
        return dict(op=op, pairs=pairs, length=max(2, tokens // (2 * pairs)), spread=rng.choice([0.0, 0.3, 0.6]),
                    vocab=vocab, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "policy":
        vocab = _log_int(rng, 2000, 160000)
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        return dict(op=op, tokens=min(_log_int(rng, 1, 8192), 8192 * 64000 // vocab), vocab=vocab, dtype=dtype,
                    kl=rng.choice([0.0, 0.02, 0.1]))
    size = rng.choice(["8b", "70b"])
    rank = rng.choice([8, 16, 32, 64, 128])
    width = sum(k + n for k, n in (LAYER_8B if size == "8b" else LAYER_70B))
    layers = max(1, min(_log_int(rng, 1, 40), int(2e8 / (width * rank))))
    return dict(op=op, layers=layers, size=size, rank=rank, bits=rng.choice([8, 32]), master=rng.random() < 0.4,
                odd=rng.choice([0, 7, 40]))


# ---------------------------------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------------------------------

def _attention_lengths(case):
    """Lengths and first rows of each sequence: lognormal around the mean, every fourth continuation a single token,
    one sequence with more queries than keys (its first rows see no key), samples starting on 128-row boundaries
    as the packer lays them out."""
    r = random.Random(case["seqs"] * 7919 + case["q_len"] * 31 + case["k_len"])
    same = case["q_len"] == case["k_len"]
    seqs, q_row, k_row = [], 0, 0
    for i in range(case["seqs"]):
        f = math.exp(r.gauss(0.0, case["spread"])) if case["spread"] else 1.0
        k = max(1, min(4 * case["k_len"], int(case["k_len"] * f)))
        if same:
            q = k
        else:
            q = 1 if i % 4 == 1 else max(1, int(case["q_len"] * f))
            if i == 2:
                q, k = min(q, 4) + 9, 4
        seqs.append((q_row, q, k_row, k))
        up = (lambda x: -(-x // 128) * 128) if same else (lambda x: x)
        q_row, k_row = q_row + up(q), k_row + up(k)
    return seqs, q_row, k_row


def _attention_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    seqs, tq, tk = _attention_lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]

    def rows(t, h, layout):
        x = torch.randn(t * h * d, device="cuda", generator=g).bfloat16()
        return x.view(h, t, d).transpose(0, 1) if layout == "heads" else x.view(t, h, d)

    if case["layout"] == "fused" and tq == tk:
        qkv = rows(tq, hq + 2 * hkv, "rows")
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        q = rows(tq, hq, "rows")
        k, v = rows(tk, hkv, case["layout"]), rows(tk, hkv, case["layout"])
    do = rows(tq, hq, "rows") if case["mode"] == "train" else None
    return dict(seqs=seqs, q=q, k=k, v=v, do=do, scale=1.0 / math.sqrt(d))


def _padded(seqs, at, n):
    """Row numbers of each sequence, padded to the longest with row -1, and which of them are real."""
    longest = max(s[at + 1] for s in seqs)
    start = torch.tensor([s[at] for s in seqs], device="cuda")[:, None]
    length = torch.tensor([s[at + 1] for s in seqs], device="cuda")[:, None]
    i = torch.arange(longest, device="cuda")[None, :]
    return torch.where(i < length, start + i, n), i < length, length


def _plain_attention(st, train):
    """All sequences at once, each padded to the longest one."""
    q, k, v, scale = st["q"], st["k"], st["v"], st["scale"]
    (tq, hq, d), (tk, hkv, _) = q.shape, k.shape
    g = hq // hkv
    qi, q_real, q_len = _padded(st["seqs"], 0, tq)
    ki, k_real, k_len = _padded(st["seqs"], 2, tk)
    n, lq, lk = len(st["seqs"]), qi.shape[1], ki.shape[1]

    def gather(x, index, h):          # -> sequence, kv head, rows of its group, d
        x = torch.cat([x.float(), torch.zeros(1, *x.shape[1:], device="cuda")])[index]
        return x.view(n, index.shape[1], hkv, h // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)

    def scatter(x, index, rows, h, last):
        x = x.view(n, hkv, h // hkv, index.shape[1], last).permute(0, 3, 1, 2, 4).reshape(n, -1, h, last)
        out = torch.zeros(rows + 1, h, last, device="cuda")
        out[index.reshape(-1)] = x.reshape(-1, h, last)
        return out[:rows]

    Q, K, V = gather(q, qi, hq), gather(k, ki, hkv), gather(v, ki, hkv)
    see = torch.arange(lk, device="cuda")[None, None, :] <= \
        torch.arange(lq, device="cuda")[None, :, None] + (k_len - q_len)[:, :, None]
    see = (see & q_real[:, :, None] & k_real[:, None, :])[:, None, None]
    S = (Q @ K.transpose(2, 3)).mul_(scale).view(n, hkv, g, lq, lk).masked_fill_(~see, -math.inf)
    top = S.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    P = S.sub_(top).exp_()
    total = P.sum(-1, keepdim=True)
    P.div_(torch.where(total > 0, total, torch.ones_like(total)))
    lse = torch.log(total) + top
    P = P.view(n, hkv, g * lq, lk)
    O = P @ V
    out_lse = torch.full((tq + 1, hq), -math.inf, device="cuda")
    out_lse[qi.reshape(-1)] = lse.view(n, hq, lq).transpose(1, 2).reshape(-1, hq)
    out_lse[tq] = -math.inf
    out = dict(o=scatter(O, qi, tq, hq, d).bfloat16(), lse=out_lse[:tq])
    if train:
        dO = gather(st["do"], qi, hq)
        dV = P.transpose(2, 3) @ dO
        dP = dO @ V.transpose(2, 3)
        dS = dP.sub_((dO * O).sum(-1, keepdim=True)).mul_(P).mul_(scale)
        out["dq"] = scatter(dS @ K, qi, tq, hq, d).bfloat16()
        out["dk"] = scatter(dS.transpose(2, 3) @ Q, ki, tk, hkv, d).bfloat16()
        out["dv"] = scatter(dV, ki, tk, hkv, d).bfloat16()
    return out


def _exact_attention(case, seed):
    """Sequence by sequence and head by head, in 64 bits."""
    if _attention_pairs(case) * case["hq"] * case["d"] * (14 if case["mode"] == "train" else 4) > 8e12:
        return None
    st = _attention_inputs(case, seed)
    q, k, v = st["q"], st["k"], st["v"]
    g = case["hq"] // case["hkv"]
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(o), torch.zeros(k.shape, dtype=torch.float64, device="cuda"), \
        torch.zeros(v.shape, dtype=torch.float64, device="cuda")
    for qs, ql, ks, kl in st["seqs"]:
        row = torch.arange(max(0, ql - kl), ql, device="cuda")      # the rows that see a key
        if row.numel() == 0:
            continue
        hidden = torch.arange(kl, device="cuda")[None] > (row + kl - ql)[:, None]
        for h in range(case["hq"]):
            Q, K, V = q[qs + row, h].double(), k[ks:ks + kl, h // g].double(), v[ks:ks + kl, h // g].double()
            S = (Q @ K.T * st["scale"]).masked_fill(hidden, -math.inf)
            L = torch.logsumexp(S, 1)
            P = torch.exp(S - L[:, None])
            o[qs + row, h], lse[qs + row, h] = P @ V, L
            if case["mode"] == "train":
                dO = st["do"][qs + row, h].double()
                dP = dO @ V.T
                dS = P * (dP - (P * dP).sum(1, keepdim=True)) * st["scale"]
                dq[qs + row, h] = dS @ K
                dk[ks:ks + kl, h // g] += dS.T @ Q
                dv[ks:ks + kl, h // g] += P.T @ dO
    out = dict(o=o, lse=lse)
    if case["mode"] == "train":
        out.update(dq=dq, dk=dk, dv=dv)
    return out


def _attention_scores(case):
    """Scores of the padded batch."""
    seqs = _attention_lengths(case)[0]
    return len(seqs) * max(s[1] for s in seqs) * max(s[3] for s in seqs) * case["hq"]


def _attention_pairs(case):
    pairs = 0
    for _, q, _, k in _attention_lengths(case)[0]:
        rows = min(q, k)                       # the rows that see a key; the last one sees all k
        pairs += rows * k - rows * (rows - 1) // 2
    return pairs


# ---------------------------------------------------------------------------------------------------------------
# losses on logits
# ---------------------------------------------------------------------------------------------------------------

def _logits(case, tokens, g):
    """Logits like a language model's: broad, with the label's raised so that its probability is often large."""
    vocab = case["vocab"]
    labels = torch.randint(0, vocab, (tokens,), device="cuda", generator=g)
    z = torch.empty(tokens, vocab, dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.float32, device="cuda")
    for i in range(0, tokens, 1024):           # in pieces: the 32-bit values of a large batch need not exist at once
        part = torch.randn(min(1024, tokens - i), vocab, device="cuda", generator=g).mul_(2.0)
        raised = torch.randn(part.shape[0], device="cuda", generator=g).mul_(3.0).add_(9.0)
        part.scatter_add_(1, labels[i:i + 1024, None], raised[:, None])
        z[i:i + 1024] = part
    logp = torch.cat([torch.gather(x.float(), 1, y[:, None])[:, 0] - torch.logsumexp(x.float(), 1)
                      for x, y in zip(z.split(1024), labels.split(1024))])
    labels = torch.where(torch.rand(tokens, device="cuda", generator=g) < 0.1, -100, labels)   # prompt, padding
    return z, labels, logp


def _preference_pairs(case):
    """(chosen row, rejected row, chosen rows, rejected rows) of each pair, with unused rows between the pairs."""
    r = random.Random(case["pairs"] * 104729 + case["length"])
    pairs, at = [], 0
    for _ in range(case["pairs"]):
        a, b = (max(1, int(case["length"] * math.exp(r.gauss(0.0, case["spread"])))) for _ in range(2))
        pairs.append((at, at + a, a, b))
        at += a + b + r.randint(0, 2)
    return pairs, at


def _preference_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pairs, tokens = _preference_pairs(case)
    z, labels, logp = _logits(case, tokens, g)
    ref = logp + 0.3 * torch.randn(tokens, device="cuda", generator=g)
    return dict(pairs=pairs, logits=z, labels=labels, ref=ref, beta=0.1, smoothing=0.1, scale=1.0 / len(pairs))


def _policy_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    tokens = case["tokens"]
    z, labels, logp = _logits(case, tokens, g)
    # log ratios to the sampling policy: in and out of the clip range [0.8, 1.28], off its two ends (where the
    # gradient jumps) by more than rounding
    ratio = 0.15 * torch.randn(tokens, device="cuda", generator=g)
    for end in (math.log(0.8), math.log(1.28)):
        near = (ratio - end).abs() < 1e-3
        ratio = torch.where(near, end + 2e-3, ratio)
    adv = torch.randn(tokens, device="cuda", generator=g)
    ref = logp + 0.2 * torch.randn(tokens, device="cuda", generator=g)
    return dict(logits=z, labels=labels, old=logp - ratio, adv=adv, ref=ref if case["kl"] else None, low=0.2,
                high=0.28, kl=case["kl"], scale=1.0 / tokens)


def _plain_logp(z, labels):
    """log p of each label (0 where there is none), the softmax, the one-hot labels' index and which rows count."""
    z = z.float()
    counts = (labels >= 0) & (labels < z.shape[1])
    index = torch.where(counts, labels, 0)[:, None]
    z = z - z.amax(1, keepdim=True)
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    logp = torch.gather(z, 1, index) - torch.log(total)
    return torch.where(counts, logp[:, 0], 0.0), e.div_(total), index, counts


def _plain_dlogits(p, index, coefficient, dtype):
    """coefficient * (one-hot - softmax), row by row."""
    d = p.mul_(-coefficient[:, None])
    return d.scatter_add_(1, index, coefficient[:, None]).to(dtype)


def _plain_preference(st):
    logp, p, index, counts = _plain_logp(st["logits"], st["labels"])
    owner = torch.full((len(logp),), len(st["pairs"]), device="cuda")
    sign = torch.zeros(len(logp), device="cuda")
    table = torch.tensor(st["pairs"], device="cuda")
    row = torch.arange(len(logp), device="cuda")[:, None]
    for at, s in ((0, 1.0), (1, -1.0)):
        inside = (row >= table[:, at]) & (row < table[:, at] + table[:, at + 2])
        owner = torch.where(inside.any(1), inside.int().argmax(1), owner)
        sign = torch.where(inside.any(1), s, sign)
    member = (owner[None] == torch.arange(len(st["pairs"]), device="cuda")[:, None]).float() * sign
    log_ratio = torch.where(counts, logp - st["ref"], 0.0)
    margin = (member * log_ratio).sum(1)
    h, eps = st["beta"] * margin, st["smoothing"]
    log_sigmoid = torch.minimum(h, torch.zeros_like(h)) - torch.log1p(torch.exp(-h.abs()))
    loss = -(1 - eps) * log_sigmoid - eps * (log_sigmoid - h)
    dh = eps - (1 - eps) + (1 - eps) * torch.sigmoid(h) - eps + eps * torch.sigmoid(h)
    per_pair = torch.cat([st["scale"] * st["beta"] * dh, torch.zeros(1, device="cuda")])
    coefficient = torch.where(counts, per_pair[owner] * sign, 0.0)
    return dict(loss=st["scale"] * loss.sum(), logp=logp, margin=margin,
                dlogits=_plain_dlogits(p, index, coefficient, st["logits"].dtype))


def _plain_policy(st):
    logp, p, index, counts = _plain_logp(st["logits"], st["labels"])
    adv = st["adv"]
    ratio = torch.exp(logp - st["old"])
    gain = torch.minimum(ratio * adv, torch.clamp(ratio, 1 - st["low"], 1 + st["high"]) * adv)
    free = torch.where(adv >= 0, ratio <= 1 + st["high"], ratio >= 1 - st["low"])
    loss, slope = -gain, -torch.where(free, ratio * adv, 0.0)
    if st["ref"] is not None:
        e = torch.exp(st["ref"] - logp)
        loss = loss + st["kl"] * (e - (st["ref"] - logp) - 1)
        slope = slope + st["kl"] * (1 - e)
    loss, slope = torch.where(counts, loss, 0.0), torch.where(counts, slope, 0.0)
    return dict(loss=st["scale"] * loss.sum(), logp=logp,
                dlogits=_plain_dlogits(p, index, st["scale"] * slope, st["logits"].dtype))


def _exact_rows(z, labels):
    """Pieces of rows in 64 bits: (first row, log softmax, label or -1)."""
    for i in range(0, z.shape[0], 512):
        x = z[i:i + 512].double()
        yield i, x - torch.logsumexp(x, 1, keepdim=True), labels[i:i + 512]


def _exact_logp(z, labels):
    out = torch.zeros(z.shape[0], dtype=torch.float64, device="cuda")
    for i, x, y in _exact_rows(z, labels):
        at = torch.nonzero(y >= 0)[:, 0]
        out[i + at] = x[at, y[at]]
    return out


def _exact_dlogits(z, labels, c):
    """In 64 bits where that is little; of a large batch the bf16 gradients rounded to 32 bits."""
    d = torch.empty(z.shape, dtype=torch.float64 if z.numel() < 2 ** 29 else torch.float32, device="cuda")
    for i, x, y in _exact_rows(z, labels):
        part = -torch.exp(x) * c[i:i + 512, None]
        at = torch.nonzero(y >= 0)[:, 0]
        part[at, y[at]] += c[i + at]
        d[i:i + 512] = part
    return d


def _exact_preference(case, seed):
    st = _preference_inputs(case, seed)
    logp = _exact_logp(st["logits"], st["labels"])
    ratio = torch.where(st["labels"] >= 0, logp - st["ref"].double(), 0.0)
    margin = torch.stack([ratio[c:c + n].sum() - ratio[r:r + m].sum() for c, r, n, m in st["pairs"]])
    h, eps = st["beta"] * margin, st["smoothing"]
    loss = (1 - eps) * torch.logaddexp(torch.zeros_like(h), -h) + eps * torch.logaddexp(torch.zeros_like(h), h)
    dh = -(1 - eps) / (1 + torch.exp(h)) + eps / (1 + torch.exp(-h))
    c = torch.zeros_like(logp)
    for (a, b, n, m), s in zip(st["pairs"], (st["scale"] * st["beta"] * dh).tolist()):
        c[a:a + n], c[b:b + m] = s, -s
    c = torch.where(st["labels"] >= 0, c, 0.0)
    return dict(loss=st["scale"] * loss.sum(), logp=logp, margin=margin,
                dlogits=_exact_dlogits(st["logits"], st["labels"], c))


def _exact_policy(case, seed):
    st = _policy_inputs(case, seed)
    logp = _exact_logp(st["logits"], st["labels"])
    old, adv = st["old"].double(), st["adv"].double()
    r = torch.exp(logp - old)
    clipped = r.clamp(1 - st["low"], 1 + st["high"])
    loss = -torch.minimum(r * adv, clipped * adv)
    slope = torch.where(r * adv <= clipped * adv, -r * adv, 0.0)
    if st["ref"] is not None:
        x = st["ref"].double() - logp
        loss, slope = loss + st["kl"] * (torch.exp(x) - x - 1), slope - st["kl"] * torch.expm1(x)
    counts = st["labels"] >= 0
    c = torch.where(counts, st["scale"] * slope, 0.0)
    return dict(loss=st["scale"] * loss[counts].sum(), logp=logp,
                dlogits=_exact_dlogits(st["logits"], st["labels"], c))


# ---------------------------------------------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------------------------------------------

def _adamw_sizes(case):
    """Numbers of values: A and B of every adapter, then some fp32 vectors of odd sizes (magnitudes, biases)."""
    layer = LAYER_8B if case["size"] == "8b" else LAYER_70B
    r = case["rank"]
    adapters = [x * r for _ in range(case["layers"]) for k, n in layer for x in (k, n)]
    return adapters, [1 + 997 * i % 4099 for i in range(case["odd"])]


def _adamw_inputs(case, seed):
    """Each group of tensors (bf16 adapters, fp32 vectors) lies in one buffer a quantity, every tensor on whole
    blocks of 256; what is between the tensors is zero and stays zero."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    groups = []
    for sizes, dtype in zip(_adamw_sizes(case), (torch.bfloat16, torch.float32)):
        if not sizes:
            continue
        starts = np.cumsum([0] + [-(-s // BLOCK) * BLOCK for s in sizes]).tolist()
        real = torch.zeros(starts[-1], device="cuda")
        for a, s in zip(starts, sizes):
            real[a:a + s] = 1.0

        def values(size):
            return torch.randn(starts[-1], device="cuda", generator=gen).mul_(size).mul_(real)

        master = values(0.02)
        # gradients whose size differs from place to place, as those of different features do
        grad = values(1e-3) * torch.exp(values(1.0))
        m, v = values(3e-4), values(1e-3).square_()
        group = dict(starts=starts, sizes=sizes, dtype=dtype, param=master.to(dtype), grad=grad.to(dtype),
                     master=master if case["master"] and dtype == torch.bfloat16 else None)
        if case["bits"] == 8:
            group["m"], group["m_scale"] = _to_8_bits(m, False)
            group["v"], group["v_scale"] = _to_8_bits(torch.sqrt(v), True)
        else:
            group["m"], group["v"] = m, v
        groups.append(group)
    return dict(groups=groups, bits=case["bits"], lr=2e-4, beta1=0.9, beta2=0.999, eps=1e-8, decay=0.01, step=10)


def _to_8_bits(x, keep_positive):
    """Blocks of 256 in e4m3 with one scale each, largest value / 448; with keep_positive no value above zero
    becomes zero (the smallest code, 2^-9, stands in for it)."""
    b = x.view(-1, BLOCK)
    top = b.abs().amax(1, keepdim=True)
    top = torch.where(top >= TINY, top, torch.zeros_like(top))
    scaled = b * torch.where(top > 0, E4M3_MAX / top, torch.zeros_like(top))
    if keep_positive:
        scaled = torch.where((b > 0) & (top > 0), scaled.clamp(min=2.0 ** -9), scaled)
    return scaled.to(torch.float8_e4m3fn).view(-1), (top * (1.0 / E4M3_MAX)).view(-1)


def _from_8_bits(codes, scale):
    return (codes.float().view(-1, BLOCK) * scale[:, None]).view(-1)


def _plain_adamw(st):
    out = []
    for s in st["groups"]:
        g = s["grad"].float()
        if st["bits"] == 8:
            m, root = _from_8_bits(s["m"], s["m_scale"]), _from_8_bits(s["v"], s["v_scale"])
            v = root * root
        else:
            m, v = s["m"], s["v"]
        m = m * st["beta1"] + g * (1 - st["beta1"])
        v = v * st["beta2"] + (g * g) * (1 - st["beta2"])
        root = torch.sqrt(v)
        p = s["master"] if s["master"] is not None else s["param"].float()
        c1, c2 = 1 - st["beta1"] ** st["step"], 1 - st["beta2"] ** st["step"]
        p = p * (1 - st["lr"] * st["decay"]) - (st["lr"] / c1) * m / (root / math.sqrt(c2) + st["eps"])
        if s["master"] is not None:
            s["master"].copy_(p)
        s["param"].copy_(p)
        if st["bits"] == 8:
            s["m"], s["m_scale"] = _to_8_bits(m, False)
            s["v"], s["v_scale"] = _to_8_bits(root, True)
        else:
            s["m"].copy_(m)
            s["v"].copy_(v)
        out.append(s)
    return _adamw_outputs(out, st["bits"])


def _adamw_outputs(groups, bits):
    """The updated buffers; of the 8-bit states the codes, as the float8 values they are, and the blocks' scales."""
    out = []
    for s in groups:
        o = dict(param=s["param"], master=s["master"], m=s["m"], v=s["v"])
        if bits == 8:
            o["m_scale"], o["v_scale"] = s["m_scale"], s["v_scale"]
        out.append(o)
    return out


def _exact_adamw(case, seed):
    if sum(map(sum, _adamw_sizes(case))) > 3e8:
        return None
    st = _adamw_inputs(case, seed)
    out = []
    for s in st["groups"]:
        g = s["grad"].double()
        if st["bits"] == 8:
            m = s["m"].double().view(-1, BLOCK).mul(s["m_scale"].double()[:, None]).view(-1)
            v = s["v"].double().view(-1, BLOCK).mul(s["v_scale"].double()[:, None]).view(-1).square()
        else:
            m, v = s["m"].double(), s["v"].double()
        m.mul_(st["beta1"]).add_(g, alpha=1 - st["beta1"])
        v.mul_(st["beta2"]).addcmul_(g, g, value=1 - st["beta2"])
        p = s["master"].double() if s["master"] is not None else s["param"].double()
        m_hat, v_hat = m / (1 - st["beta1"] ** st["step"]), v / (1 - st["beta2"] ** st["step"])
        p = p - st["lr"] * (m_hat / (v_hat.sqrt() + st["eps"]) + st["decay"] * p)
        o = dict(param=p, master=p if s["master"] is not None else None)
        if st["bits"] == 8:
            for name, x in (("m", m), ("v", v.sqrt())):
                b = x.view(-1, BLOCK)
                scale = b.abs().amax(1, keepdim=True) / E4M3_MAX
                y = b / torch.where(scale > 0, scale, 1.0)
                if name == "v":
                    y = torch.where(b > 0, y.clamp(min=2.0 ** -9), y)
                # e4m3: three fraction bits, smallest exponent -6
                size = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
                o[name], o[name + "_scale"] = (torch.round(y / size) * size).view(-1), scale.view(-1)
        else:
            o["m"], o["v"] = m, v
        out.append(o)
    return out


# ---------------------------------------------------------------------------------------------------------------
# what the tools call
# ---------------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    make = dict(attention=_attention_inputs, preference=_preference_inputs, policy=_policy_inputs,
                adamw=_adamw_inputs)[case["op"]]
    st = make(case, seed)
    st.update(op=case["op"], mode=case.get("mode"))
    if own and st["op"] == "attention":
        from lora_fine_tuning_gb300 import api
        st["table"] = api.attn_seqs(st["seqs"])             # a packed batch's table, used by every layer
    elif own and st["op"] == "preference":
        from lora_fine_tuning_gb300 import api
        st["table"] = api.pref_pairs(st["pairs"])
    elif own and st["op"] == "adamw":
        from lora_fine_tuning_gb300 import api

        def views(s, name):
            return None if s[name] is None else [s[name][a:a + n] for a, n in zip(s["starts"], s["sizes"])]

        def scales(s, name):
            return [s[name][a // BLOCK:-(-(a + n) // BLOCK)] for a, n in zip(s["starts"], s["sizes"])]

        parts = []
        for s in st["groups"]:
            keys = ("param", "grad", "m", "v", "master")
            columns = [views(s, name) or [None] * len(s["sizes"]) for name in keys]
            more = [scales(s, name) for name in ("m_scale", "v_scale")] if st["bits"] == 8 else \
                [[None] * len(s["sizes"])] * 2
            parts += [api.AdamWTensor(*row) for row in zip(*columns, *more)]
        st["table"] = api.adamw_tensors(parts)              # the optimiser's list, made once
    return st


def run(st):
    if not own:
        if st["op"] == "attention":
            return _plain_attention(st, st["mode"] == "train")
        return dict(preference=_plain_preference, policy=_plain_policy, adamw=_plain_adamw)[st["op"]](st)
    from lora_fine_tuning_gb300 import api
    if st["op"] == "attention":
        o, lse = api.attn_fwd(st["q"], st["k"], st["v"], st["table"], scale=st["scale"])
        if st["mode"] == "fwd":
            return dict(o=o, lse=lse)
        dq, dk, dv = api.attn_bwd(st["do"], st["q"], st["k"], st["v"], o, lse, st["table"], scale=st["scale"])
        return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)
    if st["op"] == "preference":
        loss, logp, margin, dlogits = api.pref_loss(st["logits"], st["labels"], st["table"], st["ref"],
                                                    beta=st["beta"], label_smoothing=st["smoothing"],
                                                    scale=st["scale"])
        return dict(loss=loss, logp=logp, margin=margin, dlogits=dlogits)
    if st["op"] == "policy":
        loss, logp, dlogits = api.policy_loss(st["logits"], st["labels"], st["old"], st["adv"], st["ref"],
                                              clip_low=st["low"], clip_high=st["high"], kl_coef=st["kl"],
                                              scale=st["scale"])
        return dict(loss=loss, logp=logp, dlogits=dlogits)
    api.adamw_step(st["table"], lr=st["lr"], beta1=st["beta1"], beta2=st["beta2"], eps=st["eps"],
                   weight_decay=st["decay"], step=st["step"])
    return _adamw_outputs(st["groups"], st["bits"])


def exact(case, seed):
    return dict(attention=_exact_attention, preference=_exact_preference, policy=_exact_policy,
                adamw=_exact_adamw)[case["op"]](case, seed)


def work(case):
    """Every input read once and every output written once; products of the pairs that are not masked."""
    if case["op"] == "attention":
        _, tq, tk = _attention_lengths(case)
        q, kv = tq * case["hq"] * case["d"] * 2, tk * case["hkv"] * case["d"] * 2
        train = case["mode"] == "train"
        # forward: Q, K, V, O; backward again Q, K, V, O, dO and the three gradients
        nbytes = 2 * q + 2 * kv + (4 * q + 4 * kv if train else 0) + tq * case["hq"] * 4
        return dict(bytes=nbytes, flops=_attention_pairs(case) * case["hq"] * case["d"] * (14 if train else 4))
    if case["op"] in ("preference", "policy"):
        tokens = _preference_pairs(case)[1] if case["op"] == "preference" else case["tokens"]
        values = tokens * case["vocab"]
        return dict(bytes=values * (4 if case["dtype"] == "bf16" else 8) + tokens * 24, flops=values * 6)
    adapters, vectors = (sum(s) for s in _adamw_sizes(case))
    states = (4 + 8 / BLOCK * 2) if case["bits"] == 8 else 16       # two states read and written
    copy = 8 if case["master"] else 2                               # the fp32 copy read and written, else p read
    return dict(bytes=adapters * (2 + 2 + copy + states) + vectors * (12 + states), flops=(adapters + vectors) * 16)
