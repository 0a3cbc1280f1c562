"""Cases that measure what stands between the adapter projections of a decoder layer, in training and for single tokens.

Five operators, each with its plain form (elementary torch operations in 32 bits) and the library's calls:

  norm     the normalised, gated and scaled block output added to the stream, and the stream's norm before the next
           block: forward ("fwd"), backward ("bwd"), or both through checkpoints in 8 bits ("ckpt")
  rope     rotary positions on queries and keys, forward and backward
  append   rotary positions on queries and keys, keys and values stored into the rows of a cache
  act8     activations into 8 bits (32 values share a power of two) and back
  lora     the adapter layer's backward from an input that was kept in 8 bits

`own` selects which of the two run() computes.
"""
import math
import random

import torch

own = False

BLOCK = 32      # values that share a scale in 8 bits


def listed():
    return [
        # the tokens of a few requests between two blocks of the 8B layer: latency
        dict(name="norm_fwd_3x4096", op="norm", mode="fwd", rows=3, width=4096, stream="bf16", y=True, post=False,
             gate=False, row_gate=False, weights=False, offset=0.0),
        # a packed batch of the 8B layer: the stream and the adapters' input kept in 8 bits, frozen weights
        dict(name="norm_ckpt_8192x4096", op="norm", mode="ckpt", rows=8192, width=4096, stream="bf16", y=True,
             post=False, gate=False, row_gate=False, weights=False, offset=0.0),
        # a width that no vector divides, fp32 stream, a weight for each row, every parameter trained
        dict(name="norm_bwd_1999x2050", op="norm", mode="bwd", rows=1999, width=2050, stream="fp32", y=True, post=True,
             gate=False, row_gate=True, weights=True, offset=1.0),
        # a large batch of the 70B layer: norms before and after the block, gates, every parameter trained
        dict(name="norm_bwd_16384x8192", op="norm", mode="bwd", rows=16384, width=8192, stream="bf16", y=True,
             post=True, gate=True, row_gate=False, weights=True, offset=0.0),
        # a packed batch, 8B heads, slices of a fused projection, halves of the head rotated against each other
        dict(name="rope_8192_fused", op="rope", rows=8192, hq=32, hkv=8, d=128, rot=128, interleaved=False, far=0,
             scaling="none", layout="fused"),
        # samples far inside long contexts, 70B heads, neighbours of the head's first half rotated
        dict(name="rope_12000_far", op="rope", rows=12000, hq=64, hkv=8, d=128, rot=64, interleaved=True,
             far=900000, scaling="parts", layout="rows"),
        # a token of each of 64 requests into the pages of a cache
        dict(name="append_64", op="append", rows=64, hq=32, hkv=8, d=128, rot=128, interleaved=False, far=4000,
             scaling="none", layout="fused", page=16),
        # a prompt's rows into the pages of a cache, small heads
        dict(name="append_5000", op="append", rows=5000, hq=24, hkv=8, d=64, rot=64, interleaved=False, far=30000,
             scaling="linear", layout="fused", page=64),
        # one short sample whose width is no multiple of the blocks
        dict(name="act8_77x1000", op="act8", rows=77, width=1000),
        # the widest activation of the 8B layer
        dict(name="act8_8192x14336", op="act8", rows=8192, width=14336),
        # one small layer
        dict(name="lora_640x512", op="lora", m=640, k=512, n=768, r=16, p=0.0),
        # a packed batch through the 8B layer's key projection, with dropout
        dict(name="lora_8192x4096", op="lora", m=8192, k=4096, n=1024, r=16, p=0.05),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm", "rope", "append", "act8", "lora"])
    if op == "norm":
        mode = rng.choice(["fwd", "bwd", "bwd", "ckpt"])
        width = rng.choice([8 * _log_int(rng, 8, 1024), 8 * _log_int(rng, 64, 1024), _log_int(rng, 65, 8192)])
        stream = "bf16" if mode == "ckpt" else rng.choice(["bf16", "bf16", "fp32"])
        y = mode == "ckpt" or rng.random() < 0.8
        case = dict(op=op, mode=mode, rows=_log_int(rng, 1, 16384), width=width, stream=stream, y=y,
                    post=y and rng.random() < 0.5, gate=y and rng.random() < 0.4, row_gate=y and rng.random() < 0.25,
                    weights=mode == "bwd" and rng.random() < 0.5, offset=rng.choice([0.0, 0.0, 1.0]))
        least = "rows"
    elif op in ("rope", "append"):
        hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([40, 64, 96, 128])
        rot = rng.choice([d, d, d // 2, d // 4 // 2 * 2])
        case = dict(op=op, rows=_log_int(rng, 1, 16384), hq=hkv * rng.choice([1, 2, 4, 7, 8]), hkv=hkv, d=d, rot=rot,
                    interleaved=rng.random() < 0.4, far=rng.choice([0, 5000, 200000, 1000000]),
                    scaling=rng.choice(["none", "linear", "base", "parts"]), layout=rng.choice(["rows", "fused"]))
        if op == "append":
            case["page"] = rng.choice([1, 16, 64, 128])
        least = "rows"
    elif op == "act8":
        case = dict(op=op, rows=_log_int(rng, 1, 16384), width=rng.choice([_log_int(rng, 33, 16384),
                                                                         8 * _log_int(rng, 16, 2048)]))
        least = "rows"
    else:
        case = dict(op=op, m=_log_int(rng, 17, 8192), k=8 * _log_int(rng, 16, 512), n=8 * _log_int(rng, 16, 256),
                    r=rng.choice([8, 16, 32, 64]), p=rng.choice([0.0, 0.05, 0.3]))
        least = "m"
    while _cost(case) > 1.5e9:
        case[least] = case[least] * 4 // 5
    return case


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 100)


# ---------------------------------------------------------------------------------------------------------------
# 8 bits: blocks of 32 values along a row share a power of two, 2^(floor(log2 of the largest) - 6); codes are whole
# numbers of at most 127 (the only value beyond it, 127.5, lies as far from 127 as from 128)
# ---------------------------------------------------------------------------------------------------------------

def _to_8_bits(x):
    """Codes (rows x whole blocks) and exponents, biased by 127 (rows x four for every 128 values)."""
    rows, width = x.shape
    blocks = -(-width // BLOCK)
    b = torch.zeros(rows, blocks * BLOCK, device=x.device)
    b[:, :width] = x
    b = b.view(rows, blocks, BLOCK)
    _, e = torch.frexp(b.abs().amax(2, keepdim=True))
    e = (e - 7).clamp(min=-126)
    codes = torch.round(torch.ldexp(b, -e)).clamp(-127, 127).to(torch.int8)
    scales = torch.full((rows, -(-width // 128) * 4), 127, dtype=torch.uint8, device=x.device)
    scales[:, :blocks] = (e + 127)[:, :, 0].to(torch.uint8)
    return codes.view(rows, -1), scales


def _from_8_bits(codes, scales, width):
    rows = codes.shape[0]
    b = codes.float().view(rows, -1, BLOCK)
    e = scales[:, :b.shape[1]].int() - 127
    return torch.ldexp(b, e[:, :, None]).view(rows, -1)[:, :width]


def _exact_8_bits(x):
    """The values that a matrix in bf16 stands for when it is held in 8 bits, in 64 bits."""
    rows, width = x.shape
    x = torch.nn.functional.pad(x.double(), (0, -width % BLOCK)).view(rows, -1, BLOCK)
    top = x.abs().amax(2, keepdim=True)
    step = torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, 1.0))) - 6)
    return (torch.round(x / step).clamp(-127, 127) * step).view(rows, -1)[:, :width]


def _act8_inputs(case, seed):
    """Activations whose channels have sizes of their own, a few of them large."""
    return dict(x=_activations(case["rows"], case["width"], torch.Generator(device="cuda").manual_seed(seed)))


def _activations(rows, width, g):
    size = torch.exp(0.5 * torch.randn(width, device="cuda", generator=g))
    size = torch.where(torch.rand(width, device="cuda", generator=g) < 0.01, size * 20, size)
    return (torch.randn(rows, width, device="cuda", generator=g) * size).bfloat16()


def _plain_act8(st):
    codes, scales = _to_8_bits(st["x"].float())
    return dict(x=_from_8_bits(codes, scales, st["x"].shape[1]).bfloat16())


def _exact_act8(case, seed):
    return dict(x=_exact_8_bits(_act8_inputs(case, seed)["x"]))


# ---------------------------------------------------------------------------------------------------------------
# norms, gates and the stream
# ---------------------------------------------------------------------------------------------------------------

def _norm_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, width = case["rows"], case["width"]

    def normal(*shape, size=1.0, mean=0.0):
        return torch.randn(*shape, device="cuda", generator=g) * size + mean

    stream = torch.float32 if case["stream"] == "fp32" else torch.bfloat16
    mean = 1.0 - case["offset"]
    st = dict(h=(_activations(rows, width, g).float() * 2).to(stream), w=normal(width, size=0.2, mean=mean).bfloat16(),
              y=_activations(rows, width, g) if case["y"] else None,
              post_w=normal(width, size=0.2, mean=mean).bfloat16() if case["post"] else None,
              gate=normal(width, size=0.3, mean=0.5) if case["gate"] else None,
              row_gate=torch.rand(rows, device="cuda", generator=g) if case["row_gate"] else None,
              res_scale=0.22, eps=1e-5, offset=case["offset"], weights=case["weights"])
    if case["mode"] != "fwd":
        st["dx"], st["dh"] = normal(rows, width).bfloat16(), normal(rows, width).to(stream)
    return st


def _plain_unit(x, eps):
    """x over its root mean square, and one over that."""
    r = torch.rsqrt((x * x).mean(1, keepdim=True) + eps)
    return x * r, r


def _plain_norm_fwd(st):
    """The stream after the block and its norm, in 32 bits."""
    h = st["h"].float()
    if st["y"] is not None:
        u = st["y"].float()
        if st["post_w"] is not None:
            u = _plain_unit(u, st["eps"])[0] * (st["post_w"].float() + st["offset"])
        if st["gate"] is not None:
            u = u * st["gate"]
        if st["row_gate"] is not None:
            u = u * st["row_gate"][:, None]
        h = h + u * st["res_scale"]
    return h, _plain_unit(h, st["eps"])[0] * (st["w"].float() + st["offset"])


def _plain_norm_bwd(st, h):
    """From the gradients of the norm (dx) and of the stream (dh); h: the stream after the block."""
    stream, s = st["h"].dtype, st["res_scale"]
    n, r = _plain_unit(h.float(), st["eps"])
    dx = st["dx"].float()
    t = dx * (st["w"].float() + st["offset"])
    dh = st["dh"].float() + r * (t - n * (t * n).mean(1, keepdim=True))
    out = dict(dh=dh.to(stream))
    if st["weights"]:
        out["dw"] = (dx * n).sum(0)
    if st["y"] is None:
        return out
    u, r = st["y"].float(), None
    if st["post_w"] is not None:
        u, r = _plain_unit(u, st["eps"])
    d = dh * s
    row = d if st["row_gate"] is None else d * st["row_gate"][:, None]
    gated = row if st["gate"] is None else row * st["gate"]
    w = None if st["post_w"] is None else st["post_w"].float() + st["offset"]
    if st["weights"]:
        if st["gate"] is not None:
            out["dgate"] = (row * u).sum(0) if w is None else (row * u).sum(0) * w
        if st["post_w"] is not None:
            out["dpost_w"] = (gated * u).sum(0)
        if st["row_gate"] is not None:
            v = u if w is None else u * w
            out["drow_gate"] = (d * (v if st["gate"] is None else v * st["gate"])).sum(1)
    if st["post_w"] is not None:
        t = gated * w
        gated = r * (t - u * (t * u).mean(1, keepdim=True))
    out["dy"] = gated.bfloat16()
    return out


def _plain_norm(st):
    if st["mode"] == "bwd":
        return _plain_norm_bwd(st, st["h"])
    h, x = _plain_norm_fwd(st)
    out = dict(h_out=h.to(st["h"].dtype), x=x.bfloat16())
    if st["mode"] == "ckpt":
        width = x.shape[1]
        out["x8"] = _from_8_bits(*_to_8_bits(out["x"].float()), width).bfloat16()
        kept = _from_8_bits(*_to_8_bits(out["h_out"].float()), width)
        out.update(_plain_norm_bwd(st, kept))
    return out


def _exact_norm(case, seed):
    """The backward as sums over the forward's own derivatives, written out by rows in 64 bits."""
    st = _norm_inputs(case, seed)
    y, h, s = st["y"], st["h"].double(), st["res_scale"]
    w = st["w"].double() + st["offset"]
    rows, width = h.shape
    one = torch.ones((), dtype=torch.float64, device="cuda")
    c = s * (st["gate"].double()[None] if case["gate"] else one) * (st["row_gate"].double()[:, None] if case["row_gate"] else one)
    v = p = None
    if y is not None:
        y = y.double()
        rms = torch.sqrt(torch.linalg.vector_norm(y, dim=1, keepdim=True) ** 2 / width + st["eps"])
        p = st["post_w"].double() + st["offset"] if case["post"] else one
        v = y / rms if case["post"] else y
    out = {}
    if case["mode"] != "bwd":
        if y is not None:
            h = h + c * p * v
        size = torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / width + st["eps"])
        out.update(h_out=h, x=h / size * w)
        if case["mode"] == "fwd":
            return out
        out["x8"] = _exact_8_bits(out["x"].bfloat16())
        h = _exact_8_bits(h.bfloat16())
    size = torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / width + st["eps"])
    dx = st["dx"].double()
    along = torch.einsum("ij,j,ij->i", dx, w, h)[:, None] / (width * size ** 3)
    dh = st["dh"].double() + dx * w / size - h * along
    out["dh"] = dh
    if case["weights"]:
        out["dw"] = torch.einsum("ij,ij->j", dx, h / size)
    if y is None:
        return out
    if case["weights"]:
        rg = st["row_gate"].double() if case["row_gate"] else torch.ones(rows, dtype=torch.float64, device="cuda")
        each = torch.einsum("ij,ij,i->j", dh, v, rg) * s
        if case["gate"]:
            out["dgate"] = each * p
        if case["post"]:
            out["dpost_w"] = each * (st["gate"].double() if case["gate"] else one)
        if case["row_gate"]:
            out["drow_gate"] = (dh * v * p * (st["gate"].double() if case["gate"] else one)).sum(1) * s
    t = dh * c * p
    out["dy"] = (t - y * (t * y).sum(1, keepdim=True) / (width * rms ** 2)) / rms if case["post"] else t
    return out


# ---------------------------------------------------------------------------------------------------------------
# rotary positions, and the cache
# ---------------------------------------------------------------------------------------------------------------

# how contexts longer than the trained ones are reached: `linear`: all positions over a factor; `base`: a larger base;
# `parts`: frequencies with few turns over the trained length as linear, those with many as they are, and a magnitude
SCALING = dict(none={}, linear=dict(scaling="linear", factor=4.0), base=dict(scaling="base", factor=8.0),
               parts=dict(scaling="parts", factor=32.0, original=8192, low=1.0, high=32.0, magnitude=1.3466))
BASE = 500000.0


def _frequencies(rot, name):
    """Radians a position of each pair."""
    s = SCALING[name]
    base, factor = BASE, s.get("factor", 1.0)
    if name == "base":
        base *= factor ** (rot / (rot - 2)) if rot > 2 else 1.0
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if name == "linear":
        f = [x / factor for x in f]
    if name == "parts":
        turns = [s["original"] * x / (2 * math.pi) for x in f]
        keep = [min(1.0, max(0.0, (t - s["low"]) / (s["high"] - s["low"]))) for t in turns]
        f = [x * k + x / factor * (1 - k) for x, k in zip(f, keep)]
    return f


def _rope_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, hq, hkv, d = case["rows"], case["hq"], case["hkv"], case["d"]

    def heads():
        if case["layout"] == "fused":
            qkv = torch.randn(rows, hq + 2 * hkv, d, device="cuda", generator=g).bfloat16()
            return qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        return tuple(torch.randn(rows, h, d, device="cuda", generator=g).bfloat16() for h in (hq, hkv, hkv))

    st = dict(rot=case["rot"], interleaved=case["interleaved"], scaling=case["scaling"],
              magnitude=SCALING[case["scaling"]].get("magnitude", 1.0),
              freq=torch.tensor(_frequencies(case["rot"], case["scaling"]), dtype=torch.float64, device="cuda"))
    st["q"], st["k"], st["v"] = heads()
    r = random.Random(seed)
    if case["op"] == "rope":
        st["dq"], st["dk"], _ = heads()
        positions = []                       # samples of a packed batch, each from its own place in its context
        while len(positions) < rows:
            first = r.randint(0, case["far"])
            positions += range(first, first + min(rows - len(positions), r.randint(1, 4096)))
        st["positions"] = torch.tensor(positions, device="cuda")
        return st
    # rows in the order of their requests; each request's rows go to pages of its own, which lie anywhere
    page, requests, at = case["page"], [], 0
    while at < rows:
        n = 1 if rows <= 256 else min(rows - at, r.randint(1, 3000))
        requests.append((r.randint(0, case["far"]), n))
        at += n
    table, positions = [], []
    for first, n in requests:
        need = (first + n - 1) // page - first // page + 1
        table += [(first, len(positions), need)]
        positions += range(first, first + n)
    total = sum(need for _, _, need in table) + 8
    free = list(range(total))
    r.shuffle(free)
    slots = []
    for (first, n), (_, _, need) in zip(requests, table):
        pages, free = free[:need], free[need:]
        slots += [pages[x // page - first // page] * page + x % page for x in range(first, first + n)]
    for i in range(7, rows, 50):             # rows of padding: not stored
        slots[i] = -1
    st["positions"], st["slots"] = torch.tensor(positions, device="cuda"), torch.tensor(slots, device="cuda")
    st["k_cache"], st["v_cache"] = (torch.randn(total * page, hkv, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    return st


def _plain_turned(x, st, back):
    """x (rows x heads x features) turned by its rows' positions; back: the transposed rotation."""
    rot = st["rot"]
    angle = st["positions"].double()[:, None] * st["freq"]
    c = (torch.cos(angle) * st["magnitude"]).float()[:, None]
    s = (torch.sin(angle) * (-st["magnitude"] if back else st["magnitude"])).float()[:, None]
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if st["interleaved"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    pair = (a * c - b * s, b * c + a * s)
    turned = torch.stack(pair, -1).flatten(-2) if st["interleaved"] else torch.cat(pair, -1)
    return torch.cat([turned, x[..., rot:]], -1).bfloat16()


def _plain_rope(st):
    if "slots" not in st:
        return dict(q=_plain_turned(st["q"], st, False), k=_plain_turned(st["k"], st, False),
                    dq=_plain_turned(st["dq"], st, True), dk=_plain_turned(st["dk"], st, True))
    real = st["slots"] >= 0
    at = st["slots"][real]
    st["k_cache"][at] = _plain_turned(st["k"], st, False)[real]
    st["v_cache"][at] = st["v"][real]
    return dict(q=_plain_turned(st["q"], st, False), k_cache=st["k_cache"], v_cache=st["v_cache"])


def _exact_rope(case, seed):
    """Pairs as complex numbers, in 64 bits."""
    st = _rope_inputs(case, seed)
    rot = case["rot"]
    turn = torch.polar(torch.full((case["rows"], rot // 2), st["magnitude"], dtype=torch.float64, device="cuda"),
                       torch.outer(st["positions"].double(), st["freq"]))[:, None]

    def turned(x, by):
        x = x.double()
        z = x[..., :rot].unflatten(-1, (-1, 2) if case["interleaved"] else (2, -1))
        z = z if case["interleaved"] else z.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * by)
        z = z if case["interleaved"] else z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), x[..., rot:]], -1)

    if case["op"] == "rope":
        return dict(q=turned(st["q"], turn), k=turned(st["k"], turn), dq=turned(st["dq"], turn.conj()),
                    dk=turned(st["dk"], turn.conj()))
    k_cache, v_cache = st["k_cache"].double(), st["v_cache"].double()
    k = turned(st["k"], turn)
    rows = torch.nonzero(st["slots"] >= 0)[:, 0]
    k_cache.index_copy_(0, st["slots"][rows], k[rows])
    v_cache.index_copy_(0, st["slots"][rows], st["v"][rows].double())
    return dict(q=turned(st["q"], turn), k_cache=k_cache, v_cache=v_cache)


# ---------------------------------------------------------------------------------------------------------------
# the adapter layer's backward
# ---------------------------------------------------------------------------------------------------------------

def _keep_bits(seed, m, k, p):
    """The dropout mask, m x k truth values: Philox4x32-10 (Salmon et al., SC 2011) of key `seed` and counter (row,
    feature / 8, 0, 0), sixteen bits of its words a feature, low half first; kept from p * 2^16 on."""
    low = 0xFFFFFFFF
    t = torch.arange(m, device="cuda")[:, None].expand(m, -(-k // 8))
    g = torch.arange(-(-k // 8), device="cuda")[None].expand(m, -1)
    c = [t, g, torch.zeros_like(t), torch.zeros_like(t)]
    key = [seed & low, seed >> 32 & low]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57      # 64-bit products, their upper halves by shift and mask
        c = [(b >> 32 & low) ^ c[1] ^ key[0], b & low, (a >> 32 & low) ^ c[3] ^ key[1], a & low]
        key = [(key[0] + 0x9E3779B9) & low, (key[1] + 0xBB67AE85) & low]
    lanes = torch.stack([x >> s & 0xFFFF for x in c for s in (0, 16)], -1)
    return (lanes >= int(p * 65536 + 0.5)).view(m, -1)[:, :k]


def _lora_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    m, k, n, r, p = (case[x] for x in ("m", "k", "n", "r", "p"))

    def normal(rows, cols, size):
        return (torch.randn(rows, cols, device="cuda", generator=g) * size).bfloat16()

    x = _activations(m, k, g)
    st = dict(dy=normal(m, n, 1.0), w=normal(k, n, k ** -0.5), a=normal(k, r, k ** -0.5), b=normal(r, n, 0.02), alpha=2.0,
              p=p, seed=seed, k=k, keep=_keep_bits(seed, m, k, p) if p else None, bits=None)
    st["codes"], st["scales"] = _to_8_bits(x.float())
    kept = x.float() / (1 - p) * st["keep"] if p else x.float()
    st["s"] = (st["alpha"] * (kept @ st["a"].float())).bfloat16()      # what the forward saved
    if p:
        st["bits"] = (st["keep"].view(m, -1, 8) * 2 ** torch.arange(8, device="cuda")).sum(-1).to(torch.uint8)
    return st


def _plain_lora(st):
    x = _from_8_bits(st["codes"], st["scales"], st["k"])
    dy, q = st["dy"].float(), 1.0 / (1.0 - st["p"])
    if st["p"]:
        x = x * q * st["keep"]
    ds = st["alpha"] * (dy @ st["b"].float().T)
    branch = ds @ st["a"].float().T
    if st["p"]:
        branch = branch * q * st["keep"]
    return dict(dx=(dy @ st["w"].float().T + branch).bfloat16(), da=(x.T @ ds).bfloat16(),
                db=(st["s"].float().T @ dy).bfloat16())


def _exact_lora(case, seed):
    """64-bit products are slow on this card: only up to some size."""
    if case["m"] * case["k"] * case["n"] > 5e10:
        return None
    st = _lora_inputs(case, seed)
    size = torch.exp2(st["scales"].double() - 127).repeat_interleave(BLOCK, 1)[:, :case["k"]]
    x = st["codes"][:, :case["k"]].double() * size
    if case["p"]:
        x = torch.where(st["keep"], x / (1 - case["p"]), 0.0)
    dy, a, b, w = (st[name].double() for name in ("dy", "a", "b", "w"))
    da = torch.einsum("ti,tr->ir", x, st["alpha"] * torch.einsum("tj,rj->tr", dy, b))
    dx = torch.einsum("tj,rj,ir->ti", dy, b, a) * st["alpha"]
    if case["p"]:
        dx = torch.where(st["keep"], dx / (1 - case["p"]), 0.0)
    return dict(dx=dx + dy @ w.T, da=da, db=torch.einsum("tr,tj->rj", st["s"].double(), dy))


# ---------------------------------------------------------------------------------------------------------------
# what the tools call
# ---------------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    make = dict(norm=_norm_inputs, rope=_rope_inputs, append=_rope_inputs, act8=_act8_inputs, lora=_lora_inputs)
    st = make[case["op"]](case, seed)
    st.update(op=case["op"], mode=case.get("mode"))
    if own and case["op"] in ("rope", "append"):
        from lora_fine_tuning_gb300 import api
        st["table"] = api.rope_table(case["rot"], BASE, interleaved=case["interleaved"], **SCALING[case["scaling"]])
    elif own and case["op"] == "lora":
        from lora_fine_tuning_gb300 import api
        st["x8"] = api.Act8(st["codes"], st["scales"], case["k"])   # as the forward's norm or act8_store left it
    return st


def run(st):
    op, mode = st["op"], st["mode"]
    if not own:
        return dict(norm=_plain_norm, rope=_plain_rope, append=_plain_rope, act8=_plain_act8, lora=_plain_lora)[op](st)
    from lora_fine_tuning_gb300 import api
    if op == "rope":
        q, k = api.rope_fwd(st["q"], st["k"], st["positions"], st["table"])
        dq, dk = api.rope_bwd(st["dq"], st["dk"], st["positions"], st["table"])
        return dict(q=q, k=k, dq=dq, dk=dk)
    if op == "append":
        q = api.rope_append(st["q"], st["k"], st["v"], st["positions"], st["slots"], st["k_cache"], st["v_cache"],
                            st["table"])
        return dict(q=q, k_cache=st["k_cache"], v_cache=st["v_cache"])
    if op == "act8":
        return dict(x=api.act8_load(api.act8_store(st["x"])))
    if op == "lora":
        dx, da, db = api.lora_bwd(st["dy"], st["x8"], st["w"], st["a"], st["b"], st["s"], st["alpha"], st["p"],
                                  st["seed"], mask_bits=st["bits"])
        return dict(dx=dx, da=da, db=db)
    block = dict(y=st["y"], post_w=st["post_w"], gate=st["gate"], row_gate=st["row_gate"], res_scale=st["res_scale"],
                 eps=st["eps"], w_offset=st["offset"])
    out, h = {}, st["h"]
    if mode != "bwd":
        kept = {}
        if mode == "ckpt":
            kept = dict(x8=api.act8(*h.shape), h8=api.act8(*h.shape))
        x, h_out = api.norm_fwd(h, st["w"], **block, **kept)
        out.update(h_out=h_out, x=x)
        if mode == "fwd":
            return out
        out["x8"], h = api.act8_load(kept["x8"]), kept["h8"]
    g = api.norm_bwd(st["dx"], h, st["w"], dh=st["dh"], want_weights=st["weights"], **block)
    out.update(dh=g.dh)
    for name in ("dy", "dw", "dpost_w", "dgate", "drow_gate"):
        if getattr(g, name) is not None:
            out[name] = getattr(g, name)
    return out


def exact(case, seed):
    make = dict(norm=_exact_norm, rope=_exact_rope, append=_exact_rope, act8=_exact_act8, lora=_exact_lora)
    return make[case["op"]](case, seed)


def work(case):
    """Every input read once and every output written once; what is kept in 8 bits is written and read once."""
    op = case["op"]
    if op == "norm":
        values, kept = case["rows"] * case["width"], 1 + 1 / BLOCK
        stream, y = 2 if case["stream"] == "bf16" else 4, 2 if case["y"] else 0
        each = 0
        if case["mode"] != "bwd":
            each += stream + y + (stream if y else 0) + 2
        if case["mode"] == "ckpt":
            each += 4 * kept + 2                       # two written, one read by the backward, one returned
        if case["mode"] != "fwd":
            each += 2 + stream + stream + 2 * y        # dx, the gradient of the stream in and out, y and dy
            each += 0 if case["mode"] == "ckpt" else stream
        vectors = case["width"] * 4 * (1 + case["post"] + case["gate"]) * (2 if case["weights"] else 1)
        return dict(bytes=values * each + vectors, flops=values * (12 if case["mode"] == "fwd" else 40))
    if op == "rope":
        # Q and K, their gradients, and all of them turned
        values = case["rows"] * (case["hq"] + case["hkv"]) * case["d"]
        return dict(bytes=values * 8 + case["rows"] * 16, flops=values * 6)
    if op == "append":
        values = case["rows"] * (case["hq"] + 2 * case["hkv"]) * case["d"]
        return dict(bytes=values * 4 + case["rows"] * 16, flops=values * 3)
    if op == "act8":
        values = case["rows"] * case["width"]
        return dict(bytes=values * (4 + 2 * (1 + 1 / BLOCK)), flops=values * 6)
    m, k, n, r = (case[x] for x in ("m", "k", "n", "r"))
    nbytes = m * n * 2 + m * k * (2 + 1 + 1 / BLOCK) + (m * k // 8 if case["p"] else 0) + k * n * 2 + m * r * 2 + 4 * r * (k + n)
    return dict(bytes=nbytes, flops=2 * m * k * n + 2 * m * r * (2 * n + 2 * k))
