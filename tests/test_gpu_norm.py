"""Norms around a block against their formulas in 64 bits, and the gradients against difference quotients of the forward's.

Tolerances.  Forward, in fp32: a sum of squares has at most 16 values a thread and 13 levels of pairs, each rounded to 2^-24: 2e-6 of
itself, half of that in 1 / rms, whose root adds 2^-22; with the products about it everything before the outputs is within
E = 4e-6 of the sizes that were added or multiplied.  h' = h + c u: E (|h| + |c u|); x: E |W| (|h| + |c u|) / rms more than 4 E |x|.
Backward: t - n mean(t n) has the size |t| + |n| mean |t n|, and what follows multiplies or sums such sizes; the chain of two norms
doubles E.  A sum over rows adds 2^-24 of the sizes for each row that a thread adds and each group: at most 64 here, 4e-6.  An output in
bf16 is rounded, 2^-8 of itself, one in fp32 2^-24.
"""
import pytest

from tests.gpu_helpers import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from lora_fine_tuning_gb300 import api, native  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
E = 4e-6


def inputs(rows, width, stream=BF, y=True, w=True, post=False, gate=False, row_gate=False, vectors=BF, offset=0.0, seed=0, res=0.3):
    g = torch.Generator(device="cuda").manual_seed(seed + rows * 131 + width)

    def normal(*shape, size=1.0, mean=0.0):
        return torch.randn(*shape, device="cuda", generator=g) * size + mean

    scale = torch.exp(normal(rows, 1))       # rows of different sizes
    st = dict(h=(normal(rows, width) * scale).to(stream), w=normal(width, size=0.3, mean=1 - offset).to(vectors) if w else None,
              y=(normal(rows, width) * scale.flip(0)).to(BF) if y else None,
              post_w=normal(width, size=0.3, mean=1 - offset).to(vectors) if post else None,
              gate=normal(width, size=0.5).to(vectors) if gate else None, row_gate=normal(rows).to(vectors) if row_gate else None,
              res_scale=res, eps=1e-5, w_offset=offset)
    return st, normal(rows, width).to(BF) if w else None, normal(rows, width).to(stream)


def wide(t):
    return None if t is None else t.double()


def forward(st):
    """The forward in 64 bits: h', x, and what the backward needs."""
    h, y = st["h"].double(), wide(st["y"])
    rows, width = h.shape
    one = torch.ones((), dtype=torch.float64, device="cuda")
    W = None if st["w"] is None else st["w"].double() + st["w_offset"]
    P = one if st["post_w"] is None else st["post_w"].double() + st["w_offset"]
    C = st["res_scale"] * (one if st["gate"] is None else st["gate"].double()[None]) * \
        (one if st["row_gate"] is None else st["row_gate"].double()[:, None])
    size = h.abs()
    v = r2 = None
    if y is not None:
        r2 = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + st["eps"]) if st["post_w"] is not None else one
        v = y * r2
        size = size + (C * P * v).abs()
        h = h + C * P * v
    r = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + st["eps"])
    return dict(h=h, v=v, r2=r2, W=W, P=P, C=C, size=size, r=r, x=None if W is None else h * r * W)


def rounding(t, like):
    return t.abs() * (2.0 ** -8 if like == BF else 2.0 ** -24)


def close(got, want, tol):
    off = (got.double() - want).abs()
    return bool((off <= tol + rounding(want, got.dtype)).all())


def check_forward(st, **out):
    x, h_out = api.norm_fwd(**st, **out)
    f = forward(st)
    if st["y"] is None:
        assert h_out is st["h"]
    else:
        assert h_out.dtype == st["h"].dtype and close(h_out, f["h"], E * f["size"])
    if st["w"] is None:
        assert x is None
    else:
        assert x.dtype == BF and close(x, f["x"], E * (4 * f["x"].abs() + (f["W"] * f["r"] * f["size"]).abs()))
    return x, h_out


def check_backward(st, dx, dh, **more):
    """norm_bwd from the stream that the forward left (rounded as it is stored)."""
    after = dict(st)
    h = forward(st)["h"].to(st["h"].dtype)
    after.pop("h")
    g = api.norm_bwd(dx, h if st["w"] is not None else None, dh=dh, **after, **more)
    f = forward(st)
    W, P, C, v, r2 = (f[k] for k in ("W", "P", "C", "v", "r2"))
    d = torch.zeros_like(f["h"]) if dh is None else dh.double()
    size, n = d.abs(), None
    if W is not None:
        hs = h.double()
        r = 1 / torch.sqrt((hs * hs).mean(1, keepdim=True) + st["eps"])
        n, t = hs * r, dx.double() * W
        d = d + r * (t - n * (t * n).mean(1, keepdim=True))
        size = size + r * (t.abs() + n.abs() * (t * n).abs().mean(1, keepdim=True))
    assert g.dh.dtype == st["h"].dtype and close(g.dh, d, E * size)
    if st["w"] is not None:
        assert close(g.dw, (dx.double() * n).sum(0), 2 * E * (dx.double() * n).abs().sum(0))
    else:
        assert g.dw is None
    if v is None:
        assert g.dy is None
        return g
    rg = 1.0 if st["row_gate"] is None else st["row_gate"].double()[:, None]
    ga = 1.0 if st["gate"] is None else st["gate"].double()
    s = st["res_scale"]
    q, qs = C * P * d, (C * P).abs() * size
    if st["post_w"] is not None:
        want = r2 * (q - v * (q * v).mean(1, keepdim=True))
        tol = r2 * (qs + v.abs() * (qs * v.abs()).mean(1, keepdim=True))
    else:
        want, tol = q, qs
    assert close(g.dy, want, 2 * E * tol)
    for got, given, factor in ((g.dgate, st["gate"], s * P), (g.dpost_w, st["post_w"], s * ga)):
        if given is None:
            assert got is None
        else:
            assert got.dtype == F32 and close(got, (rg * d * v).sum(0) * factor, 3 * E * (rg * v * factor).abs().mul(size).sum(0))
    if st["row_gate"] is None:
        assert g.drow_gate is None
    else:
        assert close(g.drow_gate, (s * ga * P * d * v).sum(1), 3 * E * ((s * ga * P * v).abs() * size).sum(1))
    return g


FORMS = [dict(y=False), dict(), dict(post=True), dict(gate=True), dict(post=True, gate=True, offset=1.0, vectors=F32),
         dict(post=True, row_gate=True), dict(gate=True, row_gate=True, stream=F32), dict(post=True, gate=True, row_gate=True, stream=F32, vectors=F32),
         dict(w=False, post=True), dict(w=False), dict(stream=F32, offset=1.0, y=False)]


@pytest.mark.parametrize("form", range(len(FORMS)))
@pytest.mark.parametrize("rows,width", [(1, 64), (5, 1), (3, 7), (37, 264), (9, 1000), (70, 1025), (130, 2048), (33, 2050), (21, 4096),
                                        (11, 5000), (40, 8192), (6, 8200), (5, 16384), (3, 16383)])
def test_forms_and_widths(form, rows, width):
    st, dx, dh = inputs(rows, width, **FORMS[form])
    check_forward(st)
    check_backward(st, dx, dh)


@pytest.mark.parametrize("rows", [1, 2, 151, 152, 153, 607, 3001])
def test_rows(rows):
    """Sums over rows: more and fewer of them than groups."""
    for width in (96, 512, 1536, 4096):
        st, dx, dh = inputs(rows, width, post=True, gate=True)
        check_backward(st, dx, dh)


def test_without_a_gradient_of_the_stream_and_without_weights_gradients():
    st, dx, dh = inputs(50, 640, post=True, gate=True, row_gate=True)
    a = check_backward(st, dx, None)
    h = forward(st)["h"].bfloat16()
    rest = {k: x for k, x in st.items() if k != "h"}
    b = api.norm_bwd(dx, h, want_weights=False, **rest)
    assert torch.equal(a.dh, b.dh) and torch.equal(a.dy, b.dy)
    assert b.dw is None and b.dgate is None and b.dpost_w is None and b.drow_gate is None
    only = api.norm_bwd(dx, h, want_weights=False, dgate=torch.empty(640, device="cuda"), **rest)
    assert torch.equal(only.dgate, a.dgate) and only.dw is None


@pytest.mark.parametrize("stream", [BF, F32])
def test_gradients_against_differences(stream):
    """Along a direction, (L(p + e) - L(p - e)) / 2e of L = <x, dx> + <h', dh> in 64 bits, p all inputs one after the other.  The quotient's
    own error is e^2 of a third derivative, 1e-6 here, the gradients' 2^-8 (bf16) of their sizes."""
    st, dx, dh = inputs(6, 72, stream=stream, post=True, gate=True, row_gate=True, vectors=F32)
    st["h"] = st["h"].float().clamp(-2, 2).to(stream) + 0
    after = {k: x for k, x in st.items() if k != "h"}
    g = api.norm_bwd(dx, forward(st)["h"].to(stream), dh=dh, **after)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for name, grad in (("h", g.dh), ("y", g.dy), ("w", g.dw), ("post_w", g.dpost_w), ("gate", g.dgate), ("row_gate", g.drow_gate)):
        way = torch.randn(st[name].shape, device="cuda", generator=gen).double()

        def loss(step):
            f = forward({**st, name: st[name].double() + step * way})
            return (f["x"] * dx.double()).sum() + (f["h"] * dh.double()).sum()

        quotient = (loss(1e-4) - loss(-1e-4)) / 2e-4
        # bf16: h' is rounded where the backward reads it, the gradients where they are stored
        size = (grad.double() * way).abs().sum()
        assert float((quotient - (grad.double() * way).sum()).abs()) <= (2.0 ** -7 if stream == BF or name == "y" else 1e-5) * float(size) + 1e-5


@pytest.mark.parametrize("width,start,ld", [(96, 0, 104), (96, 8, 120), (96, 3, 101), (95, 0, 96)])
def test_rows_apart_and_in_place(width, start, ld):
    for stream in (BF, F32):
        st, dx, dh = inputs(25, width, stream=stream, post=True, gate=True)
        after = {k: x for k, x in st.items() if k != "h"}

        def apart(t):
            whole = torch.full((25, ld), 7.0, device="cuda").to(t.dtype)
            whole[:, start:start + width] = t
            return whole, whole[:, start:start + width]

        (hw, h), (yw, y), (xw, x) = apart(st["h"]), apart(st["y"]), apart(dx)
        # the same places in other buffers: rows that are read value by value are summed in another order than whole vectors
        want = check_forward({**st, "h": apart(st["h"])[1], "y": y})
        want_g = api.norm_bwd(apart(dx)[1], apart(want[1])[1], dh=apart(dh)[1], **{**after, "y": y})
        got = api.norm_fwd(**{**st, "h": h, "y": y}, h_out=h, x=x)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[1] is h
        (dxw, dxa), (dhw, dha), (dyw, dy) = apart(dx), apart(dh), apart(dx)
        got = api.norm_bwd(dxa, h, dh=dha, dh_out=dha, dy=dy, **{**after, "y": y})
        assert all(torch.equal(a, b) for a, b in zip(got, want_g) if b is not None)
        rest = torch.ones(ld, dtype=torch.bool, device="cuda")
        rest[start:start + width] = False
        for w in (hw, yw, xw, dxw, dhw, dyw):
            assert bool((w[:, rest] == 7).all())


@pytest.mark.parametrize("width", [128, 200, 97, 4096, 2050, 8192, 9000, 16381])
@pytest.mark.parametrize("stream", [BF, F32])
def test_what_is_kept_in_8_bits(width, stream):
    """The forward's codes are act8_store's, and the backward from codes is the backward from what they stand for."""
    rows = 19
    st, dx, dh = inputs(rows, width, stream=stream, post=True, gate=True)
    x8, h8, y8 = (api.act8(rows, width) for _ in range(3))
    for a in (x8, h8, y8):
        a.codes.fill_(77), a.scales.fill_(77)
    x, h = api.norm_fwd(**st, x8=x8, h8=h8, y8=y8)
    assert torch.equal(x, api.norm_fwd(**st)[0])
    for kept, t in ((x8, x), (h8, h.bfloat16()), (y8, st["y"])):
        want = api.act8_store(t)
        assert torch.equal(kept.codes, want.codes) and torch.equal(kept.scales, want.scales)
    after = {k: t for k, t in st.items() if k not in ("h", "y")}
    a = api.norm_bwd(dx, h8, dh=dh, y=y8, **after)
    b = api.norm_bwd(dx, api.act8_load(h8).to(stream), dh=dh, y=api.act8_load(y8), **after)
    assert all(torch.equal(p, q) for p, q in zip(a, b) if p is not None)
    bad = st["h"].clone()       # a row of NaN, and one that becomes infinite, spoil their own values only: padding stays zero
    bad[3], bad[4, 0] = float("nan"), float("inf")
    api.norm_fwd(**{**st, "h": bad}, x8=x8, h8=h8)
    x, h = api.norm_fwd(**{**st, "h": bad})
    for kept, t in ((x8, x), (h8, h.bfloat16())):
        want = api.act8_store(t)
        assert torch.equal(kept.codes, want.codes) and torch.equal(kept.scales, want.scales)
    only = api.act8(rows, width)
    norm = {**st, "y": None, "post_w": None, "gate": None}
    api.norm_fwd(**norm, x8=only)
    assert torch.equal(only.codes, api.act8_store(api.norm_fwd(**norm)[0]).codes)


@pytest.mark.parametrize("width", [40, 2048, 2050])
def test_rows_of_zeros_and_what_is_not_finite(width):
    st, dx, dh = inputs(8, width, post=True, gate=True)
    want, want_h = api.norm_fwd(**st)
    bad = {**st, "h": st["h"].clone(), "y": st["y"].clone()}
    bad["h"][1], bad["y"][1] = 0, 0
    bad["h"][3, 5], bad["y"][5, 7] = float("nan"), float("inf")
    x, h = api.norm_fwd(**bad)
    assert not x[1].any() and not h[1].any()
    keep = [0, 2, 4, 6, 7]
    assert torch.equal(x[keep], want[keep]) and torch.equal(h[keep], want_h[keep])
    assert bool(torch.isnan(x[3]).all()) and not torch.isfinite(x[5]).all()
    rest = {k: t for k, t in st.items() if k not in ("h", "y")}
    good = api.norm_bwd(dx, want_h, dh=dh, y=st["y"], **rest)
    g = api.norm_bwd(dx, h, dh=dh, y=bad["y"], **rest)
    assert torch.equal(g.dh[keep], good.dh[keep]) and torch.equal(g.dy[keep], good.dy[keep])
    assert bool(torch.isfinite(g.dh[1]).all()) and bool(torch.isfinite(g.dy[1]).all())


@pytest.mark.parametrize("size", [1e19, 1e25, 1e37])
@pytest.mark.parametrize("width", [64, 2050, 4096])
def test_squares_past_fp32(size, width):
    """A row's norm does not depend on its size, up to values whose squares no fp32 holds: with eps far below, n(s v) = n(v)."""
    st, dx, dh = inputs(5, width, y=True, post=True, res=1.0)
    for name in ("h", "y"):
        st[name] = (st[name].float().clamp(-4, 4) * 2.0 ** round(torch.tensor(size).log2().item())).bfloat16()
    x, h = check_forward(st)
    f = forward(st)
    after = {k: t for k, t in st.items() if k != "h"}
    g = api.norm_bwd(dx, h, **after)
    hs = h.double()
    r = 1 / torch.sqrt((hs * hs).mean(1, keepdim=True))
    n, t = hs * r, dx.double() * f["W"]
    want = r * (t - n * (t * n).mean(1, keepdim=True))
    # results below fp32's smallest normal number have steps of 2^-149 or, in bf16, 2^-133
    tol = E * r * (t.abs() + n.abs() * (t * n).abs().mean(1, keepdim=True)) + 2.0 ** -133
    assert bool(((g.dh.double() - want).abs() <= tol + 2.0 ** -8 * want.abs()).all())
    assert close(g.dw, (dx.double() * n).sum(0), 2 * E * (dx.double() * n).abs().sum(0))


def test_the_same_from_call_to_call_on_another_stream_and_with_a_workspace():
    st, dx, dh = inputs(3000, 1024, post=True, gate=True, row_gate=True)
    _, h = api.norm_fwd(**st)
    rest = {k: t for k, t in st.items() if k != "h"}
    want = api.norm_bwd(dx, h, dh=dh, **rest)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.full((api.norm_workspace_size(3000, 1024),), 255, dtype=torch.uint8, device="cuda")
    for got in (api.norm_bwd(dx, h, dh=dh, **rest), api.norm_bwd(dx, h, dh=dh, stream=s, **rest), api.norm_bwd(dx, h, dh=dh, ws=ws, **rest)):
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_two_graphs_and_calls_between():
    calls = []
    for seed, rows in ((0, 400), (1, 300)):
        st, dx, dh = inputs(rows, 1024, post=True, gate=True, seed=seed)
        rest = {k: t for k, t in st.items() if k != "h"}
        h = api.norm_fwd(**st)[1]
        calls.append(lambda st=st, dx=dx, dh=dh, rest=rest, h=h: [*api.norm_fwd(**st), *(t for t in api.norm_bwd(dx, h, dh=dh, **rest) if t is not None)])
    want = [[t.clone() for t in f()] for f in calls]
    graphs, outs = [], []
    for f in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    big, dx, dh = inputs(9000, 4096, post=True)
    api.norm_bwd(dx, big["h"], dh=dh, **{k: t for k, t in big.items() if k != "h"})      # a larger workspace outside them
    for order in ((1, 0), (0, 1, 1, 0)):
        for i in order:
            for t in outs[i]:
                t.fill_(7)
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in order:
            assert all(torch.equal(a, b) for a, b in zip(want[i], outs[i]))


def test_two_threads_on_one_stream():
    """The launches of two threads' calls may interleave on the stream: each thread's calls have a workspace of their own."""
    import threading
    calls = []
    for seed, rows in ((0, 900), (1, 700)):
        st, dx, dh = inputs(rows, 768, post=True, gate=True, seed=seed)
        h = api.norm_fwd(**st)[1]
        calls.append(lambda dx=dx, h=h, dh=dh, rest={k: t for k, t in st.items() if k != "h"}: api.norm_bwd(dx, h, dh=dh, **rest))
    want, wrong = [f() for f in calls], []
    torch.cuda.synchronize()

    def work(i):
        for _ in range(200):
            got = calls[i]()
            torch.cuda.current_stream().synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[i]) if b is not None):
                wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_no_rows():
    st, dx, dh = inputs(0, 256, post=True, gate=True, row_gate=True)
    x, h = api.norm_fwd(**st)
    assert x.shape == h.shape == (0, 256)
    g = api.norm_bwd(dx, h, dh=dh, **{k: t for k, t in st.items() if k != "h"})
    assert g.dy.shape == (0, 256) and not g.dw.any() and not g.dgate.any() and not g.dpost_w.any() and g.drow_gate.shape == (0,)


def test_offsets_past_32_bits():
    buffer = torch.empty((1 << 31) + 4096, dtype=BF, device="cuda")
    st, dx, dh = inputs(3, 1000, post=True)
    want = api.norm_fwd(**st)
    far = buffer.as_strided((3, 1000), (1 << 30, 1))
    far.copy_(st["h"])
    got = api.norm_fwd(**{**st, "h": far}, h_out=far)
    assert torch.equal(got[0], want[0]) and torch.equal(far, want[1])


def test_refusals():
    st, dx, dh = inputs(4, 64, post=True, gate=True, row_gate=True)
    h = st["h"]
    for change in (dict(w=st["w"][:63]), dict(post_w=st["post_w"].half()), dict(gate=h), dict(row_gate=st["row_gate"][:3]), dict(y=st["y"][:3]),
                   dict(h=h.t()), dict(x8=api.act8(4, 96))):
        with pytest.raises((ValueError, TypeError)):
            api.norm_fwd(**{**st, **change})
    with pytest.raises(TypeError):
        api.norm_fwd(**{**st, "y": st["y"].float()})
    with pytest.raises(TypeError):
        api.norm_fwd(**{**st, "h": h.half()})
    for change in (dict(eps=0.0), dict(eps=float("nan")), dict(res_scale=float("inf")), dict(y=None), dict(w=None, x=torch.empty_like(h))):
        with pytest.raises(native.LoraError):
            api.norm_fwd(**{**st, **change})
    with pytest.raises(native.LoraError):
        api.norm_fwd(h, None)
    rest = {k: t for k, t in st.items() if k != "h"}
    with pytest.raises(ValueError):
        api.norm_bwd(None, None, **rest)
    with pytest.raises(TypeError):
        api.norm_bwd(dx, h, dh=dh.float(), **rest)
    for change in (dict(w=None), dict(post_w=None, dpost_w=torch.empty(64, device="cuda")), dict(dh_out=dh, dh=dh, dy=dh),
                   dict(ws=torch.zeros(512, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(native.LoraError):
            api.norm_bwd(dx, h, **{**rest, **change})


@pytest.mark.parametrize("width", [96, 97, 4096])
@pytest.mark.parametrize("stream", [BF, F32])
def test_stream_type_from_8_bits_alone(width, stream):
    """A stream kept in 8 bits without a gradient of its own, as the last norm of a decoder has it: dh_out gives the stream's type."""
    st, dx, dh = inputs(12, width, stream=stream, post=True)
    h8 = api.act8_store(st["h"].bfloat16())
    rest = {k: t for k, t in st.items() if k != "h"}
    want = api.norm_bwd(dx, h8, dh=torch.zeros_like(dh), **rest)
    got = api.norm_bwd(dx, h8, dh_out=torch.empty_like(dh), **rest)
    assert got.dh.dtype == stream and all(torch.equal(a, b) for a, b in zip(got, want) if b is not None)
    assert api.norm_bwd(dx, h8, **rest).dh.dtype == BF
