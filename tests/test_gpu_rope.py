"""Rotary positions and rows into a cache, against complex products in 64 bits.

Tolerance: sines and cosines are off by 2e-7 (angles exact to 2^-26 of a turn, sincospi to 2 steps of fp32, the magnitude's product
one), a pair's two products and their sum by three fp32 roundings of at most |a| + |b|: 1e-6 m (|a| + |b|) in all, and the result is
rounded to bf16, 2^-8 of itself.
"""
import math

import pytest

from tests.gpu_helpers import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from lora_fine_tuning_gb300 import api, native  # noqa: E402


def frequencies(rot, base=10000.0, scaling=None, factor=1.0, original=0.0, low=1.0, high=32.0, **_):
    if scaling == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "parts":
            keep = min(1.0, max(0.0, (original * f / (2 * math.pi) - low) / (high - low)))
            f = f * keep + f / factor * (1 - keep)
        out.append(f)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def turned(x, positions, rot, interleaved, back, magnitude=1.0, **how):
    """(result, tolerance) in 64 bits."""
    x = x.double()
    angle = torch.outer(positions.double(), frequencies(rot, **how))
    by = torch.polar(torch.full_like(angle, magnitude), -angle if back else angle)[:, None]
    z = x[..., :rot].unflatten(-1, (-1, 2) if interleaved else (2, -1))
    z = z if interleaved else z.transpose(-1, -2)
    size = z.abs().sum(-1, keepdim=True).expand_as(z)
    z = torch.view_as_real(torch.complex(z[..., 0], z[..., 1]) * by)
    if not interleaved:
        z, size = z.transpose(-1, -2), size.transpose(-1, -2)
    want = torch.cat([z.flatten(-2), x[..., rot:]], -1)
    size = torch.cat([size.flatten(-2), torch.zeros_like(x[..., rot:])], -1)
    return want, 2.0 ** -8 * want.abs() + 1e-6 * abs(magnitude) * size


def near(got, want):
    want, tol = want
    return bool(((got.double() - want).abs() <= tol).all())


def heads(rows, h, d, g):
    return torch.randn(rows, h, d, device="cuda", generator=g).bfloat16()


CASES = [  # rows, hq, hkv, d, rot, interleaved
    (1, 1, 1, 2, 2, False), (1, 32, 8, 128, 128, False), (3, 32, 8, 128, 128, True), (9, 6, 2, 64, 64, False),
    (17, 4, 4, 40, 40, False), (5, 3, 1, 40, 20, True), (11, 7, 1, 96, 48, False), (8, 2, 2, 96, 24, True), (6, 4, 2, 40, 10, False),
    (4, 2, 1, 36, 18, True), (4, 2, 1, 37, 6, False), (3, 1, 1, 5, 4, True), (2, 2, 1, 256, 256, False), (700, 16, 2, 128, 64, False),
    (5000, 2, 1, 64, 64, True), (257, 64, 8, 128, 128, False)]


@pytest.mark.parametrize("rows,hq,hkv,d,rot,inter", CASES)
def test_forward_and_backward(rows, hq, hkv, d, rot, inter):
    g = torch.Generator(device="cuda").manual_seed(rows * d + rot)
    q, k, dq, dk = heads(rows, hq, d, g), heads(rows, hkv, d, g), heads(rows, hq, d, g), heads(rows, hkv, d, g)
    t = torch.randint(0, 5000, (rows,), device="cuda", generator=g)
    rope = api.rope_table(rot, 500000.0, interleaved=inter)
    how = dict(rot=rot, interleaved=inter, base=500000.0)
    for x, out in zip((q, k), api.rope_fwd(q, k, t, rope)):
        assert near(out, turned(x, t, back=False, **how))
    for x, out in zip((dq, dk), api.rope_bwd(dq, dk, t, rope)):
        assert near(out, turned(x, t, back=True, **how))
    q1, none = api.rope_fwd(q, None, t.int(), rope)
    none2, k1 = api.rope_fwd(None, k, t.int(), rope)
    both = api.rope_fwd(q, k, t, rope)
    assert none is None and none2 is None and torch.equal(q1, both[0]) and torch.equal(k1, both[1])


def test_the_gradient_is_the_transposed_map():
    """<turned q, dq> = <q, turned back dq>, and the difference quotient of a linear map is the map."""
    g = torch.Generator(device="cuda").manual_seed(1)
    q, d = heads(50, 4, 64, g), heads(50, 4, 64, g)
    t = torch.randint(0, 100000, (50,), device="cuda", generator=g)
    rope = api.rope_table(64, scaling="linear", factor=3.0, magnitude=1.25)
    out, back = api.rope_fwd(q, None, t, rope)[0], api.rope_bwd(d, None, t, rope)[0]
    a, b = (out.double() * d.double()).sum(), (q.double() * back.double()).sum()
    size = (out.double() * d.double()).abs().sum() + (q.double() * back.double()).abs().sum()
    assert float((a - b).abs()) <= 2.0 ** -8 * float(size)     # each product has one rounded factor
    step = api.rope_fwd((q.float() + 2.0 ** -2 * d.float()).bfloat16(), None, t, rope)[0]
    moved = (q.float() + 2.0 ** -2 * d.float()).bfloat16().double() - q.double()
    want, _ = turned(moved, t, 64, False, False, 1.25, scaling="linear", factor=3.0)
    pair = (out.double().abs() + step.double().abs()) * 2.0 ** -8 + 1e-5 * (q.double().abs().amax() + 1)
    assert bool(((step.double() - out.double() - want).abs() <= pair).all())


@pytest.mark.parametrize("how", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
                                 dict(scaling="parts", factor=32.0, original=8192, low=1.0, high=32.0, magnitude=1.3466),
                                 dict(scaling="parts", factor=8.0, original=8192, low=1.0, high=4.0)])
def test_far_positions_and_scalings(how):
    g = torch.Generator(device="cuda").manual_seed(3)
    t = torch.tensor([0, 1, 2, 1000003, 2 ** 24 + 1, 2 ** 30, -1, -12345], device="cuda")
    q = heads(8, 2, 128, g)
    for inter in (False, True):
        rope = api.rope_table(128, 500000.0, interleaved=inter, **how)
        want, tol = turned(q, t, 128, inter, False, base=500000.0, **how)
        # the reference's own angles, up to 2^30, are off by 2^-51 of themselves (a power and two products), times |a| + |b| < 12
        tol = tol + 2.0 ** -17 * (t.double().abs() / 2 ** 30)[:, None, None]
        assert bool(((api.rope_fwd(q, None, t, rope)[0].double() - want).abs() <= tol).all())


def test_turns_are_whole_at_whole_turns():
    """A frequency of 2 pi / 64 comes back to the start every 64 positions, however far."""
    rope = api.rope_table(2)
    rope.table.turn[0] = 1 << 58
    g = torch.Generator(device="cuda").manual_seed(4)
    q = heads(6, 1, 2, g)
    t = torch.tensor([0, 64, 2 ** 40, -64, 2 ** 62, -2 ** 63], device="cuda")
    assert torch.equal(api.rope_fwd(q, None, t, rope)[0], q)


def test_fused_projection_in_place_and_padding_around_heads():
    g = torch.Generator(device="cuda").manual_seed(5)
    for d, rot in ((64, 64), (64, 32), (40, 10)):
        qkv = heads(33, 10, d, g)
        q, k, v = qkv[:, :6], qkv[:, 6:8], qkv[:, 8:]
        t = torch.randint(0, 9000, (33,), device="cuda", generator=g)
        rope = api.rope_table(rot)
        want = api.rope_fwd(q.contiguous(), k.contiguous(), t, rope)
        kept = v.clone()
        assert all(torch.equal(a, b) for a, b in zip(want, api.rope_fwd(q, k, t, rope)))
        api.rope_fwd(q, k, t, rope, Q_out=q, K_out=k)
        assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, kept)
        by_head = torch.empty(4, 33, d, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
        by_head.copy_(heads(33, 4, d, g))
        out = torch.full((33, 4, d + 3), 7.0, device="cuda").bfloat16()
        api.rope_fwd(by_head, None, t, rope, Q_out=out[:, :, :d])
        assert torch.equal(out[:, :, :d], api.rope_fwd(by_head.contiguous(), None, t, rope)[0]) and bool((out[:, :, d:] == 7).all())


@pytest.mark.parametrize("rows,hq,hkv,d,rot,inter,page", [(1, 32, 8, 128, 128, False, 16), (64, 32, 8, 128, 128, False, 16),
                                                         (7, 3, 1, 40, 20, True, 1), (500, 8, 2, 64, 32, False, 64), (33, 4, 4, 37, 6, True, 5)])
def test_rows_into_a_cache(rows, hq, hkv, d, rot, inter, page):
    g = torch.Generator(device="cuda").manual_seed(rows)
    qkv = heads(rows, hq + 2 * hkv, d, g)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    n = page * (rows // page + 3)
    kc, vc = heads(n, hkv, d, g), heads(n, hkv, d, g)
    slots = torch.randperm(n, device="cuda", generator=g)[:rows].contiguous()
    for i, bad in enumerate((-1, n, -2 ** 63, 2 ** 62)):
        if 3 * i + 2 < rows:
            slots[3 * i + 2] = bad
    t = torch.randint(0, 200000, (rows,), device="cuda", generator=g)
    rope = api.rope_table(rot, interleaved=inter)
    want_q, want_k = api.rope_fwd(q, k, t, rope)
    want_kc, want_vc = kc.clone(), vc.clone()
    real = (slots >= 0) & (slots < n)
    want_kc[slots[real]], want_vc[slots[real]] = want_k[real], v[real]
    got = api.rope_append(q, k, v, t, slots, kc, vc, rope)
    assert torch.equal(got, want_q) and torch.equal(kc, want_kc) and torch.equal(vc, want_vc)
    # caches head by head, and the turned queries in place
    kh, vh = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (want_kc, want_vc))
    api.rope_append(q, k, v, t, slots, kh, vh, rope, Q_out=q)
    assert torch.equal(q, want_q) and torch.equal(kh, want_kc) and torch.equal(vh, want_vc)


def test_rows_with_one_slot():
    """Of two rows with one slot something of either is left there, and everything else is right."""
    g = torch.Generator(device="cuda").manual_seed(10)
    q, k, v = heads(40, 4, 64, g), heads(40, 2, 64, g), heads(40, 2, 64, g)
    kc, vc = heads(60, 2, 64, g), heads(60, 2, 64, g)
    slots = torch.arange(40, device="cuda") + 10
    slots[30] = slots[5]
    t, rope = torch.arange(40, device="cuda"), api.rope_table(64)
    before = vc.clone()
    out, want = api.rope_append(q, k, v, t, slots, kc, vc, rope), api.rope_fwd(q, k, t, rope)
    rest = [i for i in range(40) if i not in (5, 30)]
    assert torch.equal(out, want[0]) and torch.equal(kc[slots[rest]], want[1][rest]) and torch.equal(vc[slots[rest]], v[rest])
    assert bool(((vc[15] == v[5]) | (vc[15] == v[30])).all()) and bool(((kc[15] == want[1][5]) | (kc[15] == want[1][30])).all())
    untouched = [i for i in range(60) if i < 10 or i == 40 or i >= 50]
    assert torch.equal(vc[untouched], before[untouched])


def test_an_empty_cache_and_no_rows():
    g = torch.Generator(device="cuda").manual_seed(6)
    q, k = heads(3, 4, 64, g), heads(3, 2, 64, g)
    rope, t = api.rope_table(64), torch.arange(3, device="cuda")
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(api.rope_append(q, k, k, t, t, none, none.clone(), rope), api.rope_fwd(q, None, t, rope)[0])
    assert api.rope_fwd(q[:0], k[:0], t[:0], rope)[0].shape == (0, 4, 64)
    cache = [heads(5, 2, 64, g) for _ in range(2)]
    assert api.rope_append(q[:0], k[:0], k[:0], t[:0], t[:0], *cache, rope).shape == (0, 4, 64)


def test_a_cache_past_32_bits():
    """Rows whose places lie beyond 2^32 bytes."""
    g = torch.Generator(device="cuda").manual_seed(7)
    q, k, v = heads(4, 2, 64, g), heads(4, 1, 64, g), heads(4, 1, 64, g)
    n = (1 << 32) // 64 // 2 + 1000
    kc, vc = (torch.zeros(n, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.tensor([n - 1, 0, n - 900, 5], device="cuda")
    t = torch.arange(4, device="cuda")
    api.rope_append(q, k, v, t, slots, kc, vc, api.rope_table(64))
    assert torch.equal(kc[slots], api.rope_fwd(None, k, t, api.rope_table(64))[1]) and torch.equal(vc[slots], v)
    assert int(kc.count_nonzero(dim=(1, 2)).count_nonzero()) == 4


def test_another_stream_and_a_graph():
    g = torch.Generator(device="cuda").manual_seed(8)
    q, k = heads(64, 8, 64, g), heads(64, 2, 64, g)
    t, rope = torch.arange(64, device="cuda"), api.rope_table(64)
    want = api.rope_fwd(q, k, t, rope)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = api.rope_fwd(q, k, t, rope, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    kc, vc, slots = heads(100, 2, 64, g), heads(100, 2, 64, g), torch.arange(64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = api.rope_append(q, k, k, t, slots, kc, vc, rope)
    t += 100
    slots += 30
    graph.replay()
    want = api.rope_fwd(q, k, t, rope)
    assert torch.equal(out, want[0]) and torch.equal(kc[30:94], want[1]) and torch.equal(vc[30:94], k)


def test_refusals():
    g = torch.Generator(device="cuda").manual_seed(9)
    q, k = heads(6, 4, 64, g), heads(6, 2, 64, g)
    t, rope = torch.arange(6, device="cuda"), api.rope_table(64)
    for call in (lambda: api.rope_fwd(q, k, t[:5], rope), lambda: api.rope_fwd(q, k, t.float(), rope),
                 lambda: api.rope_fwd(q, k[:5], t, rope), lambda: api.rope_fwd(q, k, t, rope, Q_out=q[:, :2]),
                 lambda: api.rope_append(q, k, k, t, t.int(), k, k, rope), lambda: api.rope_table(64, scaling="other")):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        api.rope_fwd(q.float(), k, t, rope)
    for call in (lambda: api.rope_fwd(q, k, t, api.rope_table(128)), lambda: api.rope_table(63), lambda: api.rope_table(0),
                 lambda: api.rope_table(258), lambda: api.rope_table(64, -1.0),
                 lambda: api.rope_append(q, k, k, t, t, k, k.clone(), rope), lambda: api.rope_table(64, scaling="linear", factor=0.0)):
        with pytest.raises(native.LoraError):
            call()
