"""Norms, rotary positions, cache rows and 8 bits through the C ABI without a GPU: every refusal is made before any CUDA call, with the code the
header gives, and the host-only table of frequencies.  No call here launches a kernel."""
import ctypes
import math
import os
from fractions import Fraction

import pytest

from lora_fine_tuning_gb300 import native


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(native.LIB_PATH):
        from lora_fine_tuning_gb300 import build
        build.build()
    return native.lib()


NAN, INF = float("nan"), float("inf")


def kept(codes=256, scales=256):
    return ctypes.byref(native.Act8(codes, scales))


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 3), (dict(rows=262145), 3), (dict(width=0), 3), (dict(width=(1 << 22) + 1, ld=1 << 23), 3), (dict(ld=99), 3), (dict(ld=1 << 38), 3),
    (dict(rows=262144, width=1 << 17, ld=1 << 17), 3), (dict(x=None), 1), (dict(x=257), 2), (dict(a=kept(codes=None)), 1),
    (dict(a=kept(scales=None)), 1), (dict(a=kept(codes=264)), 2), (dict(a=kept(scales=258)), 2), (dict(a=None), 1)])
def test_act8(lib, kw, code):
    v = dict(x=256, rows=10, width=100, ld=100, a=kept())
    v.update(kw)
    assert lib.act8_store(v["x"], v["rows"], v["width"], v["ld"], v["a"], None) == code
    assert lib.act8_load(v["a"], v["rows"], v["width"], v["x"], v["ld"], None) == code


def norm(rows=10, width=96, w=(256, 0), post=(None, 0), gate=(None, 0), row_gate=(None, 0), eps=1e-5, offset=0.0, res=1.0, stream=0, **ld):
    n = native.Norm(rows, width, *(ld.get(x, 96) for x in ("h", "y", "h_out", "x", "dx", "dh", "dh_out", "dy")))
    n.w, n.post_w, n.gate, n.row_gate = (native.Vector(p, t, 0) for p, t in (w, post, gate, row_gate))
    n.eps, n.w_offset, n.res_scale, n.stream_dtype = eps, offset, res, stream
    return ctypes.byref(n)


def fwd(lib, n, h=256, y=512, h_out=1024, x=2048, x8=None, h8=None, y8=None):
    return lib.norm_fwd(n, h, y, h_out, x, x8, h8, y8, None)


def bwd(lib, n, dx=256, dh=512, h=1024, h8=None, y=2048, y8=None, dh_out=4096, dy=8192, dw=None, dpost=None, dgate=None, drow=None, ws=256,
        ws_bytes=1 << 30):
    return lib.norm_bwd(n, dx, dh, h, h8, y, y8, dh_out, dy, dw, dpost, dgate, drow, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 3), (dict(rows=262145), 3), (dict(width=0), 3), (dict(width=16385, **{k: 20000 for k in ("h", "y", "h_out", "x")}), 3),
    (dict(stream=2), 1), (dict(eps=0.0), 1), (dict(eps=NAN), 1), (dict(eps=INF), 1), (dict(offset=NAN), 1), (dict(res=INF), 1), (dict(w=(256, 2)), 1),
    (dict(post=(256, -1)), 1), (dict(gate=(256, 7)), 1), (dict(row_gate=(256, 2)), 1), (dict(w=(257, 0)), 2), (dict(w=(258, 1)), 2),
    (dict(row_gate=(258, 1)), 2)])
def test_norm_shapes(lib, kw, code):
    assert fwd(lib, norm(**kw)) == code
    assert bwd(lib, norm(**kw)) == code


def test_norm_strides(lib):
    for name in ("h", "y", "h_out", "x"):
        assert fwd(lib, norm(**{name: 95})) == 3 and fwd(lib, norm(**{name: 1 << 38})) == 3
    for name in ("dx", "dh", "h", "y", "dh_out", "dy"):
        assert bwd(lib, norm(**{name: 95})) == 3


def test_norm_matrices(lib):
    for kw, code in ((dict(h=None), 1), (dict(h_out=None), 1), (dict(x=None), 1), (dict(h=257), 2), (dict(y=513), 2), (dict(h_out=1025), 2), (dict(x=2049), 2),
                     (dict(y=None), 1), (dict(y=None, h_out=None, y8=kept()), 1), (dict(x8=kept(codes=None)), 1), (dict(h8=kept(codes=264)), 2),
                     (dict(y8=kept(scales=258)), 2)):
        assert fwd(lib, norm(), **kw) == code, kw
    assert fwd(lib, norm(stream=1), h=258) == 2
    assert fwd(lib, norm(post=(256, 0)), y=None, h_out=None) == 1
    assert fwd(lib, norm(w=(None, 0))) == 1                                       # x without its weights
    assert fwd(lib, norm(w=(None, 0)), y=None, h_out=None, x=None) == 1           # nothing to do
    assert fwd(lib, norm(h_out=104), h_out=256) == 1                              # in place with another stride
    for kw, code in ((dict(dx=None), 1), (dict(h=None), 1), (dict(dh_out=None), 1), (dict(h8=kept()), 1), (dict(y8=kept()), 1), (dict(y=None), 1),
                     (dict(dx=257), 2), (dict(dh=513), 2), (dict(dy=8193), 2), (dict(dpost=256), 1), (dict(dgate=256), 1), (dict(drow=256), 1),
                     (dict(dw=258), 2), (dict(dy=4096), 1), (dict(dy=512), 1), (dict(dw=256, ws=None), 6), (dict(dw=256, ws=272), 6),
                     (dict(dw=256, ws_bytes=256), 6)):
        assert bwd(lib, norm(), **kw) == code, kw
    assert bwd(lib, norm(w=(None, 0))) == 1 and bwd(lib, norm(w=(None, 0)), dx=None, h=None, dw=256) == 1
    assert bwd(lib, norm(dh_out=104), dh_out=512) == 1
    assert lib.norm_fwd(None, 256, 256, 256, 256, None, None, None, None) == 1
    assert lib.norm_workspace_size(-1, 64) == 0 and lib.norm_workspace_size(10, 0) == 0 and lib.norm_workspace_size(10, 16385) == 0
    a, b = lib.norm_workspace_size(1, 64), lib.norm_workspace_size(262144, 16384)
    assert 256 < a < b < 64 << 20 and a % 256 == b % 256 == 0


def table(rot=64, base=10000.0, inter=0, **s):
    out = native.Rope()
    scaling = native.RopeScaling(s.get("kind", 0), s.get("magnitude", 1.0), s.get("factor", 1.0), s.get("original", 0.0), s.get("low", 1.0), s.get("high", 32.0))
    return native.lib().rope_table(rot, base, inter, ctypes.byref(scaling), ctypes.byref(out)), out


@pytest.mark.parametrize("kw,code", [
    (dict(rot=0), 3), (dict(rot=63), 3), (dict(rot=258), 3), (dict(base=0.0), 1), (dict(base=-2.0), 1), (dict(base=NAN), 1), (dict(base=INF), 1), (dict(inter=2), 1),
    (dict(kind=4), 1), (dict(kind=-1), 1), (dict(magnitude=NAN), 1), (dict(kind=1, factor=0.0), 1), (dict(kind=1, factor=NAN), 1),
    (dict(kind=3, original=0.0), 1), (dict(kind=3, original=100.0, low=2.0, high=2.0), 1)])
def test_table_refusals(lib, kw, code):
    assert table(**kw)[0] == code


def test_table_pointers(lib):
    assert lib.rope_table(64, 10000.0, 0, None, None) == 1
    out = native.Rope()
    assert lib.rope_table(64, 10000.0, 1, None, ctypes.byref(out)) == 0
    assert (out.rot_dim, out.interleaved, out.magnitude) == (64, 1, 1.0)


PI = Fraction(3141592653589793238462643383279502884197169399375105820974944592307816406286, 10 ** 75)


@pytest.mark.parametrize("rot,base,kw", [(2, 10000.0, {}), (64, 10000.0, {}), (128, 500000.0, {}), (256, 1e7, {}), (40, 1.0, {}), (6, 0.5, {}), (128, 1e30, {}),
                                         (64, 10000.0, dict(kind=1, factor=4.0)), (64, 10000.0, dict(kind=2, factor=8.0)),
                                         (128, 500000.0, dict(kind=3, factor=32.0, original=8192.0, magnitude=1.5)),
                                         (128, 500000.0, dict(kind=3, factor=8.0, original=8192.0, low=1.0, high=4.0))])
def test_turns(lib, rot, base, kw):
    """Frequencies by the definition in doubles; their turns are those doubles over 2 pi, modulo one, to the nearest 2^-64 (pow's last bit may
    differ between libraries: one in 2^52 of the frequency)."""
    st, got = table(rot, base, **kw)
    assert st == 0
    b = base * kw["factor"] ** (rot / (rot - 2)) if kw.get("kind") == 2 and rot > 2 else base
    for i in range(rot // 2):
        f = math.pow(b, -2.0 * i / rot)
        if kw.get("kind") == 1:
            f /= kw["factor"]
        if kw.get("kind") == 3:
            keep = min(1.0, max(0.0, (kw["original"] * f / (2 * math.pi) - kw.get("low", 1.0)) / (kw.get("high", 32.0) - kw.get("low", 1.0))))
            f = f * keep + f / kw["factor"] * (1 - keep)
        turns = Fraction(f) / (2 * PI)
        want = round(turns * 2 ** 64) % 2 ** 64
        off = (got.turn[i] - want + 2 ** 63) % 2 ** 64 - 2 ** 63
        assert abs(off) <= 1 + 8 * float(turns) * 2 ** 12, (i, off)
    assert all(got.turn[i] == 0 for i in range(rot // 2, 128))


def rope_shape(rows=10, cache=100, hq=8, hk=2, d=64, bits=64, **s):
    g = native.RopeShape(rows, cache, hq, hk, d, bits)
    for f in ("q", "k", "v", "q_out", "k_out", "v_out"):
        m = getattr(g, f)
        m.row, m.head = s.get(f, ((hq if f.startswith("q") else hk) * d, d))
    return ctypes.byref(g)


def turn(lib, g, r, q=256, k=512, pos=256, qo=1024, ko=2048):
    return [f(q, k, pos, g, r, qo, ko, None) for f in (lib.rope_fwd, lib.rope_bwd)]


def append(lib, g, r, q=256, k=512, v=768, pos=256, slots=256, qo=1024, kc=2048, vc=4096):
    return lib.rope_append(q, k, v, pos, slots, g, r, qo, kc, vc, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 3), (dict(rows=262145), 3), (dict(hq=-1), 3), (dict(hq=1025), 3), (dict(hk=1025), 3), (dict(d=0), 3), (dict(d=257), 3), (dict(d=62), 3),
    (dict(bits=16), 1), (dict(q=(511, 64)), 3), (dict(k=(64, 64)), 3), (dict(q_out=(512, 63)), 3), (dict(k_out=(0, 64)), 3), (dict(q=(-512, 64)), 3),
    (dict(q=(1 << 38, 64)), 3)])
def test_rope_shapes(lib, kw, code):
    r = ctypes.byref(table()[1])
    assert turn(lib, rope_shape(**kw), r) == [code, code]
    assert append(lib, rope_shape(**kw), r) == code


def test_rope_pointers(lib):
    r, g = ctypes.byref(table()[1]), rope_shape()
    for kw, code in ((dict(q=None), 1), (dict(k=None), 1), (dict(pos=None), 1), (dict(qo=None), 1), (dict(ko=None), 1), (dict(q=257), 2), (dict(ko=2049), 2),
                     (dict(pos=260), 2)):
        assert turn(lib, g, r, **kw) == [code, code], kw
    assert turn(lib, rope_shape(q_out=(600, 64)), r, qo=256) == [1, 1]            # in place with other strides
    assert turn(lib, None, r) == [1, 1] and turn(lib, g, None) == [1, 1] and turn(lib, rope_shape(hq=0, hk=0), r) == [3, 3]
    assert turn(lib, rope_shape(bits=32), r, pos=258) == [2, 2]
    for kw, code in ((dict(slots=None), 1), (dict(slots=260), 2), (dict(v=None), 1), (dict(v=769), 2), (dict(kc=None), 1), (dict(vc=None), 1), (dict(kc=512), 1),
                     (dict(vc=768), 1), (dict(vc=2048), 1)):
        assert append(lib, g, r, **kw) == code, kw
    assert append(lib, rope_shape(hk=0), r) == 3 and append(lib, rope_shape(cache=-1), r) == 3
    for name, value in (("rot_dim", 0), ("rot_dim", 7), ("rot_dim", 66)):
        bad = table()[1]
        setattr(bad, name, value)
        assert turn(lib, g, ctypes.byref(bad)) == [3, 3]
    for name, value in (("interleaved", 2), ("magnitude", NAN)):
        bad = table()[1]
        setattr(bad, name, value)
        assert turn(lib, g, ctypes.byref(bad)) == [1, 1]


def test_layer_backward_from_8_bits(lib):
    def call(x8, m=128):
        return lib.lora_bwd_act8(256, x8, 256, 256, 256, 256, None, 1.0, 0.0, 0, m, 128, 128, 16, 256, 256, 256, 256, 1 << 30, None)

    assert call(None) == 1 and call(kept(codes=None)) == 1 and call(kept(scales=None)) == 1
    assert call(kept(codes=264)) == 2 and call(kept(scales=258)) == 2
    assert lib.multi_lora_bwd_act8(256, None, 256, None, 0, None, 0, 0, 128, 128, 128, 256, None, 256, 256, 1 << 30, None) == 1


@pytest.mark.parametrize("kind,name", [(23, "act8_store"), (25, "norm_fwd"), (27, "norm_sums"), (28, "rope"), (29, "rope_append")])
def test_kernel_names(lib, kind, name):
    assert lib.lora_kernel_name(kind).decode() == name
