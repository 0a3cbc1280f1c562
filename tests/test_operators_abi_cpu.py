"""Attention, losses and AdamW through the C ABI without a GPU: every refusal is made before any CUDA call, with the
code the header gives, and the host-only sizes.  No call here launches a kernel."""
import os

import pytest

from lora_fine_tuning_gb300 import native


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(native.LIB_PATH):
        from lora_fine_tuning_gb300 import build
        build.build()
    return native.lib()


def shape(q_rows=300, k_rows=300, q_heads=8, kv_heads=2, head_dim=64, scale=0.125, **strides):
    s = native.AttnShape(q_rows, k_rows, q_heads, kv_heads, head_dim, scale)
    for f in ("q", "k", "v", "o", "d_o", "d_q", "d_k", "d_v"):
        heads = kv_heads if f in ("k", "v", "d_k", "d_v") else q_heads
        m = getattr(s, f)
        m.row, m.head = strides.get(f, (heads * head_dim, head_dim))
    return s


def fwd(lib, s, seqs=((0, 300, 0, 300),), n=None, Q=256, K=256, V=256, O=256, lse=256, ws=256, ws_bytes=1 << 30):
    return lib.attn_fwd(Q, K, V, s, native.attn_seqs_array(list(seqs)), len(seqs) if n is None else n, O, lse, ws,
                        ws_bytes, None)


def bwd(lib, s, seqs=((0, 300, 0, 300),), dO=256, Q=256, O=256, lse=256, dQ=256, dK=256, dV=256, ws=256,
        ws_bytes=1 << 30):
    return lib.attn_bwd(dO, Q, 256, 256, O, lse, s, native.attn_seqs_array(list(seqs)), len(seqs), dQ, dK, dV, ws,
                        ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q_rows=-1), 3), (dict(q_rows=262145), 3), (dict(k_rows=262145), 3), (dict(q_heads=0), 3),
    (dict(q_heads=1032), 3), (dict(q_heads=9), 3), (dict(kv_heads=0), 3), (dict(head_dim=60), 3),
    (dict(head_dim=136), 3), (dict(head_dim=0), 3), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
    (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1), (dict(q=(513, 64)), 2), (dict(q=(512, 60)), 2),
    (dict(q=(-512, 64)), 3), (dict(q=(512, 56)), 3), (dict(q=(504, 64)), 3), (dict(k=(64, 64)), 3),
    (dict(v=(1 << 38, 64)), 3), (dict(o=(0, 64)), 3)])
def test_attention_shapes_and_strides(lib, kw, code):
    assert fwd(lib, shape(**kw)) == code
    assert bwd(lib, shape(**kw)) == code


@pytest.mark.parametrize("kw", [dict(d_o=(504, 64)), dict(d_q=(0, 64)), dict(d_k=(64, 64)), dict(d_v=(120, 64))])
def test_attention_gradient_strides(lib, kw):
    assert bwd(lib, shape(**kw)) == 3


@pytest.mark.parametrize("seqs", [
    [(0, 301, 0, 300)], [(0, 300, 0, 301)], [(0, 100, 0, 100), (50, 100, 100, 100)],
    [(0, 100, 0, 100), (100, 100, 50, 100)], [(100, 100, 100, 100), (0, 100, 0, 100)], [(-1, 10, 0, 10)],
    [(0, -1, 0, 10)], [(0, 10, 0, -1)], [(1 << 62, 1 << 62, 0, 10)], [(0, 10, 1 << 62, 1 << 62)]])
def test_attention_tables(lib, seqs):
    assert fwd(lib, shape(), seqs) == 8
    assert bwd(lib, shape(), seqs) == 8


def test_attention_table_lengths_and_pointers(lib):
    assert fwd(lib, shape(), n=-1) == 8
    assert fwd(lib, shape(), n=1025) == 8
    assert lib.attn_fwd(256, 256, 256, shape(), None, 1, 256, 256, 256, 1 << 30, None) == 1
    assert lib.attn_fwd(256, 256, 256, None, None, 0, 256, 256, 256, 1 << 30, None) == 1
    for name in ("Q", "K", "V", "O", "lse"):
        assert fwd(lib, shape(), **{name: None}) == 1
        assert fwd(lib, shape(), **{name: 264}) == 2
    for name in ("dO", "Q", "O", "lse", "dQ", "dK", "dV"):
        assert bwd(lib, shape(), **{name: None}) == 1
        assert bwd(lib, shape(), **{name: 264}) == 2
    for call, least in ((fwd, 256), (bwd, 256 + 300 * 8 * 4)):
        for kw in (dict(ws=None), dict(ws=256 + 16), dict(ws_bytes=least - 1)):
            assert call(lib, shape(), **kw) == 6


def test_attention_workspace(lib):
    assert lib.attn_workspace_size(-1, 8) == 0
    a, b = lib.attn_workspace_size(1, 1), lib.attn_workspace_size(262144, 1024)
    assert a % 256 == 0 and 256 < a < b
    assert b >= 256 + 262144 * 1024 * 4


def logits(lib=None, logits=256, dlogits=256, rows=10, vocab=100, ld=100, dlogits_ld=100, labels=256, logp=256, dtype=0):
    return native.Logits(logits, dlogits, rows, vocab, ld, dlogits_ld, labels, logp, dtype, 0)


def pref(lib, g, pairs=((0, 5, 5, 5),), n=None, ref=256, beta=0.1, smooth=0.0, scale=1.0, loss=256, margins=256, ws=256,
         ws_bytes=1 << 30):
    return lib.pref_loss(g, native.pref_pairs_array(list(pairs)), len(pairs) if n is None else n, ref, beta, smooth, scale,
                         loss, margins, ws, ws_bytes, None)


def policy(lib, g, old=256, adv=256, ref=256, low=0.2, high=0.2, kl=0.1, scale=1.0, loss=256, ws=256, ws_bytes=1 << 30):
    return lib.policy_loss(g, old, adv, ref, low, high, kl, scale, loss, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 1), (dict(rows=-1), 3), (dict(rows=262145), 3), (dict(vocab=0), 3), (dict(vocab=262145, ld=1 << 20), 3),
    (dict(ld=99), 3), (dict(dlogits=512, dlogits_ld=99), 3), (dict(ld=1 << 38), 3), (dict(ld=104), 1),
    (dict(logits=None), 1), (dict(labels=None), 1), (dict(logp=None), 1), (dict(logits=257), 2), (dict(dlogits=513), 2),
    (dict(logits=258, dtype=1), 2), (dict(labels=260), 2), (dict(logp=258), 2)])
def test_loss_logits(lib, kw, code):
    assert pref(lib, logits(**kw)) == code
    assert policy(lib, logits(**kw)) == code


@pytest.mark.parametrize("pairs", [
    [(0, 5, 5, 6)], [(0, 5, 6, 5)], [(-1, 5, 1, 1)], [(0, 5, -1, 1)], [(0, 5, 5, 5), (9, 0, 1, 0)],
    [(1 << 62, 0, 1 << 62, 1)]])
def test_preference_tables(lib, pairs):
    assert pref(lib, logits(), pairs) == 8


def test_preference_arguments(lib):
    nan, inf = float("nan"), float("inf")
    for kw in (dict(beta=nan), dict(beta=inf), dict(scale=nan), dict(smooth=-0.1), dict(smooth=1.1), dict(smooth=nan),
               dict(loss=None), dict(margins=None)):
        assert pref(lib, logits(), **kw) == 1
    for kw in (dict(loss=258), dict(margins=258), dict(ref=258)):
        assert pref(lib, logits(), **kw) == 2
    assert pref(lib, logits(), n=-1) == 8 and pref(lib, logits(), n=1025) == 8
    assert lib.pref_loss(logits(), None, 1, 256, 0.1, 0.0, 1.0, 256, 256, 256, 1 << 30, None) == 1
    assert lib.pref_loss(None, None, 0, 256, 0.1, 0.0, 1.0, 256, 256, 256, 1 << 30, None) == 1
    need = lib.loss_workspace_size(10)
    assert pref(lib, logits(), ws=None) == 6 and pref(lib, logits(), ws=272) == 6
    assert pref(lib, logits(), ws_bytes=need - 1) == 6
    assert lib.loss_workspace_size(-1) == 0 and need % 256 == 0


def test_policy_arguments(lib):
    nan, inf = float("nan"), float("inf")
    for kw in (dict(low=nan), dict(high=nan), dict(low=-0.1), dict(high=-0.1), dict(kl=nan), dict(scale=inf),
               dict(loss=None), dict(old=None), dict(adv=None), dict(ref=None)):
        assert policy(lib, logits(), **kw) == 1, kw
    for kw in (dict(loss=258), dict(old=258), dict(adv=258), dict(ref=258)):
        assert policy(lib, logits(), **kw) == 2
    assert policy(lib, logits(), ws=None) == 6 and policy(lib, logits(), ws_bytes=256) == 6


def tensor(param=256, grad=256, m=256, v=256, m_scale=256, v_scale=256, master=None, n=1000, param_dtype=0, grad_dtype=0,
           state_bits=8):
    t = (native.AdamWTensor * 1)()
    t[0].param, t[0].grad, t[0].m, t[0].v, t[0].m_scale, t[0].v_scale, t[0].master = param, grad, m, v, m_scale, v_scale, master
    t[0].n, t[0].param_dtype, t[0].grad_dtype, t[0].state_bits = n, param_dtype, grad_dtype, state_bits
    return t


def adamw(lib, t, n=1, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, decay=0.0, step=1, grad_scale=None):
    return lib.adamw_step(t, n, lr, beta1, beta2, eps, decay, step, grad_scale, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), 3), (dict(n=(1 << 40) + 1), 3), (dict(param=None), 1), (dict(grad=None), 1), (dict(m=None), 1),
    (dict(v=None), 1), (dict(m_scale=None), 1), (dict(v_scale=None), 1), (dict(param_dtype=2), 1), (dict(grad_dtype=-1), 1),
    (dict(state_bits=16), 1), (dict(param_dtype=1, master=256), 1), (dict(param=264), 2), (dict(grad=264), 2),
    (dict(m=264), 2), (dict(v=264), 2), (dict(master=264), 2), (dict(m_scale=258), 2), (dict(v_scale=258), 2)])
def test_adamw_tensors(lib, kw, code):
    assert adamw(lib, tensor(**kw)) == code


def test_adamw_arguments(lib):
    nan, inf = float("nan"), float("inf")
    for kw in (dict(lr=nan), dict(lr=inf), dict(beta1=1.0), dict(beta1=-0.1), dict(beta1=nan), dict(beta2=1.0),
               dict(beta2=nan), dict(eps=0.0), dict(eps=nan), dict(eps=1e300), dict(decay=nan), dict(step=0), dict(n=-1)):
        assert adamw(lib, tensor(), **kw) == 1, kw
    assert adamw(lib, None) == 1
    assert adamw(lib, tensor(), grad_scale=258) == 2


@pytest.mark.parametrize("kind,name", [(13, "attn_fwd"), (14, "attn_join"), (17, "attn_fill"), (18, "loss_rows"), (22, "adamw")])
def test_kernel_names(lib, kind, name):
    assert lib.lora_kernel_name(kind).decode() == name
