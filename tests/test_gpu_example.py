"""The operators together: the example's training steps, and its block's gradients against the same block in autograd."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from lora_fine_tuning_gb300 import api  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("align_adapters", os.path.join(ROOT, "examples", "align_adapters.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_preference_training_lowers_its_loss(ex):
    losses, shift = ex.train("preference", steps=12)
    assert abs(losses[0] - 0.6931) < 0.02      # log 2: the adapters start as the frozen model (their B is zero)
    assert losses[-1] < losses[0] - 0.1 and shift > 0


def test_policy_training_raises_the_advantaged_tokens(ex):
    losses, shift = ex.train("policy", steps=12)
    assert shift > 0.01


@pytest.mark.parametrize("reference", [False, True])
def test_gradients_of_the_whole_block(ex, monkeypatch, reference):
    """Every adapter gradient of one preference step against autograd through the same block in fp64 (dropout off).
    Between the two lie the bf16 roundings of the operators' inputs and outputs: QKV, O, P, dS, logits, dlogits, dY,
    dO, dQKV and the rank-r intermediates, about a dozen of 2^-9 relative each and independent, so within 2e-2 of a
    gradient's norm.  Without a reference the second pair's margin is that of 40 rows against 200, about 140: its weight
    sigmoid(-140) is below fp32's smallest value, and zero is its right answer."""
    monkeypatch.setattr(ex, "DROPOUT", 0.0)
    gen = torch.Generator(device="cuda").manual_seed(3)
    block = ex.Block(2, gen)
    for a in block.qkv + block.out:
        a.B.copy_((torch.randn(a.B.shape, device="cuda", generator=gen) * 0.02).bfloat16())
    tokens, labels, places, rows = ex.batch([150, 130, 40, 200], gen)
    segments = [(a, -(-n // 128) * 128, i // 2) for i, (a, n) in enumerate(places)]
    pairs = [(places[0][0], places[1][0], 150, 130), (places[2][0], places[3][0], 40, 200)]
    logits, saved = block.forward(tokens, segments, places, 0)
    ref = None
    if reference:   # log p of a nearby policy
        zeros = torch.zeros(rows, device="cuda")
        logp = api.policy_loss(logits, labels, zeros, zeros, want_grad=False)[1]
        ref = logp + 0.1 * torch.randn(rows, device="cuda", generator=gen)
    loss, logp, margins, dlogits = api.pref_loss(logits, labels, pairs, ref, beta=0.1, dlogits=logits)
    block.backward(dlogits, saved, segments, places, 0)

    leaves = [(a, a.A.double().requires_grad_(), a.B.double().requires_grad_()) for a in block.qkv + block.out]

    def project(x, w, ads):
        y = x @ w.double()
        out = y.clone()
        for (a, n, i) in segments:
            _, A, B = ads[i]
            out[a:a + n] = y[a:a + n] + ex.ALPHA * (x[a:a + n] @ A) @ B
        return out

    x = block.embed[tokens].double()
    q, k, v = ex.Block.heads(project(x, block.w_qkv, leaves[:2]))
    g = ex.Q_HEADS // ex.KV_HEADS
    o = torch.zeros(rows, ex.Q_HEADS, ex.HEAD_DIM, dtype=torch.float64, device="cuda")
    for a, n in places:
        s = torch.einsum("ihd,jhd->hij", q[a:a + n], k[a:a + n].repeat_interleave(g, 1)) * ex.HEAD_DIM ** -0.5
        s = s.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), float("-inf"))
        o[a:a + n] = torch.einsum("hij,jhd->ihd", s.softmax(2), v[a:a + n].repeat_interleave(g, 1))
    z = (x + project(o.flatten(1), block.w_out, leaves[2:])) @ block.head.double()
    lp = torch.where(labels >= 0, torch.log_softmax(z, 1).gather(1, labels.clamp(min=0)[:, None])[:, 0], 0.0)
    if reference:
        lp = lp - torch.where(labels >= 0, ref, 0.0)
    want = sum(-torch.nn.functional.logsigmoid(0.1 * (lp[c:c + cn].sum() - lp[r:r + rn].sum())) for c, r, cn, rn in pairs)
    want.backward()
    for a, A, B in leaves:
        for got, leaf in ((a.dA, A), (a.dB, B)):
            least = torch.finfo(torch.float32).tiny * leaf.numel()
            assert float((got.double() - leaf.grad).norm()) <= 2e-2 * float(leaf.grad.norm()) + least
