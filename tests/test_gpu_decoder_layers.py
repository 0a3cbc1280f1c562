"""The operators of a decoder layer together, as they are used: the example's gradients against the same decoder in fp64 autograd, its training steps,
and its generation into a cache against the whole sequence at once."""
import importlib.util
import math
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
    spec = importlib.util.spec_from_file_location("decoder_layers", os.path.join(ROOT, "examples", "decoder_layers.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def decoder64(ex, model, tokens, positions, places, adapters):
    """Logits in fp64 with `adapters` (leaves) in the place of the model's."""
    def rms(x, w):
        return x / torch.sqrt((x * x).mean(1, keepdim=True) + ex.EPS) * w.double()

    def turned(x):
        f = 10000.0 ** (-2.0 * torch.arange(ex.HEAD_DIM // 2, dtype=torch.float64, device="cuda") / ex.HEAD_DIM)
        angle = torch.outer(positions.double(), f)[:, None]
        a, b = x.chunk(2, -1)
        return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1)

    h, group = model.embed[tokens].double(), ex.Q_HEADS // ex.KV_HEADS
    x = rms(h, model.norm_of(0))
    for i, layer in enumerate(model.layers):
        (a1, b1), (a2, b2) = adapters[i]
        q, k, v = ex.Decoder.heads(x @ layer.qkv.double() + ex.ALPHA * (x @ a1) @ b1)
        q, k = turned(q), turned(k)
        o = torch.zeros_like(q)
        for a, n in places:
            s = torch.einsum("ihd,jhd->hij", q[a:a + n], k[a:a + n].repeat_interleave(group, 1)) * ex.HEAD_DIM ** -0.5
            s = s.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), -math.inf)
            o[a:a + n] = torch.einsum("hij,jhd->ihd", s.softmax(2), v[a:a + n].repeat_interleave(group, 1))
        o = o.flatten(1)
        y = o @ layer.out.double() + ex.ALPHA * (o @ a2) @ b2
        h = h + ex.RES_SCALE * layer.gate.double() * rms(y, layer.post)
        x = rms(h, model.norm_of(i + 1))
    return x @ model.head.double()


@pytest.mark.parametrize("keep", ["bf16", "8 bits"])
def test_gradients_of_the_decoder(ex, keep):
    """Between the two lie the bf16 roundings of the operators' inputs and outputs, about two dozen of 2^-9 each (in the mean) and independent:
    within 2e-2 of a gradient's norm.  8 bits: a kept value is off by 2^-7 of its block's largest at most, evenly spread, 2^-7 / sqrt(3) of it in the mean,
    and a block's largest is about twice its values' mean size: 1e-2 each for x, h and y, 2e-2 together."""
    model = ex.Decoder(1)
    tokens, labels, positions, places = ex.packed([90, 41, 130], 2)
    dlogits = (torch.randn(len(tokens), ex.VOCAB, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)) * 1e-3).bfloat16()
    logits, saved = model.forward(tokens, positions, places, 0, 0.0, keep)
    model.backward(dlogits, saved, positions, places, 0, 0.0)
    leaves = [[tuple(t.double().requires_grad_() for t in pair) for pair in layer.adapters] for layer in model.layers]
    want = decoder64(ex, model, tokens, positions, places, leaves)
    assert float((logits.double() - want.detach()).norm()) <= 2e-2 * float(want.detach().norm())
    want.backward(dlogits.double())
    for layer, pairs in zip(model.layers, leaves):
        for got, leaf in zip(layer.grads, [t for pair in pairs for t in pair]):
            assert float((got.double() - leaf.grad).norm()) <= (2e-2 if keep == "bf16" else 4e-2) * float(leaf.grad.norm())


@pytest.mark.parametrize("keep", ["bf16", "8 bits"])
def test_training_runs(ex, keep):
    model, losses = ex.train(3, keep)
    assert len(losses) == 3 and all(math.isfinite(x) for x in losses)
    assert all(bool(torch.isfinite(g).all()) for _, g in model.parameters())


def test_generation_is_the_forward_of_the_whole_sequence(ex):
    """Each new row's logits against the decoder on prompt and continuation at once: the same operators on other shapes, a dozen bf16 roundings a layer
    on either side, within 2e-2 of the logits' norm."""
    model = ex.Decoder(4)
    prompts = [ex.packed([n], n)[0] for n in (33, 5, 16)]
    tokens, logits = ex.generate(model, prompts, 6)
    for p, new, got in zip(prompts, tokens, logits):
        whole = torch.cat([p, new])
        want = model.forward(whole, torch.arange(len(whole), device="cuda"), [(0, len(whole))], 0, 0.0, "bf16")[0][len(p) - 1:-1]
        assert float((got.double() - want.double()).norm()) <= 2e-2 * float(want.double().norm())


def test_a_token_step_in_a_graph(ex):
    """One token a request, captured once and replayed with other tokens, positions and slots; the cache's range a request sees is the graph's."""
    model = ex.Decoder(5)
    cache = ex.Cache([32, 32])
    gen = torch.Generator(device="cuda").manual_seed(6)
    for t in cache.k + cache.v:
        t.copy_(torch.randn(t.shape, device="cuda", generator=gen))
    tokens, positions, slots = (torch.tensor(x, device="cuda") for x in ([3, 4], [31, 31], [31, 63]))
    seqs = api.attn_seqs([(0, 1, 0, 32), (1, 1, 32, 32)])
    ex.step(model, cache, tokens, positions, slots, seqs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ex.step(model, cache, tokens, positions, slots, seqs)
    tokens += 100
    positions -= 1
    slots -= 1
    graph.replay()
    kept = [t.clone() for t in cache.k]
    assert torch.equal(out, ex.step(model, cache, tokens, positions, slots, seqs))
    assert all(torch.equal(a, b) for a, b in zip(kept, cache.k))
