"""The layer's backward from an input in 8 bits: bit for bit the backward from the bf16 values that the codes stand for, in the mode whose sums
have a fixed order, and near the oracle in either."""
import numpy as np
import pytest

from tests.gpu_helpers import assert_close, host_f64, to_dev, torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from lora_fine_tuning_gb300 import api, native, synth  # noqa: E402
from oracle import lora_oracle as O  # noqa: E402

SHAPES = [(256, 512, 512, 16, 0.1), (640, 384, 264, 16, 0.0), (129, 264, 136, 8, 0.2), (1, 128, 64, 32, 0.1), (1000, 1160, 520, 64, 0.05),
          (300, 640, 256, 128, 0.3), (513, 72, 1032, 24, 0.6), (2000, 1024, 256, 16, 0.0)]


@pytest.fixture
def fixed():
    api.lora_set_deterministic(True)
    yield
    api.lora_set_deterministic(False)


def layer(m, k, n, r, seed=3):
    raw = synth.layer_inputs(seed, m, k, n, r)
    return tuple(to_dev(raw[x]) for x in ("X", "W", "A", "B", "dY"))


@pytest.mark.parametrize("saved_mask", [False, True])
@pytest.mark.parametrize("m,k,n,r,p", SHAPES)
def test_is_the_backward_from_the_values(fixed, m, k, n, r, p, saved_mask):
    X, W, A, B, dY = layer(m, k, n, r)
    kept = api.act8_store(X)
    X2 = api.act8_load(kept)
    Y, S, bits = api.lora_fwd(X2, W, A, B, 2.0, p, 9, want_mask=saved_mask)
    want = api.lora_bwd(dY, X2, W, A, B, S, 2.0, p, 9, mask_bits=bits)
    got = api.lora_bwd(dY, kept, W, A, B, S, 2.0, p, 9, mask_bits=bits)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert api.lora_device_status(api.workspace(m, k, n, r)) == 0


@pytest.mark.parametrize("m,k,n,r,p", SHAPES)
def test_near_the_oracle(m, k, n, r, p):
    X, W, A, B, dY = layer(m, k, n, r, 4)
    kept = api.act8_store(X)
    X2 = api.act8_load(kept)
    S = api.lora_fwd(X2, W, A, B, 1.5, p, 21)[1]
    dX, dA, dB = api.lora_bwd(dY, kept, W, A, B, S, 1.5, p, 21)
    ref = O.lora_backward(*(host_f64(t) for t in (dY, X2, W, A, B)), 1.5, p, 21)
    for name, got, want in zip(("dX", "dA", "dB"), (dX, dA, dB), ref):
        assert_close(name, host_f64(got), want)


@pytest.mark.parametrize("k", [512, 200])
def test_several_adapters(fixed, k):
    n, m = 384, 128 * 7 + 40
    X, W, _, _, dY = layer(m, k, n, 16)
    g = torch.Generator(device="cuda").manual_seed(1)

    def adapters():
        g.manual_seed(1)
        return [api.Adapter((torch.randn(k, r, device="cuda", generator=g) / 20).bfloat16(),
                            (torch.randn(r, n, device="cuda", generator=g) / 20).bfloat16(), a, p)
                for r, a, p in ((16, 1.0, 0.0), (64, 2.0, 0.1), (8, 2.0, 0.3), (32, 1.0, 0.2))]

    segments = [(0, 256, 1), (256, 128, 0), (512, 256, 3), (768, 168, 1)]     # adapter 2 has no rows, rows 384..511 no adapter
    kept = api.act8_store(X)
    X2 = api.act8_load(kept)
    a, b = adapters(), adapters()
    S = api.multi_lora_fwd(X2, W, a, segments, 5)[1]
    want, got = api.multi_lora_bwd(dY, X2, W, a, segments, 5, S), api.multi_lora_bwd(dY, kept, W, b, segments, 5, S)
    assert torch.equal(got, want)
    for p, q in zip(a, b):
        assert torch.equal(p.dA, q.dA) and torch.equal(p.dB, q.dB)


def test_what_is_not_finite_spoils_its_own_features(fixed):
    """A NaN in X spoils its feature's row of dA; where the mask drops it, nothing."""
    m, k, n, r = 256, 256, 128, 16
    X, W, A, B, dY = layer(m, k, n, r)
    X[7, 33] = float("nan")
    kept = api.act8_store(X)
    X2 = api.act8_load(kept)
    S = api.lora_fwd(X2, W, A, B, 2.0, 0.0, 9)[1].nan_to_num()
    got = api.lora_bwd(dY, kept, W, A, B, S, 2.0, 0.0, 9)
    bad = torch.isnan(got[1]).any(1)
    assert bool(torch.isnan(got[1][33]).all()) and int(bad.sum()) == 1
    T = O.dropout_threshold(float(np.float32(0.5)))
    keep = O.keep_mask(9, [7], k, T)[0]
    j = int(np.flatnonzero(~keep)[0])
    X[7, 33], X[7, j] = 0.0, float("inf")
    got = api.lora_bwd(dY, api.act8_store(X), W, A, B, S, 2.0, 0.5, 9)
    assert bool(torch.isfinite(got[1]).all())


def test_refusals():
    X, W, A, B, dY = layer(256, 512, 128, 16)
    S = api.lora_fwd(X, W, A, B, 1.0, 0.0, 0)[1]
    for kept in (api.act8(256, 480), api.act8(255, 512)):
        with pytest.raises(ValueError):
            api.lora_bwd(dY, kept, W, A, B, S, 1.0, 0.0, 0)
    with pytest.raises(TypeError):          # the forward's products need X itself, and so does DoRA's backward
        api.lora_fwd(api.act8_store(X), W, A, B, 1.0, 0.0, 0)
    with pytest.raises(TypeError):
        api.dora_bwd(dY, api.act8_store(X), W, A, B, S, dY, None, None, 1.0, 0.0, 0)
    kept = api.act8_store(X)
    kept.scales = kept.scales[:, :8]
    with pytest.raises(ValueError):
        api.lora_bwd(dY, kept, W, A, B, S, 1.0, 0.0, 0)
    assert native.lib().lora_bwd_act8(256, None, 256, 256, 256, 256, None, 1.0, 0.0, 0, 128, 128, 128, 16, 256, 256, 256, 256, 1 << 30,
                                      None) == 1
