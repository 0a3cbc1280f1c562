"""Activations in 8 bits: codes, scales and the values they stand for against the format's definition, bit for bit.

Every step but the rounding to a whole number is exact (the scale is a power of two), so nothing here has a tolerance but
the format's own: half a scale, 2^-7 of the block's largest value.
"""
import ctypes

import pytest

from tests.gpu_helpers import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from lora_fine_tuning_gb300 import api, native  # noqa: E402


def defined(x):
    """Codes and scales of a bf16 matrix by the definition, in 64 bits on the host."""
    x = x.double().cpu()
    rows, width = x.shape
    blocks = -(-width // 32)
    b = torch.zeros(rows, blocks * 32, dtype=torch.float64)
    b[:, :width] = x
    b = b.view(rows, blocks, 32)
    finite = torch.isfinite(b)
    top = torch.where(finite, b.abs(), 0.0).amax(2, keepdim=True)
    e = torch.frexp(top).exponent.double() - 1 - 6                  # floor(log2 top) - 6
    e = torch.where(top > 0, e, -1e9).clamp(min=-126)
    codes = torch.round(torch.where(finite, b, 0.0) / torch.exp2(e)).clamp(-127, 127)
    codes = torch.where(finite, codes, -128.0).view(rows, -1).to(torch.int8)
    scales = torch.full((rows, -(-width // 128) * 4), 127, dtype=torch.uint8)
    scales[:, :blocks] = (e[:, :, 0] + 127).to(torch.uint8)
    return codes, scales


def values(codes, scales, width):
    rows = codes.shape[0]
    c = codes.double().view(rows, -1, 32)
    v = c * torch.exp2(scales[:, :c.shape[1]].double() - 127)[:, :, None]
    return torch.where(c == -128, float("nan"), v).view(rows, -1)[:, :width]


def check(x, kept):
    codes, scales = defined(x)
    assert torch.equal(kept.codes.cpu(), codes) and torch.equal(kept.scales.cpu(), scales)
    got = api.act8_load(kept)
    want = values(codes, scales, x.shape[1]).bfloat16()
    assert torch.equal(got.cpu().view(torch.int16)[~torch.isnan(want)], want.view(torch.int16)[~torch.isnan(want)])
    assert torch.equal(torch.isnan(got).cpu(), torch.isnan(want))
    return got


def activations(rows, width, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    size = torch.exp(2 * torch.randn(width, device="cuda", generator=g))
    return (torch.randn(rows, width, device="cuda", generator=g) * size).bfloat16()


@pytest.mark.parametrize("rows,width", [(1, 1), (1, 8), (3, 31), (5, 32), (2, 33), (7, 100), (4, 127), (9, 128), (3, 129), (77, 1000),
                                        (130, 4096), (17, 14336), (1, 8191), (300, 264)])
def test_format(rows, width):
    x = activations(rows, width, rows + width)
    got = check(x, api.act8_store(x))
    blocks = torch.nn.functional.pad(x.double(), (0, -width % 32)).view(rows, -1, 32)
    top = blocks.abs().amax(2, keepdim=True).expand_as(blocks).reshape(rows, -1)[:, :width]
    assert bool(((got.double() - x.double()).abs() <= 2.0 ** -7 * top).all())


@pytest.mark.parametrize("start,ld", [(0, 136), (8, 136), (1, 137), (3, 160)])
def test_rows_apart(start, ld):
    whole = activations(20, ld)
    x = whole[:, start:start + 100]
    check(x, api.act8_store(x))
    out = torch.full((20, ld), 7.0, device="cuda").bfloat16()
    kept = api.act8_store(x)
    assert torch.equal(api.act8_load(kept, out[:, start:start + 100]), api.act8_load(kept))
    rest = torch.ones(ld, dtype=torch.bool, device="cuda")
    rest[start:start + 100] = False
    assert bool((out[:, rest] == 7).all())


def test_slices_of_rows():
    x = activations(50, 72)
    kept = api.act8_store(x)
    part = api.Act8(kept.codes[20:30], kept.scales[20:30], 72)
    assert torch.equal(api.act8_load(part), api.act8_load(kept)[20:30])
    api.act8_store(x[:10], part)
    assert torch.equal(api.act8_load(kept)[20:30], api.act8_load(kept)[:10])


def test_the_whole_range():
    """Every bf16 value, finite or not, alone in its block and among others."""
    every = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    check(every.view(-1, 32), api.act8_store(every.view(-1, 32)))
    alone = torch.zeros(65536, 32, dtype=torch.bfloat16, device="cuda")
    alone[torch.arange(65536, device="cuda"), torch.arange(65536, device="cuda") % 32] = every
    check(alone, api.act8_store(alone))
    mixed = activations(65536 // 8, 64)
    mixed.view(-1)[::8] = every
    check(mixed, api.act8_store(mixed))


@pytest.mark.parametrize("width", [64, 61])
def test_what_is_not_finite_spoils_itself_only(width):
    x = activations(4, width)
    clean = api.act8_load(api.act8_store(x))
    y = x.clone()
    y[0, 3], y[1, 5], y[2, 40], y[3] = float("inf"), float("-inf"), float("nan"), float("nan")
    got = api.act8_load(api.act8_store(y))
    bad = ~torch.isfinite(y)
    assert bool(torch.isnan(got[bad]).all())
    same = ~bad
    for r, b in ((0, 0), (1, 0), (2, 1)):       # the blocks of the spoiled values may have another scale
        same[r, 32 * b:32 * b + 32] = False
    assert torch.equal(got[same], clean[same])
    check(y, api.act8_store(y))


def test_nothing_to_do():
    kept = api.act8_store(torch.empty(0, 40, dtype=torch.bfloat16, device="cuda"))
    assert api.act8_load(kept).shape == (0, 40)


def test_offsets_past_32_bits():
    """Rows whose last elements lie beyond 2^31 values and 2^32 bytes."""
    buffer = torch.empty((1 << 31) + 4096, dtype=torch.bfloat16, device="cuda")
    x = buffer.as_strided((3, 1000), (1 << 30, 1))
    x.copy_(activations(3, 1000))
    check(x, api.act8_store(x))
    kept = api.act8_store(activations(3, 1000, 1))
    assert torch.equal(api.act8_load(kept, x), api.act8_load(kept))


def test_another_stream_and_a_graph():
    x = activations(300, 520)
    want = api.act8_load(api.act8_store(x))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = api.act8_load(api.act8_store(x, stream=s), stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = api.act8_load(api.act8_store(x))
    x.copy_(activations(300, 520, 5))
    g.replay()
    assert torch.equal(out, api.act8_load(api.act8_store(x)))


def test_refusals():
    x = activations(4, 40)
    with pytest.raises(TypeError):
        api.act8_store(x.float())
    with pytest.raises(ValueError):
        api.act8_store(x.t())
    with pytest.raises(ValueError):
        api.act8_store(x, api.act8(4, 48))
    with pytest.raises(ValueError):
        api.act8_store(x, api.act8(5, 40))
    kept = api.act8_store(x)
    with pytest.raises(ValueError):
        api.act8_load(kept, torch.empty(4, 39, device="cuda").bfloat16())
    with pytest.raises(ValueError):
        api.act8_load(api.Act8(kept.codes[:, :32], kept.scales, 32))
    with pytest.raises(native.LoraError):
        native.check("act8_store", native.lib().act8_store(x.data_ptr(), 4, 40, 39, ctypes.byref(native.Act8(256, 256)), None))
