"""Norms around a block through the C ABI, in the calls that the header allows and the Python calls do not make: a gradient of the stream that is not
given beside a stride that is, outputs left out.  Every result is the bits of the call that is given (or asked for) everything."""
import ctypes

import pytest

from tests.gpu_helpers import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from lora_fine_tuning_gb300 import api, native  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


def vector(t):
    return native.Vector(None, 0, 0) if t is None else native.Vector(t.data_ptr(), int(t.dtype == F32), 0)


def norm(st, stream):
    """Every stride is the width, whether its matrix is given or not."""
    rows, width = st["h"].shape
    n = native.Norm(rows, width, *[width] * 8)
    n.w, n.post_w, n.gate, n.row_gate = (vector(st[k]) for k in ("w", "post_w", "gate", "row_gate"))
    n.eps, n.w_offset, n.res_scale, n.stream_dtype = 1e-5, 0.0, 0.7, int(stream == F32)
    return ctypes.byref(n)


def ptr(t):
    return None if t is None else t.data_ptr()


def kept(a):
    return None if a is None else ctypes.byref(native.Act8(a.codes.data_ptr(), a.scales.data_ptr()))


def inputs(rows, width, stream):
    g = torch.Generator(device="cuda").manual_seed(rows + width)

    def normal(*shape, dtype=BF):
        return torch.randn(*shape, device="cuda", generator=g).to(dtype)

    return dict(h=normal(rows, width, dtype=stream), y=normal(rows, width), dx=normal(rows, width), w=normal(width), post_w=normal(width, dtype=F32),
                gate=normal(width), row_gate=normal(rows, dtype=F32))


OUTPUTS = ("dh_out", "dy", "dw", "dpost_w", "dgate", "drow_gate")


def backward(st, stream, dh, leave=(), eight=False):
    """Outputs by name; those in `leave` are not asked for.  eight: h and y come in 8 bits."""
    rows, width = st["h"].shape
    out = dict(dh_out=torch.empty_like(st["h"]), dy=torch.empty_like(st["y"]), **{k: torch.empty(width, device="cuda") for k in OUTPUTS[2:5]},
               drow_gate=torch.empty(rows, device="cuda"))
    out.update({k: None for k in leave})
    h8, y8 = (api.act8_store(st[k].bfloat16()) if eight else None for k in ("h", "y"))
    size = api.norm_workspace_size(rows, width)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    native.check("norm_bwd", native.lib().norm_bwd(
        norm(st, stream), ptr(st["dx"]), ptr(dh), None if eight else ptr(st["h"]), kept(h8), None if eight else ptr(st["y"]), kept(y8),
        *(ptr(out[k]) for k in OUTPUTS), ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    return {k: t for k, t in out.items() if t is not None}


def leave_nan_in_shared_memory():
    """The largest rows' backward on NaN, on every SM: what it leaves in shared memory is NaN."""
    st = {k: torch.full_like(t, NAN) for k, t in inputs(400, 16380, F32).items()}
    backward(st, F32, st["h"])


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("width", [7, 97, 1025, 2050, 3001, 8190, 9001, 96, 4096])
def test_no_gradient_of_the_stream_is_one_of_zeros(width, stream, eight):
    st = inputs(9, width, stream)
    want = backward(st, stream, torch.zeros_like(st["h"]), eight=eight)
    leave_nan_in_shared_memory()
    got = backward(st, stream, None, eight=eight)
    for k in OUTPUTS:
        assert torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("width", [97, 2050, 4096, 9001])
def test_outputs_left_out(width, stream):
    st = inputs(9, width, stream)
    dh = torch.ones_like(st["h"])
    want = backward(st, stream, dh)
    for leave in (("dy",), ("dy", "drow_gate"), ("dw", "dgate"), ("dpost_w",), OUTPUTS[1:], OUTPUTS[2:]):
        got = backward(st, stream, dh, leave)
        assert len(got) == len(OUTPUTS) - len(leave)
        for k, t in got.items():
            assert torch.equal(t, want[k]), (k, leave)


@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("width", [97, 200, 2050, 4096, 9001])
def test_the_norm_in_8_bits_alone(width, stream):
    """x NULL beside x8: the codes and scales of the call that also writes x."""
    st = inputs(9, width, stream)

    def forward(x):
        h_out, x8 = torch.empty_like(st["h"]), api.act8(9, width)
        x8.codes.fill_(77), x8.scales.fill_(77)
        native.check("norm_fwd", native.lib().norm_fwd(norm(st, stream), ptr(st["h"]), ptr(st["y"]), ptr(h_out), ptr(x), kept(x8), None, None,
                                                       torch.cuda.current_stream().cuda_stream))
        return h_out, x8.codes, x8.scales

    x = torch.empty(9, width, dtype=BF, device="cuda")
    want = forward(x)
    assert all(torch.equal(a, b) for a, b in zip(forward(None), want))
    of_x = api.act8_store(x)
    assert torch.equal(want[1], of_x.codes) and torch.equal(want[2], of_x.scales)
