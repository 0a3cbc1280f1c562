"""The library's first call on a device prepares what every operator needs, not the norms' 140 forms; a norm's first call prepares its own."""
import ctypes
import shutil
import time

import pytest

from tests.gpu_helpers import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from lora_fine_tuning_gb300 import api, native  # noqa: E402


def test_first_calls(tmp_path):
    """Copies of the library, each with its first calls still to come.  The setup takes 2.5 ms, 28 with every form of the norms, a norm's first
    form 1.2: the quickest of three copies stays below 12."""
    times = []
    x = torch.randn(4, 64, device="cuda").bfloat16()
    w, out = torch.ones(64, device="cuda"), torch.empty(4, 64, device="cuda").bfloat16()
    norm = native.Norm(4, 64, *[64] * 8)
    norm.w, norm.eps, norm.res_scale = native.Vector(w.data_ptr(), 1, 0), 1e-5, 1.0
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    for i in range(3):
        lib = ctypes.CDLL(shutil.copy(native.LIB_PATH, tmp_path / f"copy{i}.so"))
        lib.act8_store.argtypes, lib.norm_fwd.argtypes = [vp, i64, i64, i64, vp, vp], [vp] * 9
        stream = torch.cuda.current_stream().cuda_stream
        torch.cuda.synchronize()
        start = time.perf_counter()
        assert lib.act8_store(None, 0, 64, 64, ctypes.byref(native.Act8(None, None)), stream) == 0
        middle = time.perf_counter()
        assert lib.norm_fwd(ctypes.byref(norm), x.data_ptr(), None, None, out.data_ptr(), None, None, None, stream) == 0
        torch.cuda.synchronize()
        times.append((middle - start, time.perf_counter() - middle))
        assert torch.equal(out, api.norm_fwd(x, w, eps=1e-5)[0])
    assert min(t[0] for t in times) < 12e-3 and min(t[1] for t in times) < 12e-3, times


def test_a_form_used_first_inside_a_capture():
    """Widths and types of which no other test has had the form, or has: either way the graph is right."""
    x = torch.randn(33, 4500, device="cuda").bfloat16()
    w = torch.ones(4500, device="cuda")
    api.act8_store(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = api.norm_fwd(x, w)[0]
        g = api.norm_bwd(x, x, w)
    graph.replay()
    want = api.norm_bwd(x, x, w)
    assert torch.equal(y, api.norm_fwd(x, w)[0]) and torch.equal(g.dh, want.dh) and torch.equal(g.dw, want.dw)
