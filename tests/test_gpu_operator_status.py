"""The device status word of attention and loss calls that are given no workspace."""
import pytest

from tests.gpu_helpers import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from lora_fine_tuning_gb300 import api  # noqa: E402
from tests.test_gpu_threads import attention, policy, preference  # noqa: E402


@pytest.mark.parametrize("kind", ["attn", "loss"])
def test_status_of_the_cached_workspace(kind):
    """Zero after calls; a code that a kernel left (written by the host here) is seen and cleared, and calls go on."""
    if kind == "attn":
        calls = [attention([(0, 1, 0, 5000), (1, 20, 5000, 3000)], 8, 2, 64, 9), attention([(0, 700, 0, 700)], 8, 2, 128, 1)]
        find = lambda s=None: api.attn_workspace(21, 8, stream=s)  # noqa: E731
    else:
        calls = [preference(40, 32001, torch.bfloat16, 2, 0), policy(24, 50001, torch.float32, 1)]
        find = lambda s=None: api.loss_workspace(40, stream=s)  # noqa: E731
    want = [[x.clone() for x in f()] for f in calls]
    ws = find()
    assert api.lora_device_status(ws) == 0 and not ws[:256].count_nonzero()
    ws[:4].view(torch.int32).fill_(0x0703)
    assert api.lora_device_status(find()) == 0x0703 and api.lora_device_status(find()) == 0
    for f, w in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(w, f()))
    assert find().data_ptr() == ws.data_ptr() and api.lora_device_status(ws) == 0
    side = torch.cuda.Stream()
    assert find(side).data_ptr() != ws.data_ptr() and api.lora_device_status(find(side), side) == 0


def test_no_cached_workspace_in_a_capture():
    graph = torch.cuda.CUDAGraph()
    x = torch.zeros(4, device="cuda")
    with torch.cuda.graph(graph):
        x.add_(1)
        with pytest.raises(RuntimeError):
            api.loss_workspace(10)
