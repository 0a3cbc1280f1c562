"""Every tensor of a norm, rotary position or 8-bit call is on the call's device, without a GPU: tensors are stand-ins that know their type, shape
and device only, and a library that is reached fails the test."""
import pytest

torch = pytest.importorskip("torch")

from lora_fine_tuning_gb300 import api, native  # noqa: E402
from tests import test_operator_devices as base  # noqa: E402


class Tensor(base.Tensor):
    """On the CPU where index is -1."""

    def __init__(self, shape, dtype, index=0):
        super().__init__(shape, dtype, max(index, 0))
        if index < 0:
            self.index, self.device, self.is_cuda = -1, torch.device("cpu"), False


BF16, F32, I64, I8, U8 = torch.bfloat16, torch.float32, torch.int64, torch.int8, torch.uint8


class Library:
    called = 0

    def norm_workspace_size(self, rows, width):
        return 1024

    def note(self, *args):
        self.called += 1
        return 0

    norm_fwd = norm_bwd = act8_store = act8_load = rope_fwd = rope_bwd = rope_append = lora_bwd_act8 = note


@pytest.fixture
def lib(monkeypatch):
    one = Library()
    monkeypatch.setattr(native, "lib", lambda: one)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(api, "_current_stream", lambda index: 0)
    return one


M, V, R = ((6, 64), BF16), ((64,), F32), ((6,), F32)
CODES, SCALES, WS = ((6, 64), I8), ((6, 4), U8), ((4096,), U8)
Q, KV, C, ROWS = ((6, 4, 64), BF16), ((6, 2, 64), BF16), ((90, 2, 64), BF16), ((6,), I64)
ROPE = api.Rope(native.Rope())
CALLS = {
    "norm_fwd": (lambda t: api.norm_fwd(t["h"], t["w"], y=t["y"], post_w=t["post_w"], gate=t["gate"], row_gate=t["row_gate"], h_out=t["h_out"], x=t["x"],
                                        x8=api.Act8(t["codes"], t["scales"], 64)),
                 dict(h=M, w=V, y=M, post_w=V, gate=V, row_gate=R, h_out=M, x=M, codes=CODES, scales=SCALES)),
    "norm_bwd": (lambda t: api.norm_bwd(t["dx"], t["h"], t["w"], dh=t["dh"], y=t["y"], post_w=t["post_w"], gate=t["gate"], row_gate=t["row_gate"],
                                        dh_out=t["dh_out"], dy=t["dy"], dw=t["dw"], dpost_w=t["dpost_w"], dgate=t["dgate"], drow_gate=t["drow_gate"],
                                        ws=t["ws"]),
                 dict(dx=M, h=M, w=V, dh=M, y=M, post_w=V, gate=V, row_gate=R, dh_out=M, dy=M, dw=V, dpost_w=V, dgate=V, drow_gate=R, ws=WS)),
    "norm_bwd, 8 bits": (lambda t: api.norm_bwd(t["dx"], api.Act8(t["codes"], t["scales"], 64), t["w"], dh=t["dh"], want_weights=False, dh_out=t["dh_out"]),
                         dict(codes=CODES, scales=SCALES, dx=M, w=V, dh=M, dh_out=M)),
    "act8_store": (lambda t: api.act8_store(t["X"], api.Act8(t["codes"], t["scales"], 64)), dict(X=M, codes=CODES, scales=SCALES)),
    "act8_load": (lambda t: api.act8_load(api.Act8(t["codes"], t["scales"], 64), t["out"]), dict(codes=CODES, scales=SCALES, out=M)),
    "rope_fwd": (lambda t: api.rope_fwd(t["Q"], t["K"], t["positions"], ROPE, Q_out=t["Q_out"], K_out=t["K_out"]),
                 dict(Q=Q, K=KV, positions=ROWS, Q_out=Q, K_out=KV)),
    "rope_bwd": (lambda t: api.rope_bwd(t["dQ"], t["dK"], t["positions"], ROPE, dQ_out=t["Q_out"], dK_out=t["K_out"]),
                 dict(dQ=Q, dK=KV, positions=ROWS, Q_out=Q, K_out=KV)),
    "rope_append": (lambda t: api.rope_append(t["Q"], t["K"], t["V"], t["positions"], t["slots"], t["K_cache"], t["V_cache"], ROPE, Q_out=t["Q_out"]),
                    dict(Q=Q, K=KV, V=KV, positions=ROWS, slots=ROWS, K_cache=C, V_cache=C, Q_out=Q)),
}


@pytest.mark.parametrize("name", CALLS)
def test_all_on_one_device(lib, name):
    call, given = CALLS[name]
    call({k: Tensor(*v) for k, v in given.items()})
    assert lib.called == 1


@pytest.mark.parametrize("name,other", [(n, x) for n, (_, given) in CALLS.items() for x in given])
@pytest.mark.parametrize("index", [1, -1])
def test_one_on_another_device(lib, name, other, index):
    call, given = CALLS[name]
    with pytest.raises((ValueError, TypeError)):
        call({k: Tensor(*v, index=index if k == other else 0) for k, v in given.items()})
    assert not lib.called


def test_workspace_with_holes(lib):
    call, given = CALLS["norm_bwd"]
    t = {k: Tensor(*v) for k, v in given.items()}
    t["ws"].is_contiguous = lambda: False
    with pytest.raises(ValueError, match="ws"):
        call(t)
    assert not lib.called
