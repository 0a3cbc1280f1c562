"""Every tensor of an attention, loss or AdamW call is on the call's device, without a GPU: tensors are stand-ins that know
their type, shape and device only, and a library that is reached fails the test."""
import pytest

torch = pytest.importorskip("torch")

from lora_fine_tuning_gb300 import api, native  # noqa: E402

BF16, F32, I64, U8 = torch.bfloat16, torch.float32, torch.int64, torch.uint8


class Tensor:
    is_cuda = True

    def __init__(self, shape, dtype, index=0):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index
        self.device = torch.device("cuda", index)

    def stride(self, i=None):
        s = tuple(int(torch.Size(self.shape[j + 1:]).numel()) for j in range(len(self.shape)))
        return s if i is None else s[i]

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 256


class Library:
    """Stands for the built library: sizes, and calls that are noted."""
    called = 0

    def attn_workspace_size(self, rows, heads):
        return 1024

    def loss_workspace_size(self, rows):
        return 1024

    def note(self, *args):
        self.called += 1
        return 0

    attn_fwd = attn_bwd = pref_loss = policy_loss = adamw_step = note


@pytest.fixture
def lib(monkeypatch):
    one = Library()
    monkeypatch.setattr(native, "lib", lambda: one)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(api, "_current_stream", lambda index: 0)
    return one


Q, KV, LSE = ((6, 4, 64), BF16), ((6, 2, 64), BF16), ((6, 4), F32)
ROWS, WS = ((6,), F32), ((4096,), U8)
CALLS = {
    "attn_fwd": (lambda t: api.attn_fwd(t["Q"], t["K"], t["V"], [(0, 6)], O=t["O"], lse=t["lse"], ws=t["ws"]),
                 dict(Q=Q, K=KV, V=KV, O=Q, lse=LSE, ws=WS)),
    "attn_bwd": (lambda t: api.attn_bwd(t["dO"], t["Q"], t["K"], t["V"], t["O"], t["lse"], [(0, 6)], dQ=t["dQ"], dK=t["dK"],
                                        dV=t["dV"], ws=t["ws"]),
                 dict(dO=Q, Q=Q, K=KV, V=KV, O=Q, lse=LSE, dQ=Q, dK=KV, dV=KV, ws=WS)),
    "pref_loss": (lambda t: api.pref_loss(t["logits"], t["labels"], [(0, 3, 3, 3)], t["ref_logp"], dlogits=t["dlogits"],
                                          logp=t["logp"], loss=t["loss"], margins=t["margins"], ws=t["ws"]),
                  dict(logits=((6, 50), BF16), labels=((6,), I64), ref_logp=ROWS, dlogits=((6, 50), BF16), logp=ROWS,
                       loss=((), F32), margins=((1,), F32), ws=WS)),
    "policy_loss": (lambda t: api.policy_loss(t["logits"], t["labels"], t["old_logp"], t["advantages"], t["ref_logp"],
                                              kl_coef=0.1, dlogits=t["dlogits"], logp=t["logp"], loss=t["loss"], ws=t["ws"]),
                    dict(logits=((6, 50), F32), labels=((6,), I64), old_logp=ROWS, advantages=ROWS, ref_logp=ROWS,
                         dlogits=((6, 50), F32), logp=ROWS, loss=((), F32), ws=WS)),
    "adamw_step": (lambda t: api.adamw_step([api.AdamWTensor(*(t[x] for x in ("param", "grad", "m", "v")))], lr=1e-3, step=1,
                                            grad_scale=t["grad_scale"]),
                   dict(param=ROWS, grad=ROWS, m=ROWS, v=ROWS, grad_scale=((), F32))),
}


@pytest.mark.parametrize("name", CALLS)
def test_all_on_one_device(lib, name):
    call, given = CALLS[name]
    call({k: Tensor(*v) for k, v in given.items()})
    assert lib.called == 1


@pytest.mark.parametrize("name,other", [(n, x) for n, (_, given) in CALLS.items() for x in given])
def test_one_on_another_device(lib, name, other):
    call, given = CALLS[name]
    with pytest.raises(ValueError, match="cuda:1|one device"):
        call({k: Tensor(*v, index=1 if k == other else 0) for k, v in given.items()})
    assert not lib.called


@pytest.mark.parametrize("name", ["attn_fwd", "attn_bwd", "pref_loss", "policy_loss"])
def test_workspaces_with_holes(lib, name):
    """numel() is the bytes that the library may use from the first one on: none may be missing in between."""
    call, given = CALLS[name]
    t = {k: Tensor(*v) for k, v in given.items()}
    t["ws"].is_contiguous = lambda: False
    with pytest.raises(ValueError, match="ws"):
        call(t)
    assert not lib.called
