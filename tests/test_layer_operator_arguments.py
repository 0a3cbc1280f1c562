"""Arguments of rotary positions and norms that are missing or decide a type, without a GPU: tensors are stand-ins, and where a call is refused a library that is
reached fails the test."""
import pytest

torch = pytest.importorskip("torch")

from lora_fine_tuning_gb300 import api, native  # noqa: E402
from tests.test_layer_operator_devices import BF16, C, KV, Q, ROPE, ROWS, Tensor, lib  # noqa: E402, F401

OUT = {api.rope_fwd: ("Q_out", "K_out"), api.rope_bwd: ("dQ_out", "dK_out")}
GIVEN = dict(Q=Q, K=KV, V=KV, positions=ROWS, slots=ROWS, K_cache=C, V_cache=C)


@pytest.mark.parametrize("call", [api.rope_fwd, api.rope_bwd])
def test_neither_queries_nor_keys(lib, call):  # noqa: F811
    with pytest.raises(ValueError, match="Q or K"):
        call(None, None, Tensor(*ROWS), ROPE)
    for given in ((Tensor(*Q), None), (None, Tensor(*KV))):      # either alone is a call
        call(*given, Tensor(*ROWS), ROPE, **dict(zip(OUT[call], given)))
    assert lib.called == 2


@pytest.mark.parametrize("call", [api.rope_fwd, api.rope_bwd])
@pytest.mark.parametrize("shape", [(6,), (6, 64), (6, 2, 64, 1)])
def test_keys_that_are_not_heads(lib, call, shape):  # noqa: F811
    for q, k in ((Tensor(*Q), Tensor(shape, BF16)), (None, Tensor(shape, BF16)), (Tensor(shape, BF16), Tensor(*KV))):
        with pytest.raises(ValueError):
            call(q, k, Tensor(*ROWS), ROPE, **dict(zip(OUT[call], (q, k))))
    assert not lib.called


@pytest.mark.parametrize("missing", GIVEN)
def test_append_without_an_operand(lib, missing):  # noqa: F811
    t = {k: None if k == missing else Tensor(*v) for k, v in GIVEN.items()}
    with pytest.raises(ValueError, match=missing):
        api.rope_append(*t.values(), ROPE, Q_out=Tensor(*Q))
    assert not lib.called


def test_no_positions(lib):  # noqa: F811
    with pytest.raises(ValueError, match="positions"):
        api.rope_fwd(Tensor(*Q), Tensor(*KV), None, ROPE, Q_out=Tensor(*Q), K_out=Tensor(*KV))
    assert not lib.called


@pytest.mark.parametrize("dtype,code", [(torch.bfloat16, 0), (torch.float32, 1)])
def test_stream_type_where_only_8_bits_are_given(lib, monkeypatch, dtype, code):  # noqa: F811
    """Without the stream's gradient, dh_out alone says what type the stream has."""
    seen = []
    monkeypatch.setattr(lib, "norm_bwd", lambda norm, *rest: seen.append(native.Norm.from_buffer_copy(norm).stream_dtype) or 0)
    h8, dh = api.Act8(Tensor((6, 64), torch.int8), Tensor((6, 4), torch.uint8), 64), Tensor((6, 64), dtype)
    g = api.norm_bwd(Tensor((6, 64), BF16), h8, Tensor((64,), BF16), want_weights=False, dh_out=dh)
    assert seen == [code] and g.dh is dh
    with pytest.raises(TypeError):
        api.norm_bwd(Tensor((6, 64), BF16), h8, Tensor((64,), BF16), want_weights=False, dh_out=Tensor((6, 64), torch.float16))
