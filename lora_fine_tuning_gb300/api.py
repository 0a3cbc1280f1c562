"""Tensor-level API of the LoRA linear layer (torch tensors in, torch tensors out).

The functions carry the C ABI's names and pass raw device pointers and the
current CUDA stream to it; PyTorch only allocates outputs and workspace.
"""
from __future__ import annotations

import ctypes
import struct
import threading
from dataclasses import dataclass
from typing import NamedTuple, Optional, Sequence

import torch

from . import native

_WS_CACHE: dict = {}


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check_bf16(name: str, t: torch.Tensor, shape) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA bfloat16 tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _stream(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def lora_workspace_size(m: int, k: int, n: int, r_max: int, n_adapters: int = 1) -> int:
    return int(native.lib().lora_workspace_size(m, k, n, r_max, n_adapters))


def lora_set_deterministic(on: bool) -> None:
    """Bit-reproducible reductions for every later call (see include/lora.h); sizes workspaces anew."""
    native.check("lora_set_deterministic", native.lib().lora_set_deterministic(1 if on else 0))


def lora_get_deterministic() -> bool:
    return bool(native.lib().lora_get_deterministic())


def workspace(m: int, k: int, n: int, r_max: int, n_adapters: int = 1, device=None) -> torch.Tensor:
    """A cached, zero-initialised workspace large enough for these sizes."""
    device = torch.device(device or torch.cuda.current_device())
    size = lora_workspace_size(m, k, n, r_max, n_adapters)
    key = device.index
    ws = _WS_CACHE.get(key)
    if ws is None or ws.numel() < size:
        ws = torch.zeros(max(size, 256), dtype=torch.uint8, device=device)
        _WS_CACHE[key] = ws
    return ws


def lora_fwd(X, W, A, B, alpha: float, p: float, seed: int, *, Y=None, S_saved=None, mask_bits=None,
             want_mask: bool = False, ws=None, stream=None):
    """Y = X W + alpha * (dropout(X) A) B.  Returns (Y, S_saved, mask_bits or None)."""
    m, k = X.shape
    n = W.shape[1]
    r = A.shape[1]
    _check_bf16("X", X, (m, k))
    _check_bf16("W", W, (k, n))
    _check_bf16("A", A, (k, r))
    _check_bf16("B", B, (r, n))
    Y = Y if Y is not None else torch.empty((m, n), dtype=torch.bfloat16, device=X.device)
    S_saved = S_saved if S_saved is not None else torch.empty((m, r), dtype=torch.bfloat16, device=X.device)
    if want_mask and mask_bits is None:
        mask_bits = torch.empty((m, k // 8), dtype=torch.uint8, device=X.device)
    ws = ws if ws is not None else workspace(m, k, n, r)
    st = native.lib().lora_fwd(_ptr(X), _ptr(W), _ptr(A), _ptr(B), float(alpha), float(p), int(seed) & (2**64 - 1),
                               m, k, n, r, _ptr(Y), _ptr(S_saved), _ptr(mask_bits), _ptr(ws), ws.numel(),
                               _stream(stream))
    native.check("lora_fwd", st)
    return Y, S_saved, mask_bits


def lora_bwd(dY, X, W, A, B, S_saved, alpha: float, p: float, seed: int, *, dX=None, dA=None, dB=None, ws=None,
             stream=None, mask_bits=None):
    """Gradients of lora_fwd with W frozen.  Returns (dX, dA, dB).  X: the forward's, or what act8_store or norm_fwd kept of it
    in 8 bits (Act8).  mask_bits: optional, the keep bits lora_fwd wrote for the same inputs (read instead of regenerating the mask)."""
    m, k = X.shape
    n = W.shape[1]
    r = A.shape[1]
    for name, t, shp in (("dY", dY, (m, n)), ("W", W, (k, n)), ("A", A, (k, r)), ("B", B, (r, n)), ("S_saved", S_saved, (m, r))):
        _check_bf16(name, t, shp)
    X_arg, act8_form = _layer_input(X, m, k)
    dX = dX if dX is not None else torch.empty((m, k), dtype=torch.bfloat16, device=X.device)
    dA = dA if dA is not None else torch.empty((k, r), dtype=torch.bfloat16, device=X.device)
    dB = dB if dB is not None else torch.empty((r, n), dtype=torch.bfloat16, device=X.device)
    _check_bits(mask_bits, m, k)
    ws = ws if ws is not None else workspace(m, k, n, r)
    name = "lora_bwd" + act8_form
    st = getattr(native.lib(), name)(_ptr(dY), X_arg, _ptr(W), _ptr(A), _ptr(B), _ptr(S_saved), _ptr(mask_bits),
                                     float(alpha), float(p),
                                     int(seed) & (2**64 - 1), m, k, n, r, _ptr(dX), _ptr(dA), _ptr(dB), _ptr(ws),
                                     ws.numel(), _stream(stream))
    native.check(name, st)
    return dX, dA, dB


def _layer_input(X, m: int, k: int):
    """The input of a layer's backward, bf16 or in 8 bits.  Returns what the library takes and how that form's calls end."""
    if isinstance(X, Act8):
        return _act8_arg(_On(X.codes, None), "X", X, m, k), "_act8"
    _check_bf16("X", X, (m, k))
    return _ptr(X), ""


@dataclass
class Adapter:
    """One adapter of a packed multi-adapter batch (A: k x r, B: r x n, bf16 on the device)."""
    A: torch.Tensor
    B: torch.Tensor
    alpha: float
    p: float
    dA: Optional[torch.Tensor] = None
    dB: Optional[torch.Tensor] = None

    @property
    def rank(self) -> int:
        return self.A.shape[1]


def _adapter_array(adapters: Sequence[Adapter], with_grads: bool):
    arr = (native.LoraAdapter * max(1, len(adapters)))()
    for i, a in enumerate(adapters):
        arr[i].rank = a.rank
        arr[i].alpha = a.alpha
        arr[i].p = a.p
        arr[i].A = _ptr(a.A)
        arr[i].B = _ptr(a.B)
        arr[i].dA = _ptr(a.dA) if with_grads else None
        arr[i].dB = _ptr(a.dB) if with_grads else None
    return arr


def saved_width(adapters: Sequence[Adapter]) -> int:
    return max((a.rank for a in adapters), default=0)


def multi_lora_fwd(X, W, adapters: Sequence[Adapter], segments, seed: int, *, Y=None, S_saved=None, mask_bits=None,
                   want_mask: bool = False, ws=None, stream=None):
    """Packed multi-adapter forward; segments are (row_start, rows, adapter).  Returns (Y, S_saved, mask_bits)."""
    m, k = X.shape
    n = W.shape[1]
    _check_bf16("X", X, (m, k))
    _check_bf16("W", W, (k, n))
    s_ld = saved_width(adapters)
    Y = Y if Y is not None else torch.empty((m, n), dtype=torch.bfloat16, device=X.device)
    if S_saved is None and adapters:
        S_saved = torch.empty((m, s_ld), dtype=torch.bfloat16, device=X.device)
    if want_mask and mask_bits is None:
        mask_bits = torch.zeros((m, k // 8), dtype=torch.uint8, device=X.device)
    ws = ws if ws is not None else workspace(m, k, n, max(s_ld, 8), max(1, len(adapters)))
    seg = native.segments_array(segments)
    ad = _adapter_array(adapters, False)
    st = native.lib().multi_lora_fwd(_ptr(X), _ptr(W), ad, len(adapters), seg, len(segments), int(seed) & (2**64 - 1),
                                     m, k, n, _ptr(Y), _ptr(S_saved), _ptr(mask_bits), _ptr(ws), ws.numel(),
                                     _stream(stream))
    native.check("multi_lora_fwd", st)
    return Y, S_saved, mask_bits


def multi_lora_bwd(dY, X, W, adapters: Sequence[Adapter], segments, seed: int, S_saved, *, dX=None, ws=None,
                   stream=None, mask_bits=None):
    """Packed multi-adapter backward.  Fills each adapter's dA / dB (allocated if missing); returns dX.
    X: the forward's, or what act8_store or norm_fwd kept of it in 8 bits (Act8).  mask_bits: optional, the keep bits multi_lora_fwd wrote for the same batch."""
    m, k = X.shape
    n = W.shape[1]
    _check_bf16("dY", dY, (m, n))
    X_arg, act8_form = _layer_input(X, m, k)
    _check_bf16("W", W, (k, n))
    for a in adapters:
        if a.dA is None:
            a.dA = torch.empty_like(a.A)
        if a.dB is None:
            a.dB = torch.empty_like(a.B)
    s_ld = saved_width(adapters)
    dX = dX if dX is not None else torch.empty((m, k), dtype=torch.bfloat16, device=X.device)
    ws = ws if ws is not None else workspace(m, k, n, max(s_ld, 8), max(1, len(adapters)))
    seg = native.segments_array(segments)
    ad = _adapter_array(adapters, True)
    _check_bits(mask_bits, m, k)
    name = "multi_lora_bwd" + act8_form
    st = getattr(native.lib(), name)(_ptr(dY), X_arg, _ptr(W), ad, len(adapters), seg, len(segments),
                                     int(seed) & (2**64 - 1), m, k, n, _ptr(S_saved), _ptr(mask_bits), _ptr(dX),
                                     _ptr(ws), ws.numel(), _stream(stream))
    native.check(name, st)
    return dX


_DORA_WS: dict = {}


def dora_workspace(m: int, k: int, n: int, r: int, device=None) -> torch.Tensor:
    """A cached, zero-initialised workspace for dora_fwd / dora_bwd with these sizes."""
    device = torch.device(device or torch.cuda.current_device())
    size = int(native.lib().dora_workspace_size(m, k, n, r))
    ws = _DORA_WS.get(device.index)
    if ws is None or ws.numel() < size:
        ws = torch.zeros(max(size, 256), dtype=torch.uint8, device=device)
        _DORA_WS[device.index] = ws
    return ws


def _check_bits(t, m: int, k: int) -> None:
    """The forward's keep bits handed to a backward: m x k/8 bytes, contiguous, on the device."""
    if t is None:
        return
    if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != (m, k // 8):
        raise ValueError(f"mask_bits must be a contiguous CUDA uint8 tensor of shape {(m, k // 8)}")


def _check_f32(name: str, t: torch.Tensor, n: int) -> None:
    if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{name} must be a contiguous CUDA float32 vector of {n}")


def dora_weight_norm2(W, stream=None):
    """Column norms squared of the frozen weight, fp32 (computed once per weight)."""
    k, n = W.shape
    _check_bf16("W", W, (k, n))
    out = torch.empty(n, dtype=torch.float32, device=W.device)
    native.check("dora_weight_norm2", native.lib().dora_weight_norm2(_ptr(W), k, n, _ptr(out), _stream(stream)))
    return out


def dora_fwd(X, W, A, B, mag, w_norm2, alpha: float, p: float, seed: int, *, Y=None, S_saved=None, g_saved=None,
             mask_bits=None, want_mask: bool = False, ws=None, stream=None):
    """DoRA forward: Y = g * (X W + alpha (dropout(X) A) B) with g = mag / column norms of W + alpha A B.
    Returns (Y, S_saved, g_saved, mask_bits or None)."""
    m, k = X.shape
    n = W.shape[1]
    r = A.shape[1]
    for name, t, shp in (("X", X, (m, k)), ("W", W, (k, n)), ("A", A, (k, r)), ("B", B, (r, n))):
        _check_bf16(name, t, shp)
    _check_f32("mag", mag, n)
    _check_f32("w_norm2", w_norm2, n)
    Y = Y if Y is not None else torch.empty((m, n), dtype=torch.bfloat16, device=X.device)
    S_saved = S_saved if S_saved is not None else torch.empty((m, r), dtype=torch.bfloat16, device=X.device)
    g_saved = g_saved if g_saved is not None else torch.empty(n, dtype=torch.float32, device=X.device)
    if want_mask and mask_bits is None:
        mask_bits = torch.empty((m, k // 8), dtype=torch.uint8, device=X.device)
    ws = ws if ws is not None else dora_workspace(m, k, n, r)
    st = native.lib().dora_fwd(_ptr(X), _ptr(W), _ptr(A), _ptr(B), _ptr(mag), _ptr(w_norm2), float(alpha), float(p),
                               int(seed) & (2**64 - 1), m, k, n, r, _ptr(Y), _ptr(S_saved), _ptr(g_saved),
                               _ptr(mask_bits), _ptr(ws), ws.numel(), _stream(stream))
    native.check("dora_fwd", st)
    return Y, S_saved, g_saved, mask_bits


def dora_bwd(dY, X, W, A, B, S_saved, Y, mag, g_saved, alpha: float, p: float, seed: int, *, dX=None, dA=None,
             dB=None, dmag=None, dZ=None, ws=None, stream=None, mask_bits=None):
    """DoRA backward with the column norm held constant.  Returns (dX, dA, dB, dmag).
    dZ: m x n bf16 scratch (allocated if not given).  mask_bits: optional, the keep bits dora_fwd wrote."""
    m, k = X.shape
    n = W.shape[1]
    r = A.shape[1]
    for name, t, shp in (("dY", dY, (m, n)), ("X", X, (m, k)), ("W", W, (k, n)), ("A", A, (k, r)),
                         ("B", B, (r, n)), ("S_saved", S_saved, (m, r)), ("Y", Y, (m, n))):
        _check_bf16(name, t, shp)
    _check_f32("mag", mag, n)
    _check_f32("g_saved", g_saved, n)
    dX = dX if dX is not None else torch.empty((m, k), dtype=torch.bfloat16, device=X.device)
    dA = dA if dA is not None else torch.empty((k, r), dtype=torch.bfloat16, device=X.device)
    dB = dB if dB is not None else torch.empty((r, n), dtype=torch.bfloat16, device=X.device)
    dmag = dmag if dmag is not None else torch.empty(n, dtype=torch.float32, device=X.device)
    dZ = dZ if dZ is not None else torch.empty((m, n), dtype=torch.bfloat16, device=X.device)
    _check_bf16("dZ", dZ, (m, n))
    _check_bits(mask_bits, m, k)
    ws = ws if ws is not None else dora_workspace(m, k, n, r)
    st = native.lib().dora_bwd(_ptr(dY), _ptr(X), _ptr(W), _ptr(A), _ptr(B), _ptr(S_saved), _ptr(mask_bits),
                               _ptr(Y), _ptr(mag),
                               _ptr(g_saved), float(alpha), float(p), int(seed) & (2**64 - 1), m, k, n, r, _ptr(dX),
                               _ptr(dA), _ptr(dB), _ptr(dmag), _ptr(dZ), _ptr(ws), ws.numel(), _stream(stream))
    native.check("dora_bwd", st)
    return dX, dA, dB, dmag


# ---------------------------------------------------------------------------------------------------------------
# packed causal attention
# ---------------------------------------------------------------------------------------------------------------

class _Workspaces(threading.local):
    """A host thread's cached workspaces.  A call is several launches that hand results to each other through its
    workspace, and the launches of two threads on one stream may interleave."""

    def __init__(self):
        self.cached = {}


_WORKSPACES = _Workspaces()
_GRAIN = 1 << 20   # bytes: a slightly larger batch then needs no new workspace
_WS_HEAD = 256     # bytes that are zero before a workspace's first use; the rest is scratch


class _On:
    """Allocates on the device of `t` and for the stream the call runs on: the caching allocator then hands the
    memory to nobody else before that stream is done with it."""
    __slots__ = ("index", "stream", "handle")

    def __init__(self, t: Optional[torch.Tensor], stream: Optional[torch.cuda.Stream]):
        current = torch.cuda.current_device()
        self.index = current if t is None else t.get_device()
        if self.index != current:
            raise ValueError(f"tensors are on {t.device}, the current device is cuda:{current}")
        self.stream = stream
        self.handle = _current_stream(self.index) if stream is None else stream.cuda_stream

    def empty(self, shape, dtype):
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=self.index)
        with torch.cuda.stream(self.stream):
            return torch.empty(shape, dtype=dtype, device=self.index)

    def like(self, t, rows: int, width: int, dtype):
        """A rows x width matrix; where `t` is just such a one, by the call that costs least (0.5 us of 3)."""
        if self.stream is None and type(t) is torch.Tensor and t.dtype is dtype and t.is_contiguous():
            return torch.empty_like(t)
        return self.empty((rows, width), dtype)

    def check(self, name: str, t: torch.Tensor) -> None:
        if t.get_device() != self.index:
            raise ValueError(f"{name} is on {t.device}, the call runs on cuda:{self.index}")

    def given(self, ws: torch.Tensor) -> torch.Tensor:
        """A workspace of the caller's."""
        self.check("ws", ws)
        if not ws.is_contiguous():
            raise ValueError("ws must be contiguous")
        return ws

    def capturing(self) -> bool:
        if self.stream is None:
            return torch.cuda.is_current_stream_capturing()
        with torch.cuda.stream(self.stream):
            return torch.cuda.is_current_stream_capturing()

    def workspace(self, kind: str, size: int) -> torch.Tensor:
        """The workspace of a call that was given none: cached for the calls of this thread on this stream.  A call that is
        being captured gets memory of its graph's own pool instead, zeroed by the graph before each use: a cached
        workspace may be replaced by a larger one while the graph lives, and calls outside the graph use it, too."""
        if self.capturing():
            ws = self.empty(size, torch.uint8)
            with torch.cuda.stream(self.stream):
                ws[:_WS_HEAD].zero_()
            return ws
        return self.cached(kind, size)

    def cached(self, kind: str, size: int) -> torch.Tensor:
        cached, key = _WORKSPACES.cached, (kind, self.index, self.handle)
        ws = cached.get(key)
        if ws is None or ws.numel() < size:
            ws = self.empty(-(-size // _GRAIN) * _GRAIN, torch.uint8)
            with torch.cuda.stream(self.stream):
                ws.zero_()
            cached[key] = ws
        return ws

    def public(self, kind: str, size: int) -> torch.Tensor:
        if self.capturing():
            raise RuntimeError("a captured call uses its graph's own workspace: make one before the capture and give it with ws=")
        return self.cached(kind, size)


# the handle of a device's current stream, without the objects of torch.cuda.current_stream (3 us of a call's 25)
_current_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


class AttnSeqs:
    """The sequences of a packed batch: (q_start, q_rows, k_start, k_rows) each, in row order.  Made once (1 us a sequence) and
    used by every layer's attention; a decoder whose keys grow makes one a token."""

    def __init__(self, seqs):
        self.seqs = [tuple(int(x) for x in s) for s in seqs]
        if any(len(s) != 4 for s in self.seqs):
            raise ValueError("each sequence is (q_start, q_rows, k_start, k_rows)")
        self.array = native.attn_seqs_array(self.seqs)

    def __len__(self):
        return len(self.seqs)


def attn_seqs(seqs) -> AttnSeqs:
    """A table of packed sequences from (q_start, q_rows, k_start, k_rows) tuples; (start, rows) pairs stand for
    sequences whose queries and keys are the same rows."""
    if isinstance(seqs, AttnSeqs):
        return seqs
    return AttnSeqs([(s[0], s[1], s[0], s[1]) if len(s) == 2 else s for s in seqs])


def _heads(on: _On, name: str, t: torch.Tensor, rows: int, heads: int, d: int):
    """Checks one rows x heads x head_dim operand.  Returns its strides (row, head)."""
    if t.dtype is not torch.bfloat16 or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA bfloat16 tensor")
    on.check(name, t)
    if t.shape != (rows, heads, d):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(rows, heads, d)}")
    row, head, inner = t.stride()
    if inner != 1 and d != 1:
        raise ValueError(f"the features of a head of {name} must be contiguous")
    # the stride of an extent of one is never used, and torch lets it be anything
    return row if rows > 1 else 0, head if heads > 1 else 0


# lora_attn_shape in one go: setting the fields one by one costs as much as the launch
_ATTN_SHAPE = struct.Struct("qqiiif16q")


def _attn_shape(sizes, scale, strides):
    rows, k_rows, heads, kv_heads, d = sizes
    packed = _ATTN_SHAPE.pack(rows, k_rows, heads, kv_heads, d, d ** -0.5 if scale is None else scale, *strides)
    return native.AttnShape.from_buffer_copy(packed)


_NO_STRIDES = (0,) * 8


def _attn_sizes(Q, K):
    if Q.dim() != 3 or K.dim() != 3:
        raise ValueError("Q, K and V are rows x heads x head_dim")
    rows, heads, d = Q.shape
    k_rows, kv_heads, _ = K.shape
    return rows, k_rows, heads, kv_heads, d


def _check_lse(on: _On, lse, q_rows: int, q_heads: int) -> None:
    if lse.dtype is not torch.float32 or not lse.is_cuda or not lse.is_contiguous() or lse.shape != (q_rows, q_heads):
        raise ValueError(f"lse must be a contiguous CUDA float32 tensor of shape {(q_rows, q_heads)}")
    on.check("lse", lse)


def attn_fwd(Q, K, V, seqs, *, scale: Optional[float] = None, O=None, lse=None, ws=None, stream=None):
    """Causal attention of packed sequences with grouped heads.  Q: rows x q_heads x head_dim, K and V: rows x
    kv_heads x head_dim (strided slices of a fused projection are fine); seqs: attn_seqs(...) or what it takes; scale:
    1/sqrt(head_dim) if not given.  Returns (O, lse), lse the fp32 log-sum-exp of each row and head."""
    seqs = attn_seqs(seqs)
    on = _On(Q, stream)
    sizes = rows, k_rows, heads, kv_heads, d = _attn_sizes(Q, K)
    if O is None:
        O = on.empty((rows, heads, d), torch.bfloat16)
    if lse is None:
        lse = on.empty((rows, heads), torch.float32)
    else:
        _check_lse(on, lse, rows, heads)
    shape = _attn_shape(sizes, scale, _heads(on, "Q", Q, rows, heads, d) + _heads(on, "K", K, k_rows, kv_heads, d) +
                        _heads(on, "V", V, k_rows, kv_heads, d) + _heads(on, "O", O, rows, heads, d) + _NO_STRIDES)
    ws = on.workspace("attn", attn_workspace_size(rows, heads)) if ws is None else on.given(ws)
    st = native.lib().attn_fwd(Q.data_ptr(), K.data_ptr(), V.data_ptr(), shape, seqs.array, len(seqs.seqs), O.data_ptr(),
                               lse.data_ptr(), ws.data_ptr(), ws.numel(), on.handle)
    if st:
        native.check("attn_fwd", st)
    return O, lse


def attn_bwd(dO, Q, K, V, O, lse, seqs, *, scale: Optional[float] = None, dQ=None, dK=None, dV=None, ws=None,
             stream=None):
    """Gradients of attn_fwd from dO and its O and lse.  Returns (dQ, dK, dV); dK and dV are summed over the query
    heads that share them."""
    seqs = attn_seqs(seqs)
    on = _On(Q, stream)
    sizes = rows, k_rows, heads, kv_heads, d = _attn_sizes(Q, K)
    q, kv = (rows, heads, d), (k_rows, kv_heads, d)
    if dQ is None:
        dQ = on.empty(q, torch.bfloat16)
    if dK is None:
        dK = on.empty(kv, torch.bfloat16)
    if dV is None:
        dV = on.empty(kv, torch.bfloat16)
    _check_lse(on, lse, rows, heads)
    shape = _attn_shape(sizes, scale, _heads(on, "Q", Q, *q) + _heads(on, "K", K, *kv) + _heads(on, "V", V, *kv) +
                        _heads(on, "O", O, *q) + _heads(on, "dO", dO, *q) + _heads(on, "dQ", dQ, *q) +
                        _heads(on, "dK", dK, *kv) + _heads(on, "dV", dV, *kv))
    ws = on.workspace("attn", attn_workspace_size(rows, heads)) if ws is None else on.given(ws)
    st = native.lib().attn_bwd(dO.data_ptr(), Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), lse.data_ptr(), shape,
                               seqs.array, len(seqs.seqs), dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), ws.data_ptr(),
                               ws.numel(), on.handle)
    if st:
        native.check("attn_bwd", st)
    return dQ, dK, dV


def attn_workspace_size(q_rows: int, q_heads: int) -> int:
    return int(native.lib().attn_workspace_size(q_rows, q_heads))


def attn_workspace(q_rows: int, q_heads: int, *, stream=None) -> torch.Tensor:
    """The workspace of attn_fwd and attn_bwd calls that are given none: this thread's for the stream.  A kernel whose wait
    ran out leaves its code there (lora_device_status).  A call with more rows or heads may replace it."""
    return _On(None, stream).public("attn", attn_workspace_size(q_rows, q_heads))


# ---------------------------------------------------------------------------------------------------------------
# losses on logits
# ---------------------------------------------------------------------------------------------------------------

class PrefPairs:
    """Pairs of responses: (chosen_start, rejected_start, chosen_rows, rejected_rows) each.  Made once a batch."""

    def __init__(self, pairs):
        self.pairs = [tuple(int(x) for x in q) for q in pairs]
        if any(len(q) != 4 for q in self.pairs):
            raise ValueError("each pair is (chosen_start, rejected_start, chosen_rows, rejected_rows)")
        self.array = native.pref_pairs_array(self.pairs)

    def __len__(self):
        return len(self.pairs)


def pref_pairs(pairs) -> PrefPairs:
    return pairs if isinstance(pairs, PrefPairs) else PrefPairs(pairs)


_DTYPES = {torch.bfloat16: native.BF16, torch.float32: native.F32}


def _check_rows(on: _On, name: str, t, rows: int, dtype) -> None:
    if t is None:
        return
    if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous() or t.shape != (rows,):
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} vector of {rows}")
    on.check(name, t)


def _given_f32(on: _On, name: str, t: torch.Tensor, n: int) -> torch.Tensor:
    _check_f32(name, t, n)
    on.check(name, t)
    return t


def _logits(on, logits, labels, logp, dlogits, want_grad):
    """Checks the logits and their companions.  Returns (lora_logits, logp, dlogits)."""
    if logits.dtype not in _DTYPES or not logits.is_cuda or logits.dim() != 2:
        raise TypeError("logits must be a CUDA bfloat16 or float32 matrix")
    rows, vocab = logits.shape
    if vocab > 1 and logits.stride(1) != 1:
        raise ValueError("the logits of a row must be contiguous")
    _check_rows(on, "labels", labels, rows, torch.int64)
    ld = d_ld = logits.stride(0) if rows > 1 else vocab
    if logp is None:
        logp = on.empty((rows,), torch.float32)
    else:
        _check_rows(on, "logp", logp, rows, torch.float32)
    if dlogits is None and want_grad:
        # rows as far apart as the logits' own, and as far from a 16-byte boundary (a slice may start anywhere): whole
        # vectors are then stored as they were loaded.  Else, 4096 rows of 50021 bf16 logits take 646 instead of 215 us.
        skew = logits.data_ptr() % 16 // logits.element_size()
        if ld == vocab and not skew:
            dlogits = on.empty((rows, vocab), logits.dtype)
        else:
            dlogits = on.empty((max(rows, 1) * ld + skew,), logits.dtype).as_strided((rows, vocab), (ld, 1), skew)
    elif dlogits is not None:
        if dlogits.dtype != logits.dtype or not dlogits.is_cuda or dlogits.shape != logits.shape or \
                (vocab > 1 and dlogits.stride(1) != 1):
            raise ValueError(f"dlogits must be a CUDA {logits.dtype} matrix of shape {tuple(logits.shape)}, rows contiguous")
        on.check("dlogits", dlogits)
        if rows > 1:
            d_ld = dlogits.stride(0)
    g = native.Logits(logits.data_ptr(), _ptr(dlogits), rows, vocab, ld, d_ld, labels.data_ptr(), logp.data_ptr(),
                      _DTYPES[logits.dtype], 0)
    return g, logp, dlogits


def loss_workspace_size(rows: int) -> int:
    return int(native.lib().loss_workspace_size(rows))


def loss_workspace(rows: int, *, stream=None) -> torch.Tensor:
    """The workspace of pref_loss and policy_loss calls that are given none, as attn_workspace() is attention's."""
    return _On(None, stream).public("loss", loss_workspace_size(rows))


def pref_loss(logits, labels, pairs, ref_logp=None, *, beta: float = 0.1, label_smoothing: float = 0.0,
              scale: float = 1.0, want_grad: bool = True, dlogits=None, logp=None, loss=None, margins=None, ws=None,
              stream=None):
    """Preference loss of pairs of responses (include/lora.h): scale * sum over pairs of
    -(1 - e) log sigmoid(beta margin) - e log sigmoid(-beta margin).  logits: rows x vocab, bf16 or fp32; labels: the
    token each row should predict (outside [0, vocab): the row does not count); pairs: pref_pairs(...) or what it
    takes; ref_logp: the reference policy's log p of each label.  Returns (loss, logp, margins, dlogits or None);
    dlogits=logits writes the gradient in place."""
    pairs = pref_pairs(pairs)
    on = _On(logits, stream)
    g, logp, dlogits = _logits(on, logits, labels, logp, dlogits, want_grad)
    _check_rows(on, "ref_logp", ref_logp, logits.shape[0], torch.float32)
    loss = on.empty((), torch.float32) if loss is None else _given_f32(on, "loss", loss, 1)
    margins = on.empty((len(pairs),), torch.float32) if margins is None else _given_f32(on, "margins", margins, len(pairs))
    ws = on.workspace("loss", loss_workspace_size(logits.shape[0])) if ws is None else on.given(ws)
    st = native.lib().pref_loss(g, pairs.array, len(pairs), _ptr(ref_logp), float(beta),
                                float(label_smoothing), float(scale), _ptr(loss), _ptr(margins), _ptr(ws), ws.numel(),
                                on.handle)
    native.check("pref_loss", st)
    return loss, logp, margins, dlogits


def policy_loss(logits, labels, old_logp, advantages, ref_logp=None, *, clip_low: float = 0.2, clip_high: float = 0.2,
                kl_coef: float = 0.0, scale: float = 1.0, want_grad: bool = True, dlogits=None, logp=None, loss=None,
                ws=None, stream=None):
    """Clipped policy loss with a KL term (include/lora.h): scale * sum over rows of
    -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A) + kl_coef (exp(x) - x - 1), r = exp(logp - old_logp),
    x = ref_logp - logp.  Returns (loss, logp, dlogits or None); dlogits=logits writes the gradient in place."""
    on = _On(logits, stream)
    g, logp, dlogits = _logits(on, logits, labels, logp, dlogits, want_grad)
    for name, t in (("old_logp", old_logp), ("advantages", advantages), ("ref_logp", ref_logp)):
        _check_rows(on, name, t, logits.shape[0], torch.float32)
    loss = on.empty((), torch.float32) if loss is None else _given_f32(on, "loss", loss, 1)
    ws = on.workspace("loss", loss_workspace_size(logits.shape[0])) if ws is None else on.given(ws)
    st = native.lib().policy_loss(g, _ptr(old_logp), _ptr(advantages), _ptr(ref_logp), float(clip_low),
                                  float(clip_high), float(kl_coef), float(scale), _ptr(loss), _ptr(ws), ws.numel(),
                                  on.handle)
    native.check("policy_loss", st)
    return loss, logp, dlogits


# ---------------------------------------------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------------------------------------------

ADAMW_BLOCK = 256   # values that share a scale in 8-bit states


@dataclass
class AdamWTensor:
    """One parameter with its gradient and states.  fp32 states: m and v like the parameter.  8-bit states: m and v
    (sqrt(v)) are uint8 or float8_e4m3fn codes, m_scale and v_scale fp32, one for each 256 values.  master: optional
    fp32 copy of a bf16 parameter."""
    param: torch.Tensor
    grad: torch.Tensor
    m: torch.Tensor
    v: torch.Tensor
    master: Optional[torch.Tensor] = None
    m_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None


def adamw_tensor(param, grad, *, bits: int = 32, master: bool = False) -> AdamWTensor:
    """An AdamWTensor with zero states (and, with `master`, an fp32 copy of the parameter)."""
    n, blocks = param.numel(), -(-param.numel() // ADAMW_BLOCK)
    copy = param.detach().float().clone() if master else None
    if bits == 32:
        m, v = (torch.zeros(param.shape, dtype=torch.float32, device=param.device) for _ in range(2))
        return AdamWTensor(param, grad, m, v, copy)
    if bits != 8:
        raise ValueError("bits is 8 or 32")
    m, v = (torch.zeros(n, dtype=torch.uint8, device=param.device) for _ in range(2))
    ms, vs = (torch.zeros(blocks, dtype=torch.float32, device=param.device) for _ in range(2))
    return AdamWTensor(param, grad, m, v, copy, ms, vs)


class AdamWTensors:
    """The optimiser's list of tensors, checked and laid out once for every step.  It holds their addresses: a program whose
    gradients are new tensors in each step makes the list anew (4 us a tensor), or copies them into the old ones."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        self.array = (native.AdamWTensor * max(1, len(self.tensors)))()
        given = [x for t in self.tensors for x in (t.param, t.grad, t.m, t.v, t.master, t.m_scale, t.v_scale) if x is not None]
        self.device = given[0].get_device() if given else None
        if any(x.get_device() != self.device for x in given):
            raise ValueError("the tensors of one step must be on one device")
        for a, t in zip(self.array, self.tensors):
            n = t.param.numel()
            for name in ("param", "grad"):
                x = getattr(t, name)
                if x.dtype not in _DTYPES or not x.is_cuda or not x.is_contiguous() or x.numel() != n:
                    raise ValueError(f"{name} must be a contiguous CUDA bfloat16 or float32 tensor of {n}")
            eight = t.m.dtype in (torch.uint8, torch.float8_e4m3fn)
            for name, x in (("m", t.m), ("v", t.v)):
                if x.dtype != t.m.dtype or not (eight or x.dtype == torch.float32) or not x.is_cuda or \
                        not x.is_contiguous() or x.numel() != n:
                    raise ValueError(f"{name} must be a contiguous CUDA tensor of {n}, float32 or 8-bit codes like m")
            for name, x in (("m_scale", t.m_scale), ("v_scale", t.v_scale)):
                if eight and x is None:
                    raise ValueError(f"8-bit states need {name}")
                if x is not None:
                    _check_f32(name, x, -(-n // ADAMW_BLOCK))
            if t.master is not None:
                _check_f32("master", t.master, n)
            a.param, a.grad, a.m, a.v = _ptr(t.param), _ptr(t.grad), _ptr(t.m), _ptr(t.v)
            a.m_scale, a.v_scale, a.master = _ptr(t.m_scale), _ptr(t.v_scale), _ptr(t.master)
            a.n, a.param_dtype, a.grad_dtype = n, _DTYPES[t.param.dtype], _DTYPES[t.grad.dtype]
            a.state_bits = 8 if eight else 32

    def __len__(self):
        return len(self.tensors)


def adamw_tensors(tensors) -> AdamWTensors:
    return tensors if isinstance(tensors, AdamWTensors) else AdamWTensors(tensors)


def adamw_step(tensors, *, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
               weight_decay: float = 0.0, step: int, grad_scale=None, stream=None) -> None:
    """One AdamW step (include/lora.h) over `tensors` (adamw_tensors(...) or a list of AdamWTensor), in place.
    grad_scale: optional fp32 scalar on the device that multiplies every gradient; step counts from 1."""
    tensors = adamw_tensors(tensors)
    index = torch.cuda.current_device()
    if tensors.device not in (None, index):
        raise ValueError(f"tensors are on cuda:{tensors.device}, the current device is cuda:{index}")
    if grad_scale is not None:
        _check_f32("grad_scale", grad_scale, 1)
        if grad_scale.get_device() != index:
            raise ValueError(f"grad_scale is on {grad_scale.device}, the call runs on cuda:{index}")
    st = native.lib().adamw_step(tensors.array, len(tensors), float(lr), float(beta1), float(beta2), float(eps),
                                 float(weight_decay), int(step), _ptr(grad_scale),
                                 _current_stream(index) if stream is None else stream.cuda_stream)
    native.check("adamw_step", st)


# ---------------------------------------------------------------------------------------------------------------
# activations in 8 bits
# ---------------------------------------------------------------------------------------------------------------

@dataclass
class Act8:
    """A rows x width matrix in 8 bits (include/lora.h): int8 codes, rows of the width rounded up to 32, and uint8 scales, four
    for each 128 values of a row.  Slices of whole rows of both are such a matrix, too."""
    codes: torch.Tensor
    scales: torch.Tensor
    width: int

    @property
    def shape(self):
        return torch.Size((self.codes.shape[0], self.width))

    @property
    def device(self):
        return self.codes.device


def act8(rows: int, width: int, *, stream=None) -> Act8:
    """Room for a rows x width matrix in 8 bits, on the current device."""
    on = _On(None, stream)
    return Act8(on.empty((rows, -(-width // 32) * 32), torch.int8), on.empty((rows, -(-width // 128) * 4), torch.uint8), width)


_ACT8 = struct.Struct("PP")   # lora_act8; ctypes takes the bytes for its address


def _act8_arg(on: _On, name: str, a: Act8, rows: int, width: int):
    """Checks one matrix in 8 bits.  Returns what the library takes for it."""
    codes, scales = a.codes, a.scales
    if a.width != width or codes.dtype is not torch.int8 or not codes.is_contiguous() or codes.shape != (rows, -(-width // 32) * 32):
        raise ValueError(f"{name}.codes must be a contiguous CUDA int8 tensor of shape {(rows, -(-width // 32) * 32)}, its width {width}")
    if scales.dtype is not torch.uint8 or not scales.is_contiguous() or scales.shape != (rows, -(-width // 128) * 4):
        raise ValueError(f"{name}.scales must be a contiguous CUDA uint8 tensor of shape {(rows, -(-width // 128) * 4)}")
    on.check(name, codes)
    on.check(name, scales)
    return _ACT8.pack(codes.data_ptr(), scales.data_ptr())


def _matrix(on: _On, name: str, t: torch.Tensor, rows: int, width: int, dtype) -> int:
    """Checks one rows x width operand whose rows may lie apart.  Returns its row stride."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be a CUDA {dtype} tensor")
    if t.get_device() != on.index:
        on.check(name, t)
    if t.shape != (rows, width):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(rows, width)}")
    if t.is_contiguous():
        return width
    row, inner = t.stride()
    if inner != 1 and width != 1:
        raise ValueError(f"the values of a row of {name} must be contiguous")
    return row if rows > 1 else width


def act8_store(X, out: Optional[Act8] = None, *, stream=None) -> Act8:
    """X (rows x width, bf16, rows may lie apart) in 8 bits: 32 values of a row share a power of two, codes are whole numbers up
    to 127 (include/lora.h).  Kept for a backward pass in the place of X: lora_bwd, multi_lora_bwd and norm_bwd take it."""
    on = _On(X, stream)
    if X.dim() != 2:
        raise ValueError("X is rows x width")
    rows, width = X.shape
    ld = _matrix(on, "X", X, rows, width, torch.bfloat16)
    if out is None:
        out = Act8(on.empty((rows, -(-width // 32) * 32), torch.int8), on.empty((rows, -(-width // 128) * 4), torch.uint8), width)
        arg = _ACT8.pack(out.codes.data_ptr(), out.scales.data_ptr())
    else:
        arg = _act8_arg(on, "out", out, rows, width)
    st = native.lib().act8_store(X.data_ptr(), rows, width, ld, arg, on.handle)
    if st:
        native.check("act8_store", st)
    return out


def act8_load(a: Act8, out=None, *, stream=None):
    """The bf16 values that a matrix in 8 bits stands for, exactly."""
    on = _On(a.codes, stream)
    rows, width = a.codes.shape[0], a.width
    ld = width
    if out is None:
        out = on.empty((rows, width), torch.bfloat16)
    else:
        ld = _matrix(on, "out", out, rows, width, torch.bfloat16)
    st = native.lib().act8_load(_act8_arg(on, "a", a, rows, width), rows, width, out.data_ptr(), ld, on.handle)
    if st:
        native.check("act8_load", st)
    return out


# ---------------------------------------------------------------------------------------------------------------
# norms around a block
# ---------------------------------------------------------------------------------------------------------------

# lora_norm in one go; ctypes takes the bytes for its address
_NORM = struct.Struct("10qqiiqiiqiiqiifffi")


_NO_VECTOR = (0, 0, 0)


def _vector(on: _On, name: str, t, n: int):
    """Checks one vector of weights.  Returns (address, type, 0)."""
    dtype = t.dtype
    if (dtype is not torch.bfloat16 and dtype is not torch.float32) or not t.is_contiguous() or t.shape != (n,):
        raise ValueError(f"{name} must be a contiguous CUDA bfloat16 or float32 vector of {n}")
    if t.get_device() != on.index:
        on.check(name, t)
    return t.data_ptr(), _DTYPES[dtype], 0


def _norm(on, rows, width, strides, w, post_w, gate, row_gate, eps, w_offset, res_scale, stream_dtype):
    return _NORM.pack(rows, width, *strides, *(_NO_VECTOR if w is None else _vector(on, "w", w, width)),
                      *(_NO_VECTOR if post_w is None else _vector(on, "post_w", post_w, width)),
                      *(_NO_VECTOR if gate is None else _vector(on, "gate", gate, width)),
                      *(_NO_VECTOR if row_gate is None else _vector(on, "row_gate", row_gate, rows)), eps, w_offset, res_scale,
                      _DTYPES[stream_dtype])


def norm_fwd(h, w=None, *, y=None, post_w=None, gate=None, row_gate=None, res_scale: float = 1.0, eps: float = 1e-6,
             w_offset: float = 0.0, h_out=None, x=None, x8: Optional[Act8] = None, h8: Optional[Act8] = None,
             y8: Optional[Act8] = None, stream=None):
    """A block's output joins the stream, and the stream is normed for the next block (include/lora.h):
    u = y / rms(y) (w_offset + post_w) (y itself without post_w), h' = h + res_scale gate row_gate u,
    x = h' / rms(h') (w_offset + w).  h: rows x width, bf16 or fp32; y: bf16, without it x is h's norm; w, post_w, gate: width,
    row_gate: rows, each bf16 or fp32.  x8, h8, y8 (act8(rows, width)) also receive x, h' and y in 8 bits, for the backward.
    Returns (x, h'): x None without w, h' h itself without y.  h_out=h adds in place."""
    on = _On(h, stream)
    if h.dim() != 2 or h.dtype not in _DTYPES:
        raise TypeError("h must be a CUDA bfloat16 or float32 matrix")
    rows, width = h.shape
    h_ld = width if h.is_contiguous() else _matrix(on, "h", h, rows, width, h.dtype)
    y_ld = h_out_ld = x_ld = 0
    if y is not None:
        y_ld = _matrix(on, "y", y, rows, width, torch.bfloat16)
        if h_out is None:
            h_out, h_out_ld = on.like(h, rows, width, h.dtype), width
        else:
            h_out_ld = _matrix(on, "h_out", h_out, rows, width, h.dtype)
    if x is not None:
        x_ld = _matrix(on, "x", x, rows, width, torch.bfloat16)
    elif w is not None:
        x, x_ld = on.like(h if y is None else y, rows, width, torch.bfloat16), width
    norm = _norm(on, rows, width, (h_ld, y_ld, h_out_ld, x_ld, 0, 0, 0, 0), w, post_w, gate, row_gate, eps, w_offset, res_scale,
                 h.dtype)
    if x8 is not None:
        x8 = _act8_arg(on, "x8", x8, rows, width)
    if h8 is not None:
        h8 = _act8_arg(on, "h8", h8, rows, width)
    if y8 is not None:
        y8 = _act8_arg(on, "y8", y8, rows, width)
    st = native.lib().norm_fwd(norm, h.data_ptr(), None if y is None else y.data_ptr(), None if h_out is None else h_out.data_ptr(),
                               None if x is None else x.data_ptr(), x8, h8, y8, on.handle)
    if st:
        native.check("norm_fwd", st)
    return x, h if h_out is None else h_out


class NormGrads(NamedTuple):
    """norm_bwd's results; None where the call has none."""
    dh: torch.Tensor
    dy: Optional[torch.Tensor]
    dw: Optional[torch.Tensor]
    dpost_w: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]
    drow_gate: Optional[torch.Tensor]


def norm_workspace_size(rows: int, width: int) -> int:
    return int(native.lib().norm_workspace_size(rows, width))


def norm_bwd(dx, h, w=None, *, dh=None, y=None, post_w=None, gate=None, row_gate=None, res_scale: float = 1.0,
             eps: float = 1e-6, w_offset: float = 0.0, want_weights: bool = True, dh_out=None, dy=None, dw=None, dpost_w=None,
             dgate=None, drow_gate=None, ws=None, stream=None) -> NormGrads:
    """Gradients of norm_fwd from dx and dh, those of x and h' (dh None: zero; dx and h None without w).  h: the forward's h', y its
    y, each a tensor or what act8_store or the forward kept of it in 8 bits (Act8).  Returns NormGrads: dh (of h, like
    dh or h; bf16 where there are only 8 bits, unless dh_out is fp32), dy, and with want_weights the gradients of w, post_w, gate and row_gate that were given, fp32."""
    ref = h if h is not None else dh
    if ref is None:
        raise ValueError("the gradient of x or of the stream is needed")
    on = _On(ref.codes if isinstance(ref, Act8) else ref, stream)
    rows, width = ref.shape
    # the stream's type: that of its gradient or of itself; where only 8 bits are given that of dh_out, or bf16
    typed = dh if dh is not None else dh_out if isinstance(ref, Act8) else ref
    stream_dtype = torch.bfloat16 if typed is None else typed.dtype
    if stream_dtype not in _DTYPES:
        raise TypeError("the stream is bfloat16 or float32")
    dx_ld = dh_ld = h_ld = y_ld = dy_ld = 0
    h_ptr = h8 = y_ptr = y8 = None
    if dx is not None:
        dx_ld = _matrix(on, "dx", dx, rows, width, torch.bfloat16)
    if dh is not None:
        dh_ld = _matrix(on, "dh", dh, rows, width, stream_dtype)
    if isinstance(h, Act8):
        h8 = _act8_arg(on, "h", h, rows, width)
    elif h is not None:
        h_ld, h_ptr = _matrix(on, "h", h, rows, width, stream_dtype), h.data_ptr()
    if dh_out is None:
        dh_out, dh_out_ld = on.like(dh if dh is not None else h, rows, width, stream_dtype), width
    else:
        dh_out_ld = _matrix(on, "dh_out", dh_out, rows, width, stream_dtype)
    if y is not None:
        if isinstance(y, Act8):
            y8 = _act8_arg(on, "y", y, rows, width)
        else:
            y_ld, y_ptr = _matrix(on, "y", y, rows, width, torch.bfloat16), y.data_ptr()
        if dy is None:
            dy, dy_ld = on.like(y, rows, width, torch.bfloat16), width
        else:
            dy_ld = _matrix(on, "dy", dy, rows, width, torch.bfloat16)
    norm = _norm(on, rows, width, (h_ld, y_ld, 0, 0, dx_ld, dh_ld, dh_out_ld, dy_ld), w, post_w, gate, row_gate, eps, w_offset,
                 res_scale, stream_dtype)

    if dw is not None:
        _given_f32(on, "dw", dw, width)
    if dpost_w is not None:
        _given_f32(on, "dpost_w", dpost_w, width)
    if dgate is not None:
        _given_f32(on, "dgate", dgate, width)
    if drow_gate is not None:
        _given_f32(on, "drow_gate", drow_gate, rows)
    if want_weights:
        new = (w is not None and dw is None) + (post_w is not None and dpost_w is None) + (gate is not None and dgate is None)
        if new:   # in one piece of memory
            pieces = iter((on.empty((width,), torch.float32),) if new == 1 else on.empty((new, width), torch.float32).unbind(0))
            if w is not None and dw is None:
                dw = next(pieces)
            if post_w is not None and dpost_w is None:
                dpost_w = next(pieces)
            if gate is not None and dgate is None:
                dgate = next(pieces)
        if row_gate is not None and drow_gate is None:
            drow_gate = on.empty((rows,), torch.float32)
    size = 0
    if ws is not None:
        size = on.given(ws).numel()
    elif dw is not None or dpost_w is not None or dgate is not None:
        ws = on.workspace("norm", norm_workspace_size(rows, width))
        size = ws.numel()
    st = native.lib().norm_bwd(norm, _ptr(dx), _ptr(dh), h_ptr, h8, y_ptr, y8, dh_out.data_ptr(), _ptr(dy), _ptr(dw), _ptr(dpost_w),
                               _ptr(dgate), _ptr(drow_gate), _ptr(ws), size, on.handle)
    if st:
        native.check("norm_bwd", st)
    return NormGrads(dh_out, dy, dw, dpost_w, dgate, drow_gate)


# ---------------------------------------------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------------------------------------------

class Rope:
    """The turns a position of each pair of features (include/lora.h).  Made once for a model."""

    def __init__(self, table: native.Rope):
        self.table, self.address = table, ctypes.addressof(table)


def rope_table(rot_dim: int, base: float = 10000.0, *, interleaved: bool = False, scaling: Optional[str] = None,
               factor: float = 1.0, original: float = 0.0, low: float = 1.0, high: float = 32.0,
               magnitude: float = 1.0) -> Rope:
    """Frequencies base^(-2 i / rot_dim) of the first rot_dim features of a head, in pairs (i, i + rot_dim / 2) or, interleaved,
    (2 i, 2 i + 1).  scaling for contexts longer than the trained ones: "linear" (over factor), "base" (a larger base) or "parts"
    (over factor where a pair makes fewer than `low` turns over `original` positions, as they are from `high` turns on)."""
    if scaling not in native.ROPE_SCALINGS:
        raise ValueError(f"scaling is one of {list(native.ROPE_SCALINGS)}")
    table = native.Rope()
    s = native.RopeScaling(native.ROPE_SCALINGS[scaling], magnitude, factor, original, low, high)
    native.check("rope_table", native.lib().rope_table(rot_dim, base, int(interleaved), ctypes.byref(s), ctypes.byref(table)))
    return Rope(table)


# lora_rope_shape in one go
_ROPE_SHAPE = struct.Struct("qqiiii12q")
_NO_MAT = (0, 0)


def _turned(on: _On, name: str, t: torch.Tensor, rows: int, heads: int, d: int):
    """Checks one rows x heads x head_dim operand, as _heads does.  Returns its strides (that of an extent of one is not used)."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be a CUDA bfloat16 tensor")
    if t.get_device() != on.index:
        on.check(name, t)
    if t.shape != (rows, heads, d):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(rows, heads, d)}")
    row, head, inner = t.stride()
    if inner != 1 and d != 1:
        raise ValueError(f"the features of a head of {name} must be contiguous")
    return row, head


def _positions(on: _On, positions, rows: int) -> int:
    dtype = None if positions is None else positions.dtype
    if (dtype is not torch.int64 and dtype is not torch.int32) or not positions.is_contiguous() or positions.shape != (rows,):
        raise ValueError(f"positions must be a contiguous CUDA int64 or int32 vector of {rows}")
    on.check("positions", positions)
    return 64 if dtype is torch.int64 else 32


def _rope(name, Q, K, positions, rope, Q_out, K_out, stream):
    ref = Q if Q is not None else K
    if ref is None:
        raise ValueError("Q or K is needed")
    on = _On(ref, stream)
    if ref.dim() != 3 or (K is not None and K.dim() != 3):
        raise ValueError("Q and K are rows x heads x head_dim")
    rows, _, d = ref.shape
    bits = _positions(on, positions, rows)
    hq = hk = 0
    q = qo = k = ko = _NO_MAT
    if Q is not None:
        hq = Q.shape[1]
        q = _turned(on, "Q", Q, rows, hq, d)
        if Q_out is None:
            Q_out, qo = on.empty((rows, hq, d), torch.bfloat16), (hq * d, d)
        else:
            qo = _turned(on, "Q_out", Q_out, rows, hq, d)
    if K is not None:
        hk = K.shape[1]
        k = _turned(on, "K", K, rows, hk, d)
        if K_out is None:
            K_out, ko = on.empty((rows, hk, d), torch.bfloat16), (hk * d, d)
        else:
            ko = _turned(on, "K_out", K_out, rows, hk, d)
    shape = _ROPE_SHAPE.pack(rows, 0, hq, hk, d, bits, *q, *k, 0, 0, *qo, *ko, 0, 0)
    st = getattr(native.lib(), name)(_ptr(Q), _ptr(K), positions.data_ptr(), shape, rope.address, _ptr(Q_out), _ptr(K_out), on.handle)
    if st:
        native.check(name, st)
    return Q_out, K_out


def rope_fwd(Q, K, positions, rope: Rope, *, Q_out=None, K_out=None, stream=None):
    """Q (rows x q_heads x head_dim) and K (rows x kv_heads x head_dim; either may be None) turned by the positions of their rows
    (int64 or int32, on the device).  rope: rope_table(...).  Strided slices of a fused projection are fine; Q_out=Q and K_out=K turn
    in place.  Returns (Q_out, K_out)."""
    return _rope("rope_fwd", Q, K, positions, rope, Q_out, K_out, stream)


def rope_bwd(dQ, dK, positions, rope: Rope, *, dQ_out=None, dK_out=None, stream=None):
    """Gradients of rope_fwd's Q and K from those of its outputs: the transposed rotation.  Returns (dQ_out, dK_out)."""
    return _rope("rope_bwd", dQ, dK, positions, rope, dQ_out, dK_out, stream)


def rope_append(Q, K, V, positions, slots, K_cache, V_cache, rope: Rope, *, Q_out=None, stream=None):
    """rope_fwd on the way into a cache: each row's turned K and its V go to row slots[row] (int64, on the device) of K_cache and
    V_cache (cache rows x kv_heads x head_dim; pages are runs of such rows, and attn_fwd reads one run a sequence: requests whose
    pages follow each other).  A row whose slot is outside the cache, -1 for example, is not stored; slots inside it
    must differ.  Returns the turned Q."""
    if Q is None or K is None or V is None or slots is None or K_cache is None or V_cache is None:
        raise ValueError("Q, K, V, slots, K_cache and V_cache are needed")
    on = _On(Q, stream)
    if Q.dim() != 3 or K.dim() != 3 or K_cache.dim() != 3:
        raise ValueError("Q, K, V and the caches are rows x heads x head_dim")
    rows, hq, d = Q.shape
    hk, cache_rows = K.shape[1], K_cache.shape[0]
    bits = _positions(on, positions, rows)
    _check_rows(on, "slots", slots, rows, torch.int64)
    if Q_out is None:
        Q_out, qo = on.empty((rows, hq, d), torch.bfloat16), (hq * d, d)
    else:
        qo = _turned(on, "Q_out", Q_out, rows, hq, d)
    shape = _ROPE_SHAPE.pack(
        rows, cache_rows, hq, hk, d, bits, *_turned(on, "Q", Q, rows, hq, d), *_turned(on, "K", K, rows, hk, d),
        *_turned(on, "V", V, rows, hk, d), *qo,
        *_turned(on, "K_cache", K_cache, cache_rows, hk, d), *_turned(on, "V_cache", V_cache, cache_rows, hk, d))
    st = native.lib().rope_append(Q.data_ptr(), K.data_ptr(), V.data_ptr(), positions.data_ptr(), slots.data_ptr(), shape,
                                  rope.address, Q_out.data_ptr(), K_cache.data_ptr(), V_cache.data_ptr(), on.handle)
    if st:
        native.check("rope_append", st)
    return Q_out


def lora_device_status(ws: torch.Tensor, stream=None) -> int:
    """Synchronises the stream; returns the raw device status code of the workspace (0 = fine) and clears it."""
    code = ctypes.c_int32(0)
    native.lib().lora_device_status(_ptr(ws), _stream(stream), ctypes.byref(code))
    return code.value


def lora_set_wait_limit_ns(ns: int) -> None:
    native.lib().lora_set_wait_limit_ns(int(ns))


def lora_debug_stuck_wait(ws: torch.Tensor, stream=None) -> None:
    native.check("lora_debug_stuck_wait", native.lib().lora_debug_stuck_wait(_ptr(ws), ws.numel(), _stream(stream)))
