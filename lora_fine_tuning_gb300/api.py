"""Tensor-level API of the LoRA linear layer (torch tensors in, torch tensors out).

The functions carry the C ABI's names and pass raw device pointers and the
current CUDA stream to it; PyTorch only allocates outputs and workspace.
"""
from __future__ import annotations

import ctypes
import struct
import threading
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

from . import native

_WS_CACHE: dict = {}


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check_bf16(name: str, t: torch.Tensor, shape) -> None:
    if t.dtype != torch.bfloat16 or not t.is_cuda:
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
    """Gradients of lora_fwd with W frozen.  Returns (dX, dA, dB).  mask_bits: optional, the keep bits
    lora_fwd wrote for the same inputs (read instead of regenerating the mask)."""
    m, k = X.shape
    n = W.shape[1]
    r = A.shape[1]
    for name, t, shp in (("dY", dY, (m, n)), ("X", X, (m, k)), ("W", W, (k, n)), ("A", A, (k, r)),
                         ("B", B, (r, n)), ("S_saved", S_saved, (m, r))):
        _check_bf16(name, t, shp)
    dX = dX if dX is not None else torch.empty((m, k), dtype=torch.bfloat16, device=X.device)
    dA = dA if dA is not None else torch.empty((k, r), dtype=torch.bfloat16, device=X.device)
    dB = dB if dB is not None else torch.empty((r, n), dtype=torch.bfloat16, device=X.device)
    _check_bits(mask_bits, m, k)
    ws = ws if ws is not None else workspace(m, k, n, r)
    st = native.lib().lora_bwd(_ptr(dY), _ptr(X), _ptr(W), _ptr(A), _ptr(B), _ptr(S_saved), _ptr(mask_bits),
                               float(alpha), float(p),
                               int(seed) & (2**64 - 1), m, k, n, r, _ptr(dX), _ptr(dA), _ptr(dB), _ptr(ws),
                               ws.numel(), _stream(stream))
    native.check("lora_bwd", st)
    return dX, dA, dB


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
    mask_bits: optional, the keep bits multi_lora_fwd wrote for the same batch."""
    m, k = X.shape
    n = W.shape[1]
    _check_bf16("dY", dY, (m, n))
    _check_bf16("X", X, (m, k))
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
    st = native.lib().multi_lora_bwd(_ptr(dY), _ptr(X), _ptr(W), ad, len(adapters), seg, len(segments),
                                     int(seed) & (2**64 - 1), m, k, n, _ptr(S_saved), _ptr(mask_bits), _ptr(dX),
                                     _ptr(ws), ws.numel(), _stream(stream))
    native.check("multi_lora_bwd", st)
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


def lora_device_status(ws: torch.Tensor, stream=None) -> int:
    """Synchronises the stream; returns the raw device status code of the workspace (0 = fine) and clears it."""
    code = ctypes.c_int32(0)
    native.lib().lora_device_status(_ptr(ws), _stream(stream), ctypes.byref(code))
    return code.value


def lora_set_wait_limit_ns(ns: int) -> None:
    native.lib().lora_set_wait_limit_ns(int(ns))


def lora_debug_stuck_wait(ws: torch.Tensor, stream=None) -> None:
    native.check("lora_debug_stuck_wait", native.lib().lora_debug_stuck_wait(_ptr(ws), ws.numel(), _stream(stream)))
