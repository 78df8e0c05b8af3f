"""Python binding of the MoE layer forward pass (torch tensors -> C ABI).

Marshalling only: every step of the layer runs in the CUDA library.  PyTorch
provides device memory and the current stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
from typing import Optional

import torch

from . import _lib
from ._lib import MoEDebug, check, lib

ACT = {"relu": 0, "swiglu": 1}
GATE = {"switch": 0, "renorm": 1}
DTYPE = {torch.float32: 0, torch.bfloat16: 1}
HIDDEN = {"bf16x2": 0, "bf16": 1, "f16": 2, "auto": 3}
SCORING = {"softmax": 0, "sigmoid": 1}
FP8 = torch.float8_e4m3fn


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream_handle(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


@contextlib.contextmanager
def _switched(index: int, stream):
    """``index``'s device current, and on ``stream`` if one is given (torch's
    allocations too); yields the stream's handle."""
    with contextlib.ExitStack() as stack:
        stack.enter_context(torch.cuda.device(index))
        if stream is not None:
            if stream.device.index != index:
                raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
            stack.enter_context(torch.cuda.stream(stream))
        yield torch._C._cuda_getCurrentRawStream(index)


class _Here:
    """The context of a call on the current device and its current stream."""
    __slots__ = ("handle",)

    def __init__(self, handle: int):
        self.handle = handle

    def __enter__(self):
        return self.handle

    def __exit__(self, *exc):
        return False


def _on(index: int, stream):
    """A context that runs on the tensors' device and on ``stream`` (None: that
    device's current stream) and yields the stream's handle."""
    if stream is None and torch._C._cuda_getDevice() == index:
        return _Here(torch._C._cuda_getCurrentRawStream(index))
    return _switched(index, stream)


@functools.lru_cache(maxsize=4096)
def _matmul_workspace(M: int, N: int, K: int, G: int, b_rows: int) -> int:
    return int(lib().moe_matmul_fp8_scratch_bytes(M, N, K, G, b_rows))


@functools.lru_cache(maxsize=4096)
def _balance_workspace(T: int, E: int, B: int) -> int:
    return int(lib().moe_router_balance_workspace_bytes(T, E, B))


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _device_of(name, t) -> int:
    """The index of the CUDA device that a tensor is on."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: want a tensor on a CUDA device")
    return t.get_device()


def _check_tensor(name, t, index, dtype, shape=None, contiguous=True):
    """A tensor on CUDA device ``index`` of the dtype, the shape and (by default) contiguous."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.get_device() == index
            and (shape is None or t.shape == shape) and (not contiguous or t.is_contiguous())):
        return
    if _device_of(name, t) != index:
        raise ValueError(f"{name}: want a tensor on cuda:{index}, got {t.device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: want {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: want shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: want a contiguous tensor")


def _check_room(name, t, index, nbytes):
    """A contiguous tensor on CUDA device ``index`` of at least ``nbytes`` bytes, whatever its type."""
    if _device_of(name, t) != index:
        raise ValueError(f"{name}: want a tensor on cuda:{index}, got {t.device}")
    if not t.is_contiguous() or t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name}: want a contiguous tensor of {nbytes} bytes, got {t.dtype} {tuple(t.shape)}")


def _debug_struct(debug: Optional[dict], events, stream) -> Optional[MoEDebug]:
    """moe_debug of the given device tensors and stage events (None if neither)."""
    if debug is None and events is None:
        return None
    dbg = MoEDebug()
    for name, t in (debug or {}).items():
        setattr(dbg, name, _ptr(t))
    if events is not None:
        for i, ev in enumerate(events):
            if ev is not None:
                if not ev.cuda_event:  # torch creates its CUDA event lazily, on first record
                    ev.record(torch.cuda.current_stream() if stream is None else stream)
                dbg.events[i] = ev.cuda_event
    return dbg


class MoELayer:
    """One MoE layer description (E experts, top-k, d -> d_ff -> d experts).

    act: "relu" | "swiglu" (or 0 / 1); gate_mode: "switch" | "renorm" (or 0 / 1);
    capacity_factor <= 0: dropless; dtype: torch.float32 or torch.bfloat16;
    hidden (bf16 layers): "auto" (default) holds the hidden activation in fp16
    for batches of at least 1024 rows per expert and as a hi + lo pair of
    bf16 planes otherwise; "f16" and "bf16x2" force one of those; "bf16" is
    one bf16 plane (outside the parity bar; see include/moe.h).  forward_fp8
    of over 64 tokens may round the experts' gated outputs to fp16 before it
    adds them; with "bf16x2" they stay in fp32.
    n_shared: shared experts every token visits; W1, W3, W2 then hold
    num_experts + n_shared experts, the shared ones last.
    """

    def __init__(self, num_experts: int, k: int, d: int, d_ff: int, act="swiglu", gate_mode="renorm",
                 capacity_factor: float = 0.0, dtype=torch.bfloat16, hidden="auto", n_shared: int = 0):
        self.E, self.k, self.d, self.d_ff = num_experts, k, d, d_ff
        self.act = ACT[act] if isinstance(act, str) else int(act)
        self.gate_mode = GATE[gate_mode] if isinstance(gate_mode, str) else int(gate_mode)
        self.capacity_factor = float(capacity_factor)
        self.dtype = dtype
        h = ctypes.c_void_p()
        check(lib().moe_create(num_experts, k, d, d_ff, self.act, self.gate_mode, self.capacity_factor,
                               DTYPE[dtype], ctypes.byref(h)))
        self._h = h
        self._ws = None
        self._bw = None  # backward scratch
        self._last = None  # the workspace of forward_fp8, where the last call without one of the caller's was its
        self.hidden = hidden
        check(lib().moe_set_hidden_precision(h, HIDDEN[hidden]))
        self.n_shared = int(n_shared)
        check(lib().moe_set_shared_experts(h, self.n_shared))

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and _lib._LIB is not None:
            _lib._LIB.moe_destroy(h)
            self._h = None

    def capacity(self, T: int) -> Optional[int]:
        c = lib().moe_capacity(self._h, T)
        return None if c < 0 else int(c)

    def workspace_bytes(self, T: int) -> int:
        return int(lib().moe_workspace_bytes(self._h, T))

    def workspace(self, T: int, device) -> torch.Tensor:
        n = self.workspace_bytes(T)
        if self._ws is None or self._ws.numel() < n or self._ws.device != torch.device(device):
            self._ws = torch.empty(max(n, 256), dtype=torch.uint8, device=device)
        return self._ws

    def forward(self, x, W_r, b_r, W1, W3, W2, *, out=None, stats=None, workspace=None,
                debug: Optional[dict] = None, events=None, stream=None):
        """Run the layer.  Returns (y, expert_counts, dropped, aux_loss, z_loss) as device tensors.

        debug: optional dict of device tensors named like the fields of
        moe_debug (logits_in, logits_out, lse_out, topk_idx, topk_gate,
        dest_row, drop_mask, expert_offsets, y_f32).  events: optional list of
        2 * 6 torch.cuda.Event recorded around the kernel stages.
        """
        T = x.shape[0]
        dev = x.device
        y = out if out is not None else torch.empty((T, self.d), dtype=x.dtype, device=dev)
        if stats is None:
            stats = (torch.empty(self.E, dtype=torch.int32, device=dev),
                     torch.empty(1, dtype=torch.int32, device=dev),
                     torch.empty(1, dtype=torch.float32, device=dev),
                     torch.empty(1, dtype=torch.float32, device=dev))
        counts, dropped, aux, z = stats
        ws = workspace if workspace is not None else self.workspace(T, dev)
        if workspace is None:
            self._last = None  # (balance_losses reads self._ws)
        dbg = _debug_struct(debug, events, stream)
        check(lib().moe_forward(
            self._h, T, _ptr(x), _ptr(W_r), _ptr(b_r), _ptr(W1), _ptr(W3), _ptr(W2), _ptr(y),
            _ptr(counts), _ptr(dropped), _ptr(aux), _ptr(z), _ptr(ws), ws.numel(),
            None if dbg is None else ctypes.byref(dbg), _stream_handle(stream)))
        return y, counts, dropped, aux, z

    __call__ = forward

    def workspace_bytes_w4(self, T: int) -> int:
        return int(lib().moe_workspace_bytes_w4(self._h, T))

    def forward_w4(self, x, W_r, b_r, W1q, W3q, W2q, *, out=None, stats=None, workspace=None,
                   debug: Optional[dict] = None, events=None, stream=None):
        """The layer with 4-bit expert weights: W1q, W3q (None for ReLU), W2q are
        (codes, scales) pairs from quantize_int4.  Returns like forward()."""
        T = x.shape[0]
        dev = x.device
        y = out if out is not None else torch.empty((T, self.d), dtype=x.dtype, device=dev)
        if stats is None:
            stats = (torch.empty(self.E, dtype=torch.int32, device=dev),
                     torch.empty(1, dtype=torch.int32, device=dev),
                     torch.empty(1, dtype=torch.float32, device=dev),
                     torch.empty(1, dtype=torch.float32, device=dev))
        counts, dropped, aux, z = stats
        if workspace is None:
            n = self.workspace_bytes_w4(T)
            if self._ws is None or self._ws.numel() < n or self._ws.device != dev:
                self._ws = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)
            workspace = self._ws
            self._last = None
        dbg = _debug_struct(debug, events, stream)
        q3, s3 = (None, None) if W3q is None else W3q
        check(lib().moe_forward_w4(
            self._h, T, _ptr(x), _ptr(W_r), _ptr(b_r), _ptr(W1q[0]), _ptr(W1q[1]), _ptr(q3), _ptr(s3),
            _ptr(W2q[0]), _ptr(W2q[1]), _ptr(y), _ptr(counts), _ptr(dropped), _ptr(aux), _ptr(z),
            _ptr(workspace), workspace.numel(), None if dbg is None else ctypes.byref(dbg), _stream_handle(stream)))
        return y, counts, dropped, aux, z

    def workspace_bytes_fp8(self, T: int) -> int:
        return int(lib().moe_workspace_bytes_fp8(self._h, T))

    def forward_fp8(self, x, W_r, b_r, W1q, W3q, W2q, *, out=None, stats=None, workspace=None,
                    debug: Optional[dict] = None, events=None, stream=None):
        """The layer with 8-bit expert weights: W1q, W3q (None for ReLU), W2q are
        (codes, scales) pairs from quantize_fp8(W, block_rows=128); x and the
        hidden activation are quantised on the way.  Returns like forward().
        Without ``workspace`` every call takes its own from torch's allocator,
        so calls on several streams or in several captured graphs share none."""
        dev, T, G = _device_of("x", x), x.shape[0], self.E + self.n_shared
        _check_tensor("x", x, dev, torch.bfloat16, (T, self.d))
        _check_tensor("W_r", W_r, dev, torch.float32, (self.E, self.d))
        if b_r is not None:
            _check_tensor("b_r", b_r, dev, torch.float32, (self.E,))
        for name, q, rows, cols in (("W1q", W1q, self.d_ff, self.d), ("W3q", W3q, self.d_ff, self.d),
                                    ("W2q", W2q, self.d, self.d_ff)):
            if q is not None:
                _check_tensor(name + " codes", q[0], dev, FP8, (G, rows, cols))
                _check_tensor(name + " scales", q[1], dev, torch.float32, (G, _blocks(rows), _blocks(cols)))
            elif name != "W3q":
                raise ValueError(f"forward_fp8: {name} is a (codes, scales) pair")
        if out is not None:
            _check_tensor("out", out, dev, torch.bfloat16, (T, self.d))
        if stats is not None:
            for name, t, n in zip(("expert_counts", "dropped", "aux_loss", "z_loss"), stats, (self.E, 1, 1, 1)):
                _check_room(name, t, dev, 4 * n)
        if workspace is not None:
            _check_room("workspace", workspace, dev, 0)  # (its size is the C entry's to check)
        if debug is not None:
            self._check_debug(debug, T, dev)
        with _on(dev, stream) as handle:
            y = out if out is not None else torch.empty_like(x)
            if stats is None:
                stats = (W_r.new_empty(self.E, dtype=torch.int32), W_r.new_empty(1, dtype=torch.int32),
                         W_r.new_empty(1), W_r.new_empty(1))
            counts, dropped, aux, z = stats
            if workspace is None:
                self._last = None  # (let go of the last call's before asking for this one's)
                workspace = self._last = W_r.new_empty(max(self.workspace_bytes_fp8(T), 256), dtype=torch.uint8)
            dbg = _debug_struct(debug, events, stream)
            q3, s3 = (None, None) if W3q is None else W3q
            check(lib().moe_forward_fp8(
                self._h, T, _ptr(x), _ptr(W_r), _ptr(b_r), _ptr(W1q[0]), _ptr(W1q[1]), _ptr(q3), _ptr(s3),
                _ptr(W2q[0]), _ptr(W2q[1]), _ptr(y), _ptr(counts), _ptr(dropped), _ptr(aux), _ptr(z),
                _ptr(workspace), workspace.numel(), None if dbg is None else ctypes.byref(dbg), handle))
        return y, counts, dropped, aux, z

    def backward_workspace_bytes(self, T: int) -> int:
        return int(lib().moe_backward_workspace_bytes(self._h, T))

    def backward(self, x, W_r, b_r, W1, W3, W2, dy, *, aux_coef=0.0, z_coef=0.0, workspace=None,
                 bw_workspace=None, grads=None, stream=None, dlogits=None) -> dict:
        """Gradients of <dy, y> + aux_coef * aux + z_coef * z for the last
        forward on ``workspace`` (default: this layer's own), routing held
        fixed.  It does not serve forward_fp8: refused without ``workspace``
        where that was the layer's last.  dlogits [T, E] fp32: a further gradient of the router logits
        (router_balance_backward makes one).  Returns fp32 device tensors dx, dW_r, db_r (None without a
        bias), dW1, dW3 (None for ReLU), dW2; ``grads`` may supply them."""
        if workspace is None and self._last is not None:
            raise ValueError("backward: the layer's last forward was forward_fp8, which it does not serve; "
                             "run forward() again, or pass the workspace of the one that is meant")
        T, dev = x.shape[0], x.device
        ws = workspace if workspace is not None else self._ws
        if bw_workspace is None:
            n = self.backward_workspace_bytes(T)
            if self._bw is None or self._bw.numel() < n or self._bw.device != dev:
                self._bw = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)
            bw_workspace = self._bw
        if dlogits is not None:
            _check_tensor("dlogits", dlogits, x.get_device(), torch.float32, (T, self.E))
        f32 = dict(dtype=torch.float32, device=dev)
        g = dict(grads or {})
        g.setdefault("dx", torch.empty((T, self.d), **f32))
        g.setdefault("dW_r", torch.empty(W_r.shape, **f32))
        g.setdefault("db_r", None if b_r is None else torch.empty(b_r.shape, **f32))
        g.setdefault("dW1", torch.empty(W1.shape, **f32))
        g.setdefault("dW3", None if W3 is None else torch.empty(W3.shape, **f32))
        g.setdefault("dW2", torch.empty(W2.shape, **f32))
        check(lib().moe_backward_logits(
            self._h, T, _ptr(x), _ptr(W_r), _ptr(b_r), _ptr(W1), _ptr(W3), _ptr(W2), _ptr(dy),
            float(aux_coef), float(z_coef), _ptr(dlogits), _ptr(g["dx"]), _ptr(g["dW_r"]), _ptr(g["db_r"]), _ptr(g["dW1"]),
            _ptr(g["dW3"]), _ptr(g["dW2"]), _ptr(ws), 0 if ws is None else ws.numel(), _ptr(bw_workspace),
            bw_workspace.numel(), _stream_handle(stream)))
        return g

    def balance_losses(self, T: int, workspace=None, out=None, stream=None) -> torch.Tensor:
        """The alternative balance statistics of the last forward on ``workspace``
        (default: this layer's own): a device tensor [aux over all k choices,
        CV of the assignment counts, cv^2 of the mean router probabilities]."""
        ws = workspace if workspace is not None else self._last if self._last is not None else self._ws
        dev = ws.device if ws is not None else torch.device("cuda")
        out = out if out is not None else torch.empty(3, dtype=torch.float32, device=dev)
        check(lib().moe_balance_losses(self._h, T, _ptr(ws), _ptr(out), _stream_handle(stream)))
        return out

    def _debug_form(self, T: int) -> dict:
        """Shape and dtype of every output field of moe_debug."""
        E, k = self.E, self.k
        return {
            "logits_out": ((T, E), torch.float32),
            "lse_out": ((T,), torch.float32),
            "topk_idx": ((T, k), torch.int32),
            "topk_gate": ((T, k), torch.float32),
            "dest_row": ((T, k), torch.int32),
            "drop_mask": ((T, k), torch.uint8),
            "expert_offsets": ((E + 1,), torch.int32),
            "y_f32": ((T, self.d), torch.float32),
        }

    def _check_debug(self, debug: dict, T: int, index: int) -> None:
        form = dict(self._debug_form(T), logits_in=((T, self.E), torch.float32))
        for name, t in debug.items():
            if name not in form:
                raise ValueError(f"debug: no field {name}")
            if t is not None:
                shape, dtype = form[name]
                _check_room(name, t, index, math.prod(shape) * dtype.itemsize)

    def debug_buffers(self, T: int, device) -> dict:
        """Device tensors for every output field of moe_debug."""
        return {name: torch.empty(shape, dtype=dtype, device=device)
                for name, (shape, dtype) in self._debug_form(T).items()}


def quantize_int4(W: torch.Tensor, stream=None):
    """4-bit codes (int32 view of uint32 [rows][K / 8]) and bf16 scales
    [rows][K / 128] of a bf16 weight [..., K] (rows = every leading index),
    in the format of include/moe.h."""
    K = W.shape[-1]
    lead = W.shape[:-1]
    rows = W.numel() // K if K else 0
    codes = torch.empty(lead + (K // 8,), dtype=torch.int32, device=W.device)
    scales = torch.empty(lead + (K // 128,), dtype=torch.bfloat16, device=W.device)
    check(lib().moe_quantize_int4(_ptr(W.contiguous()), rows, K, _ptr(codes), _ptr(scales), _stream_handle(stream)))
    return codes, scales


def _rows_of(t: torch.Tensor):
    """(matrices, rows, columns, row stride) of a tensor read as matrices
    [rows][columns] laid out one after another, or None if it is not."""
    shape, strides = t.shape, t.stride()
    n = len(shape)
    if n < 2 or strides[-1] != 1 and shape[-1] > 1:
        return None
    rows, cols, ld = shape[-2], shape[-1], strides[-2]
    if n == 2:
        if rows <= 1:  # one row: its stride says nothing
            ld = (cols + 15) // 16 * 16
        return (1, rows, cols, ld) if ld >= cols else None
    if t.numel() == 0:
        return math.prod(shape[:-2]), rows, cols, cols
    if rows == 1:  # the matrices' stride is the row's
        ld = next((strides[d] for d in range(n - 3, -1, -1) if shape[d] != 1), (cols + 15) // 16 * 16)
    if ld < cols:
        return None
    mats, step = 1, rows * ld
    for d in range(n - 3, -1, -1):
        if shape[d] != 1 and strides[d] != step:
            return None
        mats, step = mats * shape[d], step * shape[d]
    return mats, rows, cols, ld


def quantize_fp8(x: torch.Tensor, *, block_rows: int = 1, transpose: bool = False, stream=None):
    """e4m3 codes and fp32 scales of x [..., R, K] (bf16 or fp32): one scale for
    each 128 elements of a row (block_rows 1, activations and gradients) or for
    each 128 x 128 block (block_rows 128, weights).  transpose: of x's
    transposed matrices [..., K, R].  The codes' rows start on 16-byte
    boundaries (a view of a wider tensor where the row length is no multiple
    of 16); scales are [..., ceil(rows / block_rows), ceil(columns / 128)]."""
    dev = _device_of("x", x)
    dtype = DTYPE.get(x.dtype)
    if dtype is None or x.dim() < 2:
        raise ValueError(f"quantize_fp8: x is bf16 or fp32 with at least two dimensions, got {x.dtype} {tuple(x.shape)}")
    if block_rows != 1 and block_rows != 128:
        raise ValueError("quantize_fp8: block_rows must be 1 or 128")
    with _on(dev, stream) as handle:
        form = _rows_of(x)
        if form is None:
            x = x.contiguous()
            form = _rows_of(x)
        mats, R, K, ld = form
        rows, cols = (K, R) if transpose else (R, K)
        pitch = (cols + 15) // 16 * 16
        shape, scale_shape = (rows, pitch), ((rows + block_rows - 1) // block_rows, (cols + 127) // 128)
        if x.dim() > 2:
            lead = x.shape[:-2]
            shape, scale_shape = lead + shape, lead + scale_shape
        codes = x.new_empty(shape, dtype=FP8)
        if pitch != cols:
            codes = codes[..., :cols]
        scales = x.new_empty(scale_shape, dtype=torch.float32)
        check(lib().moe_quantize_fp8(x.data_ptr(), dtype, mats, R, K, ld, block_rows, 1 if transpose else 0,
                                     codes.data_ptr(), pitch, scales.data_ptr(), handle))
    return codes, scales


def matmul_fp8(a, b, *, offsets: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16, out=None, stream=None):
    """a [M, K] times b [N, K] transposed, both (codes, scales) pairs of
    quantize_fp8: a with block_rows 1, b with 128 or 1.  With offsets (int32
    [G + 1] on the device, ascending) b is [G, N, K] and rows offsets[g] ..
    offsets[g + 1] - 1 of a are multiplied by b[g]; rows of no group are left as
    they were in ``out``.  Returns [M, N] in out_dtype (bf16 or fp32).  The same
    sizes give a row the same bits whatever stands beside it; other batch sizes
    may cut K elsewhere and change the last ones.  The product of two scales
    must be a normal fp32 number."""
    (ac, sa), (bc, sb) = a, b
    dev = _device_of("a codes", ac)
    out_kind = DTYPE.get(out_dtype)
    if out_kind is None:
        raise ValueError(f"matmul_fp8: out_dtype is bf16 or fp32, got {out_dtype}")
    _check_tensor("a codes", ac, dev, FP8, contiguous=False)
    _check_tensor("b codes", bc, dev, FP8, contiguous=False)
    sha, shb = ac.shape, bc.shape
    if len(sha) != 2 or len(shb) != (2 if offsets is None else 3) or sha[1] != shb[-1]:
        raise ValueError(f"matmul_fp8: a [M, K] and b {'[N, K]' if offsets is None else '[G, N, K]'}, got "
                         f"{tuple(sha)} and {tuple(shb)}")
    M, K = sha
    N, kb, G = shb[-2], (K + 127) // 128, 1
    _check_tensor("a scales", sa, dev, torch.float32, (M, kb))
    b_rows = 1 if sb.dim() == len(shb) and sb.shape[-2] == N and N > 1 else 128
    scale_shape = (N if b_rows == 1 else (N + 127) // 128, kb)
    if offsets is not None:
        G = shb[0]
        scale_shape = (G,) + scale_shape
        _check_tensor("offsets", offsets, dev, torch.int32, (G + 1,))
    _check_tensor("b scales", sb, dev, torch.float32, scale_shape)
    fa, fb = _rows_of(ac), _rows_of(bc)
    if fa is None or fb is None:
        raise ValueError("matmul_fp8: the codes' rows must be contiguous, their matrices one after another")
    ld_out = N
    if out is not None:
        _check_tensor("out", out, dev, out_dtype, (M, N), contiguous=False)
        fo = _rows_of(out)
        if fo is None:
            raise ValueError("matmul_fp8: out's rows must be contiguous")
        ld_out = fo[3]
    with _on(dev, stream) as handle:
        if out is None:
            out = sa.new_empty((M, N), dtype=out_dtype)
        n = _matmul_workspace(M, N, K, G, b_rows)
        ws = sa.new_empty(n, dtype=torch.uint8) if n else None
        check(lib().moe_matmul_fp8(M, N, K, G, ac.data_ptr(), fa[3], sa.data_ptr(), bc.data_ptr(), fb[3], sb.data_ptr(),
                               b_rows, None if offsets is None else offsets.data_ptr(), out.data_ptr(), out_kind, ld_out,
                               None if ws is None else ws.data_ptr(), n, handle))
    return out


def _balance_args(name, logits, k, offsets, mask, scoring):
    dev = _device_of("logits", logits)
    if logits.dim() != 2 or logits.dtype not in DTYPE or not logits.is_contiguous():
        raise ValueError(f"{name}: logits are [T, E], fp32 or bf16 and contiguous")
    if scoring not in SCORING:
        raise ValueError(f"{name}: scoring is one of {sorted(SCORING)}")
    T, E = logits.shape
    B = 1
    if offsets is not None:
        B = offsets.numel() - 1
        if B < 0:
            raise ValueError(f"{name}: offsets are [sequences + 1]")
        _check_tensor("offsets", offsets, dev, torch.int32, (B + 1,))
    if mask is not None:
        _check_tensor("mask", mask, dev, torch.uint8 if mask.dtype == torch.uint8 else torch.bool, (T,))
    return dev, T, E, B


def router_balance(logits: torch.Tensor, k: int, *, offsets: Optional[torch.Tensor] = None,
                   mask: Optional[torch.Tensor] = None, scoring: str = "softmax", stream=None):
    """(aux, z, counts, tokens) of every sequence of a packed batch from its router
    logits [T, E] (fp32 or bf16): the balance loss over all k choices, the mean
    squared log-sum-exp, the choices of each expert [sequences, E] and the
    tokens that count.  Sequence b is tokens offsets[b] .. offsets[b + 1] - 1
    (int32 on the device; None: one sequence); mask [T]: False marks padding;
    scoring: "softmax" or "sigmoid" (normalised over the experts)."""
    dev, T, E, B = _balance_args("router_balance", logits, k, offsets, mask, scoring)
    with _on(dev, stream) as handle:
        f32, i32, new = torch.float32, torch.int32, logits.new_empty
        aux, z, counts, tokens = new(B, dtype=f32), new(B, dtype=f32), new((B, E), dtype=i32), new(B, dtype=i32)
        n = _balance_workspace(T, E, B)
        ws = new(n, dtype=torch.uint8)
        check(lib().moe_router_balance(T, E, k, logits.data_ptr(), DTYPE[logits.dtype], SCORING[scoring], B,
                                   None if offsets is None else offsets.data_ptr(),
                                   None if mask is None else mask.data_ptr(), aux.data_ptr(), z.data_ptr(),
                                   counts.data_ptr(), tokens.data_ptr(), ws.data_ptr(), n, handle))
    return aux, z, counts, tokens


def router_balance_backward(logits: torch.Tensor, counts: torch.Tensor, tokens: torch.Tensor,
                            daux: Optional[torch.Tensor], dz: Optional[torch.Tensor], k: int, *,
                            offsets: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                            scoring: str = "softmax", stream=None) -> torch.Tensor:
    """The gradient [T, E] fp32 of sum_b daux_b aux_b + dz_b z_b with respect to the
    logits, from router_balance's counts and tokens (held fixed); daux and dz
    are [sequences] fp32 or None.  Zero for padding and tokens of no sequence."""
    dev, T, E, B = _balance_args("router_balance_backward", logits, k, offsets, mask, scoring)
    _check_tensor("counts", counts, dev, torch.int32, (B, E))
    _check_tensor("tokens", tokens, dev, torch.int32, (B,))
    for name, g in (("daux", daux), ("dz", dz)):
        if g is not None:
            _check_tensor(name, g, dev, torch.float32, (B,))
    with _on(dev, stream) as handle:
        dlogits = logits.new_empty((T, E), dtype=torch.float32)
        check(lib().moe_router_balance_backward(T, E, k, logits.data_ptr(), DTYPE[logits.dtype], SCORING[scoring], B,
                                                _ptr(offsets), _ptr(mask), counts.data_ptr(), tokens.data_ptr(),
                                                _ptr(daux), _ptr(dz), dlogits.data_ptr(), handle))
    return dlogits


def status(stream=None) -> None:
    """Synchronise the stream and raise MoEError if a kernel's bounded wait ran out."""
    check(lib().moe_status(_stream_handle(stream)))


def clear_status() -> None:
    check(lib().moe_clear_status())


def launch_count() -> int:
    return int(lib().moe_launch_count())


def selftest_timeout(limit_ns: int, stream=None) -> None:
    check(lib().moe_selftest_timeout(int(limit_ns), _stream_handle(stream)))
