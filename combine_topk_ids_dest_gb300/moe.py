"""PyTorch binding of the MoE operators (include/ep_moe.h): argument marshalling only.

:class:`EpRouter` makes the ``topk_ids`` and ``topk_weights`` that
``EpComm.dispatch`` takes; :class:`EpExperts` computes the experts for a few
tokens, on all experts or on the rows one rank received; :class:`EpMoeLayer`
is both, a whole layer on one GPU; :class:`Int4Linear` is a product with 4-bit
weights. All work runs in the CUDA library on
torch's current stream of the tensors' device; torch supplies device memory
and streams only. Weights are kept by reference, not copied.

Calls on one object must be ordered on the device (one stream, or streams
with events between them): it holds one call's intermediate results. Create
objects, and let them go, outside CUDA graph captures; calls can be captured.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import EpError, check

_DTYPES = {torch.bfloat16: _lib.EP_DTYPE_BF16, torch.float16: _lib.EP_DTYPE_FP16}
_SCORING = {"softmax": _lib.EP_SCORE_SOFTMAX, "sigmoid": _lib.EP_SCORE_SIGMOID}


def _device_of(t: torch.Tensor, name: str) -> torch.device:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _weight(name, t, dtype, shape, device):
    """A weight operand: contiguous `shape` of dtype on the device."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != device \
            or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on {device}")
    return t


class _Handle:
    """A handle of the C ABI and the device it lives on."""

    _destroy = ""

    def _open(self, device: torch.device):
        self._L = _lib.load()
        self.device, self._index = device, device.index  # a tensor's device: it has an index
        self._h = None

    def destroy(self) -> None:
        """Wait for the device and free the handle; repeated calls do nothing."""
        h, self._h = getattr(self, "_h", None), None
        if h is not None:
            check(getattr(self._L, self._destroy)(h))

    def __del__(self):
        try:
            self.destroy()
        except Exception:  # interpreter shutdown
            pass

    def _live(self):
        if self._h is None:
            raise EpError(_lib.EP_ERR_STATE, f"the {type(self).__name__} was destroyed")
        return self._h

    def _rows(self, x, cols, dtype, name="x"):
        """Row count and stride of an operand [rows, cols] whose rows are contiguous."""
        if x.dtype is not dtype or x.get_device() != self._index:
            raise ValueError(f"{name} is {x.dtype} on {x.device}, expected {dtype} on {self.device}")
        shape = x.shape
        if len(shape) != 2 or shape[1] != cols:
            raise ValueError(f"{name} must be a [tokens, {cols}] tensor, got {tuple(shape)}")
        if shape[0] > 0x7FFFFFFF:
            raise ValueError(f"{name} has {shape[0]} rows, at most 2^31 - 1 fit a call")
        if x.is_contiguous():
            return shape[0], cols
        if x.stride(1) != 1 and cols != 1:
            raise ValueError(f"{name} must have contiguous rows, got strides {x.stride()}")
        return shape[0], x.stride(0)

    def _out(self, out, n, cols, dtype):
        """`out`, or a new tensor, [n, cols] of dtype, and its row stride."""
        if out is None:
            return torch.empty((n, cols), dtype=dtype, device=self.device), cols
        m, stride = self._rows(out, cols, dtype, "out")
        if m != n:
            raise ValueError(f"out must have {n} rows, got {m}")
        return out, stride

    def _call(self, fn, *args):
        """fn(handle, *args, stream) on the handle's device."""
        h, index = self._h, self._index
        if h is None:
            self._live()
        if torch._C._cuda_getDevice() != index:
            with torch.cuda.device(index):
                status = fn(h, *args, torch._C._cuda_getCurrentRawStream(index))
        else:
            status = fn(h, *args, torch._C._cuda_getCurrentRawStream(index))
        if status:
            check(status)


class EpRouter(_Handle):
    """A token's top-k experts and their weights from its hidden row.

    ``weight`` [num_experts, hidden] (bf16 or fp16) gives logits
    ``x @ weight.T`` in fp32. ``scoring`` "softmax" or "sigmoid" turns them
    into scores; ``bias`` (fp32 [num_experts], optional) is added for the
    choice only, -inf masks an expert. With ``num_groups`` > 1 the choice is
    limited to the ``top_groups`` groups of experts whose two best experts add
    up highest. The chosen scores, divided by their sum if ``renormalize``,
    times ``scale``, are the weights. Choices come in descending order, ties
    go to the lowest index; slots without an expert hold id -1, weight 0.
    """

    _destroy = "ep_router_destroy"

    def __init__(self, weight: torch.Tensor, top_k: int, scoring: str = "softmax",
                 bias: Optional[torch.Tensor] = None, num_groups: int = 1, top_groups: int = 1,
                 renormalize: bool = True, scale: float = 1.0):
        device = _device_of(weight, "weight")
        if weight.dtype not in _DTYPES or weight.dim() != 2:
            raise ValueError("weight must be a bfloat16 or float16 tensor [num_experts, hidden]")
        if scoring not in _SCORING:
            raise ValueError(f"scoring {scoring!r}: use one of {sorted(_SCORING)}")
        self.num_experts, self.hidden = (int(n) for n in weight.shape)
        self.top_k, self.dtype = int(top_k), weight.dtype
        self._weight = _weight("weight", weight, weight.dtype, weight.shape, device)
        self._bias = None if bias is None else _weight("bias", bias, torch.float32, (self.num_experts,), device)
        self._open(device)
        cfg = _lib.EpRouterConfigC(self.num_experts, self.top_k, self.hidden, _DTYPES[weight.dtype],
                                   _SCORING[scoring], int(num_groups), int(top_groups), int(bool(renormalize)),
                                   float(scale), weight.data_ptr(), 0 if bias is None else bias.data_ptr())
        h = ctypes.c_void_p()
        with torch.cuda.device(device):
            check(self._L.ep_router_create(ctypes.byref(cfg), ctypes.byref(h)))
        self._h = h.value
        self._run = self._L.ep_router_run

    def _workspace(self, n: int) -> Optional[torch.Tensor]:
        """The workspace of a call with more rows than the handle has room for itself."""
        if n <= _lib.EP_MOE_MAX_TOKENS:
            return None
        size = ctypes.c_size_t(0)
        check(self._L.ep_router_workspace_size(self._live(), n, ctypes.byref(size)))
        return torch.empty(size.value, dtype=torch.uint8, device=self.device) if size.value else None

    def __call__(self, x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
        """``x`` [tokens, hidden] -> ids int32 and weights fp32, both [tokens, top_k]."""
        n, stride = self._rows(x, self.hidden, self.dtype)
        ids, weights = self._outputs(n)
        ws = self._workspace(n)
        self._call(self._run, x.data_ptr(), stride, n, ids.data_ptr(), weights.data_ptr(),
                   0 if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel())
        return ids, weights

    def _outputs(self, n: int):
        shape, device = (n, self.top_k), self.device
        return (torch.empty(shape, dtype=torch.int32, device=device),
                torch.empty(shape, dtype=torch.float32, device=device))


class Int4Weight:
    """4-bit weights ``[..., rows, cols]`` with a scale, and optionally a zero point, per ``group`` columns:
    ``w = scale * (code - zero)``, ``zero`` 8 where none are given.

    ``codes`` uint8 [..., rows, cols/2] (the low four bits are the even column),
    ``scales`` bf16 or fp16 [..., rows, cols/group], ``zeros`` uint8 of the same
    shape or None. ``group`` (32, 64 or 128) follows from the shapes.
    """

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, zeros: Optional[torch.Tensor] = None):
        device = _device_of(codes, "codes")
        if codes.dtype is not torch.uint8 or codes.dim() < 2 or scales.dtype not in _DTYPES:
            raise ValueError("codes must be a uint8 tensor [..., rows, cols/2], scales bfloat16 or float16")
        cols, n = 2 * int(codes.shape[-1]), int(scales.shape[-1]) if scales.dim() else 0
        self.group = cols // n if n and cols % n == 0 else 0
        if self.group not in (32, 64, 128):
            raise ValueError(f"{cols} columns with {n} scales: groups must be of 32, 64 or 128 columns")
        self.shape = tuple(int(d) for d in codes.shape[:-1]) + (cols,)
        shape = self.shape[:-1] + (n,)
        self.codes = _weight("codes", codes, torch.uint8, codes.shape, device)
        self.scales = _weight("scales", scales, scales.dtype, shape, device)
        self.zeros = None if zeros is None else _weight("zeros", zeros, torch.uint8, shape, device)
        self.device = device

    def pack(self, mats: int, rows: int, gate_up: bool = False) -> torch.Tensor:
        """The weight as ``mats`` matrices of ``rows`` rows, in the operators' order (ep_weight_pack)."""
        L = _lib.load()
        w = _lib.EpIntWeightC(self.codes.data_ptr(), self.scales.data_ptr(),
                              0 if self.zeros is None else self.zeros.data_ptr(), _DTYPES[self.scales.dtype], mats, rows,
                              self.shape[-1], self.group, int(gate_up))
        need = ctypes.c_size_t(0)
        check(L.ep_weight_packed_size(ctypes.byref(w), ctypes.byref(need)))
        with torch.cuda.device(self.device):
            packed = torch.empty(need.value, dtype=torch.uint8, device=self.device)
            check(L.ep_weight_pack(ctypes.byref(w), packed.data_ptr(), need.value,
                                   torch.cuda.current_stream().cuda_stream))
        return packed

    def _c(self, packed: torch.Tensor) -> "_lib.EpWeightC":
        return _lib.EpWeightC(packed.data_ptr(), self.group, int(self.zeros is not None), _DTYPES[self.scales.dtype])


class _Workspace(_Handle):
    """A handle with a workspace that torch allocates."""

    def _create(self, cfg, size, create):
        need = ctypes.c_size_t(0)
        check(size(ctypes.byref(cfg), ctypes.byref(need)))
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            self._ws = torch.empty(need.value, dtype=torch.uint8, device=self.device)
            # the handle's counters are cleared on the default stream: this stream may still use the memory,
            # and its packing of the weights has to be done before another stream's call
            torch.cuda.current_stream().synchronize()
            check(create(ctypes.byref(cfg), self._ws.data_ptr(), need.value, ctypes.byref(h)))
        self._h = h.value


class Int4Linear(_Workspace):
    """``y = x @ W.T`` for up to ``max_tokens`` (at most 64) rows, W an :class:`Int4Weight` [outputs, inputs].

    x is bf16 or fp16, y has its type. The weight is packed here once; the
    Int4Weight is not needed afterwards.
    """

    _destroy = "ep_linear_destroy"

    def __init__(self, weight: Int4Weight, max_tokens: int = 64):
        if not isinstance(weight, Int4Weight) or len(weight.shape) != 2:
            raise ValueError("weight must be an Int4Weight [outputs, inputs]")
        self.outputs, self.inputs = weight.shape
        self.max_tokens = int(max_tokens)
        self._open(weight.device)
        self._packed = weight.pack(1, self.outputs)
        cfg = _lib.EpLinearConfigC(self.inputs, self.outputs, self.max_tokens, weight._c(self._packed))
        self._create(cfg, self._L.ep_linear_workspace_size, self._L.ep_linear_create)
        self._run = self._L.ep_linear_run

    def __call__(self, x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """``x`` [tokens, inputs] -> [tokens, outputs] (``out`` if given)."""
        dtype = x.dtype
        if dtype not in _DTYPES:
            raise ValueError(f"x is {dtype}, expected bfloat16 or float16")
        n, stride = self._rows(x, self.inputs, dtype)
        out, out_stride = self._out(out, n, self.outputs, dtype)
        self._call(self._run, _DTYPES[dtype], x.data_ptr(), stride, n, out.data_ptr(), out_stride)
        return out


class EpExperts(_Workspace):
    """The experts of an MoE layer for up to ``max_tokens`` (at most 64) tokens.

    ``gate_up`` [experts, 2*intermediate, hidden] (gate rows, then up rows) and
    ``down`` [experts, hidden, intermediate] are both bf16 tensors (kept by
    reference) or both :class:`Int4Weight` (packed here once, not needed
    afterwards). The experts are the global ids ``first_expert ..``; ids
    outside them are skipped, so one rank's experts run on the rows
    ``EpComm.dispatch`` delivered and write the rows ``EpComm.combine`` adds up.
    A receive buffer's slots all count, empty ones too: ``ep_size *
    tokens_per_rank`` is at most 64 there.
    """

    _destroy = "ep_experts_destroy"

    def __init__(self, gate_up, down, top_k: int, max_tokens: int = 64, first_expert: int = 0):
        packed = isinstance(gate_up, Int4Weight)
        if packed != isinstance(down, Int4Weight):
            raise ValueError("gate_up and down must both be tensors or both Int4Weight")
        device = gate_up.device if packed else _device_of(gate_up, "gate_up")
        if len(gate_up.shape) != 3 or gate_up.shape[1] % 2:
            raise ValueError("gate_up must be [experts, 2*intermediate, hidden]")
        E, I2, H = (int(n) for n in gate_up.shape)
        self.num_experts, self.intermediate, self.hidden = E, I2 // 2, H
        self.top_k, self.max_tokens, self.first_expert = int(top_k), int(max_tokens), int(first_expert)
        self.dtype = torch.bfloat16
        self._open(device)
        if packed:
            if down.shape != (E, H, I2 // 2) or down.device != device:
                raise ValueError(f"down must be {(E, H, I2 // 2)} on {device}, got {down.shape} on {down.device}")
            self._w = (gate_up.pack(2 * E, I2 // 2, gate_up=True), down.pack(E, H))
            cw = gate_up._c(self._w[0]), down._c(self._w[1])
        else:
            self._w = (_weight("gate_up", gate_up, torch.bfloat16, (E, I2, H), device),
                       _weight("down", down, torch.bfloat16, (E, H, I2 // 2), device))
            cw = tuple(_lib.EpWeightC(w.data_ptr(), 0, 0, 0) for w in self._w)
        cfg = _lib.EpExpertsConfigC(E, self.first_expert, self.top_k, H, I2 // 2, self.max_tokens, *cw)
        self._create(cfg, self._L.ep_experts_workspace_size, self._L.ep_experts_create)
        self._run = self._L.ep_experts_run

    def __call__(self, x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """``x`` bf16 [tokens, hidden], ``topk_ids`` int32 and ``topk_weights`` fp32 [tokens, top_k] ->
        the weighted sum of each token's experts, bf16 [tokens, hidden] (``out`` if given)."""
        n, stride = self._rows(x, self.hidden, self.dtype)
        for name, t, dtype in (("topk_ids", topk_ids, torch.int32), ("topk_weights", topk_weights, torch.float32)):
            if t.dtype is not dtype or t.get_device() != self._index or tuple(t.shape) != (n, self.top_k) \
                    or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dtype} tensor [{n}, {self.top_k}] on {self.device}")
        out, out_stride = self._out(out, n, self.hidden, self.dtype)
        self._call(self._run, x.data_ptr(), stride, topk_ids.data_ptr(), topk_weights.data_ptr(), n,
                   out.data_ptr(), out_stride)
        return out


class EpMoeLayer:
    """A whole MoE layer for a few tokens on one GPU: router, then experts."""

    def __init__(self, router: EpRouter, experts: EpExperts):
        if router.hidden != experts.hidden or router.top_k != experts.top_k or router.dtype is not experts.dtype \
                or router.device != experts.device:
            raise ValueError("router and experts must have the same hidden size, top_k, dtype and device")
        self.router, self.experts = router, experts
        self._run = experts._L.ep_layer_run

    def __call__(self, x: torch.Tensor, out: Optional[torch.Tensor] = None):
        """``x`` bf16 [tokens, hidden] -> (y bf16 [tokens, hidden] (``out`` if given), ids int32 and
        weights fp32 [tokens, top_k])."""
        router, experts = self.router, self.experts
        n, stride = router._rows(x, router.hidden, router.dtype)
        ids, weights = router._outputs(n)
        out, out_stride = experts._out(out, n, experts.hidden, experts.dtype)
        router._call(self._run, experts._live(), x.data_ptr(), stride, n, ids.data_ptr(), weights.data_ptr(),
                     out.data_ptr(), out_stride)
        return out, ids, weights
