"""Batch-invariant selected-token logprob for GB300 (sm_103a).

Thin ctypes binding over the C ABI of ``librlk.so`` (declared in
``include/rlk.h``).  Functions here only marshal torch tensors into pointers,
sizes and the current CUDA stream; every step of the computation runs in the
library's CUDA kernels.  There is no CPU fallback: if the library is missing or
the device is not compute capability 10.3 the calls raise.

The library is loaded on first use, so ``invariant_token_logprob_gb300.inputs``
(synthetic data) can be imported without it.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
from typing import NamedTuple, Optional

__all__ = ["RlkError", "lib", "logprob", "logprob_ws", "logprob_partials", "lse_merge",
           "consistency_stats", "workspace_size", "check_device_error", "take_device_errors", "vocab_tile", "row_tile",
           "logprob_backward", "backward_workspace_size", "backward_dz", "selected_token_logprob",
           "logprob_entropy", "entropy_workspace_size", "logprob_partials_shard",
           "lse_merge_sharded", "quantize_fp8_rows", "logprob_fp8", "fp8_workspace_size",
           "quantize_fp8_weight", "unpack_fp8_weight", "quantize_fp8_row_blocks",
           "quantize_fp8_weight_blocks", "logprob_fp8_block", "fp8_block_workspace_size", "consistency_stats_async",
           "stats_workspace_size", "stats_dict",
           "TokenLogprobs", "token_logprobs", "token_logprobs_backward",
           "differentiable_token_logprobs", "MAX_TOP_K",
           "quantize_w4", "dequantize_w4", "pack_w4", "unpack_w4", "linear_w4", "logprob_w4",
           "header_functions", "STAT_NAMES", "LIB_PATH", "HEADER_PATH"]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "librlk.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "rlk.h")

STAT_NAMES = ("max_abs", "mean_abs", "std_abs", "k3_mean", "sum_delta", "n_valid",
              "n_bit_mismatch", "first_mismatch")

_STATUS = {0: "RLK_OK", 1: "RLK_ERR_INVALID_ARG", 2: "RLK_ERR_ALIGNMENT",
           3: "RLK_ERR_UNSUPPORTED_DEVICE", 4: "RLK_ERR_CUDA", 5: "RLK_ERR_WORKSPACE",
           6: "RLK_ERR_TIMEOUT", 7: "RLK_ERR_TARGET_RANGE"}


class RlkError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        msg = _lib.rlk_status_string(int(status)).decode() if _lib is not None else _STATUS.get(status)
        super().__init__(f"{where}: {msg} (status {status})")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C-ABI library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'` (no CPU fallback exists)")
        L = ctypes.CDLL(LIB_PATH)
        P, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
        f32, st = ctypes.c_float, ctypes.c_int
        L.rlk_abi_version.restype = ctypes.c_int
        L.rlk_abi_version.argtypes = []
        L.rlk_status_string.restype = ctypes.c_char_p
        L.rlk_status_string.argtypes = [ctypes.c_int]
        L.rlk_row_tile.restype = ctypes.c_int
        L.rlk_row_tile.argtypes = []
        L.rlk_vocab_tile.restype = ctypes.c_int
        L.rlk_vocab_tile.argtypes = []
        L.rlk_logprob_workspace_size.restype = sz
        L.rlk_logprob_workspace_size.argtypes = [i64, i64, i64]
        L.rlk_logprob.restype = st
        L.rlk_logprob.argtypes = [P, P, P, i64, i64, i64, f32, P, P, P, P]
        L.rlk_logprob_ws.restype = st
        L.rlk_logprob_ws.argtypes = [P, P, P, i64, i64, i64, f32, P, P, P, P, sz, P]
        L.rlk_logprob_partials.restype = st
        L.rlk_logprob_partials.argtypes = [P, P, P, i64, i64, i64, f32, P, sz, P]
        L.rlk_lse_merge.restype = st
        L.rlk_lse_merge.argtypes = [P, P, i64, i64, P, P, P, P]
        L.rlk_consistency_stats.restype = st
        L.rlk_consistency_stats.argtypes = [P, P, P, i64, P, P]
        L.rlk_consistency_stats_workspace_size.restype = sz
        L.rlk_consistency_stats_workspace_size.argtypes = [i64]
        L.rlk_consistency_stats_async.restype = st
        L.rlk_consistency_stats_async.argtypes = [P, P, P, i64, P, P, sz, P]
        L.rlk_selftest_wait_timeout.restype = st
        L.rlk_selftest_wait_timeout.argtypes = [P, P, P, P, P]
        L.rlk_selftest_wait_timeout_pair.restype = st
        L.rlk_selftest_wait_timeout_pair.argtypes = [P, P, P, P, ctypes.c_int, P]
        L.rlk_check_device_error.restype = st
        L.rlk_check_device_error.argtypes = [P]
        L.rlk_take_device_errors.restype = st
        L.rlk_take_device_errors.argtypes = [P, P, P]
        L.rlk_shutdown.restype = st
        L.rlk_shutdown.argtypes = []
        L.rlk_logprob_partials_shard.restype = st
        L.rlk_logprob_partials_shard.argtypes = [P, P, P, i64, i64, i64, i64, i64, f32, P, sz, P]
        L.rlk_lse_merge_sharded.restype = st
        L.rlk_lse_merge_sharded.argtypes = [P, i64, i64, P, i64, i64, P, P, P, P]
        L.rlk_quantize_fp8_rows.restype = st
        L.rlk_quantize_fp8_rows.argtypes = [P, i64, i64, P, P, P]
        L.rlk_fp8_weight_bytes.restype = sz
        L.rlk_fp8_weight_bytes.argtypes = [i64, i64]
        L.rlk_quantize_fp8_weight.restype = st
        L.rlk_quantize_fp8_weight.argtypes = [P, i64, i64, P, P, P]
        L.rlk_logprob_fp8_workspace_size.restype = sz
        L.rlk_logprob_fp8_workspace_size.argtypes = [i64, i64, i64]
        L.rlk_logprob_fp8.restype = st
        L.rlk_logprob_fp8.argtypes = [P, P, P, P, i64, i64, i64, f32, P, P, P, P, sz, P]
        L.rlk_fp8_block_weight_scale_count.restype = sz
        L.rlk_fp8_block_weight_scale_count.argtypes = [i64, i64]
        L.rlk_quantize_fp8_row_blocks.restype = st
        L.rlk_quantize_fp8_row_blocks.argtypes = [P, i64, i64, P, P, P]
        L.rlk_quantize_fp8_weight_blocks.restype = st
        L.rlk_quantize_fp8_weight_blocks.argtypes = [P, i64, i64, P, P, P]
        L.rlk_logprob_fp8_block_workspace_size.restype = sz
        L.rlk_logprob_fp8_block_workspace_size.argtypes = [i64, i64, i64]
        L.rlk_logprob_fp8_block.restype = st
        L.rlk_logprob_fp8_block.argtypes = [P, P, P, P, i64, i64, i64, f32, P, P, P, P, sz, P]
        L.rlk_logprob_entropy_workspace_size.restype = sz
        L.rlk_logprob_entropy_workspace_size.argtypes = [i64, i64, i64]
        L.rlk_logprob_entropy.restype = st
        L.rlk_logprob_entropy.argtypes = [P, P, P, i64, i64, i64, f32, P, P, P, P, P, sz, P]
        L.rlk_logprob_backward_workspace_size.restype = sz
        L.rlk_logprob_backward_workspace_size.argtypes = [i64, i64, i64]
        L.rlk_logprob_backward_dz_ld.restype = sz
        L.rlk_logprob_backward_dz_ld.argtypes = [i64]
        L.rlk_logprob_backward.restype = st
        L.rlk_logprob_backward.argtypes = [P, P, P, P, P, i64, i64, i64, f32, P, P, ctypes.c_int,
                                           P, sz, P]
        L.rlk_token_logprobs.restype = st
        L.rlk_token_logprobs.argtypes = [P, ctypes.c_int, i64, P, P, i64, i64, i64, f32,
                                         ctypes.c_int, P, P, P, P, P, P]
        L.rlk_token_logprobs_backward.restype = st
        L.rlk_token_logprobs_backward.argtypes = [P, ctypes.c_int, i64, P, P, i64, i64, i64, f32,
                                                  P, P, P, P, P, P, P, ctypes.c_int, P, i64, P]
        L.rlk_quantize_w4.restype = st
        L.rlk_quantize_w4.argtypes = [P, ctypes.c_int, i64, i64, ctypes.c_int, P, P, P, P]
        L.rlk_dequantize_w4.restype = st
        L.rlk_dequantize_w4.argtypes = [P, P, P, ctypes.c_int, i64, i64, ctypes.c_int, P,
                                        ctypes.c_int, P]
        L.rlk_linear_w4.restype = st
        L.rlk_linear_w4.argtypes = [P, ctypes.c_int, P, P, P, i64, i64, i64, ctypes.c_int, P,
                                    ctypes.c_int, P]
        L.rlk_selftest_wait_timeout_w4.restype = st
        L.rlk_selftest_wait_timeout_w4.argtypes = [P, P, P, P, ctypes.c_int, P]
        _lib = L
    return _lib


def header_functions(path: str = HEADER_PATH) -> list:
    """Names of the functions include/rlk.h declares."""
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(rlk_[a-z_0-9]+)\s*\(", text)))


def _check(status: int, where: str):
    if status != 0:
        raise RlkError(status, where)


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def _need(t, dtype, name, ndim=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a CUDA device (no CPU path exists)")
    if t.device.index != torch.cuda.current_device():
        # the library launches on the current device; a tensor elsewhere would be
        # read through a pointer that device cannot use
        raise ValueError(f"{name} is on {t.device}, not on the current device "
                         f"cuda:{torch.cuda.current_device()} (use torch.cuda.set_device)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")


def _empty(stream, *size, **kw):
    """torch.empty in memory that belongs to `stream`, and that is not handed on either before
    work queued on the current stream by then is through with it.  A block of the current
    stream's may still be in use by work queued there when `stream` writes to it, and a
    temporary would go to that stream's next work while `stream` still uses it."""
    import torch
    with torch.cuda.stream(stream):
        t = torch.empty(*size, **kw)
    t.record_stream(torch.cuda.current_stream())
    return t


def _allocator(stream):
    """For a given stream: torch.empty if it is the current one, else _empty for it."""
    import torch
    if stream.cuda_stream == torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()):
        return torch.empty
    return functools.partial(_empty, stream)


def row_tile() -> int:
    return lib().rlk_row_tile()


def vocab_tile() -> int:
    return lib().rlk_vocab_tile()


def workspace_size(T: int, H: int, V: int) -> int:
    return lib().rlk_logprob_workspace_size(int(T), int(H), int(V))


def _check_inputs(h, W, targets):
    import torch
    _need(h, torch.bfloat16, "h", 2)
    _need(W, torch.bfloat16, "W", 2)
    _need(targets, torch.int32, "targets", 1)
    T, H = h.shape
    V, H2 = W.shape
    if H != H2 or targets.shape[0] != T:
        raise ValueError("shape mismatch: h [T,H], W [V,H], targets [T]")
    return T, H, V


def _outputs(T, device, out, stream):
    import torch
    empty = torch.empty if stream is None else _allocator(stream)
    if out is None:
        return (empty(T, dtype=torch.float32, device=device),
                empty(T, dtype=torch.float32, device=device),
                empty(T, dtype=torch.int32, device=device))
    lp, lse, am = out
    _need(lp, torch.float32, "out[0]", 1)
    _need(lse, torch.float32, "out[1]", 1)
    _need(am, torch.int32, "out[2]", 1)
    return lp, lse, am


def logprob(h, W, targets, inv_temp: float = 1.0, out=None, stream=None):
    """rlk_logprob: returns (logp f32[T], lse f32[T], argmax i32[T]) on h's device."""
    T, H, V = _check_inputs(h, W, targets)
    lp, lse, am = _outputs(T, h.device, out, stream)
    _check(lib().rlk_logprob(_ptr(h), _ptr(W), _ptr(targets), T, H, V, ctypes.c_float(inv_temp),
                             _ptr(lp), _ptr(lse), _ptr(am), _stream(stream)), "rlk_logprob")
    return lp, lse, am


def logprob_ws(h, W, targets, workspace, inv_temp: float = 1.0, out=None, stream=None):
    """rlk_logprob_ws with a caller-owned uint8 CUDA workspace tensor."""
    import torch
    T, H, V = _check_inputs(h, W, targets)
    _need(workspace, torch.uint8, "workspace", 1)
    lp, lse, am = _outputs(T, h.device, out, stream)
    _check(lib().rlk_logprob_ws(_ptr(h), _ptr(W), _ptr(targets), T, H, V, ctypes.c_float(inv_temp),
                                _ptr(lp), _ptr(lse), _ptr(am), _ptr(workspace),
                                workspace.numel(), _stream(stream)), "rlk_logprob_ws")
    return lp, lse, am


def logprob_partials(h, W, targets, inv_temp: float = 1.0, out=None, stream=None):
    """rlk_logprob_partials: returns a float32 tensor [T, NVT, 4] of {m, s, a-bits, zt}
    (view column 2 as int32 for the argmax)."""
    import torch
    empty = torch.empty if stream is None else _allocator(stream)
    T, H, V = _check_inputs(h, W, targets)
    nvt = (V + vocab_tile() - 1) // vocab_tile()
    if out is None:
        out = empty((T, nvt, 4), dtype=torch.float32, device=h.device)
    _need(out, torch.float32, "out")
    _check(lib().rlk_logprob_partials(_ptr(h), _ptr(W), _ptr(targets), T, H, V,
                                      ctypes.c_float(inv_temp), _ptr(out),
                                      out.numel() * 4, _stream(stream)), "rlk_logprob_partials")
    return out


def lse_merge(partials, targets, V: int, out=None, stream=None):
    """rlk_lse_merge over a [T, NVT, 4] float32 partial tensor."""
    import torch
    _need(partials, torch.float32, "partials", 3)
    _need(targets, torch.int32, "targets", 1)
    T = partials.shape[0]
    nvt = (V + vocab_tile() - 1) // vocab_tile()
    if partials.shape[1] != nvt or partials.shape[2] != 4 or targets.shape[0] != T:
        raise ValueError("partials must be [T, ceil(V/vocab_tile), 4] and targets [T]")
    lp, lse, am = _outputs(T, partials.device, out, stream)
    _check(lib().rlk_lse_merge(_ptr(partials), _ptr(targets), T, int(V), _ptr(lp), _ptr(lse),
                               _ptr(am), _stream(stream)), "rlk_lse_merge")
    return lp, lse, am


def consistency_stats(a, b, mask=None, stream=None):
    """rlk_consistency_stats (synchronous): a = train logp, b = rollout logp (f32 CUDA
    tensors), optional int8 mask; returns a dict keyed by STAT_NAMES."""
    import torch
    _need(a, torch.float32, "a", 1)
    _need(b, torch.float32, "b", 1)
    if a.shape != b.shape:
        raise ValueError("a and b must have the same shape")
    mp = None
    if mask is not None:
        _need(mask, torch.int8, "mask", 1)
        if mask.shape != a.shape:
            raise ValueError("mask must match a")
        mp = _ptr(mask)
    out = (ctypes.c_double * 8)()
    _check(lib().rlk_consistency_stats(_ptr(a), _ptr(b), mp, a.shape[0], out, _stream(stream)),
           "rlk_consistency_stats")
    return dict(zip(STAT_NAMES, list(out)))


def consistency_stats_async(a, b, mask=None, out=None, workspace=None, stream=None):
    """rlk_consistency_stats_async: the same statistics written, stream-ordered, into a
    float64 CUDA tensor of 8 (returned; pass `out` to reuse one).  No host sync and no
    allocation inside the library; read it with stats_dict() when needed."""
    import torch
    empty = torch.empty if stream is None else _allocator(stream)
    _need(a, torch.float32, "a", 1)
    _need(b, torch.float32, "b", 1)
    if a.shape != b.shape:
        raise ValueError("a and b must have the same shape")
    mp = None
    if mask is not None:
        _need(mask, torch.int8, "mask", 1)
        if mask.shape != a.shape:
            raise ValueError("mask must match a")
        mp = _ptr(mask)
    n = a.shape[0]
    if out is None:
        out = empty(8, dtype=torch.float64, device=a.device)
    _need(out, torch.float64, "out", 1)
    if out.numel() < 8:
        raise ValueError("out must hold 8 doubles")
    need = lib().rlk_consistency_stats_workspace_size(n)
    if workspace is None:
        workspace = empty(max(16, need), dtype=torch.uint8, device=a.device)
    _need(workspace, torch.uint8, "workspace", 1)
    _check(lib().rlk_consistency_stats_async(_ptr(a), _ptr(b), mp, n, _ptr(out), _ptr(workspace),
                                             workspace.numel(), _stream(stream)),
           "rlk_consistency_stats_async")
    return out


def stats_workspace_size(n: int) -> int:
    return lib().rlk_consistency_stats_workspace_size(int(n))


def stats_dict(out):
    """The 8 statistics of a consistency_stats_async result as a dict (synchronises)."""
    return dict(zip(STAT_NAMES, out.cpu().tolist()))


def check_device_error(stream=None):
    """Raise RlkError(RLK_ERR_TIMEOUT) if a device-side bounded wait ran out, or
    RlkError(RLK_ERR_TARGET_RANGE) if a merge saw a target >= V (synchronises)."""
    _check(lib().rlk_check_device_error(_stream(stream)), "rlk_check_device_error")


def take_device_errors(stream=None):
    """rlk_take_device_errors: read and clear the device's error records; returns
    (wait_error_bits, target_range_rows) (synchronises)."""
    bits = ctypes.c_uint32(0)
    rows = ctypes.c_uint64(0)
    _check(lib().rlk_take_device_errors(_stream(stream), ctypes.byref(bits), ctypes.byref(rows)),
           "rlk_take_device_errors")
    return int(bits.value), int(rows.value)


def backward_workspace_size(T: int, H: int, V: int) -> int:
    return lib().rlk_logprob_backward_workspace_size(int(T), int(H), int(V))


def backward_dz(workspace, T: int, V: int):
    """The bf16 [T, V] view of dz inside a backward workspace (row stride
    rlk_logprob_backward_dz_ld(V) elements)."""
    import torch
    ld = lib().rlk_logprob_backward_dz_ld(int(V))
    return workspace[:T * ld * 2].view(torch.bfloat16).view(T, ld)[:, :V]


def logprob_backward(h, W, targets, lse, grad_logp, inv_temp: float = 1.0, need_h: bool = True,
                     need_W: bool = True, grad_W=None, workspace=None, stream=None):
    """rlk_logprob_backward: returns (grad_h f32 [T,H] or None, grad_W f32 [V,H] or None,
    workspace).  Pass grad_W to accumulate into it.  dz (bf16 [T,V]) is left in the
    workspace afterwards: backward_dz(workspace, T, V)."""
    import torch
    empty = torch.empty if stream is None else _allocator(stream)
    T, H, V = _check_inputs(h, W, targets)
    _need(lse, torch.float32, "lse", 1)
    _need(grad_logp, torch.float32, "grad_logp", 1)
    gh = empty((T, H), dtype=torch.float32, device=h.device) if need_h else None
    accumulate = grad_W is not None
    if need_W and grad_W is None:
        grad_W = empty((V, H), dtype=torch.float32, device=h.device)
    if grad_W is not None:
        _need(grad_W, torch.float32, "grad_W", 2)
    if workspace is None:
        workspace = empty(backward_workspace_size(T, H, V), dtype=torch.uint8, device=h.device)
    _need(workspace, torch.uint8, "workspace", 1)
    _check(lib().rlk_logprob_backward(
        _ptr(h), _ptr(W), _ptr(targets), _ptr(lse), _ptr(grad_logp), T, H, V,
        ctypes.c_float(inv_temp), _ptr(gh) if gh is not None else None,
        _ptr(grad_W) if (need_W or accumulate) else None, 1 if accumulate else 0,
        _ptr(workspace), workspace.numel(), _stream(stream)), "rlk_logprob_backward")
    return gh, (grad_W if (need_W or accumulate) else None), workspace


def _first_derivatives(grads, inputs):
    """Gradients out of a kernel that autograd does not see.  Under create_graph they get a
    node that refuses to be differentiated: without one they would count as constants.
    (torch's once_differentiable adds its own only where the incoming gradient needs one.)"""
    import torch
    if not torch.is_grad_enabled():
        return grads

    class FirstDerivative(torch.autograd.Function):
        @staticmethod
        def forward(ctx, grad, *inputs):
            return grad.view_as(grad)

        @staticmethod
        def backward(ctx, grad):
            raise RuntimeError("this operator has first derivatives only: its gradient cannot be differentiated")

    return [None if g is None else FirstDerivative.apply(g, *inputs) for g in grads]


def _autograd_function():
    import torch

    class SelectedTokenLogprob(torch.autograd.Function):
        """logp = selected-token logprob; forward values from rlk_logprob (the
        batch-invariant kernel), gradients from rlk_logprob_backward."""

        @staticmethod
        def forward(ctx, h, W, targets, inv_temp):
            lp, lse, am = logprob(h, W, targets, inv_temp)
            ctx.save_for_backward(h, W, targets, lse)
            ctx.inv_temp = inv_temp
            return lp

        @staticmethod
        def backward(ctx, grad_lp):
            h, W, targets, lse = ctx.saved_tensors
            need_h, need_W = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
            if not (need_h or need_W):
                return None, None, None, None
            gh, gW, _ = logprob_backward(h, W, targets, lse, grad_lp.contiguous().float(),
                                         ctx.inv_temp, need_h=need_h, need_W=need_W)
            return (*_first_derivatives([gh.to(h.dtype) if need_h else None,
                                         gW.to(W.dtype) if need_W else None], [h, W, grad_lp]),
                    None, None)

    return SelectedTokenLogprob


_SelectedTokenLogprob = None


def selected_token_logprob(h, W, targets, inv_temp: float = 1.0):
    """Differentiable selected-token logprob (torch autograd): the forward is the
    batch-invariant kernel, the backward recomputes the logits on the same tiles.  First
    derivatives only."""
    global _SelectedTokenLogprob
    if _SelectedTokenLogprob is None:
        _SelectedTokenLogprob = _autograd_function()
    return _SelectedTokenLogprob.apply(h, W, targets, inv_temp)


def entropy_workspace_size(T: int, H: int, V: int) -> int:
    return lib().rlk_logprob_entropy_workspace_size(int(T), int(H), int(V))


def logprob_entropy(h, W, targets, inv_temp: float = 1.0, workspace=None, stream=None):
    """rlk_logprob_entropy: returns (logp, lse, argmax, entropy)."""
    import torch
    empty = torch.empty if stream is None else _allocator(stream)
    T, H, V = _check_inputs(h, W, targets)
    lp, lse, am = _outputs(T, h.device, None, stream)
    ent = empty(T, dtype=torch.float32, device=h.device)
    if workspace is None:
        workspace = empty(max(1, entropy_workspace_size(T, H, V)), dtype=torch.uint8,
                                device=h.device)
    _need(workspace, torch.uint8, "workspace", 1)
    _check(lib().rlk_logprob_entropy(_ptr(h), _ptr(W), _ptr(targets), T, H, V,
                                     ctypes.c_float(inv_temp), _ptr(lp), _ptr(lse), _ptr(am),
                                     _ptr(ent), _ptr(workspace), workspace.numel(),
                                     _stream(stream)), "rlk_logprob_entropy")
    return lp, lse, am, ent


def logprob_partials_shard(h, W_shard, targets, V: int, shard_begin: int, inv_temp: float = 1.0,
                           out=None, stream=None):
    """rlk_logprob_partials_shard: partials [T, ceil(rows/vocab_tile), 4] of one
    vocabulary shard W_shard = W[shard_begin : shard_begin + rows]."""
    import torch
    empty = torch.empty if stream is None else _allocator(stream)
    _need(h, torch.bfloat16, "h", 2)
    _need(W_shard, torch.bfloat16, "W_shard", 2)
    _need(targets, torch.int32, "targets", 1)
    T, H = h.shape
    rows = W_shard.shape[0]
    nvt_s = (rows + vocab_tile() - 1) // vocab_tile()
    if out is None:
        out = empty((T, nvt_s, 4), dtype=torch.float32, device=h.device)
    _need(out, torch.float32, "out")
    _check(lib().rlk_logprob_partials_shard(_ptr(h), _ptr(W_shard), _ptr(targets), T, H, int(V),
                                            int(shard_begin), rows, ctypes.c_float(inv_temp),
                                            _ptr(out), out.numel() * 4, _stream(stream)),
           "rlk_logprob_partials_shard")
    return out


def lse_merge_sharded(partials, targets, V: int, out=None, stream=None):
    """rlk_lse_merge_sharded over gathered partials [R, T, tiles_per_shard, 4]."""
    import torch
    _need(partials, torch.float32, "partials", 4)
    _need(targets, torch.int32, "targets", 1)
    R, T, nvt_s, four = partials.shape
    if four != 4 or targets.shape[0] != T:
        raise ValueError("partials must be [R, T, tiles_per_shard, 4] and targets [T]")
    lp, lse, am = _outputs(T, partials.device, out, stream)
    _check(lib().rlk_lse_merge_sharded(_ptr(partials), R, nvt_s, _ptr(targets), T, int(V),
                                       _ptr(lp), _ptr(lse), _ptr(am), _stream(stream)),
           "rlk_lse_merge_sharded")
    return lp, lse, am


def quantize_fp8_rows(x, stream=None):
    """rlk_quantize_fp8_rows: bf16 [rows, H] -> (e4m3 codes as uint8 [rows, H], f32 scales [rows])."""
    import torch
    empty = torch.empty if stream is None else _allocator(stream)
    _need(x, torch.bfloat16, "x", 2)
    rows, H = x.shape
    codes = empty((rows, H), dtype=torch.uint8, device=x.device)
    scales = empty(rows, dtype=torch.float32, device=x.device)
    _check(lib().rlk_quantize_fp8_rows(_ptr(x), rows, H, _ptr(codes), _ptr(scales),
                                       _stream(stream)), "rlk_quantize_fp8_rows")
    return codes, scales


def fp8_workspace_size(T: int, H: int, V: int) -> int:
    return lib().rlk_logprob_fp8_workspace_size(int(T), int(H), int(V))


def quantize_fp8_weight(W, out=None, stream=None):
    """rlk_quantize_fp8_weight: bf16 W [V, H] -> (tile-packed e4m3 codes as a flat uint8
    tensor, f32 scales [V]).  Pass out=(packed, scales) to reuse buffers."""
    import torch
    empty = torch.empty if stream is None else _allocator(stream)
    _need(W, torch.bfloat16, "W", 2)
    V, H = W.shape
    if out is None:
        packed = empty(lib().rlk_fp8_weight_bytes(V, H), dtype=torch.uint8, device=W.device)
        scales = empty(V, dtype=torch.float32, device=W.device)
    else:
        packed, scales = out
        _need(packed, torch.uint8, "packed", 1)
        _need(scales, torch.float32, "scales", 1)
        if packed.numel() < lib().rlk_fp8_weight_bytes(V, H) or scales.numel() < V:
            raise ValueError("out buffers too small for rlk_fp8_weight_bytes(V, H) / V")
    _check(lib().rlk_quantize_fp8_weight(_ptr(W), V, H, _ptr(packed), _ptr(scales),
                                         _stream(stream)), "rlk_quantize_fp8_weight")
    return packed, scales


def unpack_fp8_weight(packed, V: int, H: int):
    """Row-major [V, H] copy of a tile-packed fp8 weight (for inspection)."""
    bn = vocab_tile()
    nt = (V + bn - 1) // bn
    x = packed.view(nt, H // 128, bn, 128).permute(0, 2, 1, 3).reshape(nt * bn, H)
    return x[:V]


def logprob_fp8(h, W_packed, W_scales, targets, inv_temp: float = 1.0, workspace=None, out=None,
                stream=None):
    """rlk_logprob_fp8: (logp, lse, argmax) from bf16 h and a tile-packed e4m3 W
    (from quantize_fp8_weight); V = len(W_scales)."""
    import torch
    empty = torch.empty if stream is None else _allocator(stream)
    _need(h, torch.bfloat16, "h", 2)
    _need(W_packed, torch.uint8, "W_packed", 1)
    _need(W_scales, torch.float32, "W_scales", 1)
    _need(targets, torch.int32, "targets", 1)
    T, H = h.shape
    V = W_scales.shape[0]
    if W_packed.numel() < lib().rlk_fp8_weight_bytes(V, H) or targets.shape[0] != T:
        raise ValueError("W_packed must hold rlk_fp8_weight_bytes(V, H) bytes; targets [T]")
    lp, lse, am = _outputs(T, h.device, out, stream)
    if workspace is None:
        workspace = empty(max(1, fp8_workspace_size(T, H, V)), dtype=torch.uint8,
                                device=h.device)
    _need(workspace, torch.uint8, "workspace", 1)
    _check(lib().rlk_logprob_fp8(_ptr(h), _ptr(W_packed), _ptr(W_scales), _ptr(targets), T, H, V,
                                 ctypes.c_float(inv_temp), _ptr(lp), _ptr(lse), _ptr(am),
                                 _ptr(workspace), workspace.numel(), _stream(stream)),
           "rlk_logprob_fp8")
    return lp, lse, am


def quantize_fp8_row_blocks(x, stream=None):
    """rlk_quantize_fp8_row_blocks: bf16 [rows, H] -> (e4m3 codes uint8 [rows, H], f32
    scales [rows, H/128]) in 1 x 128 blocks."""
    import torch
    empty = torch.empty if stream is None else _allocator(stream)
    _need(x, torch.bfloat16, "x", 2)
    rows, H = x.shape
    codes = empty((rows, H), dtype=torch.uint8, device=x.device)
    scales = empty((rows, max(1, H // 128)), dtype=torch.float32, device=x.device)
    _check(lib().rlk_quantize_fp8_row_blocks(_ptr(x), rows, H, _ptr(codes), _ptr(scales),
                                             _stream(stream)), "rlk_quantize_fp8_row_blocks")
    return codes, scales


def quantize_fp8_weight_blocks(W, out=None, stream=None):
    """rlk_quantize_fp8_weight_blocks: bf16 W [V, H] -> (tile-packed e4m3 codes, flat
    uint8; f32 scales [ceil(V/128), H/128]) in 128 x 128 blocks."""
    import torch
    empty = torch.empty if stream is None else _allocator(stream)
    _need(W, torch.bfloat16, "W", 2)
    V, H = W.shape
    if out is None:
        packed = empty(lib().rlk_fp8_weight_bytes(V, H), dtype=torch.uint8, device=W.device)
        scales = empty(((V + 127) // 128, max(1, H // 128)), dtype=torch.float32,
                             device=W.device)
    else:
        packed, scales = out
        _need(packed, torch.uint8, "packed", 1)
        _need(scales, torch.float32, "scales")
        if (packed.numel() < lib().rlk_fp8_weight_bytes(V, H) or
                scales.numel() < lib().rlk_fp8_block_weight_scale_count(V, H)):
            raise ValueError("out buffers too small")
    _check(lib().rlk_quantize_fp8_weight_blocks(_ptr(W), V, H, _ptr(packed), _ptr(scales),
                                                _stream(stream)), "rlk_quantize_fp8_weight_blocks")
    return packed, scales


def fp8_block_workspace_size(T: int, H: int, V: int) -> int:
    return lib().rlk_logprob_fp8_block_workspace_size(int(T), int(H), int(V))


def logprob_fp8_block(h, W_packed, W_scales, targets, V: int, inv_temp: float = 1.0,
                      workspace=None, out=None, stream=None):
    """rlk_logprob_fp8_block: (logp, lse, argmax) from bf16 h and a block-quantised
    tile-packed e4m3 W with its [ceil(V/128), H/128] block scales."""
    import torch
    empty = torch.empty if stream is None else _allocator(stream)
    _need(h, torch.bfloat16, "h", 2)
    _need(W_packed, torch.uint8, "W_packed", 1)
    _need(W_scales, torch.float32, "W_scales")
    _need(targets, torch.int32, "targets", 1)
    T, H = h.shape
    if (W_packed.numel() < lib().rlk_fp8_weight_bytes(V, H) or targets.shape[0] != T or
            W_scales.numel() < lib().rlk_fp8_block_weight_scale_count(V, H)):
        raise ValueError("W_packed / W_scales too small for (V, H), or targets not [T]")
    lp, lse, am = _outputs(T, h.device, out, stream)
    if workspace is None:
        workspace = empty(max(1, fp8_block_workspace_size(T, H, V)), dtype=torch.uint8,
                                device=h.device)
    _need(workspace, torch.uint8, "workspace", 1)
    _check(lib().rlk_logprob_fp8_block(_ptr(h), _ptr(W_packed), _ptr(W_scales), _ptr(targets), T,
                                       H, int(V), ctypes.c_float(inv_temp), _ptr(lp), _ptr(lse),
                                       _ptr(am), _ptr(workspace), workspace.numel(),
                                       _stream(stream)), "rlk_logprob_fp8_block")
    return lp, lse, am


# ---------------------------------------------------------------- from logits
MAX_TOP_K = 32


class TokenLogprobs(NamedTuple):
    """Results of token_logprobs: f32 [T] logp, lse, entropy; the alternatives' ids
    (i32 [T, top_k], -1 where a row has no more tokens) and log probabilities
    (f32 [T, top_k])."""
    logp: object
    lse: object
    entropy: object
    top_ids: object
    top_logp: object


_DTYPE_CODES = {}


def _dtype_code(dtype):
    """rlk_dtype of a torch dtype (None for any other)."""
    if not _DTYPE_CODES:
        import torch
        _DTYPE_CODES.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
    return _DTYPE_CODES.get(dtype)


class _Call:
    """The checks of one call: the device its tensors must be on, found once."""
    __slots__ = ("torch", "device")

    def __init__(self):
        import torch
        self.torch = torch
        # a CUDA tensor exists only after initialisation
        self.device = torch.cuda.current_device() if torch.cuda.is_initialized() else None

    def arg(self, t, dtype, name, ndim):
        """Address of a dense tensor of this type and number of dimensions; raises as _need."""
        if not (isinstance(t, self.torch.Tensor) and t.dtype is dtype and t.dim() == ndim
                and t.get_device() == self.device and t.is_contiguous()):
            _need(t, dtype, name, ndim)
        return t.data_ptr()

    def rows(self, t, name):
        """A matrix whose rows are dense but may lie further apart than their length:
        (rlk_dtype, row stride in elements)."""
        if not isinstance(t, self.torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        code = _dtype_code(t.dtype)
        if code is None:
            raise TypeError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
        if t.dim() != 2:
            raise ValueError(f"{name} must have 2 dims")
        if t.get_device() != self.device:
            _need(t[:0].contiguous(), t.dtype, name)  # raises
        n, width = t.shape
        stride, step = t.stride()
        if (step != 1 and width > 1) or (n > 1 and stride < width):
            raise ValueError(f"{name} must have dense rows that do not overlap")
        return code, stride if n > 1 else width

    def stream(self, stream):
        if stream is not None:
            return stream.cuda_stream
        # the address alone: building the Stream object of torch.cuda.current_stream() takes
        # longer (2.9 us on Grace) than all checks of a call
        return self.torch._C._cuda_getCurrentRawStream(self.device)


def _logits_args(call, logits, targets, allowed):
    """Checked leading arguments of the two entry points, and T, V."""
    code, stride = call.rows(logits, "logits")
    i32 = call.torch.int32
    tg = call.arg(targets, i32, "targets", 1)
    T, V = logits.shape
    if targets.shape[0] != T:
        raise ValueError("shape mismatch: logits [T, V], targets [T]")
    if allowed is None:
        return (logits.data_ptr(), code, stride, tg, None, 0, T, V), T, V
    bits = call.arg(allowed, i32, "allowed", 2)
    words = allowed.shape[1]
    if allowed.shape[0] != T or words * 32 < V:
        raise ValueError("allowed must be [T, ceil(V/32)] words of allowed-token bits")
    return (logits.data_ptr(), code, stride, tg, bits, words, T, V), T, V


def token_logprobs(logits, targets, top_k: int = 0, allowed=None, inv_temp: float = 1.0, out=None,
                   stream=None):
    """rlk_token_logprobs: TokenLogprobs(logp, lse, entropy, top_ids, top_logp) of bf16,
    fp16 or fp32 logits [T, V] (dense rows, any row stride), as a tuple of tensors.

    targets i32 [T] (negative: an ignored row, logp 0); allowed: None or i32
    [T, ceil(V/32)] words of allowed-token bits (bit v % 32 of word v / 32); top_k up to
    MAX_TOP_K alternatives, the largest logits first, the lower index first among equals.
    Pass out=(logp, lse, entropy, top_ids, top_logp) to reuse tensors (the last two may
    be None for top_k = 0)."""
    call = _Call()
    torch = call.torch
    args, T, V = _logits_args(call, logits, targets, allowed)
    top_k = int(top_k)
    if not 0 <= top_k <= MAX_TOP_K:
        raise ValueError(f"top_k must lie in 0..{MAX_TOP_K}")
    f32 = torch.float32
    if out is None:
        # (five allocations: views of one cost five times as much on the host)
        dev = logits.device
        empty = torch.empty if stream is None else _allocator(stream)
        lp, lse, ent = (empty(T, dtype=f32, device=dev), empty(T, dtype=f32, device=dev),
                        empty(T, dtype=f32, device=dev))
        ids = empty((T, top_k), dtype=torch.int32, device=dev)
        top = empty((T, top_k), dtype=f32, device=dev)
        addresses = (lp.data_ptr(), lse.data_ptr(), ent.data_ptr(), ids.data_ptr(), top.data_ptr())
    else:
        lp, lse, ent, ids, top = out
        addresses = (call.arg(lp, f32, "logp", 1), call.arg(lse, f32, "lse", 1),
                     call.arg(ent, f32, "entropy", 1), None, None)
        if not lp.shape[0] == lse.shape[0] == ent.shape[0] == T:
            raise ValueError("logp, lse and entropy must be [T]")
        if top_k:
            addresses = addresses[:3] + (call.arg(ids, torch.int32, "top_ids", 2),
                                         call.arg(top, f32, "top_logp", 2))
            if ids.shape != (T, top_k) or top.shape != (T, top_k):
                raise ValueError("top_ids and top_logp must be [T, top_k]")
    _check((_lib or lib()).rlk_token_logprobs(*args, inv_temp, top_k, *addresses,
                                              call.stream(stream)), "rlk_token_logprobs")
    return TokenLogprobs(lp, lse, ent, ids, top)


def token_logprobs_backward(logits, targets, lse, entropy=None, grad_logp=None, grad_lse=None,
                            grad_entropy=None, top_ids=None, grad_top=None, allowed=None,
                            inv_temp: float = 1.0, out=None, stream=None):
    """rlk_token_logprobs_backward: the gradient with respect to the logits ([T, V] of
    their type) from those of token_logprobs' outputs (f32, each may be None).  lse and
    entropy are its outputs (entropy is needed with grad_entropy), top_ids its ids (needed
    with grad_top).  out may be a tensor to fill: `logits` itself, or one that shares no
    elements with it."""
    call = _Call()
    torch = call.torch
    empty = torch.empty if stream is None else _allocator(stream)
    args, T, V = _logits_args(call, logits, targets, allowed)
    if grad_entropy is not None and entropy is None:
        raise ValueError("grad_entropy needs entropy")
    f32 = torch.float32
    vectors = []
    for name, t in (("lse", lse), ("entropy", entropy), ("grad_logp", grad_logp),
                    ("grad_lse", grad_lse), ("grad_entropy", grad_entropy)):
        if t is None and name != "lse":
            vectors.append(None)
            continue
        vectors.append(call.arg(t, f32, name, 1))
        if t.shape[0] != T:
            raise ValueError(f"{name} must be [T]")
    top_k, ids, g_top = 0, None, None
    if grad_top is not None:
        if top_ids is None:
            raise ValueError("grad_top needs top_ids")
        ids = call.arg(top_ids, torch.int32, "top_ids", 2)
        g_top = call.arg(grad_top, f32, "grad_top", 2)
        top_k = grad_top.shape[1]
        if grad_top.shape[0] != T or top_ids.shape != grad_top.shape or top_k > MAX_TOP_K:
            raise ValueError(f"top_ids and grad_top must be [T, top_k], top_k <= {MAX_TOP_K}")
    if out is None:
        out = empty((T, V), dtype=logits.dtype, device=logits.device)
        out_stride = V
    else:
        _, out_stride = call.rows(out, "out")
        if out.dtype != logits.dtype or out.shape != logits.shape:
            raise ValueError("out must have the logits' shape and type")
    _check((_lib or lib()).rlk_token_logprobs_backward(
        *args, inv_temp, *vectors, ids, g_top, top_k, out.data_ptr(), out_stride,
        call.stream(stream)), "rlk_token_logprobs_backward")
    return out


def _token_logprobs_function():
    import torch

    class TokenLogprobsFunction(torch.autograd.Function):
        """rlk_token_logprobs with rlk_token_logprobs_backward as its gradient."""

        @staticmethod
        def forward(ctx, logits, targets, top_k, allowed, inv_temp):
            r = token_logprobs(logits, targets, top_k, allowed, inv_temp)
            ctx.save_for_backward(logits, targets, r.lse, r.entropy, r.top_ids, allowed)
            ctx.inv_temp = inv_temp
            ctx.mark_non_differentiable(r.top_ids)
            ctx.set_materialize_grads(False)
            return tuple(r)

        @staticmethod
        def backward(ctx, g_logp, g_lse, g_entropy, _, g_top):
            logits, targets, lse, entropy, ids, allowed = ctx.saved_tensors

            def dense(g):
                return None if g is None else g.contiguous().float()
            if g_logp is None and g_lse is None and g_entropy is None and g_top is None:
                return None, None, None, None, None
            if g_top is not None and g_top.shape[1] == 0:
                g_top = None
            grad = token_logprobs_backward(logits, targets, lse, entropy, dense(g_logp),
                                           dense(g_lse), dense(g_entropy),
                                           None if g_top is None else ids, dense(g_top), allowed,
                                           ctx.inv_temp)
            return (*_first_derivatives([grad], [logits, g_logp, g_lse, g_entropy, g_top]),
                    None, None, None, None)

    return TokenLogprobsFunction


_TokenLogprobsFunction = None


def differentiable_token_logprobs(logits, targets, top_k: int = 0, allowed=None,
                                  inv_temp: float = 1.0):
    """token_logprobs under torch autograd: logp, lse, entropy and top_logp carry
    gradients to the logits (top_ids does not).  First derivatives only."""
    global _TokenLogprobsFunction
    if _TokenLogprobsFunction is None:
        _TokenLogprobsFunction = _token_logprobs_function()
    return TokenLogprobs(*_TokenLogprobsFunction.apply(logits, targets, top_k, allowed, inv_temp))


# ---------------------------------------------------------------- 4-bit weights
# nibble of code k % 8 in its word: the even k in nibbles 0..3, the odd k in 4..7
_W4_NIBBLE = (0, 4, 1, 5, 2, 6, 3, 7)


def pack_w4(q):
    """Codes one to a byte (uint8 [N, K], 0..15, K % 32 == 0) as the i32 words [N, K/8] of
    linear_w4, on q's device."""
    import torch
    if q.dtype != torch.uint8 or q.dim() != 2 or q.shape[1] % 32:
        raise ValueError("q must be uint8 [N, K] with K a multiple of 32")
    words = torch.zeros(q.shape[0], q.shape[1] // 8, dtype=torch.int32, device=q.device)
    for j, nibble in enumerate(_W4_NIBBLE):
        words |= q[:, j::8].to(torch.int32) << (4 * nibble)
    return words


def unpack_w4(codes):
    """The inverse of pack_w4: uint8 [N, K] from i32 words [N, K/8]."""
    import torch
    q = torch.empty(codes.shape[0], codes.shape[1] * 8, dtype=torch.uint8, device=codes.device)
    for j, nibble in enumerate(_W4_NIBBLE):
        q[:, j::8] = ((codes >> (4 * nibble)) & 15).to(torch.uint8)
    return q


def _w4_args(call, codes, scales, zeros, group):
    """Checked (codes, scales, zeros) addresses, rlk_dtype of the scales, N, K of a 4-bit
    weight."""
    torch = call.torch
    c = call.arg(codes, torch.int32, "codes", 2)
    code = _dtype_code(scales.dtype) if isinstance(scales, torch.Tensor) else None
    if code not in (0, 1):
        raise TypeError("scales must be a bfloat16 or float16 tensor")
    s = call.arg(scales, scales.dtype, "scales", 2)
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    N, words = codes.shape
    K = words * 8
    shape = (N, (K + group - 1) // group)
    if scales.shape != shape:
        raise ValueError("scales must be [N, ceil(K/group)]")
    z = None
    if zeros is not None:
        z = call.arg(zeros, torch.uint8, "zeros", 2)
        if zeros.shape != shape:
            raise ValueError("zeros must be [N, ceil(K/group)]")
    return c, s, z, code, N, K


def quantize_w4(W, group: int = 128, asymmetric: bool = False, out=None, stream=None):
    """rlk_quantize_w4: bf16 or fp16 W [N, K] (K % 32 == 0) -> (i32 codes [N, K/8], scales
    [N, ceil(K/group)] of W's type, uint8 zero points of the same shape or None).  Pass
    out=(codes, scales, zeros) to reuse tensors."""
    call = _Call()
    torch = call.torch
    empty = torch.empty if stream is None else _allocator(stream)
    if not isinstance(W, torch.Tensor) or _dtype_code(W.dtype) not in (0, 1):
        raise TypeError("W must be a bfloat16 or float16 tensor")
    w = call.arg(W, W.dtype, "W", 2)
    N, K = W.shape
    if K % 32:
        raise ValueError("K must be a multiple of 32")
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    G = (K + group - 1) // group
    if out is None:
        codes = empty((N, K // 8), dtype=torch.int32, device=W.device)
        scales = empty((N, G), dtype=W.dtype, device=W.device)
        zeros = empty((N, G), dtype=torch.uint8, device=W.device) if asymmetric else None
    else:
        codes, scales, zeros = out
        if (zeros is not None) != bool(asymmetric):
            raise ValueError("out must hold zero points for asymmetric quantisation, and only then")
    c, s, z, code, N2, K2 = _w4_args(call, codes, scales, zeros, group)
    if (N2, K2) != (N, K) or scales.dtype != W.dtype:
        raise ValueError("out must hold codes [N, K/8] and scales of W's type")
    _check((_lib or lib()).rlk_quantize_w4(w, code, N, K, group, c, s, z, call.stream(stream)),
           "rlk_quantize_w4")
    return codes, scales, zeros


def dequantize_w4(codes, scales, zeros=None, group: int = 128, out_dtype=None, out=None,
                  stream=None):
    """rlk_dequantize_w4: the values a 4-bit weight stands for, [N, K] as the scales' type
    (default) or float32."""
    call = _Call()
    empty = call.torch.empty if stream is None else _allocator(stream)
    c, s, z, code, N, K = _w4_args(call, codes, scales, zeros, group)
    if out is None:
        out = empty((N, K), dtype=out_dtype or scales.dtype, device=codes.device)
    out_code = _dtype_code(out.dtype)
    if out_code not in (code, 2):
        raise TypeError("out_dtype must be the scales' type or float32")
    o = call.arg(out, out.dtype, "out", 2)
    if out.shape != (N, K):
        raise ValueError("out must be [N, K]")
    _check((_lib or lib()).rlk_dequantize_w4(c, s, z, code, N, K, group, o, out_code,
                                             call.stream(stream)), "rlk_dequantize_w4")
    return out


def linear_w4(x, codes, scales, zeros=None, group: int = 128, out_dtype=None, out=None,
              stream=None):
    """rlk_linear_w4: y [T, N] = x [T, K] . W^T for a 4-bit weight; x has the scales' type,
    y that type or float32 (out_dtype, default float32).  x, codes and scales start at
    16-byte boundaries, zeros at a 4-byte one."""
    call = _Call()
    empty = call.torch.empty if stream is None else _allocator(stream)
    c, s, z, code, N, K = _w4_args(call, codes, scales, zeros, group)
    a = call.arg(x, scales.dtype, "x", 2)
    T = x.shape[0]
    if x.shape[1] != K:
        raise ValueError("shape mismatch: x [T, K], codes [N, K/8]")
    if out is None:
        out = empty((T, N), dtype=out_dtype or call.torch.float32, device=x.device)
    out_code = _dtype_code(out.dtype)
    if out_code not in (code, 2):
        raise TypeError("out_dtype must be the scales' type or float32")
    o = call.arg(out, out.dtype, "out", 2)
    if out.shape != (T, N):
        raise ValueError("out must be [T, N]")
    _check((_lib or lib()).rlk_linear_w4(a, code, c, s, z, T, N, K, group, o, out_code,
                                         call.stream(stream)), "rlk_linear_w4")
    return out


def logprob_w4(h, codes, scales, targets, zeros=None, group: int = 128, top_k: int = 0,
               allowed=None, inv_temp: float = 1.0, logits=None, out=None, stream=None):
    """A decode step of a 4-bit LM head: linear_w4 into fp32 logits [T, V] (a buffer to
    reuse may be given), then token_logprobs of them.  Returns its TokenLogprobs."""
    import torch
    if logits is not None:
        _need(logits, torch.float32, "logits", 2)
    logits = linear_w4(h, codes, scales, zeros, group, out=logits, out_dtype=torch.float32,
                       stream=stream)
    return token_logprobs(logits, targets, top_k, allowed, inv_temp, out=out, stream=stream)
