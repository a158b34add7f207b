"""Training step of the routed experts on 16-bit weights (the k3moe_rows_*, k3moe_group_*, k3moe_glu_*
and k3moe_dropout calls of include/k3moe.h): tensors in, tensors out, argument marshalling only (in
csrc/experts_py.cpp).

Tensors live on one CUDA device; matrices have contiguous rows (any row stride).  Work is enqueued on
`stream` (default: the current stream), and results are allocated there.  Nothing is recorded for autograd: a
tensor that requires gradients is refused unless gradients are off (torch.no_grad, or inside an autograd
function); a given `out` counts as written in place.  Argument errors raise K3Error;
errors found on the device (row offsets out of range, a wait that ran out) are kept in a status word
per device, read by `status()`.
"""
from __future__ import annotations

import ctypes as C
import importlib.util
import os

import torch

from . import build
from .k3moe import ERR_CODE, EXPORTS, K3Error, lib

_status = {}
_native = None


def native():
    """The native binding, set up with the library's entry points (raises if it has not been built)."""
    global _native
    if _native is None:
        path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_experts.so")
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: run __graft_entry__.build() (python latent_moe_layer_gb300/build.py)")
        if not build.binding_matches():
            raise ImportError(f"{path} was built against another Python or PyTorch: build it again")
        spec = importlib.util.spec_from_file_location(__package__ + "._experts", path)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        L = lib()
        mod.setup(K3Error, _new_status, {n: C.cast(getattr(L, n), C.c_void_p).value for n in EXPORTS})
        _native = mod
    return _native


def _new_status(dev):
    """Address of device `dev`'s status word, made at the device's first call."""
    if torch.cuda.is_current_stream_capturing():
        raise K3Error(ERR_CODE["ARG"],
                      "the first call on a device allocates its status word: make it outside a capture")
    if dev not in _status:
        _status[dev] = torch.zeros(4, dtype=torch.int32, device=f"cuda:{dev}")
        torch.cuda.synchronize(dev)
    return _status[dev].data_ptr()


def status(device=None):
    """Synchronise the device, then read and clear its status word: 0 or the first device-side error
    (a K3MOE_ERR_* code) of these calls since the last read."""
    device = torch.device("cuda") if device is None else torch.device(device)
    if device.type != "cuda":
        raise K3Error(ERR_CODE["ARG"], "device: a CUDA device")
    dev = torch.cuda.current_device() if device.index is None else device.index
    if dev not in _status:
        return 0
    torch.cuda.synchronize(dev)
    st = _status[dev]
    code = int(st[0])
    if code:
        st.zero_()
        torch.cuda.synchronize(dev)
    return code


def _call(name, stream, *args):
    """A native call, with `stream` (if given) as the current stream of its device, which is the first tensor's."""
    fn = getattr(_native or native(), name)
    if stream is None:
        return fn(*args)
    if getattr(args[0], "device", stream.device) != stream.device:
        raise K3Error(ERR_CODE["ARG"], "stream: one of the tensors' device")
    with torch.cuda.stream(stream):
        return fn(*args)


# ------------------------------------------------------------------------------------------ rows
def plan_rows(idx, n_experts, first_expert=0, stream=None):
    """Expert order of a routing: idx [T, K] int32 -> (offsets [n_experts + 1], pos [T, K]), int32.

    Expert first_expert + e owns rows offsets[e] .. offsets[e + 1]; pos is each pair's row, -1 for a
    pair of another rank's expert (or a negative idx).  Rows of one expert are in (token, slot) order."""
    return _call("plan_rows", stream, idx, n_experts, first_expert)


def gather_rows(x, pos, n_rows=None, out=None, stream=None):
    """out[pos[t, k]] = x[t] for every pos >= 0; out [n_rows, D] (default T * K rows).  Rows that no
    pair names are left as they are (uninitialised in a new `out`).  Gradient: combine_rows(dout, pos)."""
    return _call("gather_rows", stream, x, pos, n_rows, out)


def combine_rows(y, pos, weights=None, out=None, stream=None):
    """z[t] = sum_k weights[t, k] y[pos[t, k]] over pos >= 0 (weights None: all 1) -> [T, D]."""
    return _call("combine_rows", stream, y, pos, weights, out)


def combine_rows_grad(dz, y, pos, weights, out=None, stream=None):
    """Gradient of combine_rows: (dy [rows of y, D], dweights [T, K] fp32).  `out` receives dy and may be y; rows that no
    pair names are left as they are (uninitialised in a new `out`)."""
    return _call("combine_rows_grad", stream, dz, y, pos, weights, out)


# ------------------------------------------------------------------------------------------ grouped products
def group_mm(x, w, offsets, out=None, out_dtype=None, stream=None):
    """y[r] = w[e] x[r] for the rows offsets[e] <= r < offsets[e + 1] of every expert e.

    x [rows, n_in], w [E, n_out, n_in] of one 16-bit type, y [rows, n_out] of that type or fp32.  Rows of
    no expert are not written."""
    return _call("group_mm", stream, x, w, offsets, out, out_dtype)


def group_mm_grad_x(dy, w, offsets, out=None, out_dtype=None, stream=None):
    """dx[r] = w[e]^T dy[r]: the gradient of group_mm for x."""
    return _call("group_mm_grad_x", stream, dy, w, offsets, out, out_dtype)


def group_mm_grad_w(dy, x, offsets, out=None, out_dtype=None, accumulate=False, stream=None):
    """dw[e] = sum over the expert's rows of dy[r] x[r]^T: the gradient of group_mm for w, [E, n_out, n_in].

    fp32 by default (or `out`'s / `out_dtype`'s type: x's).  accumulate adds to an fp32 `out`; otherwise an
    expert without rows gets zeros."""
    return _call("group_mm_grad_w", stream, dy, x, offsets, out, out_dtype, accumulate)


# ------------------------------------------------------------------------------------------ gated unit, dropout
def glu_dropout(gu, p=0.0, seed=0, offset=0, act="silu", situ_beta=4.0, situ_linear_beta=25.0, out=None, stream=None):
    """a = dropout(act(g) u), gu [rows, 2 width] = gate columns then up columns -> [rows, width].

    The mask depends on (seed, offset, element index) alone; use another offset for every call of a step."""
    return _call("glu_dropout", stream, gu, p, seed, offset, act, situ_beta, situ_linear_beta, out)


def glu_dropout_grad(da, gu, p=0.0, seed=0, offset=0, act="silu", situ_beta=4.0, situ_linear_beta=25.0, out=None,
                     stream=None):
    """Gradient of glu_dropout (with the same p, seed and offset) -> dgu [rows, 2 width]; `out` may be gu."""
    return _call("glu_dropout_grad", stream, da, gu, p, seed, offset, act, situ_beta, situ_linear_beta, out)


def dropout(x, p, seed, offset, residual=None, out=None, stream=None):
    """dropout(x) [+ residual], any contiguous shape, fp32 or 16-bit; `out` may be x or residual.  The
    gradient for x is dropout(dout, p, seed, offset)."""
    return _call("dropout", stream, x, p, seed, offset, residual, out)
