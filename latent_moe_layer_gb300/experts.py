"""Training step of the routed experts on 16-bit weights (the k3moe_rows_*, k3moe_group_*, k3moe_glu_*,
k3moe_quant8_*, k3moe_*norm* and k3moe_dropout calls of include/k3moe.h): tensors in, tensors out, argument
marshalling only (in csrc/experts_py.cpp).

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


# ------------------------------------------------------------------------------------------ gated block
def group_glu(x, w, offsets, act="silu", situ_beta=4.0, situ_linear_beta=25.0, out=None, stream=None):
    """a[r] = act(Wg x[r]) (Wu x[r]) for every expert's rows: both projections and the unit in one pass.

    x [rows, n_in], w [E, 2 width, n_in] = gate rows then up rows, of one 16-bit type -> a [rows, width].  The
    projections are not rounded on the way (group_mm then glu_dropout rounds them, and draws a dropout mask).  Nothing is
    kept for the gradient but x: less memory, and more time, than group_mm, glu_dropout and glu_dropout_grad."""
    return _call("group_glu", stream, x, w, offsets, act, situ_beta, situ_linear_beta, out)


def group_glu_grad(da, x, w, offsets, act="silu", situ_beta=4.0, situ_linear_beta=25.0, out=None, stream=None):
    """Gradient of group_glu for its projections, which are computed again -> dgu [rows, 2 width].

    The gradients for x and w are group_mm_grad_x(dgu, w, offsets) and group_mm_grad_w(dgu, x, offsets), of dgu in x's
    16 bits."""
    return _call("group_glu_grad", stream, da, x, w, offsets, act, situ_beta, situ_linear_beta, out)


# ------------------------------------------------------------------------------------------ 8-bit operands
def quant8_rows(x, kind="e4m3", stream=None):
    """x [rows, n], 16-bit -> (codes [rows, n] float8_e4m3fn or, for kind "e5m2", float8_e5m2, scales [rows,
    ceil(n / 128)] uint8): a value is code 2^(scale - 127), a scale for each 128 columns of a row.

    The scale is the smallest power of two under which nothing saturates; a value that is not finite takes no part in
    it and becomes NaN (e5m2 keeps infinities).  Rows of both results start on 16-byte boundaries."""
    return _call("quant8_rows", stream, x, kind)


def quant8_weights(w, kind="e4m3", transposed=False, stream=None):
    """w [E, n_out, n_in], 16-bit -> (codes [E, n_out, n_in], scales [E, ceil(n_out / 128), ceil(n_in / 128)] uint8):
    a scale for each 128 x 128 block, as in quant8_rows.

    transposed: a third result, the same codes as [E, n_in, n_out], whose scales are scales.transpose(1, 2)."""
    return _call("quant8_weights", stream, w, kind, transposed)


def group_mm8(x, x_scales, w, w_scales, offsets, out=None, out_dtype=None, stream=None):
    """y[r] = w[e] x[r] on 8-bit operands (quant8_rows, quant8_weights) -> [rows, n_out], bf16 (or `out`'s / `out_dtype`'s
    type: f16, fp32).

    The gradient for the rows is the same call on the quantised dy with the transposed codes and scales; that for the weights
    is group_mm_grad_w on 16-bit rows.  Scales are powers of two alone (uint8 exponents).  Codes of rows that are not on
    16-byte boundaries are refused, and x_scales' off 4-byte ones."""
    return _call("group_mm8", stream, x, x_scales, w, w_scales, offsets, out, out_dtype)


# ------------------------------------------------------------------------------------------ norms
def rms_norm(x, gain=None, eps=1e-6, out=None, stream=None):
    """gain x / sqrt(mean x^2 + eps) over each row; x [rows, D <= 16384], fp32 or 16-bit, gain [D] of x's type or fp32.
    `out` may be x."""
    return _call("rms_norm", stream, x, gain, eps, out)


def rms_norm_grad(dy, x, gain=None, eps=1e-6, add=None, out=None, stream=None):
    """Gradient of rms_norm: (dx [+ add], dgain [D] fp32 or None without a gain).  `out` may be dy, x or add."""
    return _call("rms_norm_grad", stream, dy, x, gain, eps, add, out)


def norm_residual(y, residual, gain=None, gate=None, residual_scale=1.0, next_gain=None, eps=1e-6, out=None, stream=None):
    """The norm after a block, its gate, the residual and the norm before the next block: (h, n) with
    h = residual_scale residual + gate (gain y rs(y)), n = next_gain h rs(h), rs(v) = 1 / sqrt(mean v^2 + eps).

    gate: None, fp32 [rows], or [rows, D] of y's type.  Without next_gain n is None.  `out` (for h) may be y, residual or
    gate; n comes from the h that is not rounded yet."""
    return _call("norm_residual", stream, y, residual, gain, gate, residual_scale, next_gain, eps, out)


def norm_residual_grad(dh, dn, y, h, gain=None, gate=None, residual_scale=1.0, next_gain=None, eps=1e-6, stream=None):
    """Gradient of norm_residual: (dy, dresidual, dgain, dgate, dnext_gain), None for what was not there.

    dh and dn are the gradients for h and n (either may be None, not both); h is norm_residual's (may be None without
    dn).  dgain and dnext_gain are fp32 [D], dgate of the gate's shape and type."""
    if stream is not None and getattr(y, "device", stream.device) != stream.device:         # dh may be None
        raise K3Error(ERR_CODE["ARG"], "stream: one of the tensors' device")
    return _call("norm_residual_grad", stream, dh, dn, y, h, gain, gate, residual_scale, next_gain, eps)


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
