"""Training step of the routed experts on 16-bit weights (the k3moe_rows_*, k3moe_group_*, k3moe_glu_*
and k3moe_dropout calls of include/k3moe.h): tensors in, tensors out, argument marshalling only.

Tensors live on one CUDA device; matrices have contiguous rows (any row stride).  Work is enqueued on
`stream` (default: the current stream), and results are allocated there.  Argument errors raise K3Error;
errors found on the device (row offsets out of range, a wait that ran out) are kept in a status word
per device, read by `status()`.
"""
from __future__ import annotations

import contextlib

import torch

from . import k3moe
from .k3moe import ACT_SILU, ACT_SITU, ERR_CODE, K3Error, TYPE_BF16, TYPE_F16, TYPE_F32, check, lib

_TYPE = {torch.float32: TYPE_F32, torch.bfloat16: TYPE_BF16, torch.float16: TYPE_F16}
_ACT = {"silu": ACT_SILU, "situ": ACT_SITU}
_status = {}


def _arg(ok, what):
    if not ok:
        raise K3Error(ERR_CODE["ARG"], what)


def _type(t, what):
    code = _TYPE.get(t.dtype)
    if code is None:
        raise K3Error(ERR_CODE["UNSUPPORTED"], f"{what}: {t.dtype}")
    return code


def _rows(t, what, width=None):
    """A 2-D tensor with contiguous rows -> its row stride."""
    _arg(t.is_cuda and t.dim() == 2 and (t.shape[1] <= 1 or t.stride(1) == 1), f"{what}: a CUDA matrix with contiguous rows")
    _arg(width is None or t.shape[1] == width, f"{what}: {width} columns expected")
    ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    _arg(ld >= t.shape[1], f"{what}: overlapping rows")
    return ld


def _table(t, what, dtype, shape=None):
    _arg(t.is_cuda and t.dtype == dtype and t.is_contiguous() and (shape is None or tuple(t.shape) == shape),
         f"{what}: a contiguous CUDA {dtype} tensor" + (f" of shape {shape}" if shape else ""))


def _same(ref, what, *ts):
    for t in ts:
        _arg(t is None or t.device == ref.device, f"{what}: tensors on different devices")


@contextlib.contextmanager
def _on(t, stream):
    """The device of t current, `stream` its current stream; yields the stream's handle."""
    with torch.cuda.device(t.device):
        if stream is None:
            yield torch.cuda.current_stream().cuda_stream
        else:
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


def _status_word(device):
    st = _status.get(device.index)
    if st is None:
        _arg(not torch.cuda.is_current_stream_capturing(),
             "the first call on a device allocates its status word: make it outside a capture")
        st = torch.zeros(4, dtype=torch.int32, device=device)
        torch.cuda.synchronize(device)
        _status[device.index] = st
    return st


def status(device=None):
    """Synchronise the device, then read and clear its status word: 0 or the first device-side error
    (a K3MOE_ERR_* code) of these calls since the last read."""
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else torch.device(device).index or 0)
    st = _status.get(dev.index)
    if st is None:
        return 0
    torch.cuda.synchronize(dev)
    code = int(st[0])
    if code:
        st.zero_()
        torch.cuda.synchronize(dev)
    return code


# ------------------------------------------------------------------------------------------ rows
def plan_rows(idx, n_experts, first_expert=0, stream=None):
    """Expert order of a routing: idx [T, K] int32 -> (offsets [n_experts + 1], pos [T, K]), int32.

    Expert first_expert + e owns rows offsets[e] .. offsets[e + 1]; pos is each pair's row, -1 for a
    pair of another rank's expert (or a negative idx).  Rows of one expert are in (token, slot) order."""
    _arg(idx.dim() == 2, "idx: [T, K]")
    _table(idx, "idx", torch.int32)
    T, K = idx.shape
    with _on(idx, stream) as s:
        nb = lib().k3moe_rows_plan_workspace_bytes(T, K, n_experts)
        ws = torch.empty(max(nb, 4), dtype=torch.uint8, device=idx.device)
        offsets = torch.empty(max(n_experts, 0) + 1, dtype=torch.int32, device=idx.device)
        pos = torch.empty_like(idx)
        check(lib().k3moe_rows_plan(idx.data_ptr(), T, K, first_expert, n_experts, offsets.data_ptr(), pos.data_ptr(),
                                    ws.data_ptr(), ws.numel(), s), "plan_rows")
    return offsets, pos


def gather_rows(x, pos, n_rows=None, out=None, stream=None):
    """out[pos[t, k]] = x[t] for every pos >= 0; out [n_rows, D] (default T * K rows).  Rows that no
    pair names are left as they are (uninitialised in a new `out`).  Gradient: combine_rows(dout, pos)."""
    ldx = _rows(x, "x")
    _table(pos, "pos", torch.int32)
    _arg(pos.dim() == 2 and pos.shape[0] == x.shape[0], "pos: [T, K]")
    T, K = pos.shape
    D = x.shape[1]
    with _on(x, stream) as s:
        if out is None:
            out = torch.empty((T * K if n_rows is None else n_rows, D), dtype=x.dtype, device=x.device)
        ldo = _rows(out, "out", D)
        _arg(out.dtype == x.dtype and (n_rows is None or n_rows <= out.shape[0]), "out: x's type, n_rows rows")
        _same(x, "gather_rows", pos, out)
        check(lib().k3moe_rows_gather(x.data_ptr(), ldx, pos.data_ptr(), T, K, D, _type(x, "x"), out.data_ptr(), ldo,
                                      out.shape[0] if n_rows is None else n_rows, _status_word(x.device).data_ptr(), s),
              "gather_rows")
    return out


def combine_rows(y, pos, weights=None, out=None, stream=None):
    """z[t] = sum_k weights[t, k] y[pos[t, k]] over pos >= 0 (weights None: all 1) -> [T, D]."""
    ldy = _rows(y, "y")
    _table(pos, "pos", torch.int32)
    _arg(pos.dim() == 2, "pos: [T, K]")
    T, K = pos.shape
    D = y.shape[1]
    if weights is not None:
        _table(weights, "weights", torch.float32, (T, K))
    with _on(y, stream) as s:
        if out is None:
            out = torch.empty((T, D), dtype=y.dtype, device=y.device)
        ldz = _rows(out, "out", D)
        _arg(out.dtype == y.dtype and out.shape[0] == T, "out: [T, D] of y's type")
        _same(y, "combine_rows", pos, weights, out)
        check(lib().k3moe_rows_combine(y.data_ptr(), ldy, y.shape[0], pos.data_ptr(),
                                       None if weights is None else weights.data_ptr(), T, K, D, _type(y, "y"),
                                       out.data_ptr(), ldz, _status_word(y.device).data_ptr(), s), "combine_rows")
    return out


def combine_rows_grad(dz, y, pos, weights, out=None, stream=None):
    """Gradient of combine_rows: (dy [rows of y, D], dweights [T, K] fp32).  `out` receives dy and may be y."""
    lddz, ldy = _rows(dz, "dz"), _rows(y, "y", dz.shape[1])
    _table(pos, "pos", torch.int32)
    _arg(pos.dim() == 2 and pos.shape[0] == dz.shape[0] and dz.dtype == y.dtype, "pos: [T, K]; dz of y's type")
    T, K = pos.shape
    _table(weights, "weights", torch.float32, (T, K))
    with _on(y, stream) as s:
        if out is None:
            out = torch.empty((y.shape[0], y.shape[1]), dtype=y.dtype, device=y.device)
        lddy = _rows(out, "out", y.shape[1])
        _arg(out.dtype == y.dtype and out.shape[0] == y.shape[0], "out: y's shape and type")
        _same(y, "combine_rows_grad", dz, pos, weights, out)
        dw = torch.empty((T, K), dtype=torch.float32, device=y.device)
        check(lib().k3moe_rows_combine_grad(dz.data_ptr(), lddz, y.data_ptr(), ldy, y.shape[0], pos.data_ptr(),
                                            weights.data_ptr(), T, K, y.shape[1], _type(y, "y"), out.data_ptr(), lddy,
                                            dw.data_ptr(), _status_word(y.device).data_ptr(), s), "combine_rows_grad")
    return out, dw


# ------------------------------------------------------------------------------------------ grouped products
def _weights(w):
    _arg(w.is_cuda and w.dim() == 3 and (w.shape[2] <= 1 or w.stride(2) == 1), "w: [E, n_out, n_in] with contiguous rows")
    E, N, K = w.shape
    return E, N, K, w.stride(1) if N > 1 else K, w.stride(0) if E > 1 else 0


def _group(fn, name, a, width, w, n, offsets, out, out_dtype, stream):
    E, N, K, ldw, sw = _weights(w)
    lda = _rows(a, name, width)
    _arg(a.dtype == w.dtype, f"{name}: w's type")
    _table(offsets, "offsets", torch.int32, (E + 1,))
    with _on(a, stream) as s:
        if out is None:
            out = torch.empty((a.shape[0], n), dtype=out_dtype or a.dtype, device=a.device)
        ldo = _rows(out, "out", n)
        _arg(out.shape[0] == a.shape[0] and (out_dtype is None or out.dtype == out_dtype), "out: rows and type")
        _same(a, "grouped product", w, offsets, out)
        check(fn(offsets.data_ptr(), E, a.shape[0], K, N, a.data_ptr(), lda, w.data_ptr(), ldw, sw, _type(a, name),
                 out.data_ptr(), ldo, _type(out, "out"), _status_word(a.device).data_ptr(), s), "grouped product")
    return out


def group_mm(x, w, offsets, out=None, out_dtype=None, stream=None):
    """y[r] = w[e] x[r] for the rows offsets[e] <= r < offsets[e + 1] of every expert e.

    x [rows, n_in], w [E, n_out, n_in] of one 16-bit type, y [rows, n_out] of that type or fp32.  Rows of
    no expert are not written."""
    _arg(w.dim() == 3, "w: [E, n_out, n_in]")
    return _group(lib().k3moe_group_mm, "x", x, w.shape[2], w, w.shape[1], offsets, out, out_dtype, stream)


def group_mm_grad_x(dy, w, offsets, out=None, out_dtype=None, stream=None):
    """dx[r] = w[e]^T dy[r]: the gradient of group_mm for x."""
    _arg(w.dim() == 3, "w: [E, n_out, n_in]")
    return _group(lib().k3moe_group_mm_grad_x, "dy", dy, w.shape[1], w, w.shape[2], offsets, out, out_dtype, stream)


def group_mm_grad_w(dy, x, offsets, out=None, out_dtype=None, accumulate=False, stream=None):
    """dw[e] = sum over the expert's rows of dy[r] x[r]^T: the gradient of group_mm for w, [E, n_out, n_in].

    fp32 by default (or `out`'s / `out_dtype`'s type: x's).  accumulate adds to an fp32 `out`; otherwise an
    expert without rows gets zeros."""
    lddy, ldx = _rows(dy, "dy"), _rows(x, "x")
    _arg(dy.dtype == x.dtype and dy.shape[0] == x.shape[0], "dy: x's rows and type")
    _arg(offsets.dim() == 1 and offsets.numel() > 1, "offsets: [E + 1]")
    _table(offsets, "offsets", torch.int32)
    _arg(not accumulate or out is not None, "accumulate needs out")
    E, N, K = offsets.numel() - 1, dy.shape[1], x.shape[1]
    with _on(x, stream) as s:
        if out is None:
            out = torch.empty((E, N, K), dtype=out_dtype or torch.float32, device=x.device)
        _arg(tuple(out.shape) == (E, N, K) and (out_dtype is None or out.dtype == out_dtype), "out: [E, n_out, n_in]")
        _, _, _, ldo, so = _weights(out)
        _same(x, "grouped product", dy, offsets, out)
        check(lib().k3moe_group_mm_grad_w(offsets.data_ptr(), E, x.shape[0], K, N, dy.data_ptr(), lddy, x.data_ptr(),
                                          ldx, _type(x, "x"), out.data_ptr(), ldo, so, _type(out, "out"),
                                          1 if accumulate else 0, _status_word(x.device).data_ptr(), s),
              "group_mm_grad_w")
    return out


# ------------------------------------------------------------------------------------------ gated unit, dropout
_U64 = (1 << 64) - 1


def _random(p, seed, offset):
    _arg(0.0 <= p < 1.0, "p: 0 <= p < 1")
    _arg(0 <= seed <= _U64 and 0 <= offset <= _U64, "seed, offset: 64-bit unsigned")
    return float(p), seed, offset


def glu_dropout(gu, p=0.0, seed=0, offset=0, act="silu", situ_beta=4.0, situ_linear_beta=25.0, out=None, stream=None):
    """a = dropout(act(g) u), gu [rows, 2 width] = gate columns then up columns -> [rows, width].

    The mask depends on (seed, offset, element index) alone; use another offset for every call of a step."""
    ldgu = _rows(gu, "gu")
    _arg(gu.shape[1] % 2 == 0 and gu.shape[1] > 0 and act in _ACT, "gu: [rows, 2 width]; act: silu or situ")
    width = gu.shape[1] // 2
    p, seed, offset = _random(p, seed, offset)
    with _on(gu, stream) as s:
        if out is None:
            out = torch.empty((gu.shape[0], width), dtype=gu.dtype, device=gu.device)
        lda = _rows(out, "out", width)
        _arg(out.dtype == gu.dtype and out.shape[0] == gu.shape[0], "out: gu's rows and type")
        _same(gu, "glu_dropout", out)
        check(lib().k3moe_glu_dropout(gu.data_ptr(), ldgu, gu.shape[0], width, _type(gu, "gu"), _ACT[act], situ_beta,
                                      situ_linear_beta, p, seed, offset, out.data_ptr(), lda, s), "glu_dropout")
    return out


def glu_dropout_grad(da, gu, p=0.0, seed=0, offset=0, act="silu", situ_beta=4.0, situ_linear_beta=25.0, out=None,
                     stream=None):
    """Gradient of glu_dropout (with the same p, seed and offset) -> dgu [rows, 2 width]; `out` may be gu."""
    ldgu = _rows(gu, "gu")
    _arg(gu.shape[1] % 2 == 0 and gu.shape[1] > 0 and act in _ACT, "gu: [rows, 2 width]; act: silu or situ")
    width = gu.shape[1] // 2
    ldda = _rows(da, "da", width)
    _arg(da.dtype == gu.dtype and da.shape[0] == gu.shape[0], "da: gu's rows and type")
    p, seed, offset = _random(p, seed, offset)
    with _on(gu, stream) as s:
        if out is None:
            out = torch.empty((gu.shape[0], 2 * width), dtype=gu.dtype, device=gu.device)
        ldo = _rows(out, "out", 2 * width)
        _arg(out.dtype == gu.dtype and out.shape[0] == gu.shape[0], "out: gu's shape and type")
        _same(gu, "glu_dropout_grad", da, out)
        check(lib().k3moe_glu_dropout_grad(da.data_ptr(), ldda, gu.data_ptr(), ldgu, gu.shape[0], width,
                                           _type(gu, "gu"), _ACT[act], situ_beta, situ_linear_beta, p, seed, offset,
                                           out.data_ptr(), ldo, s), "glu_dropout_grad")
    return out


def dropout(x, p, seed, offset, residual=None, out=None, stream=None):
    """dropout(x) [+ residual], any contiguous shape, fp32 or 16-bit; `out` may be x or residual.  The
    gradient for x is dropout(dout, p, seed, offset)."""
    p, seed, offset = _random(p, seed, offset)
    _arg(x.is_cuda and x.is_contiguous(), "x: a contiguous CUDA tensor")
    with _on(x, stream) as s:
        if out is None:
            out = torch.empty_like(x)
        for t in (residual, out):
            _arg(t is None or (t.is_contiguous() and t.shape == x.shape and t.dtype == x.dtype and t.device == x.device),
                 "residual, out: x's shape, type and device")
        check(lib().k3moe_dropout(x.data_ptr(), None if residual is None else residual.data_ptr(), x.numel(),
                                  _type(x, "x"), p, seed, offset, out.data_ptr(), s), "dropout")
    return out
