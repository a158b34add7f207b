"""Training step of the routed experts on 16-bit weights (the k3moe_rows_*, k3moe_group_*, k3moe_glu_*
and k3moe_dropout calls of include/k3moe.h): tensors in, tensors out, argument marshalling only.

Tensors live on one CUDA device; matrices have contiguous rows (any row stride).  Work is enqueued on
`stream` (default: the current stream), and results are allocated there.  Argument errors raise K3Error;
errors found on the device (row offsets out of range, a wait that ran out) are kept in a status word
per device, read by `status()`.
"""
from __future__ import annotations

import functools

import torch

from .k3moe import ACT_SILU, ACT_SITU, ERR_CODE, K3Error, TYPE_BF16, TYPE_F16, TYPE_F32, check, lib

_TYPE = {torch.float32: TYPE_F32, torch.bfloat16: TYPE_BF16, torch.float16: TYPE_F16}
_ACT = {"silu": ACT_SILU, "situ": ACT_SITU}
_U64 = (1 << 64) - 1
_status = {}
_ws_bytes = {}


def _refuse(what, code="ARG"):
    raise K3Error(ERR_CODE[code], what)


def _placed(fn):
    """Run fn with its first tensor's device current and, when given, `stream` as the current stream; fn's
    last argument is the stream's handle.  The common case (that device current, no stream given) costs
    two look-ups instead of two context managers."""
    @functools.wraps(fn)
    def call(t, *args, stream=None, **kw):
        dev = t.get_device()
        if dev < 0:
            _refuse(f"{fn.__name__}: CUDA tensors are needed")
        if stream is None and dev == torch._C._cuda_getDevice():
            return fn(t, *args, s=torch._C._cuda_getCurrentRawStream(dev), **kw)
        with torch.cuda.device(dev), torch.cuda.stream(stream):
            return fn(t, *args, s=torch._C._cuda_getCurrentRawStream(dev), **kw)
    return call


def _type(t, what):
    code = _TYPE.get(t.dtype)
    if code is None:
        _refuse(f"{what}: {t.dtype}", "UNSUPPORTED")
    return code


def _out(out, n, width, dtype, ref, what="out"):
    """`out` (checked) or a new [n, width] matrix of `dtype` on ref's device -> (matrix, row stride)."""
    if out is None:
        return torch.empty((n, width), dtype=dtype, device=ref.device), width     # a device number costs 2 us more
    rows, _, ld = _rows(out, what, ref.get_device(), width)
    if rows != n or out.dtype != dtype:
        _refuse(f"{what}: {n} rows of {dtype}")
    return out, ld


def _rows(t, what, dev, width=None):
    """A matrix on device `dev` with contiguous rows -> (rows, columns, row stride)."""
    if t.dim() != 2 or t.get_device() != dev:
        _refuse(f"{what}: a matrix on the call's device")
    (n, d), (ld, one) = t.shape, t.stride()
    if (one != 1 and d > 1) or (width is not None and d != width):
        _refuse(f"{what}: contiguous rows" + (f" of {width} columns" if width is not None else ""))
    if n <= 1:
        ld = d
    elif ld < d:
        _refuse(f"{what}: overlapping rows")
    return n, d, ld


def _table(t, what, dev, dtype, shape=None):
    if t.get_device() != dev or t.dtype != dtype or not t.is_contiguous() or (shape is not None and t.shape != shape):
        _refuse(f"{what}: a contiguous {dtype} tensor on the call's device" + (f" of shape {shape}" if shape else ""))


def _pairs(pos, what, dev, T=None):
    _table(pos, what, dev, torch.int32)
    if pos.dim() != 2 or (T is not None and pos.shape[0] != T):
        _refuse(f"{what}: [T, K]")
    return pos.shape


def _status_word(dev):
    st = _status.get(dev)
    if st is None:
        if torch.cuda.is_current_stream_capturing():
            _refuse("the first call on a device allocates its status word: make it outside a capture")
        st = torch.zeros(4, dtype=torch.int32, device=f"cuda:{dev}")
        torch.cuda.synchronize(dev)
        st = _status[dev] = (st, st.data_ptr())
    return st[1]


def status(device=None):
    """Synchronise the device, then read and clear its status word: 0 or the first device-side error
    (a K3MOE_ERR_* code) of these calls since the last read."""
    dev = torch.cuda.current_device() if device is None else torch.device(device).index or 0
    if dev not in _status:
        return 0
    torch.cuda.synchronize(dev)
    st = _status[dev][0]
    code = int(st[0])
    if code:
        st.zero_()
        torch.cuda.synchronize(dev)
    return code


# ------------------------------------------------------------------------------------------ rows
@_placed
def plan_rows(idx, n_experts, first_expert=0, *, s):
    """Expert order of a routing: idx [T, K] int32 -> (offsets [n_experts + 1], pos [T, K]), int32.

    Expert first_expert + e owns rows offsets[e] .. offsets[e + 1]; pos is each pair's row, -1 for a
    pair of another rank's expert (or a negative idx).  Rows of one expert are in (token, slot) order."""
    dev = idx.get_device()
    T, K = _pairs(idx, "idx", dev)
    L = lib()
    key = (T, K, n_experts)
    nb = _ws_bytes.get(key)
    if nb is None:
        if len(_ws_bytes) > 4096:
            _ws_bytes.clear()
        nb = _ws_bytes[key] = max(4, L.k3moe_rows_plan_workspace_bytes(T, K, n_experts))
    new, i32, where = torch.empty, torch.int32, idx.device
    ws, offsets = new((nb + 3) // 4, dtype=i32, device=where), new(max(n_experts, 0) + 1, dtype=i32, device=where)
    pos = torch.empty_like(idx)
    check(L.k3moe_rows_plan(idx.data_ptr(), T, K, first_expert, n_experts, offsets.data_ptr(), pos.data_ptr(),
                            ws.data_ptr(), nb, s), "plan_rows")
    return offsets, pos


@_placed
def gather_rows(x, pos, n_rows=None, out=None, *, s):
    """out[pos[t, k]] = x[t] for every pos >= 0; out [n_rows, D] (default T * K rows).  Rows that no
    pair names are left as they are (uninitialised in a new `out`).  Gradient: combine_rows(dout, pos)."""
    dev = x.get_device()
    T, D, ldx = _rows(x, "x", dev)
    K = _pairs(pos, "pos", dev, T)[1]
    if out is None:
        out = torch.empty((T * K if n_rows is None else n_rows, D), dtype=x.dtype, device=x.device)
    n, _, ldo = _rows(out, "out", dev, D)
    if out.dtype != x.dtype or (n_rows is not None and n_rows > n):
        _refuse("out: x's type and at least n_rows rows")
    check(lib().k3moe_rows_gather(x.data_ptr(), ldx, pos.data_ptr(), T, K, D, _type(x, "x"), out.data_ptr(), ldo,
                                  n if n_rows is None else n_rows, _status_word(dev), s), "gather_rows")
    return out


@_placed
def combine_rows(y, pos, weights=None, out=None, *, s):
    """z[t] = sum_k weights[t, k] y[pos[t, k]] over pos >= 0 (weights None: all 1) -> [T, D]."""
    dev = y.get_device()
    n, D, ldy = _rows(y, "y", dev)
    T, K = _pairs(pos, "pos", dev)
    if weights is not None:
        _table(weights, "weights", dev, torch.float32, (T, K))
    out, ldz = _out(out, T, D, y.dtype, y)
    check(lib().k3moe_rows_combine(y.data_ptr(), ldy, n, pos.data_ptr(), None if weights is None else weights.data_ptr(),
                                   T, K, D, _type(y, "y"), out.data_ptr(), ldz, _status_word(dev), s), "combine_rows")
    return out


@_placed
def combine_rows_grad(dz, y, pos, weights, out=None, *, s):
    """Gradient of combine_rows: (dy [rows of y, D], dweights [T, K] fp32).  `out` receives dy and may be y."""
    dev = dz.get_device()
    T, D, lddz = _rows(dz, "dz", dev)
    n, _, ldy = _rows(y, "y", dev, D)
    K = _pairs(pos, "pos", dev, T)[1]
    _table(weights, "weights", dev, torch.float32, (T, K))
    if dz.dtype != y.dtype:
        _refuse("dz: y's type")
    out, lddy = _out(out, n, D, y.dtype, y)
    dw = torch.empty_like(weights)
    check(lib().k3moe_rows_combine_grad(dz.data_ptr(), lddz, y.data_ptr(), ldy, n, pos.data_ptr(), weights.data_ptr(), T,
                                        K, D, _type(y, "y"), out.data_ptr(), lddy, dw.data_ptr(), _status_word(dev), s),
          "combine_rows_grad")
    return out, dw


# ------------------------------------------------------------------------------------------ grouped products
def _matrices(w, what, dev):
    """[E, n_out, n_in] with contiguous rows -> (E, n_out, n_in, row stride, expert stride)."""
    if w.dim() != 3 or w.get_device() != dev:
        _refuse(f"{what}: [E, n_out, n_in] on the call's device")
    (E, N, K), (sw, ld, one) = w.shape, w.stride()
    if one != 1 and K > 1:
        _refuse(f"{what}: contiguous rows")
    return E, N, K, ld if N > 1 else K, sw if E > 1 else 0


def _group(name, what, a, w, offsets, out, out_dtype, s, mm):
    dev = a.get_device()
    E, N, K, ldw, sw = _matrices(w, "w", dev)
    n, _, lda = _rows(a, what, dev, K if mm else N)
    if a.dtype != w.dtype:
        _refuse(f"{what}: w's type")
    _table(offsets, "offsets", dev, torch.int32, (E + 1,))
    width = N if mm else K
    out, ldo = _out(out, n, width, out_dtype or (a.dtype if out is None else out.dtype), a)
    check(getattr(lib(), name)(offsets.data_ptr(), E, n, K, N, a.data_ptr(), lda, w.data_ptr(), ldw, sw, _type(a, what),
                               out.data_ptr(), ldo, _type(out, "out"), _status_word(dev), s), name)
    return out


@_placed
def group_mm(x, w, offsets, out=None, out_dtype=None, *, s):
    """y[r] = w[e] x[r] for the rows offsets[e] <= r < offsets[e + 1] of every expert e.

    x [rows, n_in], w [E, n_out, n_in] of one 16-bit type, y [rows, n_out] of that type or fp32.  Rows of
    no expert are not written."""
    return _group("k3moe_group_mm", "x", x, w, offsets, out, out_dtype, s, True)


@_placed
def group_mm_grad_x(dy, w, offsets, out=None, out_dtype=None, *, s):
    """dx[r] = w[e]^T dy[r]: the gradient of group_mm for x."""
    return _group("k3moe_group_mm_grad_x", "dy", dy, w, offsets, out, out_dtype, s, False)


@_placed
def group_mm_grad_w(dy, x, offsets, out=None, out_dtype=None, accumulate=False, *, s):
    """dw[e] = sum over the expert's rows of dy[r] x[r]^T: the gradient of group_mm for w, [E, n_out, n_in].

    fp32 by default (or `out`'s / `out_dtype`'s type: x's).  accumulate adds to an fp32 `out`; otherwise an
    expert without rows gets zeros."""
    dev = dy.get_device()
    n, N, lddy = _rows(dy, "dy", dev)
    nx, K, ldx = _rows(x, "x", dev)
    if dy.dtype != x.dtype or nx != n:
        _refuse("x: dy's rows and type")
    _table(offsets, "offsets", dev, torch.int32)
    if offsets.dim() != 1 or offsets.numel() < 2:
        _refuse("offsets: [E + 1]")
    E = offsets.numel() - 1
    if out is None:
        if accumulate:
            _refuse("accumulate needs out")
        out = torch.empty((E, N, K), dtype=out_dtype or torch.float32, device=x.device)
    Eo, No, Ko, ldo, so = _matrices(out, "out", dev)
    if (Eo, No, Ko) != (E, N, K) or (out_dtype is not None and out.dtype != out_dtype):
        _refuse("out: [E, n_out, n_in] of the type asked for")
    check(lib().k3moe_group_mm_grad_w(offsets.data_ptr(), E, n, K, N, dy.data_ptr(), lddy, x.data_ptr(), ldx,
                                      _type(x, "x"), out.data_ptr(), ldo, so, _type(out, "out"), 1 if accumulate else 0,
                                      _status_word(dev), s), "group_mm_grad_w")
    return out


# ------------------------------------------------------------------------------------------ gated unit, dropout
def _random(p, seed, offset):
    if not (0.0 <= p < 1.0 and 0 <= seed <= _U64 and 0 <= offset <= _U64):
        _refuse("0 <= p < 1; seed, offset: 64-bit unsigned")


def _gated(gu, act, dev):
    n, d, ld = _rows(gu, "gu", dev)
    if d % 2 or d == 0 or act not in _ACT:
        _refuse("gu: [rows, 2 width]; act: silu or situ")
    return n, d // 2, ld


@_placed
def glu_dropout(gu, p=0.0, seed=0, offset=0, act="silu", situ_beta=4.0, situ_linear_beta=25.0, out=None, *, s):
    """a = dropout(act(g) u), gu [rows, 2 width] = gate columns then up columns -> [rows, width].

    The mask depends on (seed, offset, element index) alone; use another offset for every call of a step."""
    dev = gu.get_device()
    n, width, ldgu = _gated(gu, act, dev)
    _random(p, seed, offset)
    out, lda = _out(out, n, width, gu.dtype, gu)
    check(lib().k3moe_glu_dropout(gu.data_ptr(), ldgu, n, width, _type(gu, "gu"), _ACT[act], situ_beta,
                                  situ_linear_beta, p, seed, offset, out.data_ptr(), lda, s), "glu_dropout")
    return out


@_placed
def glu_dropout_grad(da, gu, p=0.0, seed=0, offset=0, act="silu", situ_beta=4.0, situ_linear_beta=25.0, out=None, *, s):
    """Gradient of glu_dropout (with the same p, seed and offset) -> dgu [rows, 2 width]; `out` may be gu."""
    dev = da.get_device()
    n, width, ldgu = _gated(gu, act, dev)
    na, _, ldda = _rows(da, "da", dev, width)
    if da.dtype != gu.dtype or na != n:
        _refuse("da: gu's rows and type")
    _random(p, seed, offset)
    out, ldo = _out(out, n, 2 * width, gu.dtype, gu)
    check(lib().k3moe_glu_dropout_grad(da.data_ptr(), ldda, gu.data_ptr(), ldgu, n, width, _type(gu, "gu"), _ACT[act],
                                       situ_beta, situ_linear_beta, p, seed, offset, out.data_ptr(), ldo, s),
          "glu_dropout_grad")
    return out


@_placed
def dropout(x, p, seed, offset, residual=None, out=None, *, s):
    """dropout(x) [+ residual], any contiguous shape, fp32 or 16-bit; `out` may be x or residual.  The
    gradient for x is dropout(dout, p, seed, offset)."""
    _random(p, seed, offset)
    if not x.is_contiguous():
        _refuse("x: a contiguous tensor")
    if out is None:
        out = torch.empty_like(x)
    else:
        _table(out, "out", x.get_device(), x.dtype, x.shape)
    if residual is not None:
        _table(residual, "residual", x.get_device(), x.dtype, x.shape)
    check(lib().k3moe_dropout(x.data_ptr(), None if residual is None else residual.data_ptr(), x.numel(), _type(x, "x"),
                              p, seed, offset, out.data_ptr(), s), "dropout")
    return out
