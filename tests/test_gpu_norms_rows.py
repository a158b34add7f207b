"""Norms of more rows than the GPU holds at once, so that every CTA goes on to its second and later rows and the last round is
ragged: the gradient's pipelined loop, its form with one slot in shared memory, several rows a CTA, rows off 16-byte boundaries.
Against oracle/experts.py with the bounds of test_gpu_norms.py, which hold for any number of rows.  And rows that start past
2^31 elements, against the same rows as a call of their own."""
import numpy as np
import pytest

from oracle import experts as ox

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from latent_moe_layer_gb300 import experts as ex  # noqa: E402
from test_gpu_experts import BF, F16, F32, _close, _gen, _np  # noqa: E402
from test_gpu_norms import C, GATES, _check_backward, _check_forward, _inputs, _norm_slack  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


# rows, columns, type: on 152 SMs at least two rows a CTA in the gradient, and not the same number for all CTAs
MANY = [(4001, 1536, BF), (700, 7168, F16), (500, 8192, BF), (500, 3584, F32), (500, 7168, F32), (411, 8200, BF), (411, 12288, F32),
        (50_001, 64, BF), (20_011, 200, F16), (9001, 768, F32), (9001, 1000, BF), (40_001, 33, BF), (1300, 1001, F32), (411, 9001, F16)]
ROWS = pytest.mark.parametrize("T,D,dt", MANY, ids=[f"T{t}D{d}{str(x)[6:]}" for t, d, x in MANY])


@ROWS
@GATES
def test_norm_residual_and_gradient_over_many_rows(T, D, dt, gate):
    v = _inputs(T, D, gate, dt)
    h = _check_forward(v, 0.75)
    _check_backward(v, h, 0.75)
    if gate == "row":
        _check_backward(v, h, 0.75, use_dn=False)


@ROWS
def test_rms_norm_and_gradient_over_many_rows(T, D, dt):
    v = _inputs(T, D, "none", dt)
    x, gain, dy, add, eps = v["y"], v["gain"], v["dn"], v["dh"], 1e-5
    xn, gn, dn = _np(x), _np(gain), _np(dy)
    want = ox.rms_norm(xn, gn, eps)
    _close(ex.rms_norm(x, gain, eps), want, C * np.abs(want), "norm")
    r = 1 / np.sqrt(np.mean(xn * xn, 1, keepdims=True) + eps)
    dx, dgain = ex.rms_norm_grad(dy, x, gain, eps, add=add)
    wx, wg = ox.rms_norm_grad(dn, xn, gn, eps, _np(add))
    _close(dx, wx, _norm_slack(dn, 0.0 * dn, xn, r, gn) + C * np.abs(_np(add)), "dx")
    _close(dgain, wg, (T + 64) * 2.0 ** -24 * np.abs(dn * xn * r).sum(0), "dgain")


@ROWS
@GATES
def test_a_row_does_not_depend_on_how_many_there_are(T, D, dt, gate):
    """The rows of a call are worked on alike, whichever round of a CTA they fall into: the same bits as in calls of 64 rows."""
    v = _inputs(T, D, gate, dt)
    def run(a, b):
        w = {k: (t[a:b] if torch.is_tensor(t) and t.shape[0] == T and t.shape != (D,) else t) for k, t in v.items()}
        h, n = ex.norm_residual(w["y"], w["res"], gain=v["gain"], gate=w["gate"], residual_scale=0.5, next_gain=v["next_gain"])
        got = ex.norm_residual_grad(w["dh"], w["dn"], w["y"], h, gain=v["gain"], gate=w["gate"], residual_scale=0.5, next_gain=v["next_gain"])
        return [h, n, got[0], got[1]] + ([] if gate == "none" else [got[3]]) + [ex.rms_norm_grad(w["dn"], w["y"], v["gain"])[0]]
    whole = run(0, T)
    for a in {0, 64, (T // 2) & ~7, (T - 64) & ~7}:
        for got, want in zip(run(a, min(a + 64, T)), whole):
            assert torch.equal(got, want[a:a + 64])


def test_gradients_of_rows_past_31_bits():
    T, D, last = 700_000, 3584, 40
    gen = _gen(3)
    x, dy = (torch.ones(T, D, dtype=BF, device="cuda") for _ in range(2))
    for t in (x, dy):
        t[-last:] = torch.randn(last, D, device="cuda", generator=gen).to(BF)
    gain = 1 + 0.1 * torch.randn(D, device="cuda", generator=gen)
    out = torch.full((T, D), float("nan"), dtype=BF, device="cuda")
    dx, _ = ex.rms_norm_grad(dy, x, gain, add=x, out=out)
    want, _ = ex.rms_norm_grad(dy[-last:], x[-last:], gain, add=x[-last:])
    assert torch.equal(dx[-last:], want) and not torch.isnan(dx).any()
    # norm_residual and its gradient: y and gate are x, the residual and dn are dy
    wide = out.fill_(float("nan"))
    h, n = ex.norm_residual(x, dy, gain=gain, gate=x, next_gain=gain, out=wide)
    near_h, near_n = ex.norm_residual(x[-last:], dy[-last:], gain=gain, gate=x[-last:], next_gain=gain)
    assert torch.equal(h[-last:], near_h) and torch.equal(n[-last:], near_n) and not torch.isnan(h).any()
    spoiled = [torch.full((T, D), float("nan"), dtype=BF, device="cuda") for _ in range(3)]
    del spoiled, n                                           # what the results below are allocated from
    got = ex.norm_residual_grad(dy, x, x, h, gain=gain, gate=dy, residual_scale=0.5, next_gain=gain)
    want = ex.norm_residual_grad(dy[-last:], x[-last:], x[-last:], h[-last:], gain=gain, gate=dy[-last:], residual_scale=0.5, next_gain=gain)
    for k in (0, 1, 3):
        assert torch.equal(got[k][-last:], want[k]) and not torch.isnan(got[k]).any()
    del x, dy, out, wide, h, dx, got
    torch.cuda.empty_cache()


@GATES
def test_rows_strides_past_31_bits(gate):
    """Few columns of very long rows: every matrix's stride takes its last rows past 2^31 elements."""
    T, D, ld = 66_000, 96, 32_768 + 8
    big = torch.empty(T, ld, dtype=BF, device="cuda")
    v = _inputs(T, D, gate, BF)
    w = dict(v)
    for i, k in enumerate(("y", "res", "gate", "dh", "dn")):
        if torch.is_tensor(v[k]) and v[k].dim() == 2:
            w[k] = big[:, 1024 * i:1024 * i + D]
            w[k][:] = v[k]
    # (outputs in memory of their own: one that lies between an input's rows is refused)
    other = torch.empty(T, ld, dtype=BF, device="cuda")
    hw = other[:, 8192:8192 + D].fill_(float("nan"))
    kw = dict(gain=v["gain"], residual_scale=0.5, next_gain=v["next_gain"])
    h, n = ex.norm_residual(w["y"], w["res"], gate=w["gate"], out=hw, **kw)
    wh, wn = ex.norm_residual(v["y"], v["res"], gate=v["gate"], **kw)
    assert torch.equal(h, wh) and torch.equal(n, wn)
    got = ex.norm_residual_grad(w["dh"], w["dn"], w["y"], h, gate=w["gate"], **kw)
    want = ex.norm_residual_grad(v["dh"], v["dn"], v["y"], wh, gate=v["gate"], **kw)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, want))
    dxw = other[:, 16384:16384 + D].fill_(float("nan"))
    dx, _ = ex.rms_norm_grad(w["dn"], w["y"], v["gain"], add=w["dh"], out=dxw)
    assert torch.equal(dx, ex.rms_norm_grad(v["dn"], v["y"], v["gain"], add=v["dh"])[0])
    del big, other, w, hw, h, dxw, dx
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 1001, 7168])
def test_rows_whose_squares_leave_fp32_have_norm_zero(D, dt):
    v = _inputs(9, D, "none", dt)
    v["y"][4] = 2.0 ** 70
    h, n = ex.norm_residual(v["y"], v["res"], gain=v["gain"], residual_scale=0.5, next_gain=v["next_gain"])
    assert torch.equal(h[4], (0.5 * v["res"][4].float()).to(dt)) and torch.isfinite(n).all()
    assert not ex.rms_norm(v["y"], v["gain"])[4].any()
    other = [0, 1, 2, 3, 5, 6, 7, 8]
    w = {k: (t[other] if torch.is_tensor(t) and t.shape[0] == 9 else t) for k, t in v.items()}
    assert torch.equal(h[other], _check_forward(w, 0.5))
