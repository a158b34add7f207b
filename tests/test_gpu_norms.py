"""Norms around a block on the GPU against oracle/experts.py.

A row's sums are fp32: 16 elements a thread, then trees of at most ten steps, so a mean is off by at most 26 2^-24 of the mean
of sizes, a reciprocal root by half of that and 2^-22; with the products around them every term of a result is good to C = 64
2^-24 of its size.  Sums over the rows are off by (rows + 64) 2^-24 of the sizes' sum at most."""
import numpy as np
import pytest

from oracle import experts as ox

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from latent_moe_layer_gb300 import experts as ex  # noqa: E402
from latent_moe_layer_gb300.k3moe import ERR_CODE, K3Error  # noqa: E402
from test_gpu_experts import BF, F16, F32, _close, _gen, _np  # noqa: E402

C = 64 * 2.0 ** -24
ALL = pytest.mark.parametrize("dt", [BF, F16, F32], ids=["bf16", "f16", "f32"])
GATES = pytest.mark.parametrize("gate", ["none", "row", "full"])


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def _inputs(T, D, gate, dt, gain_dt=F32):
    gen = _gen(T + D)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    v = dict(y=(r(T, D) * torch.exp2(r(T, 1) * 2)).to(dt), res=(r(T, D) * 2).to(dt), gain=(1 + 0.2 * r(D)).to(gain_dt),
             next_gain=(1 + 0.2 * r(D)).to(gain_dt), dh=r(T, D).to(dt), dn=r(T, D).to(dt))
    v["gate"] = None if gate == "none" else torch.sigmoid(r(T)) if gate == "row" else torch.sigmoid(r(T, D)).to(dt)
    return v


def _gate(g):
    return 1.0 if g is None else _np(g).reshape(len(g), -1)


def _check_forward(v, scale, eps=1e-6):
    y, res, gain, nxt, gate = _np(v["y"]), _np(v["res"]), _np(v["gain"]), _np(v["next_gain"]), _gate(v["gate"])
    h, n = ex.norm_residual(v["y"], v["res"], gain=v["gain"], gate=v["gate"], residual_scale=scale, next_gain=v["next_gain"], eps=eps)
    wh, wn = ox.norm_residual(y, res, gain, None if v["gate"] is None else _np(v["gate"]), scale, nxt, eps)
    eh = C * (np.abs(scale * res) + np.abs(wh - scale * res))
    _close(h, wh, eh, "h")
    r = 1 / np.sqrt(np.mean(wh * wh, 1, keepdims=True) + eps)
    lost = np.sqrt((eh ** 2).sum(1, keepdims=True) / np.maximum((wh ** 2).sum(1, keepdims=True), 1e-300))
    _close(n, wn, np.abs(nxt) * r * (eh + np.abs(wh) * (C + lost)), "n")
    only, none = ex.norm_residual(v["y"], v["res"], gain=v["gain"], gate=v["gate"], residual_scale=scale, eps=eps)
    assert none is None and torch.equal(only, h)
    return h


def _norm_slack(v, dv, x, r, gain):
    """Error of r (v gain - x' mean(v gain x')) from the error dv of v."""
    xh, g = np.abs(x * r), np.abs(gain)
    return r * (g * dv + xh * np.mean(g * dv * xh, 1, keepdims=True) + C * (np.abs(v) * g + xh * np.mean(np.abs(v) * g * xh, 1, keepdims=True)))


def _check_backward(v, h, scale, use_dh=True, use_dn=True, eps=1e-6):
    T = len(v["y"])
    y, hn, gain, nxt, gate = _np(v["y"]), _np(h), _np(v["gain"]), _np(v["next_gain"]), _gate(v["gate"])
    dh, dn = (_np(v["dh"]) if use_dh else 0.0 * y), (_np(v["dn"]) if use_dn else None)
    got = ex.norm_residual_grad(v["dh"] if use_dh else None, v["dn"] if use_dn else None, v["y"], h if use_dn else None, gain=v["gain"],
                                gate=v["gate"], residual_scale=scale, next_gain=v["next_gain"] if use_dn else None, eps=eps)
    dy, dres, dgain, dgate, dnext = got
    want = ox.norm_residual_grad(dh, dn, y, hn, gain, None if v["gate"] is None else _np(v["gate"]), scale, nxt, eps)
    rh, ry = (1 / np.sqrt(np.mean(t * t, 1, keepdims=True) + eps) for t in (hn, y))
    t = want[1] / scale
    dt = C * np.abs(dh)
    if use_dn:
        dt = dt + _norm_slack(dn, 0.0 * y, hn, rh, nxt)
        _close(dnext, want[4], (T + 64) * 2.0 ** -24 * np.abs(dn * hn * rh).sum(0), "dnext_gain")
    else:
        assert dnext is None
    _close(dres, want[1], scale * dt + C * np.abs(want[1]), "dres")
    yh, s, ds = np.abs(y * ry), t * gate, np.abs(gate) * dt
    _close(dy, want[0], _norm_slack(s, ds, y, ry, gain), "dy")
    _close(dgain, want[2], (ds * yh).sum(0) + (T + 64) * 2.0 ** -24 * np.abs(s * yh).sum(0), "dgain")
    if v["gate"] is None:
        assert dgate is None
    else:
        each = np.abs(gain) * yh * (dt + C * np.abs(t))
        assert dgate.shape == v["gate"].shape and dgate.dtype == v["gate"].dtype
        _close(dgate, want[3], each if v["gate"].dim() == 2 else each.sum(1), "dgate")
    return got


SIZES = [(1, 1), (1, 7168), (2, 64), (5, 7), (33, 200), (700, 33), (9, 512), (17, 520), (300, 1000), (40, 1024), (12, 3584), (300, 2048),
         (3, 8192), (6, 8200), (2, 16384), (5, 5001), (64, 13), (2000, 8)]


@ALL
@GATES
@pytest.mark.parametrize("T,D", SIZES, ids=[f"T{t}D{d}" for t, d in SIZES])
def test_norm_residual_and_gradient(T, D, gate, dt):
    v = _inputs(T, D, gate, dt)
    h = _check_forward(v, 0.75)
    _check_backward(v, h, 0.75)


@GATES
@pytest.mark.parametrize("D", [96, 2050, 7168])
def test_either_gradient_alone_and_no_gains(D, gate):
    v = _inputs(21, D, gate, BF)
    h = _check_forward(v, 1.0)
    _check_backward(v, h, 1.0, use_dn=False)
    _check_backward(v, h, 1.0, use_dh=False)
    ones = dict(v, gain=torch.ones(D, device="cuda"), next_gain=torch.ones(D, device="cuda"))
    got = ex.norm_residual_grad(v["dh"], v["dn"], v["y"], h, gate=v["gate"])
    want = ex.norm_residual_grad(v["dh"], v["dn"], v["y"], h, gain=ones["gain"], gate=v["gate"], next_gain=ones["next_gain"])
    assert got[2] is None and got[4] is None and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(ex.norm_residual(v["y"], v["res"], gate=v["gate"])[0],
                       ex.norm_residual(v["y"], v["res"], gain=ones["gain"], gate=v["gate"])[0])


@ALL
@pytest.mark.parametrize("T,D", SIZES, ids=[f"T{t}D{d}" for t, d in SIZES])
def test_rms_norm_and_gradient(T, D, dt):
    v = _inputs(T, D, "none", dt)
    x, gain, dy, add, eps = v["y"], v["gain"], v["dn"], v["dh"], 1e-5
    xn, gn, dn = _np(x), _np(gain), _np(dy)
    want = ox.rms_norm(xn, gn, eps)
    _close(ex.rms_norm(x, gain, eps), want, C * np.abs(want), "norm")
    r = 1 / np.sqrt(np.mean(xn * xn, 1, keepdims=True) + eps)
    slack = _norm_slack(dn, 0.0 * dn, xn, r, gn)
    for a in (None, add):
        dx, dgain = ex.rms_norm_grad(dy, x, gain, eps, add=a)
        wx, wg = ox.rms_norm_grad(dn, xn, gn, eps, None if a is None else _np(a))
        _close(dx, wx, slack + (0 if a is None else C * np.abs(_np(a))), "dx")
        _close(dgain, wg, (T + 64) * 2.0 ** -24 * np.abs(dn * xn * r).sum(0), "dgain")
    assert ex.rms_norm_grad(dy, x, None, eps)[1] is None
    want = ox.rms_norm(xn, None, eps)
    _close(ex.rms_norm(x, eps=eps), want, C * np.abs(want), "no gain")


@pytest.mark.parametrize("dt", [BF, F16], ids=["bf16", "f16"])
def test_gains_of_the_rows_type(dt):
    for D in (256, 777):
        v = _inputs(30, D, "full", dt, gain_dt=dt)
        h = _check_forward(v, 1.25)
        got = _check_backward(v, h, 1.25)
        assert got[2].dtype == F32 and got[4].dtype == F32


def test_views_unaligned_rows_and_in_place():
    T, D = 19, 264
    v = _inputs(T, D, "full", BF)
    h, n = ex.norm_residual(v["y"], v["res"], gain=v["gain"], gate=v["gate"], next_gain=v["next_gain"])
    for pad, at in ((8, 0), (8, 8), (5, 3)):
        wide = {}
        for k in ("y", "res", "gate", "dh", "dn"):
            t = torch.full((T, D + pad + at), float("nan"), dtype=BF, device="cuda")
            t[:, at:at + D] = v[k]
            wide[k] = t[:, at:at + D]
        out = torch.zeros(T, D + pad + at, dtype=BF, device="cuda")
        a, b = ex.norm_residual(wide["y"], wide["res"], gain=v["gain"], gate=wide["gate"], next_gain=v["next_gain"], out=out[:, at:at + D])
        # other pieces of a row a thread: the sums' order may differ in the last bit of fp32, the results in their own
        assert torch.allclose(a.float(), h.float(), rtol=2.0 ** -7, atol=1e-6) and torch.allclose(b.float(), n.float(), rtol=2.0 ** -7, atol=1e-6)
        assert not out[:, :at].any() and not out[:, at + D:].any()
        _check_backward(dict(v, **wide), a, 1.0)
    for k in ("y", "res", "gate"):                           # h over an input
        w = {x: v[x].clone() for x in ("y", "res", "gate")}
        a, b = ex.norm_residual(w["y"], w["res"], gain=v["gain"], gate=w["gate"], next_gain=v["next_gain"], out=w[k])
        assert a.data_ptr() == w[k].data_ptr() and torch.equal(a, h) and torch.equal(b, n)
    x = v["y"].clone()
    want = ex.rms_norm(x, v["gain"])
    assert torch.equal(ex.rms_norm(x, v["gain"], out=x), want) and torch.equal(x, want)
    dx, _ = ex.rms_norm_grad(v["dn"], v["y"], v["gain"], add=v["dh"])
    for k in ("dn", "y", "dh"):
        w = {x: v[x].clone() for x in ("dn", "y", "dh")}
        assert torch.equal(ex.rms_norm_grad(w["dn"], w["y"], v["gain"], add=w["dh"], out=w[k])[0], dx)


def test_rows_of_zeros_infinities_and_nan_stay_in_their_row():
    T, D = 50, 384
    v = _inputs(T, D, "full", BF)
    v["y"][3], v["res"][3] = 0, 0                            # a zero row: rs is 1 / sqrt(eps)
    v["y"][7, 5], v["res"][9, 1], v["gate"][11, 2] = float("inf"), float("nan"), float("nan")
    h, n = ex.norm_residual(v["y"], v["res"], gain=v["gain"], gate=v["gate"], next_gain=v["next_gain"])
    good = torch.ones(T, dtype=torch.bool, device="cuda")
    good[[7, 9, 11]] = False
    assert torch.isfinite(h[good]).all() and torch.isfinite(n[good]).all() and not h[3].any() and not n[3].any()
    assert torch.isnan(n[[9, 11]]).all() and torch.isnan(h[7, 5])
    got = ex.norm_residual_grad(v["dh"], v["dn"], v["y"], h, gain=v["gain"], gate=v["gate"], next_gain=v["next_gain"])
    for t in (got[0], got[1], got[3]):
        assert torch.isfinite(t[good]).all()
    clean = {k: (t[good] if torch.is_tensor(t) and t.shape[0] == T else t) for k, t in v.items()}
    _check_backward(clean, h[good], 1.0)


def test_no_rows_give_zero_gains_gradients():
    v = _inputs(3, 256, "row", BF)
    e = {k: (t[:0] if torch.is_tensor(t) and t.shape[0] == 3 else t) for k, t in v.items()}
    h, n = ex.norm_residual(e["y"], e["res"], gain=v["gain"], gate=e["gate"], next_gain=v["next_gain"])
    assert h.shape == n.shape == (0, 256)
    got = ex.norm_residual_grad(e["dh"], e["dn"], e["y"], h, gain=v["gain"], gate=e["gate"], next_gain=v["next_gain"])
    assert not got[2].any() and not got[4].any() and got[0].shape == (0, 256) and got[3].shape == (0,)
    dx, dg = ex.rms_norm_grad(e["dn"], e["y"], v["gain"])
    assert dx.shape == (0, 256) and not dg.any()


def test_bit_for_bit_other_streams_and_a_graph():
    v = _inputs(1000, 1536, "full", BF)
    run = lambda **k: ex.norm_residual_grad(v["dh"], v["dn"], v["y"], h, gain=v["gain"], gate=v["gate"], next_gain=v["next_gain"], **k)  # noqa: E731
    h, n = ex.norm_residual(v["y"], v["res"], gain=v["gain"], gate=v["gate"], next_gain=v["next_gain"])
    want = run()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(), want))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [run(stream=s) for s in streams]                   # two calls at once, a workspace each
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h, n = ex.norm_residual(v["y"], v["res"], gain=v["gain"], gate=v["gate"], next_gain=v["next_gain"])
        got = run()
    v["y"].mul_(-1.5)
    g.replay()
    torch.cuda.synchronize()
    again = ex.norm_residual(v["y"], v["res"], gain=v["gain"], gate=v["gate"], next_gain=v["next_gain"])
    assert torch.equal(again[0], h) and torch.equal(again[1], n) and all(torch.equal(a, b) for a, b in zip(run(), got))


def test_element_offsets_past_31_bits():
    T, D = 700_000, 3584
    x = torch.empty(T, D, dtype=BF, device="cuda")
    x[-40:] = torch.randn(40, D, device="cuda", generator=_gen(3)).to(BF)
    x[:-40] = 1.0
    gain = torch.ones(D, device="cuda")
    assert torch.equal(ex.rms_norm(x, gain)[-40:], ex.rms_norm(x[-40:], gain))
    dx, _ = ex.rms_norm_grad(x, x, gain, out=x)
    assert torch.isfinite(dx[-40:]).all()
    del x, dx
    torch.cuda.empty_cache()


def test_refusals_of_the_binding():
    v = _inputs(8, 64, "row", BF)
    y, res, g = v["y"], v["res"], v["gain"]
    half = g.half()
    for call in (lambda: ex.rms_norm(y, g[:63]), lambda: ex.rms_norm(y, half), lambda: ex.rms_norm(y, g, eps=0.0), lambda: ex.rms_norm(y.T),
                 lambda: ex.rms_norm(y[0]), lambda: ex.norm_residual(y, res[:4]), lambda: ex.norm_residual(y, res.half()),
                 lambda: ex.norm_residual(y, res, gate=v["gate"][:4]), lambda: ex.norm_residual(y, res, gate=v["gate"].to(BF)),
                 lambda: ex.norm_residual(y, res, gate=res.float()), lambda: ex.norm_residual(y, res, gain=g, next_gain=g.to(BF)),
                 lambda: ex.norm_residual_grad(None, None, y, res), lambda: ex.norm_residual_grad(None, y, y, None),
                 lambda: ex.norm_residual_grad(y, None, y, res, next_gain=g), lambda: ex.norm_residual_grad(y, y[:3], y, res),
                 lambda: ex.rms_norm_grad(y, y, g, add=res.float()), lambda: ex.rms_norm(y, g, out=res.float())):
        with pytest.raises(K3Error) as err:
            call()
        assert err.value.code == ERR_CODE["ARG"]
    for code, call in (("SHAPE", lambda: ex.rms_norm(torch.zeros(1, 16385, device="cuda"))), ("UNSUPPORTED", lambda: ex.rms_norm(y.double())),
                       ("ALIAS", lambda: ex.rms_norm(y[:4], out=y[1:5])), ("ALIAS", lambda: ex.norm_residual(y[:4], res[:4], out=res[2:6]))):
        with pytest.raises(K3Error) as err:
            call()
        assert err.value.code == ERR_CODE[code]
