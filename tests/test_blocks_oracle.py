"""The fp64 definitions of the 8-bit operands, the gated block and the norms around a block: the rounding against
PyTorch's own conversion, gradients against central differences; and the refusals of the library's entry points and of
the binding, which need no GPU."""
import ctypes as C

import numpy as np
import pytest

from oracle import experts as ox

ARG, SHAPE, ALIAS, WORKSPACE, UNSUPPORTED = -1, -2, -5, -6, -9
P = [C.c_void_p((i + 1) << 40) for i in range(12)]       # far apart; the refused calls never touch them


@pytest.fixture(scope="module")
def lib():
    from latent_moe_layer_gb300 import build, k3moe
    build.build()
    return k3moe.lib()


# ---------------------------------------------------------------------------------------------- definitions
@pytest.mark.parametrize("kind,name", [("e4m3", "float8_e4m3fn"), ("e5m2", "float8_e5m2")])
def test_rounding_is_the_formats(kind, name):
    torch = pytest.importorskip("torch")
    every = torch.arange(256, dtype=torch.uint8).view(getattr(torch, name)).double().numpy()
    every = every[np.isfinite(every)]
    assert np.max(every) == ox.F8[kind][2] and np.array_equal(ox.round8(every, kind), every)
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.standard_normal(4000) * 2.0 ** rng.integers(-20, 9, 4000), (every[1:] + every[:-1]) / 2])
    v = v[np.abs(v) <= ox.F8[kind][2]]                   # halfway cases among them
    assert np.array_equal(ox.round8(v, kind), torch.from_numpy(v).float().to(getattr(torch, name)).double().numpy())
    got = ox.round8(np.array([np.inf, -np.inf, np.nan]), kind)
    assert np.isnan(got[2]) and (np.isnan(got[:2]).all() if kind == "e4m3" else np.array_equal(got[:2], [np.inf, -np.inf]))


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_scale_is_the_smallest_that_saturates_nothing(kind):
    top = ox.F8[kind][2]
    for k in (-127, -126, -20, 0, 3, 100):
        assert ox.scale_exponent(top * 2.0 ** k, kind) == k
        assert ox.scale_exponent(np.nextafter(top * 2.0 ** k, np.inf), kind) == k + 1
    assert ox.scale_exponent(0.0, kind) == -127
    x = np.array([[1.0, np.nan, -3.0, np.inf] + [0.0] * 200])
    codes, scales = ox.quant8(x, kind)
    assert scales.shape == (1, 2) and scales[0, 1] == 0 and scales[0, 0] == 127 + ox.scale_exponent(3.0, kind)
    back = ox.dequant8(codes, scales)
    assert back[0, 0] == 1.0 and back[0, 2] == -3.0 and np.isnan(back[0, 1])


def _difference(f, args, i, grad, eps, tol, rng, n=20):
    for _ in range(n):
        j = tuple(rng.integers(0, s) for s in args[i].shape)
        lo, hi = [a.copy() for a in args], [a.copy() for a in args]
        lo[i][j] -= eps
        hi[i][j] += eps
        assert abs((f(*hi) - f(*lo)) / (2 * eps) - grad[j]) < tol, (i, j)


@pytest.mark.parametrize("gate", ["none", "row", "full"])
def test_norm_gradients_against_differences(gate):
    rng = np.random.default_rng(4)
    T, D = 5, 7
    y, res, gain, nxt = rng.standard_normal((T, D)), rng.standard_normal((T, D)), rng.random(D) + 0.5, rng.random(D) + 0.5
    g = {"none": np.zeros((0,)), "row": rng.random(T), "full": rng.random((T, D))}[gate]
    dh, dn = rng.standard_normal((T, D)), rng.standard_normal((T, D))
    of = lambda g: None if gate == "none" else g  # noqa: E731

    def loss(y, res, gain, nxt, g):
        h, n = ox.norm_residual(y, res, gain, of(g), 0.75, nxt, 1e-3)
        return (h * dh).sum() + (n * dn).sum()

    h, _ = ox.norm_residual(y, res, gain, of(g), 0.75, nxt, 1e-3)
    dy, dres, dgain, dgate, dnext = ox.norm_residual_grad(dh, dn, y, h, gain, of(g), 0.75, nxt, 1e-3)
    args = [y, res, gain, nxt, g]
    # values of order 10: rounding 1e-15 10 / 2e-5 and eps^2 of a third derivative of order 10, both below 1e-8
    for i, d in ((0, dy), (1, dres), (2, dgain), (3, dnext)) + (() if gate == "none" else ((4, dgate),)):
        _difference(loss, args, i, d, 1e-5, 1e-7, rng)
    dx, dg = ox.rms_norm_grad(dn, y, gain, 1e-3, add=dh)
    alone = lambda y, gain: (ox.rms_norm(y, gain, 1e-3) * dn).sum() + (y * dh).sum()  # noqa: E731
    _difference(alone, [y, gain], 0, dx, 1e-5, 1e-7, rng)
    _difference(alone, [y, gain], 1, dg, 1e-5, 1e-7, rng)


@pytest.mark.parametrize("act", ["silu", "situ"])
def test_gated_block_gradients_against_differences(act):
    rng = np.random.default_rng(5)
    off = np.array([0, 4, 4, 9])
    x, w, da = rng.standard_normal((9, 6)), rng.standard_normal((3, 10, 6)), rng.standard_normal((9, 5))
    loss = lambda x, w: (ox.group_glu(x, w, off, act) * da).sum()  # noqa: E731
    dgu = ox.group_glu_grad(da, x, w, off, act)
    _difference(loss, [x, w], 0, ox.group_mm_grad_x(dgu, w, off), 1e-6, 1e-7, rng)
    _difference(loss, [x, w], 1, ox.group_mm_grad_w(dgu, x, off), 1e-6, 1e-7, rng)


# ---------------------------------------------------------------------------------------------- refusals
def _rejects(call, cases):
    for code, changes in cases:
        for change in changes:
            assert call(**change) == code, (code, change)


def test_quant8_refusals(lib):
    def rows(x=P[0], ldx=256, rows=4, n=256, dt=1, kind=0, c=P[1], ldc=256, s=P[2], lds=2):
        return lib.k3moe_quant8_rows(x, ldx, rows, n, dt, kind, c, ldc, s, lds, None)
    _rejects(rows, [(ARG, [dict(x=None), dict(c=None), dict(s=None), dict(rows=-1), dict(n=0), dict(ldx=255), dict(ldc=255), dict(lds=1)]),
                    (UNSUPPORTED, [dict(dt=0), dict(kind=2)]),
                    (ALIAS, [dict(c=P[0]), dict(s=P[0]), dict(s=P[1]), dict(c=C.c_void_p(P[0].value + 2 * 1024 - 1))])])
    assert rows(rows=0, x=None, c=None, s=None) == 0

    def weights(w=P[0], ldw=256, sw=256 * 300, E=2, N=300, K=256, dt=1, kind=0, c=P[1], ldc=256, sc=256 * 300, t=P[2], ldt=304,
                st=304 * 256, s=P[3]):
        return lib.k3moe_quant8_weights(w, ldw, sw, E, N, K, dt, kind, c, ldc, sc, t, ldt, st, s, None)
    _rejects(weights, [(ARG, [dict(w=None), dict(c=None), dict(s=None), dict(E=0), dict(N=0), dict(K=0), dict(ldw=255), dict(ldc=255),
                              dict(ldt=299), dict(sc=256 * 299), dict(st=304 * 255), dict(sw=-1)]),
                       (UNSUPPORTED, [dict(dt=0), dict(kind=-1)]),
                       (ALIAS, [dict(c=P[0]), dict(t=P[0]), dict(s=P[0]), dict(t=P[1]), dict(s=P[1]), dict(s=P[2])])])


def test_group_mm8_refusals(lib):
    def call(off=P[0], E=4, rows=32, K=256, N=64, x=P[1], ldx=256, xk=0, xs=P[2], ldxs=4, w=P[3], ldw=256, sw=256 * 64, wk=1, ws=P[4],
             sse=2, sso=2, ssi=1, y=P[5], ldy=64, odt=1, st=P[6]):
        return lib.k3moe_group_mm8(off, E, rows, K, N, x, ldx, xk, xs, ldxs, w, ldw, sw, wk, ws, sse, sso, ssi, y, ldy, odt, st, None)
    _rejects(call, [(ARG, [dict(off=None), dict(st=None), dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(y=None), dict(E=0),
                           dict(rows=-1), dict(K=0), dict(N=0), dict(ldx=240), dict(ldw=240), dict(ldy=63), dict(ldxs=1), dict(sw=-16),
                           dict(sse=-1), dict(sso=-1), dict(ssi=-1)]),
                    (SHAPE, [dict(E=1025)]), (UNSUPPORTED, [dict(xk=2), dict(wk=2), dict(odt=3), dict(ldx=264), dict(ldw=264),
                                                            dict(sw=256 * 64 + 8), dict(x=C.c_void_p(P[1].value + 8)),
                                                            dict(w=C.c_void_p(P[3].value + 4)), dict(ldxs=3),
                                                            dict(xs=C.c_void_p(P[2].value + 2))]),
                    (ALIAS, [dict(y=P[1]), dict(y=P[2]), dict(y=P[3]), dict(y=P[4]), dict(y=P[0])])])
    assert call(rows=0, x=None, xs=None, y=None) == 0


@pytest.mark.parametrize("grad", [False, True])
def test_gated_block_refusals(lib, grad):
    def call(off=P[0], E=4, rows=32, K=64, I=40, da=P[5], ldda=40, x=P[1], ldx=64, w=P[2], ldw=64, sw=64 * 80, dt=1, act=0, b=4.0,
             lb=25.0, out=P[3], ldo=80, st=P[4]):
        if grad:
            return lib.k3moe_group_glu_grad(off, E, rows, K, I, da, ldda, x, ldx, w, ldw, sw, dt, act, b, lb, out, ldo, st, None)
        return lib.k3moe_group_glu(off, E, rows, K, I, x, ldx, w, ldw, sw, dt, act, b, lb, out, ldo, st, None)
    _rejects(call, [(ARG, [dict(off=None), dict(st=None), dict(x=None), dict(w=None), dict(out=None), dict(E=0), dict(rows=-1), dict(K=0),
                           dict(I=0), dict(I=1 << 30), dict(ldx=63), dict(ldw=63), dict(ldo=39), dict(sw=-1), dict(b=float("nan")),
                           dict(lb=float("inf"))] + ([dict(da=None), dict(ldda=39), dict(ldo=79)] if grad else [])),
                    (SHAPE, [dict(E=1025)]), (UNSUPPORTED, [dict(dt=0), dict(act=3)]),
                    (ALIAS, [dict(out=P[1]), dict(out=P[2]), dict(out=P[0])] + ([dict(out=P[5])] if grad else []))])
    assert call(rows=0, x=None, out=None, da=None) == 0


def test_norm_refusals(lib):
    def norm(x=P[0], ldx=64, g=P[1], gdt=0, eps=1e-6, rows=4, D=64, dt=1, o=P[2], ldo=64):
        return lib.k3moe_rms_norm(x, ldx, g, gdt, eps, rows, D, dt, o, ldo, None)
    bad = [dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(rows=-1), dict(D=0)]
    _rejects(norm, [(ARG, bad + [dict(x=None), dict(o=None), dict(ldx=63), dict(ldo=63)]), (SHAPE, [dict(D=16385, ldx=20000, ldo=20000)]),
                    (UNSUPPORTED, [dict(dt=3), dict(gdt=2)]),
                    (ALIAS, [dict(o=P[0], ldo=72), dict(o=C.c_void_p(P[0].value + 16)), dict(o=P[1])])])
    assert norm(rows=0, x=None, o=None) == 0

    def post(y=P[0], ldy=64, r=P[1], ldr=64, g=P[2], ng=P[3], gdt=0, gate=P[4], ldg=64, gk=2, scale=1.0, eps=1e-6, rows=4, D=64, dt=1,
             h=P[5], ldh=64, n=P[6], ldn=64):
        return lib.k3moe_norm_residual(y, ldy, r, ldr, g, ng, gdt, gate, ldg, gk, scale, eps, rows, D, dt, h, ldh, n, ldn, None)
    _rejects(post, [(ARG, bad + [dict(y=None), dict(r=None), dict(h=None), dict(gate=None), dict(gk=0), dict(gk=3), dict(ldy=63), dict(ldr=63),
                                 dict(ldg=63), dict(ldh=63), dict(ldn=63)]),
                    (UNSUPPORTED, [dict(dt=3), dict(gdt=2)]),
                    (ALIAS, [dict(h=P[6]), dict(h=P[0], ldh=72), dict(n=P[2]), dict(h=P[3]), dict(n=C.c_void_p(P[4].value + 2)),
                             dict(gk=1, h=P[4])])])
    assert lib.k3moe_norm_grad_workspace_bytes(8, 64) > 0 and lib.k3moe_norm_grad_workspace_bytes(8, 16385) == 0
    big = 1 << 30

    def grad(dy=P[0], x=P[1], g=P[2], add=P[3], dx=P[4], ldx=64, dg=P[5], ws=P[6], nb=big, eps=1e-6, rows=4, D=64, dt=1, gdt=0):
        return lib.k3moe_rms_norm_grad(dy, 64, x, 64, g, gdt, add, 64, eps, rows, D, dt, dx, ldx, dg, ws, nb, None)
    _rejects(grad, [(ARG, bad + [dict(dy=None), dict(x=None), dict(dx=None), dict(ldx=63)]),
                    (WORKSPACE, [dict(ws=None), dict(nb=64), dict(ws=C.c_void_p(P[6].value + 2))]),
                    (ALIAS, [dict(dx=P[0], ldx=72), dict(dx=P[5]), dict(dg=P[1]), dict(ws=P[5]), dict(ws=P[4]), dict(dg=P[2])])])

    def back(dh=P[0], dn=P[1], y=P[2], h=P[3], g=P[4], ng=P[5], gate=P[6], gk=2, dy=P[7], ldd=64, dr=P[8], dgate=P[9], dg=P[10], dng=P[11],
             ws=C.c_void_p(1 << 50), nb=big, eps=1e-6, rows=4, D=64, dt=1, gdt=0):
        return lib.k3moe_norm_residual_grad(dh, 64, dn, 64, y, 64, h, 64, g, ng, gdt, gate, 64, gk, 1.0, eps, rows, D, dt, dy, ldd, dr, 64,
                                            dgate, 64, dg, dng, ws, nb, None)
    _rejects(back, [(ARG, bad + [dict(dh=None, dn=None, dng=None), dict(y=None), dict(h=None), dict(dy=None), dict(dr=None), dict(dgate=None),
                                 dict(gate=None), dict(gk=0), dict(gk=5), dict(dn=None), dict(ldd=63)]),
                    (WORKSPACE, [dict(ws=None), dict(nb=8)]),
                    (ALIAS, [dict(dy=P[8]), dict(dy=P[2], ldd=72), dict(dgate=P[7]), dict(dg=P[11]), dict(dg=P[4]), dict(ws=P[2 + 5]),
                             dict(gk=1, dgate=P[6]), dict(dr=C.c_void_p(P[0].value + 16))])])


def test_binding_refuses_host_tensors_and_gradients():
    torch = pytest.importorskip("torch")
    from latent_moe_layer_gb300 import experts as ex
    from latent_moe_layer_gb300.k3moe import K3Error
    x = torch.zeros(4, 8, dtype=torch.bfloat16, requires_grad=True)
    off, s = torch.zeros(2, dtype=torch.int32), torch.zeros(4, 1, dtype=torch.uint8)
    calls = (lambda: ex.quant8_rows(x), lambda: ex.quant8_weights(x[None]), lambda: ex.group_mm8(x, s, x[None], s[None], off),
             lambda: ex.group_glu(x, x[None], off), lambda: ex.group_glu_grad(x, x, x[None], off), lambda: ex.rms_norm(x),
             lambda: ex.rms_norm_grad(x, x), lambda: ex.norm_residual(x, x), lambda: ex.norm_residual_grad(x, x, x, x))
    for call in calls:
        with pytest.raises(K3Error) as err:
            call()
        assert err.value.code == UNSUPPORTED and "gradients" in str(err.value)
        with torch.no_grad(), pytest.raises(K3Error) as err:             # then only the device is wrong
            call()
        assert err.value.code == ARG
