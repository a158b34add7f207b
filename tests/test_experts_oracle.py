"""The fp64 definitions of the expert training operators: the generator against its published known
answers, gradients against central differences, the plan against its properties; and the refusals of
the library's entry points, which need no GPU."""
import ctypes as C

import numpy as np
import pytest

from oracle import experts as ox


@pytest.mark.parametrize("counter,key,want", [
    # known answers of the authors' Random123 distribution, philox4x32 with 10 rounds
    ([0, 0, 0, 0], [0, 0], [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]),
    ([0xffffffff] * 4, [0xffffffff] * 2, [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]),
    ([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0],
     [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1])])
def test_philox_known_answers(counter, key, want):
    assert [int(v) for v in ox.philox(counter, key)] == want


def test_keep_mask_rate_and_independence():
    n = 200_000
    for p in (0.1, 0.5, 0.9):
        a = ox.keep_mask(np.arange(n), p, 7, 0)
        # binomial, five standard deviations
        assert abs(a.mean() - (1 - p)) < 5 * np.sqrt(p * (1 - p) / n)
        b = ox.keep_mask(np.arange(n), p, 7, 1)
        both = (a & b).mean()
        assert abs(both - (1 - p) ** 2) < 5 * np.sqrt((1 - p) ** 2 * (1 - (1 - p) ** 2) / n)
    assert ox.keep_mask(np.arange(100), 0.0, 7, 0).all()
    # indices past 32 bits are their own elements
    far = np.arange(64, dtype=np.uint64) + np.uint64(1 << 34)
    assert not np.array_equal(ox.keep_mask(far, 0.5, 7, 0), ox.keep_mask(np.arange(64), 0.5, 7, 0))


@pytest.mark.parametrize("act", ["silu", "situ"])
@pytest.mark.parametrize("p", [0.0, 0.4])
def test_glu_gradient_against_differences(act, p):
    rng = np.random.default_rng(1)
    gu, da = rng.standard_normal((5, 24)) * 2, rng.standard_normal((5, 12))
    got = ox.glu_dropout_grad(da, gu, p, 3, 9, act)
    eps = 1e-5
    for i in range(gu.shape[0]):
        for j in range(gu.shape[1]):
            d = np.zeros_like(gu)
            d[i, j] = eps
            diff = (ox.glu_dropout(gu + d, p, 3, 9, act) - ox.glu_dropout(gu - d, p, 3, 9, act)) / (2 * eps)
            # central difference: eps^2 f'''/6 plus 2^-53 / eps rounding, both below 1e-9 of values of order 10
            assert abs((diff * da).sum() - got[i, j]) < 1e-7


def test_combine_and_product_gradients_against_differences():
    rng = np.random.default_rng(2)
    idx = rng.integers(0, 6, (7, 3))
    offsets, pos = ox.plan_rows(idx, 4, 1)              # experts 1 .. 4 of 0 .. 5 are local
    n = int(offsets[-1])
    x, w = rng.standard_normal((n, 5)), rng.standard_normal((4, 6, 5))
    mix, dz = rng.random((7, 3)), rng.standard_normal((7, 6))

    def loss(x, w, mix):
        return (ox.combine_rows(ox.group_mm(x, w, offsets), pos, mix) * dz).sum()

    y = ox.group_mm(x, w, offsets)
    dy, dmix = ox.combine_rows_grad(dz, y, pos, mix)
    grads = (ox.group_mm_grad_x(dy, w, offsets), ox.group_mm_grad_w(dy, x, offsets), dmix)
    args, eps = (x, w, mix), 1e-6
    for a, g in enumerate(grads):
        for i in np.ndindex(args[a].shape):
            lo, hi = [v.copy() for v in args], [v.copy() for v in args]
            lo[a][i] -= eps
            hi[a][i] += eps
            assert abs((loss(*hi) - loss(*lo)) / (2 * eps) - g[i]) < 1e-7     # multilinear: rounding alone


def test_plan_properties():
    rng = np.random.default_rng(3)
    idx = rng.integers(-1, 12, (40, 4))
    offsets, pos = ox.plan_rows(idx, 5, 4)
    used = np.sort(pos[pos >= 0])
    assert np.array_equal(used, np.arange(offsets[-1]))
    assert np.array_equal(pos < 0, (idx < 4) | (idx >= 9))
    for e in range(5):
        rows = pos.reshape(-1)[idx.reshape(-1) == e + 4]
        assert np.array_equal(rows, np.arange(offsets[e], offsets[e + 1]))


# ---------------------------------------------------------------------------------------------- refusals
ARG, SHAPE, ALIAS, WORKSPACE, UNSUPPORTED = -1, -2, -5, -6, -9


@pytest.fixture(scope="module")
def lib():
    from latent_moe_layer_gb300 import build, k3moe
    build.build()
    return k3moe.lib()


P = [C.c_void_p((i + 1) << 40) for i in range(6)]        # far apart; the refused calls never touch them


def test_plan_refusals(lib):
    ws = lib.k3moe_rows_plan_workspace_bytes
    assert ws(8192, 16, 896) >= 4 * 64 * 896 and ws(0, 1, 1) > 0
    assert ws(-1, 16, 896) == 0 and ws(1 << 27, 16, 896) == 0 and ws(16, 16, 2000) == 0
    call = lambda *a: lib.k3moe_rows_plan(*a, None)  # noqa: E731
    assert call(P[0], -1, 2, 0, 4, P[1], P[2], P[3], 1 << 20) == ARG
    assert call(P[0], 4, 0, 0, 4, P[1], P[2], P[3], 1 << 20) == ARG
    assert call(P[0], 4, 2, -1, 4, P[1], P[2], P[3], 1 << 20) == ARG
    assert call(P[0], 4, 2, (1 << 31) - 2, 4, P[1], P[2], P[3], 1 << 20) == ARG
    assert call(None, 4, 2, 0, 4, P[1], P[2], P[3], 1 << 20) == ARG
    assert call(P[0], 4, 2, 0, 4, None, P[2], P[3], 1 << 20) == ARG
    assert call(P[0], 4, 2, 0, 2000, P[1], P[2], P[3], 1 << 20) == SHAPE
    assert call(P[0], 4, 2, 0, 4, P[1], P[2], None, 0) == WORKSPACE
    assert call(P[0], 4, 2, 0, 4, P[1], P[2], P[3], 8) == WORKSPACE
    assert call(P[0], 4, 2, 0, 4, P[1], P[0], P[3], 1 << 20) == ALIAS


def test_rows_refusals(lib):
    g = lambda *a: lib.k3moe_rows_gather(*a, None)  # noqa: E731
    assert g(P[0], 8, P[1], 4, 2, 8, 1, P[2], 7, 8, P[3]) == ARG          # ldo < D
    assert g(P[0], 8, P[1], 4, 2, 8, 0, P[2], 8, 8, P[3]) == UNSUPPORTED  # fp32 rows
    assert g(P[0], 8, P[1], 4, 2, 8, 1, P[0], 8, 8, P[3]) == ALIAS
    assert g(P[0], 8, None, 4, 2, 8, 1, P[2], 8, 8, P[3]) == ARG
    assert g(P[0], 8, P[1], 4, 2, 8, 1, P[2], 8, 8, None) == ARG          # no status word
    assert g(None, 8, None, 0, 2, 8, 1, None, 8, 0, None) == 0            # no tokens: nothing to do
    c = lambda *a: lib.k3moe_rows_combine(*a, None)  # noqa: E731
    assert c(P[0], 8, 8, P[1], None, 4, 2, 8, 1, P[0], 8, P[3]) == ALIAS
    assert c(P[0], 8, 8, P[1], None, 4, 2, 8, 3, P[2], 8, P[3]) == UNSUPPORTED
    assert c(P[0], 7, 8, P[1], None, 4, 2, 8, 1, P[2], 8, P[3]) == ARG
    d = lambda *a: lib.k3moe_rows_combine_grad(*a, None)  # noqa: E731
    assert d(P[0], 8, P[1], 8, 8, P[2], P[3], 4, 2, 8, 1, P[0], 8, P[4], P[5]) == ALIAS
    assert d(P[0], 8, P[1], 8, 8, P[2], P[3], 4, 2, 8, 1, P[1], 16, P[4], P[5]) == ALIAS   # y, another stride
    assert d(P[0], 8, P[1], 8, 8, P[2], P[3], 4, 2, 8, 1, C.c_void_p(P[4].value + (1 << 20)), 8, P[3], P[5]) == ALIAS
    assert d(P[0], 8, P[1], 8, 8, P[2], None, 4, 2, 8, 1, P[4], 8, P[4], P[5]) == ARG


@pytest.mark.parametrize("name", ["k3moe_group_mm", "k3moe_group_mm_grad_x"])
def test_group_refusals(lib, name):
    def call(off=P[0], E=4, rows=32, n_in=64, n_out=64, x=P[1], ldx=64, w=P[2], ldw=64, sw=4096, dt=1, y=P[3], ldy=64,
             odt=1, st=P[4]):
        return getattr(lib, name)(off, E, rows, n_in, n_out, x, ldx, w, ldw, sw, dt, y, ldy, odt, st, None)
    assert call(off=None) == ARG and call(E=0) == ARG and call(rows=-1) == ARG and call(n_in=0) == ARG
    assert call(st=None) == ARG and call(x=None) == ARG and call(w=None) == ARG and call(y=None) == ARG
    assert call(ldx=63) == ARG and call(ldw=63) == ARG and call(ldy=63) == ARG and call(sw=-1) == ARG
    assert call(E=1025) == SHAPE
    assert call(dt=0) == UNSUPPORTED and call(odt=2) == UNSUPPORTED and call(dt=5) == UNSUPPORTED
    assert call(y=P[1]) == ALIAS and call(y=C.c_void_p(P[2].value + 100)) == ALIAS
    assert call(rows=0, x=None, y=None) == 0


def test_group_grad_w_refusals(lib):
    def call(off=P[0], E=4, rows=32, n_in=64, n_out=64, dy=P[1], lddy=64, x=P[2], ldx=64, dt=1, dw=P[3], ldw=64, sw=4096,
             odt=0, acc=0, st=P[4]):
        return lib.k3moe_group_mm_grad_w(off, E, rows, n_in, n_out, dy, lddy, x, ldx, dt, dw, ldw, sw, odt, acc, st, None)
    assert call(dw=None) == ARG and call(dy=None) == ARG and call(x=None) == ARG and call(acc=2) == ARG
    assert call(lddy=63) == ARG and call(ldx=63) == ARG and call(ldw=63) == ARG and call(sw=4095) == ARG
    assert call(odt=1, acc=1) == UNSUPPORTED and call(odt=2) == UNSUPPORTED
    assert call(dw=P[2]) == ALIAS and call(E=1025) == SHAPE and call(off=None) == ARG


def test_glu_and_dropout_refusals(lib):
    def glu(gu=P[0], ld=64, rows=4, width=32, dt=1, act=0, b=4.0, lb=25.0, p=0.1, a=P[1], lda=32):
        return lib.k3moe_glu_dropout(gu, ld, rows, width, dt, act, b, lb, p, 1, 2, a, lda, None)
    assert glu(gu=None) == ARG and glu(ld=63) == ARG and glu(lda=31) == ARG and glu(width=0) == ARG and glu(rows=-1) == ARG
    assert glu(p=1.0) == ARG and glu(p=-0.1) == ARG and glu(p=float("nan")) == ARG and glu(b=float("nan")) == ARG
    assert glu(dt=0) == UNSUPPORTED and glu(act=7) == UNSUPPORTED and glu(a=P[0]) == ALIAS
    assert glu(rows=0, gu=None, a=None) == 0

    def grad(da=P[0], ldda=32, gu=P[1], ldgu=64, rows=4, width=32, dt=1, act=0, p=0.1, out=P[2], ldo=64):
        return lib.k3moe_glu_dropout_grad(da, ldda, gu, ldgu, rows, width, dt, act, 4.0, 25.0, p, 1, 2, out, ldo, None)
    assert grad(da=None) == ARG and grad(ldda=31) == ARG and grad(ldo=63) == ARG
    assert grad(out=P[0]) == ALIAS and grad(out=P[1], ldo=72) == ALIAS
    drop = lambda x, r, n, dt, p, o: lib.k3moe_dropout(x, r, n, dt, p, 1, 2, o, None)  # noqa: E731
    assert drop(None, None, 4, 0, 0.1, P[1]) == ARG and drop(P[0], None, -1, 0, 0.1, P[1]) == ARG
    assert drop(P[0], None, 4, 0, 1.0, P[1]) == ARG and drop(P[0], None, 4, 9, 0.1, P[1]) == UNSUPPORTED
    assert drop(P[0], None, 4, 0, 0.1, C.c_void_p(P[0].value + 4)) == ALIAS
    assert drop(None, None, 0, 0, 0.1, None) == 0


def test_binding_refuses_host_tensors_and_bad_arguments():
    torch = pytest.importorskip("torch")
    from latent_moe_layer_gb300 import experts as ex
    from latent_moe_layer_gb300.k3moe import K3Error
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    pos = torch.zeros(4, 2, dtype=torch.int32)
    off = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: ex.plan_rows(pos, 4), lambda: ex.gather_rows(x, pos), lambda: ex.combine_rows(x, pos),
                 lambda: ex.combine_rows_grad(x, x, pos, pos.float()), lambda: ex.group_mm(x, x[None], off),
                 lambda: ex.group_mm_grad_x(x, x[None], off), lambda: ex.group_mm_grad_w(x, x, off),
                 lambda: ex.glu_dropout(x), lambda: ex.glu_dropout_grad(x, x), lambda: ex.dropout(x, 0.1, 1, 2)):
        with pytest.raises(K3Error) as err:
            call()
        assert err.value.code == ARG
