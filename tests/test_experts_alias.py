"""Every output of the expert training operators that would be written over one of the call's own inputs or other
outputs is refused, the small tables (routing, offsets, weights, workspace) among them.  Addresses only: a refused
call touches nothing."""
import ctypes as C

import pytest

ALIAS = -5
T, K, D, E, ROWS = 4, 2, 64, 4, 32


@pytest.fixture(scope="module")
def lib():
    from latent_moe_layer_gb300 import build, k3moe
    build.build()
    return k3moe.lib()


def _check(call, outputs, others, allowed=()):
    """call(**addresses) is refused wherever an output shares memory with another argument, and only there: the
    first and the last byte of either."""
    names = {**outputs, **others}
    apart = {n: (i + 1) << 40 for i, n in enumerate(names)}
    for o in outputs:
        for n in names:
            if n == o:
                continue
            for at in (apart[n], apart[n] + names[n] - 4, apart[n] - outputs[o] + 4):
                if (o, n) in allowed and at == apart[n]:
                    continue
                a = {k: C.c_void_p(v) for k, v in {**apart, o: at}.items()}
                assert call(**a) == ALIAS, (o, n, at - apart[n])


def test_plan(lib):
    ws = lib.k3moe_rows_plan_workspace_bytes(T, K, E)
    _check(lambda idx, offsets, pos, work: lib.k3moe_rows_plan(idx, T, K, 0, E, offsets, pos, work, ws, None),
           {"offsets": 4 * (E + 1), "pos": 4 * T * K, "work": ws}, {"idx": 4 * T * K})


def test_rows(lib):
    x, rows, table = 2 * T * D, 2 * ROWS * D, 4 * T * K
    st = C.c_void_p(1 << 50)
    _check(lambda x, pos, out: lib.k3moe_rows_gather(x, D, pos, T, K, D, 1, out, D, ROWS, st, None),
           {"out": rows}, {"x": x, "pos": table})
    _check(lambda y, pos, w, z: lib.k3moe_rows_combine(y, D, ROWS, pos, w, T, K, D, 1, z, D, st, None),
           {"z": x}, {"y": rows, "pos": table, "w": table})
    _check(lambda dz, y, pos, w, dy, dw: lib.k3moe_rows_combine_grad(dz, D, y, D, ROWS, pos, w, T, K, D, 1, dy, D, dw, st, None),
           {"dy": rows, "dw": table}, {"dz": x, "y": rows, "pos": table, "w": table}, allowed=[("dy", "y")])


def test_products(lib):
    n_out = 96
    st, off, w = C.c_void_p(1 << 50), 4 * (E + 1), 2 * E * n_out * D
    _check(lambda offsets, x, w, y: lib.k3moe_group_mm(offsets, E, ROWS, D, n_out, x, D, w, D, n_out * D, 1, y, n_out, 1, st, None),
           {"y": 2 * ROWS * n_out}, {"offsets": off, "x": 2 * ROWS * D, "w": w})
    _check(lambda offsets, dy, w, dx: lib.k3moe_group_mm_grad_x(offsets, E, ROWS, D, n_out, dy, n_out, w, D, n_out * D, 1, dx, D, 1,
                                                              st, None),
           {"dx": 2 * ROWS * D}, {"offsets": off, "dy": 2 * ROWS * n_out, "w": w})
    _check(lambda offsets, dy, x, dw: lib.k3moe_group_mm_grad_w(offsets, E, ROWS, D, n_out, dy, n_out, x, D, 1, dw, D, n_out * D, 0, 0,
                                                              st, None),
           {"dw": 4 * E * n_out * D}, {"offsets": off, "dy": 2 * ROWS * n_out, "x": 2 * ROWS * D})


def test_units(lib):
    _check(lambda gu, a: lib.k3moe_glu_dropout(gu, 2 * D, ROWS, D, 1, 0, 4.0, 25.0, 0.1, 1, 2, a, D, None),
           {"a": 2 * ROWS * D}, {"gu": 4 * ROWS * D})
    _check(lambda da, gu, dgu: lib.k3moe_glu_dropout_grad(da, D, gu, 2 * D, ROWS, D, 1, 0, 4.0, 25.0, 0.1, 1, 2, dgu, 2 * D, None),
           {"dgu": 4 * ROWS * D}, {"da": 2 * ROWS * D, "gu": 4 * ROWS * D}, allowed=[("dgu", "gu")])
    _check(lambda x, r, out: lib.k3moe_dropout(x, r, 1000, 0, 0.1, 1, 2, out, None), {"out": 4000}, {"x": 4000, "r": 4000},
           allowed=[("out", "x"), ("out", "r")])
