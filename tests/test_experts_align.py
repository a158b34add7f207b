"""Every pointer of the expert training operators that is not at a multiple of its elements' bytes is refused, each by itself: a
load or store through it would fault.  Addresses only: a refused call touches nothing."""
import ctypes as C

import pytest

from latent_moe_layer_gb300.k3moe import ERR_CODE

R, D, E, T, K = 32, 256, 4, 4, 2


@pytest.fixture(scope="module")
def lib():
    from latent_moe_layer_gb300 import build, k3moe
    build.build()
    return k3moe.lib()


def _check(call, elements):
    """call(**addresses): refused with each of the addresses off by one byte (and by half an element of four)."""
    apart = {n: (i + 1) << 40 for i, n in enumerate(elements)}
    for n, size in elements.items():
        for off in {1, size // 2, size - 1} - {0}:
            got = call(**{k: C.c_void_p(v + (off if k == n else 0)) for k, v in apart.items()})
            assert got == ERR_CODE["ALIGN"], (n, off, got)


def test_rows(lib):
    ws = lib.k3moe_rows_plan_workspace_bytes(T, K, E)
    _check(lambda idx, offsets, pos, work: lib.k3moe_rows_plan(idx, T, K, 0, E, offsets, pos, work, ws, None),
           {"idx": 4, "offsets": 4, "pos": 4, "work": 4})
    _check(lambda x, pos, out, st: lib.k3moe_rows_gather(x, D, pos, T, K, D, 1, out, D, R, st, None), {"x": 2, "pos": 4, "out": 2, "st": 4})
    _check(lambda y, pos, w, z, st: lib.k3moe_rows_combine(y, D, R, pos, w, T, K, D, 1, z, D, st, None),
           {"y": 2, "pos": 4, "w": 4, "z": 2, "st": 4})
    _check(lambda dz, y, pos, w, dy, dw, st: lib.k3moe_rows_combine_grad(dz, D, y, D, R, pos, w, T, K, D, 1, dy, D, dw, st, None),
           {"dz": 2, "y": 2, "pos": 4, "w": 4, "dy": 2, "dw": 4, "st": 4})


@pytest.mark.parametrize("out", [0, 1])
def test_products(lib, out):
    n, size = 96, 2 if out else 4
    _check(lambda off, x, w, y, st: lib.k3moe_group_mm(off, E, R, D, n, x, D, w, D, n * D, 1, y, n, out, st, None),
           {"off": 4, "x": 2, "w": 2, "y": size, "st": 4})
    _check(lambda off, dy, w, dx, st: lib.k3moe_group_mm_grad_x(off, E, R, D, n, dy, n, w, D, n * D, 1, dx, D, out, st, None),
           {"off": 4, "dy": 2, "w": 2, "dx": size, "st": 4})
    _check(lambda off, dy, x, dw, st: lib.k3moe_group_mm_grad_w(off, E, R, D, n, dy, n, x, D, 1, dw, D, n * D, out, 0, st, None),
           {"off": 4, "dy": 2, "x": 2, "dw": size, "st": 4})
    a = {"x": C.c_void_p(1 << 50), "xs": C.c_void_p(1 << 51), "w": C.c_void_p(1 << 52), "ws": C.c_void_p(1 << 53)}
    _check(lambda off, y, st: lib.k3moe_group_mm8(off, E, R, D, n, a["x"], D, 0, a["xs"], 4, a["w"], D, n * D, 0, a["ws"], 2, 2, 1, y, n, out, st,
                                                 None), {"off": 4, "y": size, "st": 4})


def test_gated_block_and_units(lib):
    i = 40
    _check(lambda off, x, w, a, st: lib.k3moe_group_glu(off, E, R, D, i, x, D, w, D, 2 * i * D, 1, 0, 4.0, 25.0, a, i, st, None),
           {"off": 4, "x": 2, "w": 2, "a": 2, "st": 4})
    _check(lambda off, da, x, w, dgu, st: lib.k3moe_group_glu_grad(off, E, R, D, i, da, i, x, D, w, D, 2 * i * D, 1, 0, 4.0, 25.0, dgu, 2 * i,
                                                                   st, None), {"off": 4, "da": 2, "x": 2, "w": 2, "dgu": 2, "st": 4})
    _check(lambda gu, a: lib.k3moe_glu_dropout(gu, 2 * D, R, D, 1, 0, 4.0, 25.0, 0.1, 1, 2, a, D, None), {"gu": 2, "a": 2})
    _check(lambda da, gu, dgu: lib.k3moe_glu_dropout_grad(da, D, gu, 2 * D, R, D, 1, 0, 4.0, 25.0, 0.1, 1, 2, dgu, 2 * D, None),
           {"da": 2, "gu": 2, "dgu": 2})
    for dt, size in ((0, 4), (1, 2)):
        _check(lambda x, r, out: lib.k3moe_dropout(x, r, 1000, dt, 0.1, 1, 2, out, None), {"x": size, "r": size, "out": size})


def test_quantising(lib):
    a, b, c = (C.c_void_p(1 << i) for i in (50, 51, 52))
    _check(lambda x: lib.k3moe_quant8_rows(x, D, R, D, 1, 0, a, D, b, 4, None), {"x": 2})
    _check(lambda w: lib.k3moe_quant8_weights(w, D, D * 64, E, 64, D, 1, 0, a, D, D * 64, b, 64, 64 * D, c, None), {"w": 2})


@pytest.mark.parametrize("dt,size", [(0, 4), (1, 2)])
@pytest.mark.parametrize("kind", [1, 2])
def test_norms(lib, kind, dt, size):
    ws = lib.k3moe_norm_grad_workspace_bytes(R, D)
    g = 4 if kind == 1 else size
    work = C.c_void_p(1 << 50)
    for gdt, gs in ((0, 4), (dt, size)):
        _check(lambda x, gain, out: lib.k3moe_rms_norm(x, D, gain, gdt, 1e-6, R, D, dt, out, D, None), {"x": size, "gain": gs, "out": size})
        _check(lambda dy, x, gain, add, dx, dgain: lib.k3moe_rms_norm_grad(dy, D, x, D, gain, gdt, add, D, 1e-6, R, D, dt, dx, D, dgain, work, ws,
                                                                          None),
               {"dy": size, "x": size, "gain": gs, "add": size, "dx": size, "dgain": 4})
        _check(lambda y, res, gain, nxt, gate, h, n: lib.k3moe_norm_residual(y, D, res, D, gain, nxt, gdt, gate, D, kind, 1.0, 1e-6, R, D, dt, h,
                                                                            D, n, D, None),
               {"y": size, "res": size, "gain": gs, "nxt": gs, "gate": g, "h": size, "n": size})
        _check(lambda dh, dn, y, h, gain, nxt, gate, dy, dres, dgate, dgain, dnxt: lib.k3moe_norm_residual_grad(
                   dh, D, dn, D, y, D, h, D, gain, nxt, gdt, gate, D, kind, 1.0, 1e-6, R, D, dt, dy, D, dres, D, dgate, D, dgain, dnxt, work, ws,
                   None),
               {"dh": size, "dn": size, "y": size, "h": size, "gain": gs, "nxt": gs, "gate": g, "dy": size, "dres": size, "dgate": g,
                "dgain": 4, "dnxt": 4})
