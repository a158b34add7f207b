"""Every output of the 8-bit operands, the gated block and the norms that would be written over one of the call's own
inputs or other outputs is refused, tables, scales, gains and workspace among them.  Addresses only: a refused call touches
nothing."""
import ctypes as C

import pytest

from test_experts_alias import _check

R, D, E, I = 32, 256, 4, 40
ST = C.c_void_p(1 << 50)


@pytest.fixture(scope="module")
def lib():
    from latent_moe_layer_gb300 import build, k3moe
    build.build()
    return k3moe.lib()


def test_quantising(lib):
    _check(lambda x, codes, scales: lib.k3moe_quant8_rows(x, D, R, D, 1, 0, codes, D, scales, 4, None),
           {"codes": R * D, "scales": (R - 1) * 4 + 2}, {"x": 2 * R * D})
    _check(lambda w, codes, turned, scales: lib.k3moe_quant8_weights(w, D, D * 64, E, 64, D, 1, 0, codes, D, D * 64, turned, 64, 64 * D,
                                                                    scales, None),
           {"codes": E * D * 64, "turned": E * D * 64, "scales": E * 2}, {"w": 2 * E * D * 64})


def test_products(lib):
    n = 96
    _check(lambda offsets, x, xs, w, ws, y: lib.k3moe_group_mm8(offsets, E, R, D, n, x, D, 0, xs, 16, w, D, D * n, 0, ws, 2, 2, 1, y, n, 1,
                                                                ST, None),
           {"y": 2 * R * n}, {"offsets": 4 * (E + 1), "x": R * D, "xs": (R - 1) * 16 + 2 + 2, "w": E * n * D, "ws": E * 2})
    _check(lambda offsets, x, w, a: lib.k3moe_group_glu(offsets, E, R, D, I, x, D, w, D, 2 * I * D, 1, 0, 4.0, 25.0, a, I, ST, None),
           {"a": 2 * R * I}, {"offsets": 4 * (E + 1), "x": 2 * R * D, "w": 4 * E * I * D})
    _check(lambda offsets, da, x, w, dgu: lib.k3moe_group_glu_grad(offsets, E, R, D, I, da, I, x, D, w, D, 2 * I * D, 1, 0, 4.0, 25.0, dgu,
                                                                   2 * I, ST, None),
           {"dgu": 4 * R * I}, {"offsets": 4 * (E + 1), "da": 2 * R * I, "x": 2 * R * D, "w": 4 * E * I * D})


@pytest.mark.parametrize("by_row", [False, True])
def test_norms(lib, by_row):
    m, v, ws = 2 * R * D, 4 * D, lib.k3moe_norm_grad_workspace_bytes(R, D)
    kind, gate = (1, 4 * R) if by_row else (2, m)
    _check(lambda x, gain, out: lib.k3moe_rms_norm(x, D, gain, 0, 1e-6, R, D, 1, out, D, None), {"out": m}, {"x": m, "gain": v},
           allowed=[("out", "x")])
    _check(lambda dy, x, gain, add, dx, dgain, work: lib.k3moe_rms_norm_grad(dy, D, x, D, gain, 0, add, D, 1e-6, R, D, 1, dx, D, dgain, work,
                                                                            ws, None),
           {"dx": m, "dgain": v, "work": ws}, {"dy": m, "x": m, "gain": v, "add": m}, allowed=[("dx", n) for n in ("dy", "x", "add")])
    same = ["y", "res"] + ([] if by_row else ["gate"])
    _check(lambda y, res, gain, nxt, gate, h, n: lib.k3moe_norm_residual(y, D, res, D, gain, nxt, 0, gate, D, kind, 1.0, 1e-6, R, D, 1, h, D,
                                                                        n, D, None),
           {"h": m, "n": m}, {"y": m, "res": m, "gain": v, "nxt": v, "gate": gate}, allowed=[(o, n) for o in ("h", "n") for n in same])
    same = ["dh", "dn", "y", "h"] + ([] if by_row else ["gate"])
    outs = ["dy", "dres"] + ([] if by_row else ["dgate"])
    _check(lambda dh, dn, y, h, gain, nxt, gate, dy, dres, dgate, dgain, dnxt, work: lib.k3moe_norm_residual_grad(
               dh, D, dn, D, y, D, h, D, gain, nxt, 0, gate, D, kind, 1.0, 1e-6, R, D, 1, dy, D, dres, D, dgate, D, dgain, dnxt, work, ws, None),
           {"dy": m, "dres": m, "dgate": gate, "dgain": v, "dnxt": v, "work": ws},
           {"dh": m, "dn": m, "y": m, "h": m, "gain": v, "nxt": v, "gate": gate}, allowed=[(o, n) for o in outs for n in same])
