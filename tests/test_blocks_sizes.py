"""Products grouped by expert refuse sizes whose tiles, blocks or stages would leave 32 bits, each dimension by itself, and so do
the calls that make their operands.  Addresses only: a refused call touches nothing."""
import ctypes as C

import pytest

from latent_moe_layer_gb300.k3moe import ERR_CODE

MAX = 2 ** 31 - 1
ST = C.c_void_p(1 << 50)
P = [C.c_void_p((i + 1) << 52) for i in range(6)]                # far apart: no span reaches the next


@pytest.fixture(scope="module")
def lib():
    from latent_moe_layer_gb300 import build, k3moe
    build.build()
    return k3moe.lib()


# the last size whose round-up to 256 rows would leave 32 bits, and the largest
SIZES = pytest.mark.parametrize("size", [MAX - 255, MAX - 126, MAX - 62, MAX])


@SIZES
@pytest.mark.parametrize("which", ["rows", "n_in", "n_out"])
def test_products(lib, which, size):
    rows, n_in, n_out = (size if which == k else 8 for k in ("rows", "n_in", "n_out"))
    up = lambda n: -(-n // 16) * 16  # noqa: E731
    a, b, y = P[:3]
    assert lib.k3moe_group_mm(ST, 1, rows, n_in, n_out, a, up(n_in), b, up(n_in), 0, 1, y, up(n_out), 1, ST, None) == ERR_CODE["SHAPE"]
    assert lib.k3moe_group_mm_grad_x(ST, 1, rows, n_in, n_out, a, up(n_out), b, up(n_in), 0, 1, y, up(n_in), 1, ST, None) == ERR_CODE["SHAPE"]
    assert lib.k3moe_group_mm_grad_w(ST, 1, rows, n_in, n_out, a, up(n_out), b, up(n_in), 1, y, up(n_in), 0, 0, 0, ST, None) == ERR_CODE["SHAPE"]
    xs, ws = P[3:5]
    assert lib.k3moe_group_mm8(ST, 1, rows, n_in, n_out, a, up(n_in), 0, xs, up(n_in // 128 + 1), b, up(n_in), 0, 0, ws, 0,
                               n_in // 128 + 1, 1, y, up(n_out), 1, ST, None) == ERR_CODE["SHAPE"]


@SIZES
@pytest.mark.parametrize("which", ["rows", "n_in"])
def test_gated_block(lib, which, size):
    rows, n_in = (size if which == k else 8 for k in ("rows", "n_in"))
    ld, width = -(-n_in // 16) * 16, 8
    x, w, a, da = P[:4]
    assert lib.k3moe_group_glu(ST, 1, rows, n_in, width, x, ld, w, ld, 0, 1, 0, 4.0, 25.0, a, width, ST, None) == ERR_CODE["SHAPE"]
    assert lib.k3moe_group_glu_grad(ST, 1, rows, n_in, width, da, width, x, ld, w, ld, 0, 1, 0, 4.0, 25.0, a, 2 * width, ST,
                                    None) == ERR_CODE["SHAPE"]


@SIZES
def test_quantising(lib, size):
    ld = -(-size // 16) * 16
    x, codes, scales, turned = P[:4]
    assert lib.k3moe_quant8_rows(x, ld, 8, size, 1, 0, codes, ld, scales, ld // 128 + 1, None) == ERR_CODE["SHAPE"]
    for n_out, n_in in ((8, size), (size, 8)):
        assert lib.k3moe_quant8_weights(x, n_in, 0, 1, n_out, n_in, 1, 0, codes, n_in, 0, turned, n_out, 0, scales, None) == ERR_CODE["SHAPE"]
