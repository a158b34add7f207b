"""The gated block's results for a row and a column do not depend on what is not theirs, to the last bit: rows of other experts
and of none, and weight rows that a tile holds beside the last column's."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from latent_moe_layer_gb300 import experts as ex  # noqa: E402
from test_gpu_experts import BF, TYPES, _gen, _rand  # noqa: E402

ACTS = pytest.mark.parametrize("act", ["silu", "situ"])


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert ex.status() == 0


def _both(x, w, da, off, act):
    return ex.group_glu(x, w, off, act=act), ex.group_glu_grad(da, x, w, off, act=act)


@TYPES
@ACTS
@pytest.mark.parametrize("K,I", [(192, 136), (128, 96), (64, 40), (1024, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 1000.0])
def test_rows_of_no_expert(K, I, bad, act, dt):
    gen = _gen(K + I)
    sizes, before, after = [70, 0, 9, 131, 3], 5, 40
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32) + before
    R = int(off[-1]) + after
    x, w, da = _rand(gen, R, K, dt=dt), _rand(gen, len(sizes), 2 * I, K, dt=dt, scale=K ** -0.5), _rand(gen, R, I, dt=dt)
    off_d = torch.from_numpy(off).cuda()
    a, b = int(off[0]), int(off[-1])
    for t in (x, da):
        t[:a], t[b:] = 0, 0
    want = _both(x, w, da, off_d, act)
    for t in (x, da):
        t[:a], t[b:] = bad, bad
    for got, ref in zip(_both(x, w, da, off_d, act), want):
        assert torch.equal(got[a:b], ref[a:b])


@TYPES
@ACTS
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 1000.0])
def test_rows_of_other_experts(bad, act, dt):
    # experts 0 and 2 lie around expert 1's rows, in tiles that reach past them
    gen = _gen(7)
    K, I, sizes = 256, 48, [37, 21, 50]
    off_d = torch.tensor([0, 37, 58, 108], dtype=torch.int32, device="cuda")
    x, w, da = _rand(gen, 108, K, dt=dt), _rand(gen, 3, 2 * I, K, dt=dt, scale=K ** -0.5), _rand(gen, 108, I, dt=dt)
    want = _both(x, w, da, off_d, act)
    for t in (x, da):
        t[:37], t[58:] = bad, bad
    for got, ref in zip(_both(x, w, da, off_d, act), want):
        assert torch.equal(got[37:58], ref[37:58])


@TYPES
@ACTS
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 1000.0])
@pytest.mark.parametrize("I", [40, 72, 24])
def test_weight_rows_beside_the_last_column(I, bad, act, dt):
    # a width that is not whole blocks of 16: the last tile's gate rows run on into the up rows
    gen = _gen(I)
    K, sizes = 128, [33, 70]
    off_d = torch.tensor([0, 33, 103], dtype=torch.int32, device="cuda")
    x, w, da = _rand(gen, 103, K, dt=dt), _rand(gen, 2, 2 * I, K, dt=dt, scale=K ** -0.5), _rand(gen, 103, I, dt=dt)
    want = _both(x, w, da, off_d, act)
    w[:, I:I + 8] = bad                                      # up rows of the first eight columns
    got = _both(x, w, da, off_d, act)
    last = slice(I // 16 * 16, I)
    assert torch.equal(got[0][:, last], want[0][:, last])
    for half in (0, I):
        at = slice(last.start + half, last.stop + half)
        assert torch.equal(got[1][:, at], want[1][:, at])
