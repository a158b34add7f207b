"""The gated unit where its parts saturate or get small: results must keep their relative precision (a few
2^-22 of each factor), since 16-bit outputs show it at any size.

The argument x of tanh carries two roundings (2^-23 of it), which its derivative 1 - tanh^2 magnifies 2 |x|
times; factors add a few 2^-22: together below 2^-20 (1 + |x|), on top of half a unit in the last place."""
import numpy as np
import pytest

from oracle import experts as ox

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from latent_moe_layer_gb300 import experts as ex  # noqa: E402

BF, F16 = torch.bfloat16, torch.float16
TYPES = pytest.mark.parametrize("dt", [BF, F16], ids=["bf16", "f16"])
SEED, OFFSET = 0x123456789ABCDEF, (1 << 32) + 3


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def _np(t):
    return t.double().cpu().numpy()


def _close(got, want, relative, what):
    """Within half a unit in the last place of got's type, subnormals' included, `relative` of want, and fp32's own
    subnormals' rounding."""
    g, (bits, low) = _np(got), {BF: (8, -126), F16: (11, -14)}[got.dtype]
    unit = np.exp2(np.maximum(np.floor(np.log2(np.abs(want) * (1 + relative) + 1e-300)), low) - bits)
    bad = ~(np.abs(g - want) <= unit + relative * np.abs(want) + 2.0 ** -148)
    assert not bad.any(), (what, int(bad.sum()), bad.size, g[bad][:4], want[bad][:4])


def _signs(rng, shape):
    return rng.choice([-1.0, 1.0], shape)


@TYPES
@pytest.mark.parametrize("width", [64, 33])
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_situ_gradient_past_its_limits(width, p, dt):
    # gates of 16 to 40 (4 to 10 times their limit), up values of 3 to 8 times theirs
    rng = np.random.default_rng(width)
    rows = 96
    g = rng.uniform(16, 40, (rows, width)) * _signs(rng, (rows, width))
    u = 25.0 * rng.uniform(3, 8, (rows, width)) * _signs(rng, (rows, width))
    g[::3] = rng.standard_normal((rows // 3, width))              # one side at a time
    u[1::3] = rng.standard_normal((rows // 3, width))
    gu = torch.from_numpy(np.concatenate([g, u], 1)).cuda().to(dt)
    da = torch.from_numpy(rng.uniform(1, 2, (rows, width)) * 2.0 ** (8 if dt == F16 else 0)).cuda().to(dt)
    n, d = _np(gu), _np(da)
    kw = dict(p=p, seed=SEED, offset=OFFSET, act="situ")
    want = ox.glu_dropout_grad(d, n, p, SEED, OFFSET, "situ")
    x = np.concatenate([np.abs(n[:, :width]) / 4, np.abs(n[:, width:]) / 25], 1)
    # near its zero at g = -1.3 the gate's gradient cancels as its definition does: left to the other tests
    clear = np.concatenate([np.abs(n[:, :width] + 1.3) > 1, np.ones((rows, width), bool)], 1)
    got = ex.glu_dropout_grad(da, gu, **kw)
    _close(got[torch.from_numpy(clear).cuda()], want[clear], (2.0 ** -20 * (1 + x))[clear], "dgu")
    _close(ex.glu_dropout(gu, **kw), ox.glu_dropout(n, p, SEED, OFFSET, "situ"), 2.0 ** -20, "a")


def test_situ_of_infinite_inputs_has_its_limits():
    inf = float("inf")
    gu = torch.tensor([[inf, -inf, inf, 1.0, 1.0, 0.0, 1.0, -1.0, 2.0, 2.0, inf, inf, -inf, 1.0, inf, inf]], dtype=BF, device="cuda")
    s = 1 / (1 + np.exp(-1.0))
    f, h = 4 * np.tanh(0.25), 25 * np.tanh(0.08)
    want = np.array([[4 * h, 0, 4 * 25, s * f * 25, -s * f * 25, 0, s * f * 25, 0]])
    want[0, 7] = -(1 - s) * -f * -25                              # g = -1: sigmoid(-1) (-f) 25
    _close(ex.glu_dropout(gu, act="situ"), want, 2.0 ** -20, "a")
    da = torch.ones(1, 8, dtype=BF, device="cuda")
    got = _np(ex.glu_dropout_grad(da, gu, act="situ"))[0]
    assert np.isfinite(got).all() and got[0] == 0 and got[1] == 0 and got[2] == 0          # saturated gates
    assert (got[8 + 2:8 + 5] == 0).all()                                                    # saturated up values


@pytest.mark.parametrize("width", [64, 33])
def test_silu_keeps_gates_whose_sigmoid_is_subnormal(width):
    # e^-87.34 is fp32's smallest normal number; g e^g stays one of bf16's down to -91.8, and longer beside a large u.
    # The hardware's exponential rounds its argument, |g| log2 e: |g| 2^-23 beside the few 2^-22 of the factors.
    rng = np.random.default_rng(width)
    rows = 96
    g = rng.uniform(-94, -80, (rows, width))
    u = _signs(rng, (rows, width)) * np.exp2(rng.uniform(10, 110, (rows, width)))
    g[::4, ::3] = rng.standard_normal((rows // 4, (width + 2) // 3))           # ordinary gates beside them
    gu = torch.from_numpy(np.concatenate([g, u], 1)).cuda().to(BF)
    da = torch.from_numpy(rng.uniform(1, 2, (rows, width)) * 2.0 ** 14).cuda().to(BF)
    n, d = _np(gu), _np(da)
    slack = 2.0 ** -20 + np.abs(n[:, :width]) * 2.0 ** -23
    for p in (0.0, 0.5):
        kw = dict(p=p, seed=SEED, offset=OFFSET)
        _close(ex.glu_dropout(gu, **kw), ox.glu_dropout(n, p, SEED, OFFSET), slack, "a")
        # near its zero at g = -1.28 the gate's gradient cancels as its definition does
        clear = np.concatenate([np.abs(n[:, :width] + 1.28) > 1, np.ones((rows, width), bool)], 1)
        got, want = ex.glu_dropout_grad(da, gu, **kw), ox.glu_dropout_grad(d, n, p, SEED, OFFSET)
        _close(got[torch.from_numpy(clear).cuda()], want[clear], np.concatenate([slack, slack], 1)[clear], "dgu")


def test_silu_keeps_the_smallest_and_the_largest_results():
    # results around bf16's smallest normal numbers and near its largest: 14 bits are left at 2^-126
    g = torch.tensor([3.0, 1.0, -2.0, 5.0, 40.0, 1e30, 1e38, 2.0 ** 100], dtype=BF, device="cuda")
    u = torch.tensor([2.0 ** -125, 2.0 ** -122, 2.0 ** -120, 2.0 ** -118, 2.0 ** -128, 1e8, 2.0, 2.0 ** 27], dtype=BF, device="cuda")
    gu = torch.cat([g, u])[None].repeat(3, 1)
    n = _np(gu)
    _close(ex.glu_dropout(gu), ox.glu_dropout(n, 0, 0, 0), 2.0 ** -13, "a")
    da = torch.full((3, 8), 0.5, dtype=BF, device="cuda")
    got, want = ex.glu_dropout_grad(da, gu), ox.glu_dropout_grad(_np(da), n, 0, 0, 0)
    _close(got, want, 2.0 ** -13, "dgu")
