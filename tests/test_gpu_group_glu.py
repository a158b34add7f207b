"""The gated block in one pass on the GPU against oracle/experts.py.

The projections are fp32 sums of K products, off by at most (K + 2) 2^-23 sum |w x| (see test_gpu_experts.py).  The unit and
its derivatives are smooth, so what that moves them by is read off the definition at the four corners of the projections'
error box, a quarter more for what lies between, and its square for the curvature; the unit's own functions are good to a few
2^-22 of each factor, 2^-19 together."""
import numpy as np
import pytest

from oracle import experts as ox

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from latent_moe_layer_gb300 import experts as ex  # noqa: E402
from latent_moe_layer_gb300.k3moe import ERR_CODE, K3Error  # noqa: E402
from test_gpu_experts import BF, F16, TYPES, _close, _gen, _np, _rand  # noqa: E402

ACTS = pytest.mark.parametrize("act", ["silu", "situ"])


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert ex.status() == 0


def _inputs(sizes, K, I, dt, before=0, after=0, scale=1.0):
    gen = _gen(len(sizes) + K + I)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32) + before
    R = int(off[-1]) + after
    return (torch.from_numpy(off).cuda(), off, _rand(gen, R, K, dt=dt), _rand(gen, len(sizes), 2 * I, K, dt=dt, scale=scale * K ** -0.5),
            _rand(gen, R, I, dt=dt))


def _slack(f, gu, err, weight):
    """Bound of f's error over gu +- err; f returns arrays of gu's rows."""
    mid, I = f(gu), gu.shape[1] // 2
    worst = np.zeros_like(mid)
    for sg in (-1, 1):
        for su in (-1, 1):
            e = np.concatenate([sg * err[:, :I], su * err[:, I:]], 1)
            worst = np.maximum(worst, np.abs(f(gu + e) - mid))
    square = np.square(err[:, :I] + err[:, I:])
    curve = np.concatenate([square] * (mid.shape[1] // I), 1)
    return 1.25 * worst + np.concatenate([weight] * (mid.shape[1] // I), 1) * curve + 2.0 ** -19 * np.abs(mid)


def _check(off_d, off, x, w, da, act, **betas):
    a, b = int(off[0]), int(off[-1])
    names = {"situ_beta": "beta", "situ_linear_beta": "linear_beta"}
    more = {names[k]: v for k, v in betas.items()}
    xn, wn, dn = _np(x[:b]), _np(w), _np(da[:b])
    xn[:a] = dn[:a] = 0
    gu = ox.group_mm(xn, wn, off)
    err = (x.shape[1] + 2) * 2.0 ** -23 * ox.group_mm(np.abs(xn), np.abs(wn), off)
    fwd = lambda v: ox.glu_dropout(v, 0.0, 0, 0, act, **more)  # noqa: E731
    back = lambda v: ox.glu_dropout_grad(dn, v, 0.0, 0, 0, act, **more)  # noqa: E731
    got = ex.group_glu(x, w, off_d, act=act, **betas)
    _close(got[a:b], fwd(gu)[a:b], _slack(fwd, gu, err, np.ones_like(dn))[a:b], "a")
    dgu = ex.group_glu_grad(da, x, w, off_d, act=act, **betas)
    _close(dgu[a:b], back(gu)[a:b], _slack(back, gu, err, np.abs(dn))[a:b], "dgu")
    return got, dgu


GROUPS = [([1], 8, 8), ([0], 64, 64), ([0, 0, 5], 64, 128), ([2] * 16, 128, 96), ([3, 0, 17, 1, 0, 64], 96, 136),
          ([16, 15, 33, 129], 520, 200), ([255, 256, 257], 192, 72), ([300, 0, 511, 513, 31], 328, 320), ([1000, 7], 1096, 40),
          ([40] * 7 + [0] * 3 + [90] * 6, 256, 256), ([5] * 200, 72, 48), ([1, 0] * 64, 1024, 128), ([9], 4096, 64), ([700], 2048, 128),
          ([100, 30], 160, 50), ([64, 3], 256, 33), ([20], 72, 1)]


@TYPES
@ACTS
@pytest.mark.parametrize("sizes,K,I", GROUPS, ids=[f"E{len(s)}R{sum(s)}K{k}I{i}" for s, k, i in GROUPS])
def test_block(sizes, K, I, act, dt):
    _check(*_inputs(sizes, K, I, dt), act)


@TYPES
@ACTS
@pytest.mark.parametrize("sizes,K,I", [([3, 9], 7, 5), ([20, 0, 70], 33, 50), ([65], 129, 67)])
def test_odd_widths_off_16_byte_boundaries(sizes, K, I, act, dt):
    _check(*_inputs(sizes, K, I, dt), act)


@ACTS
@pytest.mark.parametrize("sizes,K,I", [([40], 8200, 40), ([300, 1], 16400, 24)])
def test_long_contractions(sizes, K, I, act):
    _check(*_inputs(sizes, K, I, BF), act)


@ACTS
def test_wide_gates(act):
    # gates far past the soft limits and the sigmoid's range: both ways of computing the soft-limited unit, saturated and not
    for scale in (4.0, 30.0):
        _check(*_inputs([50, 90, 3], 128, 80, BF, scale=scale), act)
    _check(*_inputs([50, 90, 3], 128, 80, F16, scale=6.0), act, **({"situ_beta": 1.5, "situ_linear_beta": 7.0} if act == "situ" else {}))


@TYPES
def test_rows_of_no_expert_are_neither_read_nor_written(dt):
    off_d, off, x, w, da = _inputs([70, 0, 9, 131], 192, 136, dt, before=5, after=40)
    a, b = int(off[0]), int(off[-1])
    for t in (x, da):
        t[:a], t[b:] = float("nan"), float("inf")
    y = torch.full((x.shape[0], 136), 3.0, dtype=dt, device="cuda")
    d = torch.full((x.shape[0], 272), 3.0, dtype=dt, device="cuda")
    ex.group_glu(x, w, off_d, out=y)
    ex.group_glu_grad(da, x, w, off_d, out=d)
    for t in (y, d):
        assert (t[:a] == 3).all() and (t[b:] == 3).all() and torch.isfinite(t).all()
    got = _check(off_d, off, x, w, da, "silu")
    assert torch.equal(got[0][a:b], y[a:b]) and torch.equal(got[1][a:b], d[a:b])


@pytest.mark.parametrize("act", ["silu", "situ"])
def test_nan_stays_in_its_row_and_column(act):
    off_d, off, x, w, da = _inputs([33, 50, 7], 128, 96, BF)
    x[40] = float("nan")
    w[2, 5] = float("nan")                                   # a gate row of expert 2: column 5 of its 7 rows
    da[3, 9] = float("nan")
    y, d = ex.group_glu(x, w, off_d, act=act), ex.group_glu_grad(da, x, w, off_d, act=act)
    bad = torch.zeros(90, 96, dtype=torch.bool, device="cuda")
    bad[40], bad[83:, 5] = True, True
    assert torch.equal(torch.isnan(y), bad)
    bad[3, 9] = True
    assert torch.equal(torch.isnan(d), torch.cat([bad, bad], 1))


@TYPES
def test_strides(dt):
    sizes, K, I = [37, 0, 200, 5], 136, 104
    off_d, off, x, w, da = _inputs(sizes, K, I, dt)
    want = _check(off_d, off, x, w, da, "silu")
    R = x.shape[0]
    for pad in (8, 3):                                       # rows on 16-byte boundaries, and off them
        wide = lambda t: torch.zeros(*t.shape[:-1], t.shape[-1] + pad, dtype=dt, device="cuda")  # noqa: E731
        xs, ws, ds, y, d = wide(x), wide(w), wide(da), torch.zeros(R, I + pad, dtype=dt, device="cuda"), torch.zeros(R, 2 * I + pad, dtype=dt, device="cuda")
        xs[:, :K], ws[..., :K], ds[:, :I] = x, w, da
        # outputs and da strided as well where x and w stay whole, and all of them
        for a, b in ((x, w), (xs[:, :K], ws[..., :K])):
            ex.group_glu(a, b, off_d, out=y[:, :I])
            ex.group_glu_grad(ds[:, :I], a, b, off_d, out=d[:, :2 * I])
            if b is w or pad == 8:
                assert torch.equal(y[:, :I], want[0]) and torch.equal(d[:, :2 * I], want[1])
            assert not y[:, I:].any() and not d[:, 2 * I:].any()
        _check(off_d, off, xs[:, :K], ws[..., :K], ds[:, :I], "situ")


def test_same_as_the_product_and_the_unit():
    # within the rounding that the two calls put between
    off_d, off, x, w, da = _inputs([300, 0, 41], 512, 256, F16)
    gu = ex.group_mm(x, w, off_d)
    a, d = ex.glu_dropout(gu), ex.glu_dropout_grad(da, gu)
    for got, want in ((ex.group_glu(x, w, off_d), a), (ex.group_glu_grad(da, x, w, off_d), d)):
        # each projection is off by 2^-11 of itself at most, the results by a few of those of their norm
        assert torch.linalg.norm(got.double() - want.double()) <= 2.0 ** -9 * torch.linalg.norm(want.double())


def test_one_weight_for_all_groups_and_bit_for_bit():
    off_d, off, x, w, da = _inputs([9, 300, 2], 264, 160, BF)
    one = w[:1].expand(3, -1, -1)
    y, d = ex.group_glu(x, one, off_d), ex.group_glu_grad(da, x, one, off_d)
    assert torch.equal(y, ex.group_glu(x, one.contiguous(), off_d)) and torch.equal(d, ex.group_glu_grad(da, x, one.contiguous(), off_d))
    for _ in range(3):
        assert torch.equal(ex.group_glu(x, one, off_d), y) and torch.equal(ex.group_glu_grad(da, x, one, off_d), d)


def test_many_experts():
    rng = np.random.default_rng(0)
    _check(*_inputs((rng.integers(0, 4, 1024) * (rng.random(1024) < 0.5)).tolist(), 64, 40, BF), "silu")


def test_offsets_out_of_range_are_reported_and_nothing_is_written():
    _, _, x, w, da = _inputs([40, 24], 64, 64, BF)
    for bad in ([0, 50, 40], [0, 40, 65], [-1, 40, 64]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        y, d = torch.full((64, 64), 3.0, dtype=BF, device="cuda"), torch.full((64, 128), 3.0, dtype=BF, device="cuda")
        for call, t in ((lambda: ex.group_glu(x, w, off, out=y), y), (lambda: ex.group_glu_grad(da, x, w, off, out=d), d)):
            call()
            assert ex.status() == ERR_CODE["RANGE"] and (t == 3).all()


def test_another_stream_and_a_graph():
    off_d, off, x, w, da = _inputs([30, 0, 99], 256, 256, BF)
    want = ex.group_glu(x, w, off_d), ex.group_glu_grad(da, x, w, off_d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ex.group_glu(x, w, off_d, stream=s), ex.group_glu_grad(da, x, w, off_d, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a = ex.group_glu(x, w, off_d)
        d = ex.group_glu_grad(a, x, w, off_d)
    x.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, ex.group_glu(x, w, off_d)) and torch.equal(d, ex.group_glu_grad(a, x, w, off_d)) and not torch.equal(a, want[0])


def test_element_offsets_past_31_bits():
    rows, K = 700_000, 3584
    x = torch.zeros(rows, K, dtype=BF, device="cuda")
    gen = _gen(9)
    x[-50:] = _rand(gen, 50, K)
    w = _rand(gen, 2, 2 * 40, K, scale=K ** -0.5)
    off = torch.tensor([rows - 50, rows - 31, rows], dtype=torch.int32, device="cuda")
    y = ex.group_glu(x, w, off)
    da = torch.ones(rows, 40, dtype=BF, device="cuda")
    dgu = ex.group_glu_grad(da, x, w, off)
    # the last rows as a call of their own: other tiles and parts of the contraction, the same error bounds
    near = np.array([0, 19, 50], dtype=np.int32)
    xn, wn, dn = _np(x[-50:]), _np(w), _np(da[-50:])
    gu, err = ox.group_mm(xn, wn, near), (K + 2) * 2.0 ** -23 * ox.group_mm(np.abs(xn), np.abs(wn), near)
    fwd = lambda v: ox.glu_dropout(v, 0.0, 0, 0)  # noqa: E731
    back = lambda v: ox.glu_dropout_grad(dn, v, 0.0, 0, 0)  # noqa: E731
    _close(y[-50:], fwd(gu), _slack(fwd, gu, err, np.ones_like(dn)), "a")
    _close(dgu[-50:], back(gu), _slack(back, gu, err, np.abs(dn)), "dgu")
    del x, y, da, dgu
    torch.cuda.empty_cache()


def test_refusals_of_the_binding():
    off_d, off, x, w, da = _inputs([30, 2], 64, 64, BF)
    for call in (lambda: ex.group_glu(x[:, :32], w, off_d), lambda: ex.group_glu(x.half(), w, off_d), lambda: ex.group_glu(x, w[:, :127], off_d),
                 lambda: ex.group_glu(x, w, off_d[:2]), lambda: ex.group_glu(x, w, off_d, act="gelu"), lambda: ex.group_glu(x, w, off_d, out=x[:, :63]),
                 lambda: ex.group_glu_grad(da[:, :63], x, w, off_d), lambda: ex.group_glu_grad(da.half(), x, w, off_d),
                 lambda: ex.group_glu_grad(da[:5], x, w, off_d), lambda: ex.group_glu(x, w, off_d, act="situ", situ_beta=float("nan"))):
        with pytest.raises(K3Error) as err:
            call()
        assert err.value.code == ERR_CODE["ARG"]
    with pytest.raises(K3Error) as err:
        ex.group_glu(x.float(), w.float(), off_d)
    assert err.value.code == ERR_CODE["UNSUPPORTED"]
