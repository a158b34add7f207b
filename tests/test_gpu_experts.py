"""GPU parity of the expert training operators (latent_moe_layer_gb300.experts) against their fp64
definitions (oracle/experts.py).

Tolerances, element by element.  An output rounded to nearest has at most half a unit in the last place
on top of its fp32 value: 2^-8, 2^-11 or 2^-24 (bf16, f16, fp32: 8, 11 and 24 significant bits) of the power
of two at or below |y|, and 2^-25 absolute where an f16 is subnormal.  A sum of n fp32 products in any order is off by at most n 2^-24 sum |a b| to first order;
tensor cores may truncate instead of rounding, which doubles that.  Elementwise functions (hardware
exponential, division, tanhf) are good to a few 2^-22 of each factor."""
import numpy as np
import pytest

from oracle import experts as ox

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from latent_moe_layer_gb300 import experts as ex  # noqa: E402
from latent_moe_layer_gb300.k3moe import ERR_CODE, K3Error  # noqa: E402

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
HALF = {BF: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}     # half a unit in the last place of 1.0
TYPES = pytest.mark.parametrize("dt", [BF, F16], ids=["bf16", "f16"])
SEED, OFFSET = 0xDEADBEEF12345678, (3 << 32) + 17


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert ex.status() == 0


def _rand(gen, *shape, dt=BF, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dt)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _np(t):
    return t.double().cpu().numpy()


def _close(got, want, slack, what=""):
    """|got - want| <= half a unit in the last place of got's type + slack, NaN nowhere."""
    g = _np(got)
    tiny = 2.0 ** -25 if got.dtype == F16 else 1e-38
    binade = np.exp2(np.floor(np.log2(np.abs(want) + slack + 1e-300)))
    tol = HALF[got.dtype] * binade + slack + tiny
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), g[bad][:4], want[bad][:4], np.broadcast_to(tol, bad.shape)[bad][:4])


# ------------------------------------------------------------------------------------------ rows
@pytest.mark.parametrize("T,K,E,first,total", [
    (0, 4, 8, 0, 8), (1, 1, 1, 0, 1), (1, 16, 896, 0, 896), (16, 16, 896, 0, 896), (37, 3, 5, 4, 12), (128, 16, 112, 224, 896),
    (129, 16, 1024, 0, 1024), (1000, 5, 7, 0, 7), (8192, 16, 896, 0, 896), (5001, 16, 448, 448, 896), (300000, 2, 33, 0, 64)])
def test_plan(T, K, E, first, total):
    rng = np.random.default_rng(T + K)
    idx = rng.integers(-1, total, (T, K)).astype(np.int32)
    idx[: T // 3] = idx[0] if T else 0                      # runs of one routing: heavy experts
    off, pos = ex.plan_rows(torch.from_numpy(idx).cuda(), E, first_expert=first)
    want_off, want_pos = ox.plan_rows(idx, E, first)
    assert np.array_equal(off.cpu().numpy(), want_off) and np.array_equal(pos.cpu().numpy(), want_pos)


def _routing(T, K, E, drop, seed):
    rng = np.random.default_rng(seed)
    idx = np.stack([rng.permutation(max(E, K))[:K] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, K), np.int32)
    idx[rng.random(idx.shape) < drop] = -1
    if T > 2:
        idx[1] = -1                                         # a token without any row
    return idx


@TYPES
@pytest.mark.parametrize("T,K,D,drop", [(1, 1, 8, 0.0), (16, 16, 3584, 0.0), (5, 3, 7, 0.3), (300, 9, 200, 0.5),
                                        (33, 32, 2056, 0.1), (4, 2, 5000, 0.0), (0, 4, 64, 0.0), (3, 40, 72, 0.2)])
def test_gather_combine_and_gradient(T, K, D, drop, dt):
    gen = _gen(T + K + D)
    E = 40
    off, pos = ex.plan_rows(torch.from_numpy(_routing(T, K, E, drop, T + D)).cuda(), E)
    n = int(off[-1])
    x = _rand(gen, T, D, dt=dt)
    buf = torch.full((n + 3, D), 7.0, dtype=dt, device="cuda")
    xs = ex.gather_rows(x, pos, out=buf)
    p = pos.cpu().numpy()
    want = np.full((n + 3, D), 7.0)
    want[p[p >= 0]] = np.repeat(_np(x)[:, None], K, 1)[p >= 0]
    assert np.array_equal(_np(xs), want)                    # copies; rows of no pair untouched
    y = _rand(gen, n + 3, D, dt=dt)
    y[n:] = float("nan")                                    # rows of no pair do not matter
    w = torch.rand(T, K, generator=gen, device="cuda")
    wn = w.double().cpu().numpy()
    ab = ox.combine_rows(np.abs(_np(y)), p, wn)
    _close(ex.combine_rows(y, pos, w), ox.combine_rows(_np(y), p, wn), K * 2.0 ** -23 * ab, "combine")
    _close(ex.combine_rows(y, pos), ox.combine_rows(_np(y), p), K * 2.0 ** -23 * ox.combine_rows(np.abs(_np(y)), p), "sum")
    dz = _rand(gen, T, D, dt=dt)
    want_dy, want_dw = ox.combine_rows_grad(_np(dz), _np(y), p, wn)
    _, ab_dw = ox.combine_rows_grad(np.abs(_np(dz)), np.abs(_np(y)), p, wn)
    dy, dw = ex.combine_rows_grad(dz, y, pos, w)
    _close(dy[:n], want_dy[:n], 2.0 ** -24 * np.abs(want_dy[:n]), "dy")
    _close(dw, want_dw, (D + 2) * 2.0 ** -23 * ab_dw, "dw")
    y2 = y.clone()                                          # in place
    dy2, dw2 = ex.combine_rows_grad(dz, y2, pos, w, out=y2)
    assert dy2.data_ptr() == y2.data_ptr() and torch.equal(y2[:n], dy[:n]) and torch.equal(dw2, dw)


def test_combine_weights_that_are_masked_do_not_matter():
    pos = torch.tensor([[0, -1], [-1, -1]], dtype=torch.int32, device="cuda")
    y = torch.ones(1, 8, dtype=BF, device="cuda")
    w = torch.tensor([[2.0, float("nan")], [float("inf"), float("-inf")]], device="cuda")
    assert torch.equal(ex.combine_rows(y, pos, w).float(), torch.tensor([[2.0] * 8, [0.0] * 8], device="cuda"))
    dz = torch.full((2, 8), float("inf"), dtype=BF, device="cuda")
    dz[0] = 1.0
    _, dw = ex.combine_rows_grad(dz, y, pos, w)
    assert dw.tolist() == [[8.0, 0.0], [0.0, 0.0]]


@TYPES
def test_rows_strides_and_unaligned_views(dt):
    gen = _gen(5)
    T, K, D = 21, 3, 64
    _, pos = ex.plan_rows(torch.from_numpy(_routing(T, K, 9, 0.2, 3)).cuda(), 9)
    n = T * K
    w = torch.rand(T, K, generator=gen, device="cuda")
    for pad, lead in ((8, 8), (5, 3)):                      # 16-byte rows, and rows at any element
        big = lambda r: _rand(gen, r, D + pad + lead, dt=dt)[:, lead:lead + D]  # noqa: E731
        x, y, dz = big(T), big(n), big(T)
        bx, bz, by = big(n).zero_(), big(T), big(n).zero_()
        assert torch.equal(ex.gather_rows(x, pos, out=bx), ex.gather_rows(x.contiguous(), pos, out=torch.zeros_like(bx)))
        assert torch.equal(ex.combine_rows(y, pos, w, out=bz), ex.combine_rows(y.contiguous(), pos, w))
        a = ex.combine_rows_grad(dz, y, pos, w, out=by)
        b = ex.combine_rows_grad(dz.contiguous(), y.contiguous(), pos, w, out=torch.zeros(n, D, dtype=dt, device="cuda"))
        assert torch.equal(a[0], b[0])
        # the two access widths group the dot product differently
        assert torch.allclose(a[1], b[1], rtol=0, atol=D * 2.0 ** -23 * 16 * D)


def test_row_numbers_out_of_range_are_reported():
    pos = torch.tensor([[0, 5]], dtype=torch.int32, device="cuda")
    x = torch.ones(1, 16, dtype=BF, device="cuda")
    out = torch.zeros(3, 16, dtype=BF, device="cuda")
    ex.gather_rows(x, pos, out=out)
    assert ex.status() == ERR_CODE["RANGE"] and ex.status() == 0
    assert out.float().sum() == 16
    assert torch.equal(ex.combine_rows(out, pos), x) and ex.status() == ERR_CODE["RANGE"]
    ex.combine_rows_grad(x, out, pos, torch.ones(1, 2, device="cuda"))
    assert ex.status() == ERR_CODE["RANGE"]


# ------------------------------------------------------------------------------------------ grouped products
GROUPS = [
    # sizes of the experts' groups, n_in, n_out
    ([1], 8, 8), ([0], 64, 64), ([0, 0, 5], 64, 128), ([2] * 16, 128, 192), ([3, 0, 17, 1, 0, 64], 96, 256),
    ([16, 15, 33, 129], 520, 264), ([255, 256, 257], 192, 136), ([300, 0, 511, 513, 31], 328, 640),
    ([1000, 7], 1096, 72), ([40] * 7 + [0] * 3 + [90] * 6, 256, 512), ([64, 128, 192], 64, 1024),
    ([5] * 200, 72, 88), ([1, 0] * 64, 1024, 256)]


def _group_inputs(sizes, K, N, dt, before=0, after=0, seed=0):
    gen = _gen(seed + K + N)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32) + before
    R = int(off[-1]) + after
    x, dy = _rand(gen, R, K, dt=dt), _rand(gen, R, N, dt=dt)
    w = _rand(gen, len(sizes), N, K, dt=dt, scale=K ** -0.5)
    return torch.from_numpy(off).cuda(), off, x, dy, w


def _check_group(off_d, off, x, dy, w, out_dtype=None):
    K, N, E = x.shape[1], dy.shape[1], w.shape[0]
    a, b = int(off[0]), int(off[-1])
    xn, dn, wn = _np(x[:b]), _np(dy[:b]), _np(w)
    xn[:a] = dn[:a] = 0
    y = ex.group_mm(x, w, off_d, out_dtype=out_dtype)
    _close(y[a:b], ox.group_mm(xn, wn, off)[a:b], (K + 2) * 2.0 ** -23 * ox.group_mm(np.abs(xn), np.abs(wn), off)[a:b], "y")
    dx = ex.group_mm_grad_x(dy, w, off_d, out_dtype=out_dtype)
    _close(dx[a:b], ox.group_mm_grad_x(dn, wn, off)[a:b],
           (N + 2) * 2.0 ** -23 * ox.group_mm_grad_x(np.abs(dn), np.abs(wn), off)[a:b], "dx")
    dw = ex.group_mm_grad_w(dy, x, off_d, out_dtype=x.dtype if out_dtype is None else out_dtype)
    rows = np.diff(off)[:, None, None]
    _close(dw, ox.group_mm_grad_w(dn, xn, off), (rows + 2) * 2.0 ** -23 * ox.group_mm_grad_w(np.abs(dn), np.abs(xn), off), "dw")
    return y, dx, dw


@TYPES
@pytest.mark.parametrize("sizes,K,N", GROUPS, ids=[f"E{len(s)}R{sum(s)}K{k}N{n}" for s, k, n in GROUPS])
def test_group_products(sizes, K, N, dt):
    off_d, off, x, dy, w = _group_inputs(sizes, K, N, dt)
    _check_group(off_d, off, x, dy, w)
    _check_group(off_d, off, x, dy, w, F32)


@TYPES
@pytest.mark.parametrize("sizes,long,short", [([1], 4096, 256), ([5], 2056, 72), ([0, 300], 3104, 520), ([257, 0, 3], 1000, 96),
                                              ([40] * 6, 2048, 600), ([513, 1, 1], 2048, 256), ([700], 1608, 640),
                                              ([256], 320, 256), ([16, 31], 2049 * 8, 40)])
def test_group_products_of_few_tiles_and_long_contractions(sizes, long, short, dt):
    for K, N in ((long, short), (short, long)):
        off_d, off, x, dy, w = _group_inputs(sizes, K, N, dt, before=3, after=20)
        a, b = int(off[0]), int(off[-1])
        for t in (x, dy):
            t[:a], t[b:] = float("nan"), float("inf")
        _check_group(off_d, off, x, dy, w)
        _check_group(off_d, off, x, dy, w, F32)
        y, dx = ex.group_mm(x, w, off_d), ex.group_mm_grad_x(dy, w, off_d)
        for _ in range(5):
            assert torch.equal(ex.group_mm(x, w, off_d)[a:b], y[a:b])
            assert torch.equal(ex.group_mm_grad_x(dy, w, off_d)[a:b], dx[a:b])


@TYPES
@pytest.mark.parametrize("sizes,K,N", [([3, 9], 7, 5), ([20, 0, 70], 33, 100), ([65], 129, 66)])
def test_group_products_of_odd_widths(sizes, K, N, dt):
    _check_group(*_group_inputs(sizes, K, N, dt))


@TYPES
def test_rows_of_no_expert_are_neither_read_nor_written(dt):
    sizes, K, N = [70, 0, 9, 131], 192, 264
    off_d, off, x, dy, w = _group_inputs(sizes, K, N, dt, before=5, after=40)
    a, b = int(off[0]), int(off[-1])
    for t in (x, dy):
        t[:a], t[b:] = float("nan"), float("inf")
    _check_group(off_d, off, x, dy, w)
    y = torch.full((x.shape[0], N), 3.0, dtype=dt, device="cuda")
    dx = torch.full((x.shape[0], K), 3.0, dtype=dt, device="cuda")
    ex.group_mm(x, w, off_d, out=y)
    ex.group_mm_grad_x(dy, w, off_d, out=dx)
    for t in (y, dx):
        assert (t[:a] == 3).all() and (t[b:] == 3).all() and torch.isfinite(t).all()


def test_infinities_and_nan_stay_in_their_row_and_expert():
    sizes, K, N = [33, 50, 7], 128, 256
    off_d, off, x, dy, w = _group_inputs(sizes, K, N, BF)
    x[40] = float("inf")                                    # expert 1
    dy[85] = float("nan")                                   # expert 2
    w[1, 0] = 0.0
    y, dx, dw = ex.group_mm(x, w, off_d), ex.group_mm_grad_x(dy, w, off_d), ex.group_mm_grad_w(dy, x, off_d)
    keep = torch.ones(90, dtype=torch.bool, device="cuda")
    keep[40] = False
    assert torch.isfinite(y[keep]).all() and torch.isnan(y[40, 0]) and not torch.isfinite(y[40]).any()
    keep[40], keep[85] = True, False
    assert torch.isfinite(dx[keep]).all() and torch.isnan(dx[85]).all()
    assert torch.isfinite(dw[0]).all() and not torch.isfinite(dw[1]).any() and torch.isnan(dw[2]).all()


@TYPES
def test_group_strides(dt):
    sizes, K, N = [37, 0, 200, 5], 136, 200
    off_d, off, x, dy, w = _group_inputs(sizes, K, N, dt)
    want = ex.group_mm(x, w, off_d), ex.group_mm_grad_x(dy, w, off_d), ex.group_mm_grad_w(dy, x, off_d)
    R = x.shape[0]
    for lead, pad in ((8, 16), (3, 2)):                     # 16-byte rows, and rows at any element
        view = lambda t: torch.nn.functional.pad(t, (lead, pad))[..., lead:lead + t.shape[-1]]  # noqa: E731
        xv, dv = view(x), view(dy)
        wv = view(torch.cat([w, w[:, :4]], 1))[:, :N]       # expert stride beyond n_out rows
        y = torch.zeros(R, N + lead + pad, dtype=dt, device="cuda")
        dx = torch.zeros(R, K + lead + pad, dtype=dt, device="cuda")
        dw = torch.zeros(4, N + 3, K + lead + pad, dtype=F32, device="cuda")
        ex.group_mm(xv, wv, off_d, out=y[:, lead:lead + N])
        ex.group_mm_grad_x(dv, wv, off_d, out=dx[:, lead:lead + K])
        ex.group_mm_grad_w(dv, xv, off_d, out=dw[:, :N, lead:lead + K])
        for got, t, width, ref in ((y, 0, N, want[0]), (dx, 1, K, want[1])):
            # another kernel may sum in another order: one ulp of the output, and fp32 noise
            assert torch.allclose(got[:, lead:lead + width].double(), ref.double(), rtol=2 * HALF[dt], atol=1e-3)
            assert not got[:, :lead].any() and not got[:, lead + width:].any()
        assert torch.allclose(dw[:, :N, lead:lead + K], want[2], rtol=1e-4, atol=1e-3)
        assert not dw[:, N:].any() and not dw[..., :lead].any() and not dw[..., lead + K:].any()


@TYPES
def test_group_products_of_odd_widths_in_16_byte_rows(dt):
    # the tensor-core path where a row's last piece is cut: widths 70 and 90 in rows of 80 and 96
    sizes, K, N = [37, 0, 300, 5], 70, 90
    off_d, off, x, dy, w = _group_inputs(sizes, K, N, dt)
    pad = lambda t, n: torch.nn.functional.pad(t, (0, n - t.shape[-1]), value=float("nan"))[..., :t.shape[-1]]  # noqa: E731
    x, dy, w = pad(x, 80), pad(dy, 96), pad(w, 80)
    _check_group(off_d, off, x, dy, w)
    dw = torch.full((4, N, 80), 5.0, device="cuda")
    ex.group_mm_grad_w(dy, x, off_d, out=dw[..., :K])
    assert (dw[..., K:] == 5).all()
    dn, xn, rows = _np(dy), _np(x), np.diff(off)[:, None, None]
    want, mag = ox.group_mm_grad_w(dn, xn, off), ox.group_mm_grad_w(np.abs(dn), np.abs(xn), off)
    _close(dw[..., :K], want, (rows + 2) * 2.0 ** -23 * mag)
    ex.group_mm_grad_w(dy, x, off_d, out=dw[..., :K], accumulate=True)
    assert (dw[..., K:] == 5).all()
    _close(dw[..., :K], 2 * want, 2 * (rows + 3) * 2.0 ** -23 * mag)


@TYPES
@pytest.mark.parametrize("sizes,K,N", [([9001], 72, 264), ([6000, 1, 0, 70, 64, 3900], 256, 256), ([7003, 2100], 200, 520),
                                       ([2600] * 5, 512, 1000), ([0, 12000], 8, 16)])
def test_grad_w_of_few_tiles_and_many_rows(sizes, K, N, dt):
    off_d, off, x, dy, _ = _group_inputs(sizes, K, N, dt, before=3, after=20)
    a, b = int(off[0]), int(off[-1])
    for t in (x, dy):
        t[:a], t[b:] = float("nan"), float("inf")
    xn, dn, rows = _np(x[:b]), _np(dy[:b]), np.diff(off)[:, None, None]
    want, mag = ox.group_mm_grad_w(dn, xn, off), ox.group_mm_grad_w(np.abs(dn), np.abs(xn), off)
    for o in (F32, dt):
        dw = ex.group_mm_grad_w(dy, x, off_d, out_dtype=o)
        _close(dw, want, (rows + 2) * 2.0 ** -23 * mag)
        assert all(torch.equal(ex.group_mm_grad_w(dy, x, off_d, out_dtype=o), dw) for _ in range(3))
    dw = torch.ones(len(sizes), N, K, device="cuda")
    ex.group_mm_grad_w(dy, x, off_d, out=dw, accumulate=True)
    _close(dw, 1 + want, (rows + 4) * 2.0 ** -23 * (1 + mag))


def test_grad_w_of_long_groups_keeps_fp32_precision():
    # sums of 512-row parts in fp32: a rounding (2^-24) per part and the parts' own truncation (n 2^-23 / 16 of
    # a running sum at most); against the norm of the result 2e-6 covers both at any length
    off_d, off, x, dy, w = _group_inputs([20011, 3, 0, 1025], 128, 256, BF)
    dw = ex.group_mm_grad_w(dy, x, off_d).double()
    for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
        want = dy[a:b].double().T @ x[a:b].double()
        assert torch.linalg.norm(dw[e] - want) <= 2e-6 * torch.linalg.norm(want)


def test_many_experts():
    rng = np.random.default_rng(0)
    sizes = (rng.integers(0, 4, 1024) * (rng.random(1024) < 0.5)).tolist()
    _check_group(*_group_inputs(sizes, 64, 72, BF))


def test_element_offsets_past_31_bits():
    # 700,000 rows of 3584: element offsets up to 2.5e9
    rows, D = 700_000, 3584
    y = torch.empty(rows, D, dtype=BF, device="cuda")
    gen = _gen(9)
    last = _rand(gen, 60, D)
    y[-60:] = last
    pos = torch.tensor([[rows - 1, rows - 60], [rows - 30, -1]], dtype=torch.int32, device="cuda")
    mix = torch.tensor([[0.5, 2.0], [1.0, 3.0]], device="cuda")
    assert torch.equal(ex.combine_rows(y, pos, mix),
                       torch.stack([last[59].float() * 0.5 + last[0].float() * 2, last[30].float()]).to(BF))
    x = _rand(gen, 2, D)
    dy, dmix = ex.combine_rows_grad(x, y, pos, mix, out=torch.empty_like(y))
    assert torch.equal(dy[rows - 30], x[1]) and torch.equal(dy[rows - 1], (x[0].float() * 0.5).to(BF))
    del dy
    ex.gather_rows(x, pos, out=y)
    assert torch.equal(y[-1], x[0]) and torch.equal(y[-60], x[0]) and torch.equal(y[-30], x[1])
    w = _rand(gen, 2, 64, D, scale=D ** -0.5)
    off = torch.tensor([rows - 50, rows - 31, rows], dtype=torch.int32, device="cuda")
    got = ex.group_mm(y, w, off)
    want = torch.cat([y[-50:-31].double() @ w[0].double().T, y[-31:].double() @ w[1].double().T])
    assert ((got[-50:].double() - want).abs() <= HALF[BF] * want.abs() + 1e-4).all()
    dx = ex.group_mm_grad_x(got, w, off)
    want = torch.cat([got[-50:-31].double() @ w[0].double(), got[-31:].double() @ w[1].double()])
    assert ((dx[-50:].double() - want).abs() <= HALF[BF] * want.abs() + 1e-4).all()
    dw = ex.group_mm_grad_w(got, y, off)
    want = got[-31:].double().T @ y[-31:].double()
    assert ((dw[1].double() - want).abs() <= 33 * 2.0 ** -23 * (got[-31:].double().abs().T @ y[-31:].double().abs())).all()
    del y, dx
    torch.cuda.empty_cache()


def test_one_weight_for_all_groups():
    off_d, off, x, dy, w = _group_inputs([9, 30, 2], 64, 128, BF)
    one = w[:1].expand(3, -1, -1)
    assert torch.equal(ex.group_mm(x, one, off_d), ex.group_mm(x, one.contiguous(), off_d))
    assert torch.equal(ex.group_mm_grad_x(dy, one, off_d), ex.group_mm_grad_x(dy, one.contiguous(), off_d))


@pytest.mark.parametrize("width", [264, 65])
def test_grad_w_accumulates(width):
    off_d, off, x, dy, w = _group_inputs([37, 0, 100], width, 136, BF)
    acc = torch.randn(3, 136, width, device="cuda", generator=_gen(1))
    before = acc.double()
    once = ex.group_mm_grad_w(dy, x, off_d)
    got = ex.group_mm_grad_w(dy, x, off_d, out=acc, accumulate=True)
    assert got.data_ptr() == acc.data_ptr()
    want = before + once.double()
    assert ((got.double() - want).abs() <= 2.0 ** -24 * want.abs()).all()      # one fp32 addition
    assert torch.equal(got[1].double(), before[1])                                    # an expert without rows


def test_offsets_out_of_range_are_reported_and_nothing_is_written():
    _, _, x, dy, w = _group_inputs([40, 24], 64, 128, BF)
    for bad in ([0, 50, 40], [0, 40, 65], [-1, 40, 64], [0, 2 ** 31 - 1, -2 ** 31]):
        off = torch.tensor(bad, dtype=torch.int64).to(torch.int32).cuda()
        y, dx = torch.full((64, 128), 3.0, dtype=BF, device="cuda"), torch.full((64, 64), 3.0, dtype=BF, device="cuda")
        dw = torch.full((2, 128, 64), 3.0, device="cuda")
        for call, t in ((lambda: ex.group_mm(x, w, off, out=y), y), (lambda: ex.group_mm_grad_x(dy, w, off, out=dx), dx),
                        (lambda: ex.group_mm_grad_w(dy, x, off, out=dw), dw)):
            call()
            assert ex.status() == ERR_CODE["RANGE"] and (t == 3).all()


def test_group_products_repeat_bit_for_bit():
    off_d, off, x, dy, w = _group_inputs([300, 1, 80, 0, 700], 512, 768, BF)
    runs = [(ex.group_mm(x, w, off_d), ex.group_mm_grad_x(dy, w, off_d), ex.group_mm_grad_w(dy, x, off_d)) for _ in range(3)]
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))


@pytest.mark.slow
def test_large_groups_on_the_gpu_against_fp64():
    # one of 64 ranks of the K3 layer with ragged loads; the fp64 product runs on the GPU
    sizes, K, N = [1, 700, 33, 0, 290, 256, 512, 129, 64, 3, 900, 17, 448, 31], 3584, 6144
    off_d, off, x, dy, w = _group_inputs(sizes, K, N, BF)
    y, dx, dw = ex.group_mm(x, w, off_d), ex.group_mm_grad_x(dy, w, off_d), ex.group_mm_grad_w(dy, x, off_d)
    for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
        xe, de, we = x[a:b].double(), dy[a:b].double(), w[e].double()
        for got, want, mag, n in ((y[a:b], xe @ we.T, xe.abs() @ we.abs().T, K), (dx[a:b], de @ we, de.abs() @ we.abs(), N),
                                  (dw[e], de.T @ xe, de.abs().T @ xe.abs(), b - a)):
            tol = HALF[got.dtype] * want.abs() + (n + 2) * 2.0 ** -23 * mag
            assert ((got.double() - want).abs() <= tol).all()


# ------------------------------------------------------------------------------------------ gated unit, dropout
def _glu_slack(gu, act, want):
    # exponential and division: a few 2^-22 relative; the situ branches are products of three factors;
    # the gradient's s + g s (1 - s) cancels, so its error goes with the terms' size (1 + |g|) |u|
    g, u = np.split(np.abs(gu), 2, 1)
    return (1 + g) * (1 + u) * 2.0 ** -20


@TYPES
@pytest.mark.parametrize("act", ["silu", "situ"])
@pytest.mark.parametrize("rows,width,p", [(1, 8, 0.0), (1, 1, 0.5), (7, 96, 0.1), (130, 264, 0.3), (33, 100, 0.9), (0, 64, 0.1),
                                          (515, 3584, 0.25)])
def test_glu_and_gradient(rows, width, p, act, dt):
    gen = _gen(rows + width)
    gu, da = _rand(gen, rows, 2 * width, dt=dt, scale=2.0), _rand(gen, rows, width, dt=dt)
    n = _np(gu)
    slack = _glu_slack(n, act, None) / (1 - p)
    want = ox.glu_dropout(n, p, SEED, OFFSET, act)
    a = ex.glu_dropout(gu, p=p, seed=SEED, offset=OFFSET, act=act)
    _close(a, want, slack, "a")
    dgu = ex.glu_dropout_grad(da, gu, p=p, seed=SEED, offset=OFFSET, act=act)
    mag = np.concatenate([slack, slack], 1) * np.concatenate([np.abs(_np(da))] * 2, 1)
    _close(dgu, ox.glu_dropout_grad(_np(da), n, p, SEED, OFFSET, act), mag, "dgu")
    if p > 0:
        keep = ox.keep_mask(np.arange(rows * width).reshape(rows, width), p, SEED, OFFSET)
        assert (_np(a)[~keep] == 0).all() and (_np(dgu)[np.concatenate([~keep, ~keep], 1)] == 0).all()
    gu2 = gu.clone()
    assert torch.equal(ex.glu_dropout_grad(da, gu2, p=p, seed=SEED, offset=OFFSET, act=act, out=gu2), dgu)


def test_glu_betas_strides_and_extremes():
    gen = _gen(3)
    gu = _rand(gen, 20, 2 * 40, scale=3.0)
    n = _np(gu)
    _close(ex.glu_dropout(gu, act="situ", situ_beta=2.5, situ_linear_beta=3.0), ox.glu_dropout(n, 0, 0, 0, "situ", 2.5, 3.0),
           _glu_slack(n, "situ", None))
    # views: 16-byte rows and rows at any element give the contiguous result
    da = _rand(gen, 20, 40)
    for lead, pad in ((8, 8), (1, 2)):
        v = torch.nn.functional.pad(gu, (lead, pad))[:, lead:lead + 80]
        d = torch.nn.functional.pad(da, (lead, pad))[:, lead:lead + 40]
        kw = dict(p=0.3, seed=1, offset=2)
        assert torch.equal(ex.glu_dropout(v, **kw), ex.glu_dropout(gu, **kw))
        assert torch.equal(ex.glu_dropout_grad(d, v, **kw), ex.glu_dropout_grad(da, gu, **kw))
    # large gates saturate, and a dropped element is 0 whatever it holds
    big = torch.tensor([[300.0, -300.0, 1e30, -1e30] * 2 + [2.0] * 8], dtype=BF, device="cuda")
    a = ex.glu_dropout(big)
    # values in bf16: 300 is exact, 1e30 rounded
    assert torch.equal(a, (torch.relu(big[:, :8].float()) * 2).to(BF))
    bad = torch.full((1, 2 * 4096), float("nan"), dtype=BF, device="cuda")
    a = ex.glu_dropout(bad, p=0.5, seed=SEED, offset=OFFSET)
    keep = torch.from_numpy(ox.keep_mask(np.arange(4096), 0.5, SEED, OFFSET)).cuda()
    assert torch.isnan(a[0][keep]).all() and (a[0][~keep] == 0).all()


@pytest.mark.parametrize("beta,linear_beta", [(1e-9, 1e20), (1e20, 1e-9), (1e6, 1e6), (2e6, 0.5), (70.0, 25.0)])
def test_glu_limits_far_from_the_usual(beta, linear_beta):
    # values below, around and above each limit; no term cancels in the unit itself, so its error is relative:
    # a few 2^-22 for each of the three factors.  The gradients' 1 - tanh^2 has that error beside 1.
    gen = _gen(11)
    rows, width = 24, 64
    around = [torch.tensor([1e-3, 0.3, 1.0, 3.0], device="cuda").repeat(width // 4) * min(b, top) for b, top in ((beta, 30.0), (linear_beta, 1e20))]
    gu = (torch.randn(rows, 2 * width, generator=gen, device="cuda") * torch.cat(around)).to(BF)
    gu[:, :4] = torch.randn(rows, 4, generator=gen, device="cuda").to(BF)
    da = _rand(gen, rows, width)
    n, d = _np(gu), _np(da)
    want = ox.glu_dropout(n, 0.25, SEED, OFFSET, "situ", beta, linear_beta)
    kw = dict(p=0.25, seed=SEED, offset=OFFSET, act="situ", situ_beta=beta, situ_linear_beta=linear_beta)
    _close(ex.glu_dropout(gu, **kw), want, 2.0 ** -20 * np.abs(want))
    g, u = np.split(n, 2, 1)
    s, f, h = 1 / (1 + np.exp(-g)), np.abs(beta * np.tanh(g / beta)), np.abs(linear_beta * np.tanh(u / linear_beta))
    slack = 2.0 ** -20 * np.abs(d) / 0.75 * s
    _close(ex.glu_dropout_grad(da, gu, **kw), ox.glu_dropout_grad(d, n, 0.25, SEED, OFFSET, "situ", beta, linear_beta),
           np.concatenate([slack * h * (1 + f), slack * f], 1))


@pytest.mark.parametrize("dt", [BF, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,p", [(1, 0.5), (3, 0.1), (4, 0.0), (1000, 0.3), (4099, 0.5), (300_001, 0.1)])
def test_dropout(n, p, dt):
    gen = _gen(n)
    x, r = _rand(gen, n, dt=dt), _rand(gen, n, dt=dt)
    for res in (None, r):
        want = ox.dropout(_np(x), p, SEED, OFFSET, None if res is None else _np(res))
        # scale rounded to fp32, one product, one sum
        slack = 2.0 ** -23 * (np.abs(_np(x)) / (1 - p) + (0 if res is None else np.abs(_np(res))))
        out = ex.dropout(x, p, SEED, OFFSET, residual=res)
        _close(out, want, slack)
        y = x.clone()
        assert torch.equal(ex.dropout(y, p, SEED, OFFSET, residual=res, out=y), out)
    q = r.clone()
    assert torch.equal(ex.dropout(x, p, SEED, OFFSET, residual=q, out=q), ex.dropout(x, p, SEED, OFFSET, residual=r))
    # an unaligned view takes the one-element path and draws the same mask
    if n > 1:
        v = torch.cat([x[:1], x])[1:]
        assert torch.equal(ex.dropout(v, p, SEED, OFFSET), ex.dropout(x, p, SEED, OFFSET))


def test_dropout_past_32_bit_indices():
    # element indices beyond 2^32 use the counter's high words
    n = (1 << 32) + 1024
    x = torch.ones(n, dtype=F16, device="cuda")
    out = ex.dropout(x, 0.5, SEED, OFFSET, out=x)
    for lo in (0, (1 << 32) - 512, n - 512):
        want = ox.keep_mask(np.arange(lo, lo + 512), 0.5, SEED, OFFSET) * 2.0
        assert np.array_equal(_np(out[lo:lo + 512]), want)
    del x, out
    torch.cuda.empty_cache()


def test_dropout_infinities():
    x = torch.full((4096,), float("inf"), device="cuda")
    out = ex.dropout(x, 0.5, SEED, OFFSET, residual=torch.ones_like(x))
    keep = torch.from_numpy(ox.keep_mask(np.arange(4096), 0.5, SEED, OFFSET)).cuda()
    assert torch.isposinf(out[keep]).all() and (out[~keep] == 1).all()


# ------------------------------------------------------------------------------------------ use
def test_another_stream_and_a_graph():
    off_d, off, x, dy, w = _group_inputs([30, 0, 99], 256, 512, BF)
    want = ex.glu_dropout(ex.group_mm(x, w, off_d), p=0.2, seed=5, offset=6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = ex.group_mm(x, w, off_d, stream=s)
    got = ex.glu_dropout(y, p=0.2, seed=5, offset=6, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = ex.glu_dropout(ex.group_mm(x, w, off_d), p=0.2, seed=5, offset=6)
    x2 = x.clone()
    x.mul_(2.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, ex.glu_dropout(ex.group_mm(x, w, off_d), p=0.2, seed=5, offset=6)) and not torch.equal(x, x2)


def test_refusals_of_the_binding():
    off_d, off, x, dy, w = _group_inputs([30, 2], 64, 128, BF)
    pos = torch.zeros(32, 2, dtype=torch.int32, device="cuda")
    for call in (lambda: ex.group_mm(x[:, :32], w, off_d), lambda: ex.group_mm(x.half(), w, off_d),
                 lambda: ex.group_mm(x, w, off_d[:2]), lambda: ex.group_mm(x, w, off_d.long()),
                 lambda: ex.group_mm(x.T, w, off_d), lambda: ex.group_mm(x, w, off_d.cpu()),
                 lambda: ex.group_mm_grad_w(dy[:5], x, off_d), lambda: ex.group_mm_grad_w(dy, x, off_d, accumulate=True),
                 lambda: ex.gather_rows(x, pos[:4]), lambda: ex.combine_rows(x, pos, torch.ones(3, 2, device="cuda")),
                 lambda: ex.glu_dropout(x[:, :63]), lambda: ex.glu_dropout(x, p=1.0), lambda: ex.glu_dropout(x, act="gelu"),
                 lambda: ex.dropout(x.T, 0.1, 1, 2), lambda: ex.dropout(x, 0.1, -1, 2), lambda: ex.dropout(x, 0.1, 1, 1 << 64)):
        with pytest.raises(K3Error) as err:
            call()
        assert err.value.code == ERR_CODE["ARG"]
    for call in (lambda: ex.group_mm(x.float(), w.float(), off_d), lambda: ex.gather_rows(x.float(), pos),
                 lambda: ex.glu_dropout(x.float()), lambda: ex.dropout(pos, 0.1, 1, 2)):
        with pytest.raises(K3Error) as err:
            call()
        assert err.value.code == ERR_CODE["UNSUPPORTED"]
