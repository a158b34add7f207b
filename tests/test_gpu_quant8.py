"""8-bit operands on the GPU: codes and scales bit for bit against oracle/experts.py, products of them against its fp64
sums.

The products of two codes are exact and so is their scaling by powers of two, so a sum of n of them is off by at most
n 2^-24 sum |a b| in fp32, twice that where the tensor cores truncate, and rounded once to the output's type."""
import numpy as np
import pytest

from oracle import experts as ox

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from latent_moe_layer_gb300 import experts as ex  # noqa: E402
from latent_moe_layer_gb300.k3moe import ERR_CODE, K3Error  # noqa: E402
from test_gpu_experts import BF, F16, F32, TYPES, _close, _gen, _np, _rand  # noqa: E402

KINDS = pytest.mark.parametrize("kind", ["e4m3", "e5m2"])


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert ex.status() == 0


def _same(got, want):
    return np.array_equal(_np(got), want, equal_nan=True)


def _spread(gen, rows, n, dt):
    """Values over most of the type's range, zeros and whole blocks of zeros among them."""
    x = torch.randn(rows, n, generator=gen, device="cuda")
    top = 15 if dt == F16 else 60
    x = x * torch.exp2(torch.randint(-top, top - 2, (rows, 1), generator=gen, device="cuda").float())
    x = x * torch.exp2(torch.randint(-12, 1, (rows, n), generator=gen, device="cuda").float())
    x = torch.where(torch.rand(rows, n, generator=gen, device="cuda") < 0.05, 0.0, x)
    if rows > 2:
        x[2] = 0
    return x.clamp(-6e4, 6e4).to(dt) if dt == F16 else x.to(dt)


# ------------------------------------------------------------------------------------------ quantising
@TYPES
@KINDS
@pytest.mark.parametrize("rows,n", [(0, 64), (1, 1), (1, 128), (3, 7), (5, 127), (4, 129), (64, 256), (7, 1001), (300, 520), (33, 3584)])
def test_rows(rows, n, kind, dt):
    x = _spread(_gen(rows + n), rows, n, dt)
    codes, scales = ex.quant8_rows(x, kind=kind)
    assert codes.shape == (rows, n) and scales.shape == (rows, -(-n // 128)) and codes.stride(0) % 16 == 0 and scales.stride(0) % 4 == 0
    want, ws = ox.quant8(_np(x), kind)
    assert np.array_equal(scales.cpu().numpy(), ws) and _same(codes, want)


@TYPES
@KINDS
def test_rows_of_extremes_and_values_that_are_not_finite(kind, dt):
    info = torch.finfo(dt)
    rows = torch.zeros(9, 256, device="cuda", dtype=dt)
    rows[0] = info.max
    rows[1] = -info.tiny
    rows[2, 3] = info.smallest_normal * info.eps              # the smallest subnormal alone
    rows[3, 5], rows[3, 200] = float("inf"), 1.0
    rows[4, :128], rows[4, 128:] = float("nan"), torch.arange(128, device="cuda") - 64
    rows[5] = float("-inf")
    rows[6] = torch.arange(256, device="cuda") / 256 - 0.5
    rows[7] = -0.0
    rows[8, 0], rows[8, 1] = 448.0, 448.0 + 448.0 * info.eps  # on and just above a power's border
    codes, scales = ex.quant8_rows(rows, kind=kind)
    want, ws = ox.quant8(_np(rows), kind)
    assert np.array_equal(scales.cpu().numpy(), ws) and _same(codes, want)
    assert torch.isnan(codes[3, 5].float()) == (kind == "e4m3") and torch.isnan(codes[4, :128].float()).all()


@TYPES
def test_strided_and_unaligned_rows(dt):
    wide = _spread(_gen(3), 40, 700, dt)
    for x in (wide[:, 8:520], wide[:, 1:258], wide[::2, 3:400], wide[5:6, 2:9]):
        codes, scales = ex.quant8_rows(x)
        want, ws = ox.quant8(_np(x), "e4m3")
        assert np.array_equal(scales.cpu().numpy(), ws) and _same(codes, want)


@TYPES
@KINDS
@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (1, 128, 128), (2, 5, 300), (3, 130, 127), (1, 257, 64), (2, 200, 520), (5, 64, 1024), (1, 640, 384)])
def test_weights(E, N, K, kind, dt):
    w = _spread(_gen(E + N + K), E * N, K, dt).reshape(E, N, K)
    want, ws = ox.quant8(_np(w), kind, 128)
    codes, scales = ex.quant8_weights(w, kind=kind)
    assert np.array_equal(scales.cpu().numpy(), ws) and _same(codes, want)
    codes2, scales2, turned = ex.quant8_weights(w, kind=kind, transposed=True)
    assert torch.equal(codes.view(torch.uint8), codes2.view(torch.uint8)) and torch.equal(scales, scales2)
    assert turned.shape == (E, K, N) and torch.equal(turned.view(torch.uint8), codes.view(torch.uint8).transpose(1, 2))


def test_weights_views():
    big = _spread(_gen(8), 3 * 150, 400, BF).reshape(3, 150, 400)
    for w in (big[:, :140, :264], big[:, 1:100, 3:200], big[::2], big[:1].expand(2, -1, -1)):
        codes, scales, turned = ex.quant8_weights(w, transposed=True)
        want, ws = ox.quant8(_np(w), "e4m3", 128)
        assert np.array_equal(scales.cpu().numpy(), ws) and _same(codes, want) and _same(turned, want.swapaxes(1, 2))


# ------------------------------------------------------------------------------------------ products
def _operands(sizes, K, N, xk="e4m3", wk="e4m3", before=0, after=0, seed=0):
    gen = _gen(seed + K + N + len(sizes))
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32) + before
    x = _rand(gen, int(off[-1]) + after, K)
    w = _rand(gen, len(sizes), N, K, scale=K ** -0.5)
    # loud rows, columns and blocks, so that every scale is another
    x = (x * torch.exp2(torch.randint(-6, 7, x.shape[:1] + (1,), generator=gen, device="cuda").float())).to(BF)
    x = (x * torch.exp2((torch.arange(K, device="cuda") // 128 % 5 * 3 - 6).float())).to(BF)
    w = (w * torch.exp2((torch.arange(K, device="cuda") // 128 % 3 * 2 - 2).float())).to(BF)
    w = (w * torch.exp2((torch.arange(N, device="cuda") // 128 % 4 * 3 - 4).float())[:, None]).to(BF)
    q, qs = ex.quant8_rows(x, kind=xk)
    return torch.from_numpy(off).cuda(), off, q, qs, ex.quant8_weights(w, kind=wk, transposed=True), w


def _check(off_d, off, q, qs, w, ws, out_dtype):
    a, b = int(off[0]), int(off[-1])
    x64, w64 = ox.dequant8(_np(q[:b]), qs[:b].cpu().numpy()), ox.dequant8(_np(w), ws.cpu().numpy(), 128)
    x64[:a] = 0
    y = ex.group_mm8(q, qs, w, ws, off_d, out_dtype=out_dtype)
    assert y.dtype == out_dtype
    want, slack = ox.group_mm(x64, w64, off)[a:b], (q.shape[1] + 2) * 2.0 ** -23 * ox.group_mm(np.abs(x64), np.abs(w64), off)[a:b]
    got = y[a:b].clone()
    if out_dtype == F16:
        # values from 65520 (halfway past the largest) on round to infinity; those within the slack of it to either
        far, near = np.abs(want) >= 65520 + slack, np.abs(np.abs(want) - 65520) <= slack
        assert np.array_equal(_np(got)[far], np.sign(want[far]) * np.inf)
        skip = torch.from_numpy(far | near).cuda()
        got[skip], want[far | near] = 0, 0
    _close(got, want, slack, "y")
    return y


GROUPS = [([1], 16, 8), ([0], 64, 64), ([0, 0, 5], 128, 128), ([2] * 16, 256, 192), ([3, 0, 17, 1, 0, 64], 96, 256),
          ([16, 15, 33, 129], 520, 264), ([239, 240, 241], 384, 136), ([300, 0, 511, 513, 31], 656, 640), ([1000, 7], 1096, 72),
          ([40] * 7 + [0] * 3 + [90] * 6, 512, 512), ([5] * 200, 144, 88), ([1, 0] * 64, 1024, 256), ([3, 9], 7, 5), ([20, 0, 70], 33, 100),
          ([65], 129, 67), ([481, 2], 2100, 300), ([7], 4096, 1024), ([300], 2056, 72)]


@pytest.mark.parametrize("out_dtype", [BF, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("sizes,K,N", GROUPS, ids=[f"E{len(s)}R{sum(s)}K{k}N{n}" for s, k, n in GROUPS])
def test_products(sizes, K, N, out_dtype):
    off_d, off, q, qs, (w, ws, wt), _ = _operands(sizes, K, N, before=2, after=19)
    _check(off_d, off, q, qs, w, ws, out_dtype)


@pytest.mark.parametrize("out_dtype", [BF, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("sizes,K,N", [([40], 8320, 72), ([300, 0, 5], 8224, 300), ([1], 16384, 128), ([7] * 40, 8256, 264)])
def test_contractions_that_16_bit_outputs_take_in_parts(sizes, K, N, out_dtype):
    off_d, off, q, qs, (w, ws, wt), _ = _operands(sizes, K, N)
    _check(off_d, off, q, qs, w, ws, out_dtype)


@pytest.mark.parametrize("sizes,K,N", [([37, 0, 260], 3584, 264), ([5, 9], 2100, 72), ([700], 520, 40)])
def test_scale_rows_on_4_byte_boundaries(sizes, K, N):
    # scales of another origin: rows of ceil(K / 128) bytes rounded up to 4, not to 16, from any such place
    off_d, off, q, qs, (w, ws, wt), _ = _operands(sizes, K, N)
    want = ex.group_mm8(q, qs, w, ws, off_d)
    n = qs.shape[1]
    for start in (0, 4):
        narrow = torch.full((qs.shape[0], -(-n // 4) * 4 + 8), 255, dtype=torch.uint8, device="cuda")[:, start:start + n]
        narrow[:] = qs
        assert torch.equal(ex.group_mm8(q, narrow, w, ws, off_d), want)


def test_many_experts():
    rng = np.random.default_rng(0)
    sizes = (rng.integers(0, 4, 1024) * (rng.random(1024) < 0.5)).tolist()
    off_d, off, q, qs, (w, ws, wt), _ = _operands(sizes, 160, 72)
    _check(off_d, off, q, qs, w, ws, BF)


@pytest.mark.parametrize("xk,wk", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
def test_products_of_either_kind(xk, wk):
    off_d, off, q, qs, (w, ws, wt), _ = _operands([70, 3, 140], 300, 200, xk, wk)
    _check(off_d, off, q, qs, w, ws, BF)


@pytest.mark.parametrize("sizes,K,N", [([33, 0, 250], 264, 392), ([5], 100, 1000), ([64] * 5, 513, 129)])
def test_transposed_weights_give_the_gradient_for_the_rows(sizes, K, N):
    off_d, off, _, _, (w, ws, wt), _ = _operands(sizes, K, N)
    dy = _rand(_gen(1), int(off[-1]), N)
    dq, dqs = ex.quant8_rows(dy, kind="e5m2")
    dx = _check(off_d, off, dq, dqs, wt, ws.transpose(1, 2), BF)
    assert dx.shape == (int(off[-1]), K)


def test_rows_of_no_expert_are_neither_read_nor_written():
    off_d, off, q, qs, (w, ws, wt), _ = _operands([70, 0, 9, 131], 192, 264, before=5, after=40)
    a, b = int(off[0]), int(off[-1])
    q.view(torch.uint8)[:a], q.view(torch.uint8)[b:], qs[:a], qs[b:] = 0x7F, 0x7F, 255, 255       # NaN codes and scales
    y = torch.full((q.shape[0], 264), 3.0, dtype=BF, device="cuda")
    ex.group_mm8(q, qs, w, ws, off_d, out=y)
    assert (y[:a] == 3).all() and (y[b:] == 3).all() and torch.isfinite(y).all()
    assert torch.equal(y[a:b], _check(off_d, off, q, qs, w, ws, BF)[a:b])


def test_nan_stays_in_its_row_and_expert():
    off_d, off, q, qs, (w, ws, wt), _ = _operands([33, 50, 7], 256, 256)
    q.view(torch.uint8)[40, 5] = 0x7F
    w.view(torch.uint8)[2, 130, 9] = 0xFF
    y = ex.group_mm8(q, qs, w, ws, off_d)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[40], bad[83:, 130] = True, True
    assert torch.equal(torch.isnan(y), bad)


def test_scales_far_from_one():
    # values near the 16-bit type's largest and smallest: the scales' product leaves fp32 neither way
    gen = _gen(5)
    x, w = _rand(gen, 20, 256), _rand(gen, 1, 64, 256)
    off = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    for sx, sw in ((2.0 ** 100, 2.0 ** -100), (2.0 ** -110, 2.0 ** 60), (2.0 ** -120, 2.0 ** 120), (2.0 ** 60, 2.0 ** 50)):
        q, qs = ex.quant8_rows((x.float() * sx).to(BF))
        v, vs = ex.quant8_weights((w.float() * sw).to(BF))
        _check(off, np.array([0, 20]), q, qs, v, vs, F32)


def test_long_contractions_keep_fp32_precision():
    # products of one sign: what truncation loses adds up
    for K in (8192, 16384 + 64):
        q = torch.full((30, K), 1.125, device="cuda").to(torch.float8_e4m3fn)
        w = torch.full((1, 128, K), 1.375, device="cuda").to(torch.float8_e4m3fn)
        qs = torch.full((30, -(-K // 512) * 4), 127, dtype=torch.uint8, device="cuda")[:, :-(-K // 128)]
        ws = torch.full((1, 1, -(-K // 128)), 126, dtype=torch.uint8, device="cuda")
        off = torch.tensor([0, 30], dtype=torch.int32, device="cuda")
        y = ex.group_mm8(q, qs, w, ws, off, out_dtype=F32)
        want = K * 1.125 * 1.375 / 2
        assert ((y.double() - want).abs() <= 2e-6 * want).all(), (y.double() - want).abs().max().item() / want


def test_one_weight_for_all_groups_and_bit_for_bit():
    off_d, off, q, qs, (w, ws, wt), _ = _operands([9, 300, 2], 520, 700)
    one, ones = w[:1].expand(3, -1, -1), ws[:1].expand(3, -1, -1)
    y = ex.group_mm8(q, qs, one, ones, off_d)
    three = torch.empty(3, *w.shape[1:-1], w.stride(1), dtype=torch.uint8, device="cuda")[..., :w.shape[2]]
    three[:] = w[:1].view(torch.uint8)
    assert torch.equal(y, ex.group_mm8(q, qs, three.view(torch.float8_e4m3fn), ones.contiguous(), off_d))
    for _ in range(3):
        assert torch.equal(ex.group_mm8(q, qs, one, ones, off_d), y)


def test_offsets_out_of_range_are_reported_and_nothing_is_written():
    _, _, q, qs, (w, ws, wt), _ = _operands([40, 24], 128, 128)
    for bad in ([0, 50, 40], [0, 40, 65], [-1, 40, 64]):
        y = torch.full((64, 128), 3.0, dtype=BF, device="cuda")
        ex.group_mm8(q, qs, w, ws, torch.tensor(bad, dtype=torch.int32, device="cuda"), out=y)
        assert ex.status() == ERR_CODE["RANGE"] and (y == 3).all()


def test_strided_outputs_another_stream_and_a_graph():
    off_d, off, q, qs, (w, ws, wt), _ = _operands([30, 0, 99], 384, 333)
    want = ex.group_mm8(q, qs, w, ws, off_d)
    wide = torch.zeros(129, 400, dtype=BF, device="cuda")
    for at in (0, 3):
        assert torch.equal(ex.group_mm8(q, qs, w, ws, off_d, out=wide[:, at:at + 333]), want)
        assert not wide[:, at + 333:].any()
        wide.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ex.group_mm8(q, qs, w, ws, off_d, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    x = _rand(_gen(2), 129, 384)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a, b = ex.quant8_rows(x)
        got = ex.group_mm8(a, b, w, ws, off_d)
    x.mul_(3.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, ex.group_mm8(*ex.quant8_rows(x), w, ws, off_d))


def test_element_offsets_past_31_bits():
    rows, K = 700_000, 3584
    q = torch.zeros(rows, K, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    qs = torch.full((rows, 28), 127, dtype=torch.uint8, device="cuda")
    last, ls = ex.quant8_rows(_rand(_gen(4), 50, K))
    q.view(torch.uint8)[-50:], qs[-50:] = last.view(torch.uint8), ls
    v = ex.quant8_weights(_rand(_gen(5), 2, 96, K, scale=K ** -0.5))
    off = torch.tensor([rows - 50, rows - 31, rows], dtype=torch.int32, device="cuda")
    y = ex.group_mm8(q, qs, *v, off)
    near = np.array([0, 19, 50], dtype=np.int32)
    x64, w64 = ox.dequant8(_np(last), ls.cpu().numpy()), ox.dequant8(_np(v[0]), v[1].cpu().numpy(), 128)
    _close(y[-50:], ox.group_mm(x64, w64, near), (K + 2) * 2.0 ** -23 * ox.group_mm(np.abs(x64), np.abs(w64), near), "y")
    x = torch.empty(rows, K, dtype=BF, device="cuda")
    x[-1] = 1.5
    a, b = ex.quant8_rows(x)
    assert (a[-1].float() * torch.exp2(b[-1, 0].float() - 127) == 1.5).all()
    del x, a, b, q, y
    torch.cuda.empty_cache()


def test_refusals_of_the_binding():
    off_d, off, q, qs, (w, ws, wt), _ = _operands([30, 2], 136, 128)
    x = _rand(_gen(0), 32, 136)
    for call in (lambda: ex.quant8_rows(x, kind="e3m4"), lambda: ex.quant8_rows(x.T), lambda: ex.quant8_weights(x),
                 lambda: ex.quant8_rows(x[:, :0]), lambda: ex.group_mm8(q[:, :128], qs, w, ws, off_d), lambda: ex.group_mm8(q, qs[:, :1], w, ws, off_d),
                 lambda: ex.group_mm8(q, qs[:5], w, ws, off_d), lambda: ex.group_mm8(q, qs, w, ws[:, :, :1], off_d),
                 lambda: ex.group_mm8(q, qs.float(), w, ws, off_d), lambda: ex.group_mm8(q, qs, w, ws, off_d[:2])):
        with pytest.raises(K3Error) as err:
            call()
        assert err.value.code == ERR_CODE["ARG"]
    narrow = q.view(torch.uint8).contiguous().view(q.dtype)                     # rows of 136 bytes
    for call in (lambda: ex.quant8_rows(x.float()), lambda: ex.group_mm8(x, qs, w, ws, off_d), lambda: ex.group_mm8(narrow, qs, w, ws, off_d),
                 lambda: ex.group_mm8(q, qs.contiguous(), w, ws, off_d), lambda: ex.group_mm8(q, qs, w, ws, off_d, out_dtype=torch.float64)):
        with pytest.raises(K3Error) as err:
            call()
        assert err.value.code == ERR_CODE["UNSUPPORTED"]
