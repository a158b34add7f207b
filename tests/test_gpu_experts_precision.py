"""Grouped products where a lost or a truncated contraction value shows: sums of small whole numbers, which
fp32 holds exactly in any order, must come out exactly; and fp32 results must be fp32-precise at any length.

The bound of the second kind: the tensor cores truncate as they add.  For products of one sign, the worst case,
that takes 3.2e-9 of the sum a contraction value in bf16 and 6.3e-9 in f16; parts of at most 512 and 256 values
(1.7e-6) are added in fp32, and those additions round to 2^-24 of a running sum each.  Against the norm of the result
2e-6 covers both at any length.  A 16-bit output of up to 8192 contraction values is the truncated sum of all,
rounded."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from latent_moe_layer_gb300 import experts as ex  # noqa: E402

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = pytest.mark.parametrize("dt", [BF, F16], ids=["bf16", "f16"])


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert ex.status() == 0


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _whole(gen, *shape, dt):
    return torch.randint(-1, 2, shape, generator=gen, device="cuda", dtype=torch.int32).to(dt)


def _offsets(sizes, before=0):
    off = (np.concatenate([[0], np.cumsum(sizes)]) + before).astype(np.int32)
    return off, torch.from_numpy(off).cuda()


def _products(off, x, dy, w):
    """fp64 y, dx, dw of every expert."""
    for e, (a, b) in enumerate(zip(off[:-1].tolist(), off[1:].tolist())):
        xe, de, we = x[a:b].double(), dy[a:b].double(), w[e].double()
        yield a, b, e, xe @ we.T, de @ we, de.T @ xe


def _check_exact(sizes, K, N, dt, pad=0):
    """All three products of whole numbers; `pad` elements in front of every row."""
    gen = _gen(K + 3 * N + len(sizes))
    off, off_d = _offsets(sizes)
    cut = lambda t: t[..., pad:]  # noqa: E731
    x, dy = cut(_whole(gen, off[-1], K + pad, dt=dt)), cut(_whole(gen, off[-1], N + pad, dt=dt))
    w = cut(_whole(gen, len(sizes), N, K + pad, dt=dt))
    y, dx, dw = (ex.group_mm(x, w, off_d, out_dtype=F32), ex.group_mm_grad_x(dy, w, off_d, out_dtype=F32),
                 ex.group_mm_grad_w(dy, x, off_d))
    # f16 holds the whole numbers up to 2048, bf16 up to 256
    y16, dx16 = ex.group_mm(x, w, off_d), ex.group_mm_grad_x(dy, w, off_d)
    for a, b, e, wy, wdx, wdw in _products(off, x, dy, w):
        assert torch.equal(y[a:b].double(), wy) and torch.equal(dx[a:b].double(), wdx), (sizes, K, N, e)
        assert torch.equal(dw[e].double(), wdw), (sizes, K, N, e)
        assert torch.equal(y16[a:b], wy.to(dt)) and torch.equal(dx16[a:b], wdx.to(dt)), (sizes, K, N, e)


@TYPES
@pytest.mark.parametrize("sizes,long,short", [
    ([1], 6144, 64), ([1], 4096, 256), ([5], 2056, 72), ([0, 300], 3104, 520), ([257, 0, 3], 1000, 96), ([40] * 6, 2048, 600),
    ([513, 1, 1], 2048, 256), ([700], 1608, 640), ([256], 320, 256), ([16, 31], 16392, 40), ([1] * 16, 4096, 512),
    ([33, 129, 17], 520, 1024), ([200] * 40, 1032, 328), ([2000, 5, 900], 584, 264), ([300, 0, 511, 513, 31], 576, 640)])
def test_whole_numbers_exactly(sizes, long, short, dt):
    _check_exact(sizes, long, short, dt)
    _check_exact(sizes, short, long, dt)


@TYPES
@pytest.mark.parametrize("n", [511, 512, 513, 1024, 1025, 2003])
def test_whole_numbers_exactly_off_16_byte_boundaries(n, dt):
    # the contraction of mm, grad_x and grad_w in turn, around the parts of 512 values
    for sizes, K, N in (([70, 0, 3], n, 66), ([70, 0, 3], 67, n), ([n, 5, n], 67, 66)):
        _check_exact(sizes, K, N, dt, pad=1)


@TYPES
def test_whole_numbers_exactly_where_an_expert_s_rows_exceed_the_cache_share(dt):
    # 32 MB of an expert's rows pass under a block of weights: 256 rows of 65,536 values, 1,024 of 16,384
    _check_exact([600, 1500, 0, 100], 65536, 520, dt)
    _check_exact([2100, 7], 16384, 16384 // 8, dt)
    _check_exact([300, 700], 264, 65536, dt)


def _norm_error(got, want):
    return float(torch.linalg.norm(got.double() - want) / torch.linalg.norm(want))


@TYPES
@pytest.mark.parametrize("sizes,K,N", [([1], 6144, 64), ([2001, 30], 1001, 2003), ([300, 5], 3584, 6144), ([40] * 6, 6144, 600), ([16, 31], 16392, 264),
                                       ([1000, 800], 16384, 512), ([700] * 14, 6144, 3584)])
def test_fp32_products_are_fp32_precise_at_any_length(sizes, K, N, dt):
    gen = _gen(K + N)
    off, off_d = _offsets(sizes)
    rnd = lambda *s, scale=1.0: (torch.randn(*s, generator=gen, device="cuda") * scale).to(dt)  # noqa: E731
    # one sign, so that truncation, which is always towards zero, cannot average out
    x, dy, w = rnd(off[-1], K).abs(), rnd(off[-1], N).abs(), rnd(len(sizes), N, K, scale=K ** -0.5).abs()
    y, dx = ex.group_mm(x, w, off_d, out_dtype=F32), ex.group_mm_grad_x(dy, w, off_d, out_dtype=F32)
    dw = ex.group_mm_grad_w(dy, x, off_d)
    for a, b, e, wy, wdx, wdw in _products(off, x, dy, w):
        assert _norm_error(y[a:b], wy) <= 2e-6, ("y", e)
        assert _norm_error(dx[a:b], wdx) <= 2e-6, ("dx", e)
        assert _norm_error(dw[e], wdw) <= 2e-6, ("dw", e)
    # a 16-bit output: the nearest of its type to a sum that has lost 6.4e-9 of itself a value, up to 8192 of them
    y16, dx16 = ex.group_mm(x, w, off_d), ex.group_mm_grad_x(dy, w, off_d)
    half = 2.0 ** -8 if dt == BF else 2.0 ** -11
    for a, b, e, wy, wdx, _ in _products(off, x, dy, w):
        for got, want, n in ((y16[a:b], wy, K), (dx16[a:b], wdx, N)):
            binade = torch.exp2(torch.floor(torch.log2(want)))
            assert ((got.double() - want).abs() <= half * binade + (6.4e-9 * min(n, 8192) + 2e-6) * want).all(), (e, n)
