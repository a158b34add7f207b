"""What lies between the rows of a matrix (the rest of its stride) takes no part in a result, whatever it holds, and outputs leave
it as it is; two calls at once on two streams do not disturb each other."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from latent_moe_layer_gb300 import experts as ex  # noqa: E402
from test_gpu_experts import BF, TYPES, _gen, _rand  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert ex.status() == 0


def _in_stride(t, pad, fill):
    """t's values with `pad` more columns of `fill` after each row."""
    wide = torch.full((*t.shape[:-1], t.shape[-1] + pad), fill, dtype=t.dtype, device="cuda")
    wide[..., :t.shape[-1]] = t
    return wide[..., :t.shape[-1]]


def _poison(codes, byte):
    """Every byte of the rows' strides that is no code."""
    base = torch.as_strided(codes.view(torch.uint8), (*codes.shape[:-1], codes.stride(-2)), codes.stride(), codes.storage_offset())
    base[..., codes.shape[-1]:] = byte


@pytest.mark.parametrize("out_dtype", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("sizes,K,N", [([33, 0, 70], 7, 9), ([65], 129, 67), ([5, 300], 520, 264), ([1], 33, 1), ([64, 64], 2100, 300)])
def test_codes_and_scales_between_rows(sizes, K, N, out_dtype):
    gen = _gen(K + N)
    off = torch.tensor([sum(sizes[:i]) for i in range(len(sizes) + 1)], dtype=torch.int32, device="cuda")
    q, qs = ex.quant8_rows(_rand(gen, sum(sizes), K))
    w, ws, wt = ex.quant8_weights(_rand(gen, len(sizes), N, K, scale=K ** -0.5), transposed=True)
    dq, dqs = ex.quant8_rows(_rand(gen, sum(sizes), N), kind="e5m2")
    run = lambda: (ex.group_mm8(q, qs, w, ws, off, out_dtype=out_dtype),  # noqa: E731
                   ex.group_mm8(dq, dqs, wt, ws.transpose(1, 2), off, out_dtype=out_dtype))
    for t in (q, w, wt, dq, qs, dqs):
        _poison(t, 0)
    want = run()
    for byte in (0x7F, 0xFF):                                # NaN of both kinds and of the scales
        for t in (q, w, wt, dq, qs, dqs):
            _poison(t, byte)
        for got, ref in zip(run(), want):
            assert torch.isfinite(got).all() and torch.equal(got, ref)


@TYPES
@pytest.mark.parametrize("act", ["silu", "situ"])
@pytest.mark.parametrize("K,I,pad", [(72, 40, 8), (129, 33, 7), (200, 96, 24), (70, 64, 2)])
def test_gated_block_between_rows(K, I, pad, act, dt):
    gen = _gen(K)
    off = torch.tensor([0, 33, 33, 103], dtype=torch.int32, device="cuda")
    x, w, da = _rand(gen, 103, K, dt=dt), _rand(gen, 3, 2 * I, K, dt=dt, scale=K ** -0.5), _rand(gen, 103, I, dt=dt)
    run = lambda a, b, c: (ex.group_glu(a, b, off, act=act), ex.group_glu_grad(c, a, b, off, act=act))  # noqa: E731
    want = run(*(_in_stride(t, pad, 0.0) for t in (x, w, da)))
    for fill in (float("nan"), float("inf")):
        for got, ref in zip(run(*(_in_stride(t, pad, fill) for t in (x, w, da))), want):
            assert torch.isfinite(got).all() and torch.equal(got, ref)


@TYPES
@pytest.mark.parametrize("D,pad", [(264, 8), (100, 3), (1001, 15), (3584, 16)])
def test_norms_between_rows(D, pad, dt):
    gen = _gen(D)
    t = {k: _rand(gen, 77, D, dt=dt) for k in ("y", "res", "gate", "dh", "dn")}
    gain = 1 + 0.1 * torch.randn(D, device="cuda", generator=gen)

    def run(fill):
        v = {k: _in_stride(m, pad, fill) for k, m in t.items()}
        out = torch.full((77, D + pad), 3.0, dtype=dt, device="cuda")
        h, n = ex.norm_residual(v["y"], v["res"], gain=gain, gate=v["gate"], next_gain=gain, out=out[:, :D])
        got = ex.norm_residual_grad(v["dh"], v["dn"], v["y"], h, gain=gain, gate=v["gate"], next_gain=gain)
        assert (out[:, D:] == 3).all()
        dx = torch.full((77, D + pad), 3.0, dtype=dt, device="cuda")
        more = ex.rms_norm_grad(v["dn"], v["y"], gain, add=v["dh"], out=dx[:, :D])
        assert (dx[:, D:] == 3).all()
        return [h, n, *got, *more, ex.rms_norm(v["y"], gain)]

    want = run(0.0)
    for got, ref in zip(run(float("nan")), want):
        assert torch.isfinite(got).all() and torch.equal(got, ref)


def test_two_calls_at_once():
    gen = _gen(1)
    K, N, sizes = 1024, 512, [700, 0, 300, 4]
    off = torch.tensor([0, 700, 700, 1000, 1004], dtype=torch.int32, device="cuda")
    x, w, da = _rand(gen, 1004, K), _rand(gen, 4, 2 * N, K, scale=K ** -0.5), _rand(gen, 1004, N)
    q, qs = ex.quant8_rows(x)
    v, vs = ex.quant8_weights(w)
    few = torch.tensor([0, 3, 3, 5, 9], dtype=torch.int32, device="cuda")
    calls = [lambda s: ex.group_mm8(q, qs, v, vs, off, stream=s), lambda s: ex.group_glu(x, w, off, stream=s),
             lambda s: ex.group_glu_grad(da, x, w, off, stream=s), lambda s: ex.group_mm8(q[:9], qs[:9], v, vs, few, stream=s),
             lambda s: ex.group_glu(x[:9], w, few, stream=s), lambda s: ex.quant8_rows(x, stream=s)[0].view(torch.uint8),
             lambda s: ex.rms_norm_grad(x, x, None, stream=s)[0]]
    want = [c(None) for c in calls]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [(i, calls[i](s)) for i in range(len(calls)) for s in streams]
        torch.cuda.synchronize()
        assert all(torch.equal(g, want[i]) for i, g in got)
