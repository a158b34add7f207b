"""The gated block, 8-bit operands and norms beside autograd: what would have to be recorded is refused, and a given output
counts as written in place."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from latent_moe_layer_gb300 import experts as ex  # noqa: E402
from latent_moe_layer_gb300.k3moe import ERR_CODE, K3Error  # noqa: E402

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def _calls():
    """(call, its float arguments, the output that may be given or None)"""
    r = lambda *s, dt=BF: torch.randn(*s, device="cuda").to(dt)  # noqa: E731
    off = torch.tensor([0, 3, 8], dtype=torch.int32, device="cuda")
    f32 = torch.float32
    q, s = ex.quant8_rows(r(8, 64))
    w, ws = ex.quant8_weights(r(2, 24, 64))
    return [(lambda x, w, out: ex.group_glu(x, w, off, out=out), [r(8, 16), r(2, 48, 16)], r(8, 24)),
            (lambda da, x, w, out: ex.group_glu_grad(da, x, w, off, out=out), [r(8, 24), r(8, 16), r(2, 48, 16)], r(8, 48)),
            (lambda out: ex.group_mm8(q, s, w, ws, off, out=out), [], r(8, 24)),
            (lambda x, g, out: ex.rms_norm(x, g, out=out), [r(8, 64), r(64, dt=f32)], r(8, 64)),
            (lambda dy, x, g, a, out: ex.rms_norm_grad(dy, x, g, add=a, out=out)[0], [r(8, 64), r(8, 64), r(64, dt=f32), r(8, 64)], r(8, 64)),
            (lambda y, res, g, m, n, out: ex.norm_residual(y, res, gain=g, gate=m, next_gain=n, out=out)[0],
             [r(8, 64), r(8, 64), r(64, dt=f32), r(8, 64), r(64, dt=f32)], r(8, 64)),
            (lambda dh, dn, y, h, g, m, n, out: ex.norm_residual_grad(dh, dn, y, h, gain=g, gate=m, next_gain=n)[0],
             [r(8, 64), r(8, 64), r(8, 64), r(8, 64), r(64, dt=f32), r(8, 64), r(64, dt=f32)], None),
            (lambda x, out: ex.quant8_rows(x)[1], [r(8, 64)], None), (lambda w, out: ex.quant8_weights(w)[1], [r(2, 24, 64)], None)]


def test_every_argument_that_needs_gradients_is_refused():
    for call, args, out in _calls():
        for i in range(len(args) + (out is not None)):
            given = [a.detach().requires_grad_(j == i) if a is not None else None for j, a in enumerate(args + [out])]
            with pytest.raises(K3Error) as err:
                call(*given)
            assert err.value.code == ERR_CODE["UNSUPPORTED"] and "gradients" in str(err.value)
            with torch.no_grad():
                assert not call(*given[:-1], None).requires_grad
    assert ex.status() == 0


def test_a_given_output_counts_as_written_in_place():
    for call, args, out in _calls():
        if out is None:
            continue
        before = out._version
        assert call(*args, out).data_ptr() == out.data_ptr() and out._version == before + 1
        assert all(a._version == 0 for a in args)
        with torch.inference_mode():
            call(*[a.clone() for a in args], out.clone())
    assert ex.status() == 0
