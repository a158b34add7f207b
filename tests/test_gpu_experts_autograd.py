"""The expert training operators beside autograd: they record nothing, so they refuse what would have to be
recorded, and a given output counts as written in place."""
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
    """(call, its float arguments, the others' keywords, the names under which an output may be given)"""
    r = lambda *s, dt=BF: torch.randn(*s, device="cuda").to(dt)  # noqa: E731
    pos = torch.arange(8, dtype=torch.int32, device="cuda").reshape(4, 2)
    off = torch.tensor([0, 3, 8], dtype=torch.int32, device="cuda")
    f32 = torch.float32
    return [(lambda x, out: ex.gather_rows(x, pos, out=out), [r(4, 16)], r(8, 16)),
            (lambda y, w, out: ex.combine_rows(y, pos, w, out=out), [r(8, 16), r(4, 2, dt=f32)], r(4, 16)),
            (lambda dz, y, w, out: ex.combine_rows_grad(dz, y, pos, w, out=out)[0], [r(4, 16), r(8, 16), r(4, 2, dt=f32)], r(8, 16)),
            (lambda x, w, out: ex.group_mm(x, w, off, out=out), [r(8, 16), r(2, 24, 16)], r(8, 24)),
            (lambda dy, w, out: ex.group_mm_grad_x(dy, w, off, out=out), [r(8, 24), r(2, 24, 16)], r(8, 16)),
            (lambda dy, x, out: ex.group_mm_grad_w(dy, x, off, out=out), [r(8, 24), r(8, 16)], r(2, 24, 16, dt=f32)),
            (lambda gu, out: ex.glu_dropout(gu, 0.1, 1, 2, out=out), [r(8, 32)], r(8, 16)),
            (lambda da, gu, out: ex.glu_dropout_grad(da, gu, 0.1, 1, 2, out=out), [r(8, 16), r(8, 32)], r(8, 32)),
            (lambda x, res, out: ex.dropout(x, 0.1, 1, 2, residual=res, out=out), [r(64), r(64)], r(64))]


def test_every_argument_that_needs_gradients_is_refused():
    for call, args, out in _calls():
        for i in range(len(args) + 1):
            given = [a.detach().requires_grad_(j == i) for j, a in enumerate(args + [out])]
            with pytest.raises(K3Error) as err:
                call(*given)
            assert err.value.code == ERR_CODE["UNSUPPORTED"] and "gradients" in str(err.value)
            with torch.no_grad():
                assert not call(*given[:-1], None).requires_grad and torch.is_tensor(call(*given))
        assert not call(*[a.detach() for a in args], None).requires_grad
    assert ex.status() == 0


def test_a_given_output_counts_as_written_in_place():
    for call, args, out in _calls():
        before = out._version
        assert call(*args, out).data_ptr() == out.data_ptr() and out._version == before + 1
        assert all(a._version == b for a, b in zip(args, [0] * len(args)))
        with torch.inference_mode():
            call(*[a.clone() for a in args], out.clone())
    gu, da = torch.randn(8, 32, device="cuda").to(BF), torch.randn(8, 16, device="cuda").to(BF)
    loss = (gu * torch.ones(32, device="cuda", dtype=BF, requires_grad=True)).sum()         # saves gu
    ex.glu_dropout_grad(da, gu, out=gu)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    assert ex.status() == 0
