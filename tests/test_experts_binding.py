"""The Python side of the expert training operators (latent_moe_layer_gb300.experts) that needs no GPU: what is
refused, and on which device and stream a call runs."""
import pytest

torch = pytest.importorskip("torch")

from latent_moe_layer_gb300 import experts as ex  # noqa: E402
from latent_moe_layer_gb300.k3moe import ERR_CODE, K3Error  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def test_a_tensor_that_needs_gradients_is_refused_not_left_out():
    x = torch.zeros(4, 8, requires_grad=True)
    pos, off = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: ex.gather_rows(x, pos), lambda: ex.combine_rows(x, pos), lambda: ex.combine_rows_grad(x, x, pos, x),
                 lambda: ex.group_mm(x, x[None], off), lambda: ex.group_mm_grad_x(x, x[None], off),
                 lambda: ex.group_mm_grad_w(x, x, off), lambda: ex.glu_dropout(x), lambda: ex.glu_dropout_grad(x, x),
                 lambda: ex.dropout(x, 0.1, 1, 2)):
        with pytest.raises(K3Error) as err:
            call()
        assert err.value.code == ERR_CODE["UNSUPPORTED"] and "gradients" in str(err.value)
        with torch.no_grad(), pytest.raises(K3Error) as err:      # then only the device is wrong
            call()
        assert err.value.code == ERR_CODE["ARG"]
