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


class _Elsewhere:
    """Stands in for a tensor or a stream of a device, of which this machine may have none."""
    def __init__(self, device):
        self.device = torch.device(device)


def test_a_stream_of_another_device_is_refused_not_ignored(monkeypatch):
    ran = []
    monkeypatch.setattr(ex, "_native", type("native", (), {"dropout": staticmethod(lambda *a: ran.append(a))}))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: torch.no_grad())         # any context manager
    with pytest.raises(K3Error) as err:
        ex.dropout(_Elsewhere("cuda:0"), 0.1, 1, 2, stream=_Elsewhere("cuda:1"))
    assert err.value.code == ERR_CODE["ARG"] and "stream" in str(err.value) and not ran
    ex.dropout(_Elsewhere("cuda:1"), 0.1, 1, 2, stream=_Elsewhere("cuda:1"))
    ex.dropout(_Elsewhere("cuda:0"), 0.1, 1, 2)
    assert len(ran) == 2


def test_status_reads_the_current_device_unless_told_another(monkeypatch):
    words = {d: torch.tensor([-10 - d, 0, 0, 0], dtype=torch.int32) for d in (0, 1)}
    monkeypatch.setattr(ex, "_status", dict(words))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda dev=None: None)
    assert ex.status("cuda") == -11 and ex.status() == 0 and int(words[0][0]) == -10
    words[1][0] = -11
    assert ex.status(torch.device("cuda")) == -11
    assert ex.status("cuda:0") == -10 and ex.status(0) == 0 and ex.status("cuda:7") == 0
    with pytest.raises(K3Error) as err:
        ex.status("cpu")
    assert err.value.code == ERR_CODE["ARG"]


def test_soft_limits_without_a_finite_reciprocal_are_refused():
    from latent_moe_layer_gb300 import k3moe
    lib, far = k3moe.lib(), [1 << 40, 2 << 40, 3 << 40]                # addresses that a refused call never touches
    inf = float("inf")
    for b, lb in ((inf, 25.0), (4.0, inf), (1e-39, 25.0), (4.0, 1e-45), (3e38, 25.0), (float("nan"), 25.0), (4.0, float("nan"))):
        assert lib.k3moe_glu_dropout(far[0], 64, 4, 32, 1, 1, b, lb, 0.1, 1, 2, far[1], 32, None) == ERR_CODE["ARG"]
        assert lib.k3moe_glu_dropout_grad(far[2], 32, far[0], 64, 4, 32, 1, 1, b, lb, 0.1, 1, 2, far[1], 64, None) == ERR_CODE["ARG"]
    for b, lb in ((0.0, -1.0), (-inf, 25.0), (2.0 ** -126, 2.0 ** 126)):
        assert lib.k3moe_glu_dropout(None, 64, 0, 32, 1, 1, b, lb, 0.1, 1, 2, None, 32, None) == 0
