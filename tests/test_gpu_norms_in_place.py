"""Norms through the C calls with outputs in place of inputs, every pairing that they allow: the same bits as apart."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_experts import BF, F16, F32  # noqa: E402
from test_gpu_norms import _inputs  # noqa: E402

CODE = {F32: 0, BF: 1, F16: 2}
# two rows a CTA and more; pipelined, one slot, rows wider than 8192, several rows a CTA, off 16-byte boundaries
SIZES = [(700, 3584, BF), (320, 7168, F32), (320, 9216, F16), (30_001, 96, BF), (3001, 1001, F32), (320, 8200, BF)]
ROWS = pytest.mark.parametrize("T,D,dt", SIZES, ids=[f"T{t}D{d}{str(x)[6:]}" for t, d, x in SIZES])


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    from latent_moe_layer_gb300 import k3moe
    return k3moe.lib()


def _p(t):
    return C.c_void_p(t.data_ptr() if t is not None else None)


def _stream():
    return C.c_void_p(torch.cuda.current_stream().cuda_stream)


@ROWS
@pytest.mark.parametrize("gate", ["row", "full"])
def test_gradient(lib, T, D, dt, gate):
    v = _inputs(T, D, gate, dt)
    v["h"] = v["res"]
    ws = torch.empty(lib.k3moe_norm_grad_workspace_bytes(T, D) // 4, device="cuda")
    kind = 1 if gate == "row" else 2

    def run(over):
        """over: output name -> the input whose memory it takes."""
        w = {k: v[k].clone() for k in ("dh", "dn", "y", "h", "gate")}
        out = {k: torch.full((T, D), float("nan"), dtype=dt, device="cuda") for k in ("dy", "dres")}
        out["dgate"] = torch.full_like(v["gate"], float("nan"))
        out.update({k: w[i] for k, i in over.items()})
        dgain, dnext = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
        rc = lib.k3moe_norm_residual_grad(_p(w["dh"]), D, _p(w["dn"]), D, _p(w["y"]), D, _p(w["h"]), D, _p(v["gain"]), _p(v["next_gain"]), 0,
                                          _p(w["gate"]), D, kind, 0.75, 1e-6, T, D, CODE[dt], _p(out["dy"]), D, _p(out["dres"]), D,
                                          _p(out["dgate"]), D, _p(dgain), _p(dnext), _p(ws), ws.numel() * 4, _stream())
        assert rc == 0
        return [out["dy"], out["dres"], out["dgate"], dgain, dnext]

    want = run({})
    ins = ["dh", "dn", "y", "h"] + (["gate"] if gate == "full" else [])
    pairs = [{o: i} for o in ["dy", "dres"] + (["dgate"] if gate == "full" else []) for i in ins]
    pairs += [{"dy": a, "dres": b} for a, b in (("y", "dh"), ("h", "dn"), ("dn", "y"), ("dh", "h"))]
    if gate == "full":
        pairs += [{"dy": "y", "dres": "dh", "dgate": "gate"}, {"dy": "dn", "dres": "gate", "dgate": "y"}]
    for over in pairs:
        for got, ref in zip(run(over), want):
            assert torch.equal(got, ref), over


@ROWS
@pytest.mark.parametrize("gate", ["row", "full"])
def test_forward(lib, T, D, dt, gate):
    v = _inputs(T, D, gate, dt)
    kind = 1 if gate == "row" else 2

    def run(over):
        w = {k: v[k].clone() for k in ("y", "res", "gate")}
        out = {k: torch.full((T, D), float("nan"), dtype=dt, device="cuda") for k in ("h", "n")}
        out.update({k: w[i] for k, i in over.items()})
        rc = lib.k3moe_norm_residual(_p(w["y"]), D, _p(w["res"]), D, _p(v["gain"]), _p(v["next_gain"]), 0, _p(w["gate"]), D, kind, 0.75, 1e-6,
                                     T, D, CODE[dt], _p(out["h"]), D, _p(out["n"]), D, _stream())
        assert rc == 0
        return [out["h"], out["n"]]

    want = run({})
    ins = ["y", "res"] + (["gate"] if gate == "full" else [])
    for over in [{o: i} for o in ("h", "n") for i in ins] + [{"h": a, "n": b} for a in ins for b in ins if a != b]:
        for got, ref in zip(run(over), want):
            assert torch.equal(got, ref), over


@ROWS
def test_rms_norm(lib, T, D, dt):
    v = _inputs(T, D, "none", dt)
    ws = torch.empty(lib.k3moe_norm_grad_workspace_bytes(T, D) // 4, device="cuda")

    def grad(over):
        w = {"dy": v["dn"].clone(), "x": v["y"].clone(), "add": v["dh"].clone()}
        dx = w.get(over, torch.full((T, D), float("nan"), dtype=dt, device="cuda"))
        dgain = torch.empty(D, device="cuda")
        assert lib.k3moe_rms_norm_grad(_p(w["dy"]), D, _p(w["x"]), D, _p(v["gain"]), 0, _p(w["add"]), D, 1e-6, T, D, CODE[dt], _p(dx), D,
                                       _p(dgain), _p(ws), ws.numel() * 4, _stream()) == 0
        return dx, dgain

    want = grad(None)
    for over in ("dy", "x", "add"):
        assert all(torch.equal(a, b) for a, b in zip(grad(over), want)), over
    x, out = v["y"].clone(), torch.empty_like(v["y"])
    for to in (out, x):
        assert lib.k3moe_rms_norm(_p(x), D, _p(v["gain"]), 0, 1e-6, T, D, CODE[dt], _p(to), D, _stream()) == 0
    assert torch.equal(out, x)
