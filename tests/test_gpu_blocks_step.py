"""The block of a layer end to end: the norm before it, dispatch, the gated block, the down product, combine, the norm after
it with gate, residual and the next norm, forwards and backwards, against the composed fp64 definitions and against
differences of the fp64 loss; the same with 8-bit products; and the example that trains with the one-pass block."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import experts as ox

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from latent_moe_layer_gb300 import experts as ex  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F16, SCALE = torch.float16, 0.75


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def _np(t):
    return t.double().cpu().numpy()


def _forward64(x, g0, w13, w2, gain, gate, nxt, idx, mix, act):
    off, pos = ox.plan_rows(idx, w13.shape[0])
    n0 = ox.rms_norm(x, g0)
    xs = np.zeros((off[-1], x.shape[1]))
    xs[pos[pos >= 0]] = np.repeat(n0[:, None], idx.shape[1], 1)[pos >= 0]
    a = ox.group_glu(xs, w13, off, act)
    y = ox.group_mm(a, w2, off)
    z = ox.combine_rows(y, pos, mix)
    h, n = ox.norm_residual(z, x, gain, gate, SCALE, nxt)
    return h, n, (off, pos, n0, xs, a, y, z)


def _backward64(dh, dn, x, g0, w13, w2, gain, gate, nxt, idx, mix, act):
    h, _, (off, pos, n0, xs, a, y, z) = _forward64(x, g0, w13, w2, gain, gate, nxt, idx, mix, act)
    dz, dres, dgain, dgate, dnext = ox.norm_residual_grad(dh, dn, z, h, gain, gate, SCALE, nxt)
    dy, dmix = ox.combine_rows_grad(dz, y, pos, mix)
    dgu = ox.group_glu_grad(ox.group_mm_grad_x(dy, w2, off), xs, w13, off, act)
    dn0 = ox.combine_rows(ox.group_mm_grad_x(dgu, w13, off), pos)
    dx, dg0 = ox.rms_norm_grad(dn0, x, g0, add=dres)
    return dict(dx=dx, dg0=dg0, dw13=ox.group_mm_grad_w(dgu, xs, off), dw2=ox.group_mm_grad_w(dy, a, off), dgain=dgain, dgate=dgate,
                dnext=dnext, dmix=dmix)


def _inputs(T=70, K=3, E=6, L=136, I=88):
    gen = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s, scale=1.0: (torch.randn(*s, generator=gen, device="cuda") * scale).to(F16)  # noqa: E731
    idx = torch.stack([torch.randperm(E, device="cuda", generator=gen)[:K] for _ in range(T)]).int()
    idx[4] = -1                                              # a dropped token: its branch is zeros
    idx[idx == 2] = 1                                        # an expert without rows, one met twice by a token
    v = dict(x=r(T, L), g0=1 + 0.1 * r(L).float(), w13=r(E, 2 * I, L, scale=L ** -0.5), w2=r(E, L, I, scale=I ** -0.5),
             gain=1 + 0.1 * r(L).float(), gate=torch.sigmoid(r(T, L).float()).to(F16), nxt=1 + 0.1 * r(L).float())
    return v, idx, torch.rand(T, K, generator=gen, device="cuda"), r(T, L), r(T, L)


@pytest.mark.parametrize("act", ["silu", "situ"])
def test_block_gradients(act):
    v, idx, mix, dh, dn = _inputs()
    off, pos = ex.plan_rows(idx, v["w13"].shape[0])
    n0 = ex.rms_norm(v["x"], v["g0"])
    rows = int(off[-1])
    xs = ex.gather_rows(n0, pos, n_rows=rows)
    a = ex.group_glu(xs, v["w13"], off, act=act)
    y = ex.group_mm(a, v["w2"], off)
    z = ex.combine_rows(y, pos, mix)
    h, n = ex.norm_residual(z, v["x"], gain=v["gain"], gate=v["gate"], residual_scale=SCALE, next_gain=v["nxt"])
    dz, dres, dgain, dgate, dnext = ex.norm_residual_grad(dh, dn, z, h, gain=v["gain"], gate=v["gate"], residual_scale=SCALE,
                                                          next_gain=v["nxt"])
    dy, dmix = ex.combine_rows_grad(dz, y, pos, mix, out=torch.empty_like(y))
    dw2 = ex.group_mm_grad_w(dy, a, off)
    dgu = ex.group_glu_grad(ex.group_mm_grad_x(dy, v["w2"], off), xs, v["w13"], off, act=act)
    dw13 = ex.group_mm_grad_w(dgu, xs, off)
    dx, dg0 = ex.rms_norm_grad(ex.combine_rows(ex.group_mm_grad_x(dgu, v["w13"], off), pos), v["x"], v["g0"], add=dres)
    args = [_np(v[k]) for k in ("x", "g0", "w13", "w2", "gain", "gate", "nxt")] + [idx.cpu().numpy(), _np(mix), act]
    wh, wn, _ = _forward64(*args)
    # up to twelve f16 roundings in a row forwards and backwards, 2^-11 of the norm each at most: 2^-7 holds them
    for got, want, name in ((h, wh, "h"), (n, wn, "n")):
        assert np.linalg.norm(_np(got) - want) <= 2.0 ** -8 * np.linalg.norm(want), name
    want = _backward64(_np(dh), _np(dn), *args)
    got = dict(dx=dx, dg0=dg0, dw13=dw13, dw2=dw2, dgain=dgain, dgate=dgate, dnext=dnext, dmix=dmix)
    for k, w in want.items():
        assert np.linalg.norm(_np(got[k]) - w) <= 2.0 ** -7 * np.linalg.norm(w), k
    assert not dw13[2].any() and not dw2[2].any() and ex.status() == 0


def test_block_in_a_graph_is_the_same():
    v, idx, mix, dh, dn = _inputs()
    rows = idx.numel()

    def step():
        off, pos = ex.plan_rows(idx, v["w13"].shape[0])
        xs = ex.gather_rows(ex.rms_norm(v["x"], v["g0"]), pos, out=buf)
        a = ex.group_glu(xs, v["w13"], off)
        h, n = ex.norm_residual(ex.combine_rows(ex.group_mm(a, v["w2"], off), pos, mix), v["x"], gain=v["gain"], gate=v["gate"],
                                next_gain=v["nxt"])
        q, s = ex.quant8_rows(n)
        return h, ex.group_mm8(q, s, *w8, one)

    buf = torch.zeros(rows, 136, dtype=F16, device="cuda")
    w8 = ex.quant8_weights(v["w13"][:1])
    one = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    want = step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(2):
        got[0].zero_(), got[1].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert ex.status() == 0


def test_block_with_8_bit_products():
    v, idx, mix, dh, dn = _inputs()
    off, pos = ex.plan_rows(idx, v["w13"].shape[0])
    rows, offn = int(off[-1]), off.cpu().numpy()
    xs = ex.gather_rows(ex.rms_norm(v["x"], v["g0"]), pos, n_rows=rows)
    q, s = ex.quant8_rows(xs)
    w, ws, wt = ex.quant8_weights(v["w13"], transposed=True)
    gu = ex.group_mm8(q, s, w, ws, off, out_dtype=F16)
    want = ox.group_mm(ox.dequant8(_np(q), s.cpu().numpy()), ox.dequant8(_np(w), ws.cpu().numpy(), 128), offn)
    assert np.linalg.norm(_np(gu) - want) <= 2.0 ** -11 * np.linalg.norm(want) * 1.01          # one rounding, and fp32 sums
    # against the unquantised product: each code is off by 2^-4 of its value at most, the two operands' errors independent
    full = ox.group_mm(_np(xs), _np(v["w13"]), offn)
    assert np.linalg.norm(_np(gu) - full) <= 2 * 2.0 ** -4 * np.linalg.norm(full)
    dgu = ex.glu_dropout_grad(_rand_like(gu[:, :88]), gu)
    dq, ds = ex.quant8_rows(dgu, kind="e5m2")
    dxs = ex.group_mm8(dq, ds, wt, ws.transpose(1, 2), off, out_dtype=F16)
    want = ox.group_mm_grad_x(ox.dequant8(_np(dq), ds.cpu().numpy()), ox.dequant8(_np(w), ws.cpu().numpy(), 128), offn)
    assert np.linalg.norm(_np(dxs) - want) <= 2.0 ** -11 * np.linalg.norm(want) * 1.01 and ex.status() == 0


def _rand_like(t):
    return torch.randn(t.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(t.dtype)


def test_fp64_block_gradients_against_differences():
    rng = np.random.default_rng(0)
    T, K, E, L, I = 6, 2, 3, 5, 4
    idx = rng.integers(-1, E, (T, K)).astype(np.int32)
    base = dict(x=rng.standard_normal((T, L)), g0=rng.random(L) + 0.5, w13=rng.standard_normal((E, 2 * I, L)),
                w2=rng.standard_normal((E, L, I)), gain=rng.random(L) + 0.5, gate=rng.random((T, L)), nxt=rng.random(L) + 0.5)
    mix, dh, dn, eps = rng.random((T, K)), rng.standard_normal((T, L)), rng.standard_normal((T, L)), 1e-6

    def loss(b, m):
        h, n, _ = _forward64(*b.values(), idx, m, "silu")
        return (h * dh).sum() + (n * dn).sum()

    grads = _backward64(dh, dn, *base.values(), idx, mix, "silu")
    for k, name in (("x", "dx"), ("g0", "dg0"), ("w13", "dw13"), ("w2", "dw2"), ("gain", "dgain"), ("gate", "dgate"), ("nxt", "dnext")):
        for _ in range(15):
            j = tuple(rng.integers(0, s) for s in base[k].shape)
            lo, hi = {q: a.copy() for q, a in base.items()}, {q: a.copy() for q, a in base.items()}
            lo[k][j] -= eps
            hi[k][j] += eps
            # rounding of a loss of order 30 over 2 eps (about 4e-9), and eps^2 of a third derivative (a token without rows has
            # a branch of zeros, whose norm's derivatives are 1e3, 1e9 ...: it is not differenced)
            if k in ("x", "w13", "w2", "g0") and (idx < 0).all(1).any():
                continue
            assert abs((loss(hi, mix) - loss(lo, mix)) / (2 * eps) - grads[name][j]) < 1e-5, (k, j)


@pytest.mark.parametrize("act", ["silu", "situ"])
def test_example_in_one_pass(act):
    spec = importlib.util.spec_from_file_location("finetune_experts", os.path.join(ROOT, "examples", "finetune_experts.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    v, idx, mix, dh, dn = _inputs()
    steps = []
    for one_pass in (False, True):
        model = example.RoutedExperts(v["w13"], v["w2"], F16, act, 0.0, 3, one_pass=one_pass)
        out, saved = model.forward(v["x"], idx, mix)
        dx, dmix = model.backward(dh, saved)
        steps.append((out, dx, dmix, *model.grad))
    for a, b in zip(*steps):
        # the projections are rounded to f16 in one and not in the other: 2^-11 each, forwards and backwards
        assert torch.linalg.norm(a.double() - b.double()) <= 2.0 ** -8 * torch.linalg.norm(a.double())
    losses, _ = example.train(steps=2, tokens=128, p=0.1, act=act, verbose=False, one_pass=True)
    assert len(losses) == 3 and all(np.isfinite(losses)) and ex.status() == 0
