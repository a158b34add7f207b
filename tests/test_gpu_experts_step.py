"""One training step of the routed experts end to end (examples/finetune_experts.py): every gradient of the
composed operators against the fp64 definitions and against differences of the fp64 loss, and a short run."""
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


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("finetune_experts", os.path.join(ROOT, "examples", "finetune_experts.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _np(t):
    return t.double().cpu().numpy()


def _loss64(h, w13, w2, idx, mix, dout, act, p, seed, offset):
    """<out, dout> in fp64, with every tensor the backward pass would need."""
    offsets, pos = ox.plan_rows(idx, w13.shape[0])
    xs = np.zeros((offsets[-1], h.shape[1]))
    xs[pos[pos >= 0]] = np.repeat(h[:, None], idx.shape[1], 1)[pos >= 0]
    gu = ox.group_mm(xs, w13, offsets)
    a = ox.glu_dropout(gu, p, seed, offset, act)
    y = ox.group_mm(a, w2, offsets)
    out = ox.dropout(ox.combine_rows(y, pos, mix), p, seed, offset + 1, h)
    return (out * dout).sum(), (offsets, pos, xs, gu, a, y)


def _grads64(h, w13, w2, idx, mix, dout, act, p, seed, offset):
    _, (offsets, pos, xs, gu, a, y) = _loss64(h, w13, w2, idx, mix, dout, act, p, seed, offset)
    dz = ox.dropout(dout, p, seed, offset + 1)
    dy, dmix = ox.combine_rows_grad(dz, y, pos, mix)
    dgu = ox.glu_dropout_grad(ox.group_mm_grad_x(dy, w2, offsets), gu, p, seed, offset, act)
    dh = ox.combine_rows(ox.group_mm_grad_x(dgu, w13, offsets), pos) + dout
    return dh, dmix, ox.group_mm_grad_w(dgu, xs, offsets), ox.group_mm_grad_w(dy, a, offsets)


@pytest.mark.parametrize("act", ["silu", "situ"])
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_step_gradients(example, act, p):
    T, K, E, L, I, seed = 45, 3, 7, 96, 72, 11
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s, scale=1.0: (torch.randn(*s, generator=gen, device="cuda") * scale).half()  # noqa: E731
    h, dout = rnd(T, L), rnd(T, L)
    idx = torch.stack([torch.randperm(E, device="cuda", generator=gen)[:K] for _ in range(T)]).int()
    idx[4] = -1                                              # a dropped token: its output is the residual
    idx[idx == 5] = 6                                        # an expert without rows, one met twice by a token
    mix = torch.rand(T, K, device="cuda", generator=gen)
    model = example.RoutedExperts(rnd(E, 2 * I, L, scale=L ** -0.5), rnd(E, L, I, scale=I ** -0.5), torch.float16, act, p, seed)
    args = (_np(h), _np(model.w13), _np(model.w2), idx.cpu().numpy(), _np(mix), _np(dout), act, p, seed, 0)
    out, saved = model.forward(h, idx, mix)
    want, _ = _loss64(*args)
    # f16 roundings of five stored tensors, each 2^-11 relative at most and independent: relative to the norms 2^-9 holds
    got = (out.double() * dout.double()).sum().item()
    assert abs(got - want) <= 2.0 ** -9 * float(torch.linalg.norm(out.double()) * torch.linalg.norm(dout.double()))
    assert torch.equal(out[4], h[4])
    dh, dmix = model.backward(dout, saved)
    for g, w, name in zip((dh, dmix, model.grad[0], model.grad[1]), _grads64(*args), ("dh", "dmix", "dw13", "dw2")):
        err = np.linalg.norm(_np(g) - w) / np.linalg.norm(w)
        # up to seven f16 roundings in a row, 2^-11 each at most: 7 2^-11 < 2^-8
        assert err <= 2.0 ** -8, (name, err)
    assert not model.grad[0][5].any() and not model.grad[1][5].any() and ex.status() == 0


def test_fp64_step_gradients_against_differences():
    rng = np.random.default_rng(0)
    T, K, E, L, I = 9, 2, 3, 6, 5
    idx = rng.integers(-1, E, (T, K)).astype(np.int32)
    base = [rng.standard_normal((T, L)), rng.standard_normal((E, 2 * I, L)), rng.standard_normal((E, L, I)), rng.random((T, K))]
    dout, eps = rng.standard_normal((T, L)), 1e-6
    loss = lambda h, w13, w2, mix: _loss64(h, w13, w2, idx, mix, dout, "silu", 0.3, 5, 8)[0]  # noqa: E731
    h, w13, w2, mix = base
    dh, dmix, dw13, dw2 = _grads64(h, w13, w2, idx, mix, dout, "silu", 0.3, 5, 8)
    for i, g in ((0, dh), (1, dw13), (2, dw2), (3, dmix)):
        for _ in range(25):
            j = tuple(rng.integers(0, n) for n in base[i].shape)
            lo, hi = [b.copy() for b in base], [b.copy() for b in base]
            lo[i][j] -= eps
            hi[i][j] += eps
            # rounding of a loss of order 10 over 2 eps, and eps^2 of the third derivative
            assert abs((loss(*hi) - loss(*lo)) / (2 * eps) - g[j]) < 1e-6


@pytest.mark.parametrize("act", ["silu", "situ"])
def test_example_learns(example, act):
    losses, _ = example.train(steps=12, tokens=384, p=0.1, act=act, verbose=False)
    assert all(np.isfinite(losses)) and losses[-1] < 0.7 * losses[0], losses
