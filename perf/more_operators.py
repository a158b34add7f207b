"""Measured cases of the 8-bit products, the gated block and the norms around a block: rows and weights to 8-bit
floating point with a power-of-two scale for each block of 128, products of such operands grouped by expert, both
projections of the gated block with its unit in one pass and its backward pass, and the norm after a block with its
gate, the residual and the norm before the next block.

Each case is run through `run` either in its plain form (elementary torch operations in 32 bits, rounded once at
the end) or, where `own` is set, through the library's entry points.  `exact` gives the same outputs from the
definitions in 64 bits.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_TOP = {"e4m3": 9, "e5m2": 16}                  # the largest value is 0.875 * 2^_TOP: 448 and 57344
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 128
EPS = 1e-6


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the routed rows of a training micro-batch on their way into the 8-bit gate and up projections
        {"name": "quant_rows_train", "op": "quant_rows", "rows": 65536, "n": 3584, "type": "bf16", "kind": "e4m3"},
        # the down projections of one of 32 ranks after an optimizer step: both orders from one read
        {"name": "quant_weights_rank", "op": "quant_weights", "E": 28, "N": 3584, "K": 3072, "type": "bf16", "kind": "e4m3",
         "transposed": True},
        # one of eight ranks at a decode batch: bound by reading the touched 8-bit weights
        {"name": "mm8_decode", "op": "mm8", "E": 112, "rows": 251, "K": 3584, "N": 6144, "type": "bf16", "kind": "e4m3",
         "out": "bf16", "skew": 0.3, "empty": 11},
        # gate and up projections of a training micro-batch on one of eight ranks, rows rounded on the way
        {"name": "mm8_train", "op": "mm8", "E": 112, "rows": 65536, "K": 3584, "N": 6144, "type": "bf16", "kind": "e4m3",
         "out": "bf16", "skew": 0.4, "empty": 0},
        # gradient of the down projection's input on one of 64 ranks: wide-range gradients, transposed weights, ragged
        {"name": "mm8_grad_x_rank", "op": "mm8_grad_x", "E": 14, "rows": 2047, "K": 3072, "N": 3584, "type": "f16",
         "kind": "e5m2", "out": "f16", "skew": 0.6, "empty": 1},
        # the gated block's projections at a decode batch on one of eight ranks
        {"name": "glu_decode", "op": "glu", "E": 112, "rows": 251, "K": 3584, "I": 3072, "type": "bf16", "act": "silu",
         "skew": 0.3, "empty": 11},
        # the same for a training micro-batch on one of sixteen ranks
        {"name": "glu_train", "op": "glu", "E": 56, "rows": 32768, "K": 3584, "I": 3072, "type": "bf16", "act": "silu",
         "skew": 0.4, "empty": 0},
        # the block's backward pass on one of 32 ranks, nothing kept from the forward pass but the rows
        {"name": "glu_grad_train", "op": "glu_grad", "E": 28, "rows": 16381, "K": 3584, "I": 3072, "type": "bf16",
         "act": "silu", "skew": 0.4, "empty": 1},
        # the soft-limited unit's backward pass on few ragged rows
        {"name": "glu_grad_situ", "op": "glu_grad", "E": 14, "rows": 1021, "K": 3584, "I": 3072, "type": "f16",
         "act": "situ", "skew": 0.6, "empty": 1},
        # between two blocks at a decode batch of 16 tokens: pure latency
        {"name": "norm_decode", "op": "norm", "T": 16, "D": 7168, "type": "bf16", "gate": "none", "scale": 1.0, "next": True},
        # between two blocks of a training micro-batch, an elementwise gate on the branch
        {"name": "norm_train", "op": "norm", "T": 8192, "D": 7168, "type": "bf16", "gate": "full", "scale": 0.75,
         "next": True},
        # its gradient for every input
        {"name": "norm_grad_train", "op": "norm_grad", "T": 8192, "D": 7168, "type": "bf16", "gate": "full", "scale": 0.75,
         "next": True},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["quant_rows", "quant_weights", "mm8", "mm8", "mm8_grad_x", "glu", "glu", "glu_grad", "norm", "norm_grad"])
    c = {"op": op, "type": rng.choice(["bf16", "f16"])}
    if op == "quant_rows":
        n = _log(rng, 1, 7168)
        c.update(rows=min(_log(rng, 1, 65536), 200_000_000 // n), n=n, kind=rng.choice(["e4m3", "e5m2"]))
    elif op == "quant_weights":
        E, N, K = _log(rng, 1, 112), _log(rng, 16, 6144), _log(rng, 16, 6144)
        while E * K * N > 300_000_000:
            E = max(1, E // 2)
        c.update(E=E, N=N, K=K, kind=rng.choice(["e4m3", "e4m3", "e5m2"]), transposed=rng.random() < 0.5)
    elif op in ("mm8", "mm8_grad_x", "glu", "glu_grad"):
        glu = op in ("glu", "glu_grad")
        E = _log(rng, 1, 112)
        K, N = _log(rng, 64, 6144, 8), _log(rng, 64, 3000 if glu else 6144, 8)
        if not glu and rng.random() < 0.3:
            K, N = K + rng.randrange(8), N + rng.randrange(8)
        while E * K * N * (1 + glu) > 400_000_000:
            E = max(1, E // 2)
        rows = _log(rng, 1, 32768)
        while rows * K * N * (1 + glu) > 300_000_000_000:
            rows = max(1, rows // 2)
        c.update(E=E, rows=rows, K=K, skew=rng.choice([0.0, 0.4, 0.8]), empty=rng.choice([0, E // 8, E // 3]))
        if glu:
            c.update(I=N, act=rng.choice(["silu", "situ"]))
        else:
            c.update(N=N, kind=rng.choice(["e4m3", "e5m2"]), out=rng.choice([c["type"], "f32"]))
    else:
        D = _log(rng, 16, 8192, rng.choice([1, 8, 8, 8]))
        T = min(_log(rng, 1, 32768), max(1, 58_000_000 // D))
        c.update(T=T, D=D, type=rng.choice(["bf16", "f16", "f32"]), gate=rng.choice(["none", "row", "full"]),
                 scale=rng.choice([1.0, 0.5, 1.25]), next=rng.random() < 0.7)
    return c


def _sizes(c):
    """Rows of each expert, largest first: a power law over the experts that have any; the same for every seed."""
    E = c["E"]
    live = max(1, E - c["empty"])
    weight = [(i + 1.0) ** -c["skew"] for i in range(live)]
    scale = c["rows"] / sum(weight)
    size = [int(w * scale) for w in weight]
    for i in range(c["rows"] - sum(size)):
        size[i % live] += 1
    return size + [0] * (E - live)


# ---------------------------------------------------------------------------------------------- inputs
def _exponent(amax, kind):
    """The smallest power of two 2^k, k >= -127, with amax <= 2^k times the format's largest value, as k + 127."""
    m, e = torch.frexp(amax)
    k = e - _TOP[kind] + (m > 0.875)
    return torch.where(amax > 0, k, torch.full_like(k, -127)).clamp(-127, 127).add(127).to(torch.uint8)


def _two_to(byte):
    """2^(byte - 127) in 32 bits."""
    return torch.where(byte > 0, byte.to(torch.int32) << 23, 1 << 22).view(torch.float32)


def _finite(x):
    return torch.where(x.abs() < math.inf, x, torch.zeros_like(x))


def _quant_rows_plain(x, kind):
    """[..., n] -> codes and the scale byte of each block of 128 along the last axis (not-finite values have no part in it)."""
    n = x.shape[-1]
    f = torch.nn.functional.pad(x.float(), (0, -n % BLOCK)).unflatten(-1, (-1, BLOCK))
    s = _exponent(_finite(f).abs().amax(-1), kind)
    v = f * _two_to(254 - s)[..., None]
    return v.flatten(-2)[..., :n].to(_F8[kind]), s


def _quant_weights_plain(w, kind):
    """[E, N, K] -> codes and the scale byte of each block of 128 x 128."""
    E, N, K = w.shape
    f = torch.nn.functional.pad(w.float(), (0, -K % BLOCK, 0, -N % BLOCK))
    f = f.unflatten(2, (-1, BLOCK)).unflatten(1, (-1, BLOCK))
    s = _exponent(_finite(f).abs().amax((2, 4)), kind)
    v = f * _two_to(254 - s)[:, :, None, :, None]
    return v.flatten(3, 4).flatten(1, 2)[:, :N, :K].to(_F8[kind]), s


def _padded_rows(codes):
    """The same codes with rows that start on 16-byte boundaries, as the framework's quantisation lays them out."""
    n = codes.shape[-1]
    wide = torch.zeros(*codes.shape[:-1], (n + 15) // 16 * 16, dtype=torch.uint8, device=codes.device)
    wide[..., :n] = codes.view(torch.uint8)
    return wide.view(codes.dtype)[..., :n]


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)
    dt = _DT[c["type"]]
    randn = lambda *s: torch.randn(*s, device="cuda", dtype=torch.float32, generator=gen)  # noqa: E731
    op = c["op"]
    st = {"case": c}
    if op == "quant_rows":
        # activations with a few loud channels
        loud = 1 + 15 * (torch.rand(c["n"], device="cuda", generator=gen) < 0.01)
        st["x"] = torch.empty(c["rows"], c["n"], dtype=dt, device="cuda")
        for r in range(0, c["rows"], 16384):
            st["x"][r:r + 16384] = randn(min(16384, c["rows"] - r), c["n"]).mul_(loud)
    elif op == "quant_weights":
        st["w"] = torch.empty(c["E"], c["N"], c["K"], dtype=dt, device="cuda")
        for e in range(c["E"]):
            st["w"][e] = randn(c["N"], c["K"]).mul_(c["K"] ** -0.5)
    elif op in ("mm8", "mm8_grad_x", "glu", "glu_grad"):
        size = _sizes(c)
        random.Random(int(seed)).shuffle(size)
        st["size"], st["cap"] = size, max(size)
        off = [0]
        for s in size:
            off.append(off[-1] + s)
        st["offsets"] = torch.tensor(off, dtype=torch.int32, device="cuda")
        E, K = c["E"], c["K"]
        if op in ("mm8", "mm8_grad_x"):
            # the weights that a program keeps: 8-bit codes and their scales, for grad_x the transposed codes
            N, grad = c["N"], op == "mm8_grad_x"
            st["x"] = randn(c["rows"], N if grad else K)
            if grad:
                st["x"] *= torch.exp2(2 * randn(c["rows"], 1))           # gradients: rows of very different size
            st["x"] = st["x"].clamp_(-6e4, 6e4).to(dt)
            codes, scales = [], []
            for e in range(E):
                q, s = _quant_weights_plain(randn(1, N, K).mul_(K ** -0.5).to(dt), "e4m3")
                codes.append(_padded_rows(q[0].view(torch.uint8).T.contiguous() if grad else q[0].view(torch.uint8)))
                scales.append(s[0])
            st["w"] = torch.empty(E, *codes[0].shape[:1], (codes[0].shape[1] + 15) // 16 * 16, dtype=torch.uint8,
                                  device="cuda")[..., :codes[0].shape[1]]
            for e in range(E):
                st["w"][e] = codes[e]
            st["w"] = st["w"].view(torch.float8_e4m3fn)
            st["ws"] = torch.stack(scales).transpose(1, 2) if grad else torch.stack(scales)
        else:
            I = c["I"]
            st["x"] = randn(c["rows"], K).to(dt)
            st["w"] = torch.empty(E, 2 * I, K, dtype=dt, device="cuda")
            for e in range(E):
                st["w"][e] = randn(2 * I, K).mul_(K ** -0.5)
            if op == "glu_grad":
                st["da"] = randn(c["rows"], I).to(dt)
    else:
        T, D = c["T"], c["D"]
        st["y"] = (randn(T, D) * torch.exp2(randn(T, 1))).to(dt)
        st["res"] = (randn(T, D) * 2).to(dt)
        st["gain"], st["next_gain"] = 1 + 0.1 * randn(D), 1 + 0.1 * randn(D) if c["next"] else None
        st["gate"] = {"none": lambda: None, "row": lambda: torch.sigmoid(randn(T)),
                      "full": lambda: torch.sigmoid(randn(T, D)).to(dt)}[c["gate"]]()
        if op == "norm_grad":
            st["h"] = _norm_plain(st)["h"]                       # kept from the forward pass
            st["dh"] = randn(T, D).to(dt)
            st["dn"] = randn(T, D).to(dt) if c["next"] else None
    return st


# ---------------------------------------------------------------------------------------------- plain forms
def _padded(t, st):
    """Rows in expert order -> [E, cap, D] in 32 bits, zero past each expert's rows."""
    off = st["offsets"].long()
    row = off[:-1, None] + torch.arange(st["cap"], device=t.device)
    inside = row < off[1:, None]
    got = t.float()[row.clamp_max(t.shape[0] - 1)]
    return torch.where(inside[..., None], got, torch.zeros_like(got))


def _unpadded(t, st, rows):
    off = st["offsets"].long()
    r = torch.arange(rows, device=t.device)
    e = torch.searchsorted(off[1:], r, right=True)
    return t[e, r - off[e]]


def _spread(scales, shape):
    """The factor of each element from the scale bytes of blocks of 128 along the last axis or the last two."""
    f = _two_to(scales).repeat_interleave(BLOCK, -1)[..., :shape[-1]]
    return f.repeat_interleave(BLOCK, -2)[..., :shape[-2], :] if scales.dim() == 3 else f


_BETA, _LINEAR = 4.0, 25.0


def _unit_plain(g, u, act):
    """(a, da/dg, da/du) of the gated unit."""
    s = 1.0 / (1.0 + torch.exp(-g))
    if act == "situ":
        tg, tu = torch.tanh(g / _BETA), torch.tanh(u / _LINEAR)
        f, h = _BETA * tg, _LINEAR * tu
        return s * f * h, h * (s * (1 - s) * f + s * (1 - tg * tg)), s * f * (1 - tu * tu)
    return g * s * u, u * (s + g * s * (1 - s)), g * s


def _gate_plain(st):
    gate = st["gate"]
    return None if gate is None else gate[:, None] if gate.dim() == 1 else gate.float()


def _norm_plain(st):
    c, dt = st["case"], _DT[st["case"]["type"]]
    y = st["y"].float()
    b = y * (1.0 / torch.sqrt((y * y).mean(1, keepdim=True) + EPS)) * st["gain"]
    gate = _gate_plain(st)
    h = c["scale"] * st["res"].float() + (b if gate is None else gate * b)
    out = {"h": h.to(dt)}
    if c["next"]:
        out["n"] = (h * (1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)) * st["next_gain"]).to(dt)
    return out


def _norm_grad_plain(st):
    c, dt = st["case"], _DT[st["case"]["type"]]
    y, t = st["y"].float(), st["dh"].float()
    out = {}
    if c["next"]:
        h, dn = st["h"].float(), st["dn"].float()
        r = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
        v = dn * st["next_gain"]
        out["dnext_gain"] = (dn * (h * r)).sum(0)
        t = t + r * (v - h * r * (v * (h * r)).mean(1, keepdim=True))
    out["dres"] = (c["scale"] * t).to(dt)
    r = 1.0 / torch.sqrt((y * y).mean(1, keepdim=True) + EPS)
    yh = y * r
    gate = _gate_plain(st)
    if gate is not None:
        dg = t * (yh * st["gain"])
        out["dgate"] = dg.sum(1) if st["gate"].dim() == 1 else dg.to(dt)
        t = t * gate
    out["dgain"] = (t * yh).sum(0)
    v = t * st["gain"]
    out["dy"] = (r * (v - yh * (v * yh).mean(1, keepdim=True))).to(dt)
    return out


def _plain(st):
    c = st["case"]
    op, dt = c["op"], _DT[c["type"]]
    if op == "quant_rows":
        q, s = _quant_rows_plain(st["x"], c["kind"])
        return {"codes": q, "scales": s}
    if op == "quant_weights":
        q, s = _quant_weights_plain(st["w"], c["kind"])
        out = {"codes": q, "scales": s}
        if c["transposed"]:
            out["codes_t"] = q.view(torch.uint8).transpose(1, 2).contiguous().view(_F8[c["kind"]])
        return out
    if op in ("mm8", "mm8_grad_x"):
        q, s = _quant_rows_plain(st["x"], c["kind"])
        x = _padded(q.float() * _spread(s, q.shape), st)
        w = st["w"].float() * _spread(st["ws"], st["w"].shape)
        return {"y": _unpadded(torch.bmm(x, w.transpose(1, 2)), st, c["rows"]).to(_DT[c["out"]])}
    if op in ("glu", "glu_grad"):
        x, w = _padded(st["x"], st), st["w"].float()
        g, u = torch.bmm(x, w.transpose(1, 2)).chunk(2, 2)
        a, dg, du = _unit_plain(g, u, c["act"])
        if op == "glu":
            return {"a": _unpadded(a, st, c["rows"]).to(dt)}
        da = _padded(st["da"], st)
        dgu = torch.cat([da * dg, da * du], 2)
        return {"dgu": _unpadded(dgu, st, c["rows"]).to(dt), "dx": _unpadded(torch.bmm(dgu, w), st, c["rows"]).to(dt),
                "dw": torch.bmm(dgu.transpose(1, 2), x).to(dt)}
    return _norm_plain(st) if op == "norm" else _norm_grad_plain(st)


# ---------------------------------------------------------------------------------------------- library calls
def _own(st):
    from latent_moe_layer_gb300 import experts as ex
    c = st["case"]
    op = c["op"]
    if op == "quant_rows":
        q, s = ex.quant8_rows(st["x"], kind=c["kind"])
        return {"codes": q, "scales": s}
    if op == "quant_weights":
        got = ex.quant8_weights(st["w"], kind=c["kind"], transposed=c["transposed"])
        return dict(zip(("codes", "scales", "codes_t"), got))
    if op in ("mm8", "mm8_grad_x"):
        q, s = ex.quant8_rows(st["x"], kind=c["kind"])
        return {"y": ex.group_mm8(q, s, st["w"], st["ws"], st["offsets"], out_dtype=_DT[c["out"]])}
    if op == "glu":
        return {"a": ex.group_glu(st["x"], st["w"], st["offsets"], act=c["act"])}
    if op == "glu_grad":
        dgu = ex.group_glu_grad(st["da"], st["x"], st["w"], st["offsets"], act=c["act"])
        return {"dgu": dgu, "dx": ex.group_mm_grad_x(dgu, st["w"], st["offsets"]),
                "dw": ex.group_mm_grad_w(dgu, st["x"], st["offsets"], out_dtype=_DT[c["type"]])}
    if op == "norm":
        h, n = ex.norm_residual(st["y"], st["res"], gain=st["gain"], gate=st["gate"], residual_scale=c["scale"],
                                next_gain=st["next_gain"], eps=EPS)
        return {"h": h, "n": n} if c["next"] else {"h": h}
    dy, dres, dgain, dgate, dnext = ex.norm_residual_grad(st["dh"], st["dn"], st["y"], st["h"], gain=st["gain"],
                                                          gate=st["gate"], residual_scale=c["scale"],
                                                          next_gain=st["next_gain"], eps=EPS)
    out = {"dy": dy, "dres": dres, "dgain": dgain}
    if dgate is not None:
        out["dgate"] = dgate
    if dnext is not None:
        out["dnext_gain"] = dnext
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------- work
def work(case):
    c, b = case, _SIZE[case["type"]]
    op = c["op"]
    up = lambda n: -(-n // BLOCK)  # noqa: E731
    if op == "quant_rows":
        n = c["rows"] * c["n"]
        return {"bytes": n * (b + 1) + c["rows"] * up(c["n"]), "flops": 2 * n}
    if op == "quant_weights":
        n = c["E"] * c["N"] * c["K"]
        return {"bytes": n * (b + 1 + c["transposed"]) + c["E"] * up(c["N"]) * up(c["K"]), "flops": 2 * n}
    if op in ("mm8", "mm8_grad_x", "glu", "glu_grad"):
        rows, K, offsets = c["rows"], c["K"], 4 * (c["E"] + 1)
        touched = sum(s > 0 for s in _sizes(c))
        if op in ("mm8", "mm8_grad_x"):
            N = c["N"]
            wide, narrow = (N, K) if op == "mm8_grad_x" else (K, N)
            return {"bytes": rows * (wide * b + narrow * _SIZE[c["out"]]) + touched * (K * N + up(K) * up(N)) + offsets,
                    "flops": 2 * rows * K * N}
        I = c["I"]
        if op == "glu":
            return {"bytes": rows * (K + I) * b + touched * 2 * I * K * b + offsets, "flops": 4 * rows * K * I + 8 * rows * I}
        # projections again, then the products for the rows and (all experts) for the weights
        return {"bytes": rows * (K + I + 2 * I + K) * b + (touched + c["E"]) * 2 * I * K * b + offsets,
                "flops": 12 * rows * K * I + 20 * rows * I}
    T, D = c["T"], c["D"]
    n, full, nxt = T * D, c["gate"] == "full", c["next"]
    if op == "norm":
        return {"bytes": n * b * (3 + full + nxt) + D * 4 * (1 + nxt), "flops": n * (7 + 4 * nxt)}
    return {"bytes": n * b * (4 + 2 * full + 2 * nxt) + D * 4 * 2 * (1 + nxt), "flops": n * (14 + 10 * nxt)}


# ---------------------------------------------------------------------------------------------- 64 bits
def _exact_codes(x, kind, rows_too):
    """Codes and scale bytes by counting: the scale is found by comparing, the code by the distance between the
    format's neighbours at the value's own power of two."""
    top = math.ldexp(0.875, _TOP[kind])
    mantissa, least = {"e4m3": (3, -6), "e5m2": (2, -14)}[kind]
    N, K = x.shape
    f = torch.zeros(-(-N // BLOCK) * BLOCK if rows_too else N, -(-K // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    f[:N, :K] = x.double()
    blocks = f.view(-1, BLOCK, f.shape[1] // BLOCK, BLOCK) if rows_too else f.view(N, 1, -1, BLOCK)
    amax = blocks.abs().amax((1, 3))
    k = torch.full(amax.shape, -127, dtype=torch.float64, device=x.device)
    k = torch.maximum(k, torch.log2((amax / top).clamp_min(1e-300)).floor() - 1)
    for _ in range(3):                                           # up until it fits
        k = torch.where(amax > top * torch.exp2(k), k + 1, k)
    wide = k.repeat_interleave(BLOCK, 1)[:, :K]
    if rows_too:
        wide = wide.repeat_interleave(BLOCK, 0)[:N]
    v = x.double() * torch.exp2(-wide)
    own_power = torch.log2(v.abs().clamp_min(2.0 ** least)).floor()
    own_power = torch.where(v.abs() >= torch.exp2(own_power + 1), own_power + 1, own_power)
    step = torch.exp2(own_power - mantissa)
    return torch.round(v / step) * step, k, wide                 # round: halves to even


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    op = c["op"]
    if op == "quant_rows":
        codes = torch.empty(c["rows"], c["n"], dtype=torch.float64, device="cuda")
        for r in range(0, c["rows"], 8192):
            codes[r:r + 8192] = _exact_codes(st["x"][r:r + 8192], c["kind"], False)[0]
        return {"codes": codes, "scales": None}
    if op == "quant_weights":
        codes = torch.stack([_exact_codes(w, c["kind"], True)[0] for w in st["w"]])
        out = {"codes": codes, "scales": None}
        if c["transposed"]:
            out["codes_t"] = codes.transpose(1, 2).contiguous()
        return out
    if op in ("mm8", "mm8_grad_x"):
        y = torch.zeros(c["rows"], st["w"].shape[1], dtype=torch.float64, device="cuda")
        r = 0
        for e, s in enumerate(st["size"]):
            if s:
                q, _, k = _exact_codes(st["x"][r:r + s], c["kind"], False)
                w, ws = st["w"][e].double(), st["ws"][e].double() - 127
                for j in range(ws.shape[1]):                     # block by block, as the definition has it
                    f = torch.exp2(ws[:, j]).repeat_interleave(BLOCK)[:w.shape[0]]
                    cols = slice(j * BLOCK, (j + 1) * BLOCK)
                    w[:, cols] *= f[:, None]
                y[r:r + s] = (q * torch.exp2(k)) @ w.T
            r += s
        return {"y": y}
    if op in ("glu", "glu_grad"):
        I, K = c["I"], c["K"]
        out = {"a": torch.zeros(c["rows"], I, dtype=torch.float64, device="cuda")}
        if op == "glu_grad":
            out = {"dgu": torch.zeros(c["rows"], 2 * I, dtype=torch.float64, device="cuda"),
                   "dx": torch.zeros(c["rows"], K, dtype=torch.float64, device="cuda"),
                   "dw": torch.zeros(c["E"], 2 * I, K, dtype=torch.float64, device="cuda")}
        r = 0
        for e, n in enumerate(st["size"]):
            if not n:
                continue
            x, w = st["x"][r:r + n].double(), st["w"][e].double()
            g, u = x @ w[:I].T, x @ w[I:].T
            s = torch.sigmoid(g)
            if c["act"] == "situ":
                f, df = _BETA * torch.tanh(g / _BETA), torch.cosh(g / _BETA).pow(-2)
                h, dh = _LINEAR * torch.tanh(u / _LINEAR), torch.cosh(u / _LINEAR).pow(-2)
            else:
                f, df, h, dh = g, torch.ones_like(g), u, torch.ones_like(u)
            if op == "glu":
                out["a"][r:r + n] = s * f * h
            else:
                da = st["da"][r:r + n].double()
                dgu = torch.cat([da * h * (s * torch.sigmoid(-g) * f + s * df), da * s * f * dh], 1)
                out["dgu"][r:r + n] = dgu
                out["dx"][r:r + n] = dgu @ w
                out["dw"][e] = dgu.T @ x
            r += n
        return out
    # the norms, a slice of the rows at a time; gradients by the chain rule through the row's own mean square
    T, D, scale = c["T"], c["D"], c["scale"]
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")  # noqa: E731
    gain = st["gain"].double()
    next_gain = st["next_gain"].double() if c["next"] else None
    if op == "norm":
        out = {"h": z(T, D), "n": z(T, D)} if c["next"] else {"h": z(T, D)}
    else:
        out = {"dy": z(T, D), "dres": z(T, D), "dgain": z(D)}
        if c["gate"] != "none":
            out["dgate"] = z(T) if c["gate"] == "row" else z(T, D)
        if c["next"]:
            out["dnext_gain"] = z(D)
    for r in range(0, T, 4096):
        sl = slice(r, min(r + 4096, T))
        y = st["y"][sl].double()
        ms = torch.linalg.vecdot(y, y)[:, None] / D + EPS
        gate = 1.0 if st["gate"] is None else st["gate"][sl].double()
        if c["gate"] == "row":
            gate = gate[:, None]
        if op == "norm":
            h = scale * st["res"][sl].double() + gate * (gain * y / ms.sqrt())
            out["h"][sl] = h
            if c["next"]:
                out["n"][sl] = next_gain * h / (torch.linalg.vecdot(h, h)[:, None] / D + EPS).sqrt()
            continue
        t = st["dh"][sl].double()
        if c["next"]:
            h, dn = st["h"][sl].double(), st["dn"][sl].double()
            hs = torch.linalg.vecdot(h, h)[:, None] / D + EPS
            out["dnext_gain"] += (dn * h / hs.sqrt()).sum(0)
            d_ms = torch.linalg.vecdot(dn * next_gain, h)[:, None] * -0.5 * hs ** -1.5
            t = t + dn * next_gain / hs.sqrt() + d_ms * 2 * h / D
        out["dres"][sl] = scale * t
        if c["gate"] != "none":
            dg = t * gain * y / ms.sqrt()
            out["dgate"][sl] = dg.sum(1) if c["gate"] == "row" else dg
        t = t * gate
        out["dgain"] += (t * y / ms.sqrt()).sum(0)
        d_ms = torch.linalg.vecdot(t * gain, y)[:, None] * -0.5 * ms ** -1.5
        out["dy"][sl] = t * gain / ms.sqrt() + d_ms * 2 * y / D
    return out
