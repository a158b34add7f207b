"""Measured cases of the expert training operators: row dispatch and combine, matrix products grouped by
expert, the gated linear unit with dropout, and dropout with a residual.

Each case is run through `run` either in its plain form (elementary torch operations in 32 bits, rounded
once at the end) or, where `own` is set, through the library's entry points.  `exact` gives the same
outputs from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 16 tokens over all 896 experts: the plan and the copies are pure latency
        {"name": "dispatch_decode", "op": "dispatch", "T": 16, "K": 16, "E": 896, "first": 0, "total": 896, "D": 3584,
         "type": "bf16", "skew": 0.0},
        # a training micro-batch of 8192 tokens with all experts local: 131,072 rows of the latent width
        {"name": "dispatch_train", "op": "dispatch", "T": 8192, "K": 16, "E": 896, "first": 0, "total": 896, "D": 3584,
         "type": "bf16", "skew": 0.0},
        # the weighted sum on one of two expert-parallel ranks: about half the pairs live elsewhere
        {"name": "combine_half", "op": "combine", "T": 4099, "K": 16, "E": 448, "first": 448, "total": 896, "D": 3584,
         "type": "f16", "skew": 0.5},
        # its gradient for the rows and for the mixture weights, with all experts local
        {"name": "combine_grad_train", "op": "combine_grad", "T": 4096, "K": 16, "E": 896, "first": 0, "total": 896,
         "D": 3584, "type": "bf16", "skew": 0.0},
        # one of eight ranks at a decode batch: two rows an expert, bound by reading the touched weights
        {"name": "mm_decode", "op": "mm", "E": 112, "rows": 251, "K": 3584, "N": 6144, "type": "bf16", "skew": 0.3,
         "empty": 11},
        # gate and up projections of a training micro-batch on one of eight ranks
        {"name": "mm_train", "op": "mm", "E": 112, "rows": 65536, "K": 3584, "N": 6144, "type": "bf16", "skew": 0.4,
         "empty": 0},
        # gradient of the down projection's input on one of 64 ranks, odd ragged groups
        {"name": "mm_grad_x_rank", "op": "mm_grad_x", "E": 14, "rows": 2047, "K": 3072, "N": 3584, "type": "f16",
         "skew": 0.6, "empty": 1},
        # weight gradient of the down projection in fp32 on one of 16 ranks, some experts without tokens
        {"name": "mm_grad_w_rank", "op": "mm_grad_w", "E": 56, "rows": 16381, "K": 3072, "N": 3584, "type": "bf16",
         "skew": 0.5, "empty": 3},
        # gated unit of a micro-batch's expert rows, SiLU, 10 % dropout
        {"name": "glu_train", "op": "glu", "rows": 32768, "I": 3072, "type": "bf16", "act": "silu", "p": 0.1},
        # gradient of the soft-limited unit on few ragged rows
        {"name": "glu_grad_situ", "op": "glu_grad", "rows": 5003, "I": 3072, "type": "f16", "act": "situ", "p": 0.25},
        # the layer output of a decode-size batch with its residual: latency
        {"name": "dropout_small", "op": "dropout", "n": 16 * 7168 - 3, "type": "bf16", "residual": True, "p": 0.1},
        # the layer output of a micro-batch with its residual
        {"name": "dropout_train", "op": "dropout", "n": 8192 * 7168, "type": "f32", "residual": True, "p": 0.1},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "combine_grad", "mm", "mm", "mm_grad_x", "mm_grad_w", "glu", "glu_grad",
                     "dropout"])
    c = {"op": op, "type": rng.choice(["bf16", "f16"])}
    if op in ("dispatch", "combine", "combine_grad"):
        total = _log(rng, 8, 896)
        share = rng.choice([1, 1, 2, 4])
        E = max(1, total // share)
        T = _log(rng, 1, 8192)
        D = _log(rng, 64, 7168, 8)
        K = rng.randint(1, min(16, total))
        while T * K * D > 400_000_000:
            T = max(1, T // 2)
        c.update(T=T, K=K, E=E, first=E * rng.randrange(share) if share > 1 else 0, total=total, D=D,
                 skew=rng.choice([0.0, 0.5, 1.0]))
    elif op in ("mm", "mm_grad_x", "mm_grad_w"):
        E = _log(rng, 1, 112)
        K, N = _log(rng, 64, 6144, 8), _log(rng, 64, 6144, 8)
        while E * K * N > 400_000_000:
            E = max(1, E // 2)
        rows = _log(rng, 1, 32768)
        while rows * K * N > 500_000_000_000:
            rows = max(1, rows // 2)
        c.update(E=E, rows=rows, K=K, N=N, skew=rng.choice([0.0, 0.4, 0.8]), empty=rng.choice([0, E // 8, E // 3]))
    elif op in ("glu", "glu_grad"):
        I = _log(rng, 32, 6144, 8)
        rows = _log(rng, 1, 32768)
        while rows * I > 100_000_000:
            rows = max(1, rows // 2)
        c.update(rows=rows, I=I, act=rng.choice(["silu", "situ"]), p=rng.choice([0.0, 0.1, 0.3, 0.5]))
    else:
        c.update(n=_log(rng, 1, 50_000_000), type=rng.choice(["bf16", "f16", "f32"]), residual=rng.random() < 0.5,
                 p=rng.choice([0.05, 0.1, 0.3, 0.5]))
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
def _routing(c, gen):
    """Top-K experts of each token from perturbed log loads, the share of them on this rank as rows."""
    load = torch.arange(1, c["total"] + 1, device="cuda", dtype=torch.float32).pow(-c["skew"]).log()
    noise = -torch.log(-torch.log(torch.rand(c["T"], c["total"], device="cuda", generator=gen).clamp(1e-7, 1 - 1e-6)))
    perm = torch.randperm(c["total"], device="cuda", generator=gen)
    idx = (load[perm] + noise).topk(c["K"], dim=1).indices.to(torch.int32).contiguous()
    return idx


def _plan_plain(idx, E, first):
    flat = idx.reshape(-1).long() - first
    local = (flat >= 0) & (flat < E)
    key = torch.where(local, flat, torch.full_like(flat, E))
    order = torch.argsort(key, stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=order.device)
    pos = torch.where(local, row, torch.full_like(row, -1)).to(torch.int32).reshape(idx.shape)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=idx.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([counts.new_zeros(1), counts[:E].cumsum(0)]).to(torch.int32)
    return offsets, pos


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)
    dt = _DT[c["type"]]
    randn = lambda *s: torch.randn(*s, device="cuda", dtype=torch.float32, generator=gen)  # noqa: E731
    op = c["op"]
    st = {"case": c}
    if op in ("dispatch", "combine", "combine_grad"):
        idx = _routing(c, gen)
        st["idx"] = idx
        if op == "dispatch":
            st["x"] = randn(c["T"], c["D"]).to(dt)
        else:
            st["pos"] = _plan_plain(idx, c["E"], c["first"])[1]
            st["y"] = randn(c["T"] * c["K"], c["D"]).to(dt)
            w = torch.rand(c["T"], c["K"], device="cuda", generator=gen) + 0.01
            st["w"] = w / w.sum(1, keepdim=True)
            if op == "combine_grad":
                st["dz"] = randn(c["T"], c["D"]).to(dt)
        if op != "combine":
            # the rank's receive buffer: room for every pair (and a spare row); rows that no pair takes stay zero
            st["buffer"] = torch.zeros(c["T"] * c["K"] + 1, c["D"], dtype=dt, device="cuda")
    elif op in ("mm", "mm_grad_x", "mm_grad_w"):
        size = _sizes(c)
        random.Random(int(seed)).shuffle(size)
        st["size"], st["cap"] = size, max(size)
        off = [0]
        for s in size:
            off.append(off[-1] + s)
        st["offsets"] = torch.tensor(off, dtype=torch.int32, device="cuda")
        if op in ("mm", "mm_grad_w"):
            st["x"] = randn(c["rows"], c["K"]).to(dt)
        if op in ("mm_grad_x", "mm_grad_w"):
            st["dy"] = randn(c["rows"], c["N"]).to(dt)
        if op in ("mm", "mm_grad_x"):
            w = torch.empty(c["E"], c["N"], c["K"], dtype=dt, device="cuda")
            for e in range(c["E"]):
                w[e] = randn(c["N"], c["K"]).mul_(c["K"] ** -0.5)
            st["w"] = w
    elif op in ("glu", "glu_grad"):
        st["gu"] = randn(c["rows"], 2 * c["I"]).to(dt)
        if op == "glu_grad":
            st["da"] = randn(c["rows"], c["I"]).to(dt)
    else:
        st["x"] = randn(c["n"]).to(dt)
        st["res"] = randn(c["n"]).to(dt) if c["residual"] else None
    # the random number stream of this step: a run's seed and a call number
    st["seed"], st["offset"] = 0x9E3779B97F4A7C15 ^ int(seed), (1 << 33) + 5
    return st


# ---------------------------------------------------------------------------------------------- plain forms
_M32 = 0xFFFFFFFF


def _keep_plain(n, p, seed, offset, device):
    """Kept elements 0 .. n - 1: Philox4x32-10 (Salmon, Moraes, Dror and Shaw 2011), counter (element / 4, offset),
    key seed, word element % 4, kept where the word is at least p 2^32."""
    b = torch.arange((n + 3) // 4, device=device, dtype=torch.int64)
    x0, x1 = b & _M32, b >> 32
    x2, x3 = torch.full_like(b, offset & _M32), torch.full_like(b, offset >> 32)
    k0, k1 = seed & _M32, seed >> 32
    for _ in range(10):
        a, d = x0 * 0xD2511F53, x2 * 0xCD9E8D57                  # 64-bit products, wrapped: all their bits
        x0, x1, x2, x3 = ((d >> 32) & _M32) ^ x1 ^ k0, d & _M32, ((a >> 32) & _M32) ^ x3 ^ k1, a & _M32
        k0, k1 = (k0 + 0x9E3779B9) & _M32, (k1 + 0xBB67AE85) & _M32
    return torch.stack([x0, x1, x2, x3], 1).reshape(-1)[:n] >= int(p * 4294967296.0)


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


_BETA, _LINEAR = 4.0, 25.0


def _plain(st):
    c = st["case"]
    op, dt = c["op"], _DT[c["type"]]
    if op == "dispatch":
        offsets, pos = _plan_plain(st["idx"], c["E"], c["first"])
        flat, n = pos.reshape(-1).long(), c["T"] * c["K"]
        st["buffer"][torch.where(flat >= 0, flat, torch.full_like(flat, n))] = st["x"].repeat_interleave(c["K"], 0)
        return {"offsets": offsets, "pos": pos, "rows": st["buffer"][:n]}
    if op == "combine":
        pos = st["pos"].long()
        w = torch.where(pos >= 0, st["w"], torch.zeros_like(st["w"]))
        return {"z": (st["y"].float()[pos.clamp_min(0)] * w[..., None]).sum(1).to(dt)}
    if op == "combine_grad":
        pos, n = st["pos"].long(), st["y"].shape[0]
        dz, flat = st["dz"].float(), pos.reshape(-1)
        st["buffer"][torch.where(flat >= 0, flat, torch.full_like(flat, n))] = \
            (dz[:, None] * st["w"][..., None]).reshape(-1, c["D"]).to(dt)
        dw = (st["y"].float()[pos.clamp_min(0)] * dz[:, None]).sum(2)
        return {"dy": st["buffer"][:n], "dw": torch.where(pos >= 0, dw, torch.zeros_like(dw))}
    if op == "mm":
        y = torch.bmm(_padded(st["x"], st), st["w"].float().transpose(1, 2))
        return {"y": _unpadded(y, st, c["rows"]).to(dt)}
    if op == "mm_grad_x":
        return {"dx": _unpadded(torch.bmm(_padded(st["dy"], st), st["w"].float()), st, c["rows"]).to(dt)}
    if op == "mm_grad_w":
        return {"dw": torch.bmm(_padded(st["dy"], st).transpose(1, 2), _padded(st["x"], st))}
    if op in ("glu", "glu_grad"):
        g, u = st["gu"].float().chunk(2, 1)
        s = 1.0 / (1.0 + torch.exp(-g))
        if c["act"] == "situ":
            tg, tu = torch.tanh(g / _BETA), torch.tanh(u / _LINEAR)
            a = s * (_BETA * tg) * (_LINEAR * tu)
        else:
            a = g * s * u
        keep = _keep_plain(g.numel(), c["p"], st["seed"], st["offset"], g.device).reshape(g.shape)
        scale = 1.0 / (1.0 - c["p"])
        if op == "glu":
            return {"a": torch.where(keep, a * scale, torch.zeros_like(a)).to(dt)}
        da = torch.where(keep, st["da"].float() * scale, torch.zeros_like(a))
        if c["act"] == "situ":
            dg = da * (_LINEAR * tu) * (s * (1 - s) * (_BETA * tg) + s * (1 - tg * tg))
            du = da * s * (_BETA * tg) * (1 - tu * tu)
        else:
            dg, du = da * u * (s + g * s * (1 - s)), da * g * s
        return {"dgu": torch.cat([dg, du], 1).to(dt)}
    x = st["x"].float()
    keep = _keep_plain(x.numel(), c["p"], st["seed"], st["offset"], x.device)
    out = torch.where(keep, x * (1.0 / (1.0 - c["p"])), torch.zeros_like(x))
    if st["res"] is not None:
        out = out + st["res"].float()
    return {"out": out.to(dt)}


# ---------------------------------------------------------------------------------------------- library calls
def _own(st):
    from latent_moe_layer_gb300 import experts as ex
    c = st["case"]
    op = c["op"]
    if op == "dispatch":
        offsets, pos = ex.plan_rows(st["idx"], c["E"], first_expert=c["first"])
        return {"offsets": offsets, "pos": pos, "rows": ex.gather_rows(st["x"], pos, out=st["buffer"][:pos.numel()])}
    if op == "combine":
        return {"z": ex.combine_rows(st["y"], st["pos"], st["w"])}
    if op == "combine_grad":
        dy, dw = ex.combine_rows_grad(st["dz"], st["y"], st["pos"], st["w"], out=st["buffer"][:st["y"].shape[0]])
        return {"dy": dy, "dw": dw}
    if op == "mm":
        return {"y": ex.group_mm(st["x"], st["w"], st["offsets"])}
    if op == "mm_grad_x":
        return {"dx": ex.group_mm_grad_x(st["dy"], st["w"], st["offsets"])}
    if op == "mm_grad_w":
        return {"dw": ex.group_mm_grad_w(st["dy"], st["x"], st["offsets"])}
    if op == "glu":
        return {"a": ex.glu_dropout(st["gu"], p=c["p"], seed=st["seed"], offset=st["offset"], act=c["act"])}
    if op == "glu_grad":
        return {"dgu": ex.glu_dropout_grad(st["da"], st["gu"], p=c["p"], seed=st["seed"], offset=st["offset"],
                                           act=c["act"])}
    return {"out": ex.dropout(st["x"], p=c["p"], seed=st["seed"], offset=st["offset"], residual=st["res"])}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------- work
def work(case):
    c, b = case, _SIZE[case["type"]]
    op = c["op"]
    if op in ("dispatch", "combine", "combine_grad"):
        pairs = c["T"] * c["K"] * min(1.0, c["E"] / c["total"])      # of them on this rank
        tok, row, table = c["T"] * c["D"] * b, pairs * c["D"] * b, c["T"] * c["K"] * 4
        if op == "dispatch":
            return {"bytes": tok + row + 2 * table + 4 * (c["E"] + 1), "flops": 0}
        if op == "combine":
            return {"bytes": tok + row + 2 * table, "flops": 2 * pairs * c["D"]}
        return {"bytes": tok + 2 * row + 3 * table, "flops": 3 * pairs * c["D"]}
    if op in ("mm", "mm_grad_x", "mm_grad_w"):
        touched = sum(s > 0 for s in _sizes(c))
        act = c["rows"] * (c["K"] + c["N"]) * b
        weight = c["E"] * c["K"] * c["N"] * 4 if op == "mm_grad_w" else touched * c["K"] * c["N"] * b
        return {"bytes": act + weight + 4 * (c["E"] + 1), "flops": 2 * c["rows"] * c["K"] * c["N"]}
    if op in ("glu", "glu_grad"):
        n = c["rows"] * c["I"]
        return {"bytes": n * b * (3 if op == "glu" else 5), "flops": n * (8 if op == "glu" else 20)}
    return {"bytes": c["n"] * b * (3 if c["residual"] else 2), "flops": 2 * c["n"]}


# ---------------------------------------------------------------------------------------------- 64 bits
def _keep_exact(n, p, seed, offset):
    """The same generator from 16-bit partial products, counters in slices."""
    def wide(x, m):                                  # high and low word of a 32 x 32-bit product
        xl, xh, ml, mh = x & 0xFFFF, x >> 16, m & 0xFFFF, m >> 16
        low = xl * ml
        mid = xh * ml + (low >> 16)
        mid2 = xl * mh + (mid & 0xFFFF)
        return xh * mh + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | (low & 0xFFFF)
    keep = torch.empty((n + 3) // 4, 4, dtype=torch.bool, device="cuda")
    for first in range(0, keep.shape[0], 1 << 23):
        i = torch.arange(first, min(first + (1 << 23), keep.shape[0]), device="cuda")
        v = [i % (1 << 32), i // (1 << 32), torch.full_like(i, offset % (1 << 32)), torch.full_like(i, offset // (1 << 32))]
        key = [seed % (1 << 32), seed // (1 << 32)]
        for _ in range(10):
            h0, l0 = wide(v[0], 0xD2511F53)
            h1, l1 = wide(v[2], 0xCD9E8D57)
            v = [h1 ^ v[1] ^ key[0], l1, h0 ^ v[3] ^ key[1], l0]
            key = [(key[0] + 0x9E3779B9) % (1 << 32), (key[1] + 0xBB67AE85) % (1 << 32)]
        for j in range(4):
            keep[first:first + i.numel(), j] = v[j] >= math.floor(p * 2 ** 32)
    return keep.reshape(-1)[:n]


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    op = c["op"]
    if op == "dispatch":
        own_rows = (st["idx"] >= c["first"]) & (st["idx"] < c["first"] + c["E"])
        t, k = own_rows.nonzero(as_tuple=True)                       # pairs in (token, slot) order
        e = st["idx"][t, k]
        order = torch.sort(e, stable=True).indices
        rows = torch.zeros(c["T"] * c["K"], c["D"], dtype=torch.float64, device="cuda")
        rows[:order.numel()] = st["x"].double()[t[order]]
        return {"offsets": None, "pos": None, "rows": rows}
    if op in ("combine", "combine_grad"):
        pos, w = st["pos"].long(), st["w"].double()
        out = {"z": torch.zeros(c["T"], c["D"], dtype=torch.float64, device="cuda")}
        if op == "combine_grad":
            out = {"dy": torch.zeros(st["y"].shape[0], c["D"], dtype=torch.float64, device="cuda"),
                   "dw": torch.zeros_like(w)}
        for k in range(c["K"]):
            t = (pos[:, k] >= 0).nonzero()[:, 0]
            r = pos[t, k]
            if op == "combine":
                out["z"][t] += w[t, k, None] * st["y"][r].double()
            else:
                out["dy"][r] = w[t, k, None] * st["dz"][t].double()
                out["dw"][t, k] = torch.linalg.vecdot(st["y"][r].double(), st["dz"][t].double())
        return out
    if op in ("mm", "mm_grad_x", "mm_grad_w"):
        shape, name = {"mm": ((c["rows"], c["N"]), "y"), "mm_grad_x": ((c["rows"], c["K"]), "dx"),
                       "mm_grad_w": ((c["E"], c["N"], c["K"]), "dw")}[op]
        out = torch.zeros(shape, dtype=torch.float64, device="cuda")
        r = 0
        for e, s in enumerate(st["size"]):
            if s == 0:
                continue
            if op == "mm":
                out[r:r + s] = st["x"][r:r + s].double() @ st["w"][e].double().T
            elif op == "mm_grad_x":
                out[r:r + s] = st["dy"][r:r + s].double() @ st["w"][e].double()
            else:
                out[e] = st["dy"][r:r + s].double().T @ st["x"][r:r + s].double()
            r += s
        return {name: out}
    if op in ("glu", "glu_grad"):
        I = c["I"]
        g, u = st["gu"][:, :I].double(), st["gu"][:, I:].double()
        keep = _keep_exact(g.numel(), c["p"], st["seed"], st["offset"]).view_as(g).double() / (1 - c["p"])
        s = torch.sigmoid(g)
        if c["act"] == "situ":
            f, df = _BETA * torch.tanh(g / _BETA), torch.cosh(g / _BETA).pow(-2)
            h, dh = _LINEAR * torch.tanh(u / _LINEAR), torch.cosh(u / _LINEAR).pow(-2)
        else:
            f, df, h, dh = g, torch.ones_like(g), u, torch.ones_like(u)
        if op == "glu":
            return {"a": s * f * h * keep}
        da = st["da"].double() * keep
        return {"dgu": torch.cat([da * h * (s * (1 - s) * f + s * df), da * s * f * dh], 1)}
    keep = _keep_exact(c["n"], c["p"], st["seed"], st["offset"]).double() / (1 - c["p"])
    out = st["x"].double() * keep
    return {"out": out if st["res"] is None else out + st["res"].double()}
