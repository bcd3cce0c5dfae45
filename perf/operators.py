"""The expert layer's operators: routing with the grouping of pairs by expert, products grouped by expert, the gated activation, the
routing-weighted combine, and products with 4-bit weights.

Each case is one pass through one operator in the form that serving or training uses; `run` computes it in elementary torch operations in
32 bits, or, where `own` is true, through the library's entry points.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}


def listed():
    return [
        # decode of one token of a 128-expert layer: logits to ids, weights and the pairs' order; latency alone counts
        {"name": "route one token", "op": "route", "T": 1, "E": 128, "k": 8, "dtype": "f32", "renorm": True, "grad": False, "pad": 0},
        # a training batch of the same layer, with the gradient of its logits
        {"name": "route training", "op": "route", "T": 16384, "E": 128, "k": 8, "dtype": "f32", "renorm": True, "grad": True, "pad": 0},
        # SiLU * up of a decode batch of 67 rows (ragged)
        {"name": "activation decode", "op": "act", "R": 67, "F": 768, "dtype": "f16", "grad": False},
        # the same of a training batch, with its gradient
        {"name": "activation training", "op": "act", "R": 24576, "F": 1408, "dtype": "bf16", "grad": True},
        # decode of 32 tokens: the experts' rows back to the tokens
        {"name": "combine decode", "op": "combine", "T": 32, "k": 8, "D": 2048, "dtype": "f16", "out": "f32", "grad": False, "pad": 0},
        # a training batch, gradients of the rows and of the routing weights
        {"name": "combine training", "op": "combine", "T": 8192, "k": 6, "D": 2048, "dtype": "bf16", "out": "bf16", "grad": True, "pad": 5},
        # decode of one token: gate/up of its 8 experts with the activation, reading 50 MB of weights
        {"name": "experts one token", "op": "experts", "T": 1, "k": 8, "E": 128, "N": 768, "K": 2048, "dtype": "f16", "out": "f16",
         "gather": True, "act": True, "grad": False, "zipf": 0.0, "pad": 0},
        # a decode batch whose experts repeat (Zipf popularity)
        {"name": "experts decode", "op": "experts", "T": 32, "k": 8, "E": 128, "N": 768, "K": 2048, "dtype": "bf16", "out": "bf16",
         "gather": True, "act": True, "grad": False, "zipf": 1.1, "pad": 0},
        # a prefill chunk of a 64-expert layer, ragged counts
        {"name": "experts prefill", "op": "experts", "T": 4096, "k": 6, "E": 64, "N": 1408, "K": 2048, "dtype": "bf16", "out": "bf16",
         "gather": True, "act": True, "grad": False, "zipf": 1.0, "pad": 0},
        # a training step of an 8-expert layer's down projection: rows, their gradient and the weights' gradient in 32 bits
        {"name": "experts training", "op": "experts", "T": 4096, "k": 2, "E": 8, "N": 4096, "K": 14336, "dtype": "bf16", "out": "bf16",
         "gather": False, "act": False, "grad": True, "zipf": 0.0, "pad": 0},
        # one token through a dense 4-bit projection (attention output, shared expert)
        {"name": "w4 one token", "op": "w4", "T": 1, "k": 1, "E": 1, "N": 4096, "K": 2048, "G": 128, "dtype": "f16", "out": "f16",
         "act": False, "zipf": 0.0, "pad": 0},
        # a decode batch through 4-bit experts, gate/up with the activation
        {"name": "w4 experts decode", "op": "w4", "T": 32, "k": 8, "E": 128, "N": 768, "K": 2048, "G": 64, "dtype": "bf16", "out": "bf16",
         "act": True, "zipf": 1.1, "pad": 0},
    ]


def _log(rng, lo, hi, step=1):
    """A whole multiple of `step` from lo to hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["route", "act", "combine", "experts", "experts", "experts", "w4", "w4"])
    if op == "route":
        E = _log(rng, 4, 512)
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(E, 10)), "dtype": rng.choice(["f32", "bf16", "f16"]),
                "renorm": rng.random() < 0.5, "grad": rng.random() < 0.5, "pad": rng.choice([0, 0, 3])}
    if op == "act":
        return {"op": op, "R": _log(rng, 1, 24576), "F": _log(rng, 8, 1408, rng.choice([1, 8, 8])), "dtype": rng.choice(["bf16", "f16"]),
                "grad": rng.random() < 0.5}
    if op == "combine":
        dtype = rng.choice(["bf16", "f16"])
        return {"op": op, "T": _log(rng, 1, 6144), "k": rng.randint(1, 8), "D": _log(rng, 64, 2048, rng.choice([1, 8, 8])), "dtype": dtype,
                "out": rng.choice([dtype, "f32"]), "grad": rng.random() < 0.5, "pad": rng.choice([0, 0, 9])}
    dtype = rng.choice(["bf16", "f16"])
    E = rng.choice([1, 3, 8, 16, 64, 128])
    k = rng.randint(1, min(E, 8))
    case = {"op": op, "T": _log(rng, 1, 4096 if op == "experts" else 256), "k": k, "E": E}
    if op == "experts":
        # at most as many weights and products as the largest listed case
        case["N"] = _log(rng, 64, 4096, rng.choice([1, 8, 16, 64]))
        case["K"] = _log(rng, 64, 4096, rng.choice([1, 8, 32, 64, 64]))
        act = rng.random() < 0.4
        return {**case, "dtype": dtype, "out": rng.choice([dtype, dtype, "f32"]), "gather": rng.random() < 0.5, "act": act,
                "grad": not act and rng.random() < 0.5, "zipf": rng.choice([0.0, 0.7, 1.1]), "pad": rng.choice([0, 0, 5])}
    G = rng.choice([32, 64, 128])
    if rng.random() < 0.5:
        case["E"] = case["k"] = 1  # one dense projection
    case["N"] = _log(rng, 48, 8192 if case["E"] <= 16 else 2048, rng.choice([1, 8, 16]))
    case["K"] = _log(rng, 256, 4096, 128)
    return {**case, "G": G, "dtype": dtype, "out": rng.choice([dtype, "f32"]), "act": rng.random() < 0.5,
            "zipf": rng.choice([0.0, 1.1]), "pad": rng.choice([0, 0, 2])}


def _ids(gen, T, k, E, zipf, pad):
    """k different experts a token, popularity falling as rank^-zipf (Gumbel keys); the last `pad` tokens are padding, with ids of -1."""
    keys = -torch.log(-torch.log(torch.rand(T, E, generator=gen, device="cuda").clamp_(1e-9, 1 - 1e-7)))
    rank = torch.randperm(E, generator=gen, device="cuda") + 1
    ids = torch.topk(keys - zipf * rank.float().log(), k, dim=1).indices.int()
    if pad:
        ids[max(1, T - pad):] = -1
    return ids


def _grouped(ids, E):
    """(bounds, order, slot, counts) of the pairs sorted by expert, earlier pairs first; pairs without an expert come last, with order and slot -1."""
    flat = ids.reshape(-1).long()
    good = (flat >= 0) & (flat < E)
    key = torch.where(good, flat, E)
    order = torch.sort(key, stable=True).indices
    bounds = (key[order][:, None] < torch.arange(E + 1, device=ids.device)[None, :]).sum(0)
    n = bounds[E]
    at = torch.arange(flat.numel(), device=ids.device)
    slot = torch.empty_like(order)
    slot[order] = at
    return (bounds.int(), torch.where(at < n, order, -1).int(), torch.where(good, slot, -1).int().reshape(ids.shape))


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(int(seed) * 7919 + 13)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype).mul_(scale)

    s = dict(case)
    op = case["op"]
    dt = DTYPES[case["dtype"]]
    i32 = {"dtype": torch.int32, "device": "cuda"}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        logits = normal(T, E, scale=2.0)
        if E > 2 * k:  # a masked expert, as a retired or unavailable one is
            logits[:, E // 2] = -math.inf
        if case["pad"]:  # padding tokens: every expert masked
            logits[max(1, T - case["pad"]):] = -math.inf
        s["logits"] = logits.to(dt)
        s["dg"] = normal(T, k)
        s["ids"], s["g"] = torch.empty(T, k, **i32), torch.empty(T, k, device="cuda")
        s["bounds"], s["order"], s["slot"] = torch.empty(E + 1, **i32), torch.empty(T * k, **i32), torch.empty(T, k, **i32)
        s["dlogits"] = torch.empty_like(s["logits"])
        return s
    if op == "act":
        R, F = case["R"], case["F"]
        s["a"], s["dh"] = normal(R, 2 * F).to(dt), normal(R, F).to(dt)
        s["h"], s["da"] = torch.empty_like(s["dh"]), torch.empty_like(s["a"])
        return s
    if op == "combine":
        T, k, D = case["T"], case["k"], case["D"]
        ids = _ids(gen, T, k, max(16, k), 0.0, case["pad"])
        _, _, s["slot"] = _grouped(ids, max(16, k))
        s["y"] = normal(T * k, D).to(dt)
        s["g"] = torch.softmax(normal(T, k), 1)
        s["dout"] = normal(T, D).to(DTYPES[case["out"]])
        s["out"] = torch.empty(T, D, device="cuda", dtype=DTYPES[case["out"]])
        s["dy"], s["dg"] = torch.zeros_like(s["y"]), torch.empty(T, k, device="cuda")
        s["out_dtype"] = DTYPES[case["out"]]
        return s
    T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
    ids = _ids(gen, T, k, E, case["zipf"], case["pad"])
    s["bounds"], s["order"], _ = _grouped(ids, E)
    s["counts"] = (s["bounds"][1:] - s["bounds"][:-1]).tolist()
    rows = 2 * N if case["act"] else N
    out = DTYPES[case["out"]]
    gathered = op == "w4" or case["gather"]
    x = normal(T if gathered else T * k, K)
    x[:, :: max(1, K // 8)] *= 8.0  # outlier channels
    s["x"] = x.to(dt)
    s["y"] = torch.zeros(T * k, N, device="cuda", dtype=out)
    if op == "experts":
        s["w"] = normal(E, rows, K, scale=K ** -0.5, dtype=dt)
        if case["grad"]:
            s["dy"] = normal(T * k, N, dtype=dt)
            s["dx"] = torch.zeros(T * k, K, device="cuda", dtype=dt)
            s["dw"] = torch.empty(E, N, K, device="cuda", dtype=torch.float32)
        return s
    G = case["G"]
    s["codes"] = torch.randint(0, 256, (E, rows, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    step = (torch.rand(E, rows, K // G, generator=gen, device="cuda") + 0.5) * (0.2 * K ** -0.5)
    s["scales"] = step.half()
    s["mins"] = (step * (-7.5 + normal(E, rows, K // G, scale=0.5))).half()
    return s


def run(s):
    op = s["op"]
    if own:
        from spectral_expert_gemv_amd import bitsmoe as bm
        if op == "route":
            bm.moe_route(s["logits"], s["k"], s["ids"], s["g"], renorm=s["renorm"], bounds=s["bounds"], order=s["order"], slot=s["slot"])
            out = [s["ids"], s["g"], s["bounds"], s["order"], s["slot"]]
            if s["grad"]:
                out.append(bm.moe_route_grad(s["logits"], s["ids"], s["dg"], s["dlogits"], renorm=s["renorm"]))
            return out
        if op == "act":
            out = [bm.silu_mul(s["a"], s["h"])]
            if s["grad"]:
                out.append(bm.silu_mul_grad(s["a"], s["dh"], s["da"]))
            return out
        if op == "combine":
            out = [bm.moe_combine(s["y"], s["slot"], s["g"], s["out"])]
            if s["grad"]:
                out += bm.moe_combine_grad(s["dout"], s["y"], s["slot"], s["g"], s["dy"], s["dg"])
            return out
        act = "silu_mul" if s["act"] else None
        if op == "w4":
            rows, div = (None, 1) if s["E"] == 1 and not s["pad"] else (s["order"], s["k"])
            return [bm.w4_matmul(s["x"], s["codes"], s["scales"], s["mins"], s["y"], None if rows is None else s["bounds"], rows, div, act)]
        rows, div = (s["order"], s["k"]) if s["gather"] else (None, 1)
        out = [bm.grouped_matmul(s["x"], s["w"], s["bounds"], s["y"], rows, div, act)]
        if s["grad"]:
            out.append(bm.grouped_matmul_dx(s["dy"], s["w"], s["bounds"], s["dx"]))
            out.append(bm.grouped_matmul_dw(s["dy"], s["x"], s["bounds"], s["dw"], rows, div))
        return out
    if op == "route":
        return _plain_route(s)
    if op == "act":
        return _plain_act(s)
    if op == "combine":
        return _plain_combine(s)
    return _plain_w4(s) if op == "w4" else _plain_experts(s)


def _plain_route(s):
    l, E, k = s["logits"].float(), s["E"], s["k"]
    top = torch.sort(l, dim=1, descending=True, stable=True)
    best, ids = top.values[:, :k], top.indices[:, :k]
    chosen = best > -math.inf
    m = top.values[:, :1]
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    every, some = torch.exp(l - m), torch.exp(best - m)
    total = (some if s["renorm"] else every).sum(1, keepdim=True)
    g = torch.where(chosen, some / total, 0.0)
    ids = torch.where(chosen, ids, -1).int()
    out = [ids, g, *_grouped(ids, E)]
    if s["grad"]:
        q = torch.zeros_like(l).scatter_add_(1, ids.long().clamp(min=0), torch.where(chosen, s["dg"], 0.0))
        if s["renorm"]:
            p = torch.zeros_like(l).scatter_add_(1, ids.long().clamp(min=0), g)
        else:
            p = torch.where(total > 0, every / total, 0.0)
        out.append((p * (q - (p * q).sum(1, keepdim=True))).to(s["logits"].dtype))
    return out


def _plain_act(s):
    F = s["F"]
    a = s["a"].float()
    g, u = a[:, :F], a[:, F:]
    sig = 1 / (1 + torch.exp(-g))
    out = [(g * sig * u).to(s["a"].dtype)]
    if s["grad"]:
        dh = s["dh"].float()
        out.append(torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], 1).to(s["a"].dtype))
    return out


def _plain_combine(s):
    y, slot, g = s["y"].float(), s["slot"].long(), s["g"]
    T, k = slot.shape
    at, there = slot.clamp(min=0), slot >= 0
    rows = y[at]
    out = [(rows * torch.where(there, g, 0.0)[:, :, None]).sum(1).to(s["out_dtype"])]
    if s["grad"]:
        dout = s["dout"].float()
        end = torch.zeros(T * k + 1, dout.shape[1], device=dout.device)
        end[torch.where(there, slot, T * k).reshape(-1)] = (g[:, :, None] * dout[:, None, :]).reshape(T * k, -1)
        out += [end[: T * k].to(s["y"].dtype), torch.where(there, (rows * dout[:, None, :]).sum(2), 0.0)]
    return out


def _by_expert(rows, w, counts, bounds):
    """rows[i] @ w[e].T for the rows of each expert, none elsewhere."""
    n = sum(counts)
    tail = torch.zeros(rows.shape[0] - n, w.shape[1], device=rows.device)
    if n <= len(counts) // 2:  # few rows: each with its own expert's weights
        e = torch.searchsorted(bounds, torch.arange(n, device=rows.device, dtype=torch.int32), right=True) - 1
        return torch.cat([torch.matmul(w[e].float(), rows[:n, :, None])[:, :, 0], tail])
    parts = rows[:n].split(counts)
    return torch.cat([a @ m.float().t() for a, m in zip(parts, w)] + [tail])


def _gated(y, act):
    if not act:
        return y
    g, u = y.chunk(2, 1)
    return g / (1 + torch.exp(-g)) * u


def _rows(s, gathered):
    x = s["x"].float()
    return x[s["order"].long().clamp(min=0) // s["k"]] if gathered else x


def _plain_experts(s):
    rows, counts = _rows(s, s["gather"]), s["counts"]
    out = [_gated(_by_expert(rows, s["w"], counts, s["bounds"]), s["act"]).to(s["y"].dtype)]
    if s["grad"]:
        n = sum(counts)
        dy = s["dy"].float()
        out.append(_by_expert(dy, s["w"].transpose(1, 2), counts, s["bounds"]).to(s["dx"].dtype))
        out.append(torch.stack([a.t() @ b for a, b in zip(dy[:n].split(counts), rows[:n].split(counts))]))
    return out


def _plain_w4(s):
    codes = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1)
    E, rows, groups = s["scales"].shape
    w = codes.reshape(E, rows, groups, -1).float() * s["scales"].float()[..., None] + s["mins"].float()[..., None]
    return [_gated(_by_expert(_rows(s, True), w.reshape(E, rows, -1), s["counts"], s["bounds"]), s["act"]).to(s["y"].dtype)]


def work(case):
    """What the path cannot do without: weights of the experts that are reached, rows in and out, products."""
    op = case["op"]
    b = SIZE[case["dtype"]]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        more = T * E * b + 4 * T * k if case["grad"] else 0
        return {"bytes": T * E * b + 16 * T * k + 4 * (E + 1) + more, "flops": T * E * (8 if case["grad"] else 4)}
    if op == "act":
        n = case["R"] * case["F"]
        return {"bytes": n * b * (6 if case["grad"] else 3), "flops": n * (18 if case["grad"] else 6)}
    if op == "combine":
        T, k, D, o = case["T"], case["k"], case["D"], SIZE[case["out"]]
        more = T * D * o + T * k * D * b + 4 * T * k if case["grad"] else 0
        return {"bytes": T * k * D * b + T * D * o + 8 * T * k + more, "flops": T * k * D * (5 if case["grad"] else 2)}
    T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
    pairs = (T - min(case["pad"], max(0, T - 1))) * k
    # experts that are reached: the expected number with the popularity that prepare() draws from
    pop = np.arange(1, E + 1, dtype=np.float64) ** -case["zipf"]
    reached = min(E, max(k, float((1 - (1 - np.minimum(1.0, k * pop / pop.sum())) ** max(1, pairs // k)).sum())))
    rows = 2 * N if case["act"] else N
    flops = 2 * pairs * rows * K
    each = rows * K * b if op == "experts" else rows * (K // 2 + 4 * (K // case["G"]))
    ins = (T if op == "w4" or case["gather"] else pairs) * K * b
    bytes_ = reached * each + ins + pairs * N * SIZE[case["out"]]
    if op == "experts" and case["grad"]:
        bytes_ += E * N * K * 4 + pairs * (N + K) * b
        flops *= 3
    return {"bytes": int(bytes_), "flops": int(flops)}


def exact(case, seed):
    """The same outputs from the definitions, in 64 bits."""
    s = prepare(case, seed)
    f64 = torch.float64
    op = case["op"]
    if op == "route":
        l = s["logits"].to(f64).cpu().numpy()
        T, E = l.shape
        k = case["k"]
        ids = np.argsort(-l, axis=1, kind="stable")[:, :k]
        z = np.take_along_axis(l, ids, 1)
        masked = np.isneginf(z)
        with np.errstate(invalid="ignore", divide="ignore"):
            p = np.exp(l - l.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
        p[np.isnan(p)] = 0.0
        part = np.take_along_axis(p, ids, 1)
        kept = part.sum(1, keepdims=True) if case["renorm"] else np.ones((T, 1))
        g = np.where(masked, 0.0, part / np.where(kept > 0, kept, 1.0))
        ids = np.where(masked, -1, ids)
        flat = ids.reshape(-1)
        bounds = np.cumsum(np.concatenate([[0], np.bincount(flat[flat >= 0], minlength=E)]))
        by = np.lexsort((np.arange(flat.size), np.where(flat < 0, E, flat)))
        slot = np.full(flat.size, -1)
        slot[by] = np.arange(flat.size)
        slot[flat < 0] = -1
        by[bounds[-1]:] = -1
        out = [ids, g, bounds, by, slot.reshape(ids.shape)]
        if case["grad"]:
            dg = np.where(masked, 0.0, s["dg"].double().cpu().numpy())
            d = np.zeros_like(l)
            row = np.arange(T)[:, None]
            if case["renorm"]:
                mean = (g * dg).sum(1, keepdims=True)
                np.add.at(d, (row, np.maximum(ids, 0)), np.where(masked, 0.0, g * (dg - mean)))
            else:
                np.add.at(d, (row, np.maximum(ids, 0)), np.where(masked, 0.0, part * dg))
                d -= p * (part * dg).sum(1, keepdims=True)
            out.append(d)
        return [torch.from_numpy(np.ascontiguousarray(v)) for v in out]
    if op == "act":
        a = s["a"].to(f64)
        g, u = a[:, : case["F"]], a[:, case["F"]:]
        sg = torch.sigmoid(g)
        out = [sg * g * u]
        if case["grad"]:
            dh = s["dh"].to(f64)
            out.append(torch.cat([dh * u * (sg + g * sg * torch.sigmoid(-g)), dh * sg * g], 1))
        return out
    if op == "combine":
        y, slot, g = s["y"].to(f64), s["slot"].long(), s["g"].to(f64)
        out = torch.zeros(case["T"], case["D"], dtype=f64, device="cuda")
        dy, dg = torch.zeros_like(y), torch.zeros_like(g)
        dout = s["dout"].to(f64)
        for j in range(case["k"]):
            t = torch.nonzero(slot[:, j] >= 0)[:, 0]
            at = slot[t, j]
            out[t] += g[t, j, None] * y[at]
            dy[at] = g[t, j, None] * dout[t]
            dg[t, j] = (dout[t] * y[at]).sum(1)
        return [out, dy, dg] if case["grad"] else [out]
    x = s["x"].to(f64)
    y = torch.zeros(s["y"].shape, dtype=f64, device="cuda")
    grads = op == "experts" and case["grad"]
    if grads:
        dy = s["dy"].to(f64)
        dx, dw = torch.zeros(s["dx"].shape, dtype=f64, device="cuda"), torch.zeros(s["dw"].shape, dtype=f64, device="cuda")
    at = 0
    for e, n in enumerate(s["counts"]):
        if n:
            here = slice(at, at + n)
            xe = x[s["order"][here].long() // case["k"]] if op == "w4" or case["gather"] else x[here]
            if op == "w4":
                q = torch.stack([s["codes"][e] % 16, s["codes"][e] // 16], 2).reshape(-1, case["K"]).to(f64)
                w = q * s["scales"][e].to(f64).repeat_interleave(case["G"], 1) + s["mins"][e].to(f64).repeat_interleave(case["G"], 1)
            else:
                w = s["w"][e].to(f64)
            v = torch.mm(xe, w.t())
            y[here] = torch.nn.functional.silu(v[:, : case["N"]]) * v[:, case["N"]:] if case["act"] else v
            if grads:
                dx[here] = torch.mm(dy[here], w)
                dw[e] = torch.mm(dy[here].t(), xe)
        at += n
    return [y, dx, dw] if grads else [y]
