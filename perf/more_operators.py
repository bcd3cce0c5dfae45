"""The expert layer's 8-bit operators and its balance loss: rows and weights to 8-bit floating point (e4m3) with a scale for each block of
128, products by expert of such operands with the gradient of their rows, and the balance loss with per-expert counts and its gradient.

Each case is one pass through one operator in the form that serving or training uses; `run` computes it in elementary torch operations in
32 bits (longer sums in 64), or, where `own` is true, through the library's entry points.

8-bit values: a group is 128 elements of a row, or a block of 128 x 128 weights (the last of an axis may be short). With a the largest
finite magnitude of the group, in float32: its scale is a / 448 and its codes are e4m3(v * (448 / a)); both factors are 1 where a < 2^-80.
Rows of codes are filled up with zeros to a multiple of 128.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
F8 = torch.float8_e4m3fn
B = 128
TINY = 2.0 ** -80


def listed():
    return [
        # a decode batch's rows on their way into 8-bit projections that share them; latency alone counts
        {"name": "rows decode", "op": "rows", "R": 32, "K": 2048, "dtype": "f16", "act": False},
        # the gated activation of a training batch, straight to the down projection's 8-bit rows
        {"name": "rows training", "op": "rows", "R": 24576, "K": 1408, "dtype": "bf16", "act": True},
        # one projection of a checkpoint while it is loaded for serving
        {"name": "weights of a projection", "op": "weights", "E": 1, "N": 4096, "K": 2048, "dtype": "bf16", "transposed": False},
        # master weights after an optimizer's step, with the transposed copy for the gradients
        {"name": "weights training", "op": "weights", "E": 8, "N": 4096, "K": 14336, "dtype": "f32", "transposed": True},
        # one token through a dense 8-bit projection (attention output, shared expert)
        {"name": "product one token dense", "op": "mm", "T": 1, "k": 1, "E": 1, "N": 4096, "K": 2048, "dtype": "f16", "out": "f16",
         "gather": True, "act": False, "grad": False, "given": False, "zipf": 0.0, "pad": 0},
        # decode of one token: gate/up of its 8 experts with the activation, 25 MB of weights
        {"name": "product one token", "op": "mm", "T": 1, "k": 8, "E": 128, "N": 768, "K": 2048, "dtype": "bf16", "out": "bf16",
         "gather": True, "act": True, "grad": False, "given": False, "zipf": 0.0, "pad": 0},
        # a decode batch whose experts repeat (Zipf popularity)
        {"name": "product decode", "op": "mm", "T": 32, "k": 8, "E": 128, "N": 768, "K": 2048, "dtype": "bf16", "out": "bf16",
         "gather": True, "act": True, "grad": False, "given": False, "zipf": 1.1, "pad": 0},
        # a prefill chunk of a 64-expert layer, ragged counts
        {"name": "product prefill", "op": "mm", "T": 4096, "k": 6, "E": 64, "N": 1408, "K": 2048, "dtype": "bf16", "out": "bf16",
         "gather": True, "act": True, "grad": False, "given": False, "zipf": 1.0, "pad": 0},
        # a training step of an 8-expert layer's down projection: rows that the activation left in 8 bits, and their gradient
        {"name": "product training", "op": "mm", "T": 4096, "k": 2, "E": 8, "N": 4096, "K": 14336, "dtype": "bf16", "out": "bf16",
         "gather": False, "act": False, "grad": True, "given": True, "zipf": 0.0, "pad": 0},
        # evaluation of a small batch's balance: loss and counts alone
        {"name": "balance small", "op": "balance", "T": 67, "E": 8, "k": 2, "S": 1, "dtype": "f32", "grad": False, "pad": 0},
        # a training batch of eight packed sequences, a loss for each, with the gradient
        {"name": "balance sequences", "op": "balance", "T": 4096, "E": 64, "k": 6, "S": 8, "dtype": "bf16", "grad": True, "pad": 37},
        # a training batch with one loss over all its tokens, with the gradient
        {"name": "balance training", "op": "balance", "T": 16384, "E": 128, "k": 8, "S": 1, "dtype": "f32", "grad": True, "pad": 0},
    ]


def _log(rng, lo, hi, step=1):
    """A whole multiple of `step` from lo to hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["rows", "weights", "mm", "mm", "mm", "mm", "balance", "balance"])
    if op == "rows":
        return {"op": op, "R": _log(rng, 1, 24576), "K": _log(rng, 8, 1408, rng.choice([1, 8, 64])), "dtype": rng.choice(["bf16", "f16", "f32"]),
                "act": rng.random() < 0.5}
    if op == "weights":
        return {"op": op, "E": rng.choice([1, 2, 5, 16]), "N": _log(rng, 16, 4096, rng.choice([1, 16, 128])),
                "K": _log(rng, 64, 4096, rng.choice([1, 16, 128])), "dtype": rng.choice(["bf16", "f16", "f32"]), "transposed": rng.random() < 0.5}
    if op == "balance":
        E, T = _log(rng, 4, 512), _log(rng, 1, 16384)
        return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(E, 10)), "S": rng.choice([1, 1, min(T, 3), _log(rng, 1, min(T, 64))]),
                "dtype": rng.choice(["f32", "bf16", "f16"]), "grad": rng.random() < 0.6, "pad": rng.choice([0, 0, 11])}
    dtype = rng.choice(["bf16", "f16"])
    E = rng.choice([1, 3, 8, 16, 64, 128])
    act = rng.random() < 0.4
    # at most as many weights and products as the largest listed case
    return {"op": op, "T": _log(rng, 1, 4096), "k": rng.randint(1, min(E, 8)), "E": E, "N": _log(rng, 64, 4096, rng.choice([1, 8, 16, 128])),
            "K": _log(rng, 64, 4096, rng.choice([1, 8, 128, 128])), "dtype": dtype, "out": rng.choice([dtype, dtype, "f32"]),
            "gather": rng.random() < 0.5, "act": act, "grad": not act and rng.random() < 0.5, "given": rng.random() < 0.4,
            "zipf": rng.choice([0.0, 0.7, 1.1]), "pad": rng.choice([0, 0, 5])}


def _ids(gen, T, k, E, zipf, pad):
    """k different experts a token, popularity falling as rank^-zipf (Gumbel keys); the last `pad` tokens are padding, with ids of -1."""
    keys = -torch.log(-torch.log(torch.rand(T, E, generator=gen, device="cuda").clamp_(1e-9, 1 - 1e-7)))
    rank = torch.randperm(E, generator=gen, device="cuda") + 1
    ids = torch.topk(keys - zipf * rank.float().log(), k, dim=1).indices.int()
    if pad:
        ids[max(1, T - pad):] = -1
    return ids


def _sorted_pairs(ids, E):
    """(bounds, order) of the pairs sorted by expert, earlier pairs first; pairs without an expert come last, with -1."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(key, stable=True).indices
    bounds = (key[order][:, None] < torch.arange(E + 1, device=ids.device)[None, :]).sum(0)
    return bounds.int(), torch.where(torch.arange(flat.numel(), device=ids.device) < bounds[E], order, -1).int()


def _up(n):
    return -(-n // B) * B


def _factors(v, dims):
    """(scale, 448 / a) of the groups over `dims`."""
    a = torch.where(torch.isfinite(v), v.abs(), 0.0).amax(dims)
    tiny = a < TINY
    top = torch.full_like(a, 448.0)  # (a tensor: torch divides by a plain number by multiplying with its reciprocal)
    return torch.where(tiny, 1.0, torch.div(a, top)), torch.where(tiny, 1.0, torch.div(top, a))


def _rows8(x):
    """(codes, scales) of rows, a scale for each 128 elements."""
    R, K = x.shape
    v = torch.nn.functional.pad(x.float(), (0, _up(K) - K)).reshape(R, -1, B)
    s, r = _factors(v, 2)
    return (v * r[:, :, None]).to(F8).reshape(R, -1), s


def _blocks8(w):
    """(codes, scales) of weights, a scale for each block of 128 x 128."""
    E, N, K = w.shape
    v = torch.nn.functional.pad(w.float(), (0, _up(K) - K, 0, _up(N) - N)).reshape(E, _up(N) // B, B, -1, B)
    s, r = _factors(v, (2, 4))
    return (v * r[:, :, None, :, None]).to(F8).reshape(E, _up(N), -1)[:, :N].contiguous(), s


def _turned8(w):
    """The same of the transposed weights."""
    return _blocks8(w.transpose(1, 2))


def _values(codes, scales, rows=B):
    """What codes of E x N x K stand for, in 32 bits: a scale for `rows` x 128 of them."""
    s = scales.repeat_interleave(rows, 1)[:, : codes.shape[1]]
    return (codes.float().unflatten(2, (-1, B)) * s[:, :, :, None]).flatten(2)


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(int(seed) * 7919 + 29)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype).mul_(scale)

    s = dict(case)
    op = case["op"]
    dt = DTYPES[case["dtype"]]
    i32 = {"dtype": torch.int32, "device": "cuda"}
    if op == "rows":
        R, K = case["R"], case["K"]
        x = normal(R, 2 * K if case["act"] else K)
        x[:, :: max(1, K // 8)] *= 20.0  # outlier channels
        x[R // 2, : min(K, B)] = 0.0
        s["x"] = x.to(dt)
        s["codes"] = torch.empty(R, _up(K), device="cuda", dtype=F8)
        s["scales"] = torch.empty(R, _up(K) // B, device="cuda")
        return s
    if op == "weights":
        E, N, K = case["E"], case["N"], case["K"]
        s["w"] = normal(E, N, K, scale=K ** -0.5).to(dt)
        s["codes"], s["scales"] = torch.empty(E, N, _up(K), device="cuda", dtype=F8), torch.empty(E, _up(N) // B, _up(K) // B, device="cuda")
        if case["transposed"]:
            s["codes_t"] = torch.empty(E, K, _up(N), device="cuda", dtype=F8)
            s["scales_t"] = torch.empty(E, _up(K) // B, _up(N) // B, device="cuda")
        return s
    T, k, E = case["T"], case["k"], case["E"]
    if op == "balance":
        S = case["S"]
        s["logits"] = (normal(T, E) + 0.7 * normal(1, E)).to(dt)  # a router that prefers some experts
        s["ids"] = torch.topk(s["logits"].float(), k, dim=1).indices.int()
        if case["pad"]:  # padding tokens: no expert, and logits of any value
            s["ids"][max(1, T - case["pad"]):] = -1
            s["logits"][max(1, T - case["pad"]):] *= 50.0
        cuts = torch.randperm(T, generator=gen, device="cuda")[: S - 1].sort().values
        s["seqs"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)]).int() if S > 1 else None
        s["loss"], s["z"], s["counts"] = torch.empty(S, device="cuda"), torch.empty(S, device="cuda"), torch.empty(S, E, **i32)
        s["tokens"] = torch.empty(S, **i32)
        s["dloss"], s["dz"] = normal(S) * 0.01, normal(S) * 0.001
        s["dlogits"] = torch.zeros_like(s["logits"])
        return s
    N, K = case["N"], case["K"]
    ids = _ids(gen, T, k, E, case["zipf"], case["pad"])
    s["bounds"], s["order"] = _sorted_pairs(ids, E)
    s["counts"] = (s["bounds"][1:] - s["bounds"][:-1]).tolist()
    x = normal(T if case["gather"] else T * k, K)
    x[:, :: max(1, K // 8)] *= 8.0  # outlier channels
    s["x"], s["x_scales"] = _rows8(x.to(dt)) if case["given"] else (x.to(dt), None)
    parts = 2 if case["act"] else 1  # gate and up rows have blocks of their own
    w = normal(E * parts, N, K, scale=K ** -0.5, dtype=torch.bfloat16)
    s["codes"], s["scales"] = _blocks8(w)
    s["codes"], s["scales"] = s["codes"].reshape(E, parts * N, -1), s["scales"].reshape(E, parts * s["scales"].shape[1], -1)
    out = DTYPES[case["out"]]
    s["y"] = torch.zeros(T * k, N, device="cuda", dtype=out)
    if case["grad"]:
        s["codes_t"], s["scales_t"] = _turned8(w)
        s["dy"] = normal(T * k, N, dtype=dt)
        s["dx"] = torch.zeros(T * k, K, device="cuda", dtype=out)
    return s


def run(s):
    op = s["op"]
    if own:
        from spectral_expert_gemv_amd import bitsmoe as bm
        if op == "rows":
            return bm.fp8_rows(s["x"], s["codes"], s["scales"], act="silu_mul" if s["act"] else None)
        if op == "weights":
            if s["transposed"]:
                return bm.fp8_weights(s["w"], s["codes"], s["scales"], s["codes_t"], s["scales_t"])
            return bm.fp8_weights(s["w"], s["codes"], s["scales"])
        if op == "balance":
            out = list(bm.moe_balance(s["logits"], s["ids"], s["seqs"], s["loss"], s["z"], s["counts"], s["tokens"]))
            if s["grad"]:
                out.append(bm.moe_balance_grad(s["logits"], s["ids"], s["counts"], s["tokens"], s["dloss"], s["dz"], s["seqs"], s["dlogits"]))
            return out
        rows, div = (s["order"], s["k"]) if s["gather"] else (None, 1)
        if s["E"] == 1 and s["gather"] and not s["pad"]:
            rows, div = None, 1  # one dense projection: its rows are the tokens
        out = [bm.fp8_matmul(s["x"], s["codes"], s["scales"], s["y"], x_scales=s["x_scales"], bounds=s["bounds"] if rows is not None or s["E"] > 1 or s["pad"] else None,
                             rows=rows, div=div, act="silu_mul" if s["act"] else None)]
        if s["grad"]:
            out.append(bm.fp8_matmul(s["dy"], s["codes_t"], s["scales_t"], s["dx"], bounds=s["bounds"]))
        return out
    return {"rows": _plain_rows, "weights": _plain_weights, "balance": _plain_balance, "mm": _plain_mm}[op](s)


def _gated(y, act):
    if not act:
        return y
    g, u = y.chunk(2, 1)
    return g / (1 + torch.exp(-g)) * u


def _plain_rows(s):
    return _rows8(_gated(s["x"].float(), s["act"]))


def _plain_weights(s):
    return [*_blocks8(s["w"]), *(_turned8(s["w"]) if s["transposed"] else ())]


def _by_expert(rows, w, counts, bounds):
    """rows[i] @ w[e].T for the rows of each expert, none elsewhere."""
    n = sum(counts)
    tail = torch.zeros(rows.shape[0] - n, w.shape[1], device=rows.device)
    if n <= len(counts) // 2:  # few rows: each with its own expert's weights
        e = torch.searchsorted(bounds, torch.arange(n, device=rows.device, dtype=torch.int32), right=True) - 1
        return torch.cat([torch.matmul(w[e], rows[:n, :, None])[:, :, 0], tail])
    return torch.cat([a @ m.t() for a, m in zip(rows[:n].split(counts), w)] + [tail])


def _plain_mm(s):
    x, xs = (s["x"], s["x_scales"]) if s["given"] else _rows8(s["x"])
    x = _values(x[None], xs[None], 1)[0]
    if s["gather"]:
        x = x[s["order"].long().clamp(min=0) // s["k"]]
    E, counts = s["E"], s["counts"]
    parts = 2 if s["act"] else 1
    codes, scales = s["codes"].unflatten(1, (parts, -1)).flatten(0, 1), s["scales"].unflatten(1, (parts, -1)).flatten(0, 1)
    w = _values(codes, scales).unflatten(0, (E, parts)).flatten(1, 2)
    out = [_gated(_by_expert(x, w, counts, s["bounds"]), s["act"]).to(s["y"].dtype)]
    if s["grad"]:
        dy, ds = _rows8(s["dy"])
        dx = _by_expert(_values(dy[None], ds[None], 1)[0], _values(s["codes_t"], s["scales_t"]), counts, s["bounds"])
        out.append(dx.to(s["dx"].dtype))
    return out


def _plain_balance(s):
    l, E, k, S = s["logits"].float(), s["E"], s["k"], s["S"]
    T = l.shape[0]
    good = (s["ids"] >= 0) & (s["ids"] < E)
    part = good.any(1)
    seq = torch.zeros(T, dtype=torch.long, device=l.device)
    if S > 1:
        seq = torch.bucketize(torch.arange(T, device=l.device, dtype=torch.int32), s["seqs"][1:], right=True)
    l = torch.where(part[:, None], l, 0.0)
    m = l.amax(1, keepdim=True)
    e = torch.exp(l - m)
    total = e.sum(1, keepdim=True)
    p, lse = e / total, m + torch.log(total)
    cuts = [0, T] if S == 1 else s["seqs"].long()

    def sums(v):  # over each sequence's tokens, in 64 bits
        return torch.cumsum(torch.cat([torch.zeros_like(v[:1]), v]).double(), 0)[cuts].diff(dim=0)

    n = sums(part.double())
    counts = sums(torch.zeros_like(l).scatter_add_(1, s["ids"].long().clamp(0, E - 1), good.float()))
    inv = torch.where(n > 0, 1 / n, 0.0)
    share = sums(torch.where(part[:, None], p, 0.0)) * inv[:, None]
    f = counts * inv[:, None] * (E / k)
    z = sums(torch.where(part, lse[:, 0].double() ** 2, 0.0)) * inv
    out = [(f * share).sum(1).float(), z.float(), counts.int(), n.int()]
    if s["grad"]:
        a, b = (s["dloss"].double() * inv).float()[seq][:, None], (2 * s["dz"].double() * inv).float()[seq][:, None]
        ft = f.float()[seq]
        d = p * (a * (ft - (p * ft).sum(1, keepdim=True)) + b * lse)
        out.append(torch.where(part[:, None], d, 0.0).to(s["logits"].dtype))
    return out


def work(case):
    """What the path cannot do without: inputs once (weights: of the experts that are reached), outputs once, products."""
    op = case["op"]
    b = SIZE[case["dtype"]]
    if op == "rows":
        R, K = case["R"], case["K"]
        return {"bytes": int(R * (K * b * (2 if case["act"] else 1) + _up(K) * (1 + 4 / B))), "flops": R * K * (8 if case["act"] else 2)}
    if op == "weights":
        E, N, K = case["E"], case["N"], case["K"]
        out = N * _up(K) + (K * _up(N) if case["transposed"] else 0)
        return {"bytes": int(E * (N * K * b + out * (1 + 4 / B ** 2))), "flops": 2 * E * N * K}
    T, k, E = case["T"], case["k"], case["E"]
    if op == "balance":
        return {"bytes": T * E * b * (2 if case["grad"] else 1) + 4 * T * k + 4 * case["S"] * (E + 3), "flops": T * E * (10 if case["grad"] else 5)}
    N, K = case["N"], case["K"]
    pairs = (T - min(case["pad"], max(0, T - 1))) * k
    # experts that are reached: the expected number with the popularity that prepare() draws from
    pop = np.arange(1, E + 1, dtype=np.float64) ** -case["zipf"]
    reached = min(E, max(k, float((1 - (1 - np.minimum(1.0, k * pop / pop.sum())) ** max(1, pairs // k)).sum())))
    rows = 2 * N if case["act"] else N
    ins = (T if case["gather"] else pairs) * (_up(K) if case["given"] else K * b)
    o = SIZE[case["out"]]
    bytes_, flops = reached * rows * _up(K) + ins + pairs * N * o, 2 * pairs * rows * K
    if case["grad"]:
        bytes_ += reached * K * _up(N) + pairs * (N * b + K * o)
        flops *= 2
    return {"bytes": int(bytes_), "flops": int(flops)}


def _e4m3(v):
    """The nearest e4m3 number (64 bits, ties to even) of values up to 448; NaN where v is not finite."""
    a = v.abs()
    exp = (torch.frexp(torch.where(torch.isfinite(a), a, 1.0))[1] - 1).clamp(min=-6)
    step = ((exp.long() + (1023 - 3)) << 52).view(torch.float64)  # 2^(exp - 3) by its bits (torch.ldexp is a step off)
    return torch.where(torch.isfinite(a), torch.copysign(torch.round(a / step) * step, v), math.nan)


def _exact_groups(v, high):
    """(values of the codes, scales) of the groups of high x 128 elements of a matrix in 64 bits; the definition's float32 steps are done
    in 64 bits, where they are exact or innocent of a second rounding, and rounded to 32."""
    r, c = v.shape
    full = torch.zeros(-(-r // high) * high, _up(c), dtype=torch.float64, device=v.device)
    full[:r, :c] = v
    g = full.reshape(-1, high, _up(c) // B, B)
    a = torch.where(torch.isfinite(g), g, 0.0).abs().amax((1, 3), keepdim=True)
    scale, factor = torch.ones_like(a), torch.ones_like(a)
    big = a >= TINY
    top = torch.full_like(a[big], 448.0)
    scale[big] = (a[big] / top).float().double()
    factor[big] = (top / a[big]).float().double()
    q = _e4m3((g * factor).float().double())
    return q.reshape(full.shape)[:r], scale[:, 0, :, 0]


def _exact_values(codes, scales, high):
    return codes.double() * scales.double().repeat_interleave(high, 0)[: codes.shape[0]].repeat_interleave(B, 1)


def exact(case, seed):
    """The same outputs from the definitions, in 64 bits."""
    s = prepare(case, seed)
    f64 = torch.float64
    op = case["op"]
    if op == "rows":
        x = s["x"].to(f64)
        if case["act"]:
            x = (torch.nn.functional.silu(x[:, : case["K"]]) * x[:, case["K"]:]).float().to(f64)
        return _exact_groups(x, 1)
    if op == "weights":
        out = [[], [], [], []]
        for w in s["w"]:
            q, sc = _exact_groups(w.to(f64), B)
            out[0].append(q.float())
            out[1].append(sc)
            if case["transposed"]:
                q, sc = _exact_groups(w.to(f64).t().contiguous(), B)
                out[2].append(q.float())
                out[3].append(sc)
        return [torch.stack(v).double() for v in out if v]
    if op == "balance":
        l, ids = s["logits"].to(f64).cpu().numpy(), s["ids"].cpu().numpy()
        T, E = l.shape
        k, S = case["k"], case["S"]
        cuts = [0, T] if s["seqs"] is None else s["seqs"].tolist()
        loss, z, counts, tokens, d = np.zeros(S), np.zeros(S), np.zeros((S, E), np.int64), np.zeros(S, np.int64), np.zeros_like(l)
        for q in range(S):
            at = np.arange(cuts[q], cuts[q + 1])
            at = at[(ids[at] >= 0).any(1)]
            tokens[q] = n = len(at)
            if n == 0:
                continue
            chosen = ids[at].reshape(-1)
            counts[q] = np.bincount(chosen[chosen >= 0], minlength=E)
            top = l[at].max(1, keepdims=True)
            lse = top[:, 0] + np.log(np.exp(l[at] - top).sum(1))
            p = np.exp(l[at] - lse[:, None])
            f = counts[q] * (E / (k * n))
            loss[q], z[q] = f @ p.mean(0), np.mean(lse ** 2)
            dl, dz = float(s["dloss"][q]), float(s["dz"][q])
            d[at] = p * (f - (p @ f)[:, None]) * (dl / n) + p * lse[:, None] * (2 * dz / n)
        out = [loss, z, counts, tokens] + ([d] if case["grad"] else [])
        return [torch.from_numpy(v) for v in out]
    E, N = case["E"], case["N"]
    q, sc = (s["x"], s["x_scales"]) if case["given"] else _exact_groups(s["x"].to(f64), 1)
    x = _exact_values(q, sc, 1)
    y = torch.zeros(s["y"].shape, dtype=f64, device="cuda")
    if case["grad"]:
        dy = _exact_values(*_exact_groups(s["dy"].to(f64), 1), 1)
        dx = torch.zeros(s["dx"].shape, dtype=f64, device="cuda")
    at = 0
    for e, n in enumerate(s["counts"]):
        if n:
            here = slice(at, at + n)
            xe = x[s["order"][here].long() // case["k"]] if case["gather"] else x[here]
            half = s["scales"].shape[1] // (2 if case["act"] else 1)
            v = torch.mm(xe, _exact_values(s["codes"][e][:N], s["scales"][e][:half], B).t())
            if case["act"]:
                v = torch.nn.functional.silu(v) * torch.mm(xe, _exact_values(s["codes"][e][N:], s["scales"][e][half:], B).t())
            y[here] = v
            if case["grad"]:
                dx[here] = torch.mm(dy[here], _exact_values(s["codes_t"][e], s["scales_t"][e], B).t())
        at += n
    return [y, dx] if case["grad"] else [y]
