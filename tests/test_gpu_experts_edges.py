"""GPU tests of the expert layer's operators where they can go wrong: weights
that cancel, infinities and NaN, empty batches, rows at any alignment, and the
router in front of the spectral path.

Tolerances as in test_gpu_experts.py: a float32 sum of n products adds at most
n 2^-23 of the sum of their magnitudes, an output rounded once half a step.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from .oracle_ref import max_rel_err, pairs_ref  # noqa: E402
from .test_gpu_experts import BF16, F16, F32, STEP, _say, bm, check, half_step, normal, ragged, rng  # noqa: E402,F401

INF, NAN = float("inf"), float("nan")


def at_offset(t, off):
    """t as rows whose first element lies `off` elements past 16-byte alignment."""
    wide = torch.full((t.shape[0], t.shape[1] + 8), NAN, dtype=t.dtype, device=t.device)
    wide[:, off:off + t.shape[1]] = t
    return wide[:, off:off + t.shape[1]]


def dequantized(codes, s, m, G):
    """(s q, m) of every weight in 64 bits."""
    q = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1).double()
    sd = s.double().repeat_interleave(G, -1)
    return sd * q, -8 * sd if m is None else m.double().repeat_interleave(G, -1)


# ------------------------------------------------------- 4-bit weights

# E, counts, K, G: one and two rows (up to and past 1024 inputs), a few, tiles of 16 and of 32
W4_ROWS = [(1, [1], 128, 128), (1, [1], 2048, 128), (1, [2], 512, 64), (3, [2, 1, 2], 2048, 64), (1, [5], 256, 32),
           (1, [14], 4096, 128), (2, [20, 40], 256, 64)]


@pytest.mark.parametrize("E, counts, K, G", W4_ROWS)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -17])
@pytest.mark.parametrize("off", [0, 3])
def test_w4_of_one_sided_groups(bm, E, counts, K, G, dtype, size, off):
    """Small weights of one sign beside one large weight a group: the codes are
    0 but for that one, and W x is the minima's sum.  Inputs near 2^-17 are
    subnormal in float16."""
    _say("one-sided", E, counts, K, G, dtype, size, off)
    g = rng(K + G)
    N = 33
    bounds, R = ragged(g, E, counts)
    w = normal(g, E, N, K).abs() * 0.01
    w[:, :, ::G] = 3.0
    x = normal(g, R, K, scale=size)
    x[:, ::G] = 0.0
    x = at_offset(x.to(dtype), off)
    codes, s, m = (torch.from_numpy(a).cuda() for a in bm.w4_pack(w.cpu().numpy(), G))
    y = bm.w4_matmul(x, codes, s, m, torch.empty(R, N, device="cuda"), bounds)
    sq, md = dequantized(codes, s, m, G)
    e = torch.repeat_interleave(torch.arange(E), torch.tensor(counts)).cuda()
    r = x.double()
    want = torch.matmul((sq + md)[e], r[:, :, None])[:, :, 0]
    mag = torch.matmul((sq + md.abs())[e], r.abs()[:, :, None])[:, :, 0]
    # K products and a few sums of groups and waves; the size of s q and m alone, not of an offset
    check(y, want, mag * ((K + 16) * STEP) + half_step(want, F32), "y")


@pytest.mark.parametrize("E, counts, K, G", W4_ROWS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_w4_bits_do_not_depend_on_alignment(bm, E, counts, K, G, dtype):
    _say("alignment", E, counts, K, G, dtype)
    g = rng(K + 1)
    bounds, R = ragged(g, E, counts)
    codes = torch.randint(0, 256, (E, 66, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(E, 66, K // G, generator=g, device="cuda") * 0.1).half()
    m = (s.float() * normal(g, E, 66, K // G)).half()
    x = normal(g, R, K, dtype=dtype)
    for act in (None, "silu_mul"):
        want = bm.w4_matmul(x, codes, s, m, bounds=bounds, act=act)
        for off in (1, 2, 4, 7):
            assert torch.equal(bm.w4_matmul(at_offset(x, off), codes, s, m, bounds=bounds, act=act), want), off


@pytest.mark.parametrize("R, off", [(70000, 1), (65535 * 32 + 77, 0), (65535 * 32 + 77, 3)])
@pytest.mark.parametrize("E", [1, 2])
def test_w4_of_many_rows(bm, R, off, E):
    """More row tiles than one dimension of a grid takes."""
    _say("many rows", R, off, E)
    g = rng(R)
    K, N = 32, 5
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(E, N, 1, generator=g, device="cuda") + 0.5).half()
    m = (s.float() * -7.5).half()
    x = at_offset(normal(g, R, K, dtype=F16), off)
    first = R // 3 if E == 2 else R
    bounds = None if E == 1 else torch.tensor([0, first, R], dtype=torch.int32, device="cuda")
    y = bm.w4_matmul(x, codes, s, m, torch.empty(R, N, device="cuda"), bounds)
    sq, md = dequantized(codes, s, m, K)
    for e, rows in ((0, slice(0, first)), (E - 1, slice(R - (R - first or R), R))):
        r = x[rows].double()
        want = r @ (sq + md)[e].t()
        check(y[rows], want, r.abs() @ (sq + md.abs())[e].t() * ((K + 16) * STEP) + half_step(want, F32), "y")


def same_kind(got, want, tol, what):
    """NaN where want is, the same infinities, finite values within tol."""
    got = got.double().cpu()
    assert torch.equal(got.isnan(), want.isnan()), what + ": NaN"
    inf = want.isinf()
    assert torch.equal(got.isinf(), inf) and torch.equal(got[inf], want[inf]), what + ": infinities"
    fine = want.isfinite()
    check(got[fine], want[fine], tol[fine], what)


@pytest.mark.parametrize("E, counts, K, G", W4_ROWS)
@pytest.mark.parametrize("dtype, off", [(F16, 0), (BF16, 0), (BF16, 5)])
@pytest.mark.parametrize("symmetric", [False, True])
def test_w4_of_infinities_and_nan(bm, E, counts, K, G, dtype, off, symmetric):
    """An output is what sum_c W x is: +-inf, NaN for 0 inf or inf - inf, and
    finite where only the sums of q x would pass float32's range."""
    _say("w4 infinities", E, counts, K, G, dtype, off, symmetric)
    g = rng(K + 9)
    N = 20
    bounds, R = ragged(g, E, counts)
    codes = torch.randint(0, 256, (E, 2 * N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = ((torch.rand(E, 2 * N, K // G, generator=g, device="cuda") + 0.5) * 2.0 ** -6).half()
    m = None if symmetric else (s.float() * (normal(g, *s.shape) - 7.5)).half()
    clean = normal(g, R, K, dtype=dtype)
    row, e = R - 1, E - 1
    sq, md = dequantized(codes[e], s[e], None if m is None else m[e], G)
    w = (sq + md).cpu()
    half = lambda t: None if t is None else t[:, :N].contiguous()  # noqa: E731
    y0 = bm.w4_matmul(clean, half(codes), half(s), half(m), bounds=bounds)
    h0 = bm.w4_matmul(clean, codes, s, m, bounds=bounds, act="silu_mul")
    kinds = {"inf": {5: INF}, "-inf": {K - 1: -INF}, "both": {1: INF, K - 2: -INF}, "nan": {3: NAN}}
    if dtype == BF16:
        kinds["large"] = {7: 3e37, K - 7: 3e37}  # 15 times this is past float32
    for kind, put in kinds.items():
        x = clean.clone()
        for c, v in put.items():
            x[row, c] = v
        terms = w * x[row].double().cpu()
        # (each product of w and the input, then their sum: as a product by a matrix would be)
        v, tol = terms.sum(1), terms.abs().sum(1) * ((K + 16) * STEP)
        x = at_offset(x, off)
        y = bm.w4_matmul(x, half(codes), half(s), half(m), bounds=bounds)
        same_kind(y[row], v[:N], tol[:N] + half_step(v[:N], dtype), kind)
        assert torch.equal(y[:row], y0[:row]), kind
        h = bm.w4_matmul(x, codes, s, m, bounds=bounds, act="silu_mul")
        assert torch.equal(h[:row], h0[:row]), kind
        if kind != "large":
            want = torch.nn.functional.silu(v[:N]) * v[N:]
            same_kind(h[row], want, torch.zeros_like(want), kind + " activated")


# ---------------------------------------------------- empty batches

@pytest.mark.parametrize("E", [1, 255, 256, 512, 513, 600, 1024, 2048])
def test_no_tokens_at_all(bm, E):
    _say("no tokens", E)
    ids = torch.empty((0, 1), dtype=torch.int32, device="cuda")
    full = lambda *n: torch.full(n, 7, dtype=torch.int32, device="cuda")  # noqa: E731
    b = full(E + 9)
    bounds, order, slot = bm.moe_group(ids, E, b[:E + 1])
    assert not bool(bounds.any()) and bool((b[E + 1:] == 7).all()) and order.numel() == slot.numel() == 0
    bounds = full(E + 1)
    bm.moe_route(torch.empty(0, E, device="cuda"), 1, bounds=bounds, order=full(0), slot=full(0, 1))
    assert not bool(bounds.any())


@pytest.mark.parametrize("E", [4, 600])
def test_a_layer_of_no_tokens(bm, E):
    from spectral_expert_gemv_amd import ExpertLayer
    g = rng(E)
    w1, w2 = normal(g, E, 16, 32, dtype=BF16), normal(g, E, 32, 8, dtype=BF16)
    layer = ExpertLayer(w1, w2)
    x, logits = torch.empty(0, 32, dtype=BF16, device="cuda"), torch.empty(0, E, device="cuda")
    assert layer.forward(x, logits, 2).shape == (0, 32)
    out, dx, dl, dw1, dw2 = layer.gradients(x, logits, 2, x)
    assert out.shape == dx.shape == (0, 32) and dl.shape == (0, E)
    assert dw1.shape == w1.shape and not bool(dw1.any()) and not bool(dw2.any())


# ------------------------------------------------- activation, router, combine

@pytest.mark.parametrize("dtype, huge", [(F16, 65504.0), (BF16, 3.3e38)])
@pytest.mark.parametrize("F", [48, 45])
def test_silu_mul_of_infinities_nan_and_the_largest(bm, dtype, huge, F):
    """As the formulas in 64 bits give it, for gates and ups up to the type's
    largest value, infinities and NaN."""
    _say("silu_mul", dtype, F)
    gates = [INF, -INF, NAN, huge, -huge, huge * 0.73, huge * 0.69, -huge * 0.73, 0.0, 1.0, -20.0, 20.0]
    ups = [1.0, -0.5, 0.0, INF, -INF, NAN, huge, 2.0 ** -10]
    pairs = torch.tensor([(g, u) for g in gates for u in ups], dtype=dtype, device="cuda")
    n = (len(pairs) + F - 1) // F
    a = torch.ones(n, 2 * F, dtype=dtype, device="cuda")
    at = torch.arange(len(pairs), device="cuda")
    a[at // F, at % F] = pairs[:, 0]
    a[at // F, F + at % F] = pairs[:, 1]
    g, u = a[:, :F].double().cpu(), a[:, F:].double().cpu()
    s = torch.sigmoid(g)
    # (what passes the type's largest value rounds to an infinity; that rounding is the second half step)
    v = (g * s * u).to(F32).to(dtype).double()
    same_kind(bm.silu_mul(a), v, half_step(v, dtype) * 2 + v.abs() * 2.0 ** -20, "h")
    dh = torch.full((n, F), 0.25, dtype=dtype, device="cuda")
    da = bm.silu_mul_grad(a, dh)
    for got, v, size in ((da[:, :F], 0.25 * u * (s * (1 + g * (1 - s))), 0.25 * u.abs() * s * (1 + (g * (1 - s)).abs())),
                         (da[:, F:], 0.25 * (g * s), 0.25 * (g * s).abs())):
        v = v.to(F32).to(dtype).double()
        same_kind(got, v, half_step(v, dtype) * 2 + size * 2.0 ** -20 + 1e-30, "da")


@pytest.mark.parametrize("D", [64, 37])
def test_combine_of_missing_rows(bm, D):
    """A slot without a row adds its weight times 0."""
    y = normal(rng(1), 6, D, dtype=F16)
    slot = torch.tensor([[0, -1], [-1, 5], [9, -1], [2, 3]], dtype=torch.int32, device="cuda")
    g = torch.tensor([[0.5, 0.0], [NAN, 2.0], [0.0, 7.0], [1.0, 1.0]], device="cuda")
    out = bm.moe_combine(y, slot, g, torch.empty(4, D, device="cuda"))
    assert torch.equal(out[0], 0.5 * y[0].float()) and not bool(out[2].any()) and bool(out[1].isnan().all())
    assert torch.equal(out[3], y[2].float() + y[3].float())


@pytest.mark.parametrize("bad", [NAN, INF])
def test_a_token_without_a_softmax_is_nan(bm, bad):
    """Its output and its dlogits are; padding is 0 and the other tokens' results
    are those of the batch without it."""
    from spectral_expert_gemv_amd import ExpertLayer
    g = rng(3)
    T, E, k, D, F = 12, 8, 2, 64, 32
    x, dout = normal(g, T, D, dtype=BF16), normal(g, T, D, dtype=BF16)
    w1, w2 = normal(g, E, 2 * F, D, dtype=BF16, scale=0.1), normal(g, E, D, F, dtype=BF16, scale=0.1)
    logits = normal(g, T, E)
    logits[7] = -INF
    other = logits.clone()
    other[4] = -INF
    logits[4, 5] = bad
    keep = torch.arange(T, device="cuda") != 4
    q = ExpertLayer.w4(w1.float().cpu().numpy(), w2.float().cpu().numpy(), group=32)
    for layer in (ExpertLayer(w1, w2), q):
        out, ref = layer.forward(x, logits, k), layer.forward(x, other, k)
        assert bool(out[4].isnan().all()) and torch.equal(out[keep], ref[keep]) and not bool(out[7].any())
    layer = ExpertLayer(w1, w2)
    got, ref = layer.gradients(x, logits, k, dout), layer.gradients(x, other, k, dout)
    assert bool(got[0][4].isnan().all()) and bool(got[2][4].isnan().all())
    for a, b in zip(got[:3], ref[:3]):
        assert torch.equal(a[keep], b[keep])
    assert torch.equal(got[3], ref[3]) and torch.equal(got[4], ref[4])


# ------------------------------------------------------------- together

def test_w4_repeats_streams_and_graphs(bm):
    """The same bits again, on another stream and from replayed graphs, for
    experts of one, two, a few and many rows of more than 1024 inputs."""
    g = rng(21)
    E, N, K, G = 6, 200, 2048, 64
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(E, N, K // G, generator=g, device="cuda") * 0.02).half()
    m = (s.float() * (normal(g, *s.shape) - 7.5)).half()
    for counts in ([1, 2, 2, 0, 5, 13], [1, 2, 40, 0, 70, 16]):
        bounds, R = ragged(g, E, counts)
        x = normal(g, R, K, dtype=BF16)
        ref = bm.w4_matmul(x, codes, s, m, bounds=bounds)
        sq, md = dequantized(codes, s, m, G)
        b = bounds.tolist()
        for e in range(E):
            r = x[b[e]:b[e + 1]].double()
            want = r @ (sq + md)[e].t()
            tol = r.abs() @ (sq + md.abs())[e].t() * ((K + 16) * STEP) + half_step(want, BF16)
            check(ref[b[e]:b[e + 1]], want, tol, "%d rows" % counts[e])
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        y = bm.w4_matmul(x, codes, s, m, bounds=bounds, stream=side)
        side.synchronize()
        assert torch.equal(y, ref)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = bm.w4_matmul(x, codes, s, m, bounds=bounds)
        for turn in range(3):
            y.fill_(NAN)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, ref), turn
            assert torch.equal(bm.w4_matmul(x, codes, s, m, bounds=bounds), ref)


@pytest.mark.parametrize("T", [1, 4, 8, 64])
def test_the_router_in_front_of_the_spectral_path(bm, T):
    """ids and weights of moe_route go into gate/up and down: a slot without an
    expert has NaN rows of h and adds nothing, a token without one gives zeros."""
    import numpy as np

    import synth
    from oracle import path
    from oracle.quantize import quantize_expert
    from spectral_expert_gemv_amd import DeviceLayer
    _say("router, gate/up, down", T)
    L = synth.make_layer(synth.LAYERS["tiny"])
    D, spec = synth.make_down(L), L.spec
    x, _ = synth.make_batch(synth.workload("tiny_t64"), L, step=2, T=T)
    logits = normal(rng(T), T, spec.E, dtype=F16)
    logits[T // 2] = -INF
    logits[T // 2, 1] = 0.5       # one expert: the second slot is empty
    if T > 1:
        logits[T - 1] = -INF      # none
    ids, g = bm.moe_route(logits, spec.k, renorm=True)
    assert ids[T // 2].tolist() == [1, -1] and g[T // 2].tolist() == [1.0, 0.0]
    dev = DeviceLayer.from_synth(L)
    h = dev.gateup(torch.from_numpy(np.ascontiguousarray(x)).cuda(), ids)
    assert bool(h[ids < 0].isnan().all()) and bool(h[ids >= 0].isfinite().all())
    phi16 = np.asarray(D.phi, np.float16)
    blob = torch.from_numpy(np.ascontiguousarray(bm.pack(D.p, D.a, D.bits))).cuda()
    phit = torch.from_numpy(np.ascontiguousarray(phi16.T)).cuda()
    out = bm.moe_down(blob, phit, h, ids, g, spec.E, spec.din, D.phi.shape[1]).cpu().numpy()
    i, hd = ids.cpu().numpy(), h.cpu().numpy()
    live = i >= 0
    pairs = [(int(t), int(j)) for t, j in zip(*np.nonzero(live))]
    # the bars of the gate/up and the down projection's own tests, by a row's largest value
    for (t, j), want in pairs_ref(L, x, i, pairs).items():
        assert max_rel_err(hd[t, j], want) <= 2e-3, (t, j)
    phat = np.stack([quantize_expert(D.p[e], D.bits[e])["phat"] for e in range(spec.E)])
    ref = path.moe_down(phi16, D.a, phat, D.bits, np.where(live[:, :, None], hd, 0.0), i, g.cpu().numpy())
    for t in range(T):
        assert max_rel_err(out[t], ref[t]) <= 5e-4, t
    assert T == 1 or not out[T - 1].any()


@pytest.mark.parametrize("counts, N, K", [([3, 0, 5], 40, 136), ([3, 0, 5], 33, 101), ([150, 0, 300], 40, 136), ([150, 0, 300], 33, 101),
                                          ([700, 1, 260], 264, 328)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_products_of_infinities_and_nan(bm, counts, N, K, dtype):
    """They reach the outputs that their rows reach, and no others: not by the
    rows and columns that fill up a tile."""
    _say("products of infinities", counts, N, K, dtype)
    g = rng(K)
    bounds, R = ragged(g, 3, counts, tail=2)
    n = R - 2
    x, dy, w = normal(g, R, K, dtype=dtype), normal(g, R, N, dtype=dtype), normal(g, 3, N, K, dtype=dtype)
    x[n:] = dy[n:] = NAN
    rows = {0: (K - 1, INF), counts[0] - 1: (K // 2, -INF), n - 1: (0, NAN)}
    good = bm.grouped_matmul(x, w, bounds), bm.grouped_matmul_dx(dy, w, bounds), bm.grouped_matmul_dw(dy, x, bounds)
    xb, dyb = x.clone(), dy.clone()
    for r, (c, v) in rows.items():
        xb[r, c] = dyb[r, c % N] = v
    y, dx = bm.grouped_matmul(xb, w, bounds), bm.grouped_matmul_dx(dyb, w, bounds)
    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    keep[n:] = False
    for r in rows:
        keep[r] = False
        e = 0 if r < counts[0] else 2
        for got, a, m in ((y, xb, w[e]), (dx, dyb, w[e].t())):
            want = (m.double().cpu() * a[r].double().cpu()).sum(1)  # no product is 0 but by chance
            same_kind(got[r], want, torch.zeros_like(want), "row %d" % r)
    assert torch.equal(y[keep], good[0][keep]) and torch.equal(dx[keep], good[1][keep])
    # dw: the columns of x, or the rows of dy, that hold them, of their experts alone
    for a, b, axis in ((dy, xb, 1), (dyb, x, 0)):
        dw = bm.grouped_matmul_dw(a, b, bounds)
        hit = torch.zeros_like(dw, dtype=torch.bool)
        for r, (c, v) in rows.items():
            e = 0 if r < counts[0] else 2
            hit[e].select(axis, c if axis else c % N).fill_(True)
        assert not bool(dw[hit].isfinite().any()) and torch.equal(dw[~hit], good[2][~hit])
