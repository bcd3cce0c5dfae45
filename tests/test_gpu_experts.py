"""GPU tests of the expert layer's operators against plain 64-bit
implementations.

Tolerances: an output rounded once is off by at most half a step, eps/2 of its
value (fp16: or half the subnormal step, 2^-25).  A float32 sum of n products
adds at most n 2^-23 of the sum of their magnitudes (every addition off by at
most one step, whatever the order); 2^-22 is allowed for each exp and
division.  Integers are equal.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
STEP = 2.0 ** -23


@pytest.fixture(scope="module")
def bm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from spectral_expert_gemv_amd import bitsmoe
    return bitsmoe


def _say(*a):
    print(*a, flush=True)


def rng(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def half_step(v, dtype):
    t = v.abs() * (torch.finfo(dtype).eps / 2)
    return t + 2.0 ** -25 if dtype == F16 else t


def check(got, want, tol, what=""):
    """Every element within tol (64 bits) of want."""
    got = got.double()
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), "%s: %d of %d off, worst %.3g of tol" % (
        what, int(bad.sum()), bad.numel(),
        float(((got - want).abs() / tol.clamp(min=1e-300)).nan_to_num(1e9).max()))


# ---------------------------------------------------------------- routing

def plain_route(l, k, renorm, scale):
    """ids, g and the choice in 64 bits, on the host."""
    l = l.double().cpu()
    order = torch.sort(l, dim=1, descending=True, stable=True)
    v, ids = order.values[:, :k], order.indices[:, :k]
    dead = torch.isinf(v) & (v < 0)
    p = torch.softmax(l, 1).nan_to_num(0.0) if bool((l > -float("inf")).any()) else torch.zeros_like(l)
    g = p.gather(1, ids)
    if renorm:
        tot = g.sum(1, keepdim=True)
        g = torch.where(tot > 0, g / tot.clamp(min=1e-300), torch.zeros_like(g))
    g = torch.where(dead, torch.zeros_like(g), g * scale)
    return torch.where(dead, torch.full_like(ids, -1), ids).int(), g


def plain_group(ids, E):
    flat = ids.cpu().reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.sort(key, stable=True).indices
    bounds = torch.tensor([int((key < e).sum()) for e in range(E + 1)], dtype=torch.int32)
    slot = torch.empty_like(order)
    slot[order] = torch.arange(order.numel())
    slot[key == E] = -1
    order[bounds[E]:] = -1
    return bounds, order.int(), slot.int().reshape(ids.shape)


@pytest.mark.parametrize("T, E, k", [(1, 1, 1), (1, 8, 2), (1, 128, 8), (3, 5, 5), (17, 16, 16), (64, 60, 4),
                                     (67, 129, 8), (33, 256, 16), (5, 256, 17), (9, 257, 6), (130, 512, 10),
                                     (4, 1000, 64), (3, 2048, 64), (1000, 64, 6), (5000, 128, 8)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("renorm", [False, True])
def test_route(bm, T, E, k, dtype, renorm):
    _say("route", T, E, k, dtype, renorm)
    g = rng(T * 7 + E)
    logits = normal(g, T, E + 3, scale=3.0)
    if E > 4:
        logits[:, 2] = -float("inf")
        logits[:, 1] = logits[:, 0]       # ties
        logits[T // 2, :] = -float("inf")  # nothing to choose
        logits[T // 3, 1:] = -float("inf")  # one expert left
        logits[T - 1, :E] = 0.0
        logits[T - 1, ::2] = -0.0         # all tie, -0 with +0
    logits = logits.to(dtype)[:, :E]      # rows of another stride
    ids, gates = bm.moe_route(logits, k, renorm=renorm, scale=2.5)
    wi, wg = plain_route(logits, k, renorm, 2.5)
    assert torch.equal(ids.cpu(), wi)
    # E additions, an exp and a division; the exponent l - max is off by half a step of up to 32
    check(gates.cpu(), wg, wg * (E * STEP + 2.0 ** -19) + 1e-30, "g")
    bounds = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    order = torch.empty(T * k, dtype=torch.int32, device="cuda")
    slot = torch.empty(T, k, dtype=torch.int32, device="cuda")
    i2, g2 = bm.moe_route(logits, k, renorm=renorm, scale=2.5, bounds=bounds, order=order, slot=slot)
    assert torch.equal(i2, ids) and torch.equal(g2, gates)
    for got, want in zip((bounds, order, slot), plain_group(wi, E)):
        assert torch.equal(got.cpu(), want)

    dg = normal(g, T, k)
    d = bm.moe_route_grad(logits, ids, dg, renorm=renorm, scale=2.5)
    l = logits.double()
    ok = ids >= 0
    pos = ids.long().clamp(min=0)
    top = l.max(1, keepdim=True).values.clamp(min=-1e30)
    e = torch.exp(l - top)
    c = torch.zeros_like(l).scatter_add_(1, pos, ok.double()) if renorm else torch.ones_like(l)
    w = c * e
    w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    q = torch.zeros_like(l).scatter_add_(1, pos, torch.where(ok, dg.double() * 2.5, 0.0))
    want = w * (q - (w * q).sum(1, keepdim=True))
    size = w * (q.abs() + (w * q.abs()).sum(1, keepdim=True))
    check(d, want, half_step(want, dtype) + size * (E * STEP + 2.0 ** -18) + 1e-30, "dlogits")


def test_route_gradient_by_differences(bm):
    """The formula's gradient against central differences of a 64-bit forward."""
    g = rng(5)
    l = normal(g, 6, 24)
    dg = normal(g, 6, 4)
    for renorm in (False, True):
        ids, _ = bm.moe_route(l, 4, renorm=renorm, scale=1.5)
        d = bm.moe_route_grad(l, ids, dg, renorm=renorm, scale=1.5).double().cpu()

        def loss(v):
            p = torch.softmax(v, 1).gather(1, ids.long().cpu())
            p = p / p.sum(1, keepdim=True) if renorm else p
            return (1.5 * p * dg.double().cpu()).sum()
        base, h = l.double().cpu(), 1e-4
        for t, e in [(0, int(ids[0, 0])), (1, 3), (2, int(ids[2, 3])), (5, 23)]:
            up, dn = base.clone(), base.clone()
            up[t, e] += h
            dn[t, e] -= h
            # central differences: error h^2 / 6 times a third derivative of order 10
            assert abs((loss(up) - loss(dn)) / (2 * h) - d[t, e]) < 1e-6


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_route_row_without_a_softmax(bm, bad):
    l = normal(rng(1), 20, 40)
    l[7, 11] = bad
    ids, g = bm.moe_route(l, 3)
    assert bool((ids[7] == -1).all()) and bool(g[7].isnan().all())
    keep = torch.arange(20, device="cuda") != 7
    wi, _ = plain_route(l[keep], 3, False, 1.0)
    assert torch.equal(ids[keep].cpu(), wi) and bool(g[keep].isfinite().all())
    d = bm.moe_route_grad(l, ids, torch.ones_like(g))
    assert bool(d[7].isnan().all()) and bool(d[keep].isfinite().all())


@pytest.mark.parametrize("P, E", [(1, 1), (63, 7), (64, 128), (65, 128), (1025, 512), (4096, 512), (4097, 3),
                                  (4100, 600), (50000, 128), (70001, 2048), (300000, 64)])
def test_group(bm, P, E):
    _say("group", P, E)
    ids = torch.randint(-2, E + 2, (P, 1), generator=rng(P), device="cuda", dtype=torch.int32)
    if P > 5000:
        ids[1000:3000] = E // 2  # a long run of one expert
    for got, want in zip(bm.moe_group(ids, E), plain_group(ids, E)):
        assert torch.equal(got.cpu(), want)


def test_group_of_nothing(bm):
    ids = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    bounds, order, slot = bm.moe_group(ids, 5)
    assert bounds.tolist() == [0] * 6 and order.numel() == 0
    bounds, order, slot = bm.moe_group(torch.full((70, 2), -1, dtype=torch.int32, device="cuda"), 5)
    assert bounds.tolist() == [0] * 6 and bool((order == -1).all()) and bool((slot == -1).all())


# ------------------------------------------------------------- activation

@pytest.mark.parametrize("R, F", [(1, 1), (1, 8), (5, 7), (67, 768), (1000, 1408), (33, 4133), (4097, 64)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("layout", ["plain", "strided", "shifted"])
def test_silu_mul(bm, R, F, dtype, layout):
    _say("silu_mul", R, F, dtype, layout)
    g = rng(R + F)
    pad, at = {"plain": (0, 0), "strided": (8, 0), "shifted": (9, 3)}[layout]
    a = normal(g, R, 2 * F + pad, dtype=dtype, scale=3.0)[:, at:at + 2 * F]
    a[0, 0] = -60.0 if dtype == F16 else -200.0
    h = torch.full((R, F + pad), 7.0, dtype=dtype, device="cuda")[:, at:at + F]
    assert bm.silu_mul(a, h) is h
    x, u = a.double()[:, :F], a.double()[:, F:]
    s = torch.sigmoid(x)
    want = x * s * u
    check(h, want, half_step(want, dtype) + want.abs() * 2.0 ** -20 + 1e-37, "h")
    dh = normal(g, R, F, dtype=dtype)
    da = bm.silu_mul_grad(a, dh)
    d = dh.double()
    wg, wu = d * u * s * (1 + x * (1 - s)), d * x * s
    size = (d * u * s).abs() * (1 + (x * (1 - s)).abs())
    check(da[:, :F], wg, half_step(wg, dtype) + size * 2.0 ** -20 + 1e-37, "dgate")
    check(da[:, F:], wu, half_step(wu, dtype) + wu.abs() * 2.0 ** -20 + 1e-37, "dup")
    b = a.clone()
    assert torch.equal(bm.silu_mul_grad(b, dh, b), da)  # in place


def test_silu_mul_leaves_rows_past_the_experts(bm):
    a = normal(rng(2), 50, 64, dtype=BF16)
    bounds = torch.tensor([0, 11, 37], dtype=torch.int32, device="cuda")
    h = torch.full((50, 32), 7.0, dtype=BF16, device="cuda")
    bm.silu_mul(a, h, bounds=bounds)
    assert torch.equal(h[:37], bm.silu_mul(a)[:37]) and bool((h[37:] == 7).all())
    da = torch.full((50, 64), 7.0, dtype=BF16, device="cuda")
    dh = normal(rng(3), 50, 32, dtype=BF16)
    bm.silu_mul_grad(a, dh, da, bounds=bounds)
    assert torch.equal(da[:37], bm.silu_mul_grad(a, dh)[:37]) and bool((da[37:] == 7).all())


# ---------------------------------------------------------------- combine

def plain_combine(y, slot, g):
    at = slot.long().clamp(min=0)
    there = ((slot >= 0) & (slot < y.shape[0])).double()
    rows = y.double()[at.clamp(max=y.shape[0] - 1)]
    return rows, there * (1.0 if g is None else g.double())


@pytest.mark.parametrize("T, k, D", [(1, 1, 1), (1, 8, 2048), (7, 3, 65), (32, 8, 2048), (500, 6, 1408), (9, 17, 4096),
                                     (3, 64, 4133), (2000, 2, 96)])
@pytest.mark.parametrize("dtype, out", [(F16, F32), (F16, F16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("pad", [0, 5])
def test_combine(bm, T, k, D, dtype, out, pad):
    _say("combine", T, k, D, dtype, out, pad)
    g = rng(T + D)
    R = T * k + 2
    y = normal(g, R, D + pad, dtype=dtype)[:, :D]
    slot = torch.randperm(R, generator=g, device="cuda")[:T * k].reshape(T, k).int()
    slot[0, 0] = -1
    slot[T - 1, k - 1] = R + 7  # as an id that is not an expert
    gates = torch.rand(T, k, generator=g, device="cuda")
    o = bm.moe_combine(y, slot, gates, torch.empty(T, D + pad, dtype=out, device="cuda")[:, :D])
    rows, w = plain_combine(y, slot, gates)
    want, size = (rows * w[:, :, None]).sum(1), (rows * w[:, :, None]).abs().sum(1)
    check(o, want, half_step(want, out) + size * (k + 1) * STEP, "out")
    rows, w1 = plain_combine(y, slot, None)
    want, size = (rows * w1[:, :, None]).sum(1), (rows * w1[:, :, None]).abs().sum(1)
    check(bm.moe_combine(y, slot, None, o), want, half_step(want, out) + size * (k + 1) * STEP, "sum")

    dout = normal(g, T, D, dtype=out)
    dy = torch.full((R, D), 7.0, dtype=dtype, device="cuda")
    _, dg = bm.moe_combine_grad(dout, y, slot, gates, dy)
    want = torch.full((R, D), 7.0, dtype=torch.float64, device="cuda")
    ok = (slot >= 0) & (slot < R)
    want[slot[ok].long()] = (gates.double()[:, :, None] * dout.double()[:, None, :])[ok]
    check(dy, want, half_step(want, dtype) + want.abs() * STEP, "dy")
    want = torch.where(ok, (rows * dout.double()[:, None, :]).sum(2), 0.0)
    size = (rows * dout.double()[:, None, :]).abs().sum(2)
    check(dg, want, half_step(want, F32) + size * D * STEP, "dg")


# --------------------------------------------------- products by expert

def plain_silu_mul_bounds(v, dv):
    """SiLU(gate) * up of [gate | up] in 64 bits and how far errors dv of its
    inputs can move it (|SiLU'| <= 1.1)."""
    F = v.shape[1] // 2
    g, u, dg, du = v[:, :F], v[:, F:], dv[:, :F], dv[:, F:]
    s = torch.nn.functional.silu(g)
    return s * u, 1.1 * u.abs() * dg + s.abs() * du + 1.1 * dg * du + (s * u).abs() * 2.0 ** -20


def ragged(g, E, counts, tail=0):
    """bounds for the counts, and R with `tail` rows past the last expert."""
    b = torch.tensor([0] + list(counts), dtype=torch.int32).cumsum(0).int()
    assert len(counts) == E
    return b.cuda(), int(b[-1]) + tail


SHAPES = [
    # E, counts, N, K: one row, empty experts, odd sizes, tile edges, long rows
    (1, [1], 1, 1),
    (1, [1], 64, 64),
    (3, [0, 5, 0], 40, 72),
    (4, [1, 0, 17, 2], 33, 31),
    (8, [1] * 8, 96, 256),
    (5, [16, 15, 17, 0, 33], 128, 264),
    (2, [64, 65], 256, 64),
    (2, [128, 129], 257, 520),
    (3, [200, 0, 77], 136, 1032),
    (2, [255, 300], 512, 192),
    (1, [513], 264, 776),
    (130, [(i * 7) % 5 for i in range(130)], 48, 128),
    (2, [700, 3], 1408, 2048),
    (16, [(i * 37) % 130 for i in range(16)], 768, 512),
]


@pytest.mark.parametrize("E, counts, N, K", SHAPES)
@pytest.mark.parametrize("dtype, out", [(F16, F16), (BF16, BF16), (F16, F32), (BF16, F32)])
def test_grouped_matmul(bm, E, counts, N, K, dtype, out):
    _say("grouped_matmul", E, sum(counts), N, K, dtype, out)
    g = rng(N + K)
    bounds, R = ragged(g, E, counts, tail=3)
    x = normal(g, R, K, dtype=dtype)
    w = normal(g, E, 2 * N, K, dtype=dtype, scale=K ** -0.5)
    w1 = w[:, :N].contiguous()
    n = R - 3
    e = torch.repeat_interleave(torch.arange(E), torch.tensor(counts)).cuda()
    k = 3
    xs = normal(g, R, K, dtype=dtype)  # gathered: pair p reads token p // 3
    order = torch.randperm(3 * R, generator=g, device="cuda")[:R].int()

    def want(rows, w):
        v = torch.zeros(n, w.shape[1], dtype=torch.float64, device="cuda")
        d = torch.zeros_like(v)
        for i in range(E):
            at = e == i
            v[at] = rows[at].double() @ w[i].double().t()
            d[at] = rows[at].double().abs() @ w[i].double().abs().t() * (K * STEP)
        return v, d

    y = torch.full((R, N), 7.0, dtype=out, device="cuda")
    bm.grouped_matmul(x, w1, bounds, y)
    v, d = want(x[:n], w1)
    check(y[:n], v, half_step(v, out) + d, "y")
    assert bool((y[n:] == 7).all())

    y = torch.full((R, N + 8), 7.0, dtype=out, device="cuda")
    bm.grouped_matmul(xs, w1, bounds, y[:, :N], order, k)
    v, d = want(xs[(order.long() // k)[:n]], w1)
    check(y[:n, :N], v, half_step(v, out) + d, "gathered")
    assert bool((y[n:] == 7).all()) and bool((y[:, N:] == 7).all())

    y = torch.full((R, N), 7.0, dtype=out, device="cuda")
    bm.grouped_matmul(xs, w, bounds, y, order, k, "silu_mul")
    v, d = want(xs[(order.long() // k)[:n]], w)
    v, d = plain_silu_mul_bounds(v, d)
    check(y[:n], v, half_step(v, out) + d + 1e-37, "silu_mul")
    assert bool((y[n:] == 7).all())


@pytest.mark.parametrize("E, counts, N, K", SHAPES)
@pytest.mark.parametrize("dtype, out", [(F16, F16), (BF16, F32), (BF16, BF16)])
def test_grouped_matmul_gradients(bm, E, counts, N, K, dtype, out):
    _say("grouped_matmul_dx, dw", E, sum(counts), N, K, dtype, out)
    g = rng(N + K + 1)
    bounds, R = ragged(g, E, counts, tail=2)
    n = R - 2
    w = normal(g, E, N, K, dtype=dtype, scale=N ** -0.5)
    dy, x = normal(g, R, N, dtype=dtype), normal(g, R, K, dtype=dtype)
    dy[n:] = float("nan")  # rows past the experts are not read
    x[n:] = float("nan")
    b = bounds.tolist()
    dx = torch.full((R, K), 7.0, dtype=out, device="cuda")
    bm.grouped_matmul_dx(dy, w, bounds, dx)
    dw = torch.full((E, N, K), 7.0, dtype=out, device="cuda")
    bm.grouped_matmul_dw(dy, x, bounds, dw)
    order = torch.randperm(2 * R, generator=g, device="cuda")[:R].int()
    xs = normal(g, R, K, dtype=dtype)
    dws = bm.grouped_matmul_dw(dy, xs, bounds, torch.full_like(dw, 7.0), order, 2)
    for i in range(E):
        at = slice(b[i], b[i + 1])
        d, v = dy[at].double(), w[i].double()
        check(dx[at], d @ v, half_step(d @ v, out) + d.abs() @ v.abs() * (N * STEP), "dx")
        for got, rows in ((dw, x[at]), (dws, xs[(order.long() // 2)[at]])):
            r = rows.double()
            want = d.t() @ r
            check(got[i], want, half_step(want, out) + d.abs().t() @ r.abs() * (counts[i] * STEP),
                  "dw of expert %d" % i)
    assert bool((dx[n:] == 7).all())


# E, rows of expert i, N, K: tiles of 256 x 256 that make a round and more, and
# left-overs that are cut in four (60, 30), in two (104, 120, 90, 88) or not (130,
# 234, 182), forward, with the activation, dx and dw
ROUNDS = [(24, 53, 300, 1032, 1032), (24, 53, 300, 776, 776), (16, 97, 290, 1000, 1288),
          (20, 71, 520, 1100, 1290), (24, 53, 300, 2568, 520)]


@pytest.mark.parametrize("E, step, most, N, K", ROUNDS)
@pytest.mark.parametrize("dtype, out", [(BF16, BF16), (F16, F32)])
def test_grouped_matmul_rounds_of_tiles(bm, E, step, most, N, K, dtype, out):
    counts = [i * step % most for i in range(E)]
    test_grouped_matmul(bm, E, counts, N, K, dtype, out)
    test_grouped_matmul_gradients(bm, E, counts, N, K, dtype, out)


@pytest.mark.parametrize("N, K", [(96, 256), (40, 31)])
def test_grouped_matmul_strides_and_bad_rows(bm, N, K):
    g = rng(4)
    bounds, R = ragged(g, 3, [20, 3, 40])
    w = normal(g, 3, N, K, dtype=BF16)
    x = normal(g, 30, K, dtype=BF16)
    order = torch.randint(0, 60, (R,), generator=g, device="cuda", dtype=torch.int32)
    good = bm.grouped_matmul(x, w, bounds, rows=order, div=2)
    for pad, at in ((8, 8), (3, 1), (1, 0)):  # strides that are and are not multiples of 16 bytes
        xs = torch.full((30, K + pad), float("nan"), dtype=BF16, device="cuda")[:, at:at + K]
        xs.copy_(x)
        ys = torch.full((R, N + pad), 7.0, dtype=BF16, device="cuda")
        bm.grouped_matmul(xs, w, bounds, ys[:, at:at + N], rows=order, div=2)
        v = x[order.long() // 2].double()
        tol = torch.cat([v[a:b].abs() @ w[i].double().abs().t() for i, (a, b) in
                         enumerate(zip(bounds[:-1].tolist(), bounds[1:].tolist()))]) * (K * STEP)
        check(ys[:, at:at + N], good.double(), tol + half_step(good.double(), BF16) * 2.0, "strided")
        keep = torch.ones(N + pad, dtype=torch.bool)
        keep[at:at + N] = False
        assert bool((ys[:, keep] == 7).all())
    bad = order.clone()
    bad[[0, 21, 62]] = torch.tensor([-1, 60, 1 << 30], dtype=torch.int32, device="cuda")
    y = bm.grouped_matmul(x, w, bounds, rows=bad, div=2)
    hit = torch.zeros(R, dtype=torch.bool, device="cuda")
    hit[[0, 21, 62]] = True
    assert bool(y[hit].isnan().all()) and torch.equal(y[~hit], good[~hit])
    dy = normal(g, R, N, dtype=BF16)
    bad[21] = order[21]
    dw = bm.grouped_matmul_dw(dy, x, bounds, rows=bad, div=2)
    ok = bm.grouped_matmul_dw(dy, x, bounds, rows=order, div=2)
    assert bool(dw[[0, 2]].isnan().all()) and torch.equal(dw[1], ok[1])


def test_grouped_matmul_wrong_bounds_stay_inside(bm):
    """Bounds that fall, or lie outside the rows, are clamped: the call returns
    and leaves what surrounds its output alone."""
    g = rng(9)
    w = normal(g, 4, 64, 128, dtype=F16)
    x = normal(g, 40, 128, dtype=F16)
    y = torch.full((60, 64), 7.0, dtype=F16, device="cuda")
    for b in ([0, 30, 10, 50, 90], [-5, -1, 20, 15, 40], [40, 0, 0, 0, 0]):
        bounds = torch.tensor(b, dtype=torch.int32, device="cuda")
        bm.grouped_matmul(x, w, bounds, y[10:50])
        bm.grouped_matmul_dx(x[:, :64], w, bounds)
        bm.grouped_matmul_dw(x[:, :64], x, bounds)
        torch.cuda.synchronize()
        assert bool((y[:10] == 7).all()) and bool((y[50:] == 7).all())


# ------------------------------------------------------- 4-bit weights

W4_SHAPES = [
    # E, counts, N, K, G
    (1, [1], 1, 32, 32),
    (1, [1], 64, 128, 128),
    (1, [1], 1000, 2048, 64),
    (1, [5], 33, 96, 32),
    (1, [17], 130, 1024, 128),
    (1, [300], 200, 640, 64),
    (4, [1, 0, 1, 1], 96, 256, 128),
    (3, [0, 70, 2], 40, 192, 64),
    (16, [(i * 5) % 9 for i in range(16)], 77, 512, 32),
    (2, [130, 1], 48, 4096, 128),
]


@pytest.mark.parametrize("E, counts, N, K, G", W4_SHAPES)
@pytest.mark.parametrize("dtype, out", [(F16, F16), (BF16, BF16), (F16, F32), (BF16, F32)])
@pytest.mark.parametrize("symmetric", [False, True])
def test_w4_matmul(bm, E, counts, N, K, G, dtype, out, symmetric):
    _say("w4", E, sum(counts), N, K, G, dtype, out, symmetric)
    g = rng(N + K + G)
    bounds, R = ragged(g, E, counts, tail=2 if E > 1 else 0)
    n = sum(counts)
    codes = torch.randint(0, 256, (E, 2 * N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = ((torch.rand(E, 2 * N, K // G, generator=g, device="cuda") + 0.5) * K ** -0.5).half()
    m = None if symmetric else (s.float() * (normal(g, *s.shape) - 7.5)).half()
    q = torch.stack([codes & 15, codes >> 4], -1).reshape(E, 2 * N, K).double()
    sd = s.double().repeat_interleave(G, 2)
    md = -8 * sd if symmetric else m.double().repeat_interleave(G, 2)
    w, size = sd * q + md, sd * q + md.abs()
    x = normal(g, R, K, dtype=dtype)
    xs = normal(g, R, K, dtype=dtype)
    order = torch.randperm(2 * R, generator=g, device="cuda")[:R].int()
    b = bounds.tolist()

    def want(rows, lo, hi):
        v, d = [], []
        for i in range(E):
            r = rows[b[i]:b[i + 1]].double()
            v.append(r @ w[i, lo:hi].t())
            # the two sums of a group are of the size of s q and |m| alone; s q may come as
            # s (q + 16) less 16 s, which is at most 32 s
            d.append(r.abs() @ (size[i, lo:hi] + 32 * sd[i, lo:hi]).t() * (K * STEP))
        return torch.cat(v), torch.cat(d)

    half = lambda t: None if t is None else t[:, :N].contiguous()  # noqa: E731
    y = torch.full((R, N + 8), 7.0, dtype=out, device="cuda")
    bm.w4_matmul(x, half(codes), half(s), half(m), y[:, :N], bounds)
    v, d = want(x, 0, N)
    check(y[:n, :N], v, half_step(v, out) + d, "y")
    assert bool((y[n:] == 7).all()) and bool((y[:, N:] == 7).all())
    if E == 1:
        y2 = bm.w4_matmul(x, codes[0, :N], s[0, :N], None if m is None else m[0, :N],
                          torch.empty(R, N, dtype=out, device="cuda"))
        assert torch.equal(y2, y[:, :N])
    y = torch.full((R, N), 7.0, dtype=out, device="cuda")
    bm.w4_matmul(xs, codes, s, m, y, bounds, order, 2, "silu_mul")
    v, d = want(xs[order.long() // 2], 0, 2 * N)
    v, d = plain_silu_mul_bounds(v, d)
    check(y[:n], v, half_step(v, out) + d + 1e-37, "silu_mul")
    assert bool((y[n:] == 7).all())


def test_w4_of_packed_weights_bad_rows_and_strides(bm):
    g = rng(12)
    w = torch.randn(50, 256, generator=torch.Generator().manual_seed(3))
    codes, s, m = (torch.from_numpy(a).cuda() for a in bm.w4_pack(w.numpy(), 64))
    x = torch.full((9, 264), float("nan"), dtype=F16, device="cuda")[:, 8:]
    x.copy_(normal(g, 9, 256))
    y = bm.w4_matmul(x, codes, s, m)
    step = s.float().repeat_interleave(64, 1)
    # a code is off by half a step of its group, the minimum by half a step of float16
    off = x.float().abs() @ (0.51 * step + 4.0 * 2 ** -11).cuda().t() + 0.01
    assert bool(((y.float() - x.float() @ w.cuda().t()).abs() <= off).all())
    bounds = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    rows = torch.arange(9, dtype=torch.int32, device="cuda")
    rows[[2, 5]] = torch.tensor([-1, 9], dtype=torch.int32, device="cuda")
    got = bm.w4_matmul(x, codes, s, m, bounds=bounds, rows=rows)
    hit = (rows < 0) | (rows > 8)
    assert bool(got[hit].isnan().all()) and torch.equal(got[~hit], y[~hit])
    for pad in (1, 4):  # rows that are not 16-byte aligned
        odd = torch.full((9, 256 + pad), float("nan"), dtype=F16, device="cuda")[:, pad:]
        odd.copy_(x)
        check(bm.w4_matmul(odd, codes, s, m), y.double(), half_step(y.double(), F16) * 2 + 256 * STEP * 100, "odd")


# ----------------------------------------------------------- together

def layer_inputs(T, E, k, D, F, dtype, seed):
    g = rng(seed)
    logits = normal(g, T, E, scale=2.0)
    logits[:, E // 2] = -float("inf")
    x = normal(g, T, D, dtype=dtype)
    w1 = normal(g, E, 2 * F, D, dtype=dtype, scale=D ** -0.5)
    w2 = normal(g, E, D, F, dtype=dtype, scale=F ** -0.5)
    dout = normal(g, T, D)
    return logits, x, w1, w2, dout


def layer_step(bm, logits, x, w1, w2, dout, k):
    """Forward and backward of a mixture-of-experts layer."""
    T, E = logits.shape
    D, F = w2.shape[1], w2.shape[2]
    i32 = dict(dtype=torch.int32, device=x.device)
    b, o, s = torch.empty(E + 1, **i32), torch.empty(T * k, **i32), torch.empty(T, k, **i32)
    ids, g = bm.moe_route(logits, k, renorm=True, bounds=b, order=o, slot=s)
    a = bm.grouped_matmul(x, w1, b, rows=o, div=k)
    h = bm.silu_mul(a, bounds=b)
    y = bm.grouped_matmul(h, w2, b)
    out = bm.moe_combine(y, s, g, torch.empty(T, D, device=x.device))
    dy, dg = bm.moe_combine_grad(dout, y, s, g)
    dh, dw2 = bm.grouped_matmul_dx(dy, w2, b), bm.grouped_matmul_dw(dy, h, b)
    da = bm.silu_mul_grad(a, dh, bounds=b)
    dxr, dw1 = bm.grouped_matmul_dx(da, w1, b), bm.grouped_matmul_dw(da, x, b, rows=o, div=k)
    dx = bm.moe_combine(dxr, s, None, torch.empty(T, D, device=x.device))
    dl = bm.moe_route_grad(logits, ids, dg, renorm=True)
    return out, dx, dw1, dw2, dl


@pytest.mark.parametrize("T, E, k, D, F", [(1, 8, 2, 64, 96), (37, 8, 2, 64, 96), (300, 16, 4, 256, 128)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_a_layer_and_its_gradients(bm, T, E, k, D, F, dtype):
    """The run of all operators against automatic differentiation of the same
    layer in 64 bits (written with dense one-hot products)."""
    _say("layer", T, E, k, D, F, dtype)
    logits, x, w1, w2, dout = layer_inputs(T, E, k, D, F, dtype, 31)
    got = layer_step(bm, logits, x, w1, w2, dout, k)
    leaves = [t.double().requires_grad_() for t in (logits, x, w1, w2)]
    l, xd, v1, v2 = leaves
    p = torch.softmax(l, 1)
    top = torch.topk(logits, k, 1).indices
    g = p.gather(1, top)
    g = g / g.sum(1, keepdim=True)
    gate = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter(1, top, g)
    out = 0
    for e in range(E):
        a = xd @ v1[e].t()
        out = out + gate[:, e:e + 1] * ((torch.nn.functional.silu(a[:, :F]) * a[:, F:]) @ v2[e].t())
    out.backward(dout.double())
    want = (out.detach(), xd.grad, v1.grad, v2.grad, l.grad.nan_to_num(0.0))
    # five roundings to 16 bits lie one after another on the longest way; each is half a
    # step of a value, so relative to the norm 5 half steps, times 2 for products of two
    # rounded factors
    tol = 10 * torch.finfo(dtype).eps / 2
    for name, a, b in zip(("out", "dx", "dw1", "dw2", "dlogits"), got, want):
        err = float((a.double() - b).norm() / b.norm())
        assert err < tol, (name, err, tol)


@pytest.mark.parametrize("T, E, k, D, F", [(1, 8, 2, 64, 96), (50, 16, 4, 256, 128), (300, 4, 2, 128, 64)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("on_stream", [False, True])
def test_expert_layer(bm, T, E, k, D, F, dtype, on_stream):
    """The layer's own forward passes (dense and 4-bit) and gradients."""
    from spectral_expert_gemv_amd import ExpertLayer
    _say("ExpertLayer", T, E, k, D, F, dtype, on_stream)
    logits, x, w1, w2, dout = layer_inputs(T, E, k, D, F, dtype, 17)
    dout = dout.to(dtype)
    stream = torch.cuda.Stream() if on_stream else None
    torch.cuda.synchronize()
    layer = ExpertLayer(w1, w2)
    out = layer.forward(x, logits, k, stream=stream)
    got = layer.gradients(x, logits, k, dout, stream=stream)
    packed = ExpertLayer.w4(w1.float().cpu().numpy(), w2.float().cpu().numpy(), group=32)
    q = packed.forward(x, logits, k, torch.empty(T, D, dtype=F32, device="cuda"), stream=stream)
    torch.cuda.synchronize()

    def plain(v1, v2):
        p = torch.softmax(logits.double(), 1)
        top = torch.topk(logits, k, 1).indices
        g = p.gather(1, top)
        gate = torch.zeros_like(p).scatter(1, top, g / g.sum(1, keepdim=True))
        o = 0
        for e in range(E):
            a = x.double() @ v1[e].double().t()
            h = torch.nn.functional.silu(a[:, :F]) * a[:, F:]
            o = o + gate[:, e:e + 1] * (h @ v2[e].double().t())
        return o

    def deq(w):
        codes, s, m = w
        c = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], codes.shape[1], -1).double()
        return c * s.double().repeat_interleave(32, 2) + m.double().repeat_interleave(32, 2)

    # the longest way has h, y and out rounded: 3 half steps, doubled as before
    tol = 6 * torch.finfo(dtype).eps / 2
    for o, want in ((out, plain(w1, w2)), (got[0], plain(w1, w2)), (q, plain(deq(packed.w1), deq(packed.w2)))):
        assert float((o.double() - want).norm() / want.norm()) < tol
    ref = layer_step(bm, logits, x, w1, w2, dout, k)
    for a, b in ((got[2], ref[4]), (got[3], ref[2]), (got[4], ref[3])):
        assert torch.equal(a, b)
    # dx is rounded to the rows' type here, to float32 there
    assert float((got[1].double() - ref[1].double()).norm() / ref[1].double().norm()) < tol
    with pytest.raises(ValueError, match="gradients"):
        packed.gradients(x, logits, k, dout)


def test_streams_graphs_and_repeats(bm):
    """The same bits eagerly, again, on another stream and from a replayed
    graph with eager work between the replays."""
    logits, x, w1, w2, dout = layer_inputs(200, 16, 4, 256, 128, BF16, 8)
    ref = layer_step(bm, logits, x, w1, w2, dout, 4)
    for a, b in zip(layer_step(bm, logits, x, w1, w2, dout, 4), ref):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer_step(bm, logits, x, w1, w2, dout, 4)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer_step(bm, logits, x, w1, w2, dout, 4)
    for turn in range(3):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            assert torch.equal(a, b), turn
        layer_step(bm, logits * 0.5, x, w1, w2, dout, 4)
        torch.cuda.synchronize()


def test_an_explicit_stream(bm):
    logits, x, w1, w2, _ = layer_inputs(600, 16, 8, 256, 128, F16, 9)
    ids, g = bm.moe_route(logits, 8)
    b, o, s = bm.moe_group(ids, 16)
    y = bm.grouped_matmul(x, w1, b, rows=o, div=8, act="silu_mul")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        i2, g2 = bm.moe_route(logits, 8, stream=stream)
        b2, o2, s2 = bm.moe_group(i2, 16, stream=stream)
        y2 = bm.grouped_matmul(x, w1, b2, rows=o2, div=8, act="silu_mul", stream=stream)
        side.synchronize()
        assert torch.equal(i2, ids) and torch.equal(o2, o) and torch.equal(y2, y)


@pytest.mark.parametrize("T", [0, 1, 9])
def test_batches_of_padding(bm, T):
    """No token at all, and tokens without any expert."""
    from spectral_expert_gemv_amd import ExpertLayer
    _, x, w1, w2, dout = layer_inputs(max(T, 1), 8, 2, 64, 96, BF16, 3)
    x, dout = x[:T], dout[:T].to(BF16)
    logits = torch.full((T, 8), -float("inf"), device="cuda")
    layer = ExpertLayer(w1, w2)
    assert layer.forward(x, logits, 2).tolist() == [[0.0] * 64] * T
    out, dx, dl, dw1, dw2 = layer.gradients(x, logits, 2, dout)
    for t, shape in ((out, (T, 64)), (dx, (T, 64)), (dl, (T, 8)), (dw1, w1.shape), (dw2, w2.shape)):
        assert t.shape == shape and not bool(t.any())
    q = ExpertLayer.w4(w1.float().cpu().numpy(), w2.float().cpu().numpy(), group=32)
    assert not bool(q.forward(x, logits, 2).any())


def test_two_streams_at_once(bm):
    """Calls of different sizes and data, interleaved on two streams."""
    jobs = []
    for i, (T, E, k) in enumerate([(300, 16, 4), (700, 16, 4)]):
        args = layer_inputs(T, E, k, 256, 128, BF16, 40 + i)
        jobs.append((torch.cuda.Stream(), args, k, layer_step(bm, *args, k)))
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for stream, args, k, _ref in jobs:
            with torch.cuda.stream(stream):
                got.append(layer_step(bm, *args, k))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for a, b in zip(g, jobs[i % 2][3]):
            assert torch.equal(a, b), i


def test_two_graphs_replayed_in_turn(bm):
    a_args = layer_inputs(64, 16, 4, 256, 128, F16, 50)
    b_args = layer_inputs(2000, 16, 4, 256, 128, F16, 51)
    refs = [layer_step(bm, *args, 4) for args in (a_args, b_args)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for args in (a_args, b_args):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer_step(bm, *args, 4))
        graphs.append(g)
    for turn in range(3):
        for g in graphs:
            g.replay()
        layer_step(bm, *a_args, 4)
        torch.cuda.synchronize()
        for got, ref in zip(outs, refs):
            for x, y in zip(got, ref):
                assert torch.equal(x, y), turn


def test_offsets_past_32_bits(bm):
    """Weights, rows and gradients of more than 2^31 elements, looked at where
    they end."""
    E, N, K = 5, 16384, 32768
    g = rng(60)
    w = torch.empty(E, N, K, dtype=BF16, device="cuda").uniform_(-0.01, 0.01, generator=g)
    counts = [2, 0, 40, 0, 70]  # the few-rows and the tiled kernel's range
    bounds, R = ragged(g, E, counts)
    x = normal(g, 70000, K, dtype=BF16)
    rows = torch.randint(69000, 70000, (R,), generator=g, device="cuda", dtype=torch.int32)
    dy = normal(g, R, N, dtype=BF16)
    at = slice(R - 70, R)
    xe = x[rows[at].long()].double()
    we = w[4, N - 300:].double()
    y = bm.grouped_matmul(x, w, bounds, rows=rows)
    want = xe @ we.t()
    check(y[at, N - 300:], want, half_step(want, BF16) + xe.abs() @ we.abs().t() * (K * STEP), "y")
    two = torch.tensor([0, 0, 0, 0, 0, 3], dtype=torch.int32, device="cuda")
    few = bm.grouped_matmul(x, w, two, rows=rows[at][:3].contiguous())
    check(few[:, N - 300:], want[:3], half_step(want[:3], BF16) + (xe.abs() @ we.abs().t())[:3] * (K * STEP), "few")
    dx = bm.grouped_matmul_dx(dy, w, bounds)
    d, wc = dy[at].double(), w[4, :, K - 200:].double()
    want = d @ wc
    check(dx[at, K - 200:], want, half_step(want, BF16) + d.abs() @ wc.abs() * (N * STEP), "dx")
    dw = bm.grouped_matmul_dw(dy, x, bounds, torch.empty_like(w), rows)
    want = d[:, N - 300:].t() @ xe
    check(dw[4, N - 300:], want, half_step(want, BF16) + d[:, N - 300:].abs().t() @ xe.abs() * (70 * STEP), "dw")
    assert not bool(dw[3, -1].any())
    slot = torch.randperm(70000, generator=g, device="cuda")[:64].reshape(32, 2).int()
    slot[31, 1] = 69999
    gates = torch.rand(32, 2, generator=g, device="cuda")
    out = bm.moe_combine(x, slot, gates)
    r, wt = plain_combine(x, slot, gates)
    want = (r * wt[:, :, None]).sum(1)
    check(out, want, half_step(want, BF16) + (r * wt[:, :, None]).abs().sum(1) * 3 * STEP, "combine")


def test_w4_offsets_past_32_bits(bm):
    E, N, K = 9, 32768, 16384
    g = rng(61)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(E, N, K // 128, generator=g, device="cuda") * 0.01).half()
    m = (s.float() * -7.5).half()
    for counts in ([0] * 8 + [1], [0] * 8 + [20]):
        bounds, R = ragged(g, E, counts)
        x = normal(g, R, K, dtype=F16)
        y = bm.w4_matmul(x, codes, s, m, torch.empty(R, N, dtype=F32, device="cuda"), bounds)
        last = slice(N - 200, N)
        q = torch.stack([codes[8, last] & 15, codes[8, last] >> 4], -1).reshape(200, K).double()
        sd = s[8, last].double().repeat_interleave(128, 1)
        md = m[8, last].double().repeat_interleave(128, 1)
        want = x.double() @ (sd * q + md).t()
        size = x.double().abs() @ (sd * q + md.abs() + 32 * sd).t()
        check(y[:, last], want, half_step(want, F32) + size * (K * STEP), "w4")
