"""GPU tests of the balance loss and its gradient against a plain 64-bit
implementation.

Tolerances: softmax in float32 is off by E 2^-23 for its sum, and by 2^-18 for
the exp of an exponent of up to 32 that is off by half a step, the exp itself
and the division; the losses are sums of such terms of one sign (z: of squares
of values off by that much).
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")
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


def check(got, want, tol, what=""):
    got = got.double()
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), "%s: %d of %d off, worst %.3g of tol" % (
        what, int(bad.sum()), bad.numel(), float(((got - want).abs() / tol.clamp(min=1e-300)).nan_to_num(1e9).max()))


def plain(l, ids, cuts, E, dloss, dz):
    """(loss, z, counts, tokens, dlogits, its size) in 64 bits on the host, a sequence at a time."""
    l, ids = l.double().cpu(), ids.cpu().long()
    k, S = ids.shape[1], len(cuts) - 1
    loss, z = torch.zeros(S, dtype=torch.float64), torch.zeros(S, dtype=torch.float64)
    counts, tokens = torch.zeros(S, E, dtype=torch.int32), torch.zeros(S, dtype=torch.int32)
    d, size = torch.zeros_like(l), torch.zeros_like(l)
    for s in range(S):
        at = torch.arange(cuts[s], cuts[s + 1])
        good = (ids[at] >= 0) & (ids[at] < E)
        at = at[good.any(1) & ~(l[at] == -INF).all(1)]
        n = len(at)
        tokens[s] = n
        if not n:
            continue
        chosen = ids[at].reshape(-1)
        chosen = chosen[(chosen >= 0) & (chosen < E)]
        counts[s] = torch.bincount(chosen, minlength=E).int()
        lse = torch.logsumexp(l[at], 1, keepdim=True)
        p = torch.exp(l[at] - lse)
        f = counts[s].double() * (E / (k * n))
        loss[s], z[s] = (f * p.mean(0)).sum(), (lse ** 2).mean()
        a, b = dloss[s].double().cpu() / n, 2 * dz[s].double().cpu() / n
        mean = (p * f).sum(1, keepdim=True)
        d[at] = p * (a * (f - mean) + b * lse)
        size[at] = p * (a.abs() * (f + mean) + b.abs() * lse.abs())
    return loss, z, counts, tokens, d, size


def make(g, T, E, k, dtype, wide=3):
    l = torch.randn(T, E + wide, generator=g, device="cuda") * 2.0
    l[:, 0] += 2.0
    l = l.to(dtype)[:, :E]
    ids = torch.topk(l.float(), k, dim=1).indices.int()
    return l, ids


def half_step(v, dtype):
    t = v.abs() * (torch.finfo(dtype).eps / 2)
    return t + 2.0 ** -25 if dtype == F16 else t


def compare(bm, l, ids, cuts, E, g, add=False):
    S, T = len(cuts) - 1, l.shape[0]
    seqs = None if cuts == [0, T] else torch.tensor(cuts, dtype=torch.int32, device="cuda")
    loss, z, counts, tokens = bm.moe_balance(l, ids, seqs)
    dloss, dz = torch.randn(S, generator=g, device="cuda"), torch.randn(S, generator=g, device="cuda") * 0.1
    wl, wz, wc, wt, wd, size = plain(l, ids, cuts, E, dloss, dz)
    assert torch.equal(counts.cpu(), wc) and torch.equal(tokens.cpu(), wt)
    rel = E * STEP + 2.0 ** -18
    check(loss.cpu(), wl, wl * rel + 1e-30, "loss")
    check(z.cpu(), wz, wz * 2.0 ** -18 + (wz.sqrt() + 1) * rel * 2, "z")
    d = bm.moe_balance_grad(l, ids, counts, tokens, dloss, dz, seqs)
    # (lse is off by its own half step and by the sum's error)
    n = max(1, int(wt.max()))
    tol = half_step(wd, l.dtype) + size * (rel * 2) + 2 * float(dz.abs().max()) * rel + 1e-30
    check(d.cpu(), wd, tol, "dlogits")
    # added to what is there
    there = torch.randn(T, E, generator=g, device="cuda").to(l.dtype)
    got = bm.moe_balance_grad(l, ids, counts, tokens, dloss, dz, seqs, there.clone(), add=True)
    want = there.double().cpu() + wd
    check(got.cpu(), want, half_step(want, l.dtype) + tol + want.abs() * STEP, "added")
    return loss, z, counts, tokens, d


@pytest.mark.parametrize("T, E, k", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (17, 16, 16), (64, 60, 4), (67, 129, 8), (33, 256, 16), (5, 257, 6), (130, 512, 10),
                                     (9, 1000, 64), (3, 2048, 64), (1000, 64, 6), (5000, 128, 8), (40000, 16, 2)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_one_sequence(bm, T, E, k, dtype):
    _say("balance", T, E, k, dtype)
    g = rng(T + E)
    l, ids = make(g, T, E, k, dtype)
    if E > 4:
        l[:, 2] = -INF          # a retired expert
        l[T // 3, 1:] = -INF    # one expert left
        ids[T // 4, 0] = -1     # a slot left over
    compare(bm, l, ids, [0, T], E, g)


@pytest.mark.parametrize("T, E, k, cuts", [(50, 8, 2, [0, 0, 1, 50]), (700, 64, 6, [0, 64, 65, 65, 300, 700]), (500, 128, 8, [0, 100, 300, 490]),
                                           (1500, 64, 6, [0, 64, 65, 65, 300, 1500]), (4096, 32, 4, [0, 1, 1, 4000, 4000, 4001, 4050, 4090, 4096]),
                                           (300, 300, 4, [5, 20, 20, 290]), (4096, 16, 2, list(range(0, 4097, 32))), (90, 2048, 8, [0, 30, 90])])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sequences(bm, T, E, k, cuts, dtype):
    """Empty ones, of one token, more than the chip's rows of work-groups; tokens in none are left as they were."""
    _say("balance of sequences", T, E, k, cuts[:8], dtype)
    g = rng(T)
    l, ids = make(g, T, E, k, dtype)
    ids[cuts[-1] - 3:] = -1  # padding
    l[cuts[-1] - 2:] = NAN
    loss, z, counts, tokens, d = compare(bm, torch.where(l.isnan(), torch.zeros_like(l), l), ids, cuts, E, g)
    seqs = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    # what padding's logits hold does not matter
    again = bm.moe_balance(l, ids, seqs)
    for a, b in zip(again, (loss, z, counts, tokens)):
        assert torch.equal(a, b)
    left = torch.full((T, E), 7.0, dtype=dtype, device="cuda")
    one = torch.ones(len(cuts) - 1, device="cuda")
    bm.moe_balance_grad(l, ids, counts, tokens, one, None, seqs, left)
    assert bool((left[: cuts[0]] == 7.0).all()) and bool((left[cuts[-1]:] == 7.0).all()) and bool(left.isfinite().all())


@pytest.mark.parametrize("T, E, k, cuts", [(50, 20, 3, [5, 20]), (50, 20, 3, [7, 7]), (250, 256, 8, [0, 250]), (257, 100, 40, [0, 257]), (1100, 100, 40, [0, 1100]), (1025, 7, 2, [0, 1025]), (30, 100, 40, [0, 30]),
                                           (400, 300, 5, [3, 390])])
@pytest.mark.parametrize("dtype", [F32, F16])
def test_one_sequence_among_the_tokens(bm, T, E, k, cuts, dtype):
    """In one launch and in two, with more slots than lanes, and ids that repeat or lie outside."""
    _say("balance of one sequence", T, E, k, cuts, dtype)
    g = rng(T + k)
    l, _ = make(g, T, E, k if k < E else 1, dtype)
    ids = torch.randint(-2, E + 2, (T, k), generator=g, device="cuda", dtype=torch.int32)
    ids[T // 3] = -1
    ids[T // 2] = E
    compare(bm, l, ids, cuts, E, g)


def test_a_workspace_at_any_word(bm):
    g = rng(77)
    l, ids = make(g, 1700, 64, 4, F32)
    want = bm.moe_balance(l, ids)
    ws = torch.empty(bm.moe_balance_workspace_size(1700, 64) + 4, dtype=torch.uint8, device="cuda")
    got = bm.moe_balance(l, ids, ws=ws[4:])
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_gradient_by_differences(bm):
    """Against central differences of a 64-bit loss with the counts held."""
    g = rng(9)
    T, E, k = 12, 20, 3
    l, ids = make(g, T, E, k, F32)
    cuts = [0, 5, 12]
    seqs = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    _, _, counts, tokens = bm.moe_balance(l, ids, seqs)
    dl, dz = torch.tensor([0.7, -1.3], device="cuda"), torch.tensor([0.2, 0.4], device="cuda")
    d = bm.moe_balance_grad(l, ids, counts, tokens, dl, dz, seqs).double().cpu()
    c = counts.double().cpu()

    def total(v):
        out = 0.0
        for s in range(2):
            r = v[cuts[s]:cuts[s + 1]]
            n = len(r)
            f = c[s] * E / (k * n)
            out = out + float(dl[s]) * (f * torch.softmax(r, 1).mean(0)).sum() + float(dz[s]) * (torch.logsumexp(r, 1) ** 2).mean()
        return out
    base, h = l.double().cpu(), 1e-4
    for t, e in [(0, int(ids[0, 0])), (4, 3), (5, 0), (11, 19)]:
        up, dn = base.clone(), base.clone()
        up[t, e] += h
        dn[t, e] -= h
        # central differences: error h^2 / 6 times a third derivative of order 10, and float32's
        assert abs((total(up) - total(dn)) / (2 * h) - d[t, e]) < 1e-6


@pytest.mark.parametrize("bad", [NAN, INF])
def test_a_token_without_a_softmax(bm, bad):
    """Its sequence's losses and its own gradient are NaN, and nothing else is."""
    g = rng(2)
    l, ids = make(g, 60, 40, 4, F32)
    l[33, 7] = bad
    l[50, :] = -INF  # takes no part
    seqs = torch.tensor([0, 30, 45, 60], dtype=torch.int32, device="cuda")
    loss, z, counts, tokens = bm.moe_balance(l, ids, seqs)
    assert loss.isnan().tolist() == [False, True, False] and z.isnan().tolist() == [False, True, False]
    assert tokens.tolist() == [30, 15, 14]
    one = torch.ones(3, device="cuda")
    d = bm.moe_balance_grad(l, ids, counts, tokens, one, one, seqs)
    assert bool(d[33].isnan().all()) and not bool(d[50].any())
    keep = torch.arange(60, device="cuda") != 33
    assert bool(d[keep].isfinite().all())


def test_perfect_balance_is_one(bm):
    E, k = 16, 2
    ids = torch.arange(E * 8, device="cuda", dtype=torch.int32).reshape(-1, k) % E
    l = torch.zeros(ids.shape[0], E, device="cuda")
    loss, z, counts, tokens = bm.moe_balance(l, ids)
    assert abs(float(loss) - 1.0) < 1e-6 and bool((counts == 8).all())
    d = bm.moe_balance_grad(l, ids, counts, tokens, torch.ones(1, device="cuda"))
    assert float(d.abs().max()) < 1e-8


def test_no_tokens(bm):
    l, ids = torch.empty(0, 8, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda")
    seqs = torch.zeros(4, dtype=torch.int32, device="cuda")
    for q, S in ((None, 1), (seqs, 3)):
        loss, z, counts, tokens = bm.moe_balance(l, ids, q)
        assert loss.tolist() == [0.0] * S and z.tolist() == [0.0] * S and not bool(counts.any()) and tokens.tolist() == [0] * S
        assert bm.moe_balance_grad(l, ids, counts, tokens, torch.ones(S, device="cuda"), seqs=q).shape == (0, 8)


def test_wrong_sequences_stay_inside(bm):
    g = rng(3)
    l, ids = make(g, 500, 32, 2, F32)
    for b in ([0, 300, 100, 5000, 400], [-5, -1, 700, 700, 7], [2 ** 31 - 1] * 5, [500, 0, 500, 0, 500]):
        seqs = torch.tensor(b, dtype=torch.int32, device="cuda")
        loss, z, counts, tokens = bm.moe_balance(l, ids, seqs)
        box = torch.full((502, 32), 7.0, device="cuda")
        bm.moe_balance_grad(l, ids, counts, tokens, torch.ones(4, device="cuda"), None, seqs, box[1:501])
        assert bool((box[0] == 7.0).all()) and bool((box[501] == 7.0).all())


def test_repeats_streams_and_graphs(bm):
    """The same bits each time: repeated, on another stream, captured and replayed."""
    g = rng(11)
    T, E, k, S = 9000, 128, 8, 3
    l, ids = make(g, T, E, k, BF16)
    seqs = torch.tensor([0, 1000, 1000, 9000], dtype=torch.int32, device="cuda")
    dl, dz = torch.ones(S, device="cuda"), torch.ones(S, device="cuda")

    def both(loss=None, z=None, counts=None, tokens=None, d=None, ws=None):
        out = bm.moe_balance(l, ids, seqs, loss, z, counts, tokens, ws)
        return list(out) + [bm.moe_balance_grad(l, ids, out[2], out[3], dl, dz, seqs, d)]
    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    bufs = [torch.empty_like(t) for t in want[:4]] + [torch.zeros_like(want[4])]
    ws = torch.empty(bm.moe_balance_workspace_size(T, E, S), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(*bufs, ws)
    for _ in range(3):
        for t in bufs:
            t.fill_(3)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(bufs, want):
            assert torch.equal(a, b)
        for a, b in zip(both(), want):
            assert torch.equal(a, b)


def test_logits_past_32_bits(bm):
    """17 GB of them: the last sequence as by itself."""
    T, E, k = 4200000, 1024, 2
    l = torch.zeros(T, E, device="cuda")
    g = rng(8)
    tail, _ = make(g, 1000, E, k, F32, wide=0)
    l[-1000:] = tail
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    ids[-1000:] = torch.topk(tail, k, dim=1).indices.int()
    seqs = torch.tensor([0, T - 1000, T], dtype=torch.int32, device="cuda")
    loss, z, counts, tokens = bm.moe_balance(l, ids, seqs)
    w = bm.moe_balance(tail, ids[-1000:].contiguous())
    assert torch.equal(counts[1:], w[2]) and torch.equal(tokens[1:], w[3]) and tokens.tolist() == [T - 1000, 1000]
    assert int(counts[0, 0]) == k * (T - 1000)
    check(loss[1:], w[0].double(), w[0].double() * 2.0 ** -16, "loss")
    check(z[1:], w[1].double(), w[1].double() * 2.0 ** -16, "z")
    one = torch.ones(2, device="cuda")
    d = bm.moe_balance_grad(l, ids, counts, tokens, one, one, seqs)
    assert torch.equal(d[-1000:], bm.moe_balance_grad(tail, ids[-1000:].contiguous(), w[2], w[3], one[:1], one[:1]))
    assert bool(d[:100].isfinite().all())
