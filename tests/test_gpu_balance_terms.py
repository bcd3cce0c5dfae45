"""GPU tests of the balance losses' gradient, element by element.

With p = softmax(l), f and lse of the definition, a = dloss / n, b = 2 dz / n:
  dl = p (a (f - m) + b lse),  m = sum p f
In float32 steps p is off by up to rel = (E + 32) 2^-23 of itself: E 2^-23 for
the sum, 2^-18 for the exp of an exponent of up to 32 that is off by half a
step, the exp itself and the division; m by as much of itself and E 2^-24 for
its sum; lse by rel (its logarithm's argument) and 2^-23 of itself.  So dl is
off by at most 2 rel (p |a| (f + m) + p |b| (|lse| + 1)), and by half a step of
its type.  The incoming gradients grow with n here, as a loss scale has it, so
that no element drowns in a type's smallest steps.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
INF = float("inf")

# (T, E, k, sequences' borders or None: every width of a lane's run of experts, whole and part ones
SHAPES = [(1, 1, 1, None), (1, 8, 2, None), (17, 16, 4, None), (64, 60, 4, None), (67, 129, 8, None), (33, 256, 16, None), (5, 257, 6, None),
          (130, 512, 10, None), (9, 1000, 64, None), (3, 2048, 64, None), (1000, 64, 6, None), (5000, 128, 8, None), (40000, 16, 2, None),
          (50, 8, 2, [0, 0, 1, 50]), (700, 64, 6, [0, 64, 65, 65, 300, 700]), (300, 300, 4, [5, 20, 20, 290]), (90, 2048, 8, [0, 30, 90])]


@pytest.fixture(scope="module")
def bm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from spectral_expert_gemv_amd import bitsmoe
    return bitsmoe


def make(T, E, k, cuts, dtype):
    """(logits, ids, counts, tokens, dloss, dz) on the host."""
    g = torch.Generator()
    g.manual_seed(T + 3 * E)
    l = torch.randn(T, E, generator=g) * 2.0
    l[:, 0] += 2.0
    l = l.to(dtype)
    if E > 4:
        l[:, 2] = -INF          # a retired expert
        l[T // 3, 1:] = -INF    # one expert left
    ids = torch.topk(l.float(), k, dim=1).indices.int()
    if T > 8:
        ids[T // 4] = -1        # padding
    cuts = cuts or [0, T]
    S = len(cuts) - 1
    counts, tokens = torch.zeros(S, E, dtype=torch.int32), torch.zeros(S, dtype=torch.int32)
    for s in range(S):
        at = ids[cuts[s]:cuts[s + 1]]
        tokens[s] = int((at >= 0).any(1).sum())
        counts[s] = torch.bincount(at[at >= 0].long(), minlength=E).int()
    n = tokens.clamp(min=1).float()
    sign = torch.where(torch.arange(S) % 2 == 0, 1.0, -1.0)
    return l, ids, counts, tokens, sign * (torch.rand(S, generator=g) + 0.5) * n, sign * (torch.rand(S, generator=g) + 0.5) * 0.1 * n


def terms(l, ids, cuts, counts, tokens, dloss, dz):
    """(p a f, p a m, p b lse, p b) of every token in 64 bits, 0 where it takes no part."""
    l = l.double()
    (T, E), k = l.shape, ids.shape[1]
    cuts = cuts or [0, T]
    out = torch.zeros(4, T, E, dtype=torch.float64)
    for s in range(len(cuts) - 1):
        n = int(tokens[s])
        at = torch.arange(cuts[s], cuts[s + 1])
        at = at[(ids[at] >= 0).any(1)]
        if not n:
            continue
        lse = torch.logsumexp(l[at], 1, keepdim=True)
        p = torch.exp(l[at] - lse)
        f = counts[s].double() * (E / (k * n))
        a, b = dloss[s].double() / n, 2 * dz[s].double() / n
        out[:, at] = torch.stack([p * a * f, p * a * (p * f).sum(1, keepdim=True), p * b * lse, p * b])
    return out


def expected(t, dtype, E):
    """(dlogits, how far off they may be)."""
    af, am, bl, b = t
    want = af - am + bl
    tol = want.abs() * (torch.finfo(dtype).eps / 2) + (2.0 ** -25 if dtype == F16 else 0.0)
    return want, tol + 2 * (E + 32) * 2.0 ** -23 * (af.abs() + am.abs() + bl.abs() + b.abs()) + 1e-36


def check(got, want, tol, what):
    off = (got.double().cpu() - want).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), "%s: %d of %d off, worst %.3g of tol" % (what, int(bad.sum()), bad.numel(), float((off / tol).nan_to_num(1e9).max()))


@pytest.mark.parametrize("T, E, k, cuts", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_every_element(bm, T, E, k, cuts, dtype):
    print("balance gradient", T, E, k, cuts, dtype, flush=True)
    l, ids, counts, tokens, dloss, dz = make(T, E, k, cuts, dtype)
    want, tol = expected(terms(l, ids, cuts, counts, tokens, dloss, dz), dtype, E)
    seqs = None if cuts is None else torch.tensor(cuts, dtype=torch.int32, device="cuda")
    l, ids, dloss, dz = (t.cuda() for t in (l, ids, dloss, dz))
    _, _, got_counts, got_tokens = bm.moe_balance(l, ids, seqs)
    assert torch.equal(got_counts.cpu(), counts) and torch.equal(got_tokens.cpu(), tokens)
    check(bm.moe_balance_grad(l, ids, got_counts, got_tokens, dloss, dz, seqs), want, tol, "dlogits")
    g = torch.Generator()
    g.manual_seed(E)
    there = torch.randn(T, E, generator=g).to("cuda", dtype)
    got = bm.moe_balance_grad(l, ids, got_counts, got_tokens, dloss, dz, seqs, there.clone(), add=True)
    total = there.double().cpu() + want
    # (the sum in float32 is rounded, then its rounding to the type)
    check(got, total, tol + total.abs() * (torch.finfo(dtype).eps / 2 + 2.0 ** -23) + (2.0 ** -25 if dtype == F16 else 0.0), "added")


@pytest.mark.parametrize("E, k", [(300, 6), (2048, 8)])
def test_wide_gradients_by_differences(bm, E, k):
    """Against central differences of 64-bit losses with the counts held: with
    step h they are off by h^2 / 6 of a third derivative, which is at most the
    size of the gradient's terms (of p a (f - m) its factor is 1 - 6p + 6p^2; of
    p b lse (1 - p)(1 - 2p), beside p b times 3p (1 - p)), and by the losses' own
    2^-50 over h."""
    T, cuts, dtype, h = 12, [0, 5, 12], F32, 1e-4
    l, ids, counts, tokens, dloss, dz = make(T, E, k, cuts, dtype)
    t = terms(l, ids, cuts, counts, tokens, dloss, dz)
    _, tol = expected(t, dtype, E)
    seqs = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    got = bm.moe_balance_grad(l.cuda(), ids.cuda(), counts.cuda(), tokens.cuda(), dloss.cuda(), dz.cuda(), seqs).double().cpu()
    g = torch.Generator()
    g.manual_seed(E)
    for i in [0, 2, 4, 5, 8, 11]:
        s = int(i >= 5)
        if int(ids[i, 0]) < 0:
            continue
        n = float(tokens[s])
        f, a, b = counts[s].double() * (E / (k * n)), float(dloss[s]) / n, float(dz[s]) / n

        def loss(v):
            lse = torch.logsumexp(v, 0)
            return float(a * (f * torch.exp(v - lse)).sum() + b * lse ** 2)
        row = l[i].double()
        picks = torch.cat([torch.topk(row, 4).indices, torch.randint(0, E, (12,), generator=g), torch.tensor([E - 1])])
        for e in picks.tolist():
            if row[e] == -INF:
                continue
            up, dn = row.clone(), row.clone()
            up[e] += h
            dn[e] -= h
            size = float(t[:, i, e].abs().sum())
            slack = h * h * size + 2.0 ** -50 * (abs(loss(row)) + 1) / h
            assert abs((loss(up) - loss(dn)) / (2 * h) - float(got[i, e])) <= float(tol[i, e]) + slack


@pytest.mark.parametrize("bad", [float("nan"), INF])
def test_a_token_that_the_router_turned_away(bm, bad):
    """Logits with a NaN or +inf: the router's ids of -1 keep the token out of the
    layer's losses, which are those of the others."""
    from spectral_expert_gemv_amd.layer import ExpertLayer
    T, E, k, D, F = 40, 8, 2, 64, 64
    g = torch.Generator()
    g.manual_seed(3)
    normal = lambda *s: torch.randn(*s, generator=g).to("cuda", F16) * 0.1  # noqa: E731
    x, dout, l = normal(T, D), normal(T, D), torch.randn(T, E, generator=g).cuda()
    l[7, 3] = bad
    l[30, 0] = bad
    layer = ExpertLayer(normal(E, 2 * F, D), normal(E, D, F))
    seqs = torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda")
    loss, z, counts, tokens = layer.gradients(x, l, k, dout, balance=0.5, z=0.1, seqs=seqs)[5]
    assert tokens.tolist() == [19, 19] and counts.sum(1).tolist() == [38, 38]
    keep = (torch.arange(T, device="cuda") != 7) & (torch.arange(T, device="cuda") != 30)
    want = layer.gradients(x[keep], l[keep], k, dout[keep], balance=0.5, z=0.1, seqs=torch.tensor([0, 19, 38], dtype=torch.int32, device="cuda"))
    for a, b in zip((loss, z), want[5]):
        # (their sums may have another order: terms of one sign, 42 additions each)
        assert bool(((a - b).abs() <= 2.0 ** -18 * b.abs()).all())
    d = layer.gradients(x, l, k, dout, balance=0.5, z=0.1, seqs=seqs)[2]
    assert bool(d[~keep].isnan().all()) and torch.equal(d[keep], want[2])
