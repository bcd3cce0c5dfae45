"""GPU tests of the balance losses over long sequences, where a sum that is kept
in float32 from token to token drifts: equal logits, whose losses are closed
forms (z = log(E)^2, and a loss of 1 for any ids), and whose additions all
round the same way.

Tolerance: at most 32 additions of a lane, 2 of its wave's tokens and 8 of the
waves stand between a token's term and float64, each off by 2^-24: 42 2^-24.
The terms: p = 1/E within 2^-23, lse = log E within a step, so its square within
2^-22 and half a step.  In all under 32 2^-23.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
REL = 2.0 ** -18


@pytest.fixture(scope="module")
def bm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from spectral_expert_gemv_amd import bitsmoe
    return bitsmoe


# 2^24 tokens are the most; of 4 or 32 tokens a turn of the work-group
@pytest.mark.parametrize("T, E, k, dtype", [(1 << 24, 8, 2, F32), (1 << 24, 100, 3, F16), (1 << 24, 257, 4, BF16), (4200000, 1024, 2, BF16), (3000001, 2047, 3, F16)])
@pytest.mark.parametrize("cuts", [None, [1, 1000, 0]])
def test_equal_logits(bm, T, E, k, dtype, cuts):
    print("balance of", T, E, k, dtype, cuts, flush=True)
    l = torch.zeros(T, E, dtype=dtype, device="cuda")
    ids = (torch.arange(T * k, device="cuda") % E).int().reshape(T, k)
    borders = [0, T] if cuts is None else [0, cuts[0], cuts[1], T]
    seqs = None if cuts is None else torch.tensor(borders, dtype=torch.int32, device="cuda")
    loss, z, counts, tokens = bm.moe_balance(l, ids, seqs)
    for s in range(len(borders) - 1):
        n = borders[s + 1] - borders[s]
        assert int(tokens[s]) == n and int(counts[s].sum()) == n * k
        assert abs(float(loss[s]) - 1.0) <= REL, (s, float(loss[s]))
        assert abs(float(z[s]) / math.log(E) ** 2 - 1.0) <= REL, (s, float(z[s]), math.log(E) ** 2)


def test_the_long_sequence_of_many(bm):
    """4.2 million tokens before 1000 others: its losses, and its gradient at its
    start, middle and end, which of equal logits is the same in every token:
    p (a (f - 1) + b log E) with p = 1 / E and the mean of f 1."""
    T, E, k = 4200000, 1024, 2
    l = torch.zeros(T, E, device="cuda", dtype=BF16)
    g = torch.Generator()
    g.manual_seed(5)
    l[-1000:] = torch.randn(1000, E, generator=g).to("cuda", BF16)
    # experts 0 .. 511 alone: f is 2 there and 0 elsewhere
    ids = (torch.arange(T * k, device="cuda") % 512).int().reshape(T, k)
    n = T - 1000
    seqs = torch.tensor([0, n, T], dtype=torch.int32, device="cuda")
    loss, z, counts, tokens = bm.moe_balance(l, ids, seqs)
    assert tokens.tolist() == [n, 1000]
    assert abs(float(loss[0]) - 1.0) <= REL and abs(float(z[0]) / math.log(E) ** 2 - 1.0) <= REL
    dloss, dz = torch.tensor([0.7, -1.0], device="cuda") * n, torch.tensor([0.05, 0.1], device="cuda") * n
    d = bm.moe_balance_grad(l, ids, counts, tokens, dloss, dz, seqs)
    a, b = float(dloss[0]) / n, 2 * float(dz[0]) / n
    f = counts[0].double().cpu() * (E / (k * n))
    want = (a * (f - 1.0) + b * math.log(E)) / E
    # half a step of the type; the terms' 2 (E + 32) 2^-23 as for any gradient
    tol = want.abs() * 2.0 ** -8 + 2 * (E + 32) * 2.0 ** -23 * (abs(a) * (f + 1.0) + abs(b) * (math.log(E) + 1)) / E
    for at in (slice(0, 300), slice(n // 2, n // 2 + 300), slice(n - 300, n)):
        assert bool(((d[at].double().cpu() - want).abs() <= tol).all())


@pytest.mark.parametrize("T, E, k, S, step", [(70000, 8, 2, 65535, 1), (200, 8, 2, 65535, 0), (69000, 300, 3, 65535, 1), (300000, 16, 2, 5000, 59)])
def test_thousands_of_sequences(bm, T, E, k, S, step):
    """Of `step` tokens each (0: of one token, far apart), against the definition
    in 64 bits.  Tolerances: (E + 32) 2^-23 of p for softmax, as in the sums of a
    few tokens; lse is off by as much and its own steps."""
    print("balance of", S, "sequences", T, E, k, flush=True)
    g = torch.Generator()
    g.manual_seed(S + E)
    l = (torch.randn(T, E, generator=g) * 2).cuda()
    ids = torch.topk(l, k, dim=1).indices.int()
    at = torch.arange(S + 1, device="cuda")
    seqs = (at * step if step else at // (S // T)).clamp(max=T).int()
    loss, z, counts, tokens = bm.moe_balance(l, ids, seqs)
    sign = torch.where(at[:S] % 2 == 0, 1.0, -1.0)
    d = bm.moe_balance_grad(l, ids, counts, tokens, sign, 0.1 * sign, seqs)

    seq = torch.bucketize(torch.arange(T, device="cuda", dtype=torch.int32), seqs[1:], right=True)
    inside = seq < S
    seq = seq.clamp(max=S - 1)

    def sums(v):
        return torch.zeros(S, *v.shape[1:], dtype=torch.float64, device="cuda").index_add_(0, seq[inside], v[inside].double())
    lse = torch.logsumexp(l.double(), 1, keepdim=True)
    p = torch.exp(l.double() - lse)
    n = sums(torch.ones(T, device="cuda"))
    c = sums(torch.zeros(T, E, device="cuda").scatter_(1, ids.long(), 1.0))
    assert torch.equal(tokens.double(), n) and torch.equal(counts.double(), c)
    inv = torch.where(n > 0, 1 / n, 0.0)
    f = c * inv[:, None] * (E / k)
    rel = (E + 32) * 2.0 ** -23
    want = (f * sums(p)).sum(1) * inv
    assert bool(((loss - want).abs() <= want * 2 * rel).all())
    want, size = sums(lse[:, 0] ** 2) * inv, sums(lse[:, 0].abs() + 1) * inv
    assert bool(((z - want).abs() <= want * 2.0 ** -18 + 2 * rel * size).all())
    a, b, ft = (sign.double() * inv)[seq][:, None], (0.2 * sign.double() * inv)[seq][:, None], f[seq]
    mean = (p * ft).sum(1, keepdim=True)
    want = torch.where(inside[:, None], p * (a * (ft - mean) + b * lse), 0.0)
    tol = 2 * rel * p * (a.abs() * (ft + mean) + b.abs() * (lse.abs() + 1)) + want.abs() * 2.0 ** -24 + 1e-36
    assert bool(((d - want).abs() <= tol).all())
