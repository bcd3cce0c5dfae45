"""GPU tests of the expert layer's operators where they can go wrong: weights
that cancel, infinities and NaN, empty batches, rows at any alignment, and the
router in front of the spectral path.

Tolerances as in test_gpu_experts.py: a float32 sum of n products adds at most
n 2^-23 of the sum of their magnitudes, an output rounded once half a step.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

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
