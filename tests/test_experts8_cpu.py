"""CPU checks of the 8-bit operators and the balance loss: what their entry
points and binding refuse before anything is enqueued, and their workspaces."""
import pytest

from spectral_expert_gemv_amd import bitsmoe as bm

from .test_experts_binding_cpu import gpu

torch = pytest.importorskip("torch")

P = 4096  # a pointer that no refused call follows
F32, F16, BF16, E4M3 = 0, 1, 2, 3
F8 = torch.float8_e4m3fn


def _status(name, *args):
    return getattr(bm._lib, "bitsmoe_" + name)(*args)


def rows(**kw):
    a = dict(dtype=F16, x=P, ldx=256, act=0, bounds=None, R=10, E=0, K=130, codes=P, ldc=256, scales=P, lds=2)
    a.update(kw)
    return _status("fp8_rows", *a.values(), None)


def weights(**kw):
    a = dict(dtype=F32, w=P, E=3, N=130, K=200, codes=P, scales=P, codes_t=P, scales_t=P)
    a.update(kw)
    return _status("fp8_weights", *a.values(), None)


def matmul(**kw):
    a = dict(x_dtype=F16, x=P, ldx=200, x_scales=None, ldxs=0, x_rows=10, rows=None, div=1, codes=P, scales=P, bounds=P, R=10, E=4, N=40,
             K=200, act=0, y=P, y_dtype=F16, ldy=40, ws=None, ws_bytes=0)
    a.update(kw)
    return _status("fp8_matmul", *a.values(), None)


def given(**kw):
    return matmul(**dict(dict(x_dtype=E4M3, ldx=256, x_scales=P, ldxs=2, y_dtype=BF16), **kw))


def balance(**kw):
    a = dict(dtype=F32, logits=P, ld=64, ids=P, seqs=None, S=1, T=100, E=64, k=4, loss=P, z=P, counts=P, tokens=P, ws=P, ws_bytes=1 << 20)
    a.update(kw)
    return _status("moe_balance", *a.values(), None)


def balance_grad(**kw):
    a = dict(dtype=F32, logits=P, ld=64, ids=P, seqs=None, S=1, T=100, E=64, k=4, counts=P, tokens=P, dloss=P, dz=P, add=0, dlogits=P, ldd=64)
    a.update(kw)
    return _status("moe_balance_grad", *a.values(), None)


@pytest.mark.parametrize("call, wrong, status", [
    (rows, dict(dtype=E4M3), bm.EINVAL), (rows, dict(dtype=-1), bm.EINVAL), (rows, dict(act=2), bm.EINVAL), (rows, dict(R=-1), bm.ESHAPE),
    (rows, dict(R=(1 << 26) + 1), bm.ESHAPE), (rows, dict(K=0), bm.ESHAPE), (rows, dict(K=(1 << 20) + 1, ldx=1 << 22), bm.ESHAPE),
    (rows, dict(ldx=129), bm.ESHAPE), (rows, dict(act=1, ldx=259), bm.ESHAPE), (rows, dict(ldc=255), bm.ESHAPE), (rows, dict(lds=1), bm.ESHAPE),
    (rows, dict(bounds=P), bm.ESHAPE), (rows, dict(x=None), bm.EINVAL), (rows, dict(codes=None), bm.EINVAL), (rows, dict(scales=None), bm.EINVAL),
    (rows, dict(codes=P + 8), bm.EINVAL), (rows, dict(ldc=264), bm.EINVAL),
    (weights, dict(dtype=E4M3), bm.EINVAL), (weights, dict(E=-1), bm.ESHAPE), (weights, dict(N=0), bm.ESHAPE), (weights, dict(K=0), bm.ESHAPE),
    (weights, dict(N=(1 << 21) + 1), bm.ESHAPE), (weights, dict(K=(1 << 21) + 1), bm.ESHAPE), (weights, dict(E=1 << 22, N=1000, K=1), bm.ESHAPE),
    (weights, dict(codes_t=None), bm.EINVAL), (weights, dict(scales_t=None), bm.EINVAL), (weights, dict(w=None), bm.EINVAL),
    (weights, dict(codes=None), bm.EINVAL), (weights, dict(scales=None), bm.EINVAL), (weights, dict(codes=P + 4), bm.EINVAL),
    (weights, dict(codes_t=P + 8), bm.EINVAL),
    (matmul, dict(x_dtype=F32), bm.EINVAL), (matmul, dict(x_dtype=4), bm.EINVAL), (matmul, dict(act=2), bm.EINVAL), (matmul, dict(y_dtype=BF16), bm.EINVAL),
    (matmul, dict(y_dtype=E4M3), bm.EINVAL), (given, dict(y_dtype=E4M3), bm.EINVAL), (matmul, dict(E=0), bm.ESHAPE), (matmul, dict(E=65536), bm.ESHAPE),
    (matmul, dict(N=0), bm.ESHAPE), (matmul, dict(K=0), bm.ESHAPE), (matmul, dict(R=-1), bm.ESHAPE), (matmul, dict(x_rows=-1, rows=P), bm.ESHAPE),
    (matmul, dict(K=(1 << 20) + 1, ldx=1 << 21), bm.ESHAPE), (matmul, dict(E=65535, R=1 << 26, x_rows=1 << 26), bm.ESHAPE),
    (matmul, dict(bounds=None), bm.EINVAL), (matmul, dict(x_rows=9), bm.ESHAPE), (matmul, dict(rows=P, div=0), bm.ESHAPE),
    (matmul, dict(rows=P, x_rows=0), bm.ESHAPE), (matmul, dict(ldx=199), bm.ESHAPE), (given, dict(ldx=240), bm.ESHAPE), (given, dict(ldxs=1), bm.ESHAPE),
    (matmul, dict(ldy=39), bm.ESHAPE), (matmul, dict(x=None), bm.EINVAL), (matmul, dict(codes=None), bm.EINVAL), (matmul, dict(scales=None), bm.EINVAL),
    (matmul, dict(y=None), bm.EINVAL), (given, dict(x_scales=None), bm.EINVAL), (matmul, dict(codes=P + 8), bm.EINVAL), (given, dict(x=P + 8), bm.EINVAL),
    (given, dict(ldx=264), bm.EINVAL),
    (balance, dict(dtype=E4M3), bm.EINVAL), (balance, dict(E=0), bm.ESHAPE), (balance, dict(E=2049, ld=4096), bm.ESHAPE), (balance, dict(k=0), bm.EINVAL),
    (balance, dict(k=65), bm.EINVAL), (balance, dict(T=-1), bm.ESHAPE), (balance, dict(T=(1 << 24) + 1), bm.ESHAPE), (balance, dict(S=0), bm.ESHAPE),
    (balance, dict(S=65536, seqs=P), bm.ESHAPE), (balance, dict(S=2), bm.EINVAL), (balance, dict(ld=63), bm.ESHAPE), (balance, dict(logits=None), bm.EINVAL),
    (balance, dict(ids=None), bm.EINVAL), (balance, dict(loss=None), bm.EINVAL), (balance, dict(z=None), bm.EINVAL), (balance, dict(counts=None), bm.EINVAL),
    (balance, dict(tokens=None), bm.EINVAL), (balance, dict(T=2000, ws=None), bm.ENOSPC), (balance, dict(T=2000, ws_bytes=10), bm.ENOSPC), (balance, dict(T=2000, ws=P + 2), bm.EINVAL),
    (balance_grad, dict(dtype=5), bm.EINVAL), (balance_grad, dict(E=2049, ld=4096, ldd=4096), bm.ESHAPE), (balance_grad, dict(k=65), bm.EINVAL),
    (balance_grad, dict(S=3), bm.EINVAL), (balance_grad, dict(ldd=63), bm.ESHAPE), (balance_grad, dict(ld=63), bm.ESHAPE),
    (balance_grad, dict(counts=None), bm.EINVAL), (balance_grad, dict(tokens=None), bm.EINVAL), (balance_grad, dict(dlogits=None), bm.EINVAL),
])
def test_refuses_before_anything_is_enqueued(call, wrong, status):
    assert call(**wrong) == status
    assert bm._lib.bitsmoe_last_error_detail()


@pytest.mark.parametrize("call, empty", [(rows, dict(R=0, x=None)), (weights, dict(E=0, w=None)), (matmul, dict(R=0, x=None, y=None)),
                                         (given, dict(R=0)), (balance_grad, dict(T=0))])
def test_nothing_to_do_is_fine(call, empty):
    assert call(**empty) == bm.OK


def test_balance_workspace():
    for T, E, S in [(1025, 1, 1), (4096, 64, 2), (100, 600, 1), (16384, 128, 1), (1 << 24, 2048, 65535), (50, 800, 300)]:
        n = bm.moe_balance_workspace_size(T, E, S)
        assert 0 < n and n % 4 == 0
    assert bm.moe_balance_workspace_size(0, 8, 1) == 0 == bm.moe_balance_workspace_size(256, 256, 1) == bm.moe_balance_workspace_size(1024, 8, 8)
    with pytest.raises(bm.BitsMoEError):
        bm.moe_balance_workspace_size(10, 3000, 1)


def f8(*shape):
    return torch.zeros(*shape).to(F8).as_subclass(type(gpu(1)))


def f32(*shape):
    return gpu(*shape, dtype=torch.float32)


def i32(*shape):
    return gpu(*shape, dtype=torch.int32)


BAD = [
    (lambda: bm.fp8_rows(gpu(4, 7), act="silu_mul"), "columns"), (lambda: bm.fp8_rows(gpu(4, 8), act="gelu"), "act"),
    (lambda: bm.fp8_rows(torch.zeros(4, 8)), "not on a GPU"), (lambda: bm.fp8_rows(gpu(4, 8, dtype=torch.float64), f8(4, 128), f32(4, 1)), "dtype"),
    (lambda: bm.fp8_rows(gpu(4, 8), f8(4, 8), f32(4, 1)), "shape"), (lambda: bm.fp8_rows(gpu(4, 8), f8(4, 128), f32(4, 2)), "shape"),
    (lambda: bm.fp8_rows(gpu(4, 8), gpu(4, 128), f32(4, 1)), "codes"), (lambda: bm.fp8_rows(gpu(8, 4).t(), f8(4, 128), f32(4, 1)), "contiguous"),
    (lambda: bm.fp8_weights(gpu(2, 4, 8), f8(2, 4, 128), f32(2, 1, 1), f8(2, 8, 128)), "together"),
    (lambda: bm.fp8_weights(gpu(2, 8, 4).transpose(1, 2), f8(2, 4, 128), f32(2, 1, 1)), "contiguous"),
    (lambda: bm.fp8_weights(gpu(2, 4, 8), f8(2, 4, 256), f32(2, 1, 1)), "codes"), (lambda: bm.fp8_weights(gpu(2, 4, 8), f8(2, 4, 128), f32(2, 1, 2)), "scales"),
    (lambda: bm.fp8_weights(gpu(2, 4, 8), f8(2, 4, 128), f32(2, 1, 1), f8(2, 4, 128), f32(2, 1, 1)), "codes_t"),
    (lambda: bm.fp8_matmul(gpu(4, 130), f8(2, 6, 128), f32(2, 1, 1), gpu(4, 6), bounds=i32(3)), "inputs"),
    (lambda: bm.fp8_matmul(gpu(4, 100), f8(2, 6, 100), f32(2, 1, 1), gpu(4, 6), bounds=i32(3)), "inputs"),
    (lambda: bm.fp8_matmul(gpu(4, 100), f8(2, 6, 128), f32(2, 1, 1), gpu(4, 6), x_scales=f32(4, 1), bounds=i32(3)), "x_scales"),
    (lambda: bm.fp8_matmul(f8(4, 128), f8(2, 6, 128), f32(2, 1, 1), gpu(4, 6), bounds=i32(3)), "x_scales"),
    (lambda: bm.fp8_matmul(f8(4, 128), f8(2, 6, 128), f32(2, 1, 1), gpu(4, 6), x_scales=gpu(4, 1), bounds=i32(3)), "float32"),
    (lambda: bm.fp8_matmul(f8(4, 128), f8(2, 6, 128), f32(2, 1, 1), gpu(4, 6), x_scales=f32(4, 2), bounds=i32(3)), "shape"),
    (lambda: bm.fp8_matmul(gpu(4, 100), f8(2, 6, 128), f32(2, 1, 1), gpu(4, 5), bounds=i32(3)), "shape"),
    (lambda: bm.fp8_matmul(gpu(4, 100), f8(2, 7, 128), f32(2, 2, 1), gpu(4, 3), bounds=i32(3), act="silu_mul"), "act"),
    (lambda: bm.fp8_matmul(gpu(4, 100), f8(2, 6, 128), f32(2, 1, 1), gpu(4, 3), bounds=i32(3), act="silu_mul"), "scales"),
    (lambda: bm.fp8_matmul(gpu(4, 100), f8(2, 6, 128), f32(2, 1, 1), gpu(4, 6), bounds=i32(4)), "bounds"),
    (lambda: bm.fp8_matmul(gpu(4, 100), gpu(2, 6, 128), f32(2, 1, 1), gpu(4, 6), bounds=i32(3)), "codes"),
    (lambda: bm.fp8_matmul(gpu(4, 100), f8(2, 6, 128), f32(2, 1, 1), gpu(5, 6), bounds=i32(3)), "rows"),
    (lambda: bm.fp8_matmul(gpu(4, 100), f8(2, 6, 128), f32(2, 1, 1), gpu(4, 6), bounds=torch.zeros(3, dtype=torch.int32)), "tensors on"),
    (lambda: bm.fp8_matmul(gpu(4, 100), f8(2, 6, 128), f32(2, 1, 1), gpu(4, 6), bounds=i32(3), ws=gpu(64)[::2]), "contiguous"),
    (lambda: bm.moe_balance(gpu(4, 8), gpu(4, 2), loss=f32(1), z=f32(1), counts=i32(1, 8), tokens=i32(1), ws=gpu(4096)), "ids"),
    (lambda: bm.moe_balance(gpu(4, 8), i32(5, 2), loss=f32(1), z=f32(1), counts=i32(1, 8), tokens=i32(1), ws=gpu(4096)), "ids"),
    (lambda: bm.moe_balance(gpu(4, 8), i32(4, 2), loss=f32(2), z=f32(1), counts=i32(1, 8), tokens=i32(1), ws=gpu(4096)), "loss"),
    (lambda: bm.moe_balance(gpu(4, 8), i32(4, 2), i32(4), f32(3), f32(3), i32(2, 8), i32(3), gpu(4096)), "counts"),
    (lambda: bm.moe_balance(gpu(4, 8), i32(4, 2), gpu(4), f32(3), f32(3), i32(3, 8), i32(3), gpu(4096)), "seqs"),
    (lambda: bm.moe_balance_grad(gpu(4, 8), i32(4, 2), i32(1, 8), i32(1), gpu(1), dlogits=gpu(4, 8)), "dloss"),
    (lambda: bm.moe_balance_grad(gpu(4, 8), i32(4, 2), i32(1, 8), i32(1), f32(1), add=True), "add"),
    (lambda: bm.moe_balance_grad(gpu(4, 8), i32(4, 2), i32(1, 8), i32(1), f32(1), dlogits=f32(4, 8)), "dtype"),
    (lambda: bm.moe_balance_grad(gpu(4, 8), i32(4, 2), i32(2, 8), i32(1), f32(1), dlogits=gpu(4, 8)), "counts"),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_binding_refuses(i):
    call, what = BAD[i]
    with pytest.raises(ValueError, match=what):
        call()


@pytest.mark.parametrize("F", [96, 128])
@pytest.mark.parametrize("which", ["w1", "w2"])
def test_layer_refuses_weights_with_gaps(F, which):
    """Whether F makes whole blocks or not: a copy of them would be made on
    another stream than the call's."""
    from spectral_expert_gemv_amd.layer import ExpertLayer
    w = dict(w1=gpu(2, 2 * F, 256), w2=gpu(2, 256, F))
    w[which] = gpu(2, w[which].shape[2], w[which].shape[1]).transpose(1, 2)
    with pytest.raises(ValueError, match="%s must be contiguous" % which):
        ExpertLayer.fp8(**w, stream=1)
