"""CPU checks of what the binding of the expert layer's operators refuses by
itself, with host tensors that say they are on a GPU."""
import pytest

from spectral_expert_gemv_amd import bitsmoe as bm

from .test_experts_cpu import combine, combine_grad, matmul, matmul_dx

torch = pytest.importorskip("torch")


class OnGpu(torch.Tensor):
    def get_device(self):
        return 0


def gpu(*shape, dtype=torch.float16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


def products(ws):
    """The three products with operands that need a workspace (odd sizes)."""
    b, i32 = gpu(3, dtype=torch.int32), torch.int32
    x, dy, w = gpu(40, 31), gpu(40, 7), gpu(2, 7, 31)
    rows = gpu(40, dtype=i32)
    return [lambda: bm.grouped_matmul(x, w, b, gpu(40, 7), rows=rows, ws=ws),
            lambda: bm.grouped_matmul_dx(dy, w, b, gpu(40, 31), ws=ws),
            lambda: bm.grouped_matmul_dw(dy, x, b, gpu(2, 7, 31), ws=ws)]


@pytest.mark.parametrize("which", [0, 1, 2])
def test_a_workspace_on_another_device_is_refused(which):
    with pytest.raises(ValueError, match="tensors on"):
        products(torch.zeros(1 << 16, dtype=torch.uint8))[which]()


@pytest.mark.parametrize("which", [0, 1, 2])
def test_a_workspace_with_holes_is_refused(which):
    """Its bytes are not those from its first one on."""
    ws = gpu(1 << 17, dtype=torch.uint8)[::2]
    with pytest.raises(ValueError, match="contiguous"):
        products(ws)[which]()


def test_a_grouping_workspace_with_holes_is_refused():
    ws, i32 = gpu(1 << 17, dtype=torch.int32)[::2], torch.int32
    out = dict(bounds=gpu(65, dtype=i32), order=gpu(10000, dtype=i32), slot=gpu(5000, 2, dtype=i32), ws=ws)
    with pytest.raises(ValueError, match="contiguous"):
        bm.moe_group(gpu(5000, 2, dtype=i32), 64, **out)
    with pytest.raises(ValueError, match="contiguous"):
        bm.moe_route(gpu(5000, 64), 2, ids=gpu(5000, 2, dtype=i32), g=gpu(5000, 2, dtype=torch.float32), **out)


@pytest.mark.parametrize("call, sizes", [
    # 65790 row tiles x 128 column tiles of 512 lanes; as many tokens as 256-lane work-groups pass 2^32 lanes
    (matmul, dict(E=65535, R=65535, x_rows=65535, N=32768, ldy=32768)),
    (matmul_dx, dict(E=65535, R=65535, K=32768, lddx=32768)),
    (combine, dict(T=1 << 24)), (combine_grad, dict(T=1 << 24)),
])
def test_what_no_grid_takes_is_refused(call, sizes):
    assert call(**sizes) == bm.ESHAPE
