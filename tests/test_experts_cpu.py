"""CPU checks of the expert layer's entry points: what they refuse before
anything is enqueued, and the host packer of 4-bit weights."""
import ctypes

import numpy as np
import pytest

from spectral_expert_gemv_amd import bitsmoe as bm

torch = pytest.importorskip("torch")

P = 4096  # a pointer that no refused call follows
F32, F16, BF16 = 0, 1, 2


def _status(name, *args):
    return getattr(bm._lib, "bitsmoe_" + name)(*args)


def route(**kw):
    a = dict(dtype=F32, logits=P, ld=64, T=3, E=64, k=4, renorm=0, scale=1.0, ids=P, g=P,
             bounds=None, order=None, slot=None, ws=None, ws_bytes=0)
    a.update(kw)
    return _status("moe_route", *a.values(), None)


def route_grad(**kw):
    a = dict(dtype=F32, logits=P, ld=64, ids=P, dg=P, T=3, E=64, k=4, renorm=0, scale=1.0,
             dlogits=P, ldd=64)
    a.update(kw)
    return _status("moe_route_grad", *a.values(), None)


def group(**kw):
    a = dict(ids=P, P=10, E=64, bounds=P, order=P, slot=P, ws=None, ws_bytes=0)
    a.update(kw)
    return _status("moe_group", *a.values(), None)


def matmul(**kw):
    a = dict(dtype=F16, x=P, ldx=64, x_rows=10, rows=None, div=1, w=P, bounds=P, R=10, E=4, N=32,
             K=64, act=0, y=P, y_dtype=F16, ldy=32, ws=None, ws_bytes=0)
    a.update(kw)
    return _status("grouped_matmul", *a.values(), None)


def matmul_dx(**kw):
    a = dict(dtype=F16, dy=P, lddy=32, w=P, bounds=P, R=10, E=4, N=32, K=64, dx=P, dx_dtype=F16,
             lddx=64, ws=None, ws_bytes=0)
    a.update(kw)
    return _status("grouped_matmul_dx", *a.values(), None)


def matmul_dw(**kw):
    a = dict(dtype=F16, dy=P, lddy=32, x=P, ldx=64, x_rows=10, rows=None, div=1, bounds=P, R=10,
             E=4, N=32, K=64, dw=P, dw_dtype=F32, ws=None, ws_bytes=0)
    a.update(kw)
    return _status("grouped_matmul_dw", *a.values(), None)


def act(**kw):
    a = dict(dtype=F16, a=P, lda=64, bounds=None, R=10, E=0, F=32, h=P, ldh=32)
    a.update(kw)
    return _status("silu_mul", *a.values(), None)


def act_grad(**kw):
    a = dict(dtype=F16, a=P, lda=64, dh=P, lddh=32, bounds=None, R=10, E=0, F=32, da=P, ldda=64)
    a.update(kw)
    return _status("silu_mul_grad", *a.values(), None)


def combine(**kw):
    a = dict(y_dtype=F16, y=P, ldy=64, R=10, slot=P, g=P, T=5, k=2, D=64, out=P, out_dtype=F16,
             ldo=64)
    a.update(kw)
    return _status("moe_combine", *a.values(), None)


def combine_grad(**kw):
    a = dict(dout=P, out_dtype=F16, ldo=64, y_dtype=F16, y=P, ldy=64, R=10, slot=P, g=P, T=5, k=2,
             D=64, dy=P, lddy=64, dg=P)
    a.update(kw)
    return _status("moe_combine_grad", *a.values(), None)


def w4(**kw):
    a = dict(dtype=F16, x=P, ldx=128, x_rows=10, rows=None, div=1, codes=P, scales=P, mins=P,
             G=64, bounds=P, R=10, E=4, N=32, K=128, act=0, y=P, y_dtype=F16, ldy=32)
    a.update(kw)
    return _status("w4_matmul", *a.values(), None)


@pytest.mark.parametrize("call, wrong, status", [
    (route, dict(dtype=3), bm.EINVAL), (route, dict(dtype=-1), bm.EINVAL),
    (route, dict(E=0, k=1), bm.ESHAPE), (route, dict(E=2049, ld=4096), bm.ESHAPE),
    (route, dict(k=0), bm.EINVAL), (route, dict(k=65), bm.EINVAL),
    (route, dict(E=3, k=4), bm.EINVAL), (route, dict(T=-1), bm.ESHAPE),
    (route, dict(T=(1 << 24) + 1), bm.ESHAPE), (route, dict(ld=63), bm.ESHAPE),
    (route, dict(logits=None), bm.EINVAL), (route, dict(ids=None), bm.EINVAL),
    (route, dict(g=None), bm.EINVAL), (route, dict(bounds=P), bm.EINVAL),
    (route, dict(bounds=P, order=P), bm.EINVAL), (route, dict(order=P, slot=P), bm.EINVAL),
    (route, dict(T=5000, bounds=P, order=P, slot=P), bm.ENOSPC),
    (route, dict(T=5000, bounds=P, order=P, slot=P, ws=None, ws_bytes=1 << 30), bm.ENOSPC),
    (route, dict(T=5000, bounds=P, order=P, slot=P, ws=P + 2, ws_bytes=1 << 30), bm.EINVAL),
    (route_grad, dict(dtype=7), bm.EINVAL), (route_grad, dict(ldd=10), bm.ESHAPE),
    (route_grad, dict(ld=10), bm.ESHAPE), (route_grad, dict(dg=None), bm.EINVAL),
    (route_grad, dict(dlogits=None), bm.EINVAL), (route_grad, dict(ids=None), bm.EINVAL),
    (group, dict(P=-1), bm.ESHAPE), (group, dict(E=0), bm.ESHAPE),
    (group, dict(E=2049), bm.ESHAPE), (group, dict(bounds=None), bm.EINVAL),
    (group, dict(ids=None), bm.EINVAL), (group, dict(order=None), bm.EINVAL),
    (group, dict(P=100000), bm.ENOSPC),
    (matmul, dict(dtype=F32), bm.EINVAL), (matmul, dict(y_dtype=BF16), bm.EINVAL),
    (matmul, dict(E=0), bm.ESHAPE), (matmul, dict(N=0), bm.ESHAPE), (matmul, dict(K=0), bm.ESHAPE),
    (matmul, dict(R=-1), bm.ESHAPE), (matmul, dict(bounds=None), bm.EINVAL),
    (matmul, dict(w=None), bm.EINVAL), (matmul, dict(x=None), bm.EINVAL),
    (matmul, dict(y=None), bm.EINVAL), (matmul, dict(ldx=63), bm.ESHAPE),
    (matmul, dict(ldy=31), bm.ESHAPE), (matmul, dict(act=2), bm.EINVAL),
    (matmul, dict(rows=P, x_rows=0), bm.ESHAPE), (matmul_dw, dict(rows=P, x_rows=0), bm.ESHAPE),
    (w4, dict(rows=P, x_rows=0), bm.ESHAPE), (matmul, dict(E=65535, R=1 << 26, x_rows=1 << 26), bm.ESHAPE),
    (w4, dict(E=65535, R=1 << 24, x_rows=1 << 24), bm.ESHAPE),
    (matmul, dict(x_rows=9), bm.ESHAPE), (matmul, dict(rows=P, div=0), bm.ESHAPE),
    (matmul, dict(rows=P, x_rows=-1), bm.ESHAPE), (matmul, dict(K=(1 << 20) + 1, ldx=1 << 21), bm.ESHAPE),
    (matmul_dx, dict(dtype=F32), bm.EINVAL), (matmul_dx, dict(dx_dtype=BF16), bm.EINVAL),
    (matmul_dx, dict(lddy=31), bm.ESHAPE), (matmul_dx, dict(lddx=63), bm.ESHAPE),
    (matmul_dx, dict(dx=None), bm.EINVAL), (matmul_dx, dict(bounds=None), bm.EINVAL),
    (matmul_dw, dict(dtype=F32), bm.EINVAL), (matmul_dw, dict(dw_dtype=BF16), bm.EINVAL),
    (matmul_dw, dict(ldx=63), bm.ESHAPE), (matmul_dw, dict(dw=None), bm.EINVAL),
    (matmul_dw, dict(x=None), bm.EINVAL), (matmul_dw, dict(x_rows=9), bm.ESHAPE),
    (matmul_dw, dict(R=0, dw=None), bm.EINVAL),
    # operands that are not 16-byte rows, without (enough of) a workspace
    (matmul, dict(R=4000, x_rows=4000, ldx=65), bm.ENOSPC), (matmul, dict(R=4000, x_rows=4000, x=P + 2), bm.ENOSPC),
    (matmul_dx, dict(N=33, lddy=40), bm.ENOSPC), (matmul_dx, dict(K=63), bm.ENOSPC),
    (matmul_dx, dict(N=33, lddy=40, ws=P, ws_bytes=100), bm.ENOSPC),
    (matmul_dx, dict(N=33, lddy=40, ws=P + 16, ws_bytes=1 << 20), bm.EINVAL),
    (matmul_dw, dict(K=63), bm.ENOSPC), (matmul_dw, dict(dy=P + 4), bm.ENOSPC),
    (act, dict(dtype=F32), bm.EINVAL), (act, dict(F=0), bm.ESHAPE), (act, dict(lda=63), bm.ESHAPE),
    (act, dict(ldh=31), bm.ESHAPE), (act, dict(bounds=P), bm.ESHAPE), (act, dict(h=None), bm.EINVAL),
    (act_grad, dict(ldda=63), bm.ESHAPE), (act_grad, dict(da=None), bm.EINVAL),
    (act_grad, dict(dh=None), bm.EINVAL),
    (combine, dict(y_dtype=F32), bm.EINVAL), (combine, dict(out_dtype=BF16), bm.EINVAL),
    (combine, dict(k=0), bm.ESHAPE), (combine, dict(D=0), bm.ESHAPE), (combine, dict(ldy=63), bm.ESHAPE),
    (combine, dict(slot=None), bm.EINVAL), (combine, dict(y=None), bm.EINVAL),
    (combine_grad, dict(dy=None), bm.EINVAL), (combine_grad, dict(lddy=63), bm.ESHAPE),
    (combine_grad, dict(dout=None), bm.EINVAL),
    (w4, dict(dtype=F32), bm.EINVAL), (w4, dict(y_dtype=BF16), bm.EINVAL), (w4, dict(G=16), bm.ESHAPE),
    (w4, dict(G=256, K=256, ldx=256), bm.ESHAPE), (w4, dict(K=96, ldx=96), bm.ESHAPE),
    (w4, dict(bounds=None), bm.EINVAL), (w4, dict(codes=P + 8), bm.EINVAL),
    (w4, dict(scales=P + 2), bm.EINVAL), (w4, dict(mins=P + 2), bm.EINVAL),
    (w4, dict(codes=None), bm.EINVAL), (w4, dict(x_rows=9), bm.ESHAPE), (w4, dict(act=5), bm.EINVAL),
    (w4, dict(rows=P, div=0), bm.ESHAPE), (w4, dict(ldx=127), bm.ESHAPE),
])
def test_refuses_before_anything_is_enqueued(call, wrong, status):
    # (without a GPU a call that went on to a launch would return EHIP)
    assert call(**wrong) == status
    assert bm._lib.bitsmoe_last_error_detail()


@pytest.mark.parametrize("call, empty", [
    (route, dict(T=0, logits=None, ids=None, g=None)), (route_grad, dict(T=0)),
    (matmul, dict(R=0, x=None, y=None, x_rows=0)), (matmul_dx, dict(R=0, dy=None, dx=None)),
    (act, dict(R=0, a=None, h=None)), (act_grad, dict(R=0)), (combine, dict(T=0)),
    (combine_grad, dict(T=0)), (w4, dict(R=0, x=None, y=None, x_rows=0)),
])
def test_nothing_to_do_is_fine(call, empty):
    assert call(**empty) == bm.OK


def test_group_workspace():
    assert bm.moe_group_workspace_size(8, 128) == 0
    assert bm.moe_group_workspace_size(4096, 512) == 0
    n = bm.moe_group_workspace_size(131072, 128)
    assert n > 0 and n % (4 * 129) == 0
    out = ctypes.c_size_t()
    assert bm._lib.bitsmoe_moe_group_workspace_size(8, 0, ctypes.byref(out)) == bm.ESHAPE
    assert bm._lib.bitsmoe_moe_group_workspace_size(8, 4, None) == bm.EINVAL


def test_matmul_workspace():
    size = ctypes.c_size_t(7)

    def need(op, a=P, lda=64, a_rows=10, b=P, ldb=64, b_rows=10, R=10, E=4, N=32, K=64, act=0):
        assert _status("grouped_matmul_workspace_size", op, a, lda, a_rows, b, ldb, b_rows, R, E, N,
                       K, act, ctypes.byref(size)) == bm.OK
        return size.value
    assert need(0) == need(1, lda=32) == need(2, lda=32) == 0
    assert need(0, K=63, lda=63) == 0              # few rows: read in place
    assert need(0, K=63, lda=63, R=4000, a_rows=4000) == 4000 * 128 + 4 * 32 * 128
    assert need(1, lda=33, N=33) == 10 * 80 // 256 * 256 + 256      # dy alone
    assert need(2, ldb=65) == 10 * 128 // 256 * 256                 # x alone
    assert _status("grouped_matmul_workspace_size", 3, P, 64, 1, P, 64, 1, 1, 1, 8, 8, 0,
                   ctypes.byref(size)) == bm.EINVAL
    assert _status("grouped_matmul_workspace_size", 0, P, 64, 1, P, 64, 1, 1, 1, 8, 8, 0,
                   None) == bm.EINVAL


def test_binding_refuses_host_tensors_and_wrong_layouts():
    x, w = torch.zeros(4, 64).half(), torch.zeros(2, 8, 64).half()
    b = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="not on a GPU"):
        bm.grouped_matmul(x, w, b)
    with pytest.raises(ValueError, match="not on a GPU"):
        bm.moe_route(torch.zeros(2, 8), 2)
    with pytest.raises(ValueError, match="act="):
        bm.grouped_matmul(x, w, b, act="relu")
    with pytest.raises(ValueError, match="act="):
        bm.grouped_matmul(x, torch.zeros(2, 7, 64).half(), b, act="silu_mul")
    with pytest.raises(ValueError, match="contiguous"):
        bm._matrix("x", torch.zeros(8, 4).t())
    with pytest.raises(ValueError, match="shape"):
        bm._matrix("x", torch.zeros(8, 4), (8, 5))
    with pytest.raises(ValueError, match="int32"):
        bm._array("ids", torch.zeros(3, dtype=torch.int64), torch.int32, (3,))
    with pytest.raises(ValueError, match="contiguous"):
        bm._array("g", torch.zeros(4, 3).t(), torch.float32, (3, 4))
    with pytest.raises(ValueError, match="dtype"):
        bm._dtype(torch.zeros(2, dtype=torch.float64))
    # one row or one column: the stride says nothing
    assert bm._matrix("x", torch.zeros(1, 8))[1] == 8
    assert bm._matrix("x", torch.zeros(5, 3)[:, :1])[1] == 3


# ------------------------------------------------------- 4-bit host packer

@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("scale", [1.0, 1e-3, 3e4])
def test_w4_pack_is_the_quantizer_rule(group, scale):
    rng = np.random.default_rng(group)
    w = (rng.standard_normal((3, 5, 256)) * scale).clip(-60000, 60000).astype(np.float32)
    w[0, 0] = 0.0            # a constant group: step 1
    w[1, 2, :group] = 0.25   # another
    w[2, 4, :group] *= 1e-7  # steps below float16's normal range
    codes, scales, mins = bm.w4_pack(w, group)
    v = w.reshape(3, 5, -1, group)
    s = ((v.max(-1) - v.min(-1)) / np.float32(15)).astype(np.float16)
    s[s == 0] = 1
    m = v.min(-1).astype(np.float16)
    q = np.clip(np.rint((v - m.astype(np.float32)[..., None]) / s.astype(np.float32)[..., None]),
                0, 15).astype(np.uint8).reshape(3, 5, 256)
    assert np.array_equal(scales.view(np.uint16), s.view(np.uint16))
    assert np.array_equal(mins, m)
    assert np.array_equal(codes & 15, q[..., 0::2]) and np.array_equal(codes >> 4, q[..., 1::2])


def test_w4_pack_refuses():
    w = np.zeros((2, 64), np.float32)
    w[1, 3] = np.nan
    with pytest.raises(bm.BitsMoEError) as e:
        bm.w4_pack(w, 32)
    assert e.value.status == bm.EBITS
    with pytest.raises(ValueError):
        bm.w4_pack(np.zeros((2, 48), np.float32), 32)
    with pytest.raises(bm.BitsMoEError):
        bm.w4_pack(np.zeros((2, 48), np.float32), 16)


SANITIZED = r"""
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include "bitsmoe.h"
int main() {
  const int groups[] = {32, 64, 128};
  for (int g : groups) {
    const int K = 256, rows = 7;
    float* w = (float*)malloc(sizeof(float) * rows * K);
    for (int i = 0; i < rows * K; ++i) w[i] = (float)((i * 2654435761u) % 2001) * 60.f - 60000.f;
    for (int i = 0; i < K; ++i) w[i] = 0.f, w[K + i] = i % 2 ? -0.f : 0.f, w[2 * K + i] = 1e-8f * i;
    unsigned char* c = (unsigned char*)malloc(rows * K / 2);
    unsigned short *s = (unsigned short*)malloc(2 * rows * K / g), *m = (unsigned short*)malloc(2 * rows * K / g);
    if (bitsmoe_w4_pack(w, rows, K, g, c, s, m)) return 1;
    if (bitsmoe_w4_pack(w, rows, K, 16, c, s, m) != BITSMOE_ESHAPE) return 2;
    if (bitsmoe_w4_pack(w, rows, K + 8, g, c, s, m) != BITSMOE_ESHAPE) return 3;
    if (bitsmoe_w4_pack(w, -1, K, g, c, s, m) != BITSMOE_ESHAPE) return 4;
    if (bitsmoe_w4_pack(w, 0, K, g, 0, 0, 0)) return 5;
    if (bitsmoe_w4_pack(w, rows, K, g, 0, s, m) != BITSMOE_EINVAL) return 6;
    w[rows * K - 1] = 60001.f;
    if (bitsmoe_w4_pack(w, rows, K, g, c, s, m) != BITSMOE_EBITS) return 7;
    free(w), free(c), free(s), free(m);
  }
  puts("ok");
  return 0;
}
"""


def test_w4_pack_under_sanitizers(tmp_path):
    import os
    import shutil
    import subprocess
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    csrc = os.path.join(root, "spectral_expert_gemv_amd", "csrc")
    src = tmp_path / "w4.cpp"
    src.write_text(SANITIZED)
    exe = str(tmp_path / "w4")
    subprocess.run([gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-I", os.path.join(root, "include"), "-I", csrc,
                    os.path.join(csrc, "common.cpp"), os.path.join(csrc, "experts", "w4_pack.cpp"),
                    str(src), "-o", exe], check=True)
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
