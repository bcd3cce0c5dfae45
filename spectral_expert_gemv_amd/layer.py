"""MoE layers resident in device memory: the packed spectral gate/up layer, and
the layer of dense or 4-bit experts (router, experts, combine) beside it.

Host work is layout only: the library packer quantizes and packs each
linear type, and Phi_gate, Phi_up (din x r each) are stored transposed and
stacked as one 2r x din fp16 array so that one projection launch produces
z_gate and z_up together.  Everything the decode step computes runs in the
library's kernels.
"""
import numpy as np

from . import bitsmoe


class DeviceLayer:
    def __init__(self, phi_gate, phi_up, a_gate, a_up, p_gate, p_up, bits_gate, bits_up,
                 device="cuda", blobs=None):
        import torch
        self.E, self.r, self.dout = p_gate.shape
        self.din = phi_gate.shape[0]
        if blobs is None:
            blobs = (bitsmoe.pack(p_gate, a_gate, bits_gate), bitsmoe.pack(p_up, a_up, bits_up))
        self.host_blobs = blobs
        phi_t = np.concatenate([np.asarray(phi_gate, np.float16).T,
                                np.asarray(phi_up, np.float16).T], axis=0)
        self.phi_t = torch.from_numpy(np.ascontiguousarray(phi_t)).to(device)
        self.blob_gate = torch.from_numpy(blobs[0]).to(device)
        self.blob_up = torch.from_numpy(blobs[1]).to(device)
        self.device = device

    @classmethod
    def from_synth(cls, layer, device="cuda"):
        return cls(layer.phi["gate"], layer.phi["up"], layer.a["gate"], layer.a["up"],
                   layer.p["gate"], layer.p["up"], layer.bits["gate"], layer.bits["up"],
                   device=device)

    def workspace(self, T, k):
        import torch
        n = bitsmoe.moe_gateup_workspace_size(T, k, self.E, self.din, self.dout, self.r)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device=self.device)
        bitsmoe.workspace_init(ws)
        return ws

    def gateup(self, x, ids, h=None, ws=None, stream=None):
        import torch
        T, k = ids.shape
        if h is None:
            h = torch.empty((T, k, self.dout), dtype=torch.float32, device=self.device)
        if ws is None:
            ws = self.workspace(T, k)
        bitsmoe.moe_gateup(self.blob_gate, self.blob_up, self.phi_t, x, ids, self.E, self.dout,
                           self.r, h, ws, stream=stream)
        return h


class ExpertLayer:
    """A mixture-of-experts layer with dense or plain 4-bit experts:

        out_t = sum over the k experts e of token t of
                g_{t,e} W2_e (SiLU(W1g_e x_t) * (W1u_e x_t)),

    with g the softmax weights of the k largest router logits.  w1: E x 2F x D
    (gate rows first), w2: E x D x F device tensors, float16 or bfloat16 (for
    4-bit experts what ExpertLayer.w4 makes of dense host weights).  Every step
    is one of the library's operators; tokens are grouped by expert once and
    read in place by the first product.  A token whose logits are all -inf gets
    zeros; one whose logits hold a NaN or +inf gets NaN (out and dlogits; its
    dx is 0, and no expert's weights and no other token's rows see it).
    """

    def __init__(self, w1, w2, renorm=True, scale=1.0, group=None):
        self.w1, self.w2 = w1, w2
        self.renorm, self.scale, self.group = renorm, scale, group
        if group is None:
            self.E, self.D, self.F = w2.shape
        else:
            self.E, self.D = w2[0].shape[:2]
            self.F = 2 * w2[0].shape[2]

    @classmethod
    def w4(cls, w1, w2, group=128, device="cuda", **kw):
        """4-bit experts from dense host weights (float32 numpy arrays)."""
        import torch

        def pack(w):
            return tuple(torch.from_numpy(a).to(device) for a in bitsmoe.w4_pack(w, group))
        return cls(pack(w1), pack(w2), group=group, **kw)

    def route(self, logits, k, stream=None):
        """(ids, g, bounds, order, slot) of T x E logits."""
        import torch
        T = logits.shape[0]
        new = bitsmoe._new
        dev, i32 = logits.get_device(), torch.int32
        bounds, order = new(self.E + 1, i32, dev, stream), new(T * k, i32, dev, stream)
        slot = new((T, k), i32, dev, stream)
        ids, g = bitsmoe.moe_route(logits, k, renorm=self.renorm, scale=self.scale, bounds=bounds,
                                   order=order, slot=slot, stream=stream)
        return ids, g, bounds, order, slot

    def _product(self, x, w, bounds, stream, **kw):
        if self.group is None:
            return bitsmoe.grouped_matmul(x, w, bounds, stream=stream, **kw)
        return bitsmoe.w4_matmul(x, *w, bounds=bounds, stream=stream, **kw)

    def forward(self, x, logits, k, out=None, stream=None):
        """out (T x D, x's dtype or out's) of tokens x (T x D)."""
        _, g, bounds, order, slot = self.route(logits, k, stream)
        h = self._product(x, self.w1, bounds, stream, rows=order, div=k, act="silu_mul")
        y = self._product(h, self.w2, bounds, stream)
        return bitsmoe.moe_combine(y, slot, g, out, stream=stream)

    def gradients(self, x, logits, k, dout, stream=None):
        """(out, dx, dlogits, dw1, dw2) of dense experts: the forward pass and
        the gradients of <dout, out>; dw1 and dw2 in float32."""
        if self.group is not None:
            raise ValueError("4-bit experts have no gradients")
        bm, s = bitsmoe, stream
        ids, g, bounds, order, slot = self.route(logits, k, s)
        a = bm.grouped_matmul(x, self.w1, bounds, rows=order, div=k, stream=s)
        h = bm.silu_mul(a, bounds=bounds, stream=s)
        y = bm.grouped_matmul(h, self.w2, bounds, stream=s)
        out = bm.moe_combine(y, slot, g, bm._new(dout.shape, dout.dtype, x.get_device(), s), stream=s)
        dy, dg = bm.moe_combine_grad(dout, y, slot, g, stream=s)
        dh = bm.grouped_matmul_dx(dy, self.w2, bounds, stream=s)
        dw2 = bm.grouped_matmul_dw(dy, h, bounds, stream=s)
        da = bm.silu_mul_grad(a, dh, bounds=bounds, stream=s)
        dw1 = bm.grouped_matmul_dw(da, x, bounds, rows=order, div=k, stream=s)
        # (a sorted row's dx is rounded to x's type before a token's rows are added up in
        # float32: half the bytes of float32 rows, at half a step of each term)
        dx = bm.moe_combine(bm.grouped_matmul_dx(da, self.w1, bounds, stream=s), slot, stream=s)
        dlogits = bm.moe_route_grad(logits, ids, dg, renorm=self.renorm, scale=self.scale, stream=s)
        return out, dx, dlogits, dw1, dw2
