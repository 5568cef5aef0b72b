"""A MoE layer resident in device memory, driven through libmpb.

PyTorch provides the device allocations and the stream; packing, routing and
the expert FFN all run in the library's kernels.
"""
from __future__ import annotations

import contextlib

import numpy as np
import torch

from . import _lib as M

XDTYPE = {"f16": M.MPB_F16, "bf16": M.MPB_BF16}
XTORCH = {"f16": torch.float16, "bf16": torch.bfloat16}


def _dev(a: np.ndarray, device) -> torch.Tensor:
    """Raw copy of a numpy array to the device (uint32/uint16 kept as int32/int16 bits)."""
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint32:
        a = a.view(np.int32)
    elif a.dtype == np.uint16:
        a = a.view(np.int16)
    return torch.from_numpy(a).to(device)


class DeviceLayer:
    """Packed pages, table images and pointer tables of one MoE layer.

    blocks: {i: (planes [8][N][Kd/32] uint32 canonical, luts list of 6
    [N][2**b] uint16)} for every i in 0..2(E+S)-1.
    q_dev: share an existing page table (e.g. several copies of one layer);
    by default a new one is created and bound with mpb_init.
    """

    def __init__(self, H, I, E, S, K, W_r, bias, q, blocks, device="cuda", q_dev=None, bind=True):
        self.H, self.I, self.E, self.S, self.K = H, I, E, S, K
        self.nb = 2 * (E + S)
        self.device = device
        self.W_r = torch.from_numpy(np.ascontiguousarray(W_r, np.float32)).to(device)
        self.bias = None if bias is None else torch.from_numpy(np.ascontiguousarray(bias, np.float32)).to(device)
        self.pages, self.luts = [], []
        plane_ptrs, lut_ptrs = [], []
        for i in range(self.nb):
            planes, luts = blocks[i]
            N, W = planes.shape[1], planes.shape[2]
            Kd = 32 * W
            canon = _dev(planes, device)
            nwords = M.mpb_plane_page_bytes(N, Kd) // 4
            pg = [torch.empty(nwords, dtype=torch.int32, device=device) for _ in range(8)]
            M.mpb_pack_block(canon, N, Kd, pg)
            del canon
            kind = i % 2  # 0: gate_up, 1: down
            imgs = []
            for b in range(3, 9):
                lut = _dev(luts[b - 3], device)
                img = torch.empty(M.mpb_table_image_bytes(kind, N, b) // 2, dtype=torch.int16, device=device)
                M.mpb_pack_table(kind, lut, N, b, img)
                imgs.append(img)
                del lut
            self.pages.append(pg)
            self.luts.append(imgs)
            plane_ptrs += [p.data_ptr() for p in pg]
            lut_ptrs += [t.data_ptr() for t in imgs]
        self.planes_table = torch.tensor(plane_ptrs, dtype=torch.int64, device=device)
        self.luts_table = torch.tensor(lut_ptrs, dtype=torch.int64, device=device)
        if q_dev is None:
            q_dev = torch.empty(self.nb, dtype=torch.int32, device=device)
            if bind:
                M.mpb_init(H, I, E, S, K, q_dev, np.asarray(q, np.int32))
        self.q_dev = q_dev
        torch.cuda.synchronize()

    @classmethod
    def from_synth(cls, layer, **kw):
        blocks = {i: (b.planes, b.luts) for i, b in layer.blocks.items()}
        return cls(layer.H, layer.I, layer.E, layer.S, layer.K, layer.W_r, layer.bias, layer.q, blocks, **kw)

    def weight_bytes(self):
        return sum(p.numel() * 4 for pg in self.pages for p in pg) + \
            sum(t.numel() * 2 for lt in self.luts for t in lt)

    # ---------------------------------------------------------------- calls
    # Where a call takes a stream, its results and workspaces are allocated for
    # that stream: a workspace freed on return is not handed out on another one
    # while the call's kernels may still run. The layer keeps none of them: calls
    # on several streams and captured graphs share no memory, and a captured call's
    # workspaces stay in its graph's pool whatever is called later.
    @staticmethod
    def _on(stream):
        return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)

    def alloc_route(self, T):
        """Router outputs for T tokens."""
        idx = torch.empty((T, self.K), dtype=torch.int32, device=self.device)
        w = torch.empty((T, self.K), dtype=torch.float32, device=self.device)
        return idx, w

    def alloc_ffn(self, T):
        out = torch.empty((T, self.H), dtype=torch.float32, device=self.device)
        ws = torch.empty(max(1, M.moe_ffn_workspace_bytes(T)), dtype=torch.uint8, device=self.device)
        return out, ws

    def alloc_fused(self, T):
        """Output and a zero-filled workspace for moe_fused (its counters must
        start at zero; each call leaves them zero)."""
        out = torch.empty((T, self.H), dtype=torch.float32, device=self.device)
        ws = torch.zeros(max(256, M.moe_fused_workspace_bytes(T)), dtype=torch.uint8, device=self.device)
        return out, ws

    def fused(self, X, xdtype, idx, w, out, ws, stream=None):
        M.moe_fused(X, XDTYPE[xdtype], self.W_r, self.bias, idx, w, self.planes_table, self.luts_table, self.q_dev,
                    out, ws, stream)

    def route(self, X, xdtype, idx, w, stream=None, ws=None):
        """moe_route; ws: a workspace of the caller's, or None for one of this call's own."""
        if ws is None:
            with self._on(stream):
                ws = torch.empty(max(1, M.moe_route_workspace_bytes(X.shape[0], self.E)), dtype=torch.uint8,
                                 device=self.device)
        M.moe_route(X, XDTYPE[xdtype], self.W_r, self.bias, self.K, idx, w, ws, stream)

    def ffn(self, X, xdtype, idx, w, out, ws, stream=None):
        M.moe_ffn(X, XDTYPE[xdtype], idx, w, self.planes_table, self.luts_table, self.q_dev, out, ws, stream)

    def forward(self, X, xdtype, stream=None):
        T = X.shape[0]
        with self._on(stream):
            idx, w = self.alloc_route(T)
            out, ws = self.alloc_ffn(T)
        self.route(X, xdtype, idx, w, stream)
        self.ffn(X, xdtype, idx, w, out, ws, stream)
        return idx, w, out

    # ---------------------------------------------------------------- the block around the layer
    def alloc_rows(self, T, xdtype):
        """[T][H] activations."""
        return torch.empty((T, self.H), dtype=XTORCH[xdtype], device=self.device)

    def norm_in(self, r, xdtype, gamma, eps=1e-6, stream=None):
        """The first block's normed input of a residual stream r [T][H]."""
        with self._on(stream):
            x = self.alloc_rows(r.shape[0], xdtype)
        M.moe_block_norm(None, r, XDTYPE[xdtype], None, None, gamma, 1.0, eps, None, x, stream)
        return x

    def adapt(self, X, xdtype, adapters, out, stream=None):
        """Adds every token's adapter to out [T][H] in place. adapters: a dict with A [n][R][H], B [n][H][R],
        adapter [T], and ranks [n] and scales [n] if they differ from R and 1."""
        A = adapters["A"]
        with self._on(stream):
            ws = torch.empty(M.moe_adapters_workspace_bytes(X.shape[0], self.H, A.shape[0], A.shape[1]),
                             dtype=torch.uint8, device=self.device)
        M.moe_adapters(X, XDTYPE[xdtype], A, adapters["B"], adapters.get("ranks"), adapters.get("scales"),
                       adapters["adapter"], out, out, ws, stream)

    def block(self, X, r, xdtype, gamma_post=None, gamma_next=None, gate=None, scale=1.0, eps=1e-6, adapters=None,
              stream=None):
        """One residual block: the layer on X [T][H] (the normed stream), its tokens' adapters, and the layer's output
        normed, gated and scaled onto the stream r [T][H]. Returns idx, w, the layer's output with the adapters', the
        stream after the block and (with gamma_next) the next block's normed input."""
        idx, w, out = self.forward(X, xdtype, stream)
        with self._on(stream):
            r_out = self.alloc_rows(r.shape[0], xdtype)
            x_next = None if gamma_next is None else self.alloc_rows(r.shape[0], xdtype)
        if adapters is not None:
            self.adapt(X, xdtype, adapters, out, stream)
        M.moe_block_norm(out, r, XDTYPE[xdtype], gate, gamma_post, gamma_next, scale, eps, r_out, x_next, stream)
        return idx, w, out, r_out, x_next

    def block_norm_grad(self, out, r_out, xdtype, dr_out, dx_next, gamma_post=None, gamma_next=None, gate=None, scale=1.0,
                        eps=1e-6, stream=None):
        """Backward pass of block's norms from its out and r_out: a dict of the gradients of r, out, the gate and the
        two norms' weights (None where there is none)."""
        T = r_out.shape[0]
        f32 = dict(dtype=torch.float32, device=self.device)
        with self._on(stream):
            g = {"r": self.alloc_rows(T, xdtype), "out": torch.empty((T, self.H), **f32),
                 "gate": None if gate is None else torch.empty_like(gate),
                 "gamma_post": None if gamma_post is None else torch.empty(self.H, **f32),
                 "gamma_next": None if gamma_next is None else torch.empty(self.H, **f32)}
            ws = torch.empty(M.moe_block_norm_grad_workspace_bytes(T, self.H), dtype=torch.uint8, device=self.device)
        M.moe_block_norm_grad(out, r_out, XDTYPE[xdtype], gate, gamma_post, gamma_next, scale, eps, dr_out, dx_next,
                              g["r"], g["out"], g["gate"], g["gamma_post"], g["gamma_next"], ws, stream)
        return g

    def router_loss(self, X, xdtype, idx, mask=None, alpha=0.01, beta=0.001, stream=None):
        """Balance and z loss of the routed batch: a dict of loss [3], counts [E + 1], prob [E] and what the gradient
        needs (logits, lse, and the call's arguments)."""
        T, f32 = X.shape[0], dict(dtype=torch.float32, device=self.device)
        with self._on(stream):
            s = {"logits": torch.empty((T, self.E), **f32), "lse": torch.empty(T, **f32),
                 "counts": torch.empty(self.E + 1, dtype=torch.int32, device=self.device),
                 "prob": torch.empty(self.E, **f32), "loss": torch.empty(3, **f32),
                 "args": (X, xdtype, idx, mask, alpha, beta)}
            ws = torch.empty(M.moe_router_loss_workspace_bytes(T, self.H, self.E), dtype=torch.uint8,
                             device=self.device)
        M.moe_router_loss(X, XDTYPE[xdtype], self.W_r, self.bias, idx, mask, alpha, beta, s["logits"], s["lse"],
                          s["counts"], s["prob"], s["loss"], ws, stream)
        return s

    def router_loss_grad(self, s, gw=None, gloss=None, stream=None):
        """Gradients (X, W_r, bias) of router_loss's loss[0] times gloss, and of the routing weights (gw [T][K])."""
        X, xdtype, idx, mask, alpha, beta = s["args"]
        f32 = dict(dtype=torch.float32, device=self.device)
        with self._on(stream):
            dX, dW, db = torch.empty(X.shape, **f32), torch.empty((self.E, self.H), **f32), torch.empty(self.E, **f32)
            ws = torch.empty(M.moe_router_loss_workspace_bytes(X.shape[0], self.H, self.E), dtype=torch.uint8,
                             device=self.device)
        M.moe_router_loss_grad(X, XDTYPE[xdtype], self.W_r, idx, mask, s["logits"], s["lse"], s["counts"], alpha, beta,
                               gw, gloss, dX, dW, db, ws, stream)
        return dX, dW, db
