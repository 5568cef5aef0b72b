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
ACT = {"none": M.MPB_ACT_NONE, "relu": M.MPB_ACT_RELU, "silu": M.MPB_ACT_SILU, "gelu": M.MPB_ACT_GELU,
       "gelu_tanh": M.MPB_ACT_GELU_TANH}
PAIRS = {"halves": M.MPB_PAIRS_HALVES, "neighbours": M.MPB_PAIRS_NEIGHBOURS}


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
        """Adds every token's adapter to out [T][N] in place (N is H for the layer itself). adapters: a dict with A
        [n][R][Kd], B [n][N][R] for X [T][Kd], adapter [T], and ranks [n] and scales [n] if they differ from R and 1."""
        A = adapters["A"]
        with self._on(stream):
            ws = torch.empty(M.moe_adapters_workspace_bytes(X.shape[0], X.shape[1], A.shape[0], A.shape[1]),
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

    # ---------------------------------------------------------------- the dense operators beside the layer
    def project(self, X, xdtype, W, bias=None, act="none", res=None, keep=False, f32=False, adapters=None, stream=None):
        """res + act(X W^T + bias) for X [T][Kd] and W [N][Kd], of X's type or (f32) fp32. adapters (see adapt) are added
        to a projection without activation, which is then fp32. keep: returns (y, z), z for project_grad."""
        T, N = X.shape[0], W.shape[0]
        if adapters is not None and ACT[act] != M.MPB_ACT_NONE:
            raise M.MpbError("project", -1, "adapters are added to a projection without activation")
        with self._on(stream):
            y = torch.empty((T, N), dtype=torch.float32 if f32 or adapters is not None else XTORCH[xdtype], device=self.device)
            z = torch.empty((T, N), dtype=XTORCH[xdtype], device=self.device) if keep else None
            ws = torch.empty(M.moe_linear_workspace_bytes(T, X.shape[1], N), dtype=torch.uint8, device=self.device)
        M.moe_linear(X, XDTYPE[xdtype], W, bias, ACT[act], res, z, y, ws, stream)
        if adapters is not None:
            self.adapt(X, xdtype, adapters, y, stream)
        return (y, z) if keep else y

    def project_grad(self, X, xdtype, W, dy, act="none", z=None, stream=None):
        """Gradients of project from dy (X's type or fp32) and, with an activation, z: a dict of X, W and bias."""
        (T, Kd), N = X.shape, W.shape[0]
        f32 = dict(dtype=torch.float32, device=self.device)
        dyt = M.MPB_F32 if dy.dtype is torch.float32 else XDTYPE[xdtype]
        with self._on(stream):
            g = {"X": torch.empty((T, Kd), dtype=XTORCH[xdtype], device=self.device), "W": torch.empty((N, Kd), **f32),
                 "bias": torch.empty(N, **f32)}
            ws = torch.empty(M.moe_linear_grad_workspace_bytes(T, Kd, N, ACT[act], dyt), dtype=torch.uint8,
                             device=self.device)
        M.moe_linear_grad(X, XDTYPE[xdtype], W, ACT[act], z, dy, g["X"], g["W"], g["bias"], ws, stream)
        return g

    def heads(self, q, k, xdtype, gamma_q=None, gamma_k=None, pos=None, freq=None, axis=None, pairs="halves", eps=1e-6,
              stream=None):
        """Norms of the heads q [T][Hq][D] and k [T][Hk][D] (views of a packed projection, k may be None) and their
        rotation by pos [A][T] (freq [Dr / 2], axis [Dr / 2] with several axes). Returns contiguous q and k."""
        with self._on(stream):
            out = [None if t is None else torch.empty(t.shape, dtype=XTORCH[xdtype], device=self.device) for t in (q, k)]
        M.moe_head_norm(q, k, XDTYPE[xdtype], gamma_q, gamma_k, eps, pos, axis, freq, PAIRS[pairs], *out, stream)
        return tuple(out)

    def heads_grad(self, q, k, xdtype, dq_out, dk_out, gamma_q=None, gamma_k=None, pos=None, freq=None, axis=None,
                   pairs="halves", eps=1e-6, stream=None):
        """Gradients of heads: a dict of q, k, gamma_q and gamma_k (None where there is none)."""
        T, Hq, D = dq_out.shape
        Hk = 0 if dk_out is None else dk_out.shape[1]
        with self._on(stream):
            g = {n: None if t is None else torch.empty(t.shape, dtype=XTORCH[xdtype], device=self.device)
                 for n, t in (("q", dq_out), ("k", dk_out))}
            g |= {n: None if t is None else torch.empty_like(t) for n, t in (("gamma_q", gamma_q), ("gamma_k", gamma_k))}
            ws = torch.empty(M.moe_head_norm_grad_workspace_bytes(T, Hq, Hk, D), dtype=torch.uint8, device=self.device)
        M.moe_head_norm_grad(q, k, XDTYPE[xdtype], gamma_q, gamma_k, eps, pos, axis, freq, PAIRS[pairs], dq_out, dk_out,
                             g["q"], g["k"], g["gamma_q"], g["gamma_k"], ws, stream)
        return g

    @staticmethod
    def _like_logits(S):
        """A tensor with S's shape, row stride and place against a 16-byte boundary; zeros between the rows, so that
        the logits of a vocabulary padded for project_grad get a gradient of the padded width."""
        if S.dim() != 2 or (S.shape[0] > 1 and S.stride(0) < S.shape[1]):
            return torch.empty_like(S)  # which the call refuses
        (T, V), ld, at = S.shape, S.stride(0), S.data_ptr() % 16 // S.element_size()
        if T == 1 and not V <= ld <= 2 * V:  # one row's stride says nothing
            ld = V
        buf = torch.empty(T * ld + at, dtype=S.dtype, device=S.device)
        if ld > V:
            torch.as_strided(buf, (T, ld - V), (ld, 1), at + V).zero_()
        return torch.as_strided(buf, (T, V), (ld, 1), at)

    def distill(self, S, ids, teacher, teacher_lse=None, weight=None, tau=1.0, grad=False, gloss=None, stream=None):
        """Loss of student logits S [T][V] (fp16, bf16 or fp32) against a teacher's top logits [T][k]: a dict of loss
        [1], kl [T], with grad the gradient dS (with S's row stride, zeros between the rows), and what distill_grad
        needs. S may be the first V columns of wider logits."""
        T, f32 = S.shape[0], dict(dtype=torch.float32, device=self.device)
        sd = {torch.float16: M.MPB_F16, torch.bfloat16: M.MPB_BF16, torch.float32: M.MPB_F32}.get(S.dtype)
        if sd is None:
            raise M.MpbError("distill", -1, f"S is {S.dtype}, not fp16, bf16 or fp32")
        with self._on(stream):
            s = {"stats": torch.empty((T, 4), **f32), "kl": torch.empty(T, **f32), "loss": torch.empty(1, **f32),
                 "dS": self._like_logits(S) if grad else None, "args": (S, sd, ids, teacher, teacher_lse, weight, tau)}
        M.moe_distill_loss(*s["args"], s["stats"], s["kl"], s["loss"], s["dS"], gloss, stream)
        return s

    def distill_grad(self, s, gloss=None, stream=None):
        """The gradient of distill's loss times gloss, as a pass of its own."""
        with self._on(stream):
            dS = self._like_logits(s["args"][0])
        M.moe_distill_loss_grad(*s["args"], s["stats"], dS, gloss, stream)
        return dS
