"""ctypes binding of libmpb (include/mpb.h). Argument marshalling only: every
step of the layer runs in the library's HIP kernels. Functions keep the C
names; tensors are passed as device pointers, streams as raw HIP handles."""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmpb.so")

MPB_F16, MPB_BF16, MPB_F32 = 0, 1, 2
MPB_GATE_NONE, MPB_GATE_TOKEN, MPB_GATE_FULL = 0, 1, 2
MPB_ACT_NONE, MPB_ACT_RELU, MPB_ACT_SILU, MPB_ACT_GELU, MPB_ACT_GELU_TANH = 0, 1, 2, 3, 4
MPB_PAIRS_HALVES, MPB_PAIRS_NEIGHBOURS = 0, 1
ERRORS = {-1: "MPB_E_ARG", -2: "MPB_E_SHAPE", -3: "MPB_E_RANGE", -4: "MPB_E_NOT_RESIDENT",
          -5: "MPB_E_WS", -6: "MPB_E_HIP", -7: "MPB_E_UNINIT", -8: "MPB_E_BUSY"}
MPB_PAGE_GPU, MPB_PAGE_CPU, MPB_PAGE_IN_TRANSFER = 0, 1, 2


class MpbError(RuntimeError):
    def __init__(self, name, code, msg):
        super().__init__(f"{name}: {ERRORS.get(code, code)}: {msg}")
        self.code = code


class LayerDesc(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("I", ctypes.c_int32), ("E", ctypes.c_int32),
                ("S", ctypes.c_int32), ("K", ctypes.c_int32)]


class PlannerParams(ctypes.Structure):
    _fields_ = [("n_buckets", ctypes.c_int32), ("bucket_frac", ctypes.c_double * 8), ("mu", ctypes.c_double * 8),
                ("floor", ctypes.c_int32 * 8), ("n_stages", ctypes.c_int32), ("stage_floor", ctypes.c_int32 * 6),
                ("eps", ctypes.c_double), ("alpha", ctypes.c_double), ("rho_min", ctypes.c_double),
                ("rho_max", ctypes.c_double), ("head_w", ((ctypes.c_double * 3) * 5) * 2),
                ("head_a", (ctypes.c_double * 5) * 2), ("head_c", (ctypes.c_double * 5) * 2),
                ("T_blk", ctypes.c_int64), ("F_blk", ctypes.c_int64), ("P_blk", ctypes.c_int64),
                ("B_kv", ctypes.c_int64)]


class PlanEntry(ctypes.Structure):
    _fields_ = [("i", ctypes.c_int32), ("from_", ctypes.c_int32), ("to", ctypes.c_int32),
                ("delta", ctypes.c_int64), ("damage", ctypes.c_double)]


class PlanSummary(ctypes.Structure):
    _fields_ = [("D", ctypes.c_int64), ("triggered", ctypes.c_int32), ("stage", ctypes.c_int32),
                ("n_plan", ctypes.c_int32), ("pad", ctypes.c_int32), ("released", ctypes.c_int64),
                ("damage", ctypes.c_double), ("stage_released", ctypes.c_int64 * 6),
                ("stage_damage", ctypes.c_double * 6)]


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_F = ctypes.c_float
_L = ctypes.c_int64


def lib() -> ctypes.CDLL:
    """Load libmpb.so; raises if it has not been built (there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m mixed_precision_bit_amd.build` (hipcc, gfx950)")
        L = ctypes.CDLL(LIB_PATH)
        sig = {
            "mpb_init": (_I, [ctypes.POINTER(LayerDesc), _P, _P, _P]),
            "mpb_plane_page_bytes": (ctypes.c_size_t, [_I, _I]),
            "mpb_pack_block": (_I, [_P, _I, _I, _P, _P]),
            "moe_route": (_I, [_P, _I, _P, _P, _I, _I, _I, _I, _P, _P, _P, _SZ, _P]),
            "moe_route_workspace_bytes": (_SZ, [_I, _I]),
            "moe_routing_mass": (_I, [_P, _P, _I, _I, _I, _P, _P]),
            "moe_ffn_workspace_bytes": (ctypes.c_size_t, [_I]),
            "moe_fused_workspace_bytes": (ctypes.c_size_t, [_I]),
            "moe_fused_counter_bytes": (ctypes.c_size_t, []),
            "moe_fused": (_I, [_P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
            "moe_ffn": (_I, [_P, _I, _I, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
            "moe_ffn_static": (_I, [_P, _I, _I, _P, _P, _P, _P, _P, _P, _P]),
            "moe_block_norm": (_I, [_P, _P, _I, _I, _I, _P, _I, _P, _P, _F, _F, _P, _P, _P]),
            "moe_block_norm_grad_workspace_bytes": (_SZ, [_I, _I]),
            "moe_block_norm_grad": (_I, [_P, _P, _I, _I, _I, _P, _I, _P, _P, _F, _F, _P, _P, _P, _P, _P, _P, _P, _P,
                                         _SZ, _P]),
            "moe_router_loss_workspace_bytes": (_SZ, [_I, _I, _I]),
            "moe_router_loss": (_I, [_P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _F, _F, _P, _P, _P, _P, _P, _P, _SZ, _P]),
            "moe_router_loss_grad": (_I, [_P, _I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _F, _P, _P, _P, _P, _P,
                                          _P, _SZ, _P]),
            "moe_adapters_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
            "moe_adapters": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _SZ, _P]),
            "moe_linear_workspace_bytes": (_SZ, [_I, _I, _I]),
            "moe_linear": (_I, [_P, _I, _P, _P, _I, _P, _I, _I, _I, _P, _P, _I, _P, _SZ, _P]),
            "moe_linear_grad_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
            "moe_linear_grad": (_I, [_P, _I, _P, _I, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _SZ, _P]),
            "moe_head_norm": (_I, [_P, _L, _P, _L, _I, _I, _I, _I, _I, _P, _P, _F, _P, _I, _P, _P, _I, _I, _P, _L, _P,
                                   _L, _P]),
            "moe_head_norm_grad_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
            "moe_head_norm_grad": (_I, [_P, _L, _P, _L, _I, _I, _I, _I, _I, _P, _P, _F, _P, _I, _P, _P, _I, _I, _P, _L,
                                        _P, _L, _P, _L, _P, _L, _P, _P, _P, _SZ, _P]),
            "moe_distill_loss": (_I, [_P, _I, _L, _P, _P, _P, _P, _I, _I, _I, _F, _P, _P, _P, _P, _P, _P]),
            "moe_distill_loss_grad": (_I, [_P, _I, _L, _P, _P, _P, _P, _I, _I, _I, _F, _P, _P, _P, _P]),
            "set_committed_bits": (_I, [_I, _I]),
            "mpb_committed_bytes": (ctypes.c_int64, [_P]),
            "mpb_get_committed_bits": (_I, [_I]),
            "mpb_dequant_block": (_I, [_P, _P, _I, _I, _I, _P, _P]),
            "mpb_table_image_bytes": (ctypes.c_int64, [_I, _I, _I]),
            "mpb_pack_table": (_I, [_I, _P, _I, _I, _P, _P]),
            "mpb_dequant_block_image": (_I, [_P, _P, _I, _I, _I, _I, _P, _P]),
            "mpb_set_resident_planes": (_I, [_I, _I]),
            "mpb_get_resident_planes": (_I, [_I]),
            "mpb_offload_pages": (_I, [_I, _I, _P, _P, _P, _P, _P]),
            "mpb_reload_pages": (_I, [_I, _I, _P, _P, _P, _P, _P]),
            "mpb_page_state": (_I, [_I, _I]),
            "mpb_plan_step": (_I, [ctypes.POINTER(LayerDesc), _P, _P, _P, _P, _P, ctypes.POINTER(PlannerParams),
                                   _P, ctypes.POINTER(PlanEntry), ctypes.POINTER(PlanSummary)]),
            "mpb_last_error": (ctypes.c_char_p, []),
            "mpb_set_kernel_events": (_I, [_P, _I]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def _check(name, rc):
    if rc < 0:
        raise MpbError(name, rc, lib().mpb_last_error().decode())
    return rc


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _host_ptrs(ptrs):
    arr = (ctypes.c_void_p * len(ptrs))(*ptrs)
    return arr


def mpb_last_error() -> str:
    return lib().mpb_last_error().decode()


def mpb_init(H, I, E, S, K, q_dev: torch.Tensor, q_init, stream=None):
    import numpy as np
    q_init = np.ascontiguousarray(q_init, dtype=np.int32)
    d = LayerDesc(H, I, E, S, K)
    return _check("mpb_init", lib().mpb_init(ctypes.byref(d), _ptr(q_dev),
                                             q_init.ctypes.data_as(ctypes.c_void_p), _stream(stream)))


def mpb_plane_page_bytes(N, Kd) -> int:
    return lib().mpb_plane_page_bytes(N, Kd)


def mpb_pack_block(canon: torch.Tensor, N, Kd, pages, stream=None):
    arr = _host_ptrs([p.data_ptr() for p in pages])
    return _check("mpb_pack_block", lib().mpb_pack_block(_ptr(canon), N, Kd, arr, _stream(stream)))


def moe_route_workspace_bytes(T, E) -> int:
    return lib().moe_route_workspace_bytes(T, E)


def moe_route(X, x_dtype, W_router, bias, K, topk_idx, topk_w, ws, stream=None):
    T, H = X.shape
    E = W_router.shape[0]
    nbytes = ws.numel() * ws.element_size()
    return _check("moe_route", lib().moe_route(_ptr(X), x_dtype, _ptr(W_router), _ptr(bias), T, H, E, K,
                                               _ptr(topk_idx), _ptr(topk_w), _ptr(ws), nbytes, _stream(stream)))


def moe_routing_mass(topk_idx, topk_w, E, mass, stream=None):
    T, K = topk_idx.shape
    return _check("moe_routing_mass", lib().moe_routing_mass(_ptr(topk_idx), _ptr(topk_w), T, E, K, _ptr(mass),
                                                             _stream(stream)))


def moe_ffn_workspace_bytes(T) -> int:
    return lib().moe_ffn_workspace_bytes(T)


def moe_ffn(X, x_dtype, topk_idx, topk_w, planes_table, luts_table, q, out, ws, stream=None):
    T = X.shape[0]
    nbytes = ws.numel() * ws.element_size()
    return _check("moe_ffn", lib().moe_ffn(_ptr(X), x_dtype, T, _ptr(topk_idx), _ptr(topk_w),
                                           _ptr(planes_table), _ptr(luts_table), _ptr(q), _ptr(out),
                                           _ptr(ws), nbytes, _stream(stream)))


def moe_ffn_static(X, x_dtype, topk_idx, topk_w, planes_table, luts_table, q, out, stream=None):
    T = X.shape[0]
    return _check("moe_ffn_static", lib().moe_ffn_static(_ptr(X), x_dtype, T, _ptr(topk_idx), _ptr(topk_w),
                                                         _ptr(planes_table), _ptr(luts_table), _ptr(q), _ptr(out),
                                                         _stream(stream)))


def moe_fused_counter_bytes() -> int:
    return lib().moe_fused_counter_bytes()


def moe_fused_workspace_bytes(T) -> int:
    return lib().moe_fused_workspace_bytes(T)


def moe_fused(X, x_dtype, W_router, bias, topk_idx, topk_w, planes_table, luts_table, q, out, ws, stream=None):
    T = X.shape[0]
    nbytes = ws.numel() * ws.element_size()
    return _check("moe_fused", lib().moe_fused(_ptr(X), x_dtype, T, _ptr(W_router), _ptr(bias), _ptr(topk_idx),
                                               _ptr(topk_w), _ptr(planes_table), _ptr(luts_table), _ptr(q),
                                               _ptr(out), _ptr(ws), nbytes, _stream(stream)))


_XT = {MPB_F16: torch.float16, MPB_BF16: torch.bfloat16}
_F32, _I32, _U8 = torch.float32, torch.int32, torch.uint8


# the current stream's handle without a Stream object around it, where this torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class _Args:
    """Checks the tensors of one call against the shapes and types the C entry
    takes them for (a C caller answers for these itself) and hands out their
    device pointers. Raw 16-bit tensors (int16) stand for either activation
    type. The call runs with the tensors' device current."""

    def __init__(self, name, *sized):
        """sized: the tensors that the sizes are read from, none of which may be missing."""
        self.name = name
        for t in sized:
            if t is None:
                self.fail("null pointer")
        self.index = sized[0].get_device()  # -1: not on a GPU

    def fail(self, msg, code=-1):
        raise MpbError(self.name, code, msg)

    def __call__(self, what, t, dtype, *shape):
        if t is None:
            return None
        if t.dtype is dtype and t.shape == shape and t.get_device() == self.index and t.is_contiguous():
            return t.data_ptr()
        if t.dtype is not dtype and not (dtype.itemsize == 2 and t.dtype is torch.int16):
            self.fail(f"{what} is {t.dtype}, not {dtype}")
        if t.shape != shape:
            self.fail(f"{what} has shape {tuple(t.shape)}, not {shape}", -2)
        if not t.is_contiguous():
            self.fail(f"{what} is not contiguous")
        if t.get_device() != self.index:
            self.fail(f"{what} is on {t.device}, other tensors on device {self.index}")
        return t.data_ptr()

    def strided(self, what, t, dtype, *shape):
        """(pointer, elements from row to row) of a tensor whose rows are contiguous, whatever lies between them."""
        if t is None:
            return None, 0
        st, row = t.stride(), shape[1] if len(shape) == 2 else shape[1] * shape[2]
        if t.dtype is dtype and t.shape == shape and t.get_device() == self.index and st[-1] == 1 and st[0] >= row and (
                len(shape) == 2 or st[1] == shape[2]) and shape[0] > 1:
            return t.data_ptr(), st[0]
        if t.dtype is not dtype and not (dtype.itemsize == 2 and t.dtype is torch.int16):
            self.fail(f"{what} is {t.dtype}, not {dtype}")
        if t.shape != shape:
            self.fail(f"{what} has shape {tuple(t.shape)}, not {shape}", -2)
        if t.get_device() != self.index:
            self.fail(f"{what} is on {t.device}, other tensors on device {self.index}")
        want = 1
        for d in range(len(shape) - 1, 0, -1):
            if st[d] != want and shape[d] > 1:
                self.fail(f"the rows of {what} are not contiguous")
            want *= shape[d]
        if shape[0] < 2:
            return t.data_ptr(), row
        if st[0] < row:
            self.fail(f"the rows of {what} overlap")
        return t.data_ptr(), st[0]

    def bytes(self, ws):
        """(pointer, bytes) of a workspace."""
        if ws is None:
            return None, 0
        if not ws.is_contiguous() or ws.get_device() != self.index:
            self.fail(f"the workspace is not contiguous on device {self.index}")
        return ws.data_ptr(), ws.numel() * ws.element_size()

    def run(self, fn, stream, *args):
        if self.index < 0:
            self.fail("tensors are on the CPU")
        if stream is not None and stream.device.index != self.index:
            self.fail(f"the stream is on {stream.device}, the tensors on device {self.index}")
        if self.index != torch.cuda.current_device():
            with torch.cuda.device(self.index):
                return self.call(fn, stream, args)
        return self.call(fn, stream, args)

    def call(self, fn, stream, args):
        rc = fn(*args, _raw_stream(self.index) if stream is None else stream.cuda_stream)
        return rc if rc >= 0 else _check(self.name, rc)


def _xtype(name, x_dtype):
    if x_dtype not in _XT:
        raise MpbError(name, -1, f"bad x_dtype {x_dtype!r}")
    return _XT[x_dtype]


def _gate(a, gate, xt, T, H, what="gate"):
    """(pointer, kind) of a gate: None, [T] fp32 or [T][H] activations."""
    if gate is None:
        return None, MPB_GATE_NONE
    if gate.dim() == 1:
        return a(what, gate, _F32, T), MPB_GATE_TOKEN
    return a(what, gate, xt, T, H), MPB_GATE_FULL


def moe_block_norm(o, r, x_dtype, gate, gamma_post, gamma_next, scale, eps, r_out, x_out, stream=None):
    """r_out = r + scale * sigmoid(gate) * norm(o), x_out = norm(r_out); gate: None, [T] fp32 or [T][H]."""
    a = _Args("moe_block_norm", r)
    xt = _xtype(a.name, x_dtype)
    if r.dim() != 2:
        a.fail("r is not [T][H]", -2)
    T, H = r.shape
    gp, kind = _gate(a, gate, xt, T, H)
    return a.run(lib().moe_block_norm, stream, a("o", o, _F32, T, H), a("r", r, xt, T, H), x_dtype, T, H, gp, kind,
                 a("gamma_post", gamma_post, _F32, H), a("gamma_next", gamma_next, _F32, H), scale, eps,
                 a("r_out", r_out, xt, T, H), a("x_out", x_out, xt, T, H))


def moe_block_norm_grad_workspace_bytes(T, H) -> int:
    return lib().moe_block_norm_grad_workspace_bytes(T, H)


def moe_block_norm_grad(o, y, x_dtype, gate, gamma_post, gamma_next, scale, eps, dr_out, dx, dr, d_o, dgate,
                        dgamma_post, dgamma_next, ws, stream=None):
    """Gradients of moe_block_norm from the stream y after the block and the gradients of r_out and x_out."""
    a = _Args("moe_block_norm_grad", dr)
    xt = _xtype(a.name, x_dtype)
    if dr.dim() != 2:
        a.fail("dr is not [T][H]", -2)
    T, H = dr.shape
    gp, kind = _gate(a, gate, xt, T, H)
    dgp, dkind = _gate(a, dgate, xt, T, H, "dgate")
    if dgate is not None and dkind != kind:
        a.fail("dgate and gate have different forms")
    wsp, wsn = a.bytes(ws)
    return a.run(lib().moe_block_norm_grad, stream, a("o", o, _F32, T, H), a("y", y, xt, T, H), x_dtype, T, H, gp, kind,
                 a("gamma_post", gamma_post, _F32, H), a("gamma_next", gamma_next, _F32, H), scale, eps,
                 a("dr_out", dr_out, xt, T, H), a("dx", dx, xt, T, H), a("dr", dr, xt, T, H),
                 a("do", d_o, _F32, T, H), dgp, a("dgamma_post", dgamma_post, _F32, H),
                 a("dgamma_next", dgamma_next, _F32, H), wsp, wsn)


def _router_args(name, X, x_dtype, W_router, topk_idx, mask):
    a = _Args(name, X, W_router, topk_idx)
    xt = _xtype(name, x_dtype)
    if X.dim() != 2 or W_router.dim() != 2 or topk_idx.dim() != 2:
        a.fail("X is [T][H], W_router [E][H], topk_idx [T][K]", -2)
    (T, H), E, K = X.shape, W_router.shape[0], topk_idx.shape[1]
    if mask is not None and mask.dtype is torch.bool:
        mask = mask.view(_U8)
    return a, T, H, E, K, (a("X", X, xt, T, H), x_dtype, a("W_router", W_router, _F32, E, H)), (
        a("topk_idx", topk_idx, _I32, T, K), a("mask", mask, _U8, T))


def moe_router_loss_workspace_bytes(T, H, E) -> int:
    return lib().moe_router_loss_workspace_bytes(T, H, E)


def moe_router_loss(X, x_dtype, W_router, bias, topk_idx, mask, alpha, beta, logits, lse, counts, prob, loss, ws,
                    stream=None):
    """Balance and z loss of a batch with the per-expert counts; mask: None or [T] uint8 or bool, 0 for padding."""
    a, T, H, E, K, head, ids = _router_args("moe_router_loss", X, x_dtype, W_router, topk_idx, mask)
    return a.run(lib().moe_router_loss, stream, *head, a("bias", bias, _F32, E), *ids, T, H, E, K, alpha, beta,
                 a("logits", logits, _F32, T, E), a("lse", lse, _F32, T), a("counts", counts, _I32, E + 1),
                 a("prob", prob, _F32, E), a("loss", loss, _F32, 3), *a.bytes(ws))


def moe_router_loss_grad(X, x_dtype, W_router, topk_idx, mask, logits, lse, counts, alpha, beta, gw, gloss, dX, dW,
                         dbias, ws, stream=None):
    """Gradients of the loss (times the scalar tensor gloss, if given) and of the routing weights (gw)."""
    a, T, H, E, K, head, ids = _router_args("moe_router_loss_grad", X, x_dtype, W_router, topk_idx, mask)
    if gloss is not None and gloss.dim():
        if gloss.numel() != 1:
            a.fail(f"gloss has shape {tuple(gloss.shape)}, not one value", -2)
        gloss = gloss.reshape(())
    return a.run(lib().moe_router_loss_grad, stream, *head, *ids, a("logits", logits, _F32, T, E),
                 a("lse", lse, _F32, T), a("counts", counts, _I32, E + 1), T, H, E, K, alpha, beta,
                 a("gw", gw, _F32, T, K), a("gloss", gloss, _F32), a("dX", dX, _F32, T, H),
                 a("dW", dW, _F32, E, H), a("dbias", dbias, _F32, E), *a.bytes(ws))


def moe_adapters_workspace_bytes(T, Kd, n, R) -> int:
    return lib().moe_adapters_workspace_bytes(T, Kd, n, R)


def moe_adapters(X, x_dtype, A, B, ranks, scales, adapter, base, out, ws, stream=None):
    """out = base + scales[a] * B[a] (A[a] x) with a = adapter[t] per token; A [n][R][Kd], B [n][N][R]."""
    a = _Args("moe_adapters", X, A, B)
    xt = _xtype(a.name, x_dtype)
    if X.dim() != 2 or A.dim() != 3 or B.dim() != 3:
        a.fail("X is [T][Kd], A [n][R][Kd], B [n][N][R]", -2)
    (T, Kd), (n, R, _), N = X.shape, A.shape, B.shape[1]
    return a.run(lib().moe_adapters, stream, a("X", X, xt, T, Kd), x_dtype, T, Kd, a("A", A, xt, n, R, Kd),
                 a("B", B, xt, n, N, R), a("ranks", ranks, _I32, n), a("scales", scales, _F32, n), n, R, N,
                 a("adapter", adapter, _I32, T), a("base", base, _F32, T, N), a("out", out, _F32, T, N), *a.bytes(ws))


def _either(a, what, t, xt, x_dtype):
    """(dtype, its number) of a tensor that has the activations' type or fp32."""
    if t is None:
        a.fail(f"{what} is missing")
    return (_F32, MPB_F32) if t.dtype is _F32 else (xt, x_dtype)


def moe_linear_workspace_bytes(T, Kd, N) -> int:
    return lib().moe_linear_workspace_bytes(T, Kd, N)


def moe_linear(X, x_dtype, W, bias, act, res, z, y, ws, stream=None):
    """z = X W^T + bias, y = res + act(z); y (and res) [T][N] of X's type or fp32, z of X's type or None."""
    a = _Args("moe_linear", X, W, y)
    xt = _xtype(a.name, x_dtype)
    if X.dim() != 2 or W.dim() != 2:
        a.fail("X is [T][Kd], W [N][Kd]", -2)
    (T, Kd), N = X.shape, W.shape[0]
    yt, yd = _either(a, "y", y, xt, x_dtype)
    return a.run(lib().moe_linear, stream, a("X", X, xt, T, Kd), x_dtype, a("W", W, xt, N, Kd), a("bias", bias, _F32, N),
                 act, a("res", res, yt, T, N), T, Kd, N, a("z", z, xt, T, N), a("y", y, yt, T, N), yd, *a.bytes(ws))


def moe_linear_grad_workspace_bytes(T, Kd, N, act, dy_dtype) -> int:
    return lib().moe_linear_grad_workspace_bytes(T, Kd, N, act, dy_dtype)


def moe_linear_grad(X, x_dtype, W, act, z, dy, dX, dW, dbias, ws, stream=None):
    """dX, dW and dbias (each may be None) of moe_linear from z as it wrote it and dy of X's type or fp32."""
    a = _Args("moe_linear_grad", X, W, dy)
    xt = _xtype(a.name, x_dtype)
    if X.dim() != 2 or W.dim() != 2:
        a.fail("X is [T][Kd], W [N][Kd]", -2)
    (T, Kd), N = X.shape, W.shape[0]
    dt, dd = _either(a, "dy", dy, xt, x_dtype)
    return a.run(lib().moe_linear_grad, stream, a("X", X, xt, T, Kd), x_dtype, a("W", W, xt, N, Kd), act,
                 a("z", z, xt, T, N), a("dy", dy, dt, T, N), dd, T, Kd, N, a("dX", dX, xt, T, Kd),
                 a("dW", dW, _F32, N, Kd), a("dbias", dbias, _F32, N), *a.bytes(ws))


def _heads(a, x_dtype, q, k, gamma_q, gamma_k, pos, axis, freq):
    """(shapes of q and k, activation type, the arguments from gamma_q to Dr but eps) of a call on heads."""
    xt = _xtype(a.name, x_dtype)
    if q.dim() != 3 or (k is not None and k.dim() != 3):
        a.fail("q is [T][Hq][D], k [T][Hk][D]", -2)
    T, Hq, D = q.shape
    Hk = 0 if k is None else k.shape[1]
    A = Dr = 0
    if freq is not None:
        if freq.dim() != 1 or pos is None or pos.dim() != 2:
            a.fail("freq is [Dr / 2], pos [A][T]", -2)
        A, Dr = pos.shape[0], 2 * freq.shape[0]
    elif pos is not None or axis is not None:
        a.fail("a rotation needs freq")
    return xt, T, Hq, Hk, D, (a("gamma_q", gamma_q, _F32, D), a("gamma_k", gamma_k, _F32, D)), (
        a("pos", pos, _I32, A, T), A, a("axis", axis, _I32, Dr // 2), a("freq", freq, _F32, Dr // 2), Dr)


def moe_head_norm(q, k, x_dtype, gamma_q, gamma_k, eps, pos, axis, freq, pairs, q_out, k_out, stream=None):
    """Norms and rotation of query and key heads [T][H][D] (views of one packed projection are fine); k may be None."""
    a = _Args("moe_head_norm", q)
    xt, T, Hq, Hk, D, gammas, rot = _heads(a, x_dtype, q, k, gamma_q, gamma_k, pos, axis, freq)
    return a.run(lib().moe_head_norm, stream, *a.strided("q", q, xt, T, Hq, D), *a.strided("k", k, xt, T, Hk, D), x_dtype,
                 T, Hq, Hk, D, *gammas, eps, *rot, pairs, *a.strided("q_out", q_out, xt, T, Hq, D),
                 *a.strided("k_out", k_out, xt, T, Hk, D))


def moe_head_norm_grad_workspace_bytes(T, Hq, Hk, D) -> int:
    return lib().moe_head_norm_grad_workspace_bytes(T, Hq, Hk, D)


def moe_head_norm_grad(q, k, x_dtype, gamma_q, gamma_k, eps, pos, axis, freq, pairs, dq_out, dk_out, dq, dk, dgamma_q,
                       dgamma_k, ws, stream=None):
    """Gradients of moe_head_norm; q (or k) may be None where its side has no gamma."""
    a = _Args("moe_head_norm_grad", dq_out)
    xt, T, Hq, Hk, D, gammas, rot = _heads(a, x_dtype, dq_out, dk_out, gamma_q, gamma_k, pos, axis, freq)
    return a.run(lib().moe_head_norm_grad, stream, *a.strided("q", q, xt, T, Hq, D), *a.strided("k", k, xt, T, Hk, D),
                 x_dtype, T, Hq, Hk, D, *gammas, eps, *rot, pairs, *a.strided("dq_out", dq_out, xt, T, Hq, D),
                 *a.strided("dk_out", dk_out, xt, T, Hk, D), *a.strided("dq", dq, xt, T, Hq, D),
                 *a.strided("dk", dk, xt, T, Hk, D), a("dgamma_q", dgamma_q, _F32, D),
                 a("dgamma_k", dgamma_k, _F32, D), *a.bytes(ws))


_ST = {**_XT, MPB_F32: torch.float32}


def _distill(a, S, s_dtype, ids, teacher, teacher_lse, weight, tau, dS, gloss):
    """(arguments up to tau, T, dS, gloss) of a distillation call."""
    if s_dtype not in _ST:
        a.fail(f"bad s_dtype {s_dtype!r}")
    st = _ST[s_dtype]
    if S.dim() != 2 or ids.dim() != 2:
        a.fail("S is [T][V], ids [T][k]", -2)
    (T, V), k = S.shape, ids.shape[1]
    p, ld = a.strided("S", S, st, T, V)
    d, dld = a.strided("dS", dS, st, T, V)
    if dS is not None and dld != ld:
        a.fail(f"dS has a row stride of {dld}, S of {ld}")
    if gloss is not None and gloss.dim():
        if gloss.numel() != 1:
            a.fail(f"gloss has shape {tuple(gloss.shape)}, not one value", -2)
        gloss = gloss.reshape(())
    return (p, s_dtype, ld, a("ids", ids, _I32, T, k), a("teacher", teacher, _F32, T, k),
            a("teacher_lse", teacher_lse, _F32, T), a("weight", weight, _F32, T), T, V, k, tau), T, d, a("gloss", gloss, _F32)


def moe_distill_loss(S, s_dtype, ids, teacher, teacher_lse, weight, tau, stats, kl, loss, dS, gloss, stream=None):
    """Loss of student logits S [T][V] against a teacher's top logits [T][k]; with dS its gradient in the same launch."""
    a = _Args("moe_distill_loss", S, ids, teacher)
    head, T, d, g = _distill(a, S, s_dtype, ids, teacher, teacher_lse, weight, tau, dS, gloss)
    return a.run(lib().moe_distill_loss, stream, *head, a("stats", stats, _F32, T, 4), a("kl", kl, _F32, T),
                 a("loss", loss, _F32, 1), d, g)


def moe_distill_loss_grad(S, s_dtype, ids, teacher, teacher_lse, weight, tau, stats, dS, gloss, stream=None):
    """The gradient of moe_distill_loss from the stats that it wrote."""
    a = _Args("moe_distill_loss_grad", S, ids, teacher)
    head, T, d, g = _distill(a, S, s_dtype, ids, teacher, teacher_lse, weight, tau, dS, gloss)
    return a.run(lib().moe_distill_loss_grad, stream, *head, a("stats", stats, _F32, T, 4), d, g)


def set_committed_bits(i, b):
    return _check("set_committed_bits", lib().set_committed_bits(i, b))


def mpb_committed_bytes(touched=None) -> int:
    import numpy as np
    if touched is None:
        return _check("mpb_committed_bytes", lib().mpb_committed_bytes(None))
    t = np.ascontiguousarray(touched, dtype=np.uint8)
    return _check("mpb_committed_bytes", lib().mpb_committed_bytes(t.ctypes.data_as(ctypes.c_void_p)))


def mpb_get_committed_bits(i) -> int:
    return _check("mpb_get_committed_bits", lib().mpb_get_committed_bits(i))


def mpb_table_image_bytes(kind, N, b) -> int:
    return _check("mpb_table_image_bytes", lib().mpb_table_image_bytes(kind, N, b))


def mpb_pack_table(kind, lut, N, b, image, stream=None):
    return _check("mpb_pack_table", lib().mpb_pack_table(kind, _ptr(lut), N, b, _ptr(image), _stream(stream)))


def mpb_dequant_block(pages, lut, N, Kd, b, out, stream=None):
    arr = _host_ptrs([p.data_ptr() for p in pages[:b]])
    return _check("mpb_dequant_block", lib().mpb_dequant_block(arr, _ptr(lut), N, Kd, b, _ptr(out),
                                                               _stream(stream)))


def mpb_dequant_block_image(pages, image, kind, N, Kd, b, out, stream=None):
    arr = _host_ptrs([p.data_ptr() for p in pages[:b]])
    return _check("mpb_dequant_block_image", lib().mpb_dequant_block_image(arr, _ptr(image), kind, N, Kd, b,
                                                                           _ptr(out), _stream(stream)))


def mpb_set_kernel_events(events):
    """events: list of 5 raw hipEvent_t handles (ints), or [] to turn recording off."""
    if not events:
        return _check("mpb_set_kernel_events", lib().mpb_set_kernel_events(None, 0))
    return _check("mpb_set_kernel_events", lib().mpb_set_kernel_events(_host_ptrs(events), len(events)))


def mpb_set_resident_planes(i, r):
    return _check("mpb_set_resident_planes", lib().mpb_set_resident_planes(i, r))


def mpb_get_resident_planes(i) -> int:
    return _check("mpb_get_resident_planes", lib().mpb_get_resident_planes(i))


def _ptr_array(ts, n):
    """n pointers (0 where the entry is None or missing) from a list of tensors."""
    ptrs = [0] * n
    for k, t in enumerate(ts):
        if t is not None:
            ptrs[k] = t.data_ptr()
    return _host_ptrs(ptrs)


def mpb_offload_pages(i, r, host_planes, dev_planes, host_tables, dev_tables, copy_stream):
    """planes: lists of 8 tensors (plane pages 0..7), tables: lists of 6
    (table images of bitwidths 3..8); None where a page does not move."""
    return _check("mpb_offload_pages", lib().mpb_offload_pages(
        i, r, _ptr_array(host_planes, 8), _ptr_array(dev_planes, 8), _ptr_array(host_tables, 6),
        _ptr_array(dev_tables, 6), _stream(copy_stream)))


def mpb_reload_pages(i, r, host_planes, dev_planes, host_tables, dev_tables, copy_stream):
    return _check("mpb_reload_pages", lib().mpb_reload_pages(
        i, r, _ptr_array(host_planes, 8), _ptr_array(dev_planes, 8), _ptr_array(host_tables, 6),
        _ptr_array(dev_tables, 6), _stream(copy_stream)))


def mpb_page_state(i, p) -> int:
    return _check("mpb_page_state", lib().mpb_page_state(i, p))


def planner_params(P: dict) -> PlannerParams:
    """Pack a dict of planner parameters (the header's field names) into the C struct."""
    c = PlannerParams()
    c.n_buckets = len(P["bucket_frac"])
    for k in range(c.n_buckets):
        c.bucket_frac[k] = P["bucket_frac"][k]
        c.mu[k] = P["mu"][k]
        c.floor[k] = P["floor"][k]
    c.n_stages = len(P["stage_floor"])
    for k in range(c.n_stages):
        c.stage_floor[k] = P["stage_floor"][k]
    c.eps, c.alpha, c.rho_min, c.rho_max = P["eps"], P["alpha"], P["rho_min"], P["rho_max"]
    for u in range(2):
        for t in range(5):
            for j in range(3):
                c.head_w[u][t][j] = P["head_w"][u][t][j]
            c.head_a[u][t] = P["head_a"][u][t]
            c.head_c[u][t] = P["head_c"][u][t]
    c.T_blk, c.F_blk, c.P_blk, c.B_kv = P["T_blk"], P["F_blk"], P["P_blk"], P["B_kv"]
    return c


def mpb_plan_step(H, I, E, S, K, q, movable, sens, mass, phi, P: dict):
    """Host planner step. q [nb] int, movable [nb] bool or None, sens [nb][6]
    (b = 3..8), mass [E], phi [nb][3]. Returns (plan, summary, queue) with plan
    a list of (i, from, to, delta, damage), summary a dict and queue an
    [n_stages][nb] int32 array."""
    import numpy as np
    nb = 2 * (E + S)
    d = LayerDesc(H, I, E, S, K)
    q = np.ascontiguousarray(q, dtype=np.int32)
    mv = None if movable is None else np.ascontiguousarray(movable, dtype=np.uint8)
    sens = np.ascontiguousarray(sens, dtype=np.float64)
    mass = np.ascontiguousarray(mass, dtype=np.float64)
    phi = np.ascontiguousarray(phi, dtype=np.float64)
    assert q.shape == (nb,) and sens.shape == (nb, 6) and mass.shape == (E,) and phi.shape == (nb, 3)
    prm = planner_params(P)
    queue = np.zeros((prm.n_stages, nb), dtype=np.int32)
    plan = (PlanEntry * nb)()
    summ = PlanSummary()

    def vp(a):
        return None if a is None else a.ctypes.data_as(ctypes.c_void_p)

    _check("mpb_plan_step", lib().mpb_plan_step(ctypes.byref(d), vp(q), vp(mv), vp(sens), vp(mass), vp(phi),
                                                ctypes.byref(prm), vp(queue), plan, ctypes.byref(summ)))
    entries = [(plan[k].i, plan[k].from_, plan[k].to, plan[k].delta, plan[k].damage) for k in range(summ.n_plan)]
    summary = {"D": summ.D, "triggered": bool(summ.triggered), "stage": summ.stage, "released": summ.released,
               "damage": summ.damage, "stage_released": list(summ.stage_released)[:prm.n_stages],
               "stage_damage": list(summ.stage_damage)[:prm.n_stages]}
    return entries, summary, queue
