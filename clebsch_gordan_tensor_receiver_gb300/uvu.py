"""Python binding of libuvu.so (argument marshalling only).

Every function named ``uvu_*`` here calls the C entry point of the same name in
``include/uvu.h`` and raises ``UVUError`` when it returns a status other than UVU_OK.  All
arithmetic runs in the library's CUDA kernels; there is no fallback path: if the library cannot
be loaded, importing this module raises.

``Plan`` is a small convenience wrapper that passes torch tensors' device pointers and the
current CUDA stream; torch is used only for memory and streams.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libuvu.so")

UVU_F32, UVU_F64, UVU_BF16, UVU_F16 = 0, 1, 2, 3
UVU_ACT_NONE, UVU_ACT_SILU = 0, 1
UVU_DX_SENDER, UVU_DX_ATOMIC, UVU_DX_STAGED = 0, 1, 2
UVU_MODULE_CONV, UVU_MODULE_HVP, UVU_MODULE_TP, UVU_MODULE_TP_SHARED = 0, 1, 2, 3
UVU_FWD_AUTO, UVU_FWD_RECEIVER, UVU_FWD_SENDER = 0, 1, 2
STATUS = {0: "UVU_OK", 1: "UVU_ERR_INVALID_ARGUMENT", 2: "UVU_ERR_UNSUPPORTED",
          3: "UVU_ERR_COMPILE", 4: "UVU_ERR_CUDA", 5: "UVU_ERR_OUT_OF_MEMORY"}

# every symbol declared in include/uvu.h
EXPORTS = (
    "uvu_plan_create", "uvu_plan_destroy", "uvu_plan_info", "uvu_plan_cg", "uvu_plan_source",
    "uvu_plan_module_source", "uvu_plan_device_status",
    "uvu_csr_from_sorted_recv", "uvu_csr_transpose_workspace", "uvu_csr_transpose",
    "uvu_csr_transpose_noalloc", "uvu_graph_validate", "uvu_conv_fwd", "uvu_conv_bwd_edge",
    "uvu_conv_bwd_dx", "uvu_conv_bwd_dx_reduce", "uvu_conv_bwd_workspace", "uvu_conv_bwd",
    "uvu_conv_hvp", "uvu_conv_hvp_workspace", "uvu_tp_fwd", "uvu_tp_bwd", "uvu_tp_bwd_workspace",
    "uvu_conv_fwd_model", "uvu_conv_fwd_sender", "uvu_conv_fwd_mode",
    "uvu_mix_fwd", "uvu_mix_bwd", "uvu_mix_workspace", "uvu_conv_uvw_fwd",
    "uvu_radial_hidden", "uvu_conv_fwd_radial", "uvu_radial_module_source",
    "uvu_radial_weights", "uvu_radial_weights_workspace", "uvu_radial_weights_bwd", "uvu_radial_weights_bwd_workspace",
    "uvu_radial_hidden_bwd", "uvu_radial_hidden_bwd_workspace",
    "uvu_group_norm_fwd", "uvu_group_norm_bwd", "uvu_group_norm_workspace", "uvu_dropout_fwd", "uvu_dropout_bwd",
    "uvu_attn_fwd", "uvu_attn_bwd", "uvu_attn_workspace", "uvu_attn_device_status",
    "uvu_embed_fwd", "uvu_embed_bwd", "uvu_embed_workspace",
    "uvu_rms_norm_fwd", "uvu_rms_norm_quant", "uvu_rms_norm_bwd", "uvu_rms_norm_workspace",
    "uvu_orthogonalize", "uvu_orthogonalize_workspace", "uvu_orthogonalize_device_status",
    "uvu_fma_rate_probe", "uvu_status_string", "uvu_last_error_message",
)


class UVUError(RuntimeError):
    def __init__(self, status: int, fn: str, msg: str):
        super().__init__(f"{fn}: {STATUS.get(status, status)}: {msg}")
        self.status = status


class AttnShape(ctypes.Structure):
    """uvu_attn_shape of include/uvu.h."""

    _fields_ = ([("dtype", ctypes.c_int), ("n_graphs", ctypes.c_int32)]
                + [(f, ctypes.c_int64) for f in ("n_q", "n_k", "max_q", "max_k")]
                + [(f, ctypes.c_int32) for f in ("q_heads", "kv_heads", "head_dim", "reserved")]
                + [("scale", ctypes.c_double)]
                + [(f, ctypes.c_int64) for f in ("q_row", "q_head", "k_row", "k_head", "v_row", "v_head", "o_row", "o_head")])


class OrthoShape(ctypes.Structure):
    """uvu_ortho_shape of include/uvu.h."""

    _fields_ = ([("dtype", ctypes.c_int)] + [(f, ctypes.c_int32) for f in ("n_matrices", "rows", "cols", "steps", "reserved")]
                + [(f, ctypes.c_double) for f in ("a", "b", "c", "eps", "scale")]
                + [(f, ctypes.c_int64) for f in ("g_matrix", "g_row", "o_matrix", "o_row")])


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libuvu.so is not built ({LIB_PATH}); run __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    sig = {
        "uvu_plan_create": [ctypes.c_char_p, ctypes.c_char_p, I, I, ctypes.POINTER(P)],
        "uvu_plan_destroy": [P],
        "uvu_plan_info": [P, P, P, P, P, P, P],
        "uvu_plan_cg": [P, I, P],
        "uvu_plan_source": [P, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_char_p)],
        "uvu_plan_module_source": [P, I, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_char_p)],
        "uvu_plan_device_status": [P, ctypes.POINTER(ctypes.c_uint), I],
        "uvu_csr_from_sorted_recv": [I64, I64, P, P, P],
        "uvu_csr_transpose_workspace": [I64, I64, ctypes.POINTER(SZ)],
        "uvu_csr_transpose": [I64, I64, P, P, P, P, P, P, SZ, P],
        "uvu_csr_transpose_noalloc": [I64, I64, P, P, P, P, P, P],
        "uvu_graph_validate": [I64, I64, P, P, P, ctypes.POINTER(I64), P],
        "uvu_conv_fwd": [P, I64, I64, P, P, P, P, P, P, P],
        "uvu_conv_bwd_edge": [P, I64, I64, P, P, P, P, P, P, P, P, P, P, P],
        "uvu_conv_bwd_dx": [P, I64, I64, P, P, P, P, P, P, P, P],
        "uvu_conv_bwd_dx_reduce": [P, I64, I64, P, P, P, P, P],
        "uvu_conv_bwd_workspace": [P, I64, I64, I, ctypes.POINTER(SZ)],
        "uvu_conv_bwd": [P, I64, I64, P, P, P, P, P, P, P, P, P, P, P, P, I, P, SZ, P],
        "uvu_conv_hvp": [P, I64, I64] + [P] * 16 + [SZ, P],
        "uvu_conv_hvp_workspace": [P, I64, I64, ctypes.POINTER(SZ)],
        "uvu_tp_fwd": [P, I64, P, P, P, I, P, P],
        "uvu_tp_bwd": [P, I64, P, P, P, I, P, P, P, P, P, SZ, P],
        "uvu_tp_bwd_workspace": [P, I64, I, ctypes.POINTER(SZ)],
        "uvu_conv_fwd_model": [P, I64, I64, ctypes.POINTER(I), ctypes.POINTER(ctypes.c_double),
                               ctypes.POINTER(ctypes.c_double)],
        "uvu_conv_fwd_sender": [P, I64, I64, P, P, P, P, P, P, P, P],
        "uvu_conv_fwd_mode": [P, I, I64, I64, P, P, P, P, P, P, P, P, P, P],
        "uvu_mix_fwd": [P, I64, I, P, P, P, P, SZ, P],
        "uvu_mix_bwd": [P, I64, I, P, P, P, P, P, P, SZ, P],
        "uvu_mix_workspace": [P, I64, I, ctypes.POINTER(SZ), ctypes.POINTER(SZ)],
        "uvu_conv_uvw_fwd": [P, I64, I64, P, P, P, P, P, P, I, P, P, P, SZ, P],
        "uvu_radial_hidden": [P, I64, P, ctypes.c_double, I, I, ctypes.POINTER(I), P, P, P],
        "uvu_conv_fwd_radial": [P, I64, I64, P, P, P, I, P, P, P, P, P],
        "uvu_radial_module_source": [P, I, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_char_p)],
        "uvu_fma_rate_probe": [I, I, I, P, ctypes.POINTER(ctypes.c_double), P],
        "uvu_radial_weights": [P, I64, P, I, P, P, P, SZ, P],
        "uvu_radial_weights_workspace": [P, I, ctypes.POINTER(SZ)],
        "uvu_radial_weights_bwd": [P, I64, P, I, P, P, P, P, P, SZ, P],
        "uvu_radial_weights_bwd_workspace": [P, I64, I, ctypes.POINTER(SZ)],
        "uvu_radial_hidden_bwd": [P, I64, P, ctypes.c_double, I, I, ctypes.POINTER(I), P, P, P, P, P, SZ, P],
        "uvu_radial_hidden_bwd_workspace": [P, I64, I, ctypes.POINTER(I), ctypes.POINTER(SZ)],
        "uvu_group_norm_fwd": [I, I64, I, I64, I, I, I, ctypes.c_double] + [P] * 8 + [SZ, P],
        "uvu_group_norm_bwd": [I, I64, I, I64, I, I, I] + [P] * 11 + [SZ, P],
        "uvu_group_norm_workspace": [I, I64, I, I64, I, I, ctypes.POINTER(SZ), ctypes.POINTER(SZ)],
        "uvu_dropout_fwd": [I, I64, I, ctypes.c_double, ctypes.c_uint64, ctypes.c_uint64, P, P, P, P],
        "uvu_dropout_bwd": [I, I64, I, ctypes.c_double, ctypes.c_uint64, ctypes.c_uint64, P, P, P],
        "uvu_attn_fwd": [ctypes.POINTER(AttnShape)] + [P] * 9 + [SZ, P],
        "uvu_attn_bwd": [ctypes.POINTER(AttnShape)] + [P] * 13 + [SZ, P],
        "uvu_attn_device_status": [ctypes.POINTER(ctypes.c_uint), I],
        "uvu_attn_workspace": [ctypes.POINTER(AttnShape), ctypes.POINTER(SZ), ctypes.POINTER(SZ)],
        "uvu_embed_fwd": [I, I64, I64, I, I, I, ctypes.c_double] + [P] * 4,
        "uvu_embed_bwd": [I, I64, I64, I, I, I, ctypes.c_double] + [P] * 4 + [SZ, P],
        "uvu_embed_workspace": [I, I64, I64, I, I, ctypes.POINTER(SZ)],
        "uvu_rms_norm_fwd": [I, I64, I, I, ctypes.c_double] + [P] * 7,
        "uvu_rms_norm_quant": [I, I64, I, I, ctypes.c_double, I] + [P] * 7,
        "uvu_rms_norm_bwd": [I, I64, I, I] + [P] * 8 + [SZ, P],
        "uvu_rms_norm_workspace": [I, I64, I, I, ctypes.POINTER(SZ)],
        "uvu_orthogonalize": [ctypes.POINTER(OrthoShape), P, P, P, SZ, P],
        "uvu_orthogonalize_workspace": [ctypes.POINTER(OrthoShape), ctypes.POINTER(SZ)],
        "uvu_orthogonalize_device_status": [ctypes.POINTER(ctypes.c_uint), I],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    lib.uvu_status_string.argtypes = [ctypes.c_int]
    lib.uvu_status_string.restype = ctypes.c_char_p
    lib.uvu_last_error_message.argtypes = []
    lib.uvu_last_error_message.restype = ctypes.c_char_p
    return lib


lib = _load()


def _check(st: int, fn: str):
    if st != 0:
        raise UVUError(st, fn, lib.uvu_last_error_message().decode())


def _wrap(name):
    f = getattr(lib, name)

    def call(*args):
        _check(f(*args), name)

    call.__name__ = name
    call.__doc__ = f"Calls {name} of include/uvu.h; raises UVUError on failure."
    return call


for _n in ("uvu_plan_destroy", "uvu_plan_info", "uvu_plan_cg", "uvu_plan_source", "uvu_plan_module_source",
           "uvu_plan_device_status",
           "uvu_csr_from_sorted_recv", "uvu_csr_transpose_workspace", "uvu_csr_transpose",
           "uvu_csr_transpose_noalloc", "uvu_graph_validate", "uvu_conv_fwd", "uvu_conv_bwd_edge",
           "uvu_conv_bwd_dx", "uvu_conv_bwd_dx_reduce", "uvu_conv_bwd_workspace", "uvu_conv_bwd",
           "uvu_conv_hvp", "uvu_conv_hvp_workspace", "uvu_tp_fwd", "uvu_tp_bwd", "uvu_tp_bwd_workspace",
           "uvu_conv_fwd_model", "uvu_conv_fwd_sender", "uvu_conv_fwd_mode",
           "uvu_mix_fwd", "uvu_mix_bwd", "uvu_mix_workspace", "uvu_conv_uvw_fwd",
           "uvu_radial_hidden", "uvu_conv_fwd_radial", "uvu_radial_module_source", "uvu_fma_rate_probe",
           "uvu_radial_weights", "uvu_radial_weights_workspace", "uvu_radial_weights_bwd",
           "uvu_radial_weights_bwd_workspace", "uvu_radial_hidden_bwd", "uvu_radial_hidden_bwd_workspace",
           "uvu_group_norm_fwd", "uvu_group_norm_bwd", "uvu_group_norm_workspace", "uvu_dropout_fwd", "uvu_dropout_bwd",
           "uvu_attn_fwd", "uvu_attn_bwd", "uvu_attn_workspace", "uvu_attn_device_status",
           "uvu_embed_fwd", "uvu_embed_bwd", "uvu_embed_workspace",
           "uvu_rms_norm_fwd", "uvu_rms_norm_quant", "uvu_rms_norm_bwd", "uvu_rms_norm_workspace",
           "uvu_orthogonalize", "uvu_orthogonalize_workspace", "uvu_orthogonalize_device_status"):
    globals()[_n] = _wrap(_n)


def fma_rate_probe(out, f64: bool, blocks: int, iters: int, stream=None) -> float:
    """Enqueue one launch of the FMA-chain probe into `out` (a device tensor of at least
    blocks * 256 elements of the dtype); returns the FMAs that launch performs."""
    n = ctypes.c_double()
    uvu_fma_rate_probe(UVU_F64 if f64 else UVU_F32, blocks, iters, _ptr(out), ctypes.byref(n), _stream(stream))
    return n.value


def uvu_plan_create(irreps_x: str, irreps_sh: str, lmax_out: int, dtype: int) -> int:
    h = ctypes.c_void_p()
    _check(lib.uvu_plan_create(irreps_x.encode(), irreps_sh.encode(), lmax_out, dtype,
                               ctypes.byref(h)), "uvu_plan_create")
    return h.value


def uvu_status_string(s: int) -> str:
    return lib.uvu_status_string(s).decode()


def uvu_last_error_message() -> str:
    return lib.uvu_last_error_message().decode()


# ----------------------------------------------------------------------- torch convenience

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _workspace(need, device, stream=None):
    """`need` bytes from torch's pool of the stream that the kernels run on.  The wrappers drop the
    reference when they return: a block of another stream's pool could then be handed out again while
    the kernels still use it."""
    import torch
    if stream is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(need, dtype=torch.uint8, device=device)


@dataclass
class PlanInfo:
    mul: int
    dim_x: int
    dim_sh: int
    dim_out: int
    n_paths: int
    paths: list


class Plan:
    """Owns a uvu plan handle; methods take torch tensors already on the current device."""

    def __init__(self, irreps_x: str, irreps_sh: str, lmax_out: int, dtype: str = "float32"):
        self.dtype_name = dtype
        self.handle = uvu_plan_create(irreps_x, irreps_sh, lmax_out,
                                      UVU_F64 if dtype == "float64" else UVU_F32)
        vals = [ctypes.c_int() for _ in range(5)]
        uvu_plan_info(self.handle, *[ctypes.byref(v) for v in vals], None)
        P = vals[4].value
        arr = (ctypes.c_int * (3 * P))()
        uvu_plan_info(self.handle, None, None, None, None, None, arr)
        self.info = PlanInfo(vals[0].value, vals[1].value, vals[2].value, vals[3].value, P,
                             [tuple(arr[3 * i:3 * i + 3]) for i in range(P)])

    def __del__(self):
        h = getattr(self, "handle", None)
        if h:
            lib.uvu_plan_destroy(h)
            self.handle = None

    def cg(self, path: int):
        import numpy as np
        l1, l2, l3 = self.info.paths[path]
        out = np.zeros((2 * l1 + 1, 2 * l2 + 1, 2 * l3 + 1))
        uvu_plan_cg(self.handle, path, out.ctypes.data_as(ctypes.c_void_p))
        return out

    def device_status(self, reset: bool = True) -> int:
        """Status word of the plan's kernels on the current device (0 = no timeout)."""
        w = ctypes.c_uint()
        uvu_plan_device_status(self.handle, ctypes.byref(w), int(reset))
        return w.value

    def source(self):
        s, l = ctypes.c_char_p(), ctypes.c_char_p()
        uvu_plan_source(self.handle, ctypes.byref(s), ctypes.byref(l))
        return s.value.decode(), l.value.decode()

    def module_source(self, module: int):
        """(source, NVRTC log) of one of the plan's modules (UVU_MODULE_*); compiles it on the host
        if needed."""
        s, l = ctypes.c_char_p(), ctypes.c_char_p()
        uvu_plan_module_source(self.handle, module, ctypes.byref(s), ctypes.byref(l))
        return s.value.decode(), l.value.decode()

    def hvp_source(self):
        return self.module_source(UVU_MODULE_HVP)

    def radial_source(self, hidden: int):
        """(source, NVRTC log) of the fused radial forward for `hidden` (fixes the plan's hidden
        width); compiles it on the host if needed."""
        s, l = ctypes.c_char_p(), ctypes.c_char_p()
        uvu_radial_module_source(self.handle, int(hidden), ctypes.byref(s), ctypes.byref(l))
        return s.value.decode(), l.value.decode()

    def radial_hidden(self, r, r_cut, p_env, widths, weights, h, stream=None):
        """Radial network h = silu(... silu(basis(r) W_1) ... W_L) (see uvu_radial_hidden);
        `widths` = [n_basis, H_1, ..., H_L] (host ints), `weights` the layers back to back."""
        wd = (ctypes.c_int * len(widths))(*[int(v) for v in widths])
        uvu_radial_hidden(self.handle, r.numel(), _ptr(r), float(r_cut), int(p_env), len(widths) - 1, wd,
                          _ptr(weights), _ptr(h), _stream(stream))

    def fwd_radial(self, n_nodes, x, Y, h, w_last, recv_offsets, src, out, stream=None):
        """Convolution with fused radial weights w = h W_last (see uvu_conv_fwd_radial)."""
        uvu_conv_fwd_radial(self.handle, n_nodes, src.numel() if src is not None else 0, _ptr(x), _ptr(Y), _ptr(h),
                            int(w_last.shape[0]), _ptr(w_last), _ptr(recv_offsets), _ptr(src), _ptr(out),
                            _stream(stream))

    def radial_weights_workspace(self, hidden) -> int:
        b = ctypes.c_size_t()
        uvu_radial_weights_workspace(self.handle, int(hidden), ctypes.byref(b))
        return b.value

    def radial_weights(self, h, w_last, w, workspace=None, stream=None):
        """Materialised last layer w = h W_last (see uvu_radial_weights)."""
        if workspace is None:
            workspace = _workspace(max(16, self.radial_weights_workspace(h.shape[1])), h.device, stream)
        uvu_radial_weights(self.handle, h.shape[0], _ptr(h), int(h.shape[1]), _ptr(w_last), _ptr(w), _ptr(workspace),
                           workspace.numel(), _stream(stream))

    def radial_weights_bwd_workspace(self, n_edges, hidden) -> int:
        b = ctypes.c_size_t()
        uvu_radial_weights_bwd_workspace(self.handle, n_edges, int(hidden), ctypes.byref(b))
        return b.value

    def radial_weights_bwd(self, h, w_last, dw, dh=None, dw_last=None, workspace=None, stream=None):
        """dh = dw W_last^T and dW_last = h^T dw (see uvu_radial_weights_bwd)."""
        E, H = h.shape
        if workspace is None:
            workspace = _workspace(max(16, self.radial_weights_bwd_workspace(E, H)), h.device, stream)
        uvu_radial_weights_bwd(self.handle, E, _ptr(h), int(H), _ptr(w_last), _ptr(dw), _ptr(dh), _ptr(dw_last),
                               _ptr(workspace), workspace.numel(), _stream(stream))

    def radial_hidden_bwd_workspace(self, n_edges, widths) -> int:
        wd = (ctypes.c_int * len(widths))(*[int(v) for v in widths])
        b = ctypes.c_size_t()
        uvu_radial_hidden_bwd_workspace(self.handle, n_edges, len(widths) - 1, wd, ctypes.byref(b))
        return b.value

    def radial_hidden_bwd(self, r, r_cut, p_env, widths, weights, dh, dr, dweights, workspace=None, stream=None):
        """Edge-length and layer gradients of <dh, h> (see uvu_radial_hidden_bwd)."""
        wd = (ctypes.c_int * len(widths))(*[int(v) for v in widths])
        if workspace is None:
            workspace = _workspace(max(16, self.radial_hidden_bwd_workspace(r.numel(), widths)), r.device, stream)
        uvu_radial_hidden_bwd(self.handle, r.numel(), _ptr(r), float(r_cut), int(p_env), len(widths) - 1, wd,
                              _ptr(weights), _ptr(dh), _ptr(dr), _ptr(dweights), _ptr(workspace), workspace.numel(),
                              _stream(stream))

    def tp_fwd(self, batch, x, y, w, out, w_shared=False, stream=None):
        """Batched tensor product (see uvu_tp_fwd)."""
        uvu_tp_fwd(self.handle, batch, _ptr(x), _ptr(y), _ptr(w), int(bool(w_shared)), _ptr(out),
                   _stream(stream))

    def tp_workspace_bytes(self, batch, w_shared) -> int:
        b = ctypes.c_size_t()
        uvu_tp_bwd_workspace(self.handle, batch, int(bool(w_shared)), ctypes.byref(b))
        return b.value

    def tp_bwd(self, batch, x, y, w, d_out, dx=None, dy=None, dw=None, w_shared=False,
               workspace=None, stream=None):
        """VJP of the batched tensor product (see uvu_tp_bwd); a shared dw needs `workspace`
        (a uint8 device tensor of tp_workspace_bytes() bytes), allocated here with torch if None."""
        ws_ptr, ws_bytes = None, 0
        need = self.tp_workspace_bytes(batch, w_shared) if dw is not None else 0
        if need:
            if workspace is None:
                workspace = _workspace(need, d_out.device, stream)
            ws_ptr, ws_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
        uvu_tp_bwd(self.handle, batch, _ptr(x), _ptr(y), _ptr(w), int(bool(w_shared)), _ptr(d_out),
                   _ptr(dx), _ptr(dy), _ptr(dw), ws_ptr, ws_bytes, _stream(stream))

    def fwd(self, n_nodes, x, Y, w, recv_offsets, src, out, stream=None):
        uvu_conv_fwd(self.handle, n_nodes, src.numel() if src is not None else 0, _ptr(x), _ptr(Y),
                     _ptr(w), _ptr(recv_offsets), _ptr(src), _ptr(out), _stream(stream))

    def fwd_model(self, n_nodes, n_edges):
        """(chosen UVU_FWD_* mode, bytes of the receiver forward, bytes of the sender forward)."""
        c, br, bs = ctypes.c_int(), ctypes.c_double(), ctypes.c_double()
        uvu_conv_fwd_model(self.handle, n_nodes, n_edges, ctypes.byref(c), ctypes.byref(br), ctypes.byref(bs))
        return c.value, br.value, bs.value

    def fwd_sender(self, n_nodes, n_edges, x, Y, w, send_offsets, send_eids, send_recv, out, stream=None):
        uvu_conv_fwd_sender(self.handle, n_nodes, n_edges, _ptr(x), _ptr(Y), _ptr(w), _ptr(send_offsets),
                            _ptr(send_eids), _ptr(send_recv), _ptr(out), _stream(stream))

    def fwd_mode(self, mode, n_nodes, n_edges, x, Y, w, graph, out, stream=None):
        """Forward by mode (UVU_FWD_*) over a Graph holding both CSRs."""
        uvu_conv_fwd_mode(self.handle, mode, n_nodes, n_edges, _ptr(x), _ptr(Y), _ptr(w),
                          _ptr(graph.recv_offsets), _ptr(graph.src), _ptr(graph.send_offsets),
                          _ptr(graph.send_eids), _ptr(graph.send_recv), _ptr(out), _stream(stream))

    def mix_workspace_bytes(self, n_nodes, w_out):
        """(forward bytes, backward bytes) of device workspace for the channel mixing."""
        f, b = ctypes.c_size_t(), ctypes.c_size_t()
        uvu_mix_workspace(self.handle, n_nodes, w_out, ctypes.byref(f), ctypes.byref(b))
        return f.value, b.value

    def _mix_ws(self, n_nodes, w_out, bwd, workspace, device, stream):
        """(pointer, bytes, the tensor, which the caller holds until its launches are done)."""
        need = self.mix_workspace_bytes(n_nodes, w_out)[1 if bwd else 0]
        if workspace is None:
            workspace = _workspace(max(need, 16), device, stream)
        return _ptr(workspace), workspace.numel() * workspace.element_size(), workspace

    def mix_fwd(self, n_nodes, w_out, inp, M, out, workspace=None, stream=None):
        """Per-path channel mixing of a UVU output (see uvu_mix_fwd); `workspace` (uint8) is
        allocated here with torch if None."""
        ws, nb, held = self._mix_ws(n_nodes, w_out, False, workspace, out.device, stream)
        uvu_mix_fwd(self.handle, n_nodes, w_out, _ptr(inp), _ptr(M), _ptr(out), ws, nb, _stream(stream))

    def mix_bwd(self, n_nodes, w_out, inp, M, d_out, d_in=None, dM=None, workspace=None, stream=None):
        """VJP of mix_fwd (see uvu_mix_bwd)."""
        ws, nb, held = self._mix_ws(n_nodes, w_out, True, workspace, d_out.device, stream)
        uvu_mix_bwd(self.handle, n_nodes, w_out, _ptr(inp), _ptr(M), _ptr(d_out), _ptr(d_in), _ptr(dM),
                    ws, nb, _stream(stream))

    def uvw_fwd(self, n_nodes, x, Y, w, recv_offsets, src, M, w_out, uvu_out, out, workspace=None, stream=None):
        """Factorised UVW convolution (see uvu_conv_uvw_fwd)."""
        ws, nb, held = self._mix_ws(n_nodes, w_out, False, workspace, out.device, stream)
        uvu_conv_uvw_fwd(self.handle, n_nodes, src.numel(), _ptr(x), _ptr(Y), _ptr(w), _ptr(recv_offsets),
                         _ptr(src), _ptr(M), w_out, _ptr(uvu_out), _ptr(out), ws, nb, _stream(stream))

    def bwd_edge(self, n_nodes, x, Y, w, recv_offsets, src, d_out, dY=None, dw=None,
                 dx_atomic=None, dx_edge=None, stream=None):
        uvu_conv_bwd_edge(self.handle, n_nodes, src.numel(), _ptr(x), _ptr(Y), _ptr(w),
                          _ptr(recv_offsets), _ptr(src), _ptr(d_out), _ptr(dY), _ptr(dw),
                          _ptr(dx_atomic), _ptr(dx_edge), _stream(stream))

    def bwd_dx(self, n_nodes, n_edges, Y, w, send_offsets, send_eids, send_recv, d_out, dx,
               stream=None):
        uvu_conv_bwd_dx(self.handle, n_nodes, n_edges, _ptr(Y), _ptr(w), _ptr(send_offsets),
                        _ptr(send_eids), _ptr(send_recv), _ptr(d_out), _ptr(dx), _stream(stream))

    def bwd_dx_reduce(self, n_nodes, n_edges, send_offsets, send_eids, dx_edge, dx, stream=None):
        uvu_conv_bwd_dx_reduce(self.handle, n_nodes, n_edges, _ptr(send_offsets), _ptr(send_eids),
                               _ptr(dx_edge), _ptr(dx), _stream(stream))

    def workspace_bytes(self, n_nodes, n_edges, dx_mode) -> int:
        b = ctypes.c_size_t()
        uvu_conv_bwd_workspace(self.handle, n_nodes, n_edges, dx_mode, ctypes.byref(b))
        return b.value

    def bwd(self, n_nodes, x, Y, w, recv_offsets, src, send_offsets, send_eids, send_recv,
            d_out, dx=None, dY=None, dw=None, dx_mode=UVU_DX_SENDER, workspace=None,
            stream=None):
        """Full VJP.  UVU_DX_STAGED needs `workspace` (a uint8 device tensor of at least
        workspace_bytes() bytes); pass None to let this wrapper allocate it with torch."""
        n_edges = src.numel()
        ws_ptr, ws_bytes = None, 0
        if dx_mode == UVU_DX_STAGED and dx is not None:
            need = self.workspace_bytes(n_nodes, n_edges, dx_mode)
            if workspace is None:
                workspace = _workspace(max(need, 16), src.device, stream)
            ws_ptr, ws_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
        uvu_conv_bwd(self.handle, n_nodes, n_edges, _ptr(x), _ptr(Y), _ptr(w),
                     _ptr(recv_offsets), _ptr(src), _ptr(send_offsets), _ptr(send_eids),
                     _ptr(send_recv), _ptr(d_out), _ptr(dx), _ptr(dY), _ptr(dw), dx_mode,
                     ws_ptr, ws_bytes, _stream(stream))


def _hvp_method(self, n_nodes, x, Y, w, recv_offsets, src, send_offsets, send_eids, d_out,
                ax=None, aY=None, aw=None, grad_d_out=None, grad_x=None, grad_Y=None, grad_w=None,
                workspace=None, stream=None):
    """Double backward: gradients of <ax,dx> + <aY,dY> + <aw,dw> (see uvu_conv_hvp)."""
    n_edges = src.numel()
    ws_ptr, ws_bytes = None, 0
    if grad_x is not None:
        b = ctypes.c_size_t()
        uvu_conv_hvp_workspace(self.handle, n_nodes, n_edges, ctypes.byref(b))
        if b.value:
            if workspace is None:
                workspace = _workspace(b.value, src.device, stream)
            ws_ptr, ws_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    uvu_conv_hvp(self.handle, n_nodes, n_edges, _ptr(x), _ptr(Y), _ptr(w), _ptr(recv_offsets),
                 _ptr(src), _ptr(send_offsets), _ptr(send_eids), _ptr(d_out), _ptr(ax), _ptr(aY),
                 _ptr(aw), _ptr(grad_d_out), _ptr(grad_x), _ptr(grad_Y), _ptr(grad_w), ws_ptr,
                 ws_bytes, _stream(stream))


Plan.hvp = _hvp_method


class Graph:
    """Receiver CSR and transposed CSR built on the device by the library's kernels."""

    def __init__(self, n_nodes: int, recv, src, stream=None):
        import torch
        dev = src.device
        self.n_nodes = n_nodes
        self.n_edges = src.numel()
        self.src = src
        self.recv_offsets = torch.empty(n_nodes + 1, dtype=torch.int32, device=dev)
        uvu_csr_from_sorted_recv(n_nodes, self.n_edges, _ptr(recv), _ptr(self.recv_offsets),
                                 _stream(stream))
        nb = ctypes.c_size_t()
        uvu_csr_transpose_workspace(n_nodes, self.n_edges, ctypes.byref(nb))
        ws = _workspace(max(nb.value, 16), dev, stream)
        self.send_offsets = torch.empty(n_nodes + 1, dtype=torch.int32, device=dev)
        self.send_eids = torch.empty(max(self.n_edges, 1), dtype=torch.int32, device=dev)
        self.send_recv = torch.empty(max(self.n_edges, 1), dtype=torch.int32, device=dev)
        uvu_csr_transpose(n_nodes, self.n_edges, _ptr(self.recv_offsets), _ptr(src),
                          _ptr(self.send_offsets), _ptr(self.send_eids), _ptr(self.send_recv),
                          _ptr(ws), nb.value, _stream(stream))
        self._ws = ws


# ------------------------------------------------------------------- node-update operators
#
# The smallest of these kernels run for 3 us, so the wrappers check what the C ABI cannot see from a
# pointer (type, device, shape, strides) and little else: a call costs the host 6 to 9 us.

_CODES = {}  # torch dtype -> uvu_dtype


def _block_dtype(t) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        import torch
        _CODES.update({torch.float32: UVU_F32, torch.bfloat16: UVU_BF16, torch.float16: UVU_F16, torch.float64: UVU_F64})
        code = _CODES.get(t.dtype)
        if code is None:
            raise TypeError(f"the node-update operators take float32, bfloat16 and float16 tensors, not {t.dtype}")
    return code


def _device(t) -> int:
    """The device number of a CUDA tensor on the current device, where the kernels are launched."""
    d = t.get_device()
    if d < 0:
        raise TypeError("the node-update operators take CUDA tensors")
    import torch
    if d != torch.cuda.current_device():
        raise ValueError(f"tensors are on device {d}, but the current device is {torch.cuda.current_device()}")
    return d


def _like(name, t, x):
    """t has x's type, device and shape and is contiguous."""
    if t.dtype != x.dtype or t.get_device() != x.get_device():
        raise TypeError(f"{name} must have the type and device of its operands")
    if t.shape != x.shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {tuple(x.shape)}, not {tuple(t.shape)}")


def _f32(name, t, shape, device):
    if _CODES.get(t.dtype) != UVU_F32 or t.get_device() != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {tuple(shape)} on the operands' device")


def _offsets(name, t, device):
    """Number of graphs of an offsets tensor."""
    import torch
    if t.dtype != torch.int32 or t.get_device() != device or t.dim() != 1 or t.numel() < 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor [n_graphs + 1] on the operands' device")
    return t.numel() - 1


def _at(t):
    return None if t is None else t.data_ptr()


def _raw_stream(stream, device):
    if stream is not None:
        return stream.cuda_stream
    import torch
    return torch._C._cuda_getCurrentRawStream(device)


def _scratch(need, workspace, device, stream=None):
    """(pointer, bytes, the tensor) of a workspace: the caller's, or one from torch."""
    if workspace is not None and (workspace.get_device() != device or not workspace.is_contiguous()):
        raise ValueError("workspace must be contiguous and on the operands' device")
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = _workspace(need, device, stream)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def group_norm_workspace_bytes(x, n_graphs, groups, max_rows=None):
    """(forward bytes, backward bytes) of device workspace for the group norm of x [N][C]."""
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    n, c = x.shape
    uvu_group_norm_workspace(_block_dtype(x), n, n_graphs, n if max_rows is None else max_rows, c, groups, ctypes.byref(f),
                             ctypes.byref(b))
    return f.value, b.value


def _norm_checks(x, gamma, beta, offsets, groups, mean, rstd):
    code, dev = _block_dtype(x), _device(x)
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be contiguous [rows][channels]")
    n, c = x.shape
    b = _offsets("offsets", offsets, dev)
    _f32("gamma", gamma, (c,), dev)
    _f32("beta", beta, (c,), dev)
    _f32("mean", mean, (b, groups), dev)
    _f32("rstd", rstd, (b, groups), dev)
    return code, dev, n, c, b


def group_norm_fwd(x, gamma, beta, offsets, groups, y, mean, rstd, act=UVU_ACT_SILU, eps=1e-5, max_rows=None,
                   workspace=None, stream=None):
    """Group norm with an activation over a packed batch (see uvu_group_norm_fwd): x, y [N][C], offsets
    [B+1] int32, mean and rstd [B][groups] fp32 (outputs); `workspace` (uint8) is allocated here with
    torch if None."""
    code, dev, n, c, b = _norm_checks(x, gamma, beta, offsets, groups, mean, rstd)
    _like("y", y, x)
    most = n if max_rows is None else max_rows
    need = group_norm_workspace_bytes(x, b, groups, most)[0] if workspace is None else 0
    ws, size, held = _scratch(need, workspace, dev, stream)
    uvu_group_norm_fwd(code, n, b, most, c, groups, act, eps, offsets.data_ptr(), x.data_ptr(), gamma.data_ptr(),
                       beta.data_ptr(), y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), ws, size, _raw_stream(stream, dev))


def group_norm_bwd(dy, x, gamma, beta, offsets, groups, mean, rstd, dx, dgamma, dbeta, act=UVU_ACT_SILU, max_rows=None,
                   workspace=None, stream=None):
    """VJP of group_norm_fwd (see uvu_group_norm_bwd)."""
    code, dev, n, c, b = _norm_checks(x, gamma, beta, offsets, groups, mean, rstd)
    _like("dy", dy, x)
    _like("dx", dx, x)
    _f32("dgamma", dgamma, (c,), dev)
    _f32("dbeta", dbeta, (c,), dev)
    most = n if max_rows is None else max_rows
    need = group_norm_workspace_bytes(x, b, groups, most)[1] if workspace is None else 0
    ws, size, held = _scratch(need, workspace, dev, stream)
    uvu_group_norm_bwd(code, n, b, most, c, groups, act, offsets.data_ptr(), x.data_ptr(), gamma.data_ptr(), beta.data_ptr(),
                       mean.data_ptr(), rstd.data_ptr(), dy.data_ptr(), dx.data_ptr(), dgamma.data_ptr(), dbeta.data_ptr(),
                       ws, size, _raw_stream(stream, dev))


def _draws(x, inner):
    n = x.numel()
    if inner < 1 or inner >= 2 ** 31 or n % inner:  # the C entry takes an int
        raise ValueError("the tensor's size must be a multiple of inner, which is in [1, 2^31)")
    return n // inner


def dropout_fwd(x, p, seed, y, offset=0, inner=1, residual=None, stream=None):
    """y = residual + dropout(x) with the mask of (seed, offset); `inner` consecutive values share a draw
    (see uvu_dropout_fwd).  All tensors contiguous and of one shape; y may be x or residual."""
    code, dev = _block_dtype(x), _device(x)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    _like("y", y, x)
    if residual is not None:
        _like("residual", residual, x)
    uvu_dropout_fwd(code, _draws(x, inner), inner, p, seed, offset, x.data_ptr(), _at(residual), y.data_ptr(),
                    _raw_stream(stream, dev))


def dropout_bwd(dy, p, seed, dx, offset=0, inner=1, stream=None):
    """VJP of dropout_fwd with respect to x; the residual's gradient is dy (see uvu_dropout_bwd)."""
    code, dev = _block_dtype(dy), _device(dy)
    if not dy.is_contiguous():
        raise ValueError("dy must be contiguous")
    _like("dx", dx, dy)
    uvu_dropout_bwd(code, _draws(dy, inner), inner, p, seed, offset, dy.data_ptr(), dx.data_ptr(),
                    _raw_stream(stream, dev))


class Attention:
    """Attention of the rows of each graph of a packed batch to that graph's states (see uvu_attn_fwd):
    q, out [Tq][q_heads][head_dim], k, v [Tk][kv_heads][head_dim] (any row and head strides, values of a
    head consecutive), q_offsets and k_offsets [B+1] int32.  max_q, max_k: lengths that no graph exceeds
    (default: all rows).  scale defaults to head_dim ** -0.5."""

    def __init__(self, q_heads, kv_heads, head_dim, q_offsets, k_offsets, max_q=None, max_k=None, scale=None):
        self.device = _device(q_offsets)
        self.n_graphs = _offsets("q_offsets", q_offsets, self.device)
        if _offsets("k_offsets", k_offsets, self.device) != self.n_graphs:
            raise ValueError("q_offsets and k_offsets must have the same number of graphs")
        self.q_offsets, self.k_offsets = q_offsets, k_offsets
        self.q_heads, self.kv_heads, self.head_dim = int(q_heads), int(kv_heads), int(head_dim)
        self.max_q, self.max_k = max_q, max_k
        self.scale = float(head_dim) ** -0.5 if scale is None else float(scale)

    def _operand(self, name, t, heads, rows, dtype):
        """Strides of [rows][heads][head_dim] with consecutive values in a head; 0 for an axis of one, whose
        stride torch leaves arbitrary."""
        if t.dtype != dtype or t.get_device() != self.device:
            raise TypeError(f"{name} must have q's type and be on the offsets' device")
        if t.shape != (rows, heads, self.head_dim):
            raise ValueError(f"{name} must be [{rows}][{heads}][{self.head_dim}], not {tuple(t.shape)}")
        r, h, d = t.stride()
        if d != 1 and self.head_dim > 1:
            raise ValueError(f"{name} must have consecutive values in a head")
        return r if rows > 1 else 0, h if heads > 1 else 0

    def _shape(self, q, k, v, out):
        _device(self.q_offsets)
        nq, nk, dt = q.shape[0], k.shape[0], q.dtype
        code = _block_dtype(q)
        qr, qh = self._operand("q", q, self.q_heads, nq, dt)
        kr, kh = self._operand("k", k, self.kv_heads, nk, dt)
        vr, vh = self._operand("v", v, self.kv_heads, nk, dt)
        orow, oh = self._operand("out", out, self.q_heads, nq, dt)
        return AttnShape(code, self.n_graphs, nq, nk, nq if self.max_q is None else self.max_q,
                         nk if self.max_k is None else self.max_k, self.q_heads, self.kv_heads, self.head_dim, 0, self.scale,
                         qr, qh, kr, kh, vr, vh, orow, oh)

    def _need(self, shape, which):
        b = (ctypes.c_size_t(), ctypes.c_size_t())
        uvu_attn_workspace(ctypes.byref(shape), ctypes.byref(b[0]), ctypes.byref(b[1]))
        return b[which].value

    def workspace_bytes(self, q, k):
        """(forward bytes, backward bytes) of device workspace for operands of q's and k's sizes."""
        s = self._shape(q, k, k, q)
        return self._need(s, 0), self._need(s, 1)

    @staticmethod
    def device_status(reset: bool = True) -> int:
        """Status word of the attention kernels on the current device (0 = no timeout)."""
        w = ctypes.c_uint()
        uvu_attn_device_status(ctypes.byref(w), int(reset))
        return w.value

    def _keep(self, keep, nk):
        if keep is None:
            return None
        if keep.element_size() != 1 or keep.dtype.is_floating_point or keep.shape != (nk,) or keep.get_device() != self.device \
                or not keep.is_contiguous():
            raise ValueError("keep must be a contiguous uint8 or bool tensor [states] on the operands' device")
        return keep.data_ptr()

    def fwd(self, q, k, v, out, lse, keep=None, workspace=None, stream=None):
        """out and lse [Tq][q_heads] (fp32); `keep` [Tk] (uint8 or bool): states with 0 take no part;
        `workspace` (uint8) is allocated here with torch if None."""
        s = self._shape(q, k, v, out)
        _block_dtype(lse)
        _f32("lse", lse, (s.n_q, self.q_heads), self.device)
        ws, size, held = _scratch(self._need(s, 0) if workspace is None else 0, workspace, self.device, stream)
        uvu_attn_fwd(ctypes.byref(s), self.q_offsets.data_ptr(), self.k_offsets.data_ptr(), self._keep(keep, s.n_k), q.data_ptr(),
                     k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), ws, size, _raw_stream(stream, self.device))

    def bwd(self, q, k, v, out, lse, d_out, dq=None, dk=None, dv=None, keep=None, workspace=None, stream=None):
        """VJP (see uvu_attn_bwd): dq, dk, dv contiguous; dq, or dk and dv, may be None."""
        s = self._shape(q, k, v, out)
        _block_dtype(lse)
        _f32("lse", lse, (s.n_q, self.q_heads), self.device)
        if self._operand("d_out", d_out, self.q_heads, s.n_q, q.dtype) != (s.o_row, s.o_head):
            raise ValueError("d_out must have the strides of out")
        for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
            if t is not None:
                _like(name, t, like)
        ws, size, held = _scratch(self._need(s, 1) if workspace is None else 0, workspace, self.device, stream)
        uvu_attn_bwd(ctypes.byref(s), self.q_offsets.data_ptr(), self.k_offsets.data_ptr(), self._keep(keep, s.n_k), q.data_ptr(),
                     k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), d_out.data_ptr(), _at(dq), _at(dk), _at(dv), ws,
                     size, _raw_stream(stream, self.device))


# ------------------------------------------------- embedding, RMS norm, weight updates

def _components(name, t):
    """(rows, channels, inner) of a contiguous [rows][channels] or [rows][channels][inner] tensor."""
    if t.dim() not in (2, 3) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous [rows][channels] or [rows][channels][inner]")
    s = t.shape
    return (s[0], s[1], 1) if len(s) == 2 else tuple(s)


def _embed_checks(index, features, table, names):
    code, dev = _block_dtype(table), _device(table)
    n, c, inner = _components(names[0], features)
    if features.dtype != table.dtype or features.get_device() != dev:
        raise TypeError(f"{names[0]} must have the type and device of {names[1]}")
    if table.dim() != 2 or table.shape[1] != c or not table.is_contiguous():
        raise ValueError(f"{names[1]} must be contiguous [rows][{c}]")
    import torch
    if index.dtype != torch.int32 or index.get_device() != dev or index.shape != (n,) or not index.is_contiguous():
        raise ValueError(f"index must be a contiguous int32 tensor [{n}] on the operands' device")
    return code, dev, n, table.shape[0], c, inner


def embed_fwd(index, table, out, scale=1.0, column=0, stream=None):
    """out[t] = scale * table[index[t]] (see uvu_embed_fwd): index [T] int32, table [rows][C], out [T][C], or
    [T][C][inner] with the values in `column` and zeros beside it.  An index outside the table gives zeros."""
    code, dev, n, rows, c, inner = _embed_checks(index, out, table, ("out", "table"))
    uvu_embed_fwd(code, n, rows, c, inner, column, scale, index.data_ptr(), table.data_ptr(), out.data_ptr(), _raw_stream(stream, dev))


def embed_workspace_bytes(dout, dtable) -> int:
    """Bytes of device workspace for embed_bwd of these gradients' sizes."""
    n, c, inner = _components("dout", dout)
    b = ctypes.c_size_t()
    uvu_embed_workspace(_block_dtype(dtable), n, dtable.shape[0], c, inner, ctypes.byref(b))
    return b.value


def embed_bwd(index, dout, dtable, scale=1.0, column=0, workspace=None, stream=None):
    """dtable[r] = scale * sum of dout[t] (its `column`) over the tokens of row r (see uvu_embed_bwd); `workspace`
    (uint8) is allocated here with torch if None."""
    code, dev, n, rows, c, inner = _embed_checks(index, dout, dtable, ("dout", "dtable"))
    need = embed_workspace_bytes(dout, dtable) if workspace is None else 0
    ws, size, held = _scratch(need, workspace, dev, stream)
    uvu_embed_bwd(code, n, rows, c, inner, column, scale, index.data_ptr(), dout.data_ptr(), dtable.data_ptr(), ws, size,
                  _raw_stream(stream, dev))


def _rms_checks(x, gamma, residual, h):
    code, dev = _block_dtype(x), _device(x)
    n, c, inner = _components("x", x)
    _f32("gamma", gamma, (c,), dev)
    if (residual is None) != (h is None):
        raise ValueError("residual and h go together: both or neither")
    if residual is not None:
        _like("residual", residual, x)
        _like("h", h, x)
    return code, dev, n, c, inner


def rms_norm_fwd(x, gamma, y, rstd=None, residual=None, h=None, eps=1e-5, stream=None):
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * gamma over the rows of x [N][C] or [N][C][inner] (see
    uvu_rms_norm_fwd); gamma [C] and rstd [N] fp32.  residual and h may be None."""
    code, dev, n, c, inner = _rms_checks(x, gamma, residual, h)
    _like("y", y, x)
    if rstd is not None:
        _f32("rstd", rstd, (n,), dev)
    uvu_rms_norm_fwd(code, n, c, inner, eps, x.data_ptr(), _at(residual), gamma.data_ptr(), _at(h), y.data_ptr(), _at(rstd),
                     _raw_stream(stream, dev))


def rms_norm_quant(x, gamma, q, scales, group=128, residual=None, h=None, eps=1e-5, stream=None):
    """rms_norm_fwd with y in 8 bits (see uvu_rms_norm_quant): q like x in float8_e4m3fn (or uint8), scales [N][groups] fp32, one
    for `group` consecutive values of a row (0: the whole row)."""
    code, dev, n, c, inner = _rms_checks(x, gamma, residual, h)
    if q.element_size() != 1 or q.get_device() != dev or q.shape != x.shape or not q.is_contiguous():
        raise ValueError(f"q must be a contiguous 8-bit tensor of shape {tuple(x.shape)} on x's device")
    if group < 0 or group >= 2 ** 31:
        raise ValueError("group must be in [0, 2^31)")
    _f32("scales", scales, (n, -(-c * inner // group) if group else 1), dev)
    uvu_rms_norm_quant(code, n, c, inner, eps, group, x.data_ptr(), _at(residual), gamma.data_ptr(), _at(h), q.data_ptr(),
                       scales.data_ptr(), _raw_stream(stream, dev))


def rms_norm_workspace_bytes(h) -> int:
    """Bytes of device workspace for rms_norm_bwd of h's size."""
    b = ctypes.c_size_t()
    uvu_rms_norm_workspace(_block_dtype(h), *_components("h", h), ctypes.byref(b))
    return b.value


def rms_norm_bwd(dy, h, gamma, rstd, dx, dgamma, dh=None, workspace=None, stream=None):
    """VJP of rms_norm_fwd for the cotangents dy of y and dh of h (see uvu_rms_norm_bwd); dx is the gradient of x and of the
    residual; `workspace` (uint8) is allocated here with torch if None."""
    code, dev, n, c, inner = _rms_checks(h, gamma, None, None)
    _like("dy", dy, h)
    _like("dx", dx, h)
    if dh is not None:
        _like("dh", dh, h)
    _f32("rstd", rstd, (n,), dev)
    _f32("dgamma", dgamma, (c,), dev)
    need = rms_norm_workspace_bytes(h) if workspace is None else 0
    ws, size, held = _scratch(need, workspace, dev, stream)
    uvu_rms_norm_bwd(code, n, c, inner, dy.data_ptr(), h.data_ptr(), gamma.data_ptr(), rstd.data_ptr(), _at(dh), dx.data_ptr(),
                     dgamma.data_ptr(), ws, size, _raw_stream(stream, dev))


MUON = (3.4445, -4.7750, 2.0315)


def _matrices(name, t):
    """(matrices, rows, cols, matrix stride, row stride) of [rows][cols] or [matrices][rows][cols] with consecutive values in a row."""
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must be [rows][cols] or [matrices][rows][cols]")
    (b, m, n), (sb, sm, sn) = ((1, *t.shape), (0, *t.stride())) if t.dim() == 2 else (tuple(t.shape), t.stride())
    if sn != 1 and n > 1:
        raise ValueError(f"{name} must have consecutive values in a row")
    return b, m, n, sb if b > 1 else 0, sm if m > 1 else n


def _ortho_shape(g, out, steps, coefficients, eps, scale):
    code, dev = _block_dtype(g), _device(g)
    if out.dtype != g.dtype or out.get_device() != dev or out.shape != g.shape:
        raise TypeError("out must have g's type, device and shape")
    b, m, n, gm, gr = _matrices("g", g)
    om, orow = _matrices("out", out)[3:]
    return dev, OrthoShape(code, b, m, n, steps, 0, *coefficients, eps, scale, gm, gr, om, orow)


def orthogonalize_workspace_bytes(g) -> int:
    """Bytes of device workspace for orthogonalize of g's type and size."""
    b, m, n = _matrices("g", g)[:3]
    size = ctypes.c_size_t()
    shape = OrthoShape(_block_dtype(g), b, m, n, 5, 0, *MUON, 0.0, 1.0, m * n, n, m * n, n)
    uvu_orthogonalize_workspace(ctypes.byref(shape), ctypes.byref(size))
    return size.value


def orthogonalize(g, out, steps=5, coefficients=MUON, eps=1e-7, scale=1.0, workspace=None, stream=None):
    """out = scale * (g made nearly orthogonal by `steps` Newton-Schulz steps), for each matrix of g [rows][cols] or
    [matrices][rows][cols] (see uvu_orthogonalize); out may be g; `workspace` (uint8) is allocated here with torch if None."""
    dev, shape = _ortho_shape(g, out, steps, coefficients, eps, scale)
    need = orthogonalize_workspace_bytes(g) if workspace is None else 0
    ws, size, held = _scratch(need, workspace, dev, stream)
    uvu_orthogonalize(ctypes.byref(shape), g.data_ptr(), out.data_ptr(), ws, size, _raw_stream(stream, dev))


def orthogonalize_device_status(reset: bool = True) -> int:
    """Status word of the orthogonalisation's kernels on the current device (0 = no timeout)."""
    w = ctypes.c_uint()
    uvu_orthogonalize_device_status(ctypes.byref(w), int(reset))
    return w.value
