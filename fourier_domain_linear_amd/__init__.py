"""MI355X-native EQ-Linear forward: a thin ctypes binding over libeqlin.so (include/eqlin.h).

The binding only marshals arguments (shape/dtype/device checks, pointers, the current HIP stream);
every step of the layer runs in the library's HIP kernels. There is no CPU fallback: if the library
is missing, every call raises.

    import fourier_domain_linear_amd as eq
    h = eq.prepare_weights(W)                 # W: cuda tensor [C_out, C_in, G], bf16 or fp32
    y = eq.forward(h, x, b)                   # x: [N, C_in, G]; b: [C_out] or None
    y2 = eq.forward_expanded(h, x, b)         # needs prepare_weights(W, expanded=True)
    dx = eq.backward_data(h, dy)              # needs prepare_weights(W, backward=True)
    dW, db = eq.backward_weights(h, x, dy)    # float32 gradients of W and b
    z = eq.forward(h, x, b, act="gelu")       # GELU(y), applied in the kernel's epilogue
    y = eq.mlp_block(h1, b1, h2, b2, x)       # EQ-Linear(C -> 4C), GELU, EQ-Linear(4C -> C)
    hc = eq.prepare_conv_weights(psi)         # p4 group convolution, psi [C_out, C_in, 4, k, k]
    y = eq.conv_forward(hc, x, b)             # x [B, H, W, C_in, 4] -> y [B, H, W, C_out, 4]

The operators between the layers of a transformer stage (include/eqlin.h has their formulas):

    y, s, rstd = eq.rmsnorm(x, gamma, residual=r)              # x, r: [N, C, G]; gamma: [C]
    q, scale, s, rstd = eq.rmsnorm_quant(x, gamma, residual=r) # q: float8_e4m3fn, one scale a token
    dx, dgamma = eq.rmsnorm_backward(dy, s, gamma, rstd, ds=ds)
    qk = eq.rotary(qk, pos, pairs=(4, 4))                      # qk: [N, H, dc, G]; pos: int32 [N, axes]
    o, lse = eq.attention(q, k, v, cu_q, cu_k, causal=False)   # q: [T, H, D] or [T, H, dc, G]
    dq, dk, dv = eq.attention_backward(do, q, k, v, o, lse, cu_q, cu_k, causal=False)

Method: "Flash EQ-Linear: Accelerating Equivariant Linear Layers via Group-wise Discrete Fourier
Transform" (explainer page, gist.science/es/paper/2607.21271).
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libeqlin.so")

EQLIN_OK = 0
EQLIN_ERR_INVALID_ARG = 1
EQLIN_ERR_UNSUPPORTED = 2
EQLIN_ERR_OUT_OF_MEMORY = 3
EQLIN_ERR_HIP = 4
EQLIN_F32 = 0
EQLIN_BF16 = 1
EQLIN_F16 = 2
EQLIN_PREPARE_EXPANDED = 1
EQLIN_PREPARE_BACKWARD = 2
EQLIN_PREPARE_D4 = 4
EQLIN_PREPARE_FIXED_KERNEL = 8
GROUPS = ("cyclic", "d4")
EQLIN_ROTARY_INVERSE = 1
EQLIN_ROTARY_D4 = 4
EQLIN_ACT_NONE = 0
EQLIN_ACT_GELU = 1
_ACTS = {None: EQLIN_ACT_NONE, "none": EQLIN_ACT_NONE, "gelu": EQLIN_ACT_GELU}

# Every symbol include/eqlin.h declares.
EXPORTED = (
    "eqlin_prepare_weights", "eqlin_forward", "eqlin_forward_expanded", "eqlin_forward_act",
    "eqlin_forward_expanded_act", "eqlin_backward_data", "eqlin_backward_data_expanded",
    "eqlin_backward_weights_workspace", "eqlin_backward_weights", "eqlin_backward_weights_static", "eqlin_destroy",
    "eqlin_export_spectral_weights", "eqlin_export_expanded_weight", "eqlin_describe",
    "eqlin_status_string", "eqlin_last_error", "eqlin_version",
    "eqlin_prepare_conv_weights", "eqlin_conv_forward", "eqlin_conv_forward_expanded",
    "eqlin_rmsnorm", "eqlin_rmsnorm_quant", "eqlin_rmsnorm_backward_workspace", "eqlin_rmsnorm_backward",
    "eqlin_rotary", "eqlin_attention_workspace", "eqlin_attention", "eqlin_attention_backward_workspace",
    "eqlin_attention_backward",
)

_lib = None

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float


class AttentionArgs(ctypes.Structure):
    """eqlin_attention_args."""
    _fields_ = [("q", _vp), ("k", _vp), ("v", _vp), ("o", _vp), ("lse", _vp),
                ("q_token_stride", _i64), ("q_head_stride", _i64), ("k_token_stride", _i64), ("k_head_stride", _i64),
                ("v_token_stride", _i64), ("v_head_stride", _i64), ("o_token_stride", _i64), ("o_head_stride", _i64),
                ("cu_q", _vp), ("cu_k", _vp), ("len_k", _vp), ("total_q", _i64), ("total_k", _i64),
                ("batch", _i32), ("heads_q", _i32), ("heads_kv", _i32), ("dim", _i32),
                ("scale", _f32), ("causal", _i32), ("dtype", _i32)]


class AttentionGrads(ctypes.Structure):
    """eqlin_attention_grads."""
    _fields_ = [("d_o", _vp), ("dq", _vp), ("dk", _vp), ("dv", _vp),
                ("do_token_stride", _i64), ("do_head_stride", _i64), ("dq_token_stride", _i64), ("dq_head_stride", _i64),
                ("dk_token_stride", _i64), ("dk_head_stride", _i64), ("dv_token_stride", _i64), ("dv_head_stride", _i64)]


class EqlinError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


def load_library() -> ctypes.CDLL:
    """Load libeqlin.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with `python -m fourier_domain_linear_amd.build` "
            "(there is no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, u32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint
    lib.eqlin_prepare_weights.argtypes = [vp, i32, i32, i32, i32, u32, vp, ctypes.POINTER(vp)]
    lib.eqlin_forward.argtypes = [vp, vp, vp, vp, i64, vp]
    lib.eqlin_forward_expanded.argtypes = [vp, vp, vp, vp, i64, vp]
    lib.eqlin_forward_act.argtypes = [vp, vp, vp, vp, i64, i32, vp]
    lib.eqlin_forward_expanded_act.argtypes = [vp, vp, vp, vp, i64, i32, vp]
    lib.eqlin_backward_data.argtypes = [vp, vp, vp, i64, vp]
    lib.eqlin_backward_data_expanded.argtypes = [vp, vp, vp, i64, vp]
    lib.eqlin_backward_weights_workspace.argtypes = [vp, i64]
    lib.eqlin_backward_weights_workspace.restype = ctypes.c_size_t
    lib.eqlin_backward_weights.argtypes = [vp, vp, vp, vp, vp, i64, vp, ctypes.c_size_t, vp]
    lib.eqlin_backward_weights_static.argtypes = [vp, vp, vp, vp, vp, i64, vp]
    lib.eqlin_prepare_conv_weights.argtypes = [vp, i32, i32, i32, i32, i32, u32, vp, ctypes.POINTER(vp)]
    lib.eqlin_conv_forward.argtypes = [vp, vp, vp, vp, i64, i32, i32, vp]
    lib.eqlin_conv_forward_expanded.argtypes = [vp, vp, vp, vp, i64, i32, i32, vp]
    lib.eqlin_destroy.argtypes = [vp]
    lib.eqlin_export_spectral_weights.argtypes = [vp, vp, vp]
    lib.eqlin_export_expanded_weight.argtypes = [vp, vp, vp]
    lib.eqlin_describe.argtypes = [vp, ctypes.c_char_p, ctypes.c_size_t]
    lib.eqlin_describe.restype = i32
    lib.eqlin_status_string.argtypes = [i32]
    lib.eqlin_status_string.restype = ctypes.c_char_p
    lib.eqlin_last_error.argtypes = []
    lib.eqlin_last_error.restype = ctypes.c_char_p
    lib.eqlin_version.argtypes = []
    lib.eqlin_version.restype = ctypes.c_char_p
    for name in ("eqlin_prepare_weights", "eqlin_forward", "eqlin_forward_expanded", "eqlin_destroy",
                 "eqlin_forward_act", "eqlin_forward_expanded_act", "eqlin_backward_data", "eqlin_backward_weights",
                 "eqlin_backward_data_expanded",
                 "eqlin_backward_weights_static", "eqlin_prepare_conv_weights", "eqlin_conv_forward",
                 "eqlin_conv_forward_expanded",
                 "eqlin_export_spectral_weights", "eqlin_export_expanded_weight"):
        getattr(lib, name).restype = i32
    szt, f32, args, grads = ctypes.c_size_t, ctypes.c_float, ctypes.POINTER(AttentionArgs), ctypes.POINTER(AttentionGrads)
    lib.eqlin_rmsnorm.argtypes = [vp, vp, vp, vp, vp, vp, i64, i32, i32, f32, i32, vp]
    lib.eqlin_rmsnorm_quant.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, f32, i32, vp]
    lib.eqlin_rmsnorm_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, vp, szt, vp]
    lib.eqlin_rmsnorm_backward_workspace.argtypes = [i64, i32, i32]
    lib.eqlin_rotary.argtypes = [vp, i64, i64, vp, i64, i64, vp, i64, i32, i32, i32, i32, ctypes.POINTER(i32),
                                 ctypes.c_double, u32, i32, vp]
    lib.eqlin_attention_workspace.argtypes = [args]
    lib.eqlin_attention.argtypes = [args, vp, szt, vp]
    lib.eqlin_attention_backward_workspace.argtypes = [args]
    lib.eqlin_attention_backward.argtypes = [args, grads, vp, szt, vp]
    for name in ("eqlin_rmsnorm", "eqlin_rmsnorm_quant", "eqlin_rmsnorm_backward", "eqlin_rotary", "eqlin_attention",
                 "eqlin_attention_backward"):
        getattr(lib, name).restype = i32
    for name in ("eqlin_rmsnorm_backward_workspace", "eqlin_attention_workspace", "eqlin_attention_backward_workspace"):
        getattr(lib, name).restype = szt
    _lib = lib
    return lib


def _check(status: int, what: str):
    if status != EQLIN_OK:
        lib = load_library()
        name = lib.eqlin_status_string(status).decode()
        detail = lib.eqlin_last_error().decode()
        raise EqlinError(status, f"{what}: {name}: {detail}")


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return EQLIN_BF16
    if dt == torch.float16:
        return EQLIN_F16
    if dt == torch.float32:
        return EQLIN_F32
    raise TypeError(f"unsupported dtype {dt} (bfloat16, float16 or float32)")


def _need_cuda(t: torch.Tensor, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class Handle:
    """Owns an eqlin_handle_t; destroyed with the object (or explicitly via destroy())."""

    def __init__(self, ptr: int, C_out: int, C_in: int, G: int, dtype: torch.dtype, device, expanded: bool,
                 backward: bool = False, group: str = "cyclic", conv_k: int = 0):
        self.ptr = ptr
        self.conv_k = conv_k
        self.C_out, self.C_in, self.G, self.group = C_out, C_in, G, group
        self.dtype, self.device, self.expanded, self.backward = dtype, device, expanded, backward

    def destroy(self):
        if self.ptr:
            load_library().eqlin_destroy(ctypes.c_void_p(self.ptr))
            self.ptr = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

    def describe(self) -> str:
        return describe(self)


def prepare_weights(W: torch.Tensor, expanded: bool = False, backward: bool = False, group: str = "cyclic",
                    fixed_kernel: bool = False) -> Handle:
    """eqlin_prepare_weights: W [C_out, C_in, G] (cuda, bf16 or fp32) -> Handle. ``expanded`` builds the
    unrolled comparator, ``backward`` the weights of backward_data. ``group``: "cyclic" (G = 1, 2, 4, 8)
    or "d4", the dihedral group of the square (G = 8, element a + 4b = r^a s^b; EQLIN_PREPARE_D4).
    ``fixed_kernel``: one forward kernel for every batch size (EQLIN_PREPARE_FIXED_KERNEL)."""
    if group not in GROUPS:
        raise ValueError(f"group must be one of {GROUPS}, got {group!r}")
    lib = load_library()
    _need_cuda(W, "W")
    if W.dim() != 3:
        raise ValueError(f"W must be [C_out, C_in, G], got {tuple(W.shape)}")
    C_out, C_in, G = W.shape
    out = ctypes.c_void_p()
    flags = (EQLIN_PREPARE_EXPANDED if expanded else 0) | (EQLIN_PREPARE_BACKWARD if backward else 0) | \
        (EQLIN_PREPARE_D4 if group == "d4" else 0) | (EQLIN_PREPARE_FIXED_KERNEL if fixed_kernel else 0)
    with torch.cuda.device(W.device):
        st = lib.eqlin_prepare_weights(ctypes.c_void_p(W.data_ptr()), C_out, C_in, G, _dtype_code(W.dtype),
                                       flags, _stream(W), ctypes.byref(out))
    _check(st, "eqlin_prepare_weights")
    return Handle(out.value, C_out, C_in, G, W.dtype, W.device, expanded, backward, group)


def _act_code(act) -> int:
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(k for k in _ACTS if k)} or None, got {act!r}")
    return _ACTS[act]


def _forward(fn, what: str, h: Handle, x: torch.Tensor, b: torch.Tensor | None, y: torch.Tensor | None,
             act: int | None = None):
    _need_cuda(x, "x")
    if x.dtype != h.dtype:
        raise TypeError(f"x dtype {x.dtype} != handle dtype {h.dtype}")
    if x.dim() != 3 or x.shape[1] != h.C_in or x.shape[2] != h.G:
        raise ValueError(f"x must be [N, {h.C_in}, {h.G}], got {tuple(x.shape)}")
    N = x.shape[0]
    if y is None:
        y = torch.empty((N, h.C_out, h.G), dtype=x.dtype, device=x.device)
    else:
        _need_cuda(y, "y")
        if y.dtype != h.dtype or tuple(y.shape) != (N, h.C_out, h.G):
            raise ValueError(f"y must be [{N}, {h.C_out}, {h.G}] of {h.dtype}")
    bp = None
    if b is not None:
        _need_cuda(b, "b")
        if b.dtype != h.dtype or tuple(b.shape) != (h.C_out,):
            raise ValueError(f"b must be [{h.C_out}] of {h.dtype}")
        bp = ctypes.c_void_p(b.data_ptr())
    args = (ctypes.c_void_p(h.ptr), ctypes.c_void_p(x.data_ptr()), bp, ctypes.c_void_p(y.data_ptr()), N)
    with torch.cuda.device(x.device):
        st = fn(*args, _stream(x)) if act is None else fn(*args, act, _stream(x))
    _check(st, what)
    return y


def forward(h: Handle, x: torch.Tensor, b: torch.Tensor | None = None, y: torch.Tensor | None = None,
            act: str | None = None):
    """eqlin_forward: y[n, o, h] = b[o] + sum_{i,g} W[o, i, (h-g) mod G] x[n, i, g] (spectral kernel).
    act="gelu" calls eqlin_forward_act instead, which applies GELU to y in the kernel's epilogue."""
    lib = load_library()
    if _act_code(act) == EQLIN_ACT_NONE:
        return _forward(lib.eqlin_forward, "eqlin_forward", h, x, b, y)
    return _forward(lib.eqlin_forward_act, "eqlin_forward_act", h, x, b, y, _act_code(act))


def forward_expanded(h: Handle, x: torch.Tensor, b: torch.Tensor | None = None, y: torch.Tensor | None = None,
                     act: str | None = None):
    """eqlin_forward_expanded: the same layer as one dense product with the unrolled weight (with
    act="gelu": eqlin_forward_expanded_act)."""
    if not h.expanded:
        raise ValueError("handle was prepared without expanded=True")
    lib = load_library()
    if _act_code(act) == EQLIN_ACT_NONE:
        return _forward(lib.eqlin_forward_expanded, "eqlin_forward_expanded", h, x, b, y)
    return _forward(lib.eqlin_forward_expanded_act, "eqlin_forward_expanded_act", h, x, b, y, _act_code(act))


def mlp_block(h1: Handle, b1: torch.Tensor | None, h2: Handle, b2: torch.Tensor | None, x: torch.Tensor,
              hidden: torch.Tensor | None = None, y: torch.Tensor | None = None, expanded: bool = False):
    """The transformer MLP block as two library calls on the current stream: hidden = GELU(layer 1 (x))
    with GELU in layer 1's epilogue, then y = layer 2 (hidden). h1: [C_h, C, G] weights, h2: [C, C_h, G].
    expanded=True runs both layers as dense products with the unrolled weights (the comparator)."""
    if h1.C_out != h2.C_in or h1.G != h2.G or h1.dtype != h2.dtype or h1.group != h2.group:
        raise ValueError("layer 2 must take layer 1's outputs (C_in, G and dtype)")
    fwd = forward_expanded if expanded else forward
    hidden = fwd(h1, x, b1, hidden, act="gelu")
    return fwd(h2, hidden, b2, y)


def backward_data(h: Handle, dy: torch.Tensor, dx: torch.Tensor | None = None) -> torch.Tensor:
    """eqlin_backward_data: dx[n, i, g] = sum_{o, h} W[o, i, (h-g) mod G] dy[n, o, h]."""
    if not h.backward:
        raise ValueError("handle was prepared without backward=True")
    _need_cuda(dy, "dy")
    if dy.dtype != h.dtype or dy.dim() != 3 or dy.shape[1] != h.C_out or dy.shape[2] != h.G:
        raise ValueError(f"dy must be [N, {h.C_out}, {h.G}] of {h.dtype}, got {tuple(dy.shape)} {dy.dtype}")
    N = dy.shape[0]
    if dx is None:
        dx = torch.empty((N, h.C_in, h.G), dtype=dy.dtype, device=dy.device)
    else:
        _need_cuda(dx, "dx")
        if dx.dtype != h.dtype or tuple(dx.shape) != (N, h.C_in, h.G):
            raise ValueError(f"dx must be [{N}, {h.C_in}, {h.G}] of {h.dtype}")
    with torch.cuda.device(dy.device):
        st = load_library().eqlin_backward_data(ctypes.c_void_p(h.ptr), ctypes.c_void_p(dy.data_ptr()),
                                                ctypes.c_void_p(dx.data_ptr()), N, _stream(dy))
    _check(st, "eqlin_backward_data")
    return dx


def backward_data_expanded(h: Handle, dy: torch.Tensor, dx: torch.Tensor | None = None) -> torch.Tensor:
    """eqlin_backward_data_expanded: the same dx as one dense product with the unrolled weight (needs
    prepare_weights(W, expanded=True, backward=True))."""
    if not (h.backward and h.expanded):
        raise ValueError("handle was prepared without expanded=True and backward=True")
    _need_cuda(dy, "dy")
    if dy.dtype != h.dtype or dy.dim() != 3 or dy.shape[1] != h.C_out or dy.shape[2] != h.G:
        raise ValueError(f"dy must be [N, {h.C_out}, {h.G}] of {h.dtype}, got {tuple(dy.shape)} {dy.dtype}")
    N = dy.shape[0]
    if dx is None:
        dx = torch.empty((N, h.C_in, h.G), dtype=dy.dtype, device=dy.device)
    else:
        _need_cuda(dx, "dx")
        if dx.dtype != h.dtype or tuple(dx.shape) != (N, h.C_in, h.G):
            raise ValueError(f"dx must be [{N}, {h.C_in}, {h.G}] of {h.dtype}")
    with torch.cuda.device(dy.device):
        st = load_library().eqlin_backward_data_expanded(ctypes.c_void_p(h.ptr), ctypes.c_void_p(dy.data_ptr()),
                                                         ctypes.c_void_p(dx.data_ptr()), N, _stream(dy))
    _check(st, "eqlin_backward_data_expanded")
    return dx


def backward_weights_workspace(h: Handle, N: int) -> int:
    """Bytes of device scratch eqlin_backward_weights needs for N tokens."""
    return int(load_library().eqlin_backward_weights_workspace(ctypes.c_void_p(h.ptr), int(N)))


def backward_weights(h: Handle, x: torch.Tensor, dy: torch.Tensor, with_bias: bool = True,
                     workspace: torch.Tensor | None = None):
    """eqlin_backward_weights -> (dW float32 [C_out, C_in, G], db float32 [C_out] or None):
    dW[o, i, d] = sum_{n, h} dy[n, o, h] x[n, i, (h-d) mod G], db[o] = sum_{n, h} dy[n, o, h]."""
    _need_cuda(x, "x")
    _need_cuda(dy, "dy")
    if x.dtype != h.dtype or dy.dtype != h.dtype:
        raise TypeError(f"x and dy must be {h.dtype}")
    if x.dim() != 3 or x.shape[1:] != (h.C_in, h.G) or dy.dim() != 3 or dy.shape[1:] != (h.C_out, h.G) \
            or x.shape[0] != dy.shape[0]:
        raise ValueError(f"x must be [N, {h.C_in}, {h.G}] and dy [N, {h.C_out}, {h.G}]")
    N = x.shape[0]
    dW = torch.empty((h.C_out, h.C_in, h.G), dtype=torch.float32, device=x.device)
    db = torch.empty((h.C_out,), dtype=torch.float32, device=x.device) if with_bias else None
    need = backward_weights_workspace(h, N)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty((need,), dtype=torch.uint8, device=x.device)
    wsp = ctypes.c_void_p(workspace.data_ptr()) if need else None
    with torch.cuda.device(x.device):
        st = load_library().eqlin_backward_weights(
            ctypes.c_void_p(h.ptr), ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(dy.data_ptr()),
            ctypes.c_void_p(dW.data_ptr()), ctypes.c_void_p(db.data_ptr()) if db is not None else None, N, wsp,
            need, _stream(x))
    _check(st, "eqlin_backward_weights")
    return dW, db


def prepare_conv_weights(psi: torch.Tensor, expanded: bool = False) -> Handle:
    """eqlin_prepare_conv_weights: psi [C_out, C_in, 4, k, k] (cuda, bf16 or fp16) -> Handle of the p4
    group convolution y[b, p, o, h] = bias[o] + sum psi[o, i, (h - g) mod 4, R^-h delta] x[b, p + delta, i, g].
    ``expanded`` also builds the unrolled comparator (conv_forward_expanded)."""
    lib = load_library()
    _need_cuda(psi, "psi")
    if psi.dim() != 5 or psi.shape[2] != 4 or psi.shape[3] != psi.shape[4]:
        raise ValueError(f"psi must be [C_out, C_in, 4, k, k], got {tuple(psi.shape)}")
    C_out, C_in, G, k, _ = psi.shape
    out = ctypes.c_void_p()
    with torch.cuda.device(psi.device):
        st = lib.eqlin_prepare_conv_weights(ctypes.c_void_p(psi.data_ptr()), C_out, C_in, G, k, _dtype_code(psi.dtype),
                                            EQLIN_PREPARE_EXPANDED if expanded else 0, _stream(psi), ctypes.byref(out))
    _check(st, "eqlin_prepare_conv_weights")
    return Handle(out.value, C_out, C_in, G, psi.dtype, psi.device, expanded, conv_k=k)


def _conv(fn, what: str, h: Handle, x: torch.Tensor, b: torch.Tensor | None, y: torch.Tensor | None):
    if not h.conv_k:
        raise ValueError("not a convolution handle (prepare_conv_weights)")
    _need_cuda(x, "x")
    if x.dtype != h.dtype or x.dim() != 5 or x.shape[3:] != (h.C_in, h.G):
        raise ValueError(f"x must be [B, H, W, {h.C_in}, {h.G}] of {h.dtype}, got {tuple(x.shape)} {x.dtype}")
    B, H, W = x.shape[:3]
    if y is None:
        y = torch.empty((B, H, W, h.C_out, h.G), dtype=x.dtype, device=x.device)
    else:
        _need_cuda(y, "y")
        if y.dtype != h.dtype or tuple(y.shape) != (B, H, W, h.C_out, h.G):
            raise ValueError(f"y must be [{B}, {H}, {W}, {h.C_out}, {h.G}] of {h.dtype}")
    bp = None
    if b is not None:
        _need_cuda(b, "b")
        if b.dtype != h.dtype or tuple(b.shape) != (h.C_out,):
            raise ValueError(f"b must be [{h.C_out}] of {h.dtype}")
        bp = ctypes.c_void_p(b.data_ptr())
    with torch.cuda.device(x.device):
        st = fn(ctypes.c_void_p(h.ptr), ctypes.c_void_p(x.data_ptr()), bp, ctypes.c_void_p(y.data_ptr()), B, H, W,
                _stream(x))
    _check(st, what)
    return y


def conv_forward(h: Handle, x: torch.Tensor, b: torch.Tensor | None = None, y: torch.Tensor | None = None):
    """eqlin_conv_forward: x [B, H, W, C_in, 4] -> y [B, H, W, C_out, 4] (the spectral kernel)."""
    return _conv(load_library().eqlin_conv_forward, "eqlin_conv_forward", h, x, b, y)


def conv_forward_expanded(h: Handle, x: torch.Tensor, b: torch.Tensor | None = None, y: torch.Tensor | None = None):
    """eqlin_conv_forward_expanded: the same through the unrolled gathered layer (needs expanded=True)."""
    if not h.expanded:
        raise ValueError("handle was prepared without expanded=True")
    return _conv(load_library().eqlin_conv_forward_expanded, "eqlin_conv_forward_expanded", h, x, b, y)


# ---- the operators between the layers of a transformer stage ----


# the current stream's handle without building a Stream object (microseconds a call); public API where it is missing
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on(index: int, fn, *args):
    """fn(*args, current stream) with device ``index`` current: the launch goes where the tensors are."""
    if torch.cuda.current_device() == index:
        return fn(*args, _raw_stream(index))
    with torch.cuda.device(index):
        return fn(*args, _raw_stream(index))


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _same(t: torch.Tensor, like: torch.Tensor, name: str, shape=None):
    """t: contiguous, on like's device, of its dtype and shape (or ``shape``)."""
    _need_cuda(t, name)
    if t.dtype != like.dtype or t.get_device() != like.get_device() or t.shape != (like.shape if shape is None else shape):
        raise ValueError(f"{name} must be {tuple(like.shape if shape is None else shape)} of {like.dtype} on {like.device}, "
                         f"got {tuple(t.shape)} {t.dtype} on {t.device}")


def _f32_out(t: torch.Tensor | None, shape, device, name: str):
    if t is None:
        return torch.empty(shape, dtype=torch.float32, device=device)
    _need_cuda(t, name)
    if t.dtype != torch.float32 or t.shape != shape or t.device != device:
        raise ValueError(f"{name} must be {tuple(shape)} of float32 on {device}")
    return t


def _norm_args(x, gamma, residual):
    _need_cuda(x, "x")
    code = _dtype_code(x.dtype)
    if x.dim() != 3:
        raise ValueError(f"x must be [N, C, G], got {tuple(x.shape)}")
    if residual is not None:
        _same(residual, x, "residual")
    if gamma is not None:
        _same(gamma, x, "gamma", (x.shape[1],))
    return code


def rmsnorm(x: torch.Tensor, gamma: torch.Tensor | None = None, residual: torch.Tensor | None = None, eps: float = 1e-6,
            y: torch.Tensor | None = None):
    """eqlin_rmsnorm -> (y, s, rstd): s = x + residual (x itself without one), rstd [N] float32 over a token's
    C * G values, y = s rstd gamma[c]. x: [N, C, G]; gamma: [C] of x's dtype or None."""
    code = _norm_args(x, gamma, residual)
    N, C, G = x.shape
    if y is None:
        y = torch.empty_like(x)
    else:
        _same(y, x, "y")
    s = x if residual is None else torch.empty_like(x)
    rstd = x.new_empty(N, dtype=torch.float32)
    st = _on(x.get_device(), load_library().eqlin_rmsnorm, x.data_ptr(), _ptr(residual), _ptr(gamma),
             None if residual is None else s.data_ptr(), y.data_ptr(), rstd.data_ptr(), N, C, G, eps, code)
    _check(st, "eqlin_rmsnorm")
    return y, s, rstd


def rmsnorm_quant(x: torch.Tensor, gamma: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                  eps: float = 1e-6):
    """eqlin_rmsnorm_quant -> (q, scale, s, rstd): rmsnorm's y as q float8_e4m3fn [N, C, G] times scale [N]
    float32 (the row's largest magnitude / 448)."""
    code = _norm_args(x, gamma, residual)
    N, C, G = x.shape
    q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    s = x if residual is None else torch.empty_like(x)
    rstd = x.new_empty(N, dtype=torch.float32)
    scale = x.new_empty(N, dtype=torch.float32)
    st = _on(x.get_device(), load_library().eqlin_rmsnorm_quant, x.data_ptr(), _ptr(residual), _ptr(gamma),
             None if residual is None else s.data_ptr(), q.data_ptr(), scale.data_ptr(), rstd.data_ptr(), N, C, G, eps, code)
    _check(st, "eqlin_rmsnorm_quant")
    return q, scale, s, rstd


def rmsnorm_backward_workspace(N: int, C: int, G: int) -> int:
    """Bytes of device scratch eqlin_rmsnorm_backward needs (0 without dgamma)."""
    return int(load_library().eqlin_rmsnorm_backward_workspace(int(N), int(C), int(G)))


def rmsnorm_backward(dy: torch.Tensor, s: torch.Tensor, gamma: torch.Tensor | None, rstd: torch.Tensor,
                     ds: torch.Tensor | None = None, with_gamma: bool = True, workspace: torch.Tensor | None = None):
    """eqlin_rmsnorm_backward -> (dx, dgamma): dx [N, C, G], the gradient of x and of the residual (ds: the
    gradient that reaches s directly), and dgamma [C] float32 (None with with_gamma=False). s, rstd: rmsnorm's."""
    code = _norm_args(s, gamma, None)
    _same(dy, s, "dy")
    if ds is not None:
        _same(ds, s, "ds")
    N, C, G = s.shape
    _f32_out(rstd, (N,), s.device, "rstd")
    dx = torch.empty_like(s)
    dgamma = torch.empty((C,), dtype=torch.float32, device=s.device) if with_gamma else None
    need = rmsnorm_backward_workspace(N, C, G) if with_gamma else 0
    workspace = _workspace(workspace, need, s.device)
    st = _on(s.get_device(), load_library().eqlin_rmsnorm_backward, s.data_ptr(), _ptr(gamma), rstd.data_ptr(), dy.data_ptr(),
             _ptr(ds), dx.data_ptr(), _ptr(dgamma), N, C, G, code, _ptr(workspace), need)
    _check(st, "eqlin_rmsnorm_backward")
    return dx, dgamma


def _workspace(workspace: torch.Tensor | None, need: int, device):
    """The caller's scratch where it is large enough, else a new one (torch's allocator keeps it for this stream)."""
    if need == 0:
        return None
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        return torch.empty((need,), dtype=torch.uint8, device=device)
    _need_cuda(workspace, "workspace")
    if workspace.device != device:
        raise ValueError(f"workspace must be on {device}")
    return workspace


def _heads(t: torch.Tensor, name: str):
    """(tokens, heads, dim) of a [T, H, D] or [T, H, dc, G] view whose heads are contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    shape, strides = t.shape, t.stride()
    if len(shape) == 3:
        dim, ok = shape[2], strides[2] == 1 or shape[2] == 1
    elif len(shape) == 4:
        dim, ok = shape[2] * shape[3], (strides[3] == 1 or shape[3] == 1) and (strides[2] == shape[3] or shape[2] == 1)
    else:
        raise ValueError(f"{name} must be [T, H, D] or [T, H, dc, G], got {tuple(shape)}")
    if not ok:
        raise ValueError(f"{name}: a head's elements must be contiguous")
    return shape[0], shape[1], dim


def _index(t: torch.Tensor, name: str, shape, index: int):
    _need_cuda(t, name)
    if t.dtype != torch.int32 or t.shape != shape or t.get_device() != index:
        raise ValueError(f"{name} must be {tuple(shape)} of int32 on device {index}, got {tuple(t.shape)} {t.dtype} on {t.device}")


def rotary(x: torch.Tensor, pos: torch.Tensor, pairs, base: float = 10000.0, group: str = "cyclic", inverse: bool = False,
           out: torch.Tensor | None = None) -> torch.Tensor:
    """eqlin_rotary: x [N, H, dc, G] (or [N, H, D], G = 1; heads contiguous, tokens and heads strided) turned by
    the positions pos, int32 [N, axes] ((row, column) last). pairs: channel pairs of each axis. inverse=True
    turns back: the backward (dx from dy). out: a tensor to write to, x itself for in place."""
    if group not in GROUPS:
        raise ValueError(f"group must be one of {GROUPS}, got {group!r}")
    N, H, D = _heads(x, "x")
    G = x.shape[3] if x.dim() == 4 else 1
    axes = len(pairs)
    _index(pos, "pos", (N, axes), x.get_device())
    if out is None:
        out = x.new_empty(x.shape)
    elif out is not x:
        _heads(out, "out")
        if out.shape != x.shape or out.dtype != x.dtype or out.device != x.device:
            raise ValueError(f"out must be {tuple(x.shape)} of {x.dtype} on {x.device}")
    flags = (EQLIN_ROTARY_INVERSE if inverse else 0) | (EQLIN_ROTARY_D4 if group == "d4" else 0)
    xs, ys = x.stride(), out.stride()
    st = _on(x.get_device(), load_library().eqlin_rotary, x.data_ptr(), xs[0], xs[1], out.data_ptr(), ys[0], ys[1],
             pos.data_ptr(), N, H, D // G if G else 0, G, axes, (ctypes.c_int * axes)(*pairs), base, flags,
             _dtype_code(x.dtype))
    _check(st, "eqlin_rotary")
    return out


def _attention_args(q, k, v, o, lse, cu_q, cu_k, len_k, causal, scale):
    Tq, Hq, D = _heads(q, "q")
    Tk, Hkv, Dk = kv = _heads(k, "k")
    dev, dt = q.get_device(), q.dtype
    if _heads(v, "v") != kv or Dk != D:
        raise ValueError(f"k and v must be [T, heads, {D}] alike, got {tuple(k.shape)} and {tuple(v.shape)}")
    if k.dtype != dt or v.dtype != dt or k.get_device() != dev or v.get_device() != dev:
        raise TypeError(f"q, k and v must be of one dtype on one device, got {dt}, {k.dtype}, {v.dtype}")
    if o is None:
        o = q.new_empty(q.shape)
    elif _heads(o, "o") != (Tq, Hq, D) or o.dtype != dt or o.get_device() != dev:
        raise ValueError(f"o must be {tuple(q.shape)} of {dt} on {q.device}")
    if lse is None:
        lse = q.new_empty((Tq, Hq), dtype=torch.float32)
    _need_cuda(cu_q, "cu_q")
    B = cu_q.numel() - 1
    if B < 0:
        raise ValueError("cu_q must hold batch + 1 entries")
    _index(cu_q, "cu_q", (B + 1,), dev)
    _index(cu_k, "cu_k", (B + 1,), dev)
    if len_k is not None:
        _index(len_k, "len_k", (B,), dev)
    qs, ks, vs, os_ = q.stride(), k.stride(), v.stride(), o.stride()
    a = AttentionArgs(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), qs[0], qs[1], ks[0], ks[1],
                      vs[0], vs[1], os_[0], os_[1], cu_q.data_ptr(), cu_k.data_ptr(), _ptr(len_k), Tq, Tk, B, Hq, Hkv, D,
                      D ** -0.5 if scale is None else scale, 1 if causal else 0, _dtype_code(dt))
    return a, o, lse


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor,
              causal: bool = False, scale: float | None = None, len_k: torch.Tensor | None = None,
              out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """eqlin_attention -> (o, lse): attention over packed sequences. q: [T, Hq, D] or [T, Hq, dc, G] (tokens and
    heads may be strided views, e.g. of a qkv layer's output), k and v: the same with Hkv heads, Hq a multiple
    of Hkv. cu_q, cu_k: int32 [batch + 1], the sequences' bounds in tokens; len_k: int32 [batch], how many keys
    of each stretch count. causal: token t of lq sees the keys j <= t + lk - lq. scale: 1/sqrt(D) if None.
    o: like q; lse: float32 [T, Hq]. Rows outside every sequence are left as they are."""
    a, out, lse = _attention_args(q, k, v, out, None, cu_q, cu_k, len_k, causal, scale)
    lib, pa = load_library(), ctypes.byref(a)
    need = lib.eqlin_attention_workspace(pa)
    workspace = _workspace(workspace, need, q.device) if need else None
    st = _on(q.get_device(), lib.eqlin_attention, pa, _ptr(workspace), need)
    if st != EQLIN_OK:
        _check(st, "eqlin_attention")
    return out, lse


def attention_backward(do: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                       lse: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor, causal: bool = False,
                       scale: float | None = None, len_k: torch.Tensor | None = None, dq: torch.Tensor | None = None,
                       dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None):
    """eqlin_attention_backward -> (dq, dk, dv) from do and the forward's tensors and arguments. dq, dk, dv:
    tensors to write to (views of one gradient of a qkv layer's output, say), else new ones."""
    if o is None or lse is None:
        raise ValueError("o and lse are the forward's")
    _f32_out(lse, q.shape[:2], q.device, "lse")
    a, o, lse = _attention_args(q, k, v, o, lse, cu_q, cu_k, len_k, causal, scale)
    grads = []
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is None:
            t = like.new_empty(like.shape)
        elif _heads(t, name) != _heads(like, name) or t.dtype != like.dtype or t.device != like.device:
            raise ValueError(f"{name} must be {tuple(like.shape)} of {like.dtype} on {like.device}")
        grads.append(t)
    dq, dk, dv = grads
    if _heads(do, "do") != _heads(q, "q") or do.dtype != q.dtype or do.device != q.device:
        raise ValueError(f"do must be {tuple(q.shape)} of {q.dtype} on {q.device}")
    g = AttentionGrads(do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), *do.stride()[:2], *dq.stride()[:2],
                       *dk.stride()[:2], *dv.stride()[:2])
    lib, pa = load_library(), ctypes.byref(a)
    need = lib.eqlin_attention_backward_workspace(pa)
    workspace = _workspace(workspace, need, q.device)
    _check(_on(q.get_device(), lib.eqlin_attention_backward, pa, ctypes.byref(g), _ptr(workspace), need),
           "eqlin_attention_backward")
    return dq, dk, dv


STATIC_SCRATCH_BYTES = 64 << 20  # EQLIN_STATIC_SCRATCH_BYTES


def backward_weights_static(h: Handle, x: torch.Tensor, dy: torch.Tensor, with_bias: bool = True):
    """eqlin_backward_weights_static: backward_weights with the library's static per-device scratch
    instead of a workspace (no device allocation in the library; the gradient tensors are allocated
    here unless passed in). Calls on one device must not overlap."""
    _need_cuda(x, "x")
    _need_cuda(dy, "dy")
    if x.dtype != h.dtype or dy.dtype != h.dtype:
        raise TypeError(f"x and dy must be {h.dtype}")
    if x.dim() != 3 or x.shape[1:] != (h.C_in, h.G) or dy.dim() != 3 or dy.shape[1:] != (h.C_out, h.G) \
            or x.shape[0] != dy.shape[0]:
        raise ValueError(f"x must be [N, {h.C_in}, {h.G}] and dy [N, {h.C_out}, {h.G}]")
    N = x.shape[0]
    dW = torch.empty((h.C_out, h.C_in, h.G), dtype=torch.float32, device=x.device)
    db = torch.empty((h.C_out,), dtype=torch.float32, device=x.device) if with_bias else None
    with torch.cuda.device(x.device):
        st = load_library().eqlin_backward_weights_static(
            ctypes.c_void_p(h.ptr), ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(dy.data_ptr()),
            ctypes.c_void_p(dW.data_ptr()), ctypes.c_void_p(db.data_ptr()) if db is not None else None, N,
            _stream(x))
    _check(st, "eqlin_backward_weights_static")
    return dW, db


def export_spectral_weights(h: Handle) -> torch.Tensor:
    """eqlin_export_spectral_weights -> float32 [G, C_out, C_in] (plane order in include/eqlin.h)."""
    out = torch.empty((h.G, h.C_out, h.C_in), dtype=torch.float32, device=h.device)
    with torch.cuda.device(h.device):
        st = load_library().eqlin_export_spectral_weights(ctypes.c_void_p(h.ptr), ctypes.c_void_p(out.data_ptr()),
                                                          _stream(out))
    _check(st, "eqlin_export_spectral_weights")
    return out


def export_expanded_weight(h: Handle) -> torch.Tensor:
    """eqlin_export_expanded_weight -> [C_out*G, C_in*G] of the handle's dtype."""
    out = torch.empty((h.C_out * h.G, h.C_in * h.G), dtype=h.dtype, device=h.device)
    with torch.cuda.device(h.device):
        st = load_library().eqlin_export_expanded_weight(ctypes.c_void_p(h.ptr), ctypes.c_void_p(out.data_ptr()),
                                                         _stream(out))
    _check(st, "eqlin_export_expanded_weight")
    return out


def describe(h: Handle) -> str:
    lib = load_library()
    buf = ctypes.create_string_buffer(512)
    lib.eqlin_describe(ctypes.c_void_p(h.ptr), buf, len(buf))
    return buf.value.decode()


def version() -> str:
    return load_library().eqlin_version().decode()


def status_string(code: int) -> str:
    return load_library().eqlin_status_string(code).decode()


def destroy(h: Handle):
    h.destroy()
