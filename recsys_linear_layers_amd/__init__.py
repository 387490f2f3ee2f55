"""bf16 GEMM and RecSys linear-compression layer for MI355X (gfx950).

Thin Python binding over liblinlayers.so, whose C ABI is declared in
include/linlayers.h.  The functions named like the C entry points
(gemm_plan_create, gemm_run, lincomp_run, ...) only marshal arguments; every
step of the computation runs in the library's HIP kernels.  ``gemm`` and
``lincomp`` are torch conveniences over them (torch supplies device memory and
the current stream).

Importing this module fails if the library has not been built
(``python recsys_linear_layers_amd/build.py``); there is no fallback path.
"""
from __future__ import annotations

import collections
import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblinlayers.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run `python {os.path.join(_HERE, 'build.py')}` "
                      "(or __graft_entry__.build()) first")

_lib = ctypes.CDLL(LIB_PATH)

LL_OK, LL_ERR_INVALID_ARG, LL_ERR_UNSUPPORTED, LL_ERR_WORKSPACE, LL_ERR_HIP, LL_ERR_NO_DEVICE = range(6)
LL_BF16, LL_F32, LL_F16 = 0, 1, 2
LL_EPI_BIAS, LL_EPI_RELU, LL_EPI_GELU, LL_EPI_SILU = 0x1, 0x10, 0x20, 0x30
ACTIVATIONS = {None: 0, "relu": LL_EPI_RELU, "gelu": LL_EPI_GELU, "silu": LL_EPI_SILU}
LL_FLAG_PACK_A = 0x1
LL_FLAG_PACK_B = 0x2
LL_FLAG_PRODUCER_CONSUMER = 0x4
LL_FLAG_COOPERATIVE = 0x8
LL_LINCOMP_NO_DEDUP = 0x1
LL_EMBED_ACCUMULATE = 0x1
LL_XENT_DX, LL_XENT_DW, LL_XENT_PACK_W = 0x1, 0x2, 0x4

_i64 = ctypes.c_int64
_vp = ctypes.c_void_p


class GemmDesc(ctypes.Structure):
    _fields_ = [("M", _i64), ("N", _i64), ("K", _i64),
                ("stride_am", _i64), ("stride_ak", _i64), ("stride_bk", _i64), ("stride_bn", _i64),
                ("stride_cm", _i64), ("stride_cn", _i64),
                ("a_type", ctypes.c_int32), ("b_type", ctypes.c_int32), ("c_type", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("epilogue", ctypes.c_uint32)]


class LincompDesc(ctypes.Structure):
    _fields_ = [("R", _i64), ("C", _i64), ("Nu", _i64), ("Ni", _i64), ("D", _i64), ("Mo", _i64),
                ("su_r", _i64), ("su_c", _i64), ("su_n", _i64),
                ("si_r", _i64), ("si_c", _i64), ("si_n", _i64),
                ("sw_n", _i64),
                ("sy_r", _i64), ("sy_c", _i64), ("sy_m", _i64),
                ("y_type", ctypes.c_int32), ("flags", ctypes.c_uint32), ("epilogue", ctypes.c_uint32)]


class LincompRaggedDesc(ctypes.Structure):
    _fields_ = [("R", _i64), ("Ctot", _i64), ("Nu", _i64), ("Ni", _i64), ("D", _i64), ("Mo", _i64),
                ("su_r", _i64), ("su_n", _i64),
                ("si_c", _i64), ("si_n", _i64),
                ("sw_n", _i64),
                ("sy_c", _i64), ("sy_m", _i64),
                ("y_type", ctypes.c_int32), ("flags", ctypes.c_uint32), ("epilogue", ctypes.c_uint32)]


class EmbedDesc(ctypes.Structure):
    _fields_ = [("V", _i64), ("T", _i64), ("D", _i64), ("stride_table", _i64), ("stride_out", _i64),
                ("type", ctypes.c_int32), ("scale", ctypes.c_float)]


class EmbedGradDesc(ctypes.Structure):
    _fields_ = [("V", _i64), ("T", _i64), ("D", _i64), ("stride_dout", _i64), ("stride_dtable", _i64),
                ("padding_id", _i64), ("type", ctypes.c_int32), ("scale", ctypes.c_float),
                ("flags", ctypes.c_uint32)]


class LayernormDesc(ctypes.Structure):
    _fields_ = [("N", _i64), ("D", _i64), ("stride_x", _i64), ("stride_y", _i64),
                ("type", ctypes.c_int32), ("param_type", ctypes.c_int32), ("eps", ctypes.c_float)]


class LayernormGradDesc(ctypes.Structure):
    _fields_ = [("N", _i64), ("D", _i64), ("stride_dy", _i64), ("stride_x", _i64), ("stride_dx", _i64),
                ("type", ctypes.c_int32), ("param_type", ctypes.c_int32)]


class XentDesc(ctypes.Structure):
    _fields_ = [("N", _i64), ("V", _i64), ("D", _i64),
                ("stride_x", _i64), ("stride_w", _i64), ("stride_dx", _i64), ("stride_dw", _i64),
                ("ignore_index", _i64), ("piece_bytes", _i64),
                ("type", ctypes.c_int32), ("dx_type", ctypes.c_int32), ("dw_type", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


_lib.ll_status_string.restype = ctypes.c_char_p
_lib.ll_status_string.argtypes = [ctypes.c_int]
_lib.ll_last_error.restype = ctypes.c_char_p
_lib.ll_last_error.argtypes = []
_lib.gemm_plan_create.argtypes = [ctypes.POINTER(_vp), ctypes.POINTER(GemmDesc)]
_lib.gemm_plan_workspace_size.argtypes = [_vp, ctypes.POINTER(ctypes.c_size_t)]
_lib.gemm_plan_describe.argtypes = [_vp, ctypes.c_char_p, ctypes.c_size_t]
_lib.gemm_run.argtypes = [_vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
_lib.gemm_run_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
_lib.gemm_run_noalloc.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp]
_lib.gemm_plan_destroy.argtypes = [_vp]
_lib.lincomp_workspace_size.argtypes = [ctypes.POINTER(LincompDesc), ctypes.POINTER(ctypes.c_size_t)]
_lib.lincomp_run.argtypes = [ctypes.POINTER(LincompDesc), _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
_lib.lincomp_ragged_run.argtypes = [ctypes.POINTER(LincompRaggedDesc), _vp, _vp, _vp, _vp, _vp, _vp]
_lib.lincomp_run_ex.argtypes = [ctypes.POINTER(LincompDesc), _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
_lib.lincomp_ragged_run_ex.argtypes = [ctypes.POINTER(LincompRaggedDesc), _vp, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.embed_run.argtypes = [ctypes.POINTER(EmbedDesc), _vp, _vp, _vp, _vp]
_lib.embed_grad_workspace_size.argtypes = [ctypes.POINTER(EmbedGradDesc), ctypes.POINTER(ctypes.c_size_t)]
_lib.embed_grad_run.argtypes = [ctypes.POINTER(EmbedGradDesc), _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
_lib.layernorm_run.argtypes = [ctypes.POINTER(LayernormDesc), *[_vp] * 7]
_lib.layernorm_grad_workspace_size.argtypes = [ctypes.POINTER(LayernormGradDesc), ctypes.POINTER(ctypes.c_size_t)]
_lib.layernorm_grad_run.argtypes = [ctypes.POINTER(LayernormGradDesc), *[_vp] * 9, ctypes.c_size_t, _vp]
_lib.xent_plan_create.argtypes = [ctypes.POINTER(_vp), ctypes.POINTER(XentDesc)]
_lib.xent_plan_workspace_size.argtypes = [_vp, ctypes.POINTER(ctypes.c_size_t)]
_lib.xent_plan_describe.argtypes = [_vp, ctypes.c_char_p, ctypes.c_size_t]
_lib.xent_run.argtypes = [*[_vp] * 10, ctypes.c_size_t, _vp]
_lib.xent_plan_destroy.argtypes = [_vp]
for _f in ("gemm_plan_create", "gemm_plan_workspace_size", "gemm_plan_describe", "gemm_run", "gemm_run_ex",
           "gemm_run_noalloc", "gemm_plan_destroy", "lincomp_workspace_size", "lincomp_run", "lincomp_ragged_run",
           "lincomp_run_ex", "lincomp_ragged_run_ex", "embed_run", "embed_grad_workspace_size", "embed_grad_run",
           "layernorm_run", "layernorm_grad_workspace_size", "layernorm_grad_run", "xent_plan_create",
           "xent_plan_workspace_size", "xent_plan_describe", "xent_run", "xent_plan_destroy"):
    getattr(_lib, _f).restype = ctypes.c_int


class LLError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {ll_status_string(status)}: {ll_last_error()}")


def ll_status_string(status: int) -> str:
    return _lib.ll_status_string(int(status)).decode()


def ll_last_error() -> str:
    return _lib.ll_last_error().decode()


def _check(status: int, what: str) -> None:
    if status != LL_OK:
        raise LLError(status, what)


# ---------------------------------------------------------------------------
# C-ABI mirrors (pointers are ints; stream is a hipStream_t value or 0)
# ---------------------------------------------------------------------------

def gemm_plan_create(desc: GemmDesc) -> int:
    h = _vp()
    _check(_lib.gemm_plan_create(ctypes.byref(h), ctypes.byref(desc)), "gemm_plan_create")
    return h.value


def gemm_plan_workspace_size(plan: int) -> int:
    n = ctypes.c_size_t()
    _check(_lib.gemm_plan_workspace_size(plan, ctypes.byref(n)), "gemm_plan_workspace_size")
    return n.value


def gemm_plan_describe(plan: int) -> str:
    buf = ctypes.create_string_buffer(512)
    _check(_lib.gemm_plan_describe(plan, buf, 512), "gemm_plan_describe")
    return buf.value.decode()


def gemm_run(plan: int, A: int, B: int, C: int, workspace: int, ws_bytes: int, stream: int) -> None:
    _check(_lib.gemm_run(plan, A, B, C, workspace, ws_bytes, stream), "gemm_run")


def gemm_run_ex(plan: int, A: int, B: int, C: int, bias: int, workspace: int, ws_bytes: int,
                stream: int = 0) -> None:
    _check(_lib.gemm_run_ex(plan, A, B, C, bias, workspace, ws_bytes, stream), "gemm_run_ex")


LL_NOALLOC_SCRATCH_BYTES = 64 << 20


def gemm_run_noalloc(plan: int, A: int, B: int, C: int, bias: int | None = None, stream: int = 0) -> None:
    _check(_lib.gemm_run_noalloc(plan, A, B, C, bias, stream), "gemm_run_noalloc")


def gemm_plan_destroy(plan: int) -> None:
    _check(_lib.gemm_plan_destroy(plan), "gemm_plan_destroy")


def lincomp_workspace_size(desc: LincompDesc) -> int:
    n = ctypes.c_size_t()
    _check(_lib.lincomp_workspace_size(ctypes.byref(desc), ctypes.byref(n)), "lincomp_workspace_size")
    return n.value


def lincomp_ragged_run(desc: LincompRaggedDesc, offsets: int, user: int, item: int, W: int, Y: int,
                       stream: int = 0) -> None:
    _check(_lib.lincomp_ragged_run(ctypes.byref(desc), offsets, user, item, W, Y, stream), "lincomp_ragged_run")


def lincomp_run(desc: LincompDesc, user: int, item: int, W: int, Y: int, workspace: int, ws_bytes: int,
                stream: int) -> None:
    _check(_lib.lincomp_run(ctypes.byref(desc), user, item, W, Y, workspace, ws_bytes, stream), "lincomp_run")


def lincomp_run_ex(desc: LincompDesc, user: int, item: int, W: int, bias: int | None, Y: int, workspace: int,
                   ws_bytes: int, stream: int) -> None:
    _check(_lib.lincomp_run_ex(ctypes.byref(desc), user, item, W, bias, Y, workspace, ws_bytes, stream),
           "lincomp_run_ex")


def lincomp_ragged_run_ex(desc: LincompRaggedDesc, offsets: int, user: int, item: int, W: int, bias: int | None,
                          Y: int, stream: int = 0) -> None:
    _check(_lib.lincomp_ragged_run_ex(ctypes.byref(desc), offsets, user, item, W, bias, Y, stream),
           "lincomp_ragged_run_ex")


def embed_run(desc: EmbedDesc, table: int, ids: int, out: int, stream: int = 0) -> None:
    _check(_lib.embed_run(ctypes.byref(desc), table, ids, out, stream), "embed_run")


def embed_grad_workspace_size(desc: EmbedGradDesc) -> int:
    n = ctypes.c_size_t()
    _check(_lib.embed_grad_workspace_size(ctypes.byref(desc), ctypes.byref(n)), "embed_grad_workspace_size")
    return n.value


def embed_grad_run(desc: EmbedGradDesc, ids: int, dout: int, dtable: int, workspace: int, ws_bytes: int,
                   stream: int = 0) -> None:
    _check(_lib.embed_grad_run(ctypes.byref(desc), ids, dout, dtable, workspace, ws_bytes, stream), "embed_grad_run")


def layernorm_run(desc: LayernormDesc, x: int, gamma: int | None, beta: int | None, y: int, mean: int | None,
                  rstd: int | None, stream: int = 0) -> None:
    _check(_lib.layernorm_run(ctypes.byref(desc), x, gamma, beta, y, mean, rstd, stream), "layernorm_run")


def layernorm_grad_workspace_size(desc: LayernormGradDesc) -> int:
    n = ctypes.c_size_t()
    _check(_lib.layernorm_grad_workspace_size(ctypes.byref(desc), ctypes.byref(n)), "layernorm_grad_workspace_size")
    return n.value


def layernorm_grad_run(desc: LayernormGradDesc, dy: int, x: int, gamma: int | None, mean: int, rstd: int, dx: int,
                       dgamma: int | None, dbeta: int | None, workspace: int, ws_bytes: int, stream: int = 0) -> None:
    _check(_lib.layernorm_grad_run(ctypes.byref(desc), dy, x, gamma, mean, rstd, dx, dgamma, dbeta, workspace,
                                   ws_bytes, stream), "layernorm_grad_run")


def xent_plan_create(desc: XentDesc) -> int:
    h = _vp()
    _check(_lib.xent_plan_create(ctypes.byref(h), ctypes.byref(desc)), "xent_plan_create")
    return h.value


def xent_plan_workspace_size(plan: int) -> int:
    n = ctypes.c_size_t()
    _check(_lib.xent_plan_workspace_size(plan, ctypes.byref(n)), "xent_plan_workspace_size")
    return n.value


def xent_plan_describe(plan: int) -> str:
    buf = ctypes.create_string_buffer(512)
    _check(_lib.xent_plan_describe(plan, buf, 512), "xent_plan_describe")
    return buf.value.decode()


def xent_run(plan: int, x: int, w: int, target: int, dloss: int | None, loss: int, lse: int | None, dx: int | None,
             dw: int | None, workspace: int, ws_bytes: int, stream: int = 0) -> None:
    _check(_lib.xent_run(plan, x, w, target, dloss, loss, lse, dx, dw, workspace, ws_bytes, stream), "xent_run")


def xent_plan_destroy(plan: int) -> None:
    _check(_lib.xent_plan_destroy(plan), "xent_plan_destroy")


# ---------------------------------------------------------------------------
# torch conveniences: build descriptors from tensor shapes/strides, keep plans,
# launch on torch's current stream.
# ---------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def _workspace(device, need: int):
    """Scratch of one call (None where it needs none), from torch's allocator on
    the current stream.  Never kept for the next call: the library lets go of
    the interpreter lock, so another thread's launches may fall between this
    call's on the same stream; and what a call allocates under graph capture
    stays with that graph's pool for as long as the graph can be replayed."""
    torch = _torch()
    return torch.empty(need, dtype=torch.uint8, device=device) if need else None


def _ptr(t):
    return None if t is None else t.data_ptr()


def _dtype_code(dt) -> int:
    torch = _torch()
    if dt == torch.bfloat16:
        return LL_BF16
    if dt == torch.float32:
        return LL_F32
    if dt == torch.float16:
        return LL_F16
    raise TypeError(f"unsupported dtype {dt}")


class GemmPlan:
    """Owns one gemm_plan.  A run on torch's current stream takes its workspace
    (packed copies, split-K partials) from torch's allocator for that call; one
    on a stream given by its handle, and callers of the raw C-ABI mirrors, use
    buffers the plan keeps on its device, one per stream and host thread: the
    C ABI asks concurrent runs for distinct workspaces."""

    def __init__(self, desc: GemmDesc, device):
        self.desc = desc
        self.handle = gemm_plan_create(desc)
        self.ws_bytes = gemm_plan_workspace_size(self.handle)
        self.device = device
        self._ws = {}

    @property
    def workspace(self):
        """The kept buffer of the current stream and thread."""
        return self.workspace_for(_torch().cuda.current_stream(self.device).cuda_stream)

    def workspace_for(self, stream: int):
        key = (stream, threading.get_ident())
        ws = self._ws.get(key)
        if ws is None:
            ws = _torch().empty(max(self.ws_bytes, 1), dtype=_torch().uint8, device=self.device)
            self._ws[key] = ws
        return ws

    def describe(self) -> str:
        return gemm_plan_describe(self.handle)

    def run(self, A, B, C, stream: int | None = None, bias=None) -> None:
        if stream is None:
            stream = _torch().cuda.current_stream(A.device).cuda_stream
            ws = _workspace(self.device, self.ws_bytes)
        else:
            ws = self.workspace_for(stream)
        if bias is not None or (self.desc.epilogue & LL_EPI_BIAS):
            gemm_run_ex(self.handle, A.data_ptr(), B.data_ptr(), C.data_ptr(),
                        bias.data_ptr() if bias is not None else None, _ptr(ws), self.ws_bytes, stream)
        else:
            gemm_run(self.handle, A.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(ws), self.ws_bytes, stream)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h and _lib is not None:  # _lib is None once the interpreter tears the module down
            _lib.gemm_plan_destroy(h)
            self.handle = None


_plans: dict = {}


def gemm_desc_for(A, B, C, flags: int = 0, epilogue: int = 0) -> GemmDesc:
    M, K = A.shape
    K2, N = B.shape
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, C {tuple(C.shape)}")
    sa, sb, sc = A.stride(), B.stride(), C.stride()
    return GemmDesc(M, N, K, sa[0], sa[1], sb[0], sb[1], sc[0], sc[1],
                    _dtype_code(A.dtype), _dtype_code(B.dtype), _dtype_code(C.dtype), flags, epilogue)


def plan_for(A, B, C, flags: int = 0, epilogue: int = 0) -> GemmPlan:
    desc = gemm_desc_for(A, B, C, flags, epilogue)
    key = (A.device.index, tuple(getattr(desc, f) for f, _ in GemmDesc._fields_))
    plan = _plans.get(key)
    if plan is None:
        plan = GemmPlan(desc, A.device)
        _plans[key] = plan
    return plan


def gemm(A, B, out=None, out_dtype=None, flags: int = 0, bias=None, act=None):
    """C = act(A @ B + bias) for 2-D bf16 (or both fp16) CUDA (HIP) tensors with
    any row/column-major strides; C is bf16 (default), fp16 or fp32.  bias:
    optional fp32 [N]; act: None, "relu", "gelu" (exact) or "silu", applied
    to the fp32 sums in the GEMM's epilogue."""
    torch = _torch()
    if out is None:
        out = torch.empty((A.shape[0], B.shape[1]), dtype=out_dtype or torch.bfloat16, device=A.device)
    epilogue = ACTIVATIONS[act]
    if bias is not None:
        if bias.dtype != torch.float32 or tuple(bias.shape) != (B.shape[1],) or not bias.is_contiguous():
            raise ValueError("bias must be a contiguous fp32 tensor of N values")
        epilogue |= LL_EPI_BIAS
    plan_for(A, B, out, flags, epilogue).run(A, B, out, bias=bias)
    return out


def _lc_epilogue(bias, act, Mo) -> int:
    torch = _torch()
    epilogue = ACTIVATIONS[act]
    if bias is not None:
        if bias.dtype != torch.float32 or tuple(bias.shape) != (Mo,) or not bias.is_contiguous():
            raise ValueError("bias must be a contiguous fp32 tensor of Mo values")
        epilogue |= LL_EPI_BIAS
    return epilogue


def lincomp_desc_for(user, item, W, Y, flags: int = 0, epilogue: int = 0) -> LincompDesc:
    """user is [R][Nu][D] (one block per request) or [R][C][Nu][D] (rows per
    candidate, e.g. the first Nu rows of a materialised input)."""
    R2, C, Ni, D2 = item.shape
    if user.dim() == 4:
        if user.shape[1] != C:
            raise ValueError("lincomp shape mismatch")
        R, _, Nu, D = user.shape
        su_r, su_c, su_n = user.stride(0), user.stride(1), user.stride(2)
    else:
        R, Nu, D = user.shape
        su_r, su_c, su_n = user.stride(0), 0, user.stride(1)
    Nin, Mo = W.shape
    if R2 != R or D2 != D or Nin != Nu + Ni or tuple(Y.shape) != (R, C, Mo, D):
        raise ValueError("lincomp shape mismatch")
    for t in (user, item, W, Y):
        if t.stride(-1) != 1:
            raise ValueError("last dimension must be contiguous")
    si, sw, sy = item.stride(), W.stride(), Y.stride()
    return LincompDesc(R, C, Nu, Ni, D, Mo, su_r, su_c, su_n, si[0], si[1], si[2], sw[0],
                       sy[0], sy[1], sy[2], _dtype_code(Y.dtype), flags, epilogue)


def lincomp(user, item, W, out=None, out_dtype=None, flags: int = 0, bias=None, act=None):
    """Y[r, c] = act(W^T . [user[r]; item[r, c]] + bias) for bf16 tensors user
    [R][Nu][D] (or [R][C][Nu][D], rows per candidate), item [R][C][Ni][D], W
    [Nu+Ni][Mo]; returns Y [R][C][Mo][D].  bias: optional fp32 [Mo], one per
    compressed row; act: None, "relu", "gelu" (exact) or "silu", applied to
    the fp32 sums before they are rounded."""
    torch = _torch()
    R, D = user.shape[0], user.shape[-1]
    C = item.shape[1]
    Mo = W.shape[1]
    if out is None:
        out = torch.empty((R, C, Mo, D), dtype=out_dtype or torch.bfloat16, device=user.device)
    desc = lincomp_desc_for(user, item, W, out, flags, _lc_epilogue(bias, act, Mo))
    need = lincomp_workspace_size(desc)
    ws = _workspace(user.device, need)
    stream = torch.cuda.current_stream(user.device).cuda_stream
    lincomp_run_ex(desc, user.data_ptr(), item.data_ptr(), W.data_ptr(),
                   bias.data_ptr() if bias is not None else None, out.data_ptr(), _ptr(ws), need, stream)
    return out



def lincomp_stacked(X, W, Nu: int, out=None, out_dtype=None, bias=None, act=None):
    """The layer's original form: X [R][C][Nu+Ni][D] holds every candidate's
    stacked input [user rows; item rows] in full.  Y[r, c] = act(W^T . X[r, c]
    + bias); each candidate computes its user rows' contribution itself."""
    return lincomp(X[:, :, :Nu], X[:, :, Nu:], W, out=out, out_dtype=out_dtype, bias=bias, act=act)


def lincomp_ragged(user, item, W, offsets, out=None, out_dtype=None, flags: int = 0, bias=None, act=None):
    """Ragged requests: user [R][Nu][D], item [Ctot][Ni][D], W [Nu+Ni][Mo] (bf16),
    offsets int64 [R+1] on the device (request r owns candidates
    offsets[r] .. offsets[r+1]-1); returns Y [Ctot][Mo][D]."""
    torch = _torch()
    R, Nu, D = user.shape
    Ctot, Ni, D2 = item.shape
    Nin, Mo = W.shape
    if D2 != D or Nin != Nu + Ni or tuple(offsets.shape) != (R + 1,) or offsets.dtype != torch.int64:
        raise ValueError("lincomp_ragged shape mismatch")
    if out is None:
        out = torch.empty((Ctot, Mo, D), dtype=out_dtype or torch.bfloat16, device=user.device)
    if tuple(out.shape) != (Ctot, Mo, D):
        raise ValueError("lincomp_ragged output shape mismatch")
    for t in (user, item, W, out):
        if t.stride(-1) != 1:
            raise ValueError("last dimension must be contiguous")
    if not offsets.is_contiguous():
        raise ValueError("offsets must be contiguous")
    su, si, sw, sy = user.stride(), item.stride(), W.stride(), out.stride()
    desc = LincompRaggedDesc(R, Ctot, Nu, Ni, D, Mo, su[0], su[1], si[0], si[1], sw[0], sy[0], sy[1],
                             _dtype_code(out.dtype), flags, _lc_epilogue(bias, act, Mo))
    stream = torch.cuda.current_stream(user.device).cuda_stream
    lincomp_ragged_run_ex(desc, offsets.data_ptr(), user.data_ptr(), item.data_ptr(), W.data_ptr(),
                          bias.data_ptr() if bias is not None else None, out.data_ptr(), stream)
    return out


# ---------------------------------------------------------------------------
# Operators around the linear layers.
# ---------------------------------------------------------------------------

def _stream_of(t):
    if not t.is_cuda:
        raise ValueError("tensors must be on a GPU")
    C, device = _torch()._C, t.get_device()
    if device != C._cuda_getDevice():  # the library launches on the current device, whatever the pointers
        raise ValueError(f"tensors on cuda:{device}, but the current device is cuda:{C._cuda_getDevice()}")
    # torch.cuda.current_stream() builds a Stream object for the same value (1.9 us, as long as some of the kernels)
    return C._cuda_getCurrentRawStream(device)


def _rows(t, what: str):
    """Row stride of a 2-D tensor whose last dimension is contiguous (one of a
    single row or column may have any stride)."""
    if t.dim() != 2:
        raise ValueError(f"{what} must be 2-D")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: last dimension must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _vector(t, n: int, what: str, dtypes):
    if tuple(t.shape) != (n,) or t.dtype not in dtypes or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{what} must be a contiguous tensor of {n} values ({', '.join(map(str, dtypes))})")


def _same_device(*ts) -> None:
    dev = ts[0].device
    for t in ts[1:]:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on different devices: {dev}, {t.device}")


def embedding(table, ids, scale: float = 1.0, out=None):
    """out[t] = scale * table[ids[t]] for table [V][D] (bf16, fp16 or fp32, any row
    stride) and int64 ids [T]; an id outside [0, V) gives a row of zeros."""
    torch = _torch()
    _vector(ids, ids.numel(), "ids", (torch.int64,))
    (V, D), T = table.shape, ids.shape[0]
    if out is None:
        out = table.new_empty((T, D))
    if tuple(out.shape) != (T, D) or out.dtype != table.dtype:
        raise ValueError("out must be [T][D] of the table's type")
    _same_device(table, ids, out)
    desc = EmbedDesc(V, T, D, _rows(table, "table"), _rows(out, "out"), _dtype_code(table.dtype), scale)
    embed_run(desc, table.data_ptr(), ids.data_ptr(), out.data_ptr(), _stream_of(table))
    return out


def embedding_grad(ids, dout, rows: int, scale: float = 1.0, padding_idx: int | None = None, out=None,
                   accumulate: bool = False):
    """Dense gradient of ``embedding`` with respect to a table of ``rows`` rows:
    scale times the sum of dout's rows per id.  Tokens with padding_idx or an id
    outside the table contribute nothing.  accumulate: add to ``out``."""
    torch = _torch()
    _vector(ids, ids.numel(), "ids", (torch.int64,))
    T, D = dout.shape
    if ids.shape[0] != T:
        raise ValueError("ids and dout differ in length")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = dout.new_empty((rows, D))
    if tuple(out.shape) != (rows, D) or out.dtype != dout.dtype:
        raise ValueError("out must be [rows][D] of dout's type")
    if padding_idx is not None and padding_idx < 0:
        raise ValueError("padding_idx must not be negative")
    _same_device(dout, ids, out)
    desc = EmbedGradDesc(rows, T, D, _rows(dout, "dout"), _rows(out, "out"), -1 if padding_idx is None else padding_idx,
                         _dtype_code(dout.dtype), scale, LL_EMBED_ACCUMULATE if accumulate else 0)
    stream = _stream_of(dout)
    need = embed_grad_workspace_size(desc)
    ws = _workspace(dout.device, need)
    embed_grad_run(desc, ids.data_ptr(), dout.data_ptr(), out.data_ptr(), _ptr(ws), need, stream)
    return out


def _norm_params(x, *params):
    """param_type of gamma and beta (None: ones, zeros)."""
    given = [p for p in params if p is not None]
    for p in given:
        _vector(p, x.shape[1], "gamma and beta", (x.dtype, _torch().float32))
        if p.dtype != given[0].dtype:
            raise ValueError("gamma and beta must have one type")
    return given[0].dtype if given else x.dtype


def layernorm(x, gamma=None, beta=None, eps: float = 1e-5, out=None):
    """y = (x - mean) * rstd * gamma + beta over the rows of x [N][D] (bf16, fp16 or
    fp32, any row stride); gamma, beta [D] of x's type or fp32, or None.  Returns
    (y, mean, rstd), the latter fp32 [N], which layernorm_grad takes."""
    torch = _torch()
    N, D = x.shape
    if out is None:
        out = x.new_empty((N, D))
    if tuple(out.shape) != (N, D) or out.dtype != x.dtype:
        raise ValueError("out must be [N][D] of x's type")
    ptype = _norm_params(x, gamma, beta)
    _same_device(x, gamma, beta, out)
    mean, rstd = torch.empty((2, N), dtype=torch.float32, device=x.device).unbind(0)
    desc = LayernormDesc(N, D, _rows(x, "x"), _rows(out, "out"), _dtype_code(x.dtype), _dtype_code(ptype), eps)
    layernorm_run(desc, x.data_ptr(), _ptr(gamma), _ptr(beta), out.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                  _stream_of(x))
    return out, mean, rstd


def layernorm_grad(dy, x, mean, rstd, gamma=None, out=None, param_grads: bool = True):
    """(dx, dgamma, dbeta) of ``layernorm`` from its input and the mean and rstd it
    returned.  dgamma and dbeta have gamma's type (x's without gamma);
    param_grads=False: dx alone, the others None."""
    torch = _torch()
    N, D = x.shape
    if tuple(dy.shape) != (N, D) or dy.dtype != x.dtype:
        raise ValueError("dy must have x's shape and type")
    if out is None:
        out = x.new_empty((N, D))
    if tuple(out.shape) != (N, D) or out.dtype != x.dtype:
        raise ValueError("out must be [N][D] of x's type")
    for t in (mean, rstd):
        _vector(t, N, "mean and rstd", (torch.float32,))
    ptype = _norm_params(x, gamma)
    _same_device(x, dy, mean, rstd, gamma, out)
    dgamma, dbeta = torch.empty((2, D), dtype=ptype, device=x.device).unbind(0) if param_grads else (None, None)
    desc = LayernormGradDesc(N, D, _rows(dy, "dy"), _rows(x, "x"), _rows(out, "out"), _dtype_code(x.dtype),
                             _dtype_code(ptype))
    stream = _stream_of(x)
    need = layernorm_grad_workspace_size(desc) if param_grads else 0
    ws = _workspace(x.device, need)
    layernorm_grad_run(desc, dy.data_ptr(), x.data_ptr(), _ptr(gamma), mean.data_ptr(), rstd.data_ptr(),
                       out.data_ptr(), _ptr(dgamma), _ptr(dbeta), _ptr(ws), need, stream)
    return out, dgamma, dbeta


class XentPlan:
    """Owns one xent_plan."""

    def __init__(self, desc: XentDesc):
        self.desc = desc
        self.handle = xent_plan_create(desc)
        self.ws_bytes = xent_plan_workspace_size(self.handle)

    def describe(self) -> str:
        return xent_plan_describe(self.handle)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h and _lib is not None:  # _lib is None once the interpreter tears the module down
            _lib.xent_plan_destroy(h)
            self.handle = None


# The plans of the latest sizes: a program whose batches differ in rows asks for a
# plan per row count, and a plan is needed for its own launches alone.
_XENT_PLANS = 256
_xent_plans: collections.OrderedDict = collections.OrderedDict()


def xent_plan_for(x, w, dx=None, dw=None, ignore_index: int = -100, piece_bytes: int = 0) -> XentPlan:
    """The plan for these tensors' sizes, strides and types (the latest are kept)."""
    N, D = x.shape
    V = w.shape[0]
    if w.shape[1] != D or w.dtype != x.dtype:
        raise ValueError("w must be [V][D] of x's type")
    code = _dtype_code(x.dtype)
    flags = (LL_XENT_DX if dx is not None else 0) | (LL_XENT_DW if dw is not None else 0)
    if w.data_ptr() % 16:
        flags |= LL_XENT_PACK_W
    key = (x.device.index, N, V, D, _rows(x, "x"), _rows(w, "w"), _rows(dx, "dx") if dx is not None else 0,
           _rows(dw, "dw") if dw is not None else 0, ignore_index, piece_bytes, code,
           _dtype_code(dx.dtype) if dx is not None else code, _dtype_code(dw.dtype) if dw is not None else code, flags)
    plan = _xent_plans.pop(key, None) or XentPlan(XentDesc(*key[1:]))
    _xent_plans[key] = plan  # the newest
    while len(_xent_plans) > _XENT_PLANS:
        try:
            _xent_plans.popitem(last=False)
        except KeyError:  # emptied by another thread
            break
    return plan


def _xent(x, w, target, dloss, dx, dw, ignore_index, piece_bytes):
    torch = _torch()
    N = x.shape[0]
    stream = _stream_of(x)
    plan = xent_plan_for(x, w, dx, dw, ignore_index, piece_bytes)
    _vector(target, N, "target", (torch.int64,))
    _same_device(x, w, target, dloss, dx, dw)
    loss, lse = torch.empty((2, N), dtype=torch.float32, device=x.device).unbind(0)
    ws = _workspace(x.device, plan.ws_bytes)
    xent_run(plan.handle, x.data_ptr(), w.data_ptr(), target.data_ptr(), _ptr(dloss), loss.data_ptr(), lse.data_ptr(),
             _ptr(dx), _ptr(dw), _ptr(ws), plan.ws_bytes, stream)
    return loss, lse


def vocab_xent(x, w, target, ignore_index: int = -100, piece_bytes: int = 0):
    """Softmax cross entropy of rows x [N][D] against the vocabulary w [V][D] (both
    bf16 or fp16, any row stride): (loss, lse), fp32 [N] each, without the
    [N][V] logits.  target: int64 [N]; ignore_index, or one outside [0, V):
    loss and lse are 0.  piece_bytes: bound of the buffers that hold a piece of
    the logits (0: 2 GiB)."""
    return _xent(x, w, target, None, None, None, ignore_index, piece_bytes)


def vocab_xent_grad(x, w, target, dloss, ignore_index: int = -100, piece_bytes: int = 0, dx=None, dw=None,
                    want_dx: bool = True, want_dw: bool = True):
    """(loss, lse, dx, dw): ``vocab_xent`` with the gradients of sum(dloss * loss)
    for fp32 dloss [N].  dx [N][D] and dw [V][D] may be given (of x's type or
    fp32); want_dx / want_dw=False: that gradient is not formed (None)."""
    torch = _torch()
    _vector(dloss, x.shape[0], "dloss", (torch.float32,))
    if want_dx and dx is None:
        dx = x.new_empty(x.shape)
    if want_dw and dw is None:
        dw = w.new_empty(w.shape)
    dx, dw = dx if want_dx else None, dw if want_dw else None
    for t, like, what in ((dx, x, "dx"), (dw, w, "dw")):
        if t is not None and (t.shape != like.shape or t.dtype not in (like.dtype, torch.float32)):
            raise ValueError(f"{what} must have its operand's shape, and its type or fp32")
    loss, lse = _xent(x, w, target, dloss, dx, dw, ignore_index, piece_bytes)
    return loss, lse, dx, dw
