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
LL_BF16, LL_F32, LL_F16, LL_E4M3, LL_E5M2 = 0, 1, 2, 3, 4
LL_EPI_BIAS, LL_EPI_RELU, LL_EPI_GELU, LL_EPI_SILU = 0x1, 0x10, 0x20, 0x30
ACTIVATIONS = {None: 0, "relu": LL_EPI_RELU, "gelu": LL_EPI_GELU, "silu": LL_EPI_SILU}
LL_GEMM8_FULL_SUMS = 0x1
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


class RmsnormDesc(ctypes.Structure):
    _fields_ = [("N", _i64), ("D", _i64),
                ("stride_x", _i64), ("stride_residual", _i64), ("stride_h", _i64), ("stride_y", _i64),
                ("stride_sn", _i64), ("stride_sb", _i64),
                ("type", ctypes.c_int32), ("param_type", ctypes.c_int32), ("y_type", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class RmsnormGradDesc(ctypes.Structure):
    _fields_ = [("N", _i64), ("D", _i64),
                ("stride_dy", _i64), ("stride_h", _i64), ("stride_dh", _i64), ("stride_dx", _i64),
                ("type", ctypes.c_int32), ("param_type", ctypes.c_int32)]


class Quant8Desc(ctypes.Structure):
    _fields_ = [("N", _i64), ("D", _i64), ("stride_x", _i64), ("stride_q", _i64), ("stride_qt", _i64),
                ("stride_sn", _i64), ("stride_sb", _i64), ("stride_tn", _i64), ("stride_tb", _i64),
                ("type", ctypes.c_int32), ("q_type", ctypes.c_int32), ("block", ctypes.c_int32)]


class Gemm8Desc(ctypes.Structure):
    _fields_ = [("M", _i64), ("N", _i64), ("K", _i64),
                ("stride_a", _i64), ("stride_b", _i64), ("stride_c", _i64),
                ("stride_am", _i64), ("stride_ab", _i64), ("stride_bn", _i64), ("stride_bb", _i64),
                ("a_type", ctypes.c_int32), ("b_type", ctypes.c_int32), ("c_type", ctypes.c_int32),
                ("b_block", ctypes.c_int32), ("flags", ctypes.c_uint32)]


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
_lib.rmsnorm_run.argtypes = [ctypes.POINTER(RmsnormDesc), *[_vp] * 8]
_lib.rmsnorm_grad_workspace_size.argtypes = [ctypes.POINTER(RmsnormGradDesc), ctypes.POINTER(ctypes.c_size_t)]
_lib.rmsnorm_grad_run.argtypes = [ctypes.POINTER(RmsnormGradDesc), *[_vp] * 8, ctypes.c_size_t, _vp]
_lib.quant8_run.argtypes = [ctypes.POINTER(Quant8Desc), *[_vp] * 6]
_lib.gemm8_workspace_size.argtypes = [ctypes.POINTER(Gemm8Desc), ctypes.POINTER(ctypes.c_size_t)]
_lib.gemm8_describe.argtypes = [ctypes.POINTER(Gemm8Desc), ctypes.c_char_p, ctypes.c_size_t]
_lib.gemm8_run.argtypes = [ctypes.POINTER(Gemm8Desc), *[_vp] * 6, ctypes.c_size_t, _vp]
for _f in ("gemm_plan_create", "gemm_plan_workspace_size", "gemm_plan_describe", "gemm_run", "gemm_run_ex",
           "gemm_run_noalloc", "gemm_plan_destroy", "lincomp_workspace_size", "lincomp_run", "lincomp_ragged_run",
           "lincomp_run_ex", "lincomp_ragged_run_ex", "embed_run", "embed_grad_workspace_size", "embed_grad_run",
           "layernorm_run", "layernorm_grad_workspace_size", "layernorm_grad_run", "xent_plan_create",
           "xent_plan_workspace_size", "xent_plan_describe", "xent_run", "xent_plan_destroy", "rmsnorm_run",
           "rmsnorm_grad_workspace_size", "rmsnorm_grad_run", "quant8_run", "gemm8_workspace_size", "gemm8_describe",
           "gemm8_run"):
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


def rmsnorm_run(desc: RmsnormDesc, x: int, residual: int | None, gamma: int | None, h: int | None, y: int,
                scale: int | None, rstd: int | None, stream: int = 0) -> None:
    _check(_lib.rmsnorm_run(ctypes.byref(desc), x, residual, gamma, h, y, scale, rstd, stream), "rmsnorm_run")


def rmsnorm_grad_workspace_size(desc: RmsnormGradDesc) -> int:
    n = ctypes.c_size_t()
    _check(_lib.rmsnorm_grad_workspace_size(ctypes.byref(desc), ctypes.byref(n)), "rmsnorm_grad_workspace_size")
    return n.value


def rmsnorm_grad_run(desc: RmsnormGradDesc, dy: int, h: int, gamma: int | None, rstd: int, dh: int | None, dx: int,
                     dgamma: int | None, workspace: int, ws_bytes: int, stream: int = 0) -> None:
    _check(_lib.rmsnorm_grad_run(ctypes.byref(desc), dy, h, gamma, rstd, dh, dx, dgamma, workspace, ws_bytes, stream),
           "rmsnorm_grad_run")


def quant8_run(desc: Quant8Desc, x: int, q: int | None, scale: int | None, qt: int | None, scale_t: int | None,
               stream: int = 0) -> None:
    _check(_lib.quant8_run(ctypes.byref(desc), x, q, scale, qt, scale_t, stream), "quant8_run")


def gemm8_workspace_size(desc: Gemm8Desc) -> int:
    n = ctypes.c_size_t()
    _check(_lib.gemm8_workspace_size(ctypes.byref(desc), ctypes.byref(n)), "gemm8_workspace_size")
    return n.value


def gemm8_describe(desc: Gemm8Desc) -> str:
    buf = ctypes.create_string_buffer(512)
    _check(_lib.gemm8_describe(ctypes.byref(desc), buf, 512), "gemm8_describe")
    return buf.value.decode()


def gemm8_run(desc: Gemm8Desc, A: int, a_scale: int, B: int, b_scale: int, C: int, workspace: int, ws_bytes: int,
              stream: int = 0) -> None:
    _check(_lib.gemm8_run(ctypes.byref(desc), A, a_scale, B, b_scale, C, workspace, ws_bytes, stream), "gemm8_run")


# ---------------------------------------------------------------------------
# torch conveniences: build descriptors from tensor shapes/strides, keep plans,
# launch on torch's current stream.
# ---------------------------------------------------------------------------

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:  # asked for several times a call: the import statement alone takes 0.3 us
        import torch
        _torch_module = torch
    return _torch_module


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


_dtype_codes: dict = {}


def _dtype_code(dt) -> int:
    if not _dtype_codes:
        torch = _torch()
        _dtype_codes.update({torch.bfloat16: LL_BF16, torch.float32: LL_F32, torch.float16: LL_F16})
    code = _dtype_codes.get(dt)
    if code is None:
        raise TypeError(f"unsupported dtype {dt}")
    return code


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
    strides = t.stride()
    if len(strides) != 2:
        raise ValueError(f"{what} must be 2-D")
    n, m = t.shape
    if m > 1 and strides[1] != 1:
        raise ValueError(f"{what}: last dimension must be contiguous")
    return strides[0] if n > 1 else max(strides[0], m)


def _vector(t, n: int, what: str, dtypes):
    if t.shape != (n,) or t.dtype not in dtypes or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{what} must be a contiguous tensor of {n} values ({', '.join(map(str, dtypes))})")


def _same_device(*ts) -> None:
    dev = ts[0].get_device()
    for t in ts:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on different devices: {ts[0].device}, {t.device}")


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
    first = None
    for p in params:
        if p is not None:
            _vector(p, x.shape[1], "gamma and beta", (x.dtype, _torch().float32))
            if first is None:
                first = p.dtype
            elif p.dtype != first:
                raise ValueError("gamma and beta must have one type")
    return x.dtype if first is None else first


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


# ---------------------------------------------------------------------------
# Linear layers in 8 bits.
# ---------------------------------------------------------------------------

_codes8: dict = {}


def _code8(dtype) -> int:
    if not _codes8:
        torch = _torch()
        _codes8.update({torch.float8_e4m3fn: LL_E4M3, torch.float8_e5m2: LL_E5M2})
    code = _codes8.get(dtype)
    if code is None:
        raise TypeError(f"unsupported 8-bit dtype {dtype} (float8_e4m3fn or float8_e5m2)")
    return code


def _blocks8(n: int) -> int:
    return -(-n // 128)


def _new8(like, rows: int, cols: int, dtype):
    """([rows][cols], row stride) in rows of a multiple of 16 bytes, as gemm8 takes them."""
    ld = -(-cols // 16) * 16
    t = like.new_empty((rows, ld), dtype=dtype)
    return (t if ld == cols else t[:, :cols]), ld


def _new_scale8(like, rows: int, cols: int, squares: bool):
    """(scales [rows][blocks of cols], their strides); row scales with the rows of one block next to each other."""
    f32, blocks = _torch().float32, _blocks8(cols)
    if squares:
        return like.new_empty((_blocks8(rows), blocks), dtype=f32), max(blocks, 1), 1
    if rows == 1:
        return like.new_empty((1, blocks), dtype=f32), 1, 1
    return like.new_empty((blocks, rows), dtype=f32).t(), 1, max(rows, 1)


def _scale_strides(t, shape, what: str):
    """Strides of 2-D fp32 scales; along a dimension of one they do not matter."""
    strides = t.stride()
    if len(strides) != 2 or t.dtype != _torch().float32:
        raise ValueError(f"{what} must be 2-D and fp32")
    return strides[0] if shape[0] > 1 else 1, strides[1] if shape[1] > 1 else 1


def _rmsnorm(x, gamma, residual, eps, y, ld_y, y_code, scale, sn, sb, residual_out):
    shape, dtype = x.shape, x.dtype
    N, D = shape
    code = _dtype_code(dtype)
    pcode = code if gamma is None else _dtype_code(_norm_params(x, gamma))
    h, ld_r, ld_h = None, 0, 0
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs a residual")
    else:
        if residual.shape != shape or residual.dtype != dtype:
            raise ValueError("residual must have x's shape and type")
        ld_r = _rows(residual, "residual")
        if residual_out is None:
            h, ld_h = _torch().empty_like(x), D
        else:
            h = residual_out
            if h.shape != shape or h.dtype != dtype:
                raise ValueError("residual_out must have x's shape and type")
            ld_h = _rows(h, "residual_out")
    _same_device(x, gamma, residual, h, y)
    stream = _stream_of(x)
    rstd = x.new_empty(N, dtype=_torch().float32)
    desc = RmsnormDesc(N, D, _rows(x, "x"), ld_r, ld_h, ld_y, sn, sb, code, pcode, code if y_code is None else y_code,
                       eps)
    rmsnorm_run(desc, x.data_ptr(), _ptr(residual), _ptr(gamma), _ptr(h), y.data_ptr(), _ptr(scale), rstd.data_ptr(),
                stream)
    return x if h is None else h, rstd


def rmsnorm(x, gamma=None, residual=None, eps: float = 1e-6, out=None, residual_out=None):
    """(y, h, rstd): h = x + residual (x itself without a residual), rounded to x's
    type, and y = h * rstd * gamma with rstd = 1 / sqrt(mean(h^2) + eps) over the
    rows of x [N][D] (bf16, fp16 or fp32, any row stride).  gamma [D] of x's type
    or fp32, or None.  residual_out: where h goes, may be residual or x.  h and
    rstd (fp32 [N]) are what rmsnorm_grad takes; out may be x without a residual,
    whose values (h) are then gone."""
    if out is None:
        out = x.new_empty(x.shape)
    elif out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError("out must have x's shape and type")
    h, rstd = _rmsnorm(x, gamma, residual, eps, out, _rows(out, "out"), None, None, 1, 1, residual_out)
    return out, h, rstd


def rmsnorm8(x, gamma=None, residual=None, eps: float = 1e-6, dtype=None, residual_out=None):
    """(q, scale, h, rstd): ``rmsnorm`` with y quantised in blocks of 128 of a row,
    as gemm8's first operand: q [N][D] of dtype (float8_e4m3fn by default, or
    float8_e5m2), scale fp32 [N][blocks]."""
    dtype = dtype or _torch().float8_e4m3fn
    code = _code8(dtype)
    N, D = x.shape
    q, ld = _new8(x, N, D, dtype)
    scale, sn, sb = _new_scale8(x, N, D, False)
    h, rstd = _rmsnorm(x, gamma, residual, eps, q, ld, code, scale, sn, sb, residual_out)
    return q, scale, h, rstd


def rmsnorm_grad(dy, h, rstd, gamma=None, dh=None, out=None, param_grads: bool = True):
    """(dx, dgamma) of ``rmsnorm`` from the h and rstd it returned.  dx is the
    gradient of h, and so of x and of the residual alike; dh: the gradient that
    reaches h by its other path, added to dx (out may be dh).  dgamma has gamma's
    type (h's without gamma); param_grads=False: dx alone, dgamma None."""
    shape, dtype = h.shape, h.dtype
    N, D = shape
    if dy.shape != shape or dy.dtype != dtype:
        raise ValueError("dy must have h's shape and type")
    if dh is not None and (dh.shape != shape or dh.dtype != dtype):
        raise ValueError("dh must have h's shape and type")
    if out is None:
        out, ld_out = h.new_empty(shape), D
    else:
        if out.shape != shape or out.dtype != dtype:
            raise ValueError("out must be [N][D] of h's type")
        ld_out = _rows(out, "out")
    _vector(rstd, N, "rstd", (_torch().float32,))
    ptype = _norm_params(h, gamma)
    _same_device(h, dy, rstd, gamma, dh, out)
    stream = _stream_of(h)
    dgamma = h.new_empty(D, dtype=ptype) if param_grads else None
    desc = RmsnormGradDesc(N, D, _rows(dy, "dy"), _rows(h, "h"), 0 if dh is None else _rows(dh, "dh"), ld_out,
                           _dtype_code(dtype), _dtype_code(ptype))
    need = rmsnorm_grad_workspace_size(desc) if param_grads else 0
    ws = _workspace(h.device, need)
    rmsnorm_grad_run(desc, dy.data_ptr(), h.data_ptr(), _ptr(gamma), rstd.data_ptr(), _ptr(dh), out.data_ptr(),
                     _ptr(dgamma), _ptr(ws), need, stream)
    return out, dgamma


def _quant8(x, squares, dtype, plain, transposed):
    dtype = dtype or _torch().float8_e4m3fn
    code = _code8(dtype)
    N, D = x.shape
    stream = _stream_of(x)
    q = s = qt = st = None
    qs, qts, sn, sb, tn, tb = 0, 0, 1, 1, 1, 1
    if plain:
        q, qs = _new8(x, N, D, dtype)
        s, sn, sb = _new_scale8(x, N, D, squares)
    if transposed:
        qt, qts = _new8(x, D, N, dtype)
        st, tn, tb = _new_scale8(x, D, N, squares)
    desc = Quant8Desc(N, D, _rows(x, "x"), qs, qts, sn, sb, tn, tb, _dtype_code(x.dtype), code, 128 if squares else 1)
    quant8_run(desc, x.data_ptr(), _ptr(q), _ptr(s), _ptr(qt), _ptr(st), stream)
    return q, s, qt, st


def quant8(x, squares: bool = False, transpose: bool = False, dtype=None):
    """(q, scale): x [N][D] (bf16, fp16 or fp32, any row stride) in 8 bits (dtype:
    float8_e4m3fn by default, or float8_e5m2) with an fp32 scale for each block: 128
    consecutive values of a row (scale [N][blocks of D]: what gemm8 takes as its
    first operand), or squares of 128 x 128 (scale [blocks of N][blocks of D]: a
    weight).  transpose: x^T [D][N] instead, the blocks along N.  A value stands
    for q * its block's scale."""
    q, s, qt, st = _quant8(x, squares, dtype, not transpose, transpose)
    return (qt, st) if transpose else (q, s)


def quant8_pair(x, squares: bool = False, dtype=None):
    """(q, scale, qt, scale_t): both forms of ``quant8``, x read once: for a weight,
    the operands of the forward product and of the inputs' gradient; for
    activations and their gradients, of their product and of the weight's gradient."""
    return _quant8(x, squares, dtype, True, True)


def gemm8_desc_for(a, a_scale, b, b_scale, out, full_sums: bool = False) -> Gemm8Desc:
    a_shape, b_shape = a.shape, b.shape
    lda, ldb = _rows16(a, a_shape, "a"), _rows16(b, b_shape, "b")
    M, K = a_shape
    N = b_shape[0]
    if b_shape[1] != K or out.shape != (M, N):
        raise ValueError(f"shape mismatch: a {tuple(a_shape)}, b {tuple(b_shape)}, out {tuple(out.shape)}")
    kb = -(-K // 128)
    sa_shape, sb_shape = a_scale.shape, b_scale.shape
    sam, sab = _scale_strides(a_scale, sa_shape, "a_scale")
    sbn, sbb = _scale_strides(b_scale, sb_shape, "b_scale")
    if sa_shape != (M, kb):
        raise ValueError(f"a_scale must be [{M}][{kb}]")
    squares = sb_shape == (-(-N // 128), kb)
    if not squares and sb_shape != (N, kb):
        raise ValueError(f"b_scale must be [{_blocks8(N)}][{kb}] or [{N}][{kb}]")
    return Gemm8Desc(M, N, K, lda, ldb, _rows(out, "out"), sam, sab, sbn, sbb, _code8(a.dtype), _code8(b.dtype),
                     _dtype_code(out.dtype), 128 if squares else 1, LL_GEMM8_FULL_SUMS if full_sums else 0)


def _rows16(t, shape, what: str):
    """_rows of an operand of gemm8; the stride of a single row, or of empty ones, does not matter."""
    strides = t.stride()
    if len(strides) != 2:
        raise ValueError(f"{what} must be 2-D")
    n, k = shape
    if k > 1 and strides[1] != 1:
        raise ValueError(f"{what}: last dimension must be contiguous")
    return strides[0] if n > 1 and k > 0 else -(-k // 16) * 16


def gemm8(a, a_scale, b, b_scale, out=None, out_dtype=None, full_sums: bool = False):
    """C = A B^T of two quantised matrices, a [M][K] (float8_e4m3fn or float8_e5m2)
    with a_scale [M][blocks of K], and b [N][K] (float8_e4m3fn), a linear layer's
    weight as stored, with b_scale [blocks of N][blocks of K] (squares) or
    [N][blocks of K] (rows), as quant8 and rmsnorm8 give them; rows at multiples of
    16 bytes.  C is bf16 (default), fp16 or fp32.

    An fp32 C has sums of fp32's precision.  Those of a 16-bit C come from the 8-bit
    matrix instruction, twice as fast, which drops from each eight products what lies
    below 2^-13 of the largest: at most 7 * 2^-13 of the sum of the products'
    magnitudes; of the result's norm 1.4e-5 on normally distributed operands and up to
    7e-5 where single columns of a stand far out.  full_sums=True: fp32's precision for
    a 16-bit C too, rounded once, at about an fp32 C's speed."""
    torch = _torch()
    if out is None:
        out = a.new_empty((a.shape[0], b.shape[0]), dtype=out_dtype or torch.bfloat16)
    desc = gemm8_desc_for(a, a_scale, b, b_scale, out, full_sums)
    _same_device(a, a_scale, b, b_scale, out)
    stream = _stream_of(a)
    need = gemm8_workspace_size(desc)
    ws = _workspace(a.device, need)
    gemm8_run(desc, a.data_ptr(), a_scale.data_ptr(), b.data_ptr(), b_scale.data_ptr(), out.data_ptr(), _ptr(ws), need,
              stream)
    return out
