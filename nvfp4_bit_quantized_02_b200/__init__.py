"""Python binding of libnvfp4 (include/nvfp4.h): NVFP4 quantization and block-scaled FP4 GEMMs
for the fprop, dgrad and wgrad GEMMs of a linear layer on a B200 (sm_100a).

Argument marshalling only: every step of the path runs in the CUDA kernels of
``libnvfp4.so``.  PyTorch provides device memory and the current stream.  Importing this
module does not load the library; the first call does, and raises if it is missing -- there is
no CPU fallback.

The functions carry the C names: ``nvfp4_quantize``, ``nvfp4_quantize_dual``,
``nvfp4_quantize_weight``, ``nvfp4_transpose_2d``, ``nvfp4_gemm``, ``nvfp4_linear_fwd``,
``nvfp4_linear_bwd``, ``nvfp4_gelu_fwd``, ``nvfp4_gelu_bwd``, ``nvfp4_poll``, for layers with one weight
per expert ``nvfp4_bf16_gemm_grouped`` and ``nvfp4_bf16_wgrad_grouped``, for the weight update
``nvfp4_adamw_step``, and for data-parallel token shards ``nvfp4_amax``, ``nvfp4_quantize_dual_shard`` (and ``nvfp4_quantize_dual_dp``, which
all-reduces the amax between them).
"""
from __future__ import annotations

import ctypes
import os
from bisect import bisect_left
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4.so")

RNE, SR = 0, 1
BLOCK_1x16, BLOCK_16x16 = 0, 1
OUT_BF16, OUT_FP32 = 0, 1
STREAM_DGRAD, STREAM_WGRAD, STREAM_RHT = 1, 2, 3
STREAM_MOMENT1, STREAM_MOMENT2 = 4, 5
STATE_FP32, STATE_FP8 = 0, 1

STATUS = {0: "OK", 1: "ERR_NULL", 2: "ERR_ALIGN", 3: "ERR_SHAPE", 4: "ERR_ARG", 5: "ERR_WORKSPACE", 6: "ERR_CUDA",
          7: "ERR_NONFINITE", 8: "ERR_TIMEOUT", 9: "ERR_UNSUPPORTED", 10: "ERR_LIMIT"}


class NVFP4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({_lib().nvfp4_status_string(status).decode()})")


class CTensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("tile_scales", ctypes.c_void_p),
                ("tensor_scale", ctypes.c_void_p), ("rows", ctypes.c_int64), ("k", ctypes.c_int64),
                ("block", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class CMXTensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64), ("k", ctypes.c_int64)]


class CLinearCtx(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int64), ("n", ctypes.c_int64), ("rht_seed", ctypes.c_uint64),
                ("xq", CTensor), ("xq_rht", CTensor), ("wq", CTensor), ("wqt", CTensor), ("dyq", CTensor),
                ("dyq_rht", CTensor), ("ws", ctypes.c_void_p), ("w_cached", ctypes.c_int32),
                ("amax_ready", ctypes.c_int32), ("y_amax_ws", ctypes.c_void_p), ("y_rht_seed", ctypes.c_uint64),
                ("dx_amax_ws", ctypes.c_void_p), ("dx_rht_seed", ctypes.c_uint64)]


class CAdamWTensor(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("w", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("amax_ws", ctypes.c_void_p), ("n", ctypes.c_int64), ("g_dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class CAdamWDynamic(ctypes.Structure):
    _fields_ = [("keep", ctypes.c_float), ("step_size", ctypes.c_float), ("v_fix", ctypes.c_float),
                ("grad_scale", ctypes.c_float), ("sr_seed", ctypes.c_uint64), ("reserved", ctypes.c_uint64)]


class CAdamWArgs(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("grad_scale", ctypes.c_double),
                ("step", ctypes.c_int64), ("sr_seed", ctypes.c_uint64), ("state", ctypes.c_int32),
                ("mode", ctypes.c_int32), ("dynamic", ctypes.c_void_p)]


_L = None


def _lib():
    global _L
    if _L is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libnvfp4.so is not built ({LIB_PATH}); run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        c = ctypes
        vp, i64, u64, u32, i32 = c.c_void_p, c.c_int64, c.c_uint64, c.c_uint32, c.c_int
        T = c.POINTER(CTensor)
        sig = {
            "nvfp4_codes_bytes": ([i64, i64], c.c_size_t),
            "nvfp4_scales_bytes": ([i64, i64], c.c_size_t),
            "nvfp4_tile_scales_bytes": ([i64, i64], c.c_size_t),
            "nvfp4_workspace_bytes": ([], c.c_size_t),
            "nvfp4_workspace_init": ([vp, vp], i32),
            "nvfp4_quantize": ([vp, i64, i64, i64, i32, i32, i32, i32, u64, u64, u32, T, vp, vp], i32),
            "nvfp4_quantize_dual": ([vp, i64, i64, i64, i32, u64, u64, u32, u32, T, T, vp, vp], i32),
            "nvfp4_quantize_weight": ([vp, i64, i64, i64, T, T, vp, vp], i32),
            "nvfp4_quantize_weight_ready": ([vp, i64, i64, i64, T, T, vp, vp], i32),
            "nvfp4_bf16_gemm_grouped": ([vp, i64, i64, vp, i32, vp, i64, i64, i32, i64, i64, vp, i64, i32, vp, vp], i32),
            "nvfp4_bf16_wgrad_grouped": ([vp, i64, vp, i64, i64, vp, i32, i64, i64, vp, i64, i64, i32, vp, vp], i32),
            "nvfp4_adamw": ([c.POINTER(CAdamWTensor), i32, c.POINTER(CAdamWArgs), vp, vp], i32),
            "nvfp4_adamw_dynamic_values": ([c.POINTER(CAdamWArgs), c.POINTER(CAdamWDynamic)], i32),
            "nvfp4_amax": ([vp, i64, i64, i64, i32, u64, vp, vp], i32),
            "nvfp4_workspace_amax_offset": ([], c.c_size_t),
            "nvfp4_quantize_dual_shard": ([vp, i64, i64, i64, i64, i64, i32, u64, u64, u32, u32, T, T, vp, vp], i32),
            "nvfp4_transpose_2d": ([T, T, vp], i32),
            "nvfp4_gemm": ([T, T, vp, i64, i32, vp, vp], i32),
            "nvfp4_gemm_reduce_scatter": ([T, T, c.POINTER(vp), i32, i64, i64, vp, vp], i32),
            "nvfp4_gemm_amax": ([T, T, vp, i64, u64, vp, vp, vp], i32),
            "nvfp4_linear_fwd": ([vp, vp, vp, c.POINTER(CLinearCtx), vp], i32),
            "nvfp4_linear_bwd": ([vp, u64, vp, vp, c.POINTER(CLinearCtx), vp], i32),
            "nvfp4_gelu_fwd": ([vp, vp, i64, vp], i32),
            "nvfp4_gelu_bwd": ([vp, vp, vp, i64, vp], i32),
            "nvfp4_gelu_fwd_amax": ([vp, vp, i64, i64, u64, vp, vp], i32),
            "nvfp4_gelu_bwd_amax": ([vp, vp, vp, i64, i64, u64, vp, vp], i32),
            "nvfp4_poll": ([vp, vp], i32),
            "nvfp4_mx_scales_bytes": ([i64, i64], c.c_size_t),
            "nvfp4_bf16_gemm": ([vp, i64, vp, i64, i64, i64, i64, vp, i64, i32, vp, vp], i32),
            "nvfp4_bf16_transpose": ([vp, i64, i64, i64, vp, i64, vp], i32),
            "nvfp4_linear_bf16_scratch_bytes": ([i64, i64, i64], c.c_size_t),
            "nvfp4_linear_bf16_fwd": ([vp, vp, vp, i64, i64, i64, vp, vp], i32),
            "nvfp4_linear_bf16_bwd": ([vp, vp, vp, vp, vp, i64, i64, i64, vp, vp, vp], i32),
            "nvfp4_mx_quantize": ([vp, i64, i64, i64, i32, i32, u64, u32, c.POINTER(CMXTensor), vp, vp], i32),
            "nvfp4_mx_quantize_dual": ([vp, i64, i64, i64, i32, u64, u32, u32, c.POINTER(CMXTensor),
                                        c.POINTER(CMXTensor), vp, vp], i32),
            "nvfp4_mx_gemm": ([c.POINTER(CMXTensor), c.POINTER(CMXTensor), vp, i64, i32, vp, vp], i32),
            "nvfp4_quantize_noalloc": ([vp, i64, i64, i64, i32, i32, i32, i32, u64, u64, u32, T, vp], i32),
            "nvfp4_poll_noalloc": ([vp], i32),
            "nvfp4_set_wait_budget_ns": ([u64], None),
            "nvfp4_status_string": ([i32], c.c_char_p),
            "nvfp4_version": ([], i32),
        }
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _L = L
    return _L


def lib():
    """The loaded ctypes library (raises ImportError if it is not built)."""
    return _lib()


def _check(status: int, what: str):
    if status != 0:
        raise NVFP4Error(status, what)


# the current stream's raw handle without building a Stream object (a tenth of the cost, which
# matters for small calls); the public route where this torch does not offer it
_RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    if _RAW_STREAM is not None:
        return _RAW_STREAM(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


# the current device's index without torch.cuda's initialisation check on every call; the public
# route where this torch does not offer it
_CUR_DEVICE = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# ---------------------------------------------------------------------------------------
# workspace
# ---------------------------------------------------------------------------------------
class Workspace:
    """256 bytes of device memory for amax slots and the sticky device flags."""

    def __init__(self, device=None):
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.buf = torch.empty(_lib().nvfp4_workspace_bytes(), dtype=torch.uint8, device=device)
        _check(_lib().nvfp4_workspace_init(_ptr(self.buf), _stream()), "nvfp4_workspace_init")
        self.addr, self.index = self.buf.data_ptr(), self.buf.get_device()

    @property
    def ptr(self):
        return _ptr(self.buf)

    def amax_words(self) -> torch.Tensor:
        """The two amax words (plain, after the RHT) as an int32 view of the device buffer: fp32
        bit patterns of non-negative values, so an integer MAX reduction is exact."""
        off = _lib().nvfp4_workspace_amax_offset()
        return self.buf[off:off + 8].view(torch.int32)


_DEFAULT_WS = {}


def default_workspace() -> Workspace:
    dev = torch.cuda.current_device()
    if dev not in _DEFAULT_WS:
        _DEFAULT_WS[dev] = Workspace()
    return _DEFAULT_WS[dev]


def nvfp4_poll(ws: Workspace | None = None, stream=None) -> int:
    """Synchronize the stream and return (and clear) the workspace's device status."""
    ws = ws or default_workspace()
    return _lib().nvfp4_poll(ws.ptr, _stream(stream))


def nvfp4_set_wait_budget_ns(ns: int):
    _lib().nvfp4_set_wait_budget_ns(int(ns))


# ---------------------------------------------------------------------------------------
# quantized operand forms
# ---------------------------------------------------------------------------------------
@dataclass
class NVFP4Tensor:
    """One quantized operand form (device buffers owned by torch)."""
    codes: torch.Tensor          # uint8 [rows][k/2]
    scales: torch.Tensor         # uint8, 128x4-tile swizzled E4M3 block scales
    tile_scales: torch.Tensor | None  # uint8 [rows/16][k/16] for 16x16 forms
    tensor_scale: torch.Tensor   # float32 [1]: decode scale s_t
    rows: int
    k: int
    block: int

    @staticmethod
    def empty(rows: int, k: int, block: int = BLOCK_1x16, device=None) -> "NVFP4Tensor":
        L = _lib()
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        codes = torch.empty(max(L.nvfp4_codes_bytes(rows, k), 1), dtype=torch.uint8, device=device)
        scales = torch.empty(max(L.nvfp4_scales_bytes(rows, k), 16), dtype=torch.uint8, device=device)
        tiles = None
        if block == BLOCK_16x16:
            tiles = torch.empty(max(L.nvfp4_tile_scales_bytes(rows, k), 1), dtype=torch.uint8, device=device)
        st = torch.empty(1, dtype=torch.float32, device=device)
        return NVFP4Tensor(codes, scales, tiles, st, rows, k, block)

    def c(self) -> CTensor:
        return CTensor(self.codes.data_ptr(), self.scales.data_ptr(),
                       self.tile_scales.data_ptr() if self.tile_scales is not None else None,
                       self.tensor_scale.data_ptr(), self.rows, self.k, self.block, 0)

    def codes_2d(self) -> torch.Tensor:
        return self.codes[: self.rows * (self.k // 2)].view(self.rows, self.k // 2)


def _bf16_2d(x: torch.Tensor):
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda:
        raise TypeError("expected a 2-D bf16 CUDA tensor")
    if x.stride(1) != 1:
        raise ValueError("inner dimension must be contiguous")
    return x.shape[0], x.shape[1], x.stride(0)


def nvfp4_quantize(x: torch.Tensor, along: int = 0, mode: int = RNE, block: int = BLOCK_1x16, rht: bool = False,
                   rht_seed: int = 0, sr_seed: int = 0, stream_id: int = 0, out: NVFP4Tensor | None = None,
                   ws: Workspace | None = None, stream=None) -> NVFP4Tensor:
    rows, cols, ld = _bf16_2d(x)
    R, K = (cols, rows) if along else (rows, cols)
    out = out or NVFP4Tensor.empty(R, K, block, x.device)
    ws = ws or default_workspace()
    ct = out.c()
    st = _lib().nvfp4_quantize(_ptr(x), rows, cols, ld, along, mode, block, int(rht), rht_seed, sr_seed, stream_id,
                               ctypes.byref(ct), ws.ptr, _stream(stream))
    _check(st, "nvfp4_quantize")
    return out


def nvfp4_quantize_dual(x: torch.Tensor, mode: int = RNE, rht_seed: int = 0, sr_seed: int = 0, stream_row: int = 0,
                        stream_col: int = 0, out_row: NVFP4Tensor | None = None, out_col: NVFP4Tensor | None = None,
                        ws: Workspace | None = None, stream=None):
    rows, cols, ld = _bf16_2d(x)
    out_row = out_row or NVFP4Tensor.empty(rows, cols, BLOCK_1x16, x.device)
    out_col = out_col or NVFP4Tensor.empty(cols, rows, BLOCK_1x16, x.device)
    ws = ws or default_workspace()
    a, b = out_row.c(), out_col.c()
    st = _lib().nvfp4_quantize_dual(_ptr(x), rows, cols, ld, mode, rht_seed, sr_seed, stream_row, stream_col,
                                    ctypes.byref(a), ctypes.byref(b), ws.ptr, _stream(stream))
    _check(st, "nvfp4_quantize_dual")
    return out_row, out_col


def nvfp4_amax(x: torch.Tensor, rht: bool = True, rht_seed: int = 0, ws: Workspace | None = None,
               stream=None) -> Workspace:
    """Pass 1 alone: the amax of x (plain, and after the RHT along rows when rht) into ws."""
    rows, cols, ld = _bf16_2d(x)
    ws = ws or default_workspace()
    _check(_lib().nvfp4_amax(_ptr(x), rows, cols, ld, 1 if rht else 0, rht_seed, ws.ptr, _stream(stream)), "nvfp4_amax")
    return ws


def nvfp4_quantize_dual_shard(x: torch.Tensor, row_offset: int, rows_total: int, mode: int = RNE, rht_seed: int = 0,
                              sr_seed: int = 0, stream_row: int = 0, stream_col: int = 0,
                              out_row: NVFP4Tensor | None = None, out_col: NVFP4Tensor | None = None,
                              ws: Workspace | None = None, stream=None):
    """Pass 2 of nvfp4_quantize_dual for rows [row_offset, row_offset + rows) of a rows_total-row
    tensor, with the (reduced) amax words already in ws."""
    rows, cols, ld = _bf16_2d(x)
    out_row = out_row or NVFP4Tensor.empty(rows, cols, BLOCK_1x16, x.device)
    out_col = out_col or NVFP4Tensor.empty(cols, rows, BLOCK_1x16, x.device)
    ws = ws or default_workspace()
    a, b = out_row.c(), out_col.c()
    st = _lib().nvfp4_quantize_dual_shard(_ptr(x), rows, cols, ld, row_offset, rows_total, mode, rht_seed, sr_seed,
                                          stream_row, stream_col, ctypes.byref(a), ctypes.byref(b), ws.ptr,
                                          _stream(stream))
    _check(st, "nvfp4_quantize_dual_shard")
    return out_row, out_col


def nvfp4_quantize_dual_dp(x: torch.Tensor, group, row_offset: int, rows_total: int, mode: int = RNE,
                           rht_seed: int = 0, sr_seed: int = 0, stream_row: int = 0, stream_col: int = 0,
                           out_row: NVFP4Tensor | None = None, out_col: NVFP4Tensor | None = None,
                           ws: Workspace | None = None, stream=None):
    """Both forms of this rank's token shard, equal to the slices of the whole batch's forms: the
    shard amax, a MAX all-reduce of the two amax words over ``group`` (torch.distributed), then
    the shard's pass 2.  Without an initialized process group there is one rank, whose shard is
    the batch, and no exchange."""
    import torch.distributed as dist
    ws = nvfp4_amax(x, True, rht_seed, ws, stream)
    if dist.is_initialized():
        dist.all_reduce(ws.amax_words(), op=dist.ReduceOp.MAX, group=group)
    return nvfp4_quantize_dual_shard(x, row_offset, rows_total, mode, rht_seed, sr_seed, stream_row, stream_col,
                                     out_row, out_col, ws, stream)


def nvfp4_quantize_weight(w: torch.Tensor, transposed: bool = True, out: NVFP4Tensor | None = None,
                          out_t: NVFP4Tensor | None = None, ws: Workspace | None = None, stream=None,
                          amax_ready: bool = False):
    """16x16 forms of a weight.  amax_ready: ws holds w's amax already (an AdamW step wrote it with w),
    and the amax pass is skipped."""
    if amax_ready and ws is None:
        raise ValueError("amax_ready needs ws, the workspace that holds w's amax")
    rows, cols, ld = _bf16_2d(w)
    out = out or NVFP4Tensor.empty(rows, cols, BLOCK_16x16, w.device)
    if transposed:
        out_t = out_t or NVFP4Tensor.empty(cols, rows, BLOCK_16x16, w.device)
    ws = ws or default_workspace()
    a = out.c()
    b = out_t.c() if transposed else None
    fn = _lib().nvfp4_quantize_weight_ready if amax_ready else _lib().nvfp4_quantize_weight
    st = fn(_ptr(w), rows, cols, ld, ctypes.byref(a), ctypes.byref(b) if b else None, ws.ptr, _stream(stream))
    _check(st, "nvfp4_quantize_weight")
    return (out, out_t) if transposed else out


def nvfp4_transpose_2d(w: NVFP4Tensor, out: NVFP4Tensor | None = None, stream=None) -> NVFP4Tensor:
    out = out or NVFP4Tensor.empty(w.k, w.rows, BLOCK_16x16, w.codes.device)
    a, b = w.c(), out.c()
    _check(_lib().nvfp4_transpose_2d(ctypes.byref(a), ctypes.byref(b), _stream(stream)), "nvfp4_transpose_2d")
    return out


def nvfp4_gemm(a: NVFP4Tensor, b: NVFP4Tensor, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
               ws: Workspace | None = None, stream=None) -> torch.Tensor:
    """D[M][N] = s_tA s_tB * A . B^T (both K-major quantized forms)."""
    M, N = a.rows, b.rows
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.codes.device)
    code = OUT_FP32 if out.dtype == torch.float32 else OUT_BF16
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("output must be bf16 or fp32")
    ws = ws or default_workspace()
    ca, cb = a.c(), b.c()
    st = _lib().nvfp4_gemm(ctypes.byref(ca), ctypes.byref(cb), _ptr(out), out.stride(0), code, ws.ptr, _stream(stream))
    _check(st, "nvfp4_gemm")
    return out


def nvfp4_gemm_amax(a: NVFP4Tensor, b: NVFP4Tensor, amax_ws: Workspace, rht_seed: int = 0,
                    out: torch.Tensor | None = None, ws: Workspace | None = None, stream=None) -> torch.Tensor:
    """D = s_tA s_tB * A . B^T in bf16, with D's plain and RHT amax written into amax_ws (as
    nvfp4_amax(D, True, rht_seed, amax_ws) would), ready for the quantize call that reads D."""
    M, N = a.rows, b.rows
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.codes.device)
    if out.dtype != torch.bfloat16:
        raise TypeError("nvfp4_gemm_amax writes bf16")
    ws = ws or default_workspace()
    ca, cb = a.c(), b.c()
    st = _lib().nvfp4_gemm_amax(ctypes.byref(ca), ctypes.byref(cb), _ptr(out), out.stride(0), rht_seed, amax_ws.ptr,
                                ws.ptr, _stream(stream))
    _check(st, "nvfp4_gemm_amax")
    return out


def nvfp4_gemm_reduce_scatter(a: NVFP4Tensor, b: NVFP4Tensor, shards, owner_rows: int,
                              ws: Workspace | None = None, stream=None) -> None:
    """shards[o] += rows [o*owner_rows, (o+1)*owner_rows) of s_tA s_tB * A . B^T (fp32 adds).

    shards: fp32 [rows_o][N] tensors with one row stride (local, or another GPU's buffer through
    a peer mapping). One owner with owner_rows >= rows accumulates the whole product into it.
    """
    if not shards:
        raise ValueError("nvfp4_gemm_reduce_scatter needs at least one shard")
    ld = shards[0].stride(0)
    for t in shards:
        if t.dtype != torch.float32 or t.dim() != 2 or t.stride(1) != 1 or t.stride(0) != ld:
            raise ValueError("shards must be fp32 2-D row-major tensors with one row stride")
        if t.shape[1] != b.rows:
            raise ValueError("each shard has N = b.rows columns")
    for o, t in enumerate(shards):
        if t.shape[0] < min(owner_rows, a.rows - o * owner_rows):
            raise ValueError(f"shard {o} holds fewer rows than its owner's share")
    addrs = (ctypes.c_void_p * len(shards))(*[t.data_ptr() for t in shards])
    ws = ws or default_workspace()
    ca, cb = a.c(), b.c()
    st = _lib().nvfp4_gemm_reduce_scatter(ctypes.byref(ca), ctypes.byref(cb), addrs, len(shards), owner_rows, ld,
                                          ws.ptr, _stream(stream))
    _check(st, "nvfp4_gemm_reduce_scatter")


def nvfp4_gelu_fwd(h: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    out = torch.empty_like(h) if out is None else out
    _check(_lib().nvfp4_gelu_fwd(_ptr(h), _ptr(out), h.numel(), _stream(stream)), "nvfp4_gelu_fwd")
    return out


def nvfp4_gelu_bwd(h: torch.Tensor, dg: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    out = torch.empty_like(h) if out is None else out
    _check(_lib().nvfp4_gelu_bwd(_ptr(h), _ptr(dg), _ptr(out), h.numel(), _stream(stream)), "nvfp4_gelu_bwd")
    return out


def nvfp4_gelu_fwd_amax(h: torch.Tensor, out: torch.Tensor | None = None, rht_seed: int = 0,
                        ws: Workspace | None = None, stream=None) -> torch.Tensor:
    """GeLU of h [rows][cols] with the plain and RHT amax of the bf16 result into ws."""
    rows, cols, ld = _bf16_2d(h)
    if ld != cols:
        raise ValueError("nvfp4_gelu_fwd_amax needs a contiguous input")
    out = torch.empty_like(h) if out is None else out
    ws = ws or default_workspace()
    _check(_lib().nvfp4_gelu_fwd_amax(_ptr(h), _ptr(out), rows, cols, rht_seed, ws.ptr, _stream(stream)),
           "nvfp4_gelu_fwd_amax")
    return out


def nvfp4_gelu_bwd_amax(h: torch.Tensor, dg: torch.Tensor, out: torch.Tensor | None = None, rht_seed: int = 0,
                        ws: Workspace | None = None, stream=None) -> torch.Tensor:
    """dg * GeLU'(h) with the plain and RHT amax of the bf16 result into ws."""
    rows, cols, ld = _bf16_2d(h)
    if ld != cols or not dg.is_contiguous():
        raise ValueError("nvfp4_gelu_bwd_amax needs contiguous inputs")
    out = torch.empty_like(h) if out is None else out
    ws = ws or default_workspace()
    _check(_lib().nvfp4_gelu_bwd_amax(_ptr(h), _ptr(dg), _ptr(out), rows, cols, rht_seed, ws.ptr, _stream(stream)),
           "nvfp4_gelu_bwd_amax")
    return out


# ---------------------------------------------------------------------------------------
# MXFP4 (the comparison format: blocks of 32, UE8M0 scales, no tensor scale)
# ---------------------------------------------------------------------------------------
@dataclass
class MXTensor:
    """One MXFP4 operand form (device buffers owned by torch)."""
    codes: torch.Tensor          # uint8 [rows][k/2]
    scales: torch.Tensor         # uint8, 128x4-tile swizzled UE8M0 block scales
    rows: int
    k: int

    @staticmethod
    def empty(rows: int, k: int, device=None) -> "MXTensor":
        L = _lib()
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        codes = torch.empty(max(L.nvfp4_codes_bytes(rows, k), 1), dtype=torch.uint8, device=device)
        scales = torch.empty(max(L.nvfp4_mx_scales_bytes(rows, k), 16), dtype=torch.uint8, device=device)
        return MXTensor(codes, scales, rows, k)

    def c(self) -> CMXTensor:
        return CMXTensor(self.codes.data_ptr(), self.scales.data_ptr(), self.rows, self.k)


def nvfp4_mx_quantize(x: torch.Tensor, along: int = 0, mode: int = RNE, sr_seed: int = 0, stream_id: int = 0,
                      out: MXTensor | None = None, ws: Workspace | None = None, stream=None) -> MXTensor:
    rows, cols, ld = _bf16_2d(x)
    R, K = (cols, rows) if along else (rows, cols)
    out = out or MXTensor.empty(R, K, x.device)
    ws = ws or default_workspace()
    ct = out.c()
    _check(_lib().nvfp4_mx_quantize(_ptr(x), rows, cols, ld, along, mode, sr_seed, stream_id, ctypes.byref(ct), ws.ptr,
                                    _stream(stream)), "nvfp4_mx_quantize")
    return out


def nvfp4_mx_quantize_dual(x: torch.Tensor, mode: int = RNE, sr_seed: int = 0, stream_row: int = 0, stream_col: int = 0,
                           out_row: MXTensor | None = None, out_col: MXTensor | None = None,
                           ws: Workspace | None = None, stream=None):
    """Both MXFP4 forms of x (along 0 and along 1) from one read."""
    rows, cols, ld = _bf16_2d(x)
    out_row = out_row or MXTensor.empty(rows, cols, x.device)
    out_col = out_col or MXTensor.empty(cols, rows, x.device)
    ws = ws or default_workspace()
    a, b = out_row.c(), out_col.c()
    _check(_lib().nvfp4_mx_quantize_dual(_ptr(x), rows, cols, ld, mode, sr_seed, stream_row, stream_col,
                                         ctypes.byref(a), ctypes.byref(b), ws.ptr, _stream(stream)),
           "nvfp4_mx_quantize_dual")
    return out_row, out_col


def nvfp4_mx_gemm(a: MXTensor, b: MXTensor, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
                  ws: Workspace | None = None, stream=None) -> torch.Tensor:
    """D[M][N] = A . B^T over MXFP4 forms (kind::mxf4 block-scaled MMA)."""
    if out is None:
        out = torch.empty((a.rows, b.rows), dtype=out_dtype, device=a.codes.device)
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("output must be bf16 or fp32")
    code = OUT_FP32 if out.dtype == torch.float32 else OUT_BF16
    ws = ws or default_workspace()
    ca, cb = a.c(), b.c()
    _check(_lib().nvfp4_mx_gemm(ctypes.byref(ca), ctypes.byref(cb), _ptr(out), out.stride(0), code, ws.ptr,
                                _stream(stream)), "nvfp4_mx_gemm")
    return out


# ---------------------------------------------------------------------------------------
# BF16 path (the layers kept in high precision)
# ---------------------------------------------------------------------------------------
def nvfp4_bf16_gemm(a: torch.Tensor, b: torch.Tensor, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
                    ws: Workspace | None = None, stream=None) -> torch.Tensor:
    """D[M][N] = A[M][K] . B[N][K]^T for bf16 A, B (tcgen05 kind::f16, fp32 accumulation)."""
    M, K, lda = _bf16_2d(a)
    N, Kb, ldb = _bf16_2d(b)
    if Kb != K:
        raise ValueError("A and B need the same K")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    code = OUT_FP32 if out.dtype == torch.float32 else OUT_BF16
    ws = ws or default_workspace()
    _check(_lib().nvfp4_bf16_gemm(_ptr(a), lda, _ptr(b), ldb, M, N, K, _ptr(out), out.stride(0), code, ws.ptr,
                                  _stream(stream)), "nvfp4_bf16_gemm")
    return out


def nvfp4_bf16_transpose(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    rows, cols, ld = _bf16_2d(x)
    out = torch.empty((cols, rows), dtype=torch.bfloat16, device=x.device) if out is None else out
    _check(_lib().nvfp4_bf16_transpose(_ptr(x), rows, cols, ld, _ptr(out), out.stride(0), _stream(stream)),
           "nvfp4_bf16_transpose")
    return out


class LinearBF16:
    """The BF16 linear layer y = x w^T with its caller-owned transpose scratch."""

    def __init__(self, T: int, d: int, n: int, device=None):
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        self.T, self.d, self.n = T, d, n
        self.scratch = torch.empty(max(_lib().nvfp4_linear_bf16_scratch_bytes(T, d, n), 16), dtype=torch.uint8,
                                   device=device)
        self.ws = Workspace(device)

    def fwd(self, x: torch.Tensor, w: torch.Tensor, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        y = torch.empty((self.T, self.n), dtype=torch.bfloat16, device=x.device) if y is None else y
        _check(_lib().nvfp4_linear_bf16_fwd(_ptr(x), _ptr(w), _ptr(y), self.T, self.d, self.n, self.ws.ptr,
                                            _stream(stream)), "nvfp4_linear_bf16_fwd")
        return y

    def bwd(self, x: torch.Tensor, w: torch.Tensor, dy: torch.Tensor, dx: torch.Tensor | None = None,
            dw: torch.Tensor | None = None, stream=None):
        dx = torch.empty((self.T, self.d), dtype=torch.bfloat16, device=x.device) if dx is None else dx
        dw = torch.empty((self.n, self.d), dtype=torch.float32, device=x.device) if dw is None else dw
        _check(_lib().nvfp4_linear_bf16_bwd(_ptr(x), _ptr(w), _ptr(dy), _ptr(dx), _ptr(dw), self.T, self.d, self.n,
                                            _ptr(self.scratch), self.ws.ptr, _stream(stream)), "nvfp4_linear_bf16_bwd")
        return dx, dw


# ---------------------------------------------------------------------------------------
# BF16 products grouped by expert (one weight per expert, token rows sorted by expert)
# ---------------------------------------------------------------------------------------
def _elsewhere(dev: int, *tensors):
    raise ValueError(f"expected tensors on the current CUDA device ({dev}), got them on {[str(t.device) for t in tensors]}")


def _call_context(dev: int, ws, stream):
    """Addresses of the workspace and the stream of a call on device `dev`."""
    if ws is None:
        ws = _DEFAULT_WS.get(dev) or default_workspace()
    elif ws.index != dev:
        raise ValueError(f"the workspace lives on CUDA device {ws.index}, the call runs on {dev}")
    if stream is not None:
        return ws.addr, stream.cuda_stream
    return ws.addr, _RAW_STREAM(dev) if _RAW_STREAM is not None else torch.cuda.current_stream().cuda_stream


def _empty(shape, dtype, device, stream):
    """torch.empty in the pool of the stream the kernel runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _offsets(t: torch.Tensor, experts: int):
    if t.dtype is not torch.int32 or t.dim() != 1 or t.numel() != experts + 1 or t.stride(0) != 1:
        raise ValueError("offsets: contiguous int32 [experts + 1]")


def nvfp4_bf16_gemm_grouped(a: torch.Tensor, b: torch.Tensor, offsets: torch.Tensor, b_kn: bool = False,
                            out_dtype=torch.bfloat16, out: torch.Tensor | None = None, ws: Workspace | None = None,
                            stream=None) -> torch.Tensor:
    """out[t] = a[t] . b[e]^T (b [E][N][K]) or a[t] . b[e] (b_kn: b [E][K][N]) for the rows t in
    [offsets[e], offsets[e + 1]) of each expert e (offsets: int32 [E + 1] on the device).  Rows that
    no expert owns are left as they were in out (undefined where out is not given)."""
    if a.dtype is not torch.bfloat16 or b.dtype is not torch.bfloat16 or a.dim() != 2 or b.dim() != 3:
        raise TypeError("expected bf16 a [rows][K] and b [E][N][K] (b_kn: [E][K][N])")
    rows, K = a.shape
    E, b_rows, b_cols = b.shape
    N, Kb = (b_cols, b_rows) if b_kn else (b_rows, b_cols)
    if Kb != K:
        raise ValueError("a and b need the same K")
    a_row, a_col = a.stride()
    b_expert, b_row, b_col = b.stride()
    if a_col != 1 or b_col != 1:
        raise ValueError("inner dimensions must be contiguous")
    _offsets(offsets, E)
    if out is not None:
        out_dtype = out.dtype
    if out_dtype is not torch.bfloat16 and out_dtype is not torch.float32:
        raise TypeError("output must be bf16 or fp32")
    if out is None:
        out = _empty((rows, N), out_dtype, a.device, stream)
    elif out.shape != (rows, N):
        raise ValueError("out: [rows][N] with a contiguous inner dimension")
    out_row, out_col = out.stride()
    if out_col != 1:
        raise ValueError("out: [rows][N] with a contiguous inner dimension")
    dev = _CUR_DEVICE()
    if a.get_device() != dev or b.get_device() != dev or offsets.get_device() != dev or out.get_device() != dev:
        _elsewhere(dev, a, b, offsets, out)
    ws_addr, raw = _call_context(dev, ws, stream)
    # a single row's or slice's stride means nothing: its width, and 0
    st = _lib().nvfp4_bf16_gemm_grouped(a.data_ptr(), a_row if rows > 1 else K, rows, offsets.data_ptr(), E, b.data_ptr(),
                                        b_row if b_rows > 1 else b_cols, b_expert if E > 1 else 0, 1 if b_kn else 0, N, K,
                                        out.data_ptr(), out_row if rows > 1 else N,
                                        OUT_FP32 if out_dtype is torch.float32 else OUT_BF16, ws_addr, raw)
    if st:
        _check(st, "nvfp4_bf16_gemm_grouped")
    return out


def nvfp4_bf16_wgrad_grouped(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor | None = None,
                             accumulate: bool = False, ws: Workspace | None = None, stream=None) -> torch.Tensor:
    """out[e] = dy_e^T . x_e in fp32 over each expert's rows (dy [rows][n], x [rows][d], out
    [E][n][d]); an expert without rows gets zeros.  accumulate: out[e] += instead."""
    if dy.dtype is not torch.bfloat16 or x.dtype is not torch.bfloat16 or dy.dim() != 2 or x.dim() != 2:
        raise TypeError("expected bf16 dy [rows][n] and x [rows][d]")
    rows, M = dy.shape
    x_rows, N = x.shape
    if x_rows != rows:
        raise ValueError("dy and x need the same rows")
    dy_row, dy_col = dy.stride()
    x_row, x_col = x.stride()
    if dy_col != 1 or x_col != 1:
        raise ValueError("inner dimensions must be contiguous")
    E = offsets.shape[0] - 1 if offsets.dim() == 1 else 0
    _offsets(offsets, E)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = _empty((max(E, 0), M, N), torch.float32, dy.device, stream)
    elif out.dtype is not torch.float32 or out.shape != (E, M, N):
        raise ValueError("out: fp32 [E][n][d] with a contiguous inner dimension")
    out_expert, out_row, out_col = out.stride()
    if out_col != 1:
        raise ValueError("out: fp32 [E][n][d] with a contiguous inner dimension")
    dev = _CUR_DEVICE()
    if dy.get_device() != dev or x.get_device() != dev or offsets.get_device() != dev or out.get_device() != dev:
        _elsewhere(dev, dy, x, offsets, out)
    ws_addr, raw = _call_context(dev, ws, stream)
    st = _lib().nvfp4_bf16_wgrad_grouped(dy.data_ptr(), dy_row if rows > 1 else M, x.data_ptr(), x_row if rows > 1 else N, rows,
                                         offsets.data_ptr(), E, M, N, out.data_ptr(), out_row if M > 1 else N,
                                         out_expert if E > 1 else 0, 1 if accumulate else 0, ws_addr, raw)
    if st:
        _check(st, "nvfp4_bf16_wgrad_grouped")
    return out


class GroupedLinearBF16:
    """The BF16 linear layer y = x w_e^T with one weight per expert (w [E][n][d] bf16): rows of x are
    sorted by expert, expert e owning rows [offsets[e], offsets[e + 1]).  Its workspace holds the
    device flags of its calls (nvfp4_poll(layer.ws))."""

    def __init__(self, experts: int, d: int, n: int, device=None):
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        self.experts, self.d, self.n = experts, d, n
        self.ws = Workspace(device)

    def _weight(self, w: torch.Tensor):
        if w.shape != (self.experts, self.n, self.d):
            raise ValueError(f"w: [{self.experts}][{self.n}][{self.d}]")

    def fwd(self, x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, y: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
        self._weight(w)
        return nvfp4_bf16_gemm_grouped(x, w, offsets, out=y, ws=self.ws, stream=stream)

    def bwd(self, x: torch.Tensor, w: torch.Tensor, dy: torch.Tensor, offsets: torch.Tensor,
            dx: torch.Tensor | None = None, dw: torch.Tensor | None = None, accumulate: bool = False, stream=None):
        """dx [rows][d] bf16 and dw [E][n][d] fp32 (accumulate: added to dw)."""
        self._weight(w)
        dx = nvfp4_bf16_gemm_grouped(dy, w, offsets, b_kn=True, out=dx, ws=self.ws, stream=stream)
        dw = nvfp4_bf16_wgrad_grouped(dy, x, offsets, out=dw, accumulate=accumulate, ws=self.ws, stream=stream)
        return dx, dw


# ---------------------------------------------------------------------------------------
# AdamW over many tensors
# ---------------------------------------------------------------------------------------
class AdamWContext:
    """The tensors of an AdamW step and their moments.

    params: fp32 master weights; grads: fp32 or bf16 gradients; weights: the bf16 weights the step
    writes (None, or None entries, for none); all contiguous, entry by entry of one size, held in
    place from step to step (the context keeps references).  What a step writes overlaps no other
    tensor of it; gradients may share memory among themselves.  state: STATE_FP32 moments, or STATE_FP8:
    E4M3 codes with an fp32 scale per 256 elements (m, and the square root of v).  m, v, m_scale and
    v_scale may be given (resuming from a checkpoint); otherwise they start at zero.  amax_ws: per
    tensor a Workspace that receives the amax of its new bf16 weights (nvfp4_quantize_weight with
    amax_ready), or None.
    """

    BLOCK = 256

    def __init__(self, params, grads, weights=None, m=None, v=None, state: int = STATE_FP32, m_scale=None,
                 v_scale=None, amax_ws=None, ws: Workspace | None = None):
        if state not in (STATE_FP32, STATE_FP8):
            raise ValueError("state is STATE_FP32 or STATE_FP8")
        k = len(params)
        fp8 = state == STATE_FP8
        dt = torch.float8_e4m3fn if fp8 else torch.float32
        zeros = lambda dtype, size: [torch.zeros(size(p.numel()), dtype=dtype, device=p.device) for p in params]
        blocks = lambda n: -(-n // self.BLOCK)
        self.state = state
        self.params, self.grads = list(params), list(grads)
        self.weights = [None] * k if weights is None else list(weights)
        self.m = zeros(dt, lambda n: n) if m is None else list(m)
        self.v = zeros(dt, lambda n: n) if v is None else list(v)
        self.m_scale = (zeros(torch.float32, blocks) if m_scale is None else list(m_scale)) if fp8 else [None] * k
        self.v_scale = (zeros(torch.float32, blocks) if v_scale is None else list(v_scale)) if fp8 else [None] * k
        self.amax_ws = [None] * k if amax_ws is None else list(amax_ws)
        for name in ("grads", "weights", "m", "v", "m_scale", "v_scale", "amax_ws"):
            if len(getattr(self, name)) != k:
                raise ValueError(f"{name}: one entry per parameter")
        named = [w.addr for w in self.amax_ws if w is not None]
        if len(set(named)) != len(named):
            raise ValueError("amax_ws: a workspace of its own for each tensor")
        flat = []      # the fields of a CAdamWTensor per tensor, as 64-bit words
        written = []   # (first address, end) of what a step writes
        dev = self.params[0].get_device() if k else -1
        for i, (p, m, v, w, ws_i) in enumerate(zip(self.params, self.m, self.v, self.weights, self.amax_ws)):
            n = p.numel()
            self._tensor(p, n, torch.float32, dev, "params", i)
            self._tensor(m, n, dt, dev, "m", i)
            self._tensor(v, n, dt, dev, "v", i)
            scales = (0, 0)
            if fp8:
                ms, vs = self.m_scale[i], self.v_scale[i]
                self._tensor(ms, blocks(n), torch.float32, dev, "m_scale", i)
                self._tensor(vs, blocks(n), torch.float32, dev, "v_scale", i)
                scales = (ms.data_ptr(), vs.data_ptr())
                written += ((ms.data_ptr(), ms.data_ptr() + 4 * blocks(n)), (vs.data_ptr(), vs.data_ptr() + 4 * blocks(n)))
            if w is not None:
                self._tensor(w, n, torch.bfloat16, dev, "weights", i)
                written.append((w.data_ptr(), w.data_ptr() + 2 * n))
            if ws_i is not None and ws_i.index != dev:
                raise ValueError(f"amax_ws[{i}]: all tensors live on one CUDA device")
            size = 1 if fp8 else 4
            written += ((p.data_ptr(), p.data_ptr() + 4 * n), (m.data_ptr(), m.data_ptr() + size * n),
                        (v.data_ptr(), v.data_ptr() + size * n))
            flat += (p.data_ptr(), 0, w.data_ptr() if w is not None else 0, m.data_ptr(), v.data_ptr(), *scales,
                     ws_i.addr if ws_i is not None else 0, n, 0)
        written = sorted(r for r in written if r[0] < r[1])
        if any(a[1] > b[0] for a, b in zip(written, written[1:])):
            raise ValueError("params, weights and moments: no two of them may overlap")
        self._written = [r[0] for r in written], [r[1] for r in written]
        self._words = (ctypes.c_int64 * max(len(flat), self._WORDS))(*flat)
        self._table = ctypes.cast(self._words, ctypes.POINTER(CAdamWTensor))
        self._count, self._dev = k, dev
        if ws is None and k:
            with torch.cuda.device(dev):
                ws = default_workspace()
        self.ws = ws
        self._args = CAdamWArgs()
        self._args.state = state
        self._args_ref = ctypes.byref(self._args)
        self.set_grads(self.grads)

    _WORDS = ctypes.sizeof(CAdamWTensor) // 8

    @staticmethod
    def _tensor(t, n, dtype, dev, name, i):
        if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
            raise ValueError(f"{name}[{i}]: expected a contiguous {dtype} tensor of {n} elements")
        if dev < 0 or t.get_device() != dev:
            raise ValueError(f"{name}[{i}]: all tensors live on one CUDA device")

    def set_grads(self, grads):
        """Gradients of the next steps, where they are not the buffers of the steps before."""
        grads = list(grads)
        if len(grads) != self._count:
            raise ValueError("grads: one entry per parameter")
        words = []
        starts, ends = self._written
        for i, g in enumerate(grads):
            bf16 = isinstance(g, torch.Tensor) and g.dtype is torch.bfloat16
            n = self._words[self._WORDS * i + 8]
            self._tensor(g, n, torch.bfloat16 if bf16 else torch.float32, self._dev, "grads", i)
            addr = g.data_ptr()
            at = bisect_left(starts, addr + (2 if bf16 else 4) * n)     # what is written before the gradient's end
            if n and at and ends[at - 1] > addr:
                raise ValueError(f"grads[{i}]: overlaps a tensor that the step writes")
            words.append((addr, OUT_BF16 if bf16 else OUT_FP32))
        for i, (addr, kind) in enumerate(words):
            self._words[self._WORDS * i + 1] = addr
            self._words[self._WORDS * i + 9] = kind      # g_dtype, reserved = 0
        self.grads = grads

    def moment(self, i: int, which: str) -> torch.Tensor:
        """Moment "m" or "v" of tensor i as fp32 values (a copy)."""
        t = getattr(self, which)[i]
        if self.state == STATE_FP32:
            return t.clone()
        n = t.numel()
        x = t.reshape(-1).float() * getattr(self, which + "_scale")[i].repeat_interleave(self.BLOCK)[:n]
        return (x * x if which == "v" else x).view(t.shape)

    def dynamic(self, lr: float, step: int, beta1: float = 0.9, beta2: float = 0.95, weight_decay: float = 0.1,
                grad_scale: float = 1.0, sr_seed: int = 0) -> torch.Tensor:
        """A step's values as 32 bytes of host memory: copied into a device buffer that a captured
        nvfp4_adamw_step reads (its `dynamic`), they are what the next replay uses."""
        a = CAdamWArgs(lr, beta1, beta2, 0.0, weight_decay, grad_scale, step, sr_seed & 0xFFFFFFFFFFFFFFFF, self.state, RNE, None)
        out = CAdamWDynamic()
        _check(_lib().nvfp4_adamw_dynamic_values(ctypes.byref(a), ctypes.byref(out)), "nvfp4_adamw_dynamic_values")
        return torch.frombuffer(bytearray(bytes(out)), dtype=torch.uint8)


def nvfp4_adamw_step(ctx: AdamWContext, lr: float = 0.0, step: int = 1, beta1: float = 0.9, beta2: float = 0.95,
                     eps: float = 1e-8, weight_decay: float = 0.1, grad_scale: float = 1.0, mode: int = SR,
                     sr_seed: int = 0, dynamic: torch.Tensor | None = None, stream=None) -> None:
    """One AdamW step (decoupled weight decay, bias-corrected moments; step counts from 1) over the
    context's tensors, in place.  mode and sr_seed: rounding of 8-bit moments (give each step
    another seed).  dynamic: 32 device bytes (AdamWContext.dynamic) that replace lr, step,
    weight_decay, grad_scale and sr_seed, read when the kernel runs."""
    if ctx._count == 0:
        return
    dev = _CUR_DEVICE()
    if ctx._dev != dev:
        raise ValueError(f"the tensors live on CUDA device {ctx._dev}, the current device is {dev}")
    a = ctx._args
    a.lr, a.beta1, a.beta2, a.eps, a.weight_decay, a.grad_scale = lr, beta1, beta2, eps, weight_decay, grad_scale
    a.step, a.sr_seed, a.mode = step, sr_seed & 0xFFFFFFFFFFFFFFFF, mode
    if dynamic is not None:
        if dynamic.dtype != torch.uint8 or dynamic.numel() != 32 or not dynamic.is_contiguous() or dynamic.get_device() != dev:
            raise ValueError("dynamic: 32 contiguous uint8 on the tensors' device")
        a.dynamic = dynamic.data_ptr()
    else:
        a.dynamic = None
    ws_addr, raw = _call_context(dev, ctx.ws, stream)
    st = _lib().nvfp4_adamw(ctx._table, ctx._count, ctx._args_ref, ws_addr, raw)
    if st:
        _check(st, "nvfp4_adamw")


# ---------------------------------------------------------------------------------------
# linear layer
# ---------------------------------------------------------------------------------------
class LinearContext:
    """Caller-owned buffers of one NVFP4 linear layer y = x w^T (T tokens, d in, n out)."""

    def __init__(self, T: int, d: int, n: int, rht_seed: int = 0, device=None):
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        self.T, self.d, self.n = T, d, n
        self.xq = NVFP4Tensor.empty(T, d, BLOCK_1x16, device)
        self.xq_rht = NVFP4Tensor.empty(d, T, BLOCK_1x16, device)
        self.wq = NVFP4Tensor.empty(n, d, BLOCK_16x16, device)
        self.wqt = NVFP4Tensor.empty(d, n, BLOCK_16x16, device)
        self.dyq = NVFP4Tensor.empty(T, n, BLOCK_1x16, device)
        self.dyq_rht = NVFP4Tensor.empty(n, T, BLOCK_1x16, device)
        self.ws = Workspace(device)
        self.ctx = CLinearCtx(T, d, n, rht_seed, self.xq.c(), self.xq_rht.c(), self.wq.c(), self.wqt.c(),
                              self.dyq.c(), self.dyq_rht.c(), self.ws.buf.data_ptr(), 0, 0)

    @property
    def w_cached(self) -> bool:
        return bool(self.ctx.w_cached)

    @w_cached.setter
    def w_cached(self, v: bool):
        self.ctx.w_cached = 1 if v else 0

    @property
    def amax_ready(self) -> bool:
        """The next call's input has its amax words in this context's workspace already (a fused
        producer wrote them); the call skips its amax pass and clears the flag."""
        return bool(self.ctx.amax_ready)

    @amax_ready.setter
    def amax_ready(self, v: bool):
        self.ctx.amax_ready = 1 if v else 0

    def feed(self, consumer: "LinearContext"):
        """This layer's y is consumer's x and consumer's dx is this layer's dy (a stack of layers):
        this layer's fprop GEMM writes y's amax words into consumer's workspace, and consumer's
        dgrad GEMM writes dx's into this layer's, so the consuming quantize calls skip their amax
        passes (the caller sets amax_ready on the consuming context before its call)."""
        self.ctx.y_amax_ws = consumer.ws.ptr
        self.ctx.y_rht_seed = consumer.ctx.rht_seed
        consumer.ctx.dx_amax_ws = self.ws.ptr
        consumer.ctx.dx_rht_seed = self.ctx.rht_seed
        # each context now holds the other's workspace address: keep both workspaces alive
        self._feeds = consumer
        consumer._fed_by = self


# ---------------------------------------------------------------------------------------
# data parallelism over tokens
# ---------------------------------------------------------------------------------------
def dp_token_rows(T_local: int, rank: int, world: int):
    """(row_offset, rows_total) of this rank's token shard in the whole batch: ranks hold equal
    consecutive shards in rank order."""
    return rank * T_local, world * T_local


def dp_dw_rows(n: int, rank: int, world: int):
    """The rows [r0, r1) of dW that the reduce-scatter leaves on this rank (n % world == 0)."""
    if n % world:
        raise ValueError("out-features must divide evenly over the ranks")
    per = n // world
    return rank * per, (rank + 1) * per


class DPLinear:
    """The NVFP4 linear layer y = x w^T under data parallelism: each rank holds T consecutive tokens
    of a world * T-token batch and a replica of w.

    - X and dY: the tensor scale comes from the whole batch, so the plain and RHT amax of each
      rank's shard are all-reduced with an integer MAX between the two quantize passes, and SR
      fields are indexed in the whole batch's forms: every rank's forms are its slice of the forms
      one GPU would compute for the whole batch.
    - W: quantized on every rank from the same replica (identical forms, no exchange).
    - dW: each rank's wgrad GEMM gives the partial sum over its tokens; the partials are
      reduce-scattered (fp32 sum) over the group, each rank keeping rows dp_dw_rows(n, rank,
      world).  dw_reduce="nccl": the wgrad GEMM stores the partial, and an NCCL reduce-scatter
      overlaps the dgrad GEMM.  dw_reduce="fused": the wgrad GEMM's epilogue adds each output
      tile into its owner's shard directly (nvfp4_gemm_reduce_scatter into the ranks' symmetric
      buffers, through peer addresses), so the exchange runs inside the GEMM; a 4-byte all-reduce
      after the dgrad GEMM is the barrier that orders every rank's adds before the owner reads
      its shard.  Two shard buffers alternate between steps, so a buffer is zeroed one whole
      step (one barrier) before any rank adds into it again.
    """

    def __init__(self, T: int, d: int, n: int, group=None, rht_seed: int = 0, device=None,
                 dw_reduce: str = "nccl"):
        import torch.distributed as dist
        if dw_reduce not in ("nccl", "fused"):
            raise ValueError("dw_reduce is 'nccl' or 'fused'")
        self.group = group
        self.world = dist.get_world_size(group) if dist.is_initialized() else 1
        self.rank = dist.get_rank(group) if dist.is_initialized() else 0
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        self.T, self.d, self.n, self.rht_seed = T, d, n, rht_seed
        self.ctx = LinearContext(T, d, n, rht_seed=rht_seed, device=device)
        r0, r1 = dp_dw_rows(n, self.rank, self.world)
        self.dw = torch.empty((r1 - r0, d), dtype=torch.float32, device=device)
        self.dw_reduce = dw_reduce
        if dw_reduce == "nccl":
            self.dw_partial = torch.empty((n, d), dtype=torch.float32, device=device)
            return
        per = r1 - r0
        if per % 32 or self.world > 8:
            raise ValueError("the fused reduce-scatter needs n / world % 32 == 0 and at most 8 ranks")
        self._rs_bufs, self._rs_peers, self._rs_step = [], [], 0
        for _ in range(2):
            if dist.is_initialized():
                import torch.distributed._symmetric_memory as symm_mem
                buf = symm_mem.empty((per, d), dtype=torch.float32, device=device)
                buf.zero_()
                h = symm_mem.rendezvous(buf, group if group is not None else dist.group.WORLD)
                peers = [buf if p == self.rank else h.get_buffer(p, (per, d), torch.float32)
                         for p in range(self.world)]
            else:
                buf = torch.zeros((per, d), dtype=torch.float32, device=device)
                peers = [buf]
            self._rs_bufs.append(buf)
            self._rs_peers.append(peers)
        self._rs_flag = torch.zeros(1, dtype=torch.float32, device=device)
        if dist.is_initialized():
            torch.cuda.synchronize(device)
            dist.barrier(group)   # every shard is zero before any rank adds into it

    def fwd(self, x: torch.Tensor, w: torch.Tensor, y: torch.Tensor | None = None) -> torch.Tensor:
        c = self.ctx
        off, total = dp_token_rows(self.T, self.rank, self.world)
        nvfp4_quantize_dual_dp(x, self.group, off, total, mode=RNE, rht_seed=self.rht_seed, out_row=c.xq,
                               out_col=c.xq_rht, ws=c.ws)
        nvfp4_quantize_weight(w, out=c.wq, out_t=c.wqt, ws=c.ws)
        return nvfp4_gemm(c.xq, c.wq, out=y, ws=c.ws)

    def bwd(self, dy: torch.Tensor, sr_seed: int, dx: torch.Tensor | None = None):
        """dX for this rank's tokens; this rank's rows of the batch's dW land in self.dw."""
        import torch.distributed as dist
        c = self.ctx
        off, total = dp_token_rows(self.T, self.rank, self.world)
        nvfp4_quantize_dual_dp(dy, self.group, off, total, mode=SR, rht_seed=self.rht_seed, sr_seed=sr_seed,
                               stream_row=STREAM_DGRAD, stream_col=STREAM_WGRAD, out_row=c.dyq, out_col=c.dyq_rht,
                               ws=c.ws)
        if self.dw_reduce == "fused":
            j = self._rs_step & 1
            self._rs_step += 1
            nvfp4_gemm_reduce_scatter(c.dyq_rht, c.xq_rht, self._rs_peers[j], self.dw.shape[0], ws=c.ws)
            dx = nvfp4_gemm(c.dyq, c.wqt, out=dx, ws=c.ws)
            if dist.is_initialized():
                dist.all_reduce(self._rs_flag, group=self.group)   # every rank's adds are complete
            self.dw.copy_(self._rs_bufs[j])
            self._rs_bufs[j].zero_()
            return dx
        nvfp4_gemm(c.dyq_rht, c.xq_rht, out=self.dw_partial, ws=c.ws)
        work = None
        if self.world > 1:
            work = dist.reduce_scatter_tensor(self.dw, self.dw_partial, op=dist.ReduceOp.SUM, group=self.group,
                                              async_op=True)
        dx = nvfp4_gemm(c.dyq, c.wqt, out=dx, ws=c.ws)
        if work is not None:
            work.wait()
        else:
            self.dw.copy_(self.dw_partial)
        return dx


def nvfp4_linear_fwd(ctx: LinearContext, x: torch.Tensor, w: torch.Tensor | None, y: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    if y is None:
        y = torch.empty((ctx.T, ctx.n), dtype=torch.bfloat16, device=x.device)
    st = _lib().nvfp4_linear_fwd(_ptr(x), _ptr(w), _ptr(y), ctypes.byref(ctx.ctx), _stream(stream))
    _check(st, "nvfp4_linear_fwd")
    return y


def nvfp4_linear_bwd(ctx: LinearContext, dy: torch.Tensor, sr_seed: int, dx: torch.Tensor | None = None,
                     dw: torch.Tensor | None = None, stream=None):
    if dx is None:
        dx = torch.empty((ctx.T, ctx.d), dtype=torch.bfloat16, device=dy.device)
    if dw is None:
        dw = torch.empty((ctx.n, ctx.d), dtype=torch.float32, device=dy.device)
    st = _lib().nvfp4_linear_bwd(_ptr(dy), sr_seed, _ptr(dx), _ptr(dw), ctypes.byref(ctx.ctx), _stream(stream))
    _check(st, "nvfp4_linear_bwd")
    return dx, dw
