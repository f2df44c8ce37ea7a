"""Python binding of libbsg (include/bsg.h): block-scaled grouped quantize and
grouped GEMM for MoE expert products on MI355X.

Argument marshalling only.  Every function has the name of its C entry point,
takes torch tensors (device memory) and enqueues on the current torch stream;
outputs the caller does not pass are allocated with torch.  Every step of the
computation runs in the HIP library: if ``libbsg.so`` is missing or fails to
load, every call raises.
"""

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libbsg.so")

BSG_FPROP_TN = 0
BSG_WGRAD_NT = 1
BSG_OUT_BF16 = 0
BSG_OUT_F32 = 1
BSG_DGRAD_NN = 2
BSG_WGRAD_NT_E5M2 = 3
BSG_OUT_F16 = 2
BSG_IN_BF16 = 0
BSG_IN_F16 = 1
BSG_IN_F32 = 2
BSG_GRAD_BF16 = 0
BSG_GRAD_F16 = 1
BSG_GRAD_F32 = 2
BSG_MAX_LORA_RANK = 256
BSG_MAX_TOP_K = 16
BSG_MAX_INT8_K = 131056
BSG_MAX_GROUPS = 256
BSG_COLWISE_PAD = 128
DEV_NEGATIVE_SIZE = 1
DEV_OVER_CAPACITY = 2
DEV_BAD_PADDING = 4
DEV_NONFINITE = 8
DEV_BAD_ADAPTER = 16

EXPORTS = ("bsg_last_error", "bsg_version", "group_offsets_i32_to_i64", "grouped_quantize_mxfp8",
           "grouped_quantize_mxfp8_rowwise_e5m2",
           "grouped_quantize_nvfp4_rowscaled", "grouped_quantize_nvfp4_rowscaled_colwise",
           "grouped_quantize_nvfp4_pertensor",
           "grouped_gemm_mxfp8", "grouped_gemm_mxfp8_ex", "grouped_gemm_nvfp4_rowscaled",
           "grouped_gemm_nvfp4_rowscaled_wgrad", "grouped_gemm_nvfp4_pertensor",
           "grouped_gemm_nvfp4_rowscaled_noalloc", "grouped_quantize_nvfp4_pertensor_rht",
           "grouped_quantize_nvfp4_pertensor_2d", "grouped_quantize_mxfp8_colwise_e5m2",
           "grouped_gemm_nvfp4_rowscaled_ex", "grouped_gemm_nvfp4_rowscaled_wgrad_ex",
           "grouped_gemm_mxfp8_workspace_size", "grouped_gemm_mxfp8_ws",
           "grouped_gemm_nvfp4_workspace_size", "grouped_gemm_nvfp4_rowscaled_ws",
           "grouped_gemm_nvfp4_pertensor_ws",
           "grouped_gemm_16bit_workspace_size", "grouped_gemm_16bit_tile_rows", "grouped_gemm_16bit",
           "grouped_lora_gemm_16bit_workspace_size", "grouped_lora_gemm_16bit_tile_rows",
           "grouped_lora_gemm_16bit",
           "grad_clip_plan_fill", "grad_clip_workspace_size", "grad_norm", "clip_grad_norm",
           "moe_router_topk_workspace_size", "moe_router_topk", "moe_router_topk_backward",
           "grouped_quantize_int8", "grouped_gemm_int8_workspace_size", "grouped_gemm_int8_tile_rows",
           "grouped_gemm_int8", "grouped_gemm_int8_dynamic_workspace_size",
           "grouped_gemm_int8_dynamic", "grouped_swiglu_checkpoint_mxfp8",
           "grouped_swiglu_checkpoint_mxfp8_backward")
BSG_NOALLOC_SCRATCH_BYTES = 64 << 20

_lib = None


class BsgError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__("bsg status %d: %s" % (code, msg))
        self.code = code


def load_library(path=LIB_PATH):
    """Loads libbsg.so once; raises if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("libbsg.so not built at %s (run python -m block_scaled_grouped_amd.build)"
                           % path)
    lib = ctypes.CDLL(path)
    P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.bsg_last_error.restype = ctypes.c_char_p
    lib.bsg_last_error.argtypes = []
    lib.bsg_version.restype = I32
    lib.bsg_version.argtypes = []
    lib.group_offsets_i32_to_i64.restype = I32
    lib.group_offsets_i32_to_i64.argtypes = [P, I64, I64, I64, P, P, I64, P, P]
    lib.grouped_quantize_mxfp8.restype = I32
    lib.grouped_quantize_mxfp8.argtypes = [P, I64, I64, I64, P, P, P, P, I64, P, P, P, P]
    lib.grouped_quantize_mxfp8_rowwise_e5m2.restype = I32
    lib.grouped_quantize_mxfp8_rowwise_e5m2.argtypes = [P, I64, I64, I64, P, P, P, P, P]
    lib.grouped_quantize_mxfp8_colwise_e5m2.restype = I32
    lib.grouped_quantize_mxfp8_colwise_e5m2.argtypes = [P, I64, I64, I64, P, P, I64, P, P, P, P]
    lib.grouped_quantize_nvfp4_rowscaled.restype = I32
    lib.grouped_quantize_nvfp4_rowscaled.argtypes = [P, I64, I64, I64, P, P, P, P, P, P]
    lib.grouped_quantize_nvfp4_rowscaled_colwise.restype = I32
    lib.grouped_quantize_nvfp4_rowscaled_colwise.argtypes = [P, I64, I64, I64, P, P, I64, P, P, P,
                                                             P, P]
    lib.grouped_gemm_mxfp8.restype = I32
    lib.grouped_gemm_mxfp8.argtypes = [I32, I64, P, P, P, P, P, I64, I64, I64, P, I32, P, P]
    lib.grouped_gemm_mxfp8_workspace_size.restype = ctypes.c_size_t
    lib.grouped_gemm_mxfp8_workspace_size.argtypes = []
    lib.grouped_gemm_mxfp8_ws.restype = I32
    lib.grouped_gemm_mxfp8_ws.argtypes = [I32, I64, P, P, P, P, P, I64, I64, I64, P, I32, P,
                                          ctypes.c_size_t, P, P]
    lib.grouped_gemm_mxfp8_ex.restype = I32
    lib.grouped_gemm_mxfp8_ex.argtypes = [I32, I64, P, P, P, P, P, I64, I64, I64, P, I32, P, P, P,
                                          P, P]
    lib.grouped_gemm_nvfp4_rowscaled.restype = I32
    lib.grouped_gemm_nvfp4_rowscaled.argtypes = [I64, P, P, P, P, I64, I64, P, P, P, P, P, I64, I32,
                                                 P, P, P]
    lib.grouped_quantize_nvfp4_pertensor.restype = I32
    lib.grouped_quantize_nvfp4_pertensor.argtypes = [P, I64, I64, I64, P, P, P, P, P, P]
    lib.grouped_quantize_nvfp4_pertensor_rht.restype = I32
    lib.grouped_quantize_nvfp4_pertensor_rht.argtypes = [P, I64, I64, I64, P, ctypes.c_uint32, P, P,
                                                         P, P, P]
    lib.grouped_quantize_nvfp4_pertensor_2d.restype = I32
    lib.grouped_quantize_nvfp4_pertensor_2d.argtypes = [P, I64, I64, I64, P, P, P, P, P, P]
    lib.grouped_gemm_nvfp4_pertensor.restype = I32
    lib.grouped_gemm_nvfp4_pertensor.argtypes = [I64, P, P, P, P, I64, I64, P, P, P, P, P, I64, I32,
                                                 P, P]
    lib.grouped_gemm_nvfp4_rowscaled_ex.restype = I32
    lib.grouped_gemm_nvfp4_rowscaled_ex.argtypes = [I64, P, P, P, P, I64, I64, P, P, P, P, P, I64,
                                                    I32, P, I32, P, P]
    lib.grouped_gemm_nvfp4_rowscaled_wgrad_ex.restype = I32
    lib.grouped_gemm_nvfp4_rowscaled_wgrad_ex.argtypes = [I64, P, P, P, P, P, P, P, I64, I64, I64,
                                                          P, I32, I32, P, P]
    lib.grouped_gemm_nvfp4_rowscaled_noalloc.restype = I32
    lib.grouped_gemm_nvfp4_rowscaled_noalloc.argtypes = [I64, P, P, P, P, I64, I64, P, P, P, P, P,
                                                         I64, I32, P, P]
    lib.grouped_gemm_nvfp4_workspace_size.restype = ctypes.c_size_t
    lib.grouped_gemm_nvfp4_workspace_size.argtypes = []
    lib.grouped_gemm_nvfp4_rowscaled_ws.restype = I32
    lib.grouped_gemm_nvfp4_rowscaled_ws.argtypes = [I64, P, P, P, P, I64, I64, P, P, P, P, P, I64,
                                                    I32, I32, P, ctypes.c_size_t, P, P]
    lib.grouped_gemm_nvfp4_pertensor_ws.restype = I32
    lib.grouped_gemm_nvfp4_pertensor_ws.argtypes = [I64, P, P, P, P, I64, I64, P, P, P, P, P, I64,
                                                    I32, P, ctypes.c_size_t, P, P]
    lib.grouped_gemm_nvfp4_rowscaled_wgrad.restype = I32
    lib.grouped_gemm_nvfp4_rowscaled_wgrad.argtypes = [I64, P, P, P, P, P, P, P, I64, I64, I64, P,
                                                       I32, P, P]
    SZ = ctypes.c_size_t
    lib.grouped_gemm_16bit_workspace_size.restype = SZ
    lib.grouped_gemm_16bit_workspace_size.argtypes = []
    lib.grouped_gemm_16bit_tile_rows.restype = I32
    lib.grouped_gemm_16bit_tile_rows.argtypes = [I32, I64, I64, I64, I64, I32]
    lib.grouped_gemm_16bit.restype = I32
    lib.grouped_gemm_16bit.argtypes = [I32, I32, I64, P, I64, P, I64, I64, P, I64, I64, I64, P, P,
                                       I64, I64, I32, P, SZ, P, P]
    lib.grouped_lora_gemm_16bit_workspace_size.restype = SZ
    lib.grouped_lora_gemm_16bit_workspace_size.argtypes = [I64, I64, I64, I64]
    lib.grouped_lora_gemm_16bit_tile_rows.restype = I32
    lib.grouped_lora_gemm_16bit_tile_rows.argtypes = [I64, I64, I64]
    lib.grouped_lora_gemm_16bit.restype = I32
    lib.grouped_lora_gemm_16bit.argtypes = [I32, I64, P, I64, P, I64, P, P, I64, I64, P, P, P, I64,
                                            I64, I64, P, I64, I32, P, SZ, P, P]
    lib.grad_clip_plan_fill.restype = I32
    lib.grad_clip_plan_fill.argtypes = [I64, P, P, P, P, P, SZ, P]
    lib.grad_clip_workspace_size.restype = SZ
    lib.grad_clip_workspace_size.argtypes = []
    lib.grad_norm.restype = I32
    lib.grad_norm.argtypes = [P, I64, P, SZ, P, P, P, P]
    lib.clip_grad_norm.restype = I32
    lib.clip_grad_norm.argtypes = [P, I64, ctypes.c_float, P, P, SZ, P, P, P]
    lib.moe_router_topk_workspace_size.restype = SZ
    lib.moe_router_topk_workspace_size.argtypes = [I64, I64]
    lib.moe_router_topk.restype = I32
    lib.moe_router_topk.argtypes = [I32, P, I64, I64, I64, I64, P, I32, P, P, P, P, P, P, P, SZ, P, P]
    lib.moe_router_topk_backward.restype = I32
    lib.moe_router_topk_backward.argtypes = [I32, P, I64, I64, I64, I64, P, I32, P, P, P, P, P, P, I64,
                                             P]
    lib.grouped_quantize_int8.restype = I32
    lib.grouped_quantize_int8.argtypes = [I32, P, I64, I64, I64, I64, P, P, P, P, P]
    lib.grouped_gemm_int8_workspace_size.restype = SZ
    lib.grouped_gemm_int8_workspace_size.argtypes = []
    lib.grouped_gemm_int8_tile_rows.restype = I32
    lib.grouped_gemm_int8_tile_rows.argtypes = [I64, I64, I64, I64, I32]
    lib.grouped_gemm_int8.restype = I32
    lib.grouped_gemm_int8.argtypes = [I64, P, I64, P, P, I64, I64, P, P, I64, I64, I64, P, I64, I32, P,
                                      SZ, P, P]
    lib.grouped_gemm_int8_dynamic_workspace_size.restype = SZ
    lib.grouped_gemm_int8_dynamic_workspace_size.argtypes = [I64, I64]
    lib.grouped_gemm_int8_dynamic.restype = I32
    lib.grouped_gemm_int8_dynamic.argtypes = [I32, I64, P, I64, P, I64, I64, P, P, I64, I64, I64, P,
                                              I64, I32, P, SZ, P, P]
    lib.grouped_swiglu_checkpoint_mxfp8.restype = I32
    lib.grouped_swiglu_checkpoint_mxfp8.argtypes = [I32, P, I64, P, I64, P, I64, I64, P, I64, P, P, P,
                                                    P]
    lib.grouped_swiglu_checkpoint_mxfp8_backward.restype = I32
    lib.grouped_swiglu_checkpoint_mxfp8_backward.argtypes = [I32, P, P, P, P, I64, I64, P, I64, I64, P,
                                                             I64, P, I64, P, P, P]
    _lib = lib
    return lib


def _check(rc):
    if rc != 0:
        raise BsgError(rc, _lib.bsg_last_error().decode())


def _ptr(t):
    return None if t is None else t.data_ptr() or None


def _stream(t):
    import torch
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("bsg operates on device tensors")


def _dtype_name(dt):
    return str(dt).replace("torch.", "")


def _req(t, name, nbytes, dtype=None, optional=False):
    """Checks, before anything is launched, that tensor t can hold what the C
    call will touch: a contiguous device tensor of at least nbytes bytes (and of
    the given torch dtype).  A buffer that is too small would otherwise be read
    or written out of bounds on the device."""
    if t is None:
        if optional:
            return
        raise ValueError("%s is required" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if dtype is not None:
        allowed = dtype if isinstance(dtype, tuple) else (dtype,)
        if t.dtype not in allowed:
            raise ValueError("%s must be %s, not %s" % (
                name, " or ".join(_dtype_name(d) for d in allowed), _dtype_name(t.dtype)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    have = t.nbytes
    if have < nbytes:
        raise ValueError("%s holds %d bytes; the call touches %d" % (name, have, int(nbytes)))


def _i64():
    import torch
    return torch.int64


def _f32():
    import torch
    return torch.float32


def _bf16_2d(x, name="x"):
    import torch
    if x.dim() != 2:
        raise ValueError("%s must be 2-D [rows, cols]" % name)
    _req(x, name, 0, torch.bfloat16)
    return x.shape


def _out_dtype(out_dtype):
    import torch
    if out_dtype == BSG_OUT_F32:
        return torch.float32, 4
    if out_dtype == BSG_OUT_BF16:
        return torch.bfloat16, 2
    raise ValueError("unknown out_dtype %r" % (out_dtype,))


def mx_scale_row_bytes(cols):
    """Stored E8M0 bytes per row of a rowwise MXFP8 tensor (cols / 32 rounded up to 4)."""
    return ((cols // 32 + 3) // 4) * 4


def mx_scale_shape(rows, cols):
    """Shape of rowwise MXFP8 scales: [NQ][rows] words of 4 bytes, NQ = ceil(cols / 128)."""
    return (mx_scale_row_bytes(cols) // 4, rows, 4)


def group_offsets_i32_to_i64(sizes, multiplier=1, pad_to=1, capacity=0, sizes_i64=None,
                             offsets=None, status=None):
    """int32 [G] sizes -> (int64 [G] sizes * multiplier, int64 [G+1] offsets)."""
    import torch
    lib = load_library()
    _req(sizes, "sizes", 0, torch.int32)
    G = sizes.numel()
    if sizes_i64 is None:
        sizes_i64 = torch.empty(G, dtype=torch.int64, device=sizes.device)
    if offsets is None:
        offsets = torch.empty(G + 1, dtype=torch.int64, device=sizes.device)
    _req(sizes_i64, "sizes_i64", 8 * G, torch.int64)
    _req(offsets, "offsets", 8 * (G + 1), torch.int64)
    _req(status, "status", 4, optional=True)
    _check(lib.group_offsets_i32_to_i64(_ptr(sizes), G, multiplier, pad_to, _ptr(sizes_i64),
                                        _ptr(offsets), capacity, _ptr(status), _stream(sizes)))
    return sizes_i64, offsets


def grouped_quantize_mxfp8(x, offsets, G=None, rowwise=True, padded_offsets=None,
                           col_rows_cap=None, row_data=None, row_scales=None, col_data=None,
                           col_scales=None, status=None):
    """bf16 [rows_cap, cols] -> dict with "row_data"/"row_scales" (rowwise) and
    "col_data"/"col_scales" (when padded_offsets is given), uint8 tensors."""
    import torch
    lib = load_library()
    rows_cap, cols = _bf16_2d(x)
    G = offsets.numel() - 1 if G is None else G
    _req(offsets, "offsets", 8 * (G + 1), _i64())
    out = {}
    if rowwise:
        if row_data is None:
            row_data = torch.empty((rows_cap, cols), dtype=torch.uint8, device=x.device)
        if row_scales is None:
            row_scales = torch.empty(mx_scale_shape(rows_cap, cols), dtype=torch.uint8,
                                     device=x.device)
        out["row_data"], out["row_scales"] = row_data, row_scales
    else:
        row_data = row_scales = None
    if padded_offsets is not None:
        if col_rows_cap is None:
            col_rows_cap = rows_cap + BSG_COLWISE_PAD * G
        if col_data is None:
            col_data = torch.empty(col_rows_cap * cols, dtype=torch.uint8, device=x.device)
        if col_scales is None:
            col_scales = torch.empty(col_rows_cap * cols // 32, dtype=torch.uint8, device=x.device)
        out["col_data"], out["col_scales"] = col_data, col_scales
        out["col_rows_cap"] = col_rows_cap
        _req(padded_offsets, "padded_offsets", 8 * (G + 1), _i64())
        _req(col_data, "col_data", col_rows_cap * cols)
        _req(col_scales, "col_scales", col_rows_cap * cols // 32)
    if rowwise:
        _req(row_data, "row_data", rows_cap * cols)
        _req(row_scales, "row_scales", rows_cap * mx_scale_row_bytes(cols))
    _req(status, "status", 4, optional=True)
    _check(lib.grouped_quantize_mxfp8(_ptr(x), rows_cap, cols, G, _ptr(offsets), _ptr(row_data),
                                      _ptr(row_scales), _ptr(padded_offsets),
                                      col_rows_cap or 0, _ptr(col_data), _ptr(col_scales),
                                      _ptr(status), _stream(x)))
    return out


def grouped_quantize_mxfp8_rowwise_e5m2(x, offsets, G=None, row_data=None, row_scales=None,
                                        status=None):
    """bf16 [rows_cap, cols] gradient -> (E5M2 [rows_cap, cols], E8M0 scale words as
    grouped_quantize_mxfp8's rowwise output)."""
    import torch
    lib = load_library()
    rows_cap, cols = _bf16_2d(x)
    G = offsets.numel() - 1 if G is None else G
    _req(offsets, "offsets", 8 * (G + 1), torch.int64)
    if row_data is None:
        row_data = torch.empty((rows_cap, cols), dtype=torch.uint8, device=x.device)
    if row_scales is None:
        row_scales = torch.empty(mx_scale_shape(rows_cap, cols), dtype=torch.uint8, device=x.device)
    _req(row_data, "row_data", rows_cap * cols)
    _req(row_scales, "row_scales", rows_cap * mx_scale_row_bytes(cols))
    _req(status, "status", 4, optional=True)
    _check(lib.grouped_quantize_mxfp8_rowwise_e5m2(_ptr(x), rows_cap, cols, G, _ptr(offsets),
                                                   _ptr(row_data), _ptr(row_scales), _ptr(status),
                                                   _stream(x)))
    return row_data, row_scales


def grouped_quantize_mxfp8_colwise_e5m2(x, offsets, padded_offsets, G=None, col_rows_cap=None,
                                        col_data=None, col_scales=None, status=None):
    """bf16 [rows_cap, cols] gradient -> its E5M2 columnwise copy (col_data,
    col_scales) in grouped_quantize_mxfp8's columnwise layout."""
    import torch
    lib = load_library()
    rows_cap, cols = _bf16_2d(x)
    G = offsets.numel() - 1 if G is None else G
    _req(offsets, "offsets", 8 * (G + 1), torch.int64)
    _req(padded_offsets, "padded_offsets", 8 * (G + 1), torch.int64)
    if col_rows_cap is None:
        col_rows_cap = rows_cap + BSG_COLWISE_PAD * G
    if col_data is None:
        col_data = torch.empty(col_rows_cap * cols, dtype=torch.uint8, device=x.device)
    if col_scales is None:
        col_scales = torch.empty(col_rows_cap * cols // 32, dtype=torch.uint8, device=x.device)
    _req(col_data, "col_data", col_rows_cap * cols)
    _req(col_scales, "col_scales", col_rows_cap * cols // 32)
    _req(status, "status", 4, optional=True)
    _check(lib.grouped_quantize_mxfp8_colwise_e5m2(_ptr(x), rows_cap, cols, G, _ptr(offsets),
                                                   _ptr(padded_offsets), col_rows_cap,
                                                   _ptr(col_data), _ptr(col_scales), _ptr(status),
                                                   _stream(x)))
    return col_data, col_scales


def grouped_quantize_nvfp4_rowscaled(x, offsets, G=None, data=None, block_scales=None, outer=None,
                                     status=None):
    """bf16 [rows_cap, cols] -> (E2M1 [rows_cap, cols/2], E4M3 [rows_cap, cols/16], f32 [rows_cap])."""
    import torch
    lib = load_library()
    rows_cap, cols = _bf16_2d(x)
    G = offsets.numel() - 1 if G is None else G
    _req(offsets, "offsets", 8 * (G + 1), torch.int64)
    if data is None:
        data = torch.empty((rows_cap, cols // 2), dtype=torch.uint8, device=x.device)
    if block_scales is None:
        block_scales = torch.empty((rows_cap, cols // 16), dtype=torch.uint8, device=x.device)
    if outer is None:
        outer = torch.empty(rows_cap, dtype=torch.float32, device=x.device)
    _req(data, "data", rows_cap * cols // 2)
    _req(block_scales, "block_scales", rows_cap * cols // 16)
    _req(outer, "outer", 4 * rows_cap, torch.float32)
    _req(status, "status", 4, optional=True)
    _check(lib.grouped_quantize_nvfp4_rowscaled(_ptr(x), rows_cap, cols, G, _ptr(offsets),
                                                _ptr(data), _ptr(block_scales), _ptr(outer),
                                                _ptr(status), _stream(x)))
    return data, block_scales, outer


def grouped_quantize_nvfp4_pertensor(x, offsets, G=None, data=None, block_scales=None, amax=None,
                                     status=None):
    """bf16 [rows_cap, cols] -> (E2M1 [rows_cap, cols/2], E4M3 [rows_cap, cols/16], f32 amax [G])."""
    import torch
    lib = load_library()
    rows_cap, cols = _bf16_2d(x)
    G = offsets.numel() - 1 if G is None else G
    _req(offsets, "offsets", 8 * (G + 1), torch.int64)
    if data is None:
        data = torch.empty((rows_cap, cols // 2), dtype=torch.uint8, device=x.device)
    if block_scales is None:
        block_scales = torch.empty((rows_cap, cols // 16), dtype=torch.uint8, device=x.device)
    if amax is None:
        amax = torch.empty(G, dtype=torch.float32, device=x.device)
    _req(data, "data", rows_cap * cols // 2)
    _req(block_scales, "block_scales", rows_cap * cols // 16)
    _req(amax, "amax", 4 * G, torch.float32)
    _req(status, "status", 4, optional=True)
    _check(lib.grouped_quantize_nvfp4_pertensor(_ptr(x), rows_cap, cols, G, _ptr(offsets),
                                                _ptr(data), _ptr(block_scales), _ptr(amax),
                                                _ptr(status), _stream(x)))
    return data, block_scales, amax


def _pertensor_variant(cfn, x, offsets, G, data, block_scales, amax, status, *extra):
    import torch
    rows_cap, cols = _bf16_2d(x)
    G = offsets.numel() - 1 if G is None else G
    _req(offsets, "offsets", 8 * (G + 1), torch.int64)
    if data is None:
        data = torch.empty((rows_cap, cols // 2), dtype=torch.uint8, device=x.device)
    if block_scales is None:
        block_scales = torch.empty((rows_cap, cols // 16), dtype=torch.uint8, device=x.device)
    if amax is None:
        amax = torch.empty(G, dtype=torch.float32, device=x.device)
    _req(data, "data", rows_cap * cols // 2)
    _req(block_scales, "block_scales", rows_cap * cols // 16)
    _req(amax, "amax", 4 * G, torch.float32)
    _req(status, "status", 4, optional=True)
    args = [_ptr(x), rows_cap, cols, G, _ptr(offsets)] + list(extra) + [
        _ptr(data), _ptr(block_scales), _ptr(amax), _ptr(status), _stream(x)]
    _check(cfn(*args))
    return data, block_scales, amax


def grouped_quantize_nvfp4_pertensor_rht(x, offsets, rht_sign_mask, G=None, data=None,
                                         block_scales=None, amax=None, status=None):
    """Per-tensor NVFP4 of the rows' randomized Hadamard transform (16-element
    blocks, signs from the 16-bit mask): outputs as
    grouped_quantize_nvfp4_pertensor.  See include/bsg.h."""
    lib = load_library()
    return _pertensor_variant(lib.grouped_quantize_nvfp4_pertensor_rht, x, offsets, G, data,
                              block_scales, amax, status, ctypes.c_uint32(int(rht_sign_mask)))


def grouped_quantize_nvfp4_pertensor_2d(x, offsets, G=None, data=None, block_scales=None, amax=None,
                                        status=None):
    """Per-tensor NVFP4 with one E4M3 scale per 16 x 16 block (written into each
    row of the block): outputs as grouped_quantize_nvfp4_pertensor.  See
    include/bsg.h."""
    lib = load_library()
    return _pertensor_variant(lib.grouped_quantize_nvfp4_pertensor_2d, x, offsets, G, data,
                              block_scales, amax, status)


def grouped_quantize_nvfp4_rowscaled_colwise(x, offsets, padded_offsets, G=None, col_rows_cap=None,
                                             data=None, block_scales=None, outer=None, status=None):
    """bf16 [rows_cap, cols] -> per-expert transposed copies: (E2M1 bytes
    [col_rows_cap * cols / 2], E4M3 [col_rows_cap * cols / 16], f32 outer [G, cols]).
    See include/bsg.h for the block layout."""
    import torch
    lib = load_library()
    rows_cap, cols = _bf16_2d(x)
    G = offsets.numel() - 1 if G is None else G
    _req(offsets, "offsets", 8 * (G + 1), torch.int64)
    _req(padded_offsets, "padded_offsets", 8 * (G + 1), torch.int64)
    if col_rows_cap is None:
        col_rows_cap = rows_cap + BSG_COLWISE_PAD * G
    if data is None:
        data = torch.empty(col_rows_cap * cols // 2, dtype=torch.uint8, device=x.device)
    if block_scales is None:
        block_scales = torch.empty(col_rows_cap * cols // 16, dtype=torch.uint8, device=x.device)
    if outer is None:
        outer = torch.empty((G, cols), dtype=torch.float32, device=x.device)
    _req(data, "data", col_rows_cap * cols // 2)
    _req(block_scales, "block_scales", col_rows_cap * cols // 16)
    _req(outer, "outer", 4 * G * cols, torch.float32)
    _req(status, "status", 4, optional=True)
    _check(lib.grouped_quantize_nvfp4_rowscaled_colwise(
        _ptr(x), rows_cap, cols, G, _ptr(offsets), _ptr(padded_offsets), col_rows_cap, _ptr(data),
        _ptr(block_scales), _ptr(outer), _ptr(status), _stream(x)))
    return data, block_scales, outer


def _mx_gemm_bytes(mode, G, rows_cap, n, k):
    """Bytes grouped_gemm_mxfp8 reads from a, a_scales, b, b_scales, and the
    output's element count (include/bsg.h gives the layouts)."""
    nq = (k + 127) // 128
    if mode == BSG_FPROP_TN:
        return (rows_cap * k, 4 * nq * rows_cap, G * n * k, 4 * nq * G * n, rows_cap * n)
    if mode == BSG_DGRAD_NN:
        kpad = 128 * nq   # the weights' columnwise copy pads each expert to 128 tokens
        return (rows_cap * k, 4 * nq * rows_cap, G * n * kpad, G * n * kpad // 32, rows_cap * n)
    if mode in (BSG_WGRAD_NT, BSG_WGRAD_NT_E5M2):
        return (rows_cap * n, rows_cap * n // 32, rows_cap * k, rows_cap * k // 32, G * n * k)
    raise ValueError("unknown mode %r" % (mode,))


def _mx_gemm_check(mode, G, a, a_scales, b, b_scales, offsets, rows_cap, n, k, out, out_dtype,
                   status):
    na, nas, nb, nbs, nout = _mx_gemm_bytes(mode, G, rows_cap, n, k)
    _req(a, "a", na)
    _req(a_scales, "a_scales", nas)
    _req(b, "b", nb)
    _req(b_scales, "b_scales", nbs)
    _req(offsets, "offsets", 8 * (G + 1), _i64())
    dt, esz = _out_dtype(out_dtype)
    _req(out, "out", esz * nout, dt)
    _req(status, "status", 4, optional=True)


def gemm_workspace(device=None):
    """A uint8 device tensor of max(grouped_gemm_mxfp8_workspace_size(),
    grouped_gemm_nvfp4_workspace_size(), grouped_gemm_16bit_workspace_size()) bytes
    (256-byte aligned: torch's caching allocator aligns blocks to 512), for the
    `workspace` argument of grouped_gemm_mxfp8, grouped_gemm_nvfp4_rowscaled,
    grouped_gemm_nvfp4_pertensor, grouped_gemm_16bit and grouped_gemm_int8 (which needs
    as much as grouped_gemm_16bit).  Calls that may run at the same time (on different
    streams) need a workspace each."""
    import torch
    lib = load_library()
    n = max(int(lib.grouped_gemm_mxfp8_workspace_size()),
            int(lib.grouped_gemm_nvfp4_workspace_size()),
            int(lib.grouped_gemm_16bit_workspace_size()))
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def grouped_gemm_mxfp8(mode, a, a_scales, b, b_scales, offsets, rows_cap, n, k, out=None,
                       out_dtype=BSG_OUT_BF16, G=None, status=None, workspace=None):
    """FPROP_TN, DGRAD_NN: out [rows_cap, n]; WGRAD_NT: out [G, n, k].  With a
    `workspace` (gemm_workspace()), grouped_gemm_mxfp8_ws: the last round of
    tiles is split along the contraction.  See include/bsg.h."""
    import torch
    lib = load_library()
    _need_cuda(a, a_scales, b, b_scales, offsets)
    G = offsets.numel() - 1 if G is None else G
    if out is None:
        dt = _out_dtype(out_dtype)[0]
        shape = (G, n, k) if mode in (BSG_WGRAD_NT, BSG_WGRAD_NT_E5M2) else (rows_cap, n)
        out = torch.empty(shape, dtype=dt, device=a.device)
    _mx_gemm_check(mode, G, a, a_scales, b, b_scales, offsets, rows_cap, n, k, out, out_dtype,
                   status)
    if workspace is not None:
        _need_cuda(workspace)
        _check(lib.grouped_gemm_mxfp8_ws(mode, G, _ptr(a), _ptr(a_scales), _ptr(b), _ptr(b_scales),
                                         _ptr(offsets), rows_cap, n, k, _ptr(out), out_dtype,
                                         _ptr(workspace),
                                         workspace.numel() * workspace.element_size(),
                                         _ptr(status), _stream(a)))
        return out
    _check(lib.grouped_gemm_mxfp8(mode, G, _ptr(a), _ptr(a_scales), _ptr(b), _ptr(b_scales),
                                  _ptr(offsets), rows_cap, n, k, _ptr(out), out_dtype, _ptr(status),
                                  _stream(a)))
    return out


def grouped_gemm_mxfp8_ex(mode, a, a_scales, b, b_scales, offsets, rows_cap, n, k, out,
                          out_dtype=BSG_OUT_BF16, alpha=None, beta=None, bias=None, G=None,
                          status=None):
    """grouped_gemm_mxfp8 with out = alpha[g] * S + beta[g] * out + bias[g]
    (float32 [G] alpha / beta, [G, output columns] bias; None = 1 / 0 / none).
    `out` is required (it is read where beta != 0).  See include/bsg.h."""
    lib = load_library()
    _need_cuda(a, a_scales, b, b_scales, offsets, out)
    G = offsets.numel() - 1 if G is None else G
    _mx_gemm_check(mode, G, a, a_scales, b, b_scales, offsets, rows_cap, n, k, out, out_dtype,
                   status)
    _req(alpha, "alpha", 4 * G, _f32(), optional=True)
    _req(beta, "beta", 4 * G, _f32(), optional=True)
    _req(bias, "bias", 4 * G * (k if mode in (BSG_WGRAD_NT, BSG_WGRAD_NT_E5M2) else n), _f32(),
         optional=True)
    _check(lib.grouped_gemm_mxfp8_ex(mode, G, _ptr(a), _ptr(a_scales), _ptr(b), _ptr(b_scales),
                                     _ptr(offsets), rows_cap, n, k, _ptr(out), out_dtype,
                                     _ptr(alpha), _ptr(beta), _ptr(bias), _ptr(status),
                                     _stream(a)))
    return out


def _nv_gemm_check(G, a, a_scales, a_outer, offsets, rows_cap, k, b, b_scales, b_outer, npg, out,
                   ld_out, out_dtype, status, per_tensor):
    nb = sum(npg)
    _req(a, "a", rows_cap * k // 2)
    _req(a_scales, "a_scales", rows_cap * k // 16)
    _req(a_outer, "a_amax" if per_tensor else "a_outer", 4 * (G if per_tensor else rows_cap),
         _f32())
    _req(offsets, "offsets", 8 * (G + 1), _i64())
    _req(b, "b", nb * k // 2)
    _req(b_scales, "b_scales", nb * k // 16)
    _req(b_outer, "b_amax" if per_tensor else "b_outer", 4 * (G if per_tensor else nb), _f32())
    dt, esz = _out_dtype(out_dtype)
    _req(out, "out", esz * rows_cap * ld_out, dt)
    _req(status, "status", 4, optional=True)


def grouped_gemm_nvfp4_rowscaled(a, a_scales, a_outer, offsets, k, b, b_scales, b_outer,
                                 n_per_group, out=None, ld_out=None, out_dtype=BSG_OUT_BF16,
                                 scratch=None, G=None, status=None, accumulate=False,
                                 workspace=None):
    """Row-scaled NVFP4 fprop: out [rows_cap, ld_out]; n_per_group is a host list.
    accumulate=True adds Y to out's previous contents (grouped_gemm_nvfp4_rowscaled_ex).
    With a `workspace` (gemm_workspace(), fused epilogue only),
    grouped_gemm_nvfp4_rowscaled_ws: the last round of tiles is split along the
    contraction."""
    import torch
    lib = load_library()
    _need_cuda(a, a_scales, a_outer, offsets, b, b_scales, b_outer)
    rows_cap = a.shape[0]
    G = offsets.numel() - 1 if G is None else G
    npg = [int(v) for v in n_per_group]
    if len(npg) != G:
        raise ValueError("n_per_group needs G entries")
    if ld_out is None:
        ld_out = max(npg) if out is None else out.shape[1]
    if out is None:
        dt = _out_dtype(out_dtype)[0]
        out = torch.empty((rows_cap, ld_out), dtype=dt, device=a.device)
    _nv_gemm_check(G, a, a_scales, a_outer, offsets, rows_cap, k, b, b_scales, b_outer, npg, out,
                   ld_out, out_dtype, status, per_tensor=False)
    _req(scratch, "scratch", 4 * rows_cap * ld_out, torch.float32, optional=True)
    host_n = (ctypes.c_int64 * G)(*npg)
    if workspace is not None:
        if scratch is not None:
            raise ValueError("a workspace serves the fused epilogue only (no scratch)")
        _need_cuda(workspace)
        _check(lib.grouped_gemm_nvfp4_rowscaled_ws(
            G, _ptr(a), _ptr(a_scales), _ptr(a_outer), _ptr(offsets), rows_cap, k, _ptr(b),
            _ptr(b_scales), _ptr(b_outer), ctypes.cast(host_n, ctypes.c_void_p), _ptr(out), ld_out,
            out_dtype, 1 if accumulate else 0, _ptr(workspace),
            workspace.nbytes, _ptr(status), _stream(a)))
        return out
    if accumulate:
        _check(lib.grouped_gemm_nvfp4_rowscaled_ex(
            G, _ptr(a), _ptr(a_scales), _ptr(a_outer), _ptr(offsets), rows_cap, k, _ptr(b),
            _ptr(b_scales), _ptr(b_outer), ctypes.cast(host_n, ctypes.c_void_p), _ptr(out), ld_out,
            out_dtype, _ptr(scratch), 1, _ptr(status), _stream(a)))
        return out
    _check(lib.grouped_gemm_nvfp4_rowscaled(G, _ptr(a), _ptr(a_scales), _ptr(a_outer),
                                            _ptr(offsets), rows_cap, k, _ptr(b), _ptr(b_scales),
                                            _ptr(b_outer), ctypes.cast(host_n, ctypes.c_void_p),
                                            _ptr(out), ld_out, out_dtype, _ptr(scratch),
                                            _ptr(status), _stream(a)))
    return out


def grouped_gemm_nvfp4_rowscaled_noalloc(a, a_scales, a_outer, offsets, k, b, b_scales, b_outer,
                                         n_per_group, out, ld_out=None, out_dtype=BSG_OUT_BF16,
                                         G=None, status=None):
    """grouped_gemm_nvfp4_rowscaled's two-step (FP32 S) flow with S in the
    library's static device scratch: allocates nothing, so `out` is required.
    rows_cap * ld_out * 4 must fit BSG_NOALLOC_SCRATCH_BYTES; calls that overlap
    on one GPU race.  See include/bsg.h."""
    lib = load_library()
    _need_cuda(a, a_scales, a_outer, offsets, b, b_scales, b_outer, out)
    rows_cap = a.shape[0]
    G = offsets.numel() - 1 if G is None else G
    npg = [int(v) for v in n_per_group]
    if len(npg) != G:
        raise ValueError("n_per_group needs G entries")
    if ld_out is None:
        ld_out = out.shape[1]
    _nv_gemm_check(G, a, a_scales, a_outer, offsets, rows_cap, k, b, b_scales, b_outer, npg, out,
                   ld_out, out_dtype, status, per_tensor=False)
    host_n = (ctypes.c_int64 * G)(*npg)
    _check(lib.grouped_gemm_nvfp4_rowscaled_noalloc(
        G, _ptr(a), _ptr(a_scales), _ptr(a_outer), _ptr(offsets), rows_cap, k, _ptr(b),
        _ptr(b_scales), _ptr(b_outer), ctypes.cast(host_n, ctypes.c_void_p), _ptr(out), ld_out,
        out_dtype, _ptr(status), _stream(a)))
    return out


def grouped_gemm_nvfp4_pertensor(a, a_scales, a_amax, offsets, k, b, b_scales, b_amax, n_per_group,
                                 out=None, ld_out=None, out_dtype=BSG_OUT_BF16, G=None,
                                 status=None, workspace=None):
    """Per-tensor NVFP4 fprop (alpha per group from the two amax arrays): out
    [rows_cap, ld_out]; n_per_group is a host list.  With a `workspace`
    (gemm_workspace()), grouped_gemm_nvfp4_pertensor_ws: the last round of tiles
    is split along the contraction."""
    import torch
    lib = load_library()
    _need_cuda(a, a_scales, a_amax, offsets, b, b_scales, b_amax)
    rows_cap = a.shape[0]
    G = offsets.numel() - 1 if G is None else G
    npg = [int(v) for v in n_per_group]
    if len(npg) != G:
        raise ValueError("n_per_group needs G entries")
    if ld_out is None:
        ld_out = max(npg) if out is None else out.shape[1]
    if out is None:
        dt = _out_dtype(out_dtype)[0]
        out = torch.empty((rows_cap, ld_out), dtype=dt, device=a.device)
    _nv_gemm_check(G, a, a_scales, a_amax, offsets, rows_cap, k, b, b_scales, b_amax, npg, out,
                   ld_out, out_dtype, status, per_tensor=True)
    host_n = (ctypes.c_int64 * G)(*npg)
    if workspace is not None:
        _need_cuda(workspace)
        _check(lib.grouped_gemm_nvfp4_pertensor_ws(
            G, _ptr(a), _ptr(a_scales), _ptr(a_amax), _ptr(offsets), rows_cap, k, _ptr(b),
            _ptr(b_scales), _ptr(b_amax), ctypes.cast(host_n, ctypes.c_void_p), _ptr(out), ld_out,
            out_dtype, _ptr(workspace), workspace.nbytes, _ptr(status),
            _stream(a)))
        return out
    _check(lib.grouped_gemm_nvfp4_pertensor(G, _ptr(a), _ptr(a_scales), _ptr(a_amax),
                                            _ptr(offsets), rows_cap, k, _ptr(b), _ptr(b_scales),
                                            _ptr(b_amax), ctypes.cast(host_n, ctypes.c_void_p),
                                            _ptr(out), ld_out, out_dtype, _ptr(status),
                                            _stream(a)))
    return out


def grouped_gemm_nvfp4_rowscaled_wgrad(a, a_scales, a_outer, b, b_scales, b_outer, padded_offsets,
                                       n, k, col_rows_cap=None, out=None, out_dtype=BSG_OUT_BF16,
                                       G=None, status=None, accumulate=False):
    """Row-scaled NVFP4 wgrad from the columnwise copies: out [G, n, k];
    accumulate=True adds to out's previous contents
    (grouped_gemm_nvfp4_rowscaled_wgrad_ex).  See include/bsg.h."""
    import torch
    lib = load_library()
    _need_cuda(a, a_scales, a_outer, b, b_scales, b_outer, padded_offsets)
    G = padded_offsets.numel() - 1 if G is None else G
    if col_rows_cap is None:
        col_rows_cap = a.numel() * 2 // n
    if out is None:
        dt = _out_dtype(out_dtype)[0]
        out = torch.empty((G, n, k), dtype=dt, device=a.device)
    _req(a, "a", col_rows_cap * n // 2)
    _req(a_scales, "a_scales", col_rows_cap * n // 16)
    _req(a_outer, "a_outer", 4 * G * n, torch.float32)
    _req(b, "b", col_rows_cap * k // 2)
    _req(b_scales, "b_scales", col_rows_cap * k // 16)
    _req(b_outer, "b_outer", 4 * G * k, torch.float32)
    _req(padded_offsets, "padded_offsets", 8 * (G + 1), torch.int64)
    dt, esz = _out_dtype(out_dtype)
    _req(out, "out", esz * G * n * k, dt)
    _req(status, "status", 4, optional=True)
    if accumulate:
        _check(lib.grouped_gemm_nvfp4_rowscaled_wgrad_ex(
            G, _ptr(a), _ptr(a_scales), _ptr(a_outer), _ptr(b), _ptr(b_scales), _ptr(b_outer),
            _ptr(padded_offsets), col_rows_cap, n, k, _ptr(out), out_dtype, 1, _ptr(status),
            _stream(a)))
        return out
    _check(lib.grouped_gemm_nvfp4_rowscaled_wgrad(
        G, _ptr(a), _ptr(a_scales), _ptr(a_outer), _ptr(b), _ptr(b_scales), _ptr(b_outer),
        _ptr(padded_offsets), col_rows_cap, n, k, _ptr(out), out_dtype, _ptr(status), _stream(a)))
    return out


def _types_16bit(t, name, out_dtype, like=None):
    """(in_dtype, out_dtype code, torch output type) of a 16-bit operand; out_dtype None: its own
    or, where there is one, that of `like` (an addend or an output)."""
    import torch
    if out_dtype is None and like is not None and like.dtype == torch.float32:
        out_dtype = BSG_OUT_F32
    if t.dtype == torch.bfloat16:
        code, same = BSG_IN_BF16, BSG_OUT_BF16
    elif t.dtype == torch.float16:
        code, same = BSG_IN_F16, BSG_OUT_F16
    else:
        raise ValueError("%s must be bfloat16 or float16, not %s" % (name, _dtype_name(t.dtype)))
    if out_dtype is None or out_dtype == same:
        return code, same, t.dtype
    if out_dtype == BSG_OUT_F32:
        return code, out_dtype, torch.float32
    raise ValueError("out_dtype %r is neither the operands' type nor BSG_OUT_F32" % (out_dtype,))


def _strided(t, name, dims, dtype, index):
    """Row (and matrix) strides of a tensor on device `index` whose rows are contiguous: (ld,
    stride).  A size-1 dimension's stride is never used and torch leaves it arbitrary, so a
    dense one stands in."""
    if t.dim() != dims:
        raise ValueError("%s must be %d-D, not %d-D" % (name, dims, t.dim()))
    if t.get_device() != index:
        raise ValueError("%s must be a device tensor, on cuda:%d" % (name, index) if index >= 0
                         else "%s must be a device tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, not %s" % (name, _dtype_name(dtype), _dtype_name(t.dtype)))
    if dims == 2:
        (rows, cols), (ld, one) = t.shape, t.stride()
    else:
        (groups, rows, cols), (stride, ld, one) = t.shape, t.stride()
    if one != 1 and cols > 1:
        raise ValueError("the rows of %s must be contiguous" % name)
    if rows <= 1:
        ld = max(cols, 1)
    if dims == 2:
        return ld, 0
    return ld, (stride if groups > 1 else rows * ld)


def _dense(t, name, nbytes, dtype, index):
    """_req for a tensor that has to be on device `index`; returns its address."""
    if t.dtype != dtype or t.get_device() != index or not t.is_contiguous() or t.nbytes < nbytes:
        _req(t, name, nbytes, dtype)
        raise ValueError("%s is on %s, not on cuda:%d" % (name, t.device, index))
    return t.data_ptr()


def _device_index(t, name):
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    return t.get_device()


def _same_device(ref, **others):
    index = ref.get_device()
    for name, t in others.items():
        if t is not None and t.get_device() != index:
            raise ValueError("%s is on %s, not on %s" % (name, t.device, ref.device))


def _out_or_new(out, shape, dtype, ref, name="out"):
    if out is None:
        return ref.new_empty(shape, dtype=dtype)
    if tuple(out.shape) != tuple(shape):
        raise ValueError("%s is %s; the call writes %s" % (name, tuple(out.shape), tuple(shape)))
    return out


def grouped_gemm_16bit(mode, a, b, offsets, c=None, out=None, out_dtype=None, workspace=None,
                       status=None):
    """Grouped products of bf16 or fp16 operands over the row groups of `offsets`:

    BSG_FPROP_TN  a [rows, k], b [G, n, k]  -> [rows, n]: group g's rows times b[g]^T
    BSG_DGRAD_NN  a [rows, k], b [G, k, n]  -> [rows, n]: group g's rows times b[g]
    BSG_WGRAD_NT  a [rows, n], b [rows, k]  -> [G, n, k]: a^T b over group g's rows

    c: an addend in the output's type and shape (pass the same tensor as `out` to
    accumulate).  out_dtype: the operands' type or BSG_OUT_F32; None takes that of `out`
    or `c` where given, else the operands'.  Rows may be strided (strides multiples of 8
    elements).  See include/bsg.h."""
    import torch
    lib = load_library()
    code, od, odt = _types_16bit(a, "a", out_dtype, out if out is not None else c)
    dt, dev = a.dtype, _device_index(a, "a")
    lda, _ = _strided(a, "a", 2, dt, dev)
    off = _dense(offsets, "offsets", 16, torch.int64, dev)
    G = offsets.numel() - 1
    rows, acols = a.shape
    if mode == BSG_WGRAD_NT:
        ldb, stride_b = _strided(b, "b", 2, dt, dev)
        n, k = acols, b.shape[1]
        if b.shape[0] != rows:
            raise ValueError("a has %d rows, b has %d" % (rows, b.shape[0]))
        shape = (G, n, k)
    elif mode == BSG_FPROP_TN or mode == BSG_DGRAD_NN:
        ldb, stride_b = _strided(b, "b", 3, dt, dev)
        k = acols
        groups, n, bk = b.shape
        if mode == BSG_DGRAD_NN:
            n, bk = bk, n
        if groups != G or bk != k:
            raise ValueError("b is %s; %d groups contracting %d are needed" % (tuple(b.shape), G, k))
        shape = (rows, n)
    else:
        raise ValueError("mode %r has no 16-bit product" % (mode,))
    out = _out_or_new(out, shape, odt, a)
    ldo, stride_o = _strided(out, "out", len(shape), odt, dev)
    if c is not None:
        if tuple(c.shape) != shape:
            raise ValueError("c is %s; the output is %s" % (tuple(c.shape), shape))
        if _strided(c, "c", len(shape), odt, dev) != (ldo, stride_o):
            raise ValueError("c must have the strides of out")
    if n == 0 or k == 0:
        raise ValueError("n and k must be positive")
    optr = out.data_ptr()
    _check(lib.grouped_gemm_16bit(
        mode, code, G, a.data_ptr() or optr, lda, b.data_ptr() or optr, ldb, stride_b, off, rows, n,
        k, None if c is None else c.data_ptr(), optr, ldo, stride_o, od,
        None if workspace is None else _dense(workspace, "workspace", 0, workspace.dtype, dev),
        0 if workspace is None else workspace.nbytes,
        None if status is None else _dense(status, "status", 4, status.dtype, dev),
        _stream(a)) if optr else 0)
    return out


def grouped_gemm_16bit_tile_rows(mode, groups, rows_cap, n, k, workspace=True):
    """Rows of the output tiles (32, 64, 128 or 256) that grouped_gemm_16bit takes for these
    sizes on the current device.  It goes by rows_cap, the rows of the tensors, however few of
    them the offsets leave live: pass a view of the rows that can be live."""
    rows = load_library().grouped_gemm_16bit_tile_rows(mode, groups, rows_cap, n, k, 1 if workspace else 0)
    if rows == 0:
        raise ValueError("no 16-bit product of mode %r, %r groups, rows_cap=%r, n=%r, k=%r" % (
            mode, groups, rows_cap, n, k))
    return rows


def grouped_lora_gemm_16bit_tile_rows(rows_cap, n, k):
    """As grouped_gemm_16bit_tile_rows, for grouped_lora_gemm_16bit."""
    rows = load_library().grouped_lora_gemm_16bit_tile_rows(rows_cap, n, k)
    if rows == 0:
        raise ValueError("no adapted projection of rows_cap=%r, n=%r, k=%r" % (rows_cap, n, k))
    return rows


def grouped_lora_gemm_16bit_workspace(rows_cap, n, k, rank, device=None):
    """A uint8 device tensor for the `workspace` argument of grouped_lora_gemm_16bit, with
    up to rows_cap rows and a rank of up to `rank`.  Calls that may run at the same time (on
    different streams) need a workspace each."""
    import torch
    nbytes = int(load_library().grouped_lora_gemm_16bit_workspace_size(rows_cap, n, k, rank))
    if nbytes == 0:
        raise ValueError("no workspace for rows_cap=%r, n=%r, k=%r, rank=%r" % (rows_cap, n, k, rank))
    return torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")


def grouped_lora_gemm_16bit(x, w, lora_a, lora_b, offsets, adapter, scale, out=None, out_dtype=None,
                            workspace=None, status=None):
    """x w^T plus, for the rows of request g (offsets[g] .. offsets[g+1]) with adapter
    a = adapter[g] >= 0, scale[a] (x lora_a[a]^T) lora_b[a]^T -> [rows, n].

    x [rows, k], w [n, k] (rows may be strided), lora_a [adapters, rank, k] and lora_b
    [adapters, n, rank] of one 16-bit type; adapter int32 [G], scale float32 [adapters].
    workspace: grouped_lora_gemm_16bit_workspace(rows, n, k, rank), or None for a new
    one (some 67 MB a call).  See include/bsg.h."""
    import torch
    lib = load_library()
    code, od, odt = _types_16bit(x, "x", out_dtype, out)
    dt, dev = x.dtype, _device_index(x, "x")
    ldx, _ = _strided(x, "x", 2, dt, dev)
    ldw, _ = _strided(w, "w", 2, dt, dev)
    (rows, k), (n, wk) = x.shape, w.shape
    if lora_a.dim() != 3 or lora_b.dim() != 3:
        raise ValueError("lora_a and lora_b must be 3-D")
    count, rank, ak = lora_a.shape
    if wk != k or ak != k or tuple(lora_b.shape) != (count, n, rank):
        raise ValueError("x %s, w %s, lora_a %s and lora_b %s do not fit" % (
            tuple(x.shape), tuple(w.shape), tuple(lora_a.shape), tuple(lora_b.shape)))
    G = offsets.numel() - 1
    out = _out_or_new(out, (rows, n), odt, x)
    ldo, _ = _strided(out, "out", 2, odt, dev)
    if workspace is None:
        workspace = grouped_lora_gemm_16bit_workspace(rows, n, k, rank, x.device)
    args = (_dense(lora_a, "lora_a", 0, dt, dev), _dense(lora_b, "lora_b", 0, dt, dev), count, rank,
            _dense(offsets, "offsets", 16, torch.int64, dev),
            _dense(adapter, "adapter", 4 * G, torch.int32, dev),
            _dense(scale, "scale", 4 * count, torch.float32, dev), rows, n, k, out.data_ptr(), ldo, od,
            _dense(workspace, "workspace", 0, workspace.dtype, dev), workspace.nbytes,
            None if status is None else _dense(status, "status", 4, status.dtype, dev), _stream(x))
    if rows:
        _check(lib.grouped_lora_gemm_16bit(code, G, x.data_ptr(), ldx, w.data_ptr(), ldw, *args))
    return out


class GradClipPlan:
    """The chunk table of a set of gradients on the device, and the workspace of its calls.

    Valid while the tensors stay where they are; it keeps them alive.  Calls on one plan
    share its workspace: run them on one stream at a time."""

    def __init__(self, tensors, outs, table, num_chunks, workspace):
        self.tensors, self.outs = tensors, outs
        self.table, self.num_chunks, self.workspace = table, num_chunks, workspace


def grad_clip_plan(tensors, outs=None, device=None):
    """Plan for grad_norm and clip_grad_norm over contiguous bf16, fp16 or float32 device
    tensors (any number, any sizes, aligned to their elements).  outs: where the clipped
    gradients go (same types and sizes); None clips in place.  An output may share memory
    with its own tensor only, so a tensor that is used twice (tied weights) is listed once.
    device: needed only where there are no tensors."""
    import torch
    lib = load_library()
    tensors = list(tensors)
    outs = tensors if outs is None else list(outs)
    if len(outs) != len(tensors):
        raise ValueError("%d tensors and %d outputs" % (len(tensors), len(outs)))
    codes = {torch.bfloat16: BSG_GRAD_BF16, torch.float16: BSG_GRAD_F16, torch.float32: BSG_GRAD_F32}
    for i, (t, o) in enumerate(zip(tensors, outs)):
        _req(t, "tensor %d" % i, 0, tuple(codes))
        _req(o, "output %d" % i, 0, t.dtype)
        if o.numel() != t.numel():
            raise ValueError("tensor %d has %d elements, its output %d" % (i, t.numel(), o.numel()))
        _same_device(tensors[0], **{"tensor %d" % i: t, "output %d" % i: o})
    count = len(tensors)
    src = (ctypes.c_void_p * max(count, 1))(*[t.data_ptr() for t in tensors])
    dst = (ctypes.c_void_p * max(count, 1))(*[o.data_ptr() for o in outs])
    numels = (ctypes.c_int64 * max(count, 1))(*[t.numel() for t in tensors])
    dtypes = (ctypes.c_int32 * max(count, 1))(*[codes[t.dtype] for t in tensors])
    chunks = ctypes.c_int64(0)
    _check(lib.grad_clip_plan_fill(count, src, dst, numels, dtypes, None, 0, ctypes.byref(chunks)))
    nbytes = 24 * max(chunks.value, 1)
    table = torch.zeros(nbytes, dtype=torch.uint8)
    _check(lib.grad_clip_plan_fill(count, src, dst, numels, dtypes,
                                   ctypes.c_void_p(table.data_ptr()), nbytes, ctypes.byref(chunks)))
    dev = tensors[0].device if tensors else torch.device(device or "cuda")
    workspace = torch.empty(int(lib.grad_clip_workspace_size()), dtype=torch.uint8, device=dev)
    return GradClipPlan(tensors, outs, table.to(dev), chunks.value, workspace)


def _grad_outputs(plan, norm, status):
    import torch
    if norm is None:
        norm = torch.empty((), dtype=torch.float32, device=plan.table.device)
    _req(norm, "norm", 4, torch.float32)
    _req(status, "status", 4, optional=True)
    _same_device(plan.table, norm=norm, status=status)
    return norm


def grad_norm(plan, norm=None, sumsq=None, status=None):
    """The 2-norm over all tensors of the plan (float32 scalar tensor).  sumsq: a float64
    tensor that receives the sum of squares too (for sums over ranks)."""
    import torch
    norm = _grad_outputs(plan, norm, status)
    _req(sumsq, "sumsq", 8, torch.float64, optional=True)
    _same_device(plan.table, sumsq=sumsq)
    _check(load_library().grad_norm(_ptr(plan.table), plan.num_chunks, _ptr(plan.workspace),
                                    plan.workspace.numel(), _ptr(norm), _ptr(sumsq), _ptr(status),
                                    _stream(plan.table)))
    return norm


def clip_grad_norm(plan, max_norm, sumsq=None, norm=None, status=None):
    """Scales the plan's tensors by min(1, max_norm / (norm + 1e-6)) into its outputs and
    returns the norm before it.  sumsq: a float64 tensor holding the sum of squares to go
    by (e.g. grad_norm's, added over ranks); None computes it."""
    import torch
    norm = _grad_outputs(plan, norm, status)
    _req(sumsq, "sumsq", 8, torch.float64, optional=True)
    _same_device(plan.table, sumsq=sumsq)
    _check(load_library().clip_grad_norm(_ptr(plan.table), plan.num_chunks, max_norm, _ptr(sumsq),
                                         _ptr(plan.workspace), plan.workspace.numel(), _ptr(norm),
                                         _ptr(status), _stream(plan.table)))
    return norm


def _launch(fn, index, *args):
    """fn(*args, stream) on device `index`, on its current stream; kernels are launched on the
    device that is current."""
    import torch
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            _check(fn(*args, torch._C._cuda_getCurrentRawStream(index)))
    else:
        _check(fn(*args, torch._C._cuda_getCurrentRawStream(index)))


_makers = {}


def _maker(index, dtype):
    """new_empty of a tensor of that type on device `index`: a call of it without a type takes half a
    microsecond less than one with a type, which is a good part of a small call."""
    make = _makers.get((index, dtype))
    if make is None:
        import torch
        make = torch.empty(0, dtype=dtype, device=torch.device("cuda", index)).new_empty
        _makers[index, dtype] = make
    return make


def _maybe(t, name, nbytes, dtype, index):
    """_dense for a tensor that may be left out."""
    return None if t is None else _dense(t, name, nbytes, dtype, index)


def _rows(t, name, dtype, index):
    """(row stride, rows, columns) of a 2-D tensor on device `index` whose rows are contiguous."""
    if t.dtype is dtype and t.get_device() == index and t.is_contiguous() and t.dim() == 2:
        rows, cols = t.shape
        return cols or 1, rows, cols
    ld, _ = _strided(t, name, 2, dtype, index)
    return ld, t.shape[0], t.shape[1]


def _output(t, rows, cols, dtype, index, name="out"):
    """(tensor [rows, cols], row stride): a new one, or the given one after its checks."""
    if t is None:
        return _maker(index, dtype)(rows, cols), cols
    ld, r, c = _rows(t, name, dtype, index)
    if r != rows or c != cols:
        raise ValueError("%s is %s; the call writes %s" % (name, tuple(t.shape), (rows, cols)))
    return t, ld


def _buffer(t, rows, cols, dtype, index, name):
    """(tensor, address) of a dense output [rows, cols] or, without cols, [rows]."""
    if t is None:
        make = _maker(index, dtype)
        t = make(rows) if cols is None else make(rows, cols)
        return t, t.data_ptr()
    return t, _dense(t, name, rows * (cols or 1) * t.element_size(), dtype, index)


def _status(t, index):
    return None if t is None else _dense(t, "status", 4, t.dtype, index)


def _router_args(logits, mask, index):
    """(in_dtype, row stride, tokens, experts, the mask's address)"""
    import torch
    dtype = logits.dtype
    code = (BSG_IN_F32 if dtype is torch.float32 else BSG_IN_BF16 if dtype is torch.bfloat16
            else BSG_IN_F16 if dtype is torch.float16 else None)
    if code is None:
        raise ValueError("logits must be bfloat16, float16 or float32, not %s" % _dtype_name(dtype))
    ld, tokens, experts = _rows(logits, "logits", dtype, index)
    m = None
    if mask is not None:
        if mask.dtype not in (torch.bool, torch.uint8):
            raise ValueError("mask must be bool or uint8, not %s" % _dtype_name(mask.dtype))
        m = _dense(mask, "mask", tokens, mask.dtype, index)
    return code, ld, tokens, experts, m


def moe_router_topk_workspace(tokens, experts, device=None):
    """A uint8 device tensor for the `workspace` argument of moe_router_topk, with up to that many
    tokens and experts.  Calls that may run at the same time need a workspace each."""
    import torch
    nbytes = int(load_library().moe_router_topk_workspace_size(tokens, experts))
    if nbytes == 0:
        raise ValueError("no workspace for %r tokens and %r experts" % (tokens, experts))
    return torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")


def moe_router_topk(logits, top_k, mask=None, normalize=True, workspace=None, status=None):
    """Each token's top_k of the experts by its logits [tokens, experts] (bf16, fp16 or float32; rows
    may be strided), and what balances them.  mask [tokens] (bool or uint8): tokens to route.  Returns

    experts    int32 [tokens, top_k], in descending order (ties: the lowest index first; -1: none)
    weights    float32 [tokens, top_k]: softmax probabilities; normalize: over the chosen ones' sum
    counts     int32 [experts]: the sizes that group_offsets_i32_to_i64 takes
    prob_sums  float32 [experts], live int32 [1]: sums over the tokens that are routed
    loss       float32 [1]: experts / (top_k live^2) * sum(counts * prob_sums)

    as a dict.  See include/bsg.h."""
    import torch
    lib = load_library()
    dev = _device_index(logits, "logits")
    code, ld, tokens, E, m = _router_args(logits, mask, dev)
    if workspace is None:
        workspace = moe_router_topk_workspace(tokens, max(E, 1), logits.device)
    ints, floats = _maker(dev, torch.int32), _maker(dev, torch.float32)
    experts, weights, counts = ints(tokens, top_k), floats(tokens, top_k), ints(E)
    prob_sums, live, loss = floats(E), ints(1), floats(1)
    _launch(lib.moe_router_topk, dev, code, logits.data_ptr(), ld, tokens, E, top_k, m,
            1 if normalize else 0, experts.data_ptr(), weights.data_ptr(), counts.data_ptr(),
            prob_sums.data_ptr(), live.data_ptr(), loss.data_ptr(),
            _dense(workspace, "workspace", 0, workspace.dtype, dev), workspace.nbytes,
            _status(status, dev))
    return {"experts": experts, "weights": weights, "counts": counts, "prob_sums": prob_sums,
            "live": live, "loss": loss}


def moe_router_topk_backward(logits, experts, counts, live, d_weights=None, d_loss=None, mask=None,
                             normalize=True, out=None):
    """d_logits of sum(d_weights * weights) + d_loss * loss, with the experts and counts that
    moe_router_topk gave (counts and live may be sums over ranks).  d_weights float32
    [tokens, top_k], d_loss float32 [1] on the device; either may be left out.  out: not logits."""
    import torch
    lib = load_library()
    dev = _device_index(logits, "logits")
    code, ld, tokens, E, m = _router_args(logits, mask, dev)
    if experts.dim() != 2 or experts.shape[0] != tokens:
        raise ValueError("experts is %s, the logits have %d rows" % (tuple(experts.shape), tokens))
    top_k = experts.shape[1]
    if d_weights is not None and tuple(d_weights.shape) != (tokens, top_k):
        raise ValueError("d_weights is %s, experts %s" % (tuple(d_weights.shape), (tokens, top_k)))
    out, ldo = _output(out, tokens, E, logits.dtype, dev)
    args = (_dense(experts, "experts", 4 * tokens * top_k, torch.int32, dev),
            _maybe(d_weights, "d_weights", 4 * tokens * top_k, torch.float32, dev),
            _dense(counts, "counts", 4 * E, torch.int32, dev), _dense(live, "live", 4, torch.int32, dev),
            _maybe(d_loss, "d_loss", 4, torch.float32, dev), out.data_ptr(), ldo)
    if tokens:
        _launch(lib.moe_router_topk_backward, dev, code, logits.data_ptr(), ld, tokens, E, top_k, m,
                1 if normalize else 0, *args)
    return out


def _in_16bit(t, name):
    import torch
    if t.dtype is torch.bfloat16:
        return BSG_IN_BF16
    if t.dtype is torch.float16:
        return BSG_IN_F16
    raise ValueError("%s must be bfloat16 or float16, not %s" % (name, _dtype_name(t.dtype)))


def grouped_quantize_int8(x, offsets=None, data=None, scales=None, status=None):
    """Rows of x [rows, cols] (bf16 or fp16; rows may be strided) in 8-bit integers with a float32
    scale each: (data int8 [rows, cols], scales [rows]).  offsets: only rows in
    [offsets[0], offsets[-1]); None: all.  Weights [G, n, k] go in as G * n rows."""
    import torch
    lib = load_library()
    code, dev = _in_16bit(x, "x"), _device_index(x, "x")
    ld, rows, cols = _rows(x, "x", x.dtype, dev)
    data, dptr = _buffer(data, rows, cols, torch.int8, dev, "data")
    scales, sptr = _buffer(scales, rows, None, torch.float32, dev, "scales")
    off, G = None, 0
    if offsets is not None:
        off, G = _dense(offsets, "offsets", 16, torch.int64, dev), offsets.numel() - 1
    st = _status(status, dev)
    if rows:
        _launch(lib.grouped_quantize_int8, dev, code, x.data_ptr(), ld, rows, cols, G, off, dptr, sptr, st)
    return data, scales


def _int8_weights(w, w_scales, offsets, k, index):
    """(groups, n, row stride, group stride, addresses of the scales and offsets) of an int8
    product's checked weights."""
    import torch
    ldw, stride_w = _strided(w, "w", 3, torch.int8, index)
    G, n, wk = w.shape
    if offsets.numel() - 1 != G or wk != k:
        raise ValueError("w is %s; %d groups contracting %d are needed" % (
            tuple(w.shape), offsets.numel() - 1, k))
    return (G, n, ldw, stride_w, _dense(w_scales, "w_scales", 4 * G * n, torch.float32, index),
            _dense(offsets, "offsets", 16, torch.int64, index))


def _int8_output(out, rows, n, out_dtype, default, index):
    """(out, row stride, out_dtype): out_dtype None is that of `out` or, without one, the default."""
    import torch
    codes = {torch.bfloat16: BSG_OUT_BF16, torch.float16: BSG_OUT_F16, torch.float32: BSG_OUT_F32}
    if out_dtype is None:
        out_dtype = default if out is None else codes.get(out.dtype)
    odt = (torch.bfloat16 if out_dtype == BSG_OUT_BF16 else torch.float16 if out_dtype == BSG_OUT_F16
           else torch.float32 if out_dtype == BSG_OUT_F32 else None)
    if odt is None:
        raise ValueError("out_dtype %r is not BSG_OUT_BF16, BSG_OUT_F16 or BSG_OUT_F32" % (out_dtype,))
    return _output(out, rows, n, odt, index) + (out_dtype,)


def grouped_gemm_int8(a, a_scales, w, w_scales, offsets, out=None, out_dtype=None, workspace=None,
                      status=None):
    """Group g's rows of a [rows, k] int8 times w[g]^T (w [G, n, k] int8), each times its row's scale
    and its channel's: a_scales float32 [rows], w_scales float32 [G, n] -> [rows, n].  out_dtype:
    BSG_OUT_BF16 (default), BSG_OUT_F16 or BSG_OUT_F32.  workspace: gemm_workspace(), or None
    (no contraction is split).  See include/bsg.h."""
    import torch
    lib = load_library()
    dev = _device_index(a, "a")
    lda, rows, k = _rows(a, "a", torch.int8, dev)
    G, n, ldw, stride_w, sptr, off = _int8_weights(w, w_scales, offsets, k, dev)
    out, ldo, od = _int8_output(out, rows, n, out_dtype, BSG_OUT_BF16, dev)
    scales = _dense(a_scales, "a_scales", 4 * rows, torch.float32, dev)
    ws, nbytes = None, 0
    if workspace is not None:
        ws, nbytes = _dense(workspace, "workspace", 0, workspace.dtype, dev), workspace.nbytes
    st = _status(status, dev)
    if rows:
        _launch(lib.grouped_gemm_int8, dev, G, a.data_ptr(), lda, scales, w.data_ptr(), ldw, stride_w,
                sptr, off, rows, n, k, out.data_ptr(), ldo, od, ws, nbytes, st)
    return out


def grouped_gemm_int8_tile_rows(groups, rows_cap, n, k, workspace=True):
    """As grouped_gemm_16bit_tile_rows, for grouped_gemm_int8 and grouped_gemm_int8_dynamic."""
    rows = load_library().grouped_gemm_int8_tile_rows(groups, rows_cap, n, k, 1 if workspace else 0)
    if rows == 0:
        raise ValueError("no int8 product of %r groups, rows_cap=%r, n=%r, k=%r" % (groups, rows_cap, n, k))
    return rows


def grouped_gemm_int8_dynamic_workspace(rows_cap, k, device=None):
    """A uint8 device tensor for the `workspace` argument of grouped_gemm_int8_dynamic, with up to
    rows_cap rows and a contraction of up to k.  Calls that may run at the same time need a
    workspace each."""
    import torch
    nbytes = int(load_library().grouped_gemm_int8_dynamic_workspace_size(rows_cap, k))
    if nbytes == 0:
        raise ValueError("no workspace for rows_cap=%r, k=%r" % (rows_cap, k))
    return torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")


def grouped_gemm_int8_dynamic(x, w, w_scales, offsets, out=None, out_dtype=None, workspace=None,
                              status=None):
    """grouped_gemm_int8 of 16-bit tokens x [rows, k] (bf16 or fp16; rows may be strided), quantized
    on the way as grouped_quantize_int8 does.  out_dtype: None for the type of `out` or, without
    one, of x.  workspace: grouped_gemm_int8_dynamic_workspace(rows, k), or None for a new one
    (some 67 MB and the tokens' integers a call)."""
    lib = load_library()
    code, dev = _in_16bit(x, "x"), _device_index(x, "x")
    ldx, rows, k = _rows(x, "x", x.dtype, dev)
    G, n, ldw, stride_w, sptr, off = _int8_weights(w, w_scales, offsets, k, dev)
    out, ldo, od = _int8_output(out, rows, n, out_dtype,
                                BSG_OUT_F16 if code == BSG_IN_F16 else BSG_OUT_BF16, dev)
    if workspace is None:
        workspace = grouped_gemm_int8_dynamic_workspace(rows, k, x.device)
    ws, st = _dense(workspace, "workspace", 0, workspace.dtype, dev), _status(status, dev)
    if rows:
        _launch(lib.grouped_gemm_int8_dynamic, dev, code, G, x.data_ptr(), ldx, w.data_ptr(), ldw,
                stride_w, sptr, off, rows, n, k, out.data_ptr(), ldo, od, ws, workspace.nbytes, st)
    return out


def grouped_swiglu_checkpoint_mxfp8(h, offsets, row_weights=None, out=None, data=None, scales=None,
                                    keep=True, status=None):
    """out = row_weights * silu(g) * u of h = [g | u] ([rows, 2 f], bf16 or fp16; rows may be strided),
    and h in 8 bits for grouped_swiglu_checkpoint_mxfp8_backward: (out [rows, f], data uint8
    [rows, 2 f] E4M3 codes, scales uint8 [rows, f / 16] E8M0 bytes).  keep=False: (out, None, None).
    Only rows in [offsets[0], offsets[-1]).  See include/bsg.h."""
    import torch
    lib = load_library()
    code, dev = _in_16bit(h, "h"), _device_index(h, "h")
    ldh, rows, f2 = _rows(h, "h", h.dtype, dev)
    f = f2 // 2
    if f2 % 64 != 0 or f2 == 0:
        raise ValueError("h has %d columns, not two times a multiple of 32" % f2)
    out, ldo = _output(out, rows, f, h.dtype, dev)
    dptr = sptr = None
    if keep:
        data, dptr = _buffer(data, rows, f2, torch.uint8, dev, "data")
        scales, sptr = _buffer(scales, rows, f // 16, torch.uint8, dev, "scales")
    else:
        data = scales = None
    w = _maybe(row_weights, "row_weights", 4 * rows, torch.float32, dev)
    off, st = _dense(offsets, "offsets", 16, torch.int64, dev), _status(status, dev)
    if rows:
        _launch(lib.grouped_swiglu_checkpoint_mxfp8, dev, code, h.data_ptr(), ldh, w,
                offsets.numel() - 1, off, rows, f, out.data_ptr(), ldo, dptr, sptr, st)
    return out, data, scales


def grouped_swiglu_checkpoint_mxfp8_backward(data, scales, d_out, offsets, row_weights=None,
                                             recompute=False, d_h=None, d_row_weights=None, out=None,
                                             status=None):
    """(d_h [rows, 2 f], d_row_weights [rows], out [rows, f]) from what
    grouped_swiglu_checkpoint_mxfp8 kept and the gradient d_out [rows, f] (bf16 or fp16; rows may be
    strided) of its output.  d_row_weights: None without row_weights; out (the activation again, for
    the second product's weight gradient): None unless recompute or given."""
    import torch
    lib = load_library()
    code, dev = _in_16bit(d_out, "d_out"), _device_index(d_out, "d_out")
    ldd, rows, f = _rows(d_out, "d_out", d_out.dtype, dev)
    if f % 32 != 0 or f == 0:
        raise ValueError("d_out has %d columns, not a multiple of 32" % f)
    d_h, ldh = _output(d_h, rows, 2 * f, d_out.dtype, dev, "d_h")
    ldo, optr = f, None
    if recompute or out is not None:
        out, ldo = _output(out, rows, f, d_out.dtype, dev)
        optr = out.data_ptr()
    w = wptr = None
    if row_weights is None:
        d_row_weights = None
    else:
        w = _dense(row_weights, "row_weights", 4 * rows, torch.float32, dev)
        d_row_weights, wptr = _buffer(d_row_weights, rows, None, torch.float32, dev, "d_row_weights")
    dptr = _dense(data, "data", rows * 2 * f, torch.uint8, dev)
    sptr = _dense(scales, "scales", rows * (f // 16), torch.uint8, dev)
    off, st = _dense(offsets, "offsets", 16, torch.int64, dev), _status(status, dev)
    if rows:
        _launch(lib.grouped_swiglu_checkpoint_mxfp8_backward, dev, code, dptr, sptr, w, d_out.data_ptr(),
                ldd, offsets.numel() - 1, off, rows, f, d_h.data_ptr(), ldh, optr, ldo, wptr, st)
    return d_h, d_row_weights, out
