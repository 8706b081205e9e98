"""Thin Python binding over libmx355 (C ABI in include/mx.h).

Argument marshalling only: every step of the path runs in the HIP kernels of
libmx355.so.  PyTorch supplies device memory (tensors are passed as raw device
pointers) and the current HIP stream.  There is no fallback: if the library
or a GPU is missing, calls raise.
"""
from __future__ import annotations

import array
import ctypes
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmx355.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "mx.h")

MX_F32, MX_BF16 = 0, 1
RNE, SR = 0, 1
# scale storage orders (include/mx.h): 2D B scales; staged ([stage][row][8 bytes]);
# column-wise groups padded to 256 tokens
SCALES_B_2D, SCALES_STAGED, GROUPS_PAD256 = 1, 2, 4
# the router's scores (include/mx.h, mx_score)
SOFTMAX, SIGMOID = 0, 1
STATUS = {0: "MX_OK", 1: "MX_ERR_NULL", 2: "MX_ERR_SHAPE", 3: "MX_ERR_ALIGN",
          4: "MX_ERR_DTYPE", 5: "MX_ERR_UNSUPPORTED", 6: "MX_ERR_LAUNCH"}


class MXError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__("%s returned %s" % (fn, STATUS.get(code, code)))
        self.code = code


_lib = None


def lib():
    """Load libmx355.so (built in-tree by __graft_entry__.build())."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libmx355.so is not built; run "
                               "python -m mxfp4_precision_numerics_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        P, i64, u64, u32, i32, c_int = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64,
                                        ctypes.c_uint32, ctypes.c_int32, ctypes.c_int)
        L.mx_version.restype = c_int
        L.mx_status_str.argtypes = [c_int]
        L.mx_status_str.restype = ctypes.c_char_p
        L.mx_rht_sign_mask.argtypes = [u64]
        L.mx_rht_sign_mask.restype = u32
        L.mx_rht.argtypes = [P, c_int, P, i64, i64, u32, c_int, P]
        L.mx_quantize_1d.argtypes = [P, c_int, i64, i64, c_int, P, i32, i64, P, c_int, u32, c_int,
                                     u64, u32, u64, P, i64, P, P]
        L.mx_quantize_2d.argtypes = [P, c_int, i64, i64, i64, P, i64, P, P, i64, P, P]
        L.mx_quantize_2d_deosc.argtypes = [P, c_int, i64, i64, i64, P, i64, P, c_int, P, i64, P, P, i64, P,
                                           P, P]
        L.mx_dequantize.argtypes = [P, i64, P, i64, i64, i64, c_int, P, c_int, P]
        L.mx_quantize_1d_dual.argtypes = [P, c_int, i64, i64, P, i32, i64, c_int, u32, c_int, u32, u64, P, P,
                                          c_int, u32, u64, P, i64, P, u64, c_int, P]
        L.mx_quantize_1d_ex.argtypes = [P, c_int, i64, i64, c_int, u32, c_int, u64, u32, u64,
                                        ctypes.c_float, i64, P, P, P, P]
        L.mx_dequantize_1d_ex.argtypes = [P, P, P, i64, i64, i64, P, P]
        L.mx_grouped_gemm.argtypes = [P, i64, P, P, P, i64, P, c_int, P, i32, c_int, i64, i64, i64,
                                      ctypes.c_float, P, c_int, P]
        L.mx_grouped_gemm_q.argtypes = [P, i64, P, P, P, i64, P, c_int, P, i32, i64, i64, i64,
                                        ctypes.c_float, P, P, i64, P, P]
        f32 = ctypes.c_float
        L.mx_route.argtypes = [P, c_int, i64, i32, i64, P, c_int, i32, i32, i32, i32, c_int, f32, P, P, P]
        L.mx_route_bwd.argtypes = [P, c_int, i64, i32, i64, c_int, i32, c_int, f32, P, P, P, i64, P]
        L.mx_route_plan_workspace.argtypes = [i64, i32, i32]
        L.mx_route_plan_workspace.restype = i64
        L.mx_route_plan.argtypes = [P, i64, i32, i32, P, P, P, P, P]
        L.mx_combine.argtypes = [P, c_int, i64, i64, i64, P, P, i64, i32, P, i64, P, c_int, i64, P]
        L.mx_combine_bwd.argtypes = [P, c_int, i64, P, c_int, i64, i64, i64, P, P, i64, i32, P, P, i64, P, P]
        L.mx_grad_workspace.argtypes = [i32]
        L.mx_grad_workspace.restype = i64
        L.mx_grad_norm.argtypes = [P, P, P, i32, P, P, P]
        L.mx_grad_clip.argtypes = [P, P, P, i32, P, f32, P, P, P]
        for name in ("mx_rht", "mx_quantize_1d", "mx_quantize_2d", "mx_quantize_2d_deosc", "mx_dequantize",
                     "mx_quantize_1d_ex", "mx_dequantize_1d_ex", "mx_quantize_1d_dual",
                     "mx_grouped_gemm", "mx_grouped_gemm_q", "mx_route", "mx_route_bwd", "mx_route_plan",
                     "mx_combine", "mx_combine_bwd", "mx_grad_norm", "mx_grad_clip"):
            getattr(L, name).restype = c_int
        for name, restype, argtypes in (
                ("mx_balance_workspace", i64, [i64, i32]),
                ("mx_balance", c_int, [P, c_int, i64, i32, i64, c_int, P, i32, P, P, P, P, P]),
                ("mx_balance_bwd", c_int, [P, c_int, i64, i32, i64, c_int, P, P, f32, P, i64, P, i64, P]),
                ("mx_cache_write", c_int, [P, P, i64, i64, P, i64, i64, c_int, i64, P, P]),
                ("mx_cache_read", c_int, [P, P, i64, i64, P, i64, i64, c_int, i64, P, P]),
                ("mx_cache_attention_workspace", i64, [P, c_int, i64, i32, i32]),
                ("mx_cache_attention", c_int, [P, P, c_int, i64, i32, i64, i64, P, i32, i32, P, i64, i32, P, f32, c_int,
                                               i32, P, P, i64, i64, P, P, P])):
            if hasattr(L, name):      # (not in a library built of the other sources alone)
                getattr(L, name).restype, getattr(L, name).argtypes = restype, argtypes
        _lib = L
    return _lib


def declared_functions():
    """Function names declared in include/mx.h."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*[A-Za-z_][\w\s\*]*?\b(mx_\w+)\s*\(", text, re.M)))


def _check(fn, code):
    if code != 0:
        raise MXError(fn, code)


# ---------------------------------------------------------------------------
# torch plumbing
# ---------------------------------------------------------------------------
_torch_module = _dtype_codes = None


def _torch():
    """torch, imported at the first call that needs it."""
    global _torch_module, _dtype_codes
    if _torch_module is None:
        import torch
        _dtype_codes = {torch.float32: MX_F32, torch.bfloat16: MX_BF16}
        _torch_module = torch
    return _torch_module


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream():
    # the current device's current stream as a handle; building a
    # torch.cuda.Stream for it would take ten times as long
    C = _torch()._C
    return C._cuda_getCurrentRawStream(C._cuda_getDevice())


def _dtype_code(t):
    _torch()
    try:
        return _dtype_codes[t.dtype]
    except KeyError:
        raise TypeError("expected float32 or bfloat16, got %s" % t.dtype) from None


def _dev(t, name):
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _codes(t, name):
    """A code tensor [..., rows, row_bytes] whose rows may be padded: its
    rows are contiguous and any row pitch (stride between rows, in bytes) is
    allowed, and leading dimensions are contiguous over pitched rows (a
    row-slice view t = buf[..., :row_bytes] of a wider buffer).  Returns the
    row pitch to pass to the library, 0 when the rows are contiguous."""
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if t.dtype.itemsize != 1 or t.dim() < 2 or t.stride(-1) != 1:
        raise ValueError("%s must be uint8 [..., rows, bytes] with contiguous rows" % name)
    ld = t.stride(-2)
    expect = ld * t.shape[-2]
    for d in range(t.dim() - 3, -1, -1):
        if t.shape[d] > 1 and t.stride(d) != expect:
            raise ValueError("%s: leading dimensions must be contiguous over its rows" % name)
        expect *= t.shape[d]
    return 0 if ld == t.shape[-1] else ld


def _shaped(t, shape, dtype, name, pitched=False):
    """Check a tensor against the extent the library reads or writes: this
    shape (a leading batch of 1 may be left out) and dtype, on the device,
    contiguous, or for a code array with rows that may be padded.  Returns
    the code rows' pitch (0 when unpadded or not a code array)."""
    shape = tuple(int(v) for v in shape)
    got = tuple(t.shape)
    if got != shape and not (len(shape) == 3 and shape[0] == 1 and got == shape[1:]):
        raise ValueError("%s: expected shape %s, got %s" % (name, shape, got))
    if t.dtype != dtype:
        raise TypeError("%s: expected %s, got %s" % (name, dtype, t.dtype))
    if pitched:
        return _codes(t, name)
    _dev(t, name)
    return 0


def rht_sign_mask(seed: int) -> int:
    return int(lib().mx_rht_sign_mask(seed))


def _index_vector(t, name, min_numel=0):
    """A device int32 vector (offsets, row indices): a tensor of another type
    would be read as int32 words and mis-group silently."""
    torch = _torch()
    if t.dtype != torch.int32 or t.dim() != 1 or t.numel() < min_numel:
        raise ValueError("%s must be a 1-D int32 tensor%s" %
                         (name, " of at least %d elements" % min_numel if min_numel else ""))
    return _dev(t, name)


def rht(x, sign_mask: int, inverse: bool = False, out=None):
    torch = _torch()
    _dev(x, "x")
    rows, cols = x.shape
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.float32, device=x.device)
    else:
        _shaped(out, (rows, cols), torch.float32, "out")
    _check("mx_rht", lib().mx_rht(_ptr(x), _dtype_code(x), _ptr(out), rows, cols, sign_mask,
                                  int(inverse), _stream()))
    return out


def _scale_flags(b_scale_2d, staged):
    return (SCALES_B_2D if b_scale_2d else 0) | (SCALES_STAGED if staged else 0)


def padded_capacity(rows: int, num_groups: int, group_pad: int = 32) -> int:
    """A token capacity that holds any grouping of `rows` tokens into
    `num_groups` groups each padded to a multiple of group_pad (32 or 256),
    rounded up to a multiple of 256 tokens: every row of the column-wise
    codes is then a whole number of 128-byte lines, and the number of
    32-token blocks is even (the grouped GEMM moves scale bytes in pairs)."""
    return (rows + (group_pad - 1) * num_groups + 255) // 256 * 256


def quantize_1d(x, block_axis: int = 1, group_offsets=None, kp: int = 0, use_rht: bool = False,
                sign_mask: int = 0, rnd: int = RNE, seed: int = 0, stream_id: int = 0,
                index_base: int = 0, codes=None, scales=None, row_index=None, staged: bool = False,
                group_pad: int = 32):
    """Returns (codes, scales) uint8 device tensors; see mx_quantize_1d.
    row_index (column-wise only): gather x's rows through it; the grouped
    positions then number row_index.numel().  A row-wise codes output may
    have padded rows, e.g. buf[:, :cols // 2] of a wider buffer (its row
    stride, a multiple of 16, is passed as the pitch; the padding is not
    written).  staged: scales in the staged order (include/mx.h), row-wise
    [ceil(cols / 256), rows, 8], column-wise [kp // 256 + groups, cols, 8].
    group_pad (column-wise): 32, or 256 to start every group on a whole K
    stage of the weight-gradient GEMM."""
    torch = _torch()
    _dev(x, "x")
    rows, cols = x.shape
    if row_index is not None:
        _index_vector(row_index, "row_index")
        rows = row_index.numel()
    ng = 0
    if block_axis == 1:
        shape_c, shape_s = (rows, cols // 2), (rows, cols // 32)
        if staged:
            shape_s = ((cols + 255) // 256, rows, 8)
    else:
        _index_vector(group_offsets, "group_offsets", min_numel=2)
        ng = group_offsets.numel() - 1
        if group_pad not in (32, 256):
            raise ValueError("group_pad is 32 or 256")
        if not kp:
            kp = padded_capacity(rows, ng, group_pad)
        shape_c, shape_s = (cols, kp // 2), (cols, kp // 32)
        if staged:
            shape_s = (kp // 256 + ng, cols, 8)
    if codes is None:
        codes = torch.empty(shape_c, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(shape_s, dtype=torch.uint8, device=x.device)
    # codes may be a row-slice view of a wider buffer (padded rows)
    codes_ld = _shaped(codes, shape_c, torch.uint8, "codes", pitched=True)
    _shaped(scales, shape_s, torch.uint8, "scales")
    _check("mx_quantize_1d", lib().mx_quantize_1d(
        _ptr(x), _dtype_code(x), rows, cols,
        block_axis | (SCALES_STAGED if staged else 0) | (GROUPS_PAD256 if group_pad == 256 else 0),
        _ptr(group_offsets), ng, kp,
        _ptr(row_index), int(use_rht), sign_mask, rnd, seed, stream_id, index_base, _ptr(codes), codes_ld,
        _ptr(scales), _stream()))
    return codes, scales


def quantize_1d_dual(x, group_offsets, kp: int = 0, use_rht: bool = False, sign_mask: int = 0,
                     col_rnd: int = RNE, col_stream_id: int = 0, row_rnd: int = RNE, row_stream_id: int = 0,
                     seed: int = 0, col_index_base: int = 0, row_index_base: int = 0, col_codes=None,
                     col_scales=None, row_codes=None, row_scales=None, staged: bool = False, group_pad: int = 32):
    """Column-wise (grouped, transposed, optional RHT) and row-wise (no RHT)
    1x32 quantization of x from one read (see mx_quantize_1d_dual).
    Returns (col_codes, col_scales, row_codes, row_scales); row_codes may
    have padded rows (a row-slice view of a wider buffer).  staged: both
    outputs' scales in the staged order (column-wise [kp // 256 + groups,
    cols, 8], row-wise [ceil(cols / 256), rows, 8]); group_pad: the
    column-wise output's group padding, 32 or 256 tokens."""
    torch = _torch()
    _dev(x, "x")
    rows, cols = x.shape
    _index_vector(group_offsets, "group_offsets", min_numel=2)
    ng = group_offsets.numel() - 1
    if group_pad not in (32, 256):
        raise ValueError("group_pad is 32 or 256")
    kp = kp or padded_capacity(rows, ng, group_pad)
    u8, dev = torch.uint8, x.device
    shape_cs = (kp // 256 + ng, cols, 8) if staged else (cols, kp // 32)
    shape_rs = ((cols + 255) // 256, rows, 8) if staged else (rows, cols // 32)
    col_codes = col_codes if col_codes is not None else torch.empty((cols, kp // 2), dtype=u8, device=dev)
    col_scales = col_scales if col_scales is not None else torch.empty(shape_cs, dtype=u8, device=dev)
    row_codes = row_codes if row_codes is not None else torch.empty((rows, cols // 2), dtype=u8, device=dev)
    row_scales = row_scales if row_scales is not None else torch.empty(shape_rs, dtype=u8, device=dev)
    _shaped(col_codes, (cols, kp // 2), u8, "col_codes")
    _shaped(col_scales, shape_cs, u8, "col_scales")
    ld = _shaped(row_codes, (rows, cols // 2), u8, "row_codes", pitched=True)
    _shaped(row_scales, shape_rs, u8, "row_scales")
    flags = (SCALES_STAGED if staged else 0) | (GROUPS_PAD256 if group_pad == 256 else 0)
    _check("mx_quantize_1d_dual", lib().mx_quantize_1d_dual(
        _ptr(x), _dtype_code(x), rows, cols, _ptr(group_offsets), ng, kp, int(use_rht), sign_mask, col_rnd,
        col_stream_id, col_index_base, _ptr(col_codes), _ptr(col_scales), row_rnd, row_stream_id,
        row_index_base, _ptr(row_codes), ld, _ptr(row_scales), seed, flags, _stream()))
    return col_codes, col_scales, row_codes, row_scales


def quantize_2d(w, layout=True, transposed=True):
    """w [batch x rows x cols] or [rows x cols]; returns (codes, scales,
    codes_t, scales_t), None for a layout not asked for."""
    torch = _torch()
    _dev(w, "w")
    b, r, c = (1,) + tuple(w.shape) if w.dim() == 2 else tuple(w.shape)
    dev = w.device
    codes = torch.empty((b, r, c // 2), dtype=torch.uint8, device=dev) if layout else None
    scales = torch.empty((b, r // 32, c // 32), dtype=torch.uint8, device=dev) if layout else None
    codes_t = torch.empty((b, c, r // 2), dtype=torch.uint8, device=dev) if transposed else None
    scales_t = torch.empty((b, c // 32, r // 32), dtype=torch.uint8, device=dev) if transposed else None
    return quantize_2d_into(w, codes, scales, codes_t, scales_t)


def quantize_2d_into(w, codes, scales, codes_t, scales_t):
    """As quantize_2d, into caller-provided buffers (either pair may be None).
    codes and codes_t may have padded rows (row-slice views of wider buffers)."""
    torch = _torch()
    _dev(w, "w")
    squeeze = w.dim() == 2
    w3 = w.unsqueeze(0) if squeeze else w
    b, r, c = w3.shape
    u8 = torch.uint8
    ld = 0 if codes is None else _shaped(codes, (b, r, c // 2), u8, "codes", pitched=True)
    ld_t = 0 if codes_t is None else _shaped(codes_t, (b, c, r // 2), u8, "codes_t", pitched=True)
    if scales is not None:
        _shaped(scales, (b, r // 32, c // 32), u8, "scales")
    if scales_t is not None:
        _shaped(scales_t, (b, c // 32, r // 32), u8, "scales_t")
    _check("mx_quantize_2d", lib().mx_quantize_2d(
        _ptr(w3), _dtype_code(w3), b, r, c, _ptr(codes), ld, _ptr(scales), _ptr(codes_t), ld_t,
        _ptr(scales_t), _stream()))
    out = [codes, scales, codes_t, scales_t]
    if squeeze:
        out = [t[0] if t is not None and t.dim() == 3 else t for t in out]
    return tuple(out)


def quantize_1d_ex(x, use_rht: bool = False, sign_mask: int = 0, rnd: int = RNE, seed: int = 0,
                   stream_id: int = 0, index_base: int = 0, clip_ratio: float = 1.0, macro_block: int = 0,
                   codes=None, scales=None, macro_r=None):
    """Row-wise 1x32 quantization with outlier clipping and macro-block
    scaling (see mx_quantize_1d_ex).  Returns (codes, scales, macro_r or
    None)."""
    torch = _torch()
    _dev(x, "x")
    rows, cols = x.shape
    dev = x.device
    codes = codes if codes is not None else torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
    scales = scales if scales is not None else torch.empty((rows, cols // 32), dtype=torch.uint8, device=dev)
    _shaped(codes, (rows, cols // 2), torch.uint8, "codes")
    _shaped(scales, (rows, cols // 32), torch.uint8, "scales")
    if macro_block:
        if cols % macro_block:
            raise ValueError("macro_block must divide cols")
        macro_r = macro_r if macro_r is not None else torch.empty((rows, cols // macro_block),
                                                                  dtype=torch.float32, device=dev)
        _shaped(macro_r, (rows, cols // macro_block), torch.float32, "macro_r")
    else:
        macro_r = None
    _check("mx_quantize_1d_ex", lib().mx_quantize_1d_ex(
        _ptr(x), _dtype_code(x), rows, cols, int(use_rht), sign_mask, rnd, seed, stream_id, index_base,
        float(clip_ratio), int(macro_block), _ptr(codes), _ptr(scales), _ptr(macro_r), _stream()))
    return codes, scales, macro_r


def dequantize_1d_ex(codes, scales, macro_r=None, macro_block: int = 0, out=None):
    """fp32 decode of quantize_1d_ex's output: deq(code, scale) / r."""
    torch = _torch()
    _dev(codes, "codes")
    rows, half = codes.shape
    cols = half * 2
    _shaped(scales, (rows, cols // 32), torch.uint8, "scales")
    if macro_block:
        _shaped(macro_r, (rows, cols // macro_block), torch.float32, "macro_r")
    out = out if out is not None else torch.empty((rows, cols), dtype=torch.float32, device=codes.device)
    _shaped(out, (rows, cols), torch.float32, "out")
    _check("mx_dequantize_1d_ex", lib().mx_dequantize_1d_ex(
        _ptr(codes), _ptr(scales), _ptr(macro_r) if macro_block else None, rows, cols, int(macro_block),
        _ptr(out), _stream()))
    return out


def quantize_2d_deosc(w, prev_codes, prev_scales, margin64: int, codes=None, scales=None,
                      codes_t=None, scales_t=None, transposed=True, flips=True):
    """32x32 quantization with the de-oscillation band against the previous
    step's as-given codes and scales (see mx_quantize_2d_deosc).  codes /
    scales default to new tensors; passing prev_codes / prev_scales again
    updates them in place.  Returns (codes, scales, codes_t, scales_t,
    flips), None for what was not asked for."""
    torch = _torch()
    _dev(w, "w")
    squeeze = w.dim() == 2
    w3 = w.unsqueeze(0) if squeeze else w
    b, r, c = w3.shape
    u8, dev = torch.uint8, w.device

    def as3(t):
        return t.unsqueeze(0) if t is not None and t.dim() == 2 else t

    prev_codes, prev_scales = as3(prev_codes), as3(prev_scales)
    codes = as3(codes) if codes is not None else torch.empty((b, r, c // 2), dtype=u8, device=dev)
    scales = as3(scales) if scales is not None else torch.empty((b, r // 32, c // 32), dtype=u8, device=dev)
    if transposed:
        codes_t = as3(codes_t) if codes_t is not None else torch.empty((b, c, r // 2), dtype=u8, device=dev)
        scales_t = as3(scales_t) if scales_t is not None else torch.empty((b, c // 32, r // 32), dtype=u8,
                                                                          device=dev)
    else:
        codes_t = scales_t = None
    fl = torch.empty((b, r // 32, c // 32), dtype=torch.int16, device=dev) if flips else None
    pld = _shaped(prev_codes, (b, r, c // 2), u8, "prev_codes", pitched=True)
    _shaped(prev_scales, (b, r // 32, c // 32), u8, "prev_scales")
    ld = _shaped(codes, (b, r, c // 2), u8, "codes", pitched=True)
    _shaped(scales, (b, r // 32, c // 32), u8, "scales")
    ld_t = 0 if codes_t is None else _shaped(codes_t, (b, c, r // 2), u8, "codes_t", pitched=True)
    if scales_t is not None:
        _shaped(scales_t, (b, c // 32, r // 32), u8, "scales_t")
    _check("mx_quantize_2d_deosc", lib().mx_quantize_2d_deosc(
        _ptr(w3), _dtype_code(w3), b, r, c, _ptr(prev_codes), pld, _ptr(prev_scales), int(margin64),
        _ptr(codes), ld, _ptr(scales), _ptr(codes_t), ld_t, _ptr(scales_t), _ptr(fl), _stream()))
    out = [codes, scales, codes_t, scales_t, fl]
    if squeeze:
        out = [t[0] if t is not None and t.dim() == 3 else t for t in out]
    return tuple(out)


def dequantize(codes, scales, block_rows: int = 1, out_dtype=None, out=None):
    """Per mx_dequantize; codes may have padded rows."""
    torch = _torch()
    ld = _codes(codes, "codes")
    out_dtype = out_dtype or torch.float32
    squeeze = codes.dim() == 2
    c3 = codes.unsqueeze(0) if squeeze else codes
    b, r, half = c3.shape
    _shaped(scales, (b, r // block_rows, half * 2 // 32), torch.uint8, "scales")
    if out is None:
        out = torch.empty((b, r, half * 2), dtype=out_dtype, device=codes.device)
    else:
        _shaped(out, (b, r, half * 2), out.dtype, "out")
    _check("mx_dequantize", lib().mx_dequantize(
        _ptr(c3), ld, _ptr(scales), b, r, half * 2, block_rows, _ptr(out), _dtype_code(out),
        _stream()))
    return out[0] if squeeze and out.dim() == 3 else out


def _gemm_operands(a_codes, a_scales, a_row_index, b_codes, b_scales, group_offsets, M, N, K,
                   b_scale_2d, group_dim_k, staged=False):
    """Check A, B and their scales against M, N, K and the group count (the
    extents the kernel reads); returns (a_ld, b_ld, G).  Staged scales are
    [stages, rows, 8]: K // 256 + G stages with groups along K, ceil(K / 256)
    along M."""
    torch = _torch()
    u8 = torch.uint8
    _index_vector(group_offsets, "group_offsets", min_numel=2)
    G = group_offsets.numel() - 1
    a_rows = M
    if a_row_index is not None:
        _index_vector(a_row_index, "a_row_index")
        if a_row_index.numel() != M:
            raise ValueError("a_row_index must be int32 [M]")
        a_rows = a_codes.shape[0]
    a_ld = _shaped(a_codes, (a_rows, K // 2), u8, "a_codes", pitched=True)
    stages = (K // 256 + G) if group_dim_k else (K + 255) // 256
    _shaped(a_scales, (stages, a_rows, 8) if staged else (a_rows, K // 32), u8, "a_scales")
    if group_dim_k:
        b_ld = _shaped(b_codes, (N, K // 2), u8, "b_codes", pitched=True)
        _shaped(b_scales, (stages, N, 8) if staged else (N, K // 32), u8, "b_scales")
    else:
        b_ld = _shaped(b_codes, (G, N, K // 2), u8, "b_codes", pitched=True)
        _shaped(b_scales, (G, N // 32, K // 32) if b_scale_2d else (G, N, K // 32), u8, "b_scales")
    return a_ld, b_ld, G


def grouped_gemm(a_codes, a_scales, b_codes, b_scales, group_offsets, M, N, K,
                 a_row_index=None, b_scale_2d=False, group_dim_k=False, alpha=1.0,
                 out_dtype=None, out=None, staged=False):
    """C (bf16 by default, or out_dtype float32) per mx_grouped_gemm.  a_codes
    and b_codes may have padded rows (row-slice views of wider buffers); rows
    padded to whole 128-byte lines are read fastest."""
    torch = _torch()
    a_ld, b_ld, G = _gemm_operands(a_codes, a_scales, a_row_index, b_codes, b_scales, group_offsets,
                                   M, N, K, b_scale_2d, group_dim_k, staged)
    shape = (G, M, N) if group_dim_k else (M, N)
    if out is None:
        out = torch.empty(shape, dtype=out_dtype or torch.bfloat16, device=a_codes.device)
    else:
        _shaped(out, shape, out_dtype or out.dtype, "out")
    _check("mx_grouped_gemm", lib().mx_grouped_gemm(
        _ptr(a_codes), a_ld, _ptr(a_scales), _ptr(a_row_index), _ptr(b_codes), b_ld, _ptr(b_scales),
        _scale_flags(b_scale_2d, staged), _ptr(group_offsets), G, int(bool(group_dim_k)), M, N, K,
        float(alpha), _ptr(out), _dtype_code(out), _stream()))
    return out


def grouped_gemm_q(a_codes, a_scales, b_codes, b_scales, group_offsets, M, N, K,
                   a_row_index=None, b_scale_2d=False, alpha=1.0, with_bf16=True,
                   out=None, codes=None, scales=None, staged=False):
    """Grouped GEMM (groups split M) whose bf16 output is also written as
    row-wise MXFP4 (1x32 along N, RTNE) by the GEMM's epilogue.  Returns
    (c or None, codes [M x N/2], scales [M x N/32]); out / codes / scales
    are optional preallocated outputs."""
    torch = _torch()
    a_ld, b_ld, G = _gemm_operands(a_codes, a_scales, a_row_index, b_codes, b_scales, group_offsets,
                                   M, N, K, b_scale_2d, False, staged)
    dev = a_codes.device
    c = None
    if with_bf16:
        c = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        _shaped(c, (M, N), torch.bfloat16, "out")
    codes = codes if codes is not None else torch.empty((M, N // 2), dtype=torch.uint8, device=dev)
    c_ld = _shaped(codes, (M, N // 2), torch.uint8, "codes", pitched=True)
    scales = scales if scales is not None else torch.empty((M, N // 32), dtype=torch.uint8, device=dev)
    _shaped(scales, (M, N // 32), torch.uint8, "scales")
    _check("mx_grouped_gemm_q", lib().mx_grouped_gemm_q(
        _ptr(a_codes), a_ld, _ptr(a_scales), _ptr(a_row_index), _ptr(b_codes), b_ld, _ptr(b_scales),
        _scale_flags(b_scale_2d, staged), _ptr(group_offsets), G, M, N, K, float(alpha),
        _ptr(c), _ptr(codes), c_ld, _ptr(scales), _stream()))
    return c, codes, scales


# ---------------------------------------------------------------------------
# Routing, the experts' rows back into tokens, gradient clipping
# ---------------------------------------------------------------------------
# These calls can be as short as their launch, so what they allocate and check
# takes the quickest way there is.
def _new(device, dtype, rows, cols):
    return _torch().empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _new_vector(device, dtype, n):
    return _torch().empty_strided((n,), (1,), dtype=dtype, device=device)


def _same(t, shape, dtype, name):
    """_shaped, one comparison where all is well."""
    if t.shape != shape or t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        _shaped(t, shape, dtype, name)


def _rows(t, name, shape=None, dtype=None):
    """A device matrix with contiguous rows any pitch apart; returns the pitch
    in elements (0 when the rows are contiguous)."""
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError("%s: expected shape %s, got %s" % (name, shape or "[rows, cols]", tuple(t.shape)))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s: expected %s, got %s" % (name, dtype, t.dtype))
    if t.is_contiguous():
        return 0
    rows, cols = t.shape
    ld = t.stride(0)
    if (cols > 1 and t.stride(1) != 1) or (rows > 1 and ld < cols):
        raise ValueError("%s must have contiguous rows that do not overlap" % name)
    return ld if rows > 1 and ld != cols else 0


def route(logits, top_k: int, score: int = SOFTMAX, bias=None, groups: int = 1, top_groups: int = 1,
          group_best: int = 1, renorm: bool = True, scale: float = 1.0, ids=None, weights=None):
    """The top_k experts of each token and their weights from the router's
    logits [tokens, experts] (fp32 or bf16; rows may be padded): ids int32
    and weights fp32 [tokens, top_k].  See mx_route for scores, bias, groups
    and what happens to masked experts."""
    torch = _torch()
    ld = _rows(logits, "logits")
    tokens, experts = logits.shape
    if bias is not None:
        _same(bias, (experts,), torch.float32, "bias")
    if ids is None:
        ids = _new(logits.device, torch.int32, tokens, top_k)
    else:
        _same(ids, (tokens, top_k), torch.int32, "ids")
    if weights is None:
        weights = torch.empty_like(ids, dtype=torch.float32)
    else:
        _same(weights, (tokens, top_k), torch.float32, "weights")
    _check("mx_route", lib().mx_route(
        _ptr(logits), _dtype_code(logits), tokens, experts, ld, _ptr(bias), score, groups, top_groups, group_best,
        top_k, int(bool(renorm)), scale, _ptr(ids), _ptr(weights), _stream()))
    return ids, weights


def route_bwd(logits, ids, dweights, score: int = SOFTMAX, renorm: bool = True, scale: float = 1.0, dlogits=None):
    """The gradient of route's weights with respect to the logits, for the ids
    it chose: dlogits [tokens, experts] of the logits' type (see
    mx_route_bwd)."""
    torch = _torch()
    ld = _rows(logits, "logits")
    tokens, experts = logits.shape
    if ids.dim() != 2:
        raise ValueError("ids must be [tokens, top_k]")
    top_k = ids.shape[1]
    _same(ids, (tokens, top_k), torch.int32, "ids")
    _same(dweights, (tokens, top_k), torch.float32, "dweights")
    dld = 0
    if dlogits is None:
        dlogits = _new(logits.device, logits.dtype, tokens, experts)
    else:
        dld = _rows(dlogits, "dlogits", (tokens, experts), logits.dtype)
    _check("mx_route_bwd", lib().mx_route_bwd(
        _ptr(logits), _dtype_code(logits), tokens, experts, ld, score, top_k, int(bool(renorm)), scale, _ptr(ids),
        _ptr(dweights), _ptr(dlogits), dld, _stream()))
    return dlogits


def route_plan(ids, num_experts: int, offsets=None, row_index=None, slot=None, workspace=None):
    """The dispatch plan of ids [tokens, top_k] (-1: no expert): offsets
    [num_experts + 1] (the group_offsets of the quantizers and the grouped
    GEMM), row_index [tokens * top_k] (their row gather) and slot [tokens,
    top_k] (where combine finds each assignment's row, -1: nowhere), all
    int32; see mx_route_plan.  workspace: uint8, at least
    mx_route_plan_workspace bytes, or None to allocate it."""
    torch = _torch()
    if ids.dim() != 2 or ids.dtype != torch.int32:
        raise ValueError("ids must be int32 [tokens, top_k]")
    _dev(ids, "ids")
    tokens, top_k = ids.shape
    dev, i32 = ids.device, torch.int32
    if offsets is None:
        offsets = _new_vector(dev, i32, num_experts + 1)
    else:
        _same(offsets, (num_experts + 1,), i32, "offsets")
    if row_index is None:
        row_index = _new_vector(dev, i32, tokens * top_k)
    else:
        _same(row_index, (tokens * top_k,), i32, "row_index")
    if slot is None:
        slot = torch.empty_like(ids)
    else:
        _same(slot, (tokens, top_k), i32, "slot")
    need = lib().mx_route_plan_workspace(tokens, top_k, num_experts)
    workspace = _workspace(workspace, need, dev)
    _check("mx_route_plan", lib().mx_route_plan(
        _ptr(ids), tokens, top_k, num_experts, _ptr(offsets), _ptr(row_index), _ptr(slot), _ptr(workspace),
        _stream()))
    return offsets, row_index, slot


def _workspace(t, need, device):
    """A uint8 device buffer of at least `need` bytes."""
    torch = _torch()
    if t is None:
        return None if need == 0 else _new_vector(device, torch.uint8, need)
    if t.dtype != torch.uint8 or t.numel() < need:
        raise ValueError("workspace must be uint8 of at least %d bytes" % need)
    return _dev(t, "workspace")


def _slots(slot, weights):
    torch = _torch()
    if slot.dim() != 2:
        raise ValueError("slot must be [tokens, top_k]")
    tokens, top_k = slot.shape
    _same(slot, (tokens, top_k), torch.int32, "slot")
    if weights is not None:
        _same(weights, (tokens, top_k), torch.float32, "weights")
    return tokens, top_k


def combine(y, slot, weights=None, residual=None, out_dtype=None, out=None):
    """out[t] = residual[t] + sum_j weights[t, j] * y[slot[t, j]]: the experts'
    rows y [rows, cols] back into tokens (see mx_combine).  weights None: 1.
    out is of y's type unless out_dtype or out says otherwise; residual has
    out's type.  Rows may be padded."""
    torch = _torch()
    tokens, top_k = _slots(slot, weights)
    y_ld = _rows(y, "y")
    rows, cols = y.shape
    out_ld = 0
    if out is None:
        out = _new(y.device, out_dtype or y.dtype, tokens, cols)
    else:
        out_ld = _rows(out, "out", (tokens, cols), out_dtype)
    res_ld = _rows(residual, "residual", (tokens, cols), out.dtype) if residual is not None else 0
    _check("mx_combine", lib().mx_combine(
        _ptr(y), _dtype_code(y), rows, cols, y_ld, _ptr(slot), _ptr(weights), tokens, top_k, _ptr(residual), res_ld,
        _ptr(out), _dtype_code(out), out_ld, _stream()))
    return out


def combine_bwd(dout, y, slot, weights=None, used_rows=None, dy=None, dweights=None, need_dweights: bool = True):
    """Gradient of combine: (dy [rows, cols] of y's type, dweights fp32
    [tokens, top_k]) from dout [tokens, cols] (see mx_combine_bwd).
    used_rows: an int32 device tensor of one element, the number of rows that
    slots name (the plan's offsets[-1:]); the rows of dy after it become 0.
    Without it rows that no slot names are left unwritten.  dy may be y.
    need_dweights=False: dweights is None and y is not read."""
    torch = _torch()
    tokens, top_k = _slots(slot, weights)
    y_ld = _rows(y, "y")
    rows, cols = y.shape
    dout_ld = _rows(dout, "dout", (tokens, cols))
    if used_rows is not None:
        _index_vector(used_rows, "used_rows", min_numel=1)
    dy_ld = 0
    if dy is None:
        dy = _new(y.device, y.dtype, rows, cols)
    else:
        dy_ld = _rows(dy, "dy", (rows, cols), y.dtype)
    if dweights is not None:
        _same(dweights, (tokens, top_k), torch.float32, "dweights")
    elif need_dweights:
        dweights = torch.empty_like(slot, dtype=torch.float32)
    _check("mx_combine_bwd", lib().mx_combine_bwd(
        _ptr(dout), _dtype_code(dout), dout_ld, _ptr(y), _dtype_code(y), rows, cols, y_ld, _ptr(slot),
        _ptr(weights), tokens, top_k, _ptr(used_rows), _ptr(dy), dy_ld, _ptr(dweights), _stream()))
    return dy, dweights


def _grad_list(grads, name, device=None):
    """The host arrays of a gradient list (any shapes, contiguous, fp32 and
    bf16 mixed) and its device's index: all of one device, the given one if
    there is one."""
    codes = _dtype_codes
    grads = list(grads)
    devices = {g.get_device() if g.is_contiguous() else -1 for g in grads}
    if -1 in devices:
        raise ValueError("%s must be contiguous device tensors" % name)
    if len(devices) > 1 or (device is not None and devices and device not in devices):
        raise ValueError("%s must be on one device, that of the other arguments" % name)
    try:
        types = array.array("i", [codes[g.dtype] for g in grads])
    except KeyError as e:
        raise TypeError("%s: expected float32 or bfloat16, got %s" % (name, e.args[0])) from None
    return (grads, types, array.array("q", [g.numel() for g in grads]),
            array.array("Q", [g.data_ptr() for g in grads]), devices.pop() if devices else None)


def grad_norm(grads, norm=None, workspace=None):
    """The L2 norm over all elements of the tensors in grads (contiguous, on
    one device): a 0-dim fp32 device tensor (see mx_grad_norm).  workspace:
    uint8, at least mx_grad_workspace bytes, or None to allocate it."""
    return _grad_call("mx_grad_norm", grads, None, None, norm, workspace)


def grad_clip(grads, max_norm: float, outs=None, norm=None, workspace=None):
    """Scales the tensors in grads by min(1, max_norm / (norm + 1e-6)), in
    place or into the tensors of outs (same types and sizes), and returns
    their norm before that as a 0-dim fp32 device tensor.  A norm that is not
    finite leaves the values as they are (see mx_grad_clip).  All tensors are
    contiguous and on one device.  What is written may not overlap another
    tensor: in place no gradient may be in the list twice."""
    return _grad_call("mx_grad_clip", grads, outs, float(max_norm), norm, workspace)


def _grad_call(fn, grads, outs, max_norm, norm, workspace):
    torch = _torch()
    if norm is not None:
        _shaped(norm, (), torch.float32, "norm")
    grads, types, numels, ptrs, device = _grad_list(grads, "grads", None if norm is None else norm.get_device())
    n, outs_at = len(grads), None
    if outs is not None:
        outs, out_types, out_numels, out_ptrs, _ = _grad_list(outs, "outs", device)
        if out_types != types or out_numels != numels:
            raise ValueError("outs must match grads in number, types and sizes")
        outs_at = out_ptrs.buffer_info()[0]
    if norm is None:
        norm = torch.empty((), dtype=torch.float32, device=grads[0].device if n else "cuda")
    workspace = _workspace(workspace, lib().mx_grad_workspace(n), norm.device)
    head = (ptrs.buffer_info()[0], types.buffer_info()[0], numels.buffer_info()[0], n)
    if fn == "mx_grad_norm":
        code = lib().mx_grad_norm(*head, _ptr(workspace), _ptr(norm), _stream())
    else:
        code = lib().mx_grad_clip(*head, outs_at, max_norm, _ptr(workspace), _ptr(norm), _stream())
    _check(fn, code)
    return norm


# ---------------------------------------------------------------------------
# The balance loss
# ---------------------------------------------------------------------------
def _here(device, **tensors):
    """Refuses tensors that are not on this device (its index), and a device
    other than the current one, whose stream the call would go to."""
    if device != _torch()._C._cuda_getDevice():
        raise ValueError("the tensors are not on the current device")
    for name, t in tensors.items():
        if t is not None and t.get_device() != device:
            raise ValueError("%s is on another device" % name)


def balance(logits, ids, score: int = SOFTMAX, counts=None, slope=None, loss=None, workspace=None):
    """The balance loss of a router over its tokens (see mx_balance): (loss, a
    0-dim fp32 device tensor, 1 for an even balance; counts int32 [experts],
    the assignments of each expert in ids [tokens, top_k]; slope fp32
    [experts], what balance_bwd needs).  logits [tokens, experts], fp32 or
    bf16, rows may be padded.  workspace: uint8, at least
    mx_balance_workspace bytes, or None to allocate it."""
    torch = _torch()
    ld = _rows(logits, "logits")
    tokens, experts = logits.shape
    if ids.dim() != 2:
        raise ValueError("ids must be [tokens, top_k]")
    top_k = ids.shape[1]
    _same(ids, (tokens, top_k), torch.int32, "ids")
    dev = logits.device
    if counts is None:
        counts = _new_vector(dev, torch.int32, experts)
    else:
        _same(counts, (experts,), torch.int32, "counts")
    if slope is None:
        slope = _new_vector(dev, torch.float32, experts)
    else:
        _same(slope, (experts,), torch.float32, "slope")
    if loss is None:
        loss = torch.empty((), dtype=torch.float32, device=dev)
    else:
        _shaped(loss, (), torch.float32, "loss")
    workspace = _workspace(workspace, lib().mx_balance_workspace(tokens, experts), dev)
    _here(logits.get_device(), ids=ids, counts=counts, slope=slope, loss=loss, workspace=workspace)
    _check("mx_balance", lib().mx_balance(
        _ptr(logits), _dtype_code(logits), tokens, experts, ld, score, _ptr(ids), top_k, _ptr(counts), _ptr(slope),
        _ptr(loss), _ptr(workspace), _stream()))
    return loss, counts, slope


def balance_bwd(logits, slope, score: int = SOFTMAX, dloss=None, scale: float = 1.0, add=None, dlogits=None):
    """Gradient of scale * dloss * balance with respect to the logits, plus add
    (see mx_balance_bwd): dlogits [tokens, experts] of the logits' type.
    dloss: an fp32 device tensor of one element, or None for 1.  add: the
    router's own gradient (route_bwd); dlogits may be add, which then becomes
    the sum."""
    torch = _torch()
    ld = _rows(logits, "logits")
    tokens, experts = logits.shape
    _same(slope, (experts,), torch.float32, "slope")
    if dloss is not None and (dloss.dtype != torch.float32 or dloss.numel() != 1):
        raise ValueError("dloss must be one float32")
    add_ld = _rows(add, "add", (tokens, experts), logits.dtype) if add is not None else 0
    dld = 0
    if dlogits is None:
        dlogits = _new(logits.device, logits.dtype, tokens, experts)
    else:
        dld = _rows(dlogits, "dlogits", (tokens, experts), logits.dtype)
    _here(logits.get_device(), slope=slope, dloss=dloss, add=add, dlogits=dlogits)
    _check("mx_balance_bwd", lib().mx_balance_bwd(
        _ptr(logits), _dtype_code(logits), tokens, experts, ld, score, _ptr(slope), _ptr(dloss), float(scale),
        _ptr(add), add_ld, _ptr(dlogits), dld, _stream()))
    return dlogits


# ---------------------------------------------------------------------------
# The key/value cache and the attention over it
# ---------------------------------------------------------------------------
class _CacheStruct(ctypes.Structure):
    """mx_cache."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k_codes", "k_scales", "v_codes", "v_scales")] +
                [("pages", ctypes.c_int64)] +
                [(n, ctypes.c_int32) for n in ("heads", "page_size", "head_dim", "use_rht")] +
                [("sign_mask", ctypes.c_uint32)])


class KVCache:
    """A paged key/value cache in MXFP4 over four uint8 device tensors (see
    mx_cache): codes [pages, heads, page_size, head_dim // 2] and scales
    [pages, heads, head_dim // 32, page_size], of keys and of values.  With
    use_rht what it holds is transformed (sign_mask).

    It describes these tensors' storage as it is now: its fields cannot be
    set, and calls refuse it once a tensor's storage has been replaced."""

    _FIELDS = frozenset(("k_codes", "k_scales", "v_codes", "v_scales", "pages", "heads", "page_size", "head_dim",
                         "use_rht", "sign_mask", "device_index"))

    def __init__(self, k_codes, k_scales, v_codes, v_scales, use_rht: bool = False, sign_mask: int = 0):
        torch = _torch()
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be [pages, heads, page_size, head_dim // 2]")
        pages, heads, page_size, half = k_codes.shape
        for name, t in (("k_codes", k_codes), ("v_codes", v_codes)):
            _shaped(t, (pages, heads, page_size, half), torch.uint8, name)
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            _shaped(t, (pages, heads, half // 16, page_size), torch.uint8, name)
        device = k_codes.get_device()
        if any(t.get_device() != device for t in (k_scales, v_codes, v_scales)):
            raise ValueError("the cache's tensors are on different devices")
        tensors = (k_codes, k_scales, v_codes, v_scales)
        at = tuple(t.data_ptr() for t in tensors)
        struct = _CacheStruct(*[p or None for p in at], pages, heads, page_size, 2 * half, bool(use_rht), int(sign_mask))
        vars(self).update(k_codes=k_codes, k_scales=k_scales, v_codes=v_codes, v_scales=v_scales, device_index=device,
                          pages=pages, heads=heads, page_size=page_size, head_dim=2 * half, use_rht=bool(use_rht),
                          sign_mask=int(sign_mask), _tensors=tensors, _struct=struct, _addresses=at)

    def __setattr__(self, name, value):
        if name in self._FIELDS:
            raise AttributeError("a KVCache's %s cannot be set; make another KVCache" % name)
        super().__setattr__(name, value)

    @property
    def _at(self):
        """The address of the mx_cache, for a call."""
        a, b, c, d = self._tensors
        if (a.data_ptr(), b.data_ptr(), c.data_ptr(), d.data_ptr()) != self._addresses:
            raise ValueError("the storage of the cache's tensors has been replaced; make another KVCache")
        return ctypes.addressof(self._struct)


def kv_cache(pages: int, heads: int, page_size: int, head_dim: int, use_rht: bool = False, sign_mask: int = 0,
             device="cuda"):
    """A new KVCache; every slot reads as 0."""
    torch = _torch()
    shapes = ((pages, heads, page_size, head_dim // 2), (pages, heads, head_dim // 32, page_size)) * 2
    return KVCache(*[torch.zeros(s, dtype=torch.uint8, device=device) for s in shapes], use_rht=use_rht,
                   sign_mask=sign_mask)


def _heads(t, name, shape=None, dtype=None, written=False):
    """The pitches (token, head) of a device tensor [tokens, heads, dim] with
    contiguous rows in any order, 0 for the default ones.  written: its rows
    may not overlap."""
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if t.dim() != 3 or (shape is not None and t.shape != shape):
        raise ValueError("%s: expected shape %s, got %s" % (name, shape or "[tokens, heads, dim]", tuple(t.shape)))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s: expected %s, got %s" % (name, dtype, t.dtype))
    if t.is_contiguous():
        return 0, 0
    (tokens, heads, dim), (ld, head_ld, one) = t.shape, t.stride()
    ld, head_ld = ld if tokens > 1 else 0, head_ld if heads > 1 else 0
    if one != 1 or (tokens > 1 and ld < dim) or (heads > 1 and head_ld < dim):
        raise ValueError("%s must have contiguous rows that do not overlap" % name)
    if written and tokens > 1 and heads > 1 and ld < (heads - 1) * head_ld + dim and head_ld < (tokens - 1) * ld + dim:
        raise ValueError("%s must have rows that do not overlap" % name)
    return ld, head_ld


def _slot_vector(slots, tokens):
    torch = _torch()
    _same(slots, (tokens,), torch.int32, "slots")
    return slots


def cache_write(cache, k, v, slots):
    """Quantizes the keys and values k, v [tokens, heads, head_dim] (fp32 or
    bf16, any pitches) into the cache's slots (int32 [tokens]: page * page_size
    + offset; -1 or another one outside the cache: not written).  See
    mx_cache_write."""
    k_ld, k_head = _heads(k, "k")
    tokens = k.shape[0]
    shape = (tokens, cache.heads, cache.head_dim)
    if k.shape != shape:
        raise ValueError("k: expected shape %s, got %s" % (shape, tuple(k.shape)))
    v_ld, v_head = _heads(v, "v", shape, k.dtype)
    _slot_vector(slots, tokens)
    _here(cache.device_index, k=k, v=v, slots=slots)
    _check("mx_cache_write", lib().mx_cache_write(
        cache._at, _ptr(k), k_ld, k_head, _ptr(v), v_ld, v_head, _dtype_code(k), tokens, _ptr(slots), _stream()))


def cache_read(cache, slots, out_dtype=None, k=None, v=None):
    """The keys and values in the slots (int32 [tokens]), decoded: k, v
    [tokens, heads, head_dim] of out_dtype (bf16 by default), zeros where a
    slot is outside the cache.  k, v: tensors to write, any pitches.  See
    mx_cache_read."""
    torch = _torch()
    if slots.dim() != 1:
        raise ValueError("slots must be [tokens]")
    tokens = slots.shape[0]
    _slot_vector(slots, tokens)
    shape = (tokens, cache.heads, cache.head_dim)
    given = k if k is not None else v
    out_dtype = out_dtype or (torch.bfloat16 if given is None else given.dtype)
    pitches = []
    for name, t in (("k", k), ("v", v)):
        pitches.append((0, 0) if t is None else _heads(t, name, shape, out_dtype, written=True))
    k = torch.empty(shape, dtype=out_dtype, device=slots.device) if k is None else k
    v = torch.empty_like(k, memory_format=torch.contiguous_format) if v is None else v
    _here(cache.device_index, k=k, v=v, slots=slots)
    _check("mx_cache_read", lib().mx_cache_read(
        cache._at, _ptr(k), *pitches[0], _ptr(v), *pitches[1], _dtype_code(k), tokens, _ptr(slots), _stream()))
    return k, v


def cache_attention(cache, q, page_table, lengths, scale=None, q_offsets=None, max_queries=None, causal: bool = True,
                    window: int = 0, sinks=None, out=None, lse=None, need_lse: bool = False, workspace=None):
    """Attention of the query rows q [tokens, q_heads, head_dim] (fp32 or bf16,
    any pitches) over the cache: (out of q's shape and type, lse fp32 [tokens,
    q_heads] or None).  page_table int32 [seqs, pages of a sequence], lengths
    int32 [seqs]: the tokens of each sequence in the cache, its queries' own
    included.  q_offsets int32 [seqs + 1]: the rows of each sequence; None: one
    each.  scale: 1 / sqrt(head_dim) by default.  causal, window, sinks (fp32
    [q_heads]) as in mx_cache_attention.  max_queries: the most rows of a
    sequence, which a batch of short ones should pass (without it the kernel
    is chosen as if one sequence had all rows).  fp32 queries are computed and
    returned to fp32 precision.  workspace: uint8, at least
    mx_cache_attention_workspace bytes, or None to allocate it."""
    torch = _torch()
    q_ld, q_head = _heads(q, "q")
    tokens, q_heads, dim = q.shape
    if dim != cache.head_dim:
        raise ValueError("q: expected a head_dim of %d, got %d" % (cache.head_dim, dim))
    table_ld = _rows(page_table, "page_table", None, torch.int32)
    seqs, table_pages = page_table.shape
    _same(lengths, (seqs,), torch.int32, "lengths")
    if q_offsets is not None:
        _same(q_offsets, (seqs + 1,), torch.int32, "q_offsets")
    if max_queries is None:
        max_queries = 1 if q_offsets is None else 0
    for name, value in (("window", window), ("max_queries", max_queries)):
        if not 0 <= value < 2 ** 31:
            raise ValueError("%s must be from 0 to 2^31 - 1" % name)
    if sinks is not None:
        _same(sinks, (q_heads,), torch.float32, "sinks")
    out_ld = out_head = 0
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        out_ld, out_head = _heads(out, "out", q.shape, q.dtype, written=True)
    if lse is not None:
        _same(lse, (tokens, q_heads), torch.float32, "lse")
    elif need_lse:
        lse = _new(q.device, torch.float32, tokens, q_heads)
    at = cache._at
    need = lib().mx_cache_attention_workspace(at, _dtype_code(q), tokens, q_heads, max_queries)
    workspace = _workspace(workspace, need, q.device)
    _here(cache.device_index, q=q, page_table=page_table, lengths=lengths, q_offsets=q_offsets, sinks=sinks, out=out,
          lse=lse, workspace=workspace)
    _check("mx_cache_attention", lib().mx_cache_attention(
        at, _ptr(q), _dtype_code(q), tokens, q_heads, q_ld, q_head, _ptr(q_offsets), max_queries, seqs,
        _ptr(page_table), table_ld, table_pages, _ptr(lengths), dim ** -0.5 if scale is None else float(scale),
        int(bool(causal)), window, _ptr(sinks), _ptr(out), out_ld, out_head, _ptr(lse), _ptr(workspace), _stream()))
    return out, lse
