"""Row operators of libmoe_fp8.so (include/moe_ops.h): token rows into expert
order and back with their gradients, microscaled 4-bit quantisation, and the
product of two microscaled 4-bit matrices.

One function per entry point.  Tensors are checked here (type, shape, layout,
device), before the library's own checks; outputs are allocated where none
is passed, on the stream the call runs on.  Matrices of bf16, f16 or f32 rows
may have a row stride; everything else is densely packed.  The functions take
no part in autograd: the gradients are entry points of their own.
"""
import ctypes

import torch

from . import _check, lib

MOE_DTYPE_BF16 = 0
MOE_DTYPE_F16 = 1
MOE_DTYPE_F32 = 2
MOE_DTYPE_U8 = 3

EXPORTED_SYMBOLS = (
    "moe_permute", "moe_permute_bwd", "moe_unpermute", "moe_unpermute_bwd",
    "moe_quantize_mxfp4", "moe_dequantize_mxfp4", "moe_gemm_mxfp4",
)

_DTYPES = {torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_F16,
           torch.float32: MOE_DTYPE_F32}
_DTYPES_U8 = {**_DTYPES, torch.uint8: MOE_DTYPE_U8}

_ops = None


def ops_lib():
    """libmoe_fp8.so with the argument types of the row operators set."""
    global _ops
    if _ops is None:
        L = lib()
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        L.moe_permute.argtypes = [i32] * 5 + [vp, i64, vp, vp, vp, vp, i64, vp]
        L.moe_permute_bwd.argtypes = [i32] * 5 + [vp, i64, vp, vp, i64, vp]
        L.moe_unpermute.argtypes = [i32] * 5 + [vp, i64, vp, vp, vp, i64, vp]
        L.moe_unpermute_bwd.argtypes = [i32] * 5 + [vp, i64, vp, i64, vp, vp, vp, vp, vp, i64, vp,
                                                    vp]
        L.moe_quantize_mxfp4.argtypes = [i32] * 3 + [vp, i64, vp, vp, vp]
        L.moe_dequantize_mxfp4.argtypes = [i32] * 3 + [vp, vp, vp, i64, vp]
        L.moe_gemm_mxfp4.argtypes = [i32] * 5 + [vp] * 7 + [i64, vp]
        for name in EXPORTED_SYMBOLS:
            getattr(L, name).restype = ctypes.c_int
        _ops = L
    return _ops


def _rows(t, name, device, dtypes=_DTYPES, dtype=None, shape=None):
    """Checks a matrix of rows; returns its row stride in elements."""
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected "
                         f"{shape if shape is not None else '[rows, width]'}")
    if t.dtype not in dtypes or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{name}: dtype {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    n, w = t.shape
    if (w > 1 and t.stride(1) != 1) or (n > 1 and t.stride(0) < w):
        raise ValueError(f"{name}: strides {t.stride()}, expected rows of adjacent elements "
                         "that do not overlap (call .contiguous())")
    return t.stride(0) if n > 1 else w


def _dense(t, name, device, dtype, numel=None, shape=None):
    """Checks a densely packed tensor; returns its address."""
    if t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: {t.dtype}, strides {t.stride()}, expected contiguous {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if (numel is not None and t.numel() != numel) or (shape is not None and tuple(t.shape) != shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected "
                         f"{shape if shape is not None else f'{numel} elements'}")
    return t.data_ptr()


class _Call:
    """The device and stream of one call: enters the tensors' device (and,
    where a stream is given, that stream, so that outputs allocated inside
    belong to it) and marks the tensors as used there."""

    def __init__(self, t, stream):
        dev = t.device
        if dev.type != "cuda":
            raise ValueError(f"tensors are on {dev}, expected a GPU")
        self.device = dev
        self.guard = None
        if stream is None:
            if dev.index != torch.cuda.current_device():
                self.guard = torch.cuda.device(dev)
            self.stream = None
        else:
            if isinstance(stream, int):
                stream = (torch.cuda.ExternalStream(stream, device=dev) if stream
                          else torch.cuda.default_stream(dev))
            if stream.device != dev:
                raise ValueError(f"stream on {stream.device}, tensors on {dev}")
            self.stream = stream
            self.guard = torch.cuda.stream(stream)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def handle(self, *tensors):
        """The stream's handle; the tensors passed are kept for it."""
        if self.stream is None:
            return torch.cuda.current_stream(self.device).cuda_stream
        for t in tensors:
            if t is not None:
                t.record_stream(self.stream)
        return self.stream.cuda_stream


def _slots(src_row, num_tokens, device):
    """Checks src_row [T*K] (any shape); returns its address and K."""
    n = src_row.numel()
    if num_tokens < 0 or (num_tokens == 0 and n) or (num_tokens and (n == 0 or n % num_tokens)):
        raise ValueError(f"src_row: {n} slots for {num_tokens} tokens")
    return _dense(src_row, "src_row", device, torch.int32), max(1, n // max(1, num_tokens))


def _used(offsets, device):
    """Address of the used-row count: the last entry of moe_route's offsets."""
    if offsets is None:
        return None
    if offsets.numel() < 1:
        raise ValueError("offsets: empty")
    return _dense(offsets, "offsets", device, torch.int32) + 4 * (offsets.numel() - 1)


def moe_permute(x, row_src, src_row, offsets, out=None, stream=None):
    """Token rows x [T, W] into the pool order of moe_route's lists: returns
    xp [pool_rows, W] with x[f // K] in row src_row[f], zeros in the padding
    rows below offsets[-1] (offsets None: all rows) and the rows from there on
    left as they were (a new xp: unset).  dtype bf16, f16, f32 or uint8."""
    with _Call(x, stream) as c:
        T, W = x.shape if x.dim() == 2 else (0, 0)
        x_ld = _rows(x, "x", c.device, _DTYPES_U8)
        src, K = _slots(src_row, T, c.device)
        R = row_src.numel()
        if out is None:
            out = torch.empty(R, W, dtype=x.dtype, device=c.device)
        ld = _rows(out, "out", c.device, _DTYPES_U8, x.dtype, (R, W))
        _check(ops_lib().moe_permute(
            T, K, R, W, _DTYPES_U8[x.dtype], x.data_ptr(), x_ld,
            _dense(row_src, "row_src", c.device, torch.int32), src, _used(offsets, c.device),
            out.data_ptr(), ld, c.handle(x, row_src, src_row, offsets, out)), "moe_permute")
    return out


def _token_sums(fn, what, rows, src_row, num_tokens, w, out, stream):
    with _Call(rows, stream) as c:
        ld = _rows(rows, "rows", c.device)
        R, W = rows.shape
        src, K = _slots(src_row, num_tokens, c.device)
        if out is None:
            out = torch.empty(num_tokens, W, dtype=rows.dtype, device=c.device)
        out_ld = _rows(out, "out", c.device, _DTYPES, rows.dtype, (num_tokens, W))
        args = [num_tokens, K, R, W, _DTYPES[rows.dtype], rows.data_ptr(), ld, src]
        if fn == "moe_unpermute":
            args.append(None if w is None else
                        _dense(w, "topk_w", c.device, torch.float32, num_tokens * K))
        _check(getattr(ops_lib(), fn)(*args, out.data_ptr(), out_ld,
                                      c.handle(rows, src_row, w, out)), what)
    return out


def moe_permute_bwd(dxp, src_row, num_tokens, out=None, stream=None):
    """Gradient of moe_permute: dx [T, W], each token's sum of its slots' rows
    of dxp [pool_rows, W] (f32 sums, rounded once)."""
    return _token_sums("moe_permute_bwd", "moe_permute_bwd", dxp, src_row, num_tokens, None, out,
                       stream)


def moe_unpermute(yp, src_row, num_tokens, topk_w=None, out=None, stream=None):
    """Expert rows yp [pool_rows, W] back to tokens: y [T, W], each token's sum
    of topk_w[t, j] (f32; None: 1) times its slots' rows."""
    return _token_sums("moe_unpermute", "moe_unpermute", yp, src_row, num_tokens, topk_w, out,
                       stream)


def moe_unpermute_bwd(dy, yp, row_src, src_row, offsets, topk_w=None, dyp=None, dw=None,
                      need_dyp=True, need_dw=True, stream=None):
    """Gradients of moe_unpermute for dy [T, W]: (dyp [pool_rows, W], dw f32
    [T, K]); dyp's padding rows below offsets[-1] are zeros, its rows from
    there on left as they were.  need_dyp / need_dw False: that one is None
    (without need_dw, yp is not read and may be None)."""
    with _Call(dy, stream) as c:
        ld = _rows(dy, "dy", c.device)
        T, W = dy.shape
        src, K = _slots(src_row, T, c.device)
        rs = _dense(row_src, "row_src", c.device, torch.int32)
        R = row_src.numel()
        yp_ld = dyp_ld = 0
        if need_dw:
            yp_ld = _rows(yp, "yp", c.device, _DTYPES, dy.dtype, (R, W))
            if dw is None:
                dw = torch.empty(T, K, dtype=torch.float32, device=c.device)
            _dense(dw, "dw", c.device, torch.float32, T * K)
        if need_dyp:
            if dyp is None:
                dyp = torch.empty(R, W, dtype=dy.dtype, device=c.device)
            dyp_ld = _rows(dyp, "dyp", c.device, _DTYPES, dy.dtype, (R, W))
        w = None if topk_w is None else _dense(topk_w, "topk_w", c.device, torch.float32, T * K)
        _check(ops_lib().moe_unpermute_bwd(
            T, K, R, W, _DTYPES[dy.dtype], dy.data_ptr(), ld,
            yp.data_ptr() if need_dw else None, yp_ld, rs, src, _used(offsets, c.device), w,
            dyp.data_ptr() if need_dyp else None, dyp_ld, dw.data_ptr() if need_dw else None,
            c.handle(dy, yp if need_dw else None, row_src, src_row, offsets, topk_w, dyp, dw)),
            "moe_unpermute_bwd")
    return (dyp if need_dyp else None), (dw if need_dw else None)


def moe_quantize_mxfp4(x, codes=None, sf=None, stream=None):
    """Rows x [M, C] (bf16, f16 or f32, C a multiple of 32) to packed e2m1
    codes uint8 [M, C/2] and UE8M0 scale codes uint8 [M, C/32]."""
    with _Call(x, stream) as c:
        ld = _rows(x, "x", c.device)
        M, C = x.shape
        if codes is None:
            codes = torch.empty(M, C // 2, dtype=torch.uint8, device=c.device)
        if sf is None:
            sf = torch.empty(M, C // 32, dtype=torch.uint8, device=c.device)
        _check(ops_lib().moe_quantize_mxfp4(
            M, C, _DTYPES[x.dtype], x.data_ptr(), ld,
            _dense(codes, "codes", c.device, torch.uint8, shape=(M, C // 2)),
            _dense(sf, "sf", c.device, torch.uint8, shape=(M, C // 32)),
            c.handle(x, codes, sf)), "moe_quantize_mxfp4")
    return codes, sf


def moe_dequantize_mxfp4(codes, sf, dtype=torch.bfloat16, out=None, stream=None):
    """The values [M, C] of e2m1 codes [M, C/2] and UE8M0 codes [M, C/32]."""
    with _Call(codes, stream) as c:
        if codes.dim() != 2 or dtype not in _DTYPES:
            raise ValueError(f"codes: shape {tuple(codes.shape)}; dtype {dtype}")
        M, C = codes.shape[0], 2 * codes.shape[1]
        if out is None:
            out = torch.empty(M, C, dtype=dtype, device=c.device)
        ld = _rows(out, "out", c.device, _DTYPES, dtype, (M, C))
        _check(ops_lib().moe_dequantize_mxfp4(
            M, C, _DTYPES[dtype], _dense(codes, "codes", c.device, torch.uint8),
            _dense(sf, "sf", c.device, torch.uint8, shape=(M, C // 32)), out.data_ptr(), ld,
            c.handle(codes, sf, out)), "moe_dequantize_mxfp4")
    return out


def moe_gemm_mxfp4(a, a_sf, b, b_sf, offsets=None, counts=None, dtype=None, out=None,
                   stream=None):
    """y [R, N] = a b^T of 4-bit microscaled a [R, K/2], a_sf [R, K/32] and
    b [N, K/2], b_sf [N, K/32] (dense), or b [E, N, K/2], b_sf [E, N, K/32]
    with offsets int32 [E+1] and counts int32 [E] (None: the segments'
    whole lengths): expert e's rows offsets[e] .. + counts[e], the other rows
    of y left as they were (a new y: unset).  y's type: out's, else dtype,
    else bf16."""
    with _Call(a, stream) as c:
        if a.dim() != 2 or b.dim() != (2 if offsets is None else 3):
            raise ValueError(f"a: shape {tuple(a.shape)}, b: shape {tuple(b.shape)}, expected "
                             "[rows, k/2] and [n, k/2], or [experts, n, k/2] with offsets")
        if offsets is None and counts is not None:
            raise ValueError("counts without offsets")
        R, K, N = a.shape[0], 2 * a.shape[1], b.shape[-2]
        E = 1 if offsets is None else b.shape[0]
        lead = () if offsets is None else (E,)
        if dtype is None:
            dtype = torch.bfloat16 if out is None else out.dtype
        if dtype not in _DTYPES:
            raise ValueError(f"dtype {dtype}")
        if out is None:
            out = torch.empty(R, N, dtype=dtype, device=c.device)
        ld = _rows(out, "out", c.device, _DTYPES, dtype, (R, N))
        u8, i32 = torch.uint8, torch.int32
        _check(ops_lib().moe_gemm_mxfp4(
            E, R, N, K, _DTYPES[dtype], _dense(a, "a", c.device, u8),
            _dense(a_sf, "a_sf", c.device, u8, shape=(R, K // 32)),
            _dense(b, "b", c.device, u8, shape=lead + (N, K // 2)),
            _dense(b_sf, "b_sf", c.device, u8, shape=lead + (N, K // 32)),
            None if offsets is None else _dense(offsets, "offsets", c.device, i32, E + 1),
            None if counts is None else _dense(counts, "counts", c.device, i32, E),
            out.data_ptr(), ld, c.handle(a, a_sf, b, b_sf, offsets, counts, out)),
            "moe_gemm_mxfp4")
    return out
