"""Row operators of libmoe_fp8.so (include/moe_ops.h): token rows into expert
order and back with their gradients, microscaled 4-bit quantisation, the
product of two microscaled 4-bit matrices, and around the experts' products the
router's choice, the residual norm and SwiGLU with 8-bit rows, each with its
gradient, and the experts' weight gradients from 8-bit rows.

One function per entry point.  Tensors are checked here (type, shape, layout,
device), before the library's own checks; outputs are allocated where none
is passed, on the stream the call runs on.  Matrices of bf16, f16 or f32 rows
may have a row stride; everything else is densely packed.  The functions take
no part in autograd: the gradients are entry points of their own.  So a call
whose gradient would be lost is refused (grad mode on, and a float tensor of a
permutation or an output requires grad): make it under torch.no_grad() or in an
autograd.Function, whose backward calls the gradient's entry point.
Quantisation, whose codes have no gradient, takes such an input.
"""
import ctypes

import torch

from . import MOE_ERR_INVALID_ARG, _check, lib

MOE_DTYPE_BF16 = 0
MOE_DTYPE_F16 = 1
MOE_DTYPE_F32 = 2
MOE_DTYPE_U8 = 3
MOE_SCORE_SOFTMAX = 0
MOE_SCORE_SIGMOID = 1
MOE_SF_F32_128 = 0
MOE_SF_UE8M0_32 = 1

EXPORTED_SYMBOLS = (
    "moe_permute", "moe_permute_bwd", "moe_unpermute", "moe_unpermute_bwd",
    "moe_quantize_mxfp4", "moe_dequantize_mxfp4", "moe_gemm_mxfp4", "moe_gemm_mxfp4_info",
    "moe_gate", "moe_gate_bwd", "moe_rms_norm", "moe_rms_norm_bwd",
    "moe_rms_norm_bwd_workspace_bytes", "moe_swiglu", "moe_swiglu_bwd",
    "moe_gemm_wgrad", "moe_gemm_wgrad_workspace_bytes",
)

_DTYPES = {torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_F16,
           torch.float32: MOE_DTYPE_F32}
_DTYPES_16 = {torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_F16}
_DTYPES_U8 = {**_DTYPES, torch.uint8: MOE_DTYPE_U8}

_ops = None


def ops_lib():
    """libmoe_fp8.so with the argument types of the row operators set."""
    global _ops
    if _ops is None:
        L = lib()
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        f32, size = ctypes.c_float, ctypes.c_size_t
        L.moe_permute.argtypes = [i32] * 5 + [vp, i64, vp, vp, vp, vp, i64, vp]
        L.moe_permute_bwd.argtypes = [i32] * 5 + [vp, i64, vp, vp, i64, vp]
        L.moe_unpermute.argtypes = [i32] * 5 + [vp, i64, vp, vp, vp, i64, vp]
        L.moe_unpermute_bwd.argtypes = [i32] * 5 + [vp, i64, vp, i64, vp, vp, vp, vp, vp, i64, vp,
                                                    vp]
        L.moe_quantize_mxfp4.argtypes = [i32] * 3 + [vp, i64, vp, vp, vp]
        L.moe_dequantize_mxfp4.argtypes = [i32] * 3 + [vp, vp, vp, i64, vp]
        L.moe_gemm_mxfp4.argtypes = [i32] * 5 + [vp] * 6 + [i32, vp, i64, vp]
        L.moe_gemm_mxfp4_info.argtypes = [i32] * 4 + [vp] * 2
        L.moe_gate.argtypes = [i32] * 4 + [vp, i64, vp, vp] + [i32] * 5 + [f32, vp, vp, vp]
        L.moe_gate_bwd.argtypes = [i32] * 4 + [vp, i64, vp, vp, i32, i32, f32, vp, i64, vp]
        L.moe_rms_norm.argtypes = ([i32] * 3 + [vp, i64, vp, i64, vp, i32, f32, vp, i64, vp, vp, i64,
                                                vp, vp, i32, vp])
        L.moe_rms_norm_bwd.argtypes = ([i32] * 3 + [vp, i64, vp, i64, vp, i32, vp, vp, i64, vp, i64, vp,
                                                    vp, size, vp])
        L.moe_rms_norm_bwd_workspace_bytes.argtypes = [i32, i32, vp]
        L.moe_swiglu.argtypes = [i32] * 3 + [vp, i64, f32, vp, vp, vp, i64] + [vp] * 4 + [i32, vp]
        L.moe_swiglu_bwd.argtypes = [i32] * 3 + [vp, i64, vp, i64, vp, vp, i32, f32, vp, vp, vp, i64, vp]
        L.moe_gemm_wgrad.argtypes = ([i32] * 5 + [vp, i64, vp, vp, i32, vp, vp, i32, vp, i32, vp, size, vp])
        L.moe_gemm_wgrad_workspace_bytes.argtypes = [i32] * 4 + [vp]
        for name in EXPORTED_SYMBOLS:
            getattr(L, name).restype = ctypes.c_int
        _ops = L
    return _ops


# The raw handle of a device's current stream; torch.cuda.current_stream
# builds a Stream object for it, a third of a small call's host time.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)

# The current device's number without torch.cuda's check that it is initialised
# (a tensor on a GPU shows that it is).
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _here(t, stream):
    """Whether a call with tensor t and this stream argument runs on the
    current device and its current stream."""
    if not t.is_cuda:
        raise ValueError(f"tensors are on {t.device}, expected a GPU")
    return stream is None and t.get_device() == _current_device()


def _elsewhere(fn, t, stream, *args, **kw):
    """fn(*args, **kw) on t's device and, if one is given, on `stream`, which
    is then the current one (new outputs belong to it) and is recorded as a
    user of every tensor of the call."""
    dev = t.device
    if stream is None:
        with torch.cuda.device(dev):
            return fn(*args, **kw)
    if isinstance(stream, int):
        stream = (torch.cuda.ExternalStream(stream, device=dev) if stream
                  else torch.cuda.default_stream(dev))
    if stream.device != dev:
        raise ValueError(f"stream on {stream.device}, tensors on {dev}")
    with torch.cuda.stream(stream):
        out = fn(*args, **kw)
    for v in (*args, *kw.values(), *(out if isinstance(out, tuple) else (out,))):
        if isinstance(v, torch.Tensor):
            v.record_stream(stream)
    return out


# Tells autograd that the library wrote a caller's tensors: what it saved of them
# is then refused in a backward pass, as after torch's own in-place writes.
_wrote = getattr(torch._C, "_increment_version", None) or torch.autograd.graph.increment_version


def _lost(name):
    """Refuses a tensor that requires grad, with grad mode on."""
    raise ValueError(f"{name}: requires grad, and the call would record no graph (make it under "
                     "torch.no_grad(), or in an autograd.Function with the gradient's entry point)")


def _rows(t, name, dev, dtype, rows, width, codes=False):
    """Checks a [rows, width] matrix of rows; returns its row stride in elements.
    codes: the call's results are codes, which have no gradient."""
    if t.requires_grad and not codes and torch.is_grad_enabled():
        _lost(name)
    if t.dtype is not dtype or t.shape != (rows, width) or t.get_device() != dev:
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)} on {t.device}, expected {dtype} "
                         f"{(rows, width)} on device {dev}")
    ld, one = t.stride()
    if (one != 1 and width > 1) or (ld < width and rows > 1):
        raise ValueError(f"{name}: strides {t.stride()}, expected rows of adjacent elements "
                         "that do not overlap (call .contiguous())")
    return ld if rows > 1 else width


_MAX = (1 << 31) - 1


def _int32(name, size):
    """Refuses a size (the largest of a call's) that the C ABI's int32 arguments
    cannot hold: ctypes would wrap it."""
    if size > _MAX:
        raise ValueError(f"{name}: {size}, beyond 32 bits")


def _matrix(t, name, dtypes):
    """The dtype code and shape of an input matrix of rows."""
    if t.dim() != 2 or t.dtype not in dtypes:
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)}, expected [rows, width] of "
                         f"{', '.join(str(d) for d in dtypes)}")
    rows, width = t.shape
    _int32(name, max(rows, width))
    return dtypes[t.dtype], rows, width


def _dense(t, name, dev, dtype, n):
    """Checks a densely packed tensor of n elements (or of shape n); returns its address."""
    if (t.dtype is not dtype or not t.is_contiguous() or t.get_device() != dev or
            (t.shape != n if isinstance(n, tuple) else t.numel() != n)):
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)}, strides {t.stride()} on {t.device}, "
                         f"expected contiguous {dtype} of {n if isinstance(n, tuple) else f'{n} elements'} "
                         f"on device {dev}")
    return t.data_ptr()


def _slots(src_row, num_tokens, dev):
    """Checks src_row [T*K] (any shape); returns its address and K."""
    n = src_row.numel()
    _int32("src_row", n)
    if num_tokens < 0 or (n % num_tokens or n == 0 if num_tokens else n):
        raise ValueError(f"src_row: {n} slots for {num_tokens} tokens")
    return _dense(src_row, "src_row", dev, torch.int32, n), n // num_tokens if num_tokens else 1


def _weights(topk_w, dev, n):
    """Checks topk_w (n elements, or None: all 1); returns its address."""
    if topk_w is None:
        return None
    if topk_w.requires_grad and torch.is_grad_enabled():
        _lost("topk_w")
    return _dense(topk_w, "topk_w", dev, torch.float32, n)


def _used(offsets, dev):
    """Address of the used-row count: the last entry of moe_route's offsets."""
    if offsets is None:
        return None
    n = offsets.numel()
    if n < 1:
        raise ValueError("offsets: empty")
    return _dense(offsets, "offsets", dev, torch.int32, n) + 4 * (n - 1)


_SF_BLOCK = {MOE_SF_F32_128: (128, torch.float32), MOE_SF_UE8M0_32: (32, torch.uint8)}


def _out(t, name, dev, like, rows, width):
    """A given output matrix of rows, checked, or a new one (which needs no check), of
    like's type: the tensor, its address and its row stride."""
    if t is None:
        t = (torch.empty_like(like) if like.shape == (rows, width) and like.is_contiguous() else
             torch.empty((rows, width), dtype=like.dtype, device=like.device))
        return t, t.data_ptr(), width
    return t, t.data_ptr(), _rows(t, name, dev, like.dtype, rows, width)


def _out_dense(t, name, dev, dtype, shape, device):
    """A given densely packed output, checked, or a new one: the tensor and its address."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        return t, t.data_ptr()
    if t.requires_grad and torch.is_grad_enabled():
        _lost(name)
    return t, _dense(t, name, dev, dtype, shape)


def _out_codes(codes, sf, name, dev, rows, cols, sf_format, device):
    """The given (checked) or new code and scale tensors of 8-bit rows in a format, and
    their addresses."""
    if sf_format not in _SF_BLOCK:
        raise ValueError(f"sf_format {sf_format}")
    block, dtype = _SF_BLOCK[sf_format]
    codes, codes_at = _out_dense(codes, name + "codes", dev, torch.uint8, (rows, cols), device)
    sf, sf_at = _out_dense(sf, name + "sf", dev, dtype, (rows, cols // block), device)
    return codes, sf, codes_at, sf_at


def _codes_at(codes, sf, name, dev, rows, cols, sf_format):
    """Checks 8-bit rows of a format; returns their addresses."""
    block, dtype = _SF_BLOCK[sf_format]
    return (_dense(codes, name + "codes", dev, torch.uint8, (rows, cols)),
            _dense(sf, name + "sf", dev, dtype, (rows, cols // block)))


def _sf_format(sf, name):
    """The format that a scale tensor's type tells."""
    for fmt, (_, dtype) in _SF_BLOCK.items():
        if sf.dtype is dtype:
            return fmt
    raise ValueError(f"{name}: {sf.dtype}, expected float32 (per 128 columns) or uint8 (UE8M0, per 32)")


def _norm_weight(weight, dev, dtype, width):
    """Checks a norm's weight (its rows' type or f32; None: 1); returns address and dtype code."""
    if weight is None:
        return None, MOE_DTYPE_F32
    if weight.requires_grad and torch.is_grad_enabled():
        _lost("weight")
    t = torch.float32 if weight.dtype is torch.float32 else dtype
    return _dense(weight, "weight", dev, t, (width,)), _DTYPES[t]


def moe_permute(x, row_src, src_row, offsets, out=None, stream=None):
    """Token rows x [T, W] into the pool order of moe_route's lists: returns
    xp [pool_rows, W] with x[f // K] in row src_row[f], zeros in the padding
    rows below offsets[-1] (offsets None: all rows) and the rows from there on
    left as they were (a new xp: unset).  dtype bf16, f16, f32 or uint8."""
    if not _here(x, stream):
        return _elsewhere(moe_permute, x, stream, x, row_src, src_row, offsets, out)
    dev = x.get_device()
    dt, T, W = _matrix(x, "x", _DTYPES_U8)
    src, K = _slots(src_row, T, dev)
    R = row_src.numel()
    _int32("row_src", R)
    given = out
    if out is None:
        out = torch.empty(R, W, dtype=x.dtype, device=x.device)
    _check(ops_lib().moe_permute(
        T, K, R, W, dt, x.data_ptr(), _rows(x, "x", dev, x.dtype, T, W),
        _dense(row_src, "row_src", dev, torch.int32, R), src, _used(offsets, dev),
        out.data_ptr(), _rows(out, "out", dev, x.dtype, R, W), _raw_stream(dev)), "moe_permute")
    if given is not None:
        _wrote((given,))
    return out


def moe_permute_bwd(dxp, src_row, num_tokens, out=None, stream=None):
    """Gradient of moe_permute: dx [T, W], each token's sum of its slots' rows
    of dxp [pool_rows, W] (f32 sums, rounded once)."""
    if not _here(dxp, stream):
        return _elsewhere(moe_permute_bwd, dxp, stream, dxp, src_row, num_tokens, out)
    dev = dxp.get_device()
    dt, R, W = _matrix(dxp, "dxp", _DTYPES)
    src, K = _slots(src_row, num_tokens, dev)
    given = out
    if out is None:
        out = torch.empty(num_tokens, W, dtype=dxp.dtype, device=dxp.device)
    _check(ops_lib().moe_permute_bwd(
        num_tokens, K, R, W, dt, dxp.data_ptr(), _rows(dxp, "dxp", dev, dxp.dtype, R, W), src,
        out.data_ptr(), _rows(out, "out", dev, dxp.dtype, num_tokens, W), _raw_stream(dev)),
        "moe_permute_bwd")
    if given is not None:
        _wrote((given,))
    return out


def moe_unpermute(yp, src_row, num_tokens, topk_w=None, out=None, stream=None):
    """Expert rows yp [pool_rows, W] back to tokens: y [T, W], each token's sum
    of topk_w[t, j] (f32; None: 1) times its slots' rows."""
    if not _here(yp, stream):
        return _elsewhere(moe_unpermute, yp, stream, yp, src_row, num_tokens, topk_w, out)
    dev = yp.get_device()
    dt, R, W = _matrix(yp, "yp", _DTYPES)
    src, K = _slots(src_row, num_tokens, dev)
    given = out
    if out is None:
        out = torch.empty(num_tokens, W, dtype=yp.dtype, device=yp.device)
    _check(ops_lib().moe_unpermute(
        num_tokens, K, R, W, dt, yp.data_ptr(), _rows(yp, "yp", dev, yp.dtype, R, W), src,
        _weights(topk_w, dev, num_tokens * K),
        out.data_ptr(), _rows(out, "out", dev, yp.dtype, num_tokens, W), _raw_stream(dev)),
        "moe_unpermute")
    if given is not None:
        _wrote((given,))
    return out


def moe_unpermute_bwd(dy, yp, row_src, src_row, offsets, topk_w=None, dyp=None, dw=None,
                      need_dyp=True, need_dw=True, stream=None):
    """Gradients of moe_unpermute for dy [T, W]: (dyp [pool_rows, W], dw f32
    [T, K]); dyp's padding rows below offsets[-1] are zeros, its rows from
    there on left as they were.  need_dyp / need_dw False: that one is None
    (without need_dw, yp is not read and may be None).  row_src None: dyp's
    padding rows are left as they were too (a new dyp: unset), and the pool has
    as many rows as yp, or as dyp where there is no yp."""
    if not _here(dy, stream):
        return _elsewhere(moe_unpermute_bwd, dy, stream, dy, yp, row_src, src_row, offsets, topk_w,
                          dyp, dw, need_dyp, need_dw)
    dev = dy.get_device()
    if not (need_dyp or need_dw):
        _check(MOE_ERR_INVALID_ARG, "moe_unpermute_bwd")
    dt, T, W = _matrix(dy, "dy", _DTYPES)
    src, K = _slots(src_row, T, dev)
    if need_dw and yp is None:
        raise ValueError("yp: None, needed for dw (need_dw=False leaves dw out)")
    pool = next((t for t in (row_src, yp, dyp) if t is not None), None)
    if pool is None:
        raise ValueError("none of row_src, yp and dyp, which the pool's rows are known by")
    R = row_src.numel() if row_src is not None else pool.shape[0] if pool.dim() else 0
    _int32("row_src", R)
    given = tuple(t for t, need in ((dyp, need_dyp), (dw, need_dw)) if need and t is not None)
    yp_at = dyp_at = dw_at = None
    yp_ld = dyp_ld = 0
    if need_dw:
        yp_at, yp_ld = yp.data_ptr(), _rows(yp, "yp", dev, dy.dtype, R, W)
        if dw is None:
            # (no tokens: src_row is empty and only topk_w knows the slots per token)
            k = topk_w.shape[1] if T == 0 and topk_w is not None and topk_w.dim() == 2 else K
            dw = torch.empty(T, k, dtype=torch.float32, device=dy.device)
        elif dw.requires_grad and torch.is_grad_enabled():
            _lost("dw")
        dw_at = _dense(dw, "dw", dev, torch.float32, T * K)
    if need_dyp:
        if dyp is None:
            dyp = torch.empty(R, W, dtype=dy.dtype, device=dy.device)
        dyp_at, dyp_ld = dyp.data_ptr(), _rows(dyp, "dyp", dev, dy.dtype, R, W)
    _check(ops_lib().moe_unpermute_bwd(
        T, K, R, W, dt, dy.data_ptr(), _rows(dy, "dy", dev, dy.dtype, T, W), yp_at, yp_ld,
        None if row_src is None else _dense(row_src, "row_src", dev, torch.int32, R), src,
        _used(offsets, dev),
        _weights(topk_w, dev, T * K),
        dyp_at, dyp_ld, dw_at, _raw_stream(dev)), "moe_unpermute_bwd")
    if given:
        _wrote(given)
    return (dyp if need_dyp else None), (dw if need_dw else None)


def moe_quantize_mxfp4(x, codes=None, sf=None, stream=None):
    """Rows x [M, C] (bf16, f16 or f32, C a multiple of 32) to packed e2m1
    codes uint8 [M, C/2] and UE8M0 scale codes uint8 [M, C/32]."""
    if not _here(x, stream):
        return _elsewhere(moe_quantize_mxfp4, x, stream, x, codes, sf)
    dev, u8 = x.get_device(), torch.uint8
    dt, M, C = _matrix(x, "x", _DTYPES)
    given = tuple(t for t in (codes, sf) if t is not None)
    if codes is None:
        codes = torch.empty(M, C // 2, dtype=u8, device=x.device)
    if sf is None:
        sf = torch.empty(M, C // 32, dtype=u8, device=x.device)
    _check(ops_lib().moe_quantize_mxfp4(
        M, C, dt, x.data_ptr(), _rows(x, "x", dev, x.dtype, M, C, codes=True),
        _dense(codes, "codes", dev, u8, (M, C // 2)), _dense(sf, "sf", dev, u8, (M, C // 32)),
        _raw_stream(dev)), "moe_quantize_mxfp4")
    if given:
        _wrote(given)
    return codes, sf


def moe_dequantize_mxfp4(codes, sf, dtype=torch.bfloat16, out=None, stream=None):
    """The values [M, C] of e2m1 codes [M, C/2] and UE8M0 codes [M, C/32]."""
    if not _here(codes, stream):
        return _elsewhere(moe_dequantize_mxfp4, codes, stream, codes, sf, dtype, out)
    dev, u8 = codes.get_device(), torch.uint8
    if codes.dim() != 2 or dtype not in _DTYPES:
        raise ValueError(f"codes: shape {tuple(codes.shape)}; dtype {dtype}")
    M, C = codes.shape[0], 2 * codes.shape[1]
    _int32("codes", max(M, C))
    given = out
    if out is None:
        out = torch.empty(M, C, dtype=dtype, device=codes.device)
    _check(ops_lib().moe_dequantize_mxfp4(
        M, C, _DTYPES[dtype], _dense(codes, "codes", dev, u8, (M, C // 2)),
        _dense(sf, "sf", dev, u8, (M, C // 32)), out.data_ptr(),
        _rows(out, "out", dev, dtype, M, C), _raw_stream(dev)), "moe_dequantize_mxfp4")
    if given is not None:
        _wrote((given,))
    return out


def moe_gemm_mxfp4(a, a_sf, b, b_sf, offsets=None, counts=None, dtype=None, out=None,
                   slots=0, stream=None):
    """y [R, N] = a b^T of 4-bit microscaled a [R, K/2], a_sf [R, K/32] and
    b [N, K/2], b_sf [N, K/32] (dense), or b [E, N, K/2], b_sf [E, N, K/32]
    with offsets int32 [E+1] and counts int32 [E] (None: the segments'
    whole lengths): expert e's rows offsets[e] .. + counts[e], the other rows
    of y left as they were (a new y: unset).  y's type: out's, else dtype,
    else bf16.  slots: an upper bound of the counts' sum (T * K), where a pool
    with padding has more rows than that (0: R; without counts not used)."""
    if not _here(a, stream):
        return _elsewhere(moe_gemm_mxfp4, a, stream, a, a_sf, b, b_sf, offsets, counts, dtype, out,
                          slots)
    dev, u8, i32 = a.get_device(), torch.uint8, torch.int32
    if a.dim() != 2 or b.dim() != (2 if offsets is None else 3):
        raise ValueError(f"a: shape {tuple(a.shape)}, b: shape {tuple(b.shape)}, expected "
                         "[rows, k/2] and [n, k/2], or [experts, n, k/2] with offsets")
    if offsets is None and counts is not None:
        raise ValueError("counts without offsets")
    R, k2 = a.shape
    N, nb = b.shape[-2], k2 // 16
    E, lead = (1, ()) if offsets is None else (b.shape[0], (b.shape[0],))
    _int32("sizes", max(E, R, N, 2 * k2, abs(slots)))
    if dtype is None:
        dtype = torch.bfloat16 if out is None else out.dtype
    if dtype not in _DTYPES:
        raise ValueError(f"dtype {dtype}")
    given = out
    if out is None:
        out = torch.empty(R, N, dtype=dtype, device=a.device)
    _check(ops_lib().moe_gemm_mxfp4(
        E, R, N, 2 * k2, _DTYPES[dtype], _dense(a, "a", dev, u8, (R, k2)),
        _dense(a_sf, "a_sf", dev, u8, (R, nb)), _dense(b, "b", dev, u8, lead + (N, k2)),
        _dense(b_sf, "b_sf", dev, u8, lead + (N, nb)),
        None if offsets is None else _dense(offsets, "offsets", dev, i32, E + 1),
        None if counts is None else _dense(counts, "counts", dev, i32, E), slots,
        out.data_ptr(), _rows(out, "out", dev, dtype, R, N), _raw_stream(dev)), "moe_gemm_mxfp4")
    if given is not None:
        _wrote((given,))
    return out


def moe_gemm_mxfp4_info(rows, n, k, groups=0):
    """Rows and columns of y per workgroup in a moe_gemm_mxfp4 call of these
    sizes (groups 0: dense), as {"tile_m", "tile_n"}."""
    _int32("sizes", max(map(abs, (rows, n, k, groups))))
    m, w = ctypes.c_int32(), ctypes.c_int32()
    _check(ops_lib().moe_gemm_mxfp4_info(groups, rows, n, k, ctypes.addressof(m),
                                         ctypes.addressof(w)), "moe_gemm_mxfp4_info")
    return {"tile_m": m.value, "tile_n": w.value}


def moe_gate(logits, top_k, bias=None, mask=None, score=MOE_SCORE_SOFTMAX, groups=1, top_groups=1,
             group_top=1, renorm=True, scale=1.0, topk_idx=None, topk_w=None, stream=None):
    """The router's choice: (topk_idx int32 [T, K], topk_w f32 [T, K]) of logits
    [T, E], largest first, ties to the lower id, -1 and 0 where no expert is left.
    Scores are the logits' softmax or sigmoid; bias f32 [E] shifts them for the choice
    alone; groups > 1: the top_groups groups with the largest sums of their group_top
    best experts are chosen from; renorm: weights divided by their sum; scale: times
    that.  mask bool or uint8 [T]: tokens with 0 get no expert."""
    if not _here(logits, stream):
        return _elsewhere(moe_gate, logits, stream, logits, top_k, bias, mask, score, groups, top_groups,
                          group_top, renorm, scale, topk_idx, topk_w)
    dev = logits.get_device()
    dt, T, E = _matrix(logits, "logits", _DTYPES)
    _int32("sizes", max(map(abs, (top_k, score, groups, top_groups, group_top))))
    if top_k > E:  # (before outputs of that size)
        _check(MOE_ERR_INVALID_ARG, "moe_gate")
    slots = (T, max(top_k, 0))
    if mask is not None and mask.dtype is torch.bool:
        mask = mask.view(torch.uint8)
    given = tuple(t for t in (topk_idx, topk_w) if t is not None)
    topk_idx, idx_at = _out_dense(topk_idx, "topk_idx", dev, torch.int32, slots, logits.device)
    topk_w, w_at = _out_dense(topk_w, "topk_w", dev, torch.float32, slots, logits.device)
    _check(ops_lib().moe_gate(
        T, E, top_k, dt, logits.data_ptr(), _rows(logits, "logits", dev, logits.dtype, T, E),
        None if bias is None else _dense(bias, "bias", dev, torch.float32, (E,)),
        None if mask is None else _dense(mask, "mask", dev, torch.uint8, (T,)),
        score, groups, top_groups, group_top, bool(renorm), scale, idx_at, w_at, _raw_stream(dev)), "moe_gate")
    if given:
        _wrote(given)
    return topk_idx, topk_w


def moe_gate_bwd(logits, topk_idx, dw, score=MOE_SCORE_SOFTMAX, renorm=True, scale=1.0, out=None, stream=None):
    """Gradient of moe_gate's weights: dlogits [T, E] for dw f32 [T, K], the choice
    topk_idx int32 [T, K] fixed."""
    if not _here(logits, stream):
        return _elsewhere(moe_gate_bwd, logits, stream, logits, topk_idx, dw, score, renorm, scale, out)
    dev = logits.get_device()
    dt, T, E = _matrix(logits, "logits", _DTYPES)
    if topk_idx.dim() != 2:
        raise ValueError(f"topk_idx: shape {tuple(topk_idx.shape)}, expected [T, K]")
    K = topk_idx.shape[1]
    _int32("sizes", max(K, abs(score)))
    if dw.requires_grad and torch.is_grad_enabled():
        _lost("dw")
    given = out
    out, out_at, out_ld = _out(out, "out", dev, logits, T, E)
    _check(ops_lib().moe_gate_bwd(
        T, E, K, dt, logits.data_ptr(), _rows(logits, "logits", dev, logits.dtype, T, E),
        _dense(topk_idx, "topk_idx", dev, torch.int32, (T, K)), _dense(dw, "dw", dev, torch.float32, (T, K)),
        score, bool(renorm), scale, out_at, out_ld, _raw_stream(dev)), "moe_gate_bwd")
    if given is not None:
        _wrote((given,))
    return out


def moe_rms_norm(x, weight=None, residual=None, eps=1e-6, need_y=True, sf_format=None, z=None, rstd=None, y=None,
                 codes=None, sf=None, stream=None):
    """Residual and root-mean-square norm of rows x [T, W]: (z, rstd, y, codes, sf).
    z = x + residual (None without a residual; z=residual or z=x: in place), rstd f32
    [T], y = z * rstd * weight in x's type (need_y), and y in 8 bits in a format
    (sf_format MOE_SF_F32_128: f32 scales per 128 columns, MOE_SF_UE8M0_32: UE8M0 codes
    per 32; None: codes and sf None).  weight [W] in x's type or f32 (None: 1)."""
    if not _here(x, stream):
        return _elsewhere(moe_rms_norm, x, stream, x, weight, residual, eps, need_y, sf_format, z, rstd, y, codes,
                          sf)
    dev = x.get_device()
    dt, T, W = _matrix(x, "x", _DTYPES)
    eight = sf_format is not None
    given = tuple(t for t in (z, rstd, y if need_y else None, *((codes, sf) if eight else ())) if t is not None)
    res_at = z_at = y_at = codes_at = sf_at = None
    res_ld = z_ld = y_ld = 0
    if residual is not None:
        res_at, res_ld = residual.data_ptr(), _rows(residual, "residual", dev, x.dtype, T, W)
        z, z_at, z_ld = _out(z, "z", dev, x, T, W)
    elif z is not None:
        raise ValueError("z: without a residual it is x")
    rstd, rstd_at = _out_dense(rstd, "rstd", dev, torch.float32, (T,), x.device)
    if need_y:
        y, y_at, y_ld = _out(y, "y", dev, x, T, W)
    if eight:
        codes, sf, codes_at, sf_at = _out_codes(codes, sf, "", dev, T, W, sf_format, x.device)
    w_at, w_dt = _norm_weight(weight, dev, x.dtype, W)
    _check(ops_lib().moe_rms_norm(
        T, W, dt, x.data_ptr(), _rows(x, "x", dev, x.dtype, T, W), res_at, res_ld, w_at, w_dt, eps, z_at, z_ld,
        rstd_at, y_at, y_ld, codes_at, sf_at, sf_format or 0, _raw_stream(dev)), "moe_rms_norm")
    if given:
        _wrote(given)
    return z, rstd, (y if need_y else None), (codes if eight else None), (sf if eight else None)


def moe_rms_norm_bwd_workspace_bytes(rows, width):
    """Bytes of workspace that moe_rms_norm_bwd needs for the weight's gradient."""
    _int32("sizes", max(map(abs, (rows, width))))
    n = ctypes.c_size_t()
    _check(ops_lib().moe_rms_norm_bwd_workspace_bytes(rows, width, ctypes.addressof(n)),
           "moe_rms_norm_bwd_workspace_bytes")
    return n.value


def moe_rms_norm_bwd(dy, z, rstd, weight=None, dz=None, dx=None, dw=None, need_dx=True, need_dw=True,
                     workspace=None, stream=None):
    """Gradients of moe_rms_norm for dy [T, W], through the z (without a residual: x) and
    rstd it returned: (dx [T, W], dw f32 [W]); dx is that of x and of the residual
    alike, dz [T, W] the gradient that reaches z on its other way (None: 0).  need_dx /
    need_dw False: that one is None.  workspace uint8, at least
    moe_rms_norm_bwd_workspace_bytes (None: allocated)."""
    if not _here(dy, stream):
        return _elsewhere(moe_rms_norm_bwd, dy, stream, dy, z, rstd, weight, dz, dx, dw, need_dx, need_dw,
                          workspace)
    dev = dy.get_device()
    if not (need_dx or need_dw):
        _check(MOE_ERR_INVALID_ARG, "moe_rms_norm_bwd")
    dt, T, W = _matrix(dy, "dy", _DTYPES)
    given = tuple(t for t, need in ((dx, need_dx), (dw, need_dw)) if need and t is not None)
    dz_at = dx_at = dw_at = ws_at = None
    dz_ld = dx_ld = ws_bytes = 0
    if dz is not None:
        dz_at, dz_ld = dz.data_ptr(), _rows(dz, "dz", dev, dy.dtype, T, W)
    if need_dx:
        dx, dx_at, dx_ld = _out(dx, "dx", dev, dy, T, W)
    if need_dw:
        dw, dw_at = _out_dense(dw, "dw", dev, torch.float32, (W,), dy.device)
        if workspace is None:
            workspace = torch.empty(moe_rms_norm_bwd_workspace_bytes(T, W), dtype=torch.uint8, device=dy.device)
        ws_bytes = workspace.numel()
        ws_at = _dense(workspace, "workspace", dev, torch.uint8, ws_bytes)
    w_at, w_dt = _norm_weight(weight, dev, dy.dtype, W)
    _check(ops_lib().moe_rms_norm_bwd(
        T, W, dt, dy.data_ptr(), _rows(dy, "dy", dev, dy.dtype, T, W), z.data_ptr(),
        _rows(z, "z", dev, dy.dtype, T, W), w_at, w_dt, _dense(rstd, "rstd", dev, torch.float32, (T,)), dz_at, dz_ld,
        dx_at, dx_ld, dw_at, ws_at, ws_bytes, _raw_stream(dev)), "moe_rms_norm_bwd")
    if given:
        _wrote(given)
    return (dx if need_dx else None), (dw if need_dw else None)


def moe_swiglu(gu, row_src=None, offsets=None, clamp=0.0, sf_format=None, need_h=True, need_h8=False,
               need_gu8=False, h=None, h_codes=None, h_sf=None, gu_codes=None, gu_sf=None, stream=None):
    """h = silu(gate) * up of pool rows gu [R, 2 I] (gate, then up): (h, h_codes, h_sf,
    gu_codes, gu_sf), those not needed None.  need_h: h [R, I] in gu's type; need_h8: h
    in 8 bits in sf_format, the second product's rows; need_gu8: gu in 8 bits, for
    moe_swiglu_bwd.  Rows with row_src < 0 and from offsets[-1] on (None: no such
    rows) are left as they were in every output (a new output: unset).  clamp > 0: gate and up
    are clamped to [-clamp, clamp] first."""
    if not _here(gu, stream):
        return _elsewhere(moe_swiglu, gu, stream, gu, row_src, offsets, clamp, sf_format, need_h, need_h8, need_gu8, h,
                          h_codes, h_sf, gu_codes, gu_sf)
    dev = gu.get_device()
    dt, R, W = _matrix(gu, "gu", _DTYPES)
    if W % 2:
        raise ValueError(f"gu: {W} columns, expected gate and up")
    inner = W // 2
    given = tuple(t for t, need in ((h, need_h), (h_codes, need_h8), (h_sf, need_h8), (gu_codes, need_gu8),
                                    (gu_sf, need_gu8)) if need and t is not None)
    h_at = hc_at = hsf_at = gc_at = gsf_at = None
    h_ld = 0
    if need_h:
        h, h_at, h_ld = _out(h, "h", dev, gu, R, inner)
    if need_h8:
        h_codes, h_sf, hc_at, hsf_at = _out_codes(h_codes, h_sf, "h_", dev, R, inner, sf_format, gu.device)
    if need_gu8:
        gu_codes, gu_sf, gc_at, gsf_at = _out_codes(gu_codes, gu_sf, "gu_", dev, R, W, sf_format, gu.device)
    _check(ops_lib().moe_swiglu(
        R, inner, dt, gu.data_ptr(), _rows(gu, "gu", dev, gu.dtype, R, W), clamp,
        None if row_src is None else _dense(row_src, "row_src", dev, torch.int32, R), _used(offsets, dev), h_at, h_ld,
        hc_at, hsf_at, gc_at, gsf_at, sf_format or 0, _raw_stream(dev)), "moe_swiglu")
    if given:
        _wrote(given)
    return (h if need_h else None, *((h_codes, h_sf) if need_h8 else (None, None)),
            *((gu_codes, gu_sf) if need_gu8 else (None, None)))


def moe_swiglu_bwd(dh, gu=None, gu_codes=None, gu_sf=None, row_src=None, offsets=None, clamp=0.0, out=None,
                   stream=None):
    """Gradient of moe_swiglu: dgu [R, 2 I] for dh [R, I], at the input gu, or at its
    8-bit copy gu_codes [R, 2 I], gu_sf (f32 per 128 columns or UE8M0 per 32).  Rows
    without a slot are left as they were; out=gu: in place."""
    if not _here(dh, stream):
        return _elsewhere(moe_swiglu_bwd, dh, stream, dh, gu, gu_codes, gu_sf, row_src, offsets, clamp, out)
    dev = dh.get_device()
    dt, R, inner = _matrix(dh, "dh", _DTYPES)
    _int32("dh", 2 * inner)
    if (gu is None) == (gu_codes is None) or (gu_codes is None) != (gu_sf is None):
        raise ValueError("gu, or gu_codes and gu_sf: exactly one of the two")
    given, fmt, gu_at, gu_ld, at = out, 0, None, 0, (None, None)
    if gu is not None:
        gu_at, gu_ld = gu.data_ptr(), _rows(gu, "gu", dev, dh.dtype, R, 2 * inner)
    else:
        fmt = _sf_format(gu_sf, "gu_sf")
        at = _codes_at(gu_codes, gu_sf, "gu_", dev, R, 2 * inner, fmt)
    out, out_at, out_ld = _out(out, "out", dev, dh, R, 2 * inner)
    _check(ops_lib().moe_swiglu_bwd(
        R, inner, dt, dh.data_ptr(), _rows(dh, "dh", dev, dh.dtype, R, inner), gu_at, gu_ld, *at, fmt, clamp,
        None if row_src is None else _dense(row_src, "row_src", dev, torch.int32, R), _used(offsets, dev),
        out_at, out_ld, _raw_stream(dev)), "moe_swiglu_bwd")
    if given is not None:
        _wrote((given,))
    return out


def moe_gemm_wgrad_workspace_bytes(groups, rows, n, k):
    """Bytes of workspace that a moe_gemm_wgrad call of these sizes needs."""
    _int32("sizes", max(map(abs, (groups, rows, n, k))))
    size = ctypes.c_size_t()
    _check(ops_lib().moe_gemm_wgrad_workspace_bytes(groups, rows, n, k, ctypes.addressof(size)),
           "moe_gemm_wgrad_workspace_bytes")
    return size.value


def moe_gemm_wgrad(dy, x, x_sf, offsets=None, counts=None, dtype=None, out=None, accumulate=False,
                   workspace=None, stream=None):
    """Weight gradients from 8-bit rows: dw [N, K] = dy^T x of dy [R, N] (bf16 or f16) and
    x [R, K] e4m3 with x_sf (f32 per 128 columns or UE8M0 per 32), or dw [E, N, K] with
    offsets int32 [E+1] and counts int32 [E] (None: the segments' whole lengths), each
    expert's from its rows, zeros for one without.  dw's type: out's, else dtype,
    else f32.  accumulate: out is added to.  workspace uint8, at least
    moe_gemm_wgrad_workspace_bytes (None: allocated)."""
    if not _here(dy, stream):
        return _elsewhere(moe_gemm_wgrad, dy, stream, dy, x, x_sf, offsets, counts, dtype, out, accumulate,
                          workspace)
    dev, i32 = dy.get_device(), torch.int32
    dt, R, N = _matrix(dy, "dy", _DTYPES_16)
    if x.dim() != 2:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected [rows, k]")
    if offsets is None and counts is not None:
        raise ValueError("counts without offsets")
    if accumulate and out is None:
        raise ValueError("accumulate without out")
    K = x.shape[1]
    E = 1
    if offsets is not None:
        E = offsets.numel() - 1
        if E < 1:
            raise ValueError(f"offsets: {E + 1} entries")
    _int32("sizes", max(E, K))
    if dtype is None:
        dtype = torch.float32 if out is None else out.dtype
    if dtype not in _DTYPES:
        raise ValueError(f"dtype {dtype}")
    shape = (N, K) if offsets is None else (E, N, K)
    given, fmt = out, _sf_format(x_sf, "x_sf")
    out, out_at = _out_dense(out, "out", dev, dtype, shape, dy.device)
    x_at, sf_at = _codes_at(x, x_sf, "x_", dev, R, K, fmt)
    need = moe_gemm_wgrad_workspace_bytes(E, R, N, K)
    ws_at, ws_bytes = None, 0
    if need:
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dy.device)
        ws_bytes = workspace.numel()
        ws_at = _dense(workspace, "workspace", dev, torch.uint8, ws_bytes)
    _check(ops_lib().moe_gemm_wgrad(
        E, R, N, K, dt, dy.data_ptr(), _rows(dy, "dy", dev, dy.dtype, R, N), x_at, sf_at, fmt,
        None if offsets is None else _dense(offsets, "offsets", dev, i32, E + 1),
        None if counts is None else _dense(counts, "counts", dev, i32, E), bool(accumulate),
        out_at, _DTYPES[dtype], ws_at, ws_bytes, _raw_stream(dev)), "moe_gemm_wgrad")
    if given is not None:
        _wrote((given,))
    return out
