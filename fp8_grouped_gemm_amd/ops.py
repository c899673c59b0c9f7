"""Row operators of libmoe_fp8.so (include/moe_ops.h): token rows into expert
order and back with their gradients, microscaled 4-bit quantisation, and the
product of two microscaled 4-bit matrices.

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

EXPORTED_SYMBOLS = (
    "moe_permute", "moe_permute_bwd", "moe_unpermute", "moe_unpermute_bwd",
    "moe_quantize_mxfp4", "moe_dequantize_mxfp4", "moe_gemm_mxfp4", "moe_gemm_mxfp4_info",
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
        L.moe_gemm_mxfp4.argtypes = [i32] * 5 + [vp] * 6 + [i32, vp, i64, vp]
        L.moe_gemm_mxfp4_info.argtypes = [i32] * 4 + [vp] * 2
        for name in EXPORTED_SYMBOLS:
            getattr(L, name).restype = ctypes.c_int
        _ops = L
    return _ops


# The raw handle of a device's current stream; torch.cuda.current_stream
# builds a Stream object for it, a third of a small call's host time.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _here(t, stream):
    """Whether a call with tensor t and this stream argument runs on the
    current device and its current stream."""
    if not t.is_cuda:
        raise ValueError(f"tensors are on {t.device}, expected a GPU")
    return stream is None and t.get_device() == torch.cuda.current_device()


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
