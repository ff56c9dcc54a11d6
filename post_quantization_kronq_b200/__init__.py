"""KronQ per-layer quantization pass on NVIDIA B200 (sm_100a).

Python binding of libkronq.so: one wrapper per C entry point, same names,
argument marshalling only (torch tensors -> device pointers, the current CUDA
stream).  Every step of the pass runs in the library's CUDA kernels; PyTorch
supplies device memory and streams.  See ``include/kronq.h`` for the
contract of each call.
"""
from __future__ import annotations

import ctypes

from ._lib import (BF16, BIIP_MODES, F32, MXFP4, NVFP4, ORDERED_FP32, R_FORM, U_GIVEN, WRITE_E,
                   KronqError, QuantParams, check, lib)

__all__ = [
    "KronqError", "QuantParams", "U_GIVEN", "ORDERED_FP32", "WRITE_E", "R_FORM",
    "kronq_accumulate_factors", "kronq_sensitivity", "kronq_trace_tokens",
    "kronq_sensitivity_from_traces", "kronq_allocate_bits",
    "kronq_allocate_topn_types", "kronq_biip_workspace_bytes", "kronq_biip_forward",
    "kronq_biip_inverse", "kronq_quantize_workspace_bytes", "kronq_quantize_layer",
    "kronq_quantize_layer_static", "kronq_quantize_act_order_workspace_bytes",
    "kronq_quantize_layer_act_order", "kronq_quantize_two_sided_workspace_bytes", "kronq_quantize_two_sided",
    "kronq_pack", "kronq_unpack", "kronq_device_status", "kronq_wait_selftest",
    "kronq_kfac_loss_workspace_bytes",
    "kronq_kfac_loss", "kronq_launch_count", "kronq_last_error", "kronq_version", "workspace", "words_per_row",
    "EST_INPUT", "EST_MARGINAL", "EST_FROBENIUS", "EST_FLIPFLOP",
    "kronq_kron_factors_workspace_bytes", "kronq_kron_factors",
    "kronq_decode_matvec_workspace_bytes", "kronq_decode_matvec",
    "MXFP4", "NVFP4", "kronq_fp4_code_row_bytes", "kronq_fp4_scale_row_bytes",
    "kronq_fp4_quantize_workspace_bytes", "kronq_fp4_quantize", "kronq_fp4_dequantize",
    "kronq_fp4_matmul_workspace_bytes", "kronq_fp4_matmul", "kronq_fp4_matvec_workspace_bytes",
    "kronq_fp4_matvec", "kronq_fp4_grouped_matmul",
]

# kronq_estimator (Table 1 rows of the "WaterKron and FlipFlop Hessian" page)
EST_INPUT, EST_MARGINAL, EST_FROBENIUS, EST_FLIPFLOP = 0, 1, 2, 3


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _rowmajor(t, name):
    """The C ABI takes dense row-major arrays; refuse anything else loudly."""
    if t is not None and not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous row-major tensor")
    if t is not None and not t.is_cuda:
        raise ValueError(f"{name} must live in device memory")
    return t


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def workspace(nbytes: int, device="cuda"):
    """A device byte buffer for the calls that take a workspace (256-byte aligned)."""
    import torch
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def words_per_row(n: int, bits: int) -> int:
    return (n * bits + 31) // 32


def kronq_version() -> str:
    return lib.kronq_version().decode()


def kronq_launch_count() -> int:
    return int(lib.kronq_launch_count())


def kronq_last_error() -> str:
    return lib.kronq_last_error().decode(errors="replace")


def kronq_accumulate_factors(A, H, zero_first: bool = False, lda: int | None = None, stream=None):
    """H (d x d float32) += A^T A for A (T x d, bf16 or float32, row stride lda)."""
    T, d = A.shape
    if A.stride(1) != 1:
        raise ValueError("A must have unit stride along d (row-major token rows)")
    _rowmajor(H, "H")
    lda = A.stride(0) if lda is None else lda
    check(lib.kronq_accumulate_factors(_ptr(A), _dtype_code(A), T, d, lda, _ptr(H),
                                       1 if zero_first else 0, _stream(stream)))


def kronq_sensitivity(HX, HG, ws=None, stream=None):
    """(tr(H_X), tr(H_G), tr(H_G) * tr(H_X)) as Python floats (synchronises)."""
    _rowmajor(HX, "HX"), _rowmajor(HG, "HG")
    out = (ctypes.c_double * 3)()
    ws = workspace(256, HX.device) if ws is None else ws
    check(lib.kronq_sensitivity(_ptr(HX), HX.shape[0], _ptr(HG), HG.shape[0], out, _ptr(ws),
                                ws.numel(), _stream(stream)))
    return out[0], out[1], out[2]


def kronq_trace_tokens(A, trace, zero_first: bool = True, ws=None, stream=None):
    """trace (one device float64) (+)= sum_t |a_t|^2 = tr(A^T A) for tokens A (T x d)."""
    T, d = A.shape
    if A.stride(1) != 1:
        raise ValueError("A must have unit stride along d (row-major token rows)")
    _rowmajor(trace, "trace")
    ws = workspace(int(lib.kronq_trace_tokens_workspace_bytes()), A.device) if ws is None else ws
    check(lib.kronq_trace_tokens(_ptr(A), _dtype_code(A), T, d, A.stride(0), _ptr(trace),
                                 1 if zero_first else 0, _ptr(ws), ws.numel(), _stream(stream)))


def kronq_sensitivity_from_traces(traces, stream=None):
    """(tr(H_X), tr(H_G), tr(H_G) * tr(H_X)) from two device float64 traces (synchronises)."""
    _rowmajor(traces, "traces")
    out = (ctypes.c_double * 3)()
    check(lib.kronq_sensitivity_from_traces(_ptr(traces), out, _stream(stream)))
    return out[0], out[1], out[2]


def kronq_allocate_bits(sens, sizes, avg_bits: float = 2.5, bmin: int = 2, bmax: int = 4):
    L = len(sens)
    s = (ctypes.c_double * L)(*[float(v) for v in sens])
    z = (ctypes.c_int64 * L)(*[int(v) for v in sizes])
    out = (ctypes.c_int * L)()
    check(lib.kronq_allocate_bits(s, z, L, float(avg_bits), bmin, bmax, out))
    return list(out)


def kronq_allocate_topn_types(sens, type_ids, n_types: int, base_bits: int, N: int):
    L = len(sens)
    s = (ctypes.c_double * L)(*[float(v) for v in sens])
    t = (ctypes.c_int * L)(*[int(v) for v in type_ids])
    out = (ctypes.c_int * L)()
    check(lib.kronq_allocate_topn_types(s, t, L, n_types, base_bits, N, out))
    return list(out)


def kronq_biip_workspace_bytes(m: int, n: int) -> int:
    return int(lib.kronq_biip_workspace_bytes(m, n))


def kronq_biip_forward(W, Wt, HX, HG, seed: int, alpha: float, mode: str, d_in, d_out, ws=None,
                       stream=None):
    m, n = W.shape
    for t, name in ((W, "W"), (Wt, "Wt"), (HX, "HX"), (HG, "HG"), (d_in, "d_in"), (d_out, "d_out")):
        _rowmajor(t, name)
    ws = workspace(kronq_biip_workspace_bytes(m, n), W.device) if ws is None else ws
    check(lib.kronq_biip_forward(_ptr(W), _dtype_code(W), _ptr(Wt), m, n, _ptr(HX), _ptr(HG),
                                 int(seed), float(alpha), BIIP_MODES[mode], _ptr(d_in), _ptr(d_out),
                                 _ptr(ws), ws.numel(), _stream(stream)))


def kronq_biip_inverse(W, seed: int, mode: str, d_in, d_out, ws=None, stream=None):
    m, n = W.shape
    _rowmajor(W, "W")
    ws = workspace(kronq_biip_workspace_bytes(m, n), W.device) if ws is None else ws
    check(lib.kronq_biip_inverse(_ptr(W), m, n, int(seed), BIIP_MODES[mode], _ptr(d_in),
                                 _ptr(d_out), _ptr(ws), ws.numel(), _stream(stream)))


def kronq_quantize_workspace_bytes(m: int, n: int, params: QuantParams) -> int:
    return int(lib.kronq_quantize_workspace_bytes(m, n, ctypes.byref(params)))


def kronq_quantize_layer(Wt, HX, params: QuantParams, codes, scales, zeros, info, E=None, ws=None,
                         stream=None):
    m, n = Wt.shape
    for t, name in ((Wt, "Wt"), (HX, "HX"), (codes, "codes"), (scales, "scales"), (zeros, "zeros"),
                    (info, "info"), (E, "E")):
        _rowmajor(t, name)
    ws = workspace(kronq_quantize_workspace_bytes(m, n, params), Wt.device) if ws is None else ws
    check(lib.kronq_quantize_layer(_ptr(Wt), _ptr(HX), m, n, ctypes.byref(params), _ptr(codes),
                                   _ptr(scales), _ptr(zeros), _ptr(E), _ptr(info), _ptr(ws),
                                   ws.numel(), _stream(stream)))


def kronq_quantize_layer_static(Wt, HX, params: QuantParams, codes, scales, zeros, info, E=None,
                                stream=None):
    """kronq_quantize_layer without a workspace, for callers that cannot
    allocate device memory: the scratch is the library's 64 MiB static device
    array (shared by all calls on a device; overlapping calls race)."""
    m, n = Wt.shape
    for t, name in ((Wt, "Wt"), (HX, "HX"), (codes, "codes"), (scales, "scales"), (zeros, "zeros"),
                    (info, "info"), (E, "E")):
        _rowmajor(t, name)
    check(lib.kronq_quantize_layer_static(_ptr(Wt), _ptr(HX), m, n, ctypes.byref(params),
                                          _ptr(codes), _ptr(scales), _ptr(zeros), _ptr(E),
                                          _ptr(info), _stream(stream)))


def kronq_quantize_act_order_workspace_bytes(m: int, n: int, params: QuantParams) -> int:
    return int(lib.kronq_quantize_act_order_workspace_bytes(m, n, ctypes.byref(params)))


def kronq_quantize_layer_act_order(Wt, HX, params: QuantParams, codes, scales, zeros, g_idx, info,
                                   E=None, perm=None, ws=None, stream=None):
    """kronq_quantize_layer with the act-order sweep order; outputs in the
    original column order, scales/zeros per sweep-order group, g_idx (n int32)."""
    m, n = Wt.shape
    for t, name in ((Wt, "Wt"), (HX, "HX"), (codes, "codes"), (scales, "scales"), (zeros, "zeros"),
                    (g_idx, "g_idx"), (info, "info"), (E, "E"), (perm, "perm")):
        _rowmajor(t, name)
    if ws is None:
        ws = workspace(kronq_quantize_act_order_workspace_bytes(m, n, params), Wt.device)
    check(lib.kronq_quantize_layer_act_order(_ptr(Wt), _ptr(HX), m, n, ctypes.byref(params), _ptr(codes),
                                             _ptr(scales), _ptr(zeros), _ptr(E), _ptr(g_idx), _ptr(perm),
                                             _ptr(info), _ptr(ws), ws.numel(), _stream(stream)))


def kronq_quantize_two_sided_workspace_bytes(m: int, n: int, params: QuantParams) -> int:
    return int(lib.kronq_quantize_two_sided_workspace_bytes(m, n, ctypes.byref(params)))


def kronq_quantize_two_sided(Wt, HX, HG, params: QuantParams, codes, scales, zeros, info, E=None, ws=None,
                             stream=None):
    """Two-sided rounding under H_X (x) H_G; info holds two int32 (H_X, H_G)."""
    m, n = Wt.shape
    for t, name in ((Wt, "Wt"), (HX, "HX"), (HG, "HG"), (codes, "codes"), (scales, "scales"),
                    (zeros, "zeros"), (info, "info"), (E, "E")):
        _rowmajor(t, name)
    if info.numel() < 2:
        raise ValueError("info: two int32 (H_X, H_G)")
    if ws is None:
        ws = workspace(kronq_quantize_two_sided_workspace_bytes(m, n, params), Wt.device)
    check(lib.kronq_quantize_two_sided(_ptr(Wt), _ptr(HX), _ptr(HG), m, n, ctypes.byref(params), _ptr(codes),
                                       _ptr(scales), _ptr(zeros), _ptr(E), _ptr(info), _ptr(ws), ws.numel(),
                                       _stream(stream)))


def kronq_pack(codes, bits: int, out, stream=None):
    m, n = codes.shape
    _rowmajor(codes, "codes"), _rowmajor(out, "out")
    check(lib.kronq_pack(_ptr(codes), m, n, bits, _ptr(out), _stream(stream)))


def kronq_unpack(words, m: int, n: int, bits: int, codes, stream=None):
    check(lib.kronq_unpack(_ptr(words), m, n, bits, _ptr(codes), _stream(stream)))


def kronq_device_status(stream=None) -> int:
    v = ctypes.c_int(0)
    check(lib.kronq_device_status(ctypes.byref(v), _stream(stream)))
    return v.value


def kronq_wait_selftest(which: int, limit_ns: int, ws, stream=None):
    """One CTA whose bounded wait (0: mbarrier, 1: cross-CTA counter) is never
    satisfied gives up after limit_ns; read the result with kronq_device_status."""
    check(lib.kronq_wait_selftest(int(which), int(limit_ns), _ptr(ws), ws.numel() * ws.element_size(),
                                  _stream(stream)))


def kronq_kron_factors_workspace_bytes(T: int, n: int, m: int) -> int:
    return int(lib.kronq_kron_factors_workspace_bytes(T, n, m))


def kronq_kron_factors(X, G, est: int, iters: int, A, B, info, ws=None, stream=None):
    """Kronecker factors (A n x n, B m x m, fp32 out) of E[x x^T (x) g g^T]
    from bf16 tokens X (T x n) and G (T x m); info (device int) 0 on success."""
    import torch
    T, n = X.shape
    m = G.shape[1]
    if X.dtype != torch.bfloat16 or G.dtype != torch.bfloat16:
        raise ValueError("X and G must be bfloat16")
    for t, name in ((X, "X"), (G, "G"), (A, "A"), (B, "B"), (info, "info")):
        _rowmajor(t, name)
    ws = workspace(kronq_kron_factors_workspace_bytes(T, n, m), X.device) if ws is None else ws
    check(lib.kronq_kron_factors(_ptr(X), _ptr(G), T, n, m, int(est), int(iters), _ptr(A), _ptr(B),
                                 _ptr(info), _ptr(ws), ws.numel(), _stream(stream)))


def kronq_decode_matvec_workspace_bytes(m: int, n: int) -> int:
    return int(lib.kronq_decode_matvec_workspace_bytes(m, n))


def kronq_decode_matvec(packed, scales, zeros, n: int, bits: int, group: int, seed: int, mode: str,
                        d_in, d_out, x, y, ws=None, stream=None):
    """y (m, float32) = D_o^-1 U^T Q V D_i^-1 x from packed codes (int32 words)."""
    m = packed.shape[0]
    for t, name in ((packed, "packed"), (scales, "scales"), (zeros, "zeros"), (d_in, "d_in"),
                    (d_out, "d_out"), (x, "x"), (y, "y")):
        _rowmajor(t, name)
    ws = workspace(kronq_decode_matvec_workspace_bytes(m, n), x.device) if ws is None else ws
    check(lib.kronq_decode_matvec(_ptr(packed), _ptr(scales), _ptr(zeros), m, n, bits, group, seed,
                                  BIIP_MODES[mode], _ptr(d_in), _ptr(d_out), _ptr(x), _dtype_code(x),
                                  _ptr(y), _ptr(ws), ws.numel(), _stream(stream)))


def kronq_kfac_loss_workspace_bytes(m: int, n: int) -> int:
    return int(lib.kronq_kfac_loss_workspace_bytes(m, n))


def kronq_kfac_loss(E, HG, ws=None, stream=None) -> float:
    m, n = E.shape
    _rowmajor(E, "E"), _rowmajor(HG, "HG")
    ws = workspace(kronq_kfac_loss_workspace_bytes(m, n), E.device) if ws is None else ws
    out = ctypes.c_double(0.0)
    check(lib.kronq_kfac_loss(_ptr(E), _ptr(HG), m, n, ctypes.byref(out), _ptr(ws), ws.numel(),
                              _stream(stream)))
    return out.value


# ------------------------------------------------------------ microscaled 4-bit floating point
# These calls run once per layer and decoded token, so their marshalling is
# kept short: plain integers for pointers, sizes worked out here, torch looked
# up once.
_torch = None


def _fp4_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def kronq_fp4_code_row_bytes(n: int) -> int:
    return int(lib.kronq_fp4_code_row_bytes(n))


def kronq_fp4_scale_row_bytes(fmt: int, n: int) -> int:
    return int(lib.kronq_fp4_scale_row_bytes(fmt, n))


def _fp4_call(fn, device, stream, *args):
    """One library call with the tensors' device current, on the given stream or that device's current one."""
    cuda = (_torch or _fp4_torch())._C
    index = device.index
    if stream is None:
        raw = cuda._cuda_getCurrentRawStream(index)
    elif stream.device == device:
        raw = stream.cuda_stream
    else:
        raise ValueError(f"stream of {stream.device} for tensors on {device}")
    if cuda._cuda_getDevice() == index:
        status = fn(*args, raw)
    else:
        with _torch.cuda.device(device):
            status = fn(*args, raw)
    if status:
        check(status)


def _fp4_matrix(t, name):
    """(pointer, rows, columns, row stride) of a device matrix with dense rows."""
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a matrix in device memory")
    rows, n = t.shape
    ld, one = t.stride()
    if one != 1 and n > 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    # a single row may carry any stride: pass one that keeps its alignment
    return t.data_ptr(), rows, n, ld if rows > 1 else (n + 15) & ~15


def _fp4_pair(codes, scales, name, fmt, lead, n, device):
    """Pointers of a quantised matrix's codes and scales, whose shapes are lead + (row bytes,)."""
    if fmt == NVFP4:
        shape = lead + (((n + 255) >> 8) << 4,)
    elif fmt == MXFP4:
        shape = lead + (((n + 511) >> 9) << 4,)
    else:
        raise ValueError("fmt must be MXFP4 or NVFP4")
    uint8 = (_torch or _fp4_torch()).uint8
    if codes.shape != lead + (((n + 31) >> 5) << 4,) or codes.dtype is not uint8 or not codes.is_contiguous():
        raise ValueError(f"{name} codes must be contiguous uint8 of shape {lead + (((n + 31) >> 5) << 4,)}, got "
                         f"{codes.dtype} {tuple(codes.shape)}")
    if scales.shape != shape or scales.dtype is not uint8 or not scales.is_contiguous():
        raise ValueError(f"{name} scales must be contiguous uint8 of shape {shape}, got {scales.dtype} "
                         f"{tuple(scales.shape)}")
    if codes.device != device or scales.device != device:
        raise ValueError(f"{name} must live on {device}")
    return codes.data_ptr(), scales.data_ptr()


def _fp4_scale(t, name, fmt, count, device):
    if t is None:
        if fmt == NVFP4:
            raise ValueError(f"{name}: NVFP4 has a float32 tensor scale")
        return None
    if fmt != NVFP4:
        raise ValueError(f"{name}: MXFP4 has no tensor scale")
    if t.dtype is not _torch.float32 or t.numel() != count or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must hold {count} float32 on {device}")
    return t.data_ptr()


def _fp4_ws(ws, need, args, device, stream):
    """(pointer, bytes, owner) of the workspace; allocated where none is given
    and one is needed, on the call's stream, since it is freed before the
    kernels there have run."""
    if ws is None:
        nbytes = need(*args)
        if nbytes == 0:
            return None, 0, None
        if stream is None:
            ws = workspace(nbytes, device)
        else:
            with _torch.cuda.stream(stream):
                ws = workspace(nbytes, device)
    elif ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous on {device}")
    return ws.data_ptr(), ws.nbytes, ws


def _fp4_dtype(t):
    dt = t.dtype
    if dt is _torch.bfloat16:
        return BF16
    if dt is _torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {dt}")


def kronq_fp4_quantize_workspace_bytes(rows: int, n: int, fmt: int) -> int:
    return int(lib.kronq_fp4_quantize_workspace_bytes(rows, n, fmt))


def kronq_fp4_quantize(x, fmt: int, codes, scales, gscale=None, gscale_given: bool = False, deq=None, ws=None,
                       stream=None):
    """codes, scales (and NVFP4's gscale, unless given) of x (rows x n, bf16 or
    float32, dense rows); deq (x's type) receives the values they stand for."""
    px, rows, n, ldx = _fp4_matrix(x, "x")
    dev = x.device
    pc, ps = _fp4_pair(codes, scales, "output", fmt, (rows,), n, dev)
    pg = _fp4_scale(gscale, "gscale", fmt, 1, dev)
    pd, ldd = None, 0
    if deq is not None:
        pd, _, _, ldd = _fp4_matrix(deq, "deq")
        if deq.shape != x.shape or deq.dtype != x.dtype or deq.device != dev:
            raise ValueError("deq must have x's shape, type and device")
    pw, nw = None, 0
    if pg is not None and not gscale_given:
        pw, nw, ws = _fp4_ws(ws, kronq_fp4_quantize_workspace_bytes, (rows, n, fmt), dev, stream)
    _fp4_call(lib.kronq_fp4_quantize, dev, stream, px, _fp4_dtype(x), rows, n, ldx, fmt, pc, ps, pg,
              1 if gscale_given else 0, pd, ldd, pw, nw)


def kronq_fp4_dequantize(codes, scales, fmt: int, out, gscale=None, stream=None):
    """out (rows x n, bf16 or float32, dense rows) = the values of codes and scales."""
    po, rows, n, ldo = _fp4_matrix(out, "out")
    dev = out.device
    pc, ps = _fp4_pair(codes, scales, "input", fmt, (rows,), n, dev)
    pg = _fp4_scale(gscale, "gscale", fmt, 1, dev)
    _fp4_call(lib.kronq_fp4_dequantize, dev, stream, pc, ps, pg, fmt, rows, n, po, _fp4_dtype(out), ldo)


def kronq_fp4_matmul_workspace_bytes(T: int, m: int, n: int, fmt: int) -> int:
    return int(lib.kronq_fp4_matmul_workspace_bytes(T, m, n, fmt))


def kronq_fp4_matmul(xc, xs, wc, wsc, fmt: int, n: int, y, xg=None, wg=None, ws=None, stream=None):
    """y (T x m, bf16 or float32, dense rows) = X W^T for quantised X (T x n)
    and W (m x n), each as codes, scales and (NVFP4) a tensor scale."""
    py, T, m, ldy = _fp4_matrix(y, "y")
    dev = y.device
    pxc, pxs = _fp4_pair(xc, xs, "X", fmt, (T,), n, dev)
    pwc, pws = _fp4_pair(wc, wsc, "W", fmt, (m,), n, dev)
    pxg, pwg = _fp4_scale(xg, "xg", fmt, 1, dev), _fp4_scale(wg, "wg", fmt, 1, dev)
    pw, nw, ws = _fp4_ws(ws, kronq_fp4_matmul_workspace_bytes, (T, m, n, fmt), dev, stream)
    _fp4_call(lib.kronq_fp4_matmul, dev, stream, pxc, pxs, pxg, pwc, pws, pwg, fmt, T, m, n, py, _fp4_dtype(y),
              ldy, pw, nw)


def kronq_fp4_matvec_workspace_bytes(T: int, m: int, n: int, fmt: int) -> int:
    return int(lib.kronq_fp4_matvec_workspace_bytes(T, m, n, fmt))


def kronq_fp4_matvec(x, wc, wsc, fmt: int, y, wg=None, ws=None, stream=None):
    """y (T x m, bf16 or float32) = X W^T for at most 16 tokens X (T x n, bf16
    or float32, not quantised) and quantised W (m x n)."""
    px, T, n, ldx = _fp4_matrix(x, "x")
    py, Ty, m, ldy = _fp4_matrix(y, "y")
    dev = y.device
    if Ty != T or x.device != dev:
        raise ValueError("x and y must have the same rows and device")
    pwc, pws = _fp4_pair(wc, wsc, "W", fmt, (m,), n, dev)
    pwg = _fp4_scale(wg, "wg", fmt, 1, dev)
    pw, nw, ws = _fp4_ws(ws, kronq_fp4_matvec_workspace_bytes, (T, m, n, fmt), dev, stream)
    _fp4_call(lib.kronq_fp4_matvec, dev, stream, px, _fp4_dtype(x), ldx, pwc, pws, pwg, fmt, T, m, n, py,
              _fp4_dtype(y), ldy, pw, nw)


def kronq_fp4_grouped_matmul(xc, xs, offsets, wc, wsc, fmt: int, n: int, y, xg=None, wg=None, stream=None):
    """Rows [offsets[e], offsets[e + 1]) of y = those of X times expert e's
    weights: wc, wsc (E x m x row bytes), wg (E float32, NVFP4), offsets
    (E + 1 int32).  Rows of no group are left as they were."""
    import torch
    py, T, m, ldy = _fp4_matrix(y, "y")
    dev = y.device
    E = offsets.numel() - 1
    if offsets.dtype != torch.int32 or offsets.device != dev or not offsets.is_contiguous():
        raise ValueError(f"offsets must be contiguous int32 on {dev}")
    pxc, pxs = _fp4_pair(xc, xs, "X", fmt, (T,), n, dev)
    pwc, pws = _fp4_pair(wc, wsc, "W", fmt, (E, m), n, dev)
    pxg, pwg = _fp4_scale(xg, "xg", fmt, 1, dev), _fp4_scale(wg, "wg", fmt, E, dev)
    _fp4_call(lib.kronq_fp4_grouped_matmul, dev, stream, pxc, pxs, pxg, offsets.data_ptr(), E, pwc, pws, pwg, fmt, T,
              m, n, py, _fp4_dtype(y), ldy)
