"""ctypes binding of libnvfp4moe.so (see include/nvfp4moe.h for the contract).

Argument marshalling only: shape/dtype/device checks, output allocation with
torch (device memory), the current stream, and status-code -> exception.
"""

import ctypes
import functools
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnvfp4moe.so")
TENSORS_LIB_PATH = os.path.join(os.path.dirname(LIB_PATH), "libnvfp4moe_tensors.so")

NVFP4MOE_F32 = 0
NVFP4MOE_BF16 = 1
_OUTER_PER_ROW, _OUTER_PER_GROUP = 0, 1
_LAYOUT_TRANSPOSED, _LAYOUT_PER_GROUP = 0, 1
_ROWWISE, _COLWISE_GROUPED = 0, 1
_EINVAL, _EUNSUPPORTED = 1, 2
_SCORES = {"softmax": 0, "sigmoid": 1}
_FORMATS = {3: 0, 2: 1}                 # parts of a weight: NVFP4 (with outer scales), MXFP4
_ACTS = {"none": 0, "relu2": 1, "silu": 2}

_c_i64 = ctypes.c_int64
_c_int = ctypes.c_int
_c_u32 = ctypes.c_uint32
_c_u64 = ctypes.c_uint64
_c_size = ctypes.c_size_t
_c_f32 = ctypes.c_float
_p = ctypes.c_void_p

# name -> argument types (all return int status, except where noted)
SIGNATURES = {
    "nvfp4moe_abi_version": ([], _c_int),
    "nvfp4moe_status_string": ([_c_int], ctypes.c_char_p),
    "nvfp4_quantize": ([_p, _c_int, _c_i64, _c_i64, _c_int, _c_i64, _p, _p, _p, _p], _c_int),
    "nvfp4moe_permute_workspace_size": ([_c_i64, _c_int, _c_int], _c_size),
    "moe_permute": ([_p, _c_i64, _c_int, _c_int, _c_int, _p, _p, _p, _c_i64, _p, _p, _p, _p,
                     _p, _p, _p, _p, _p, _c_size, _p], _c_int),
    "moe_permute_noalloc": ([_p, _c_i64, _c_int, _c_int, _c_int, _p, _p, _p, _c_i64, _p, _p, _p,
                             _p, _p, _p, _p, _p, _p], _c_int),
    "moe_fwd_grouped_gemm": ([_p, _p, _p, _p, _p, _p, _p, _c_int, _c_i64, _c_i64, _c_i64, _p,
                              _c_int, _p], _c_int),
    "mxfp8_requant_sr": ([_p, _p, _p, _c_int, _c_i64, _c_i64, _c_i64, _p, _p, _c_int, _c_i64,
                          _c_u64, _c_u32, _p, _p, _p], _c_int),
    "mxfp8_quantize": ([_p, _c_int, _c_i64, _c_i64, _c_int, _p, _p, _c_int, _c_i64, _p, _p, _p],
                       _c_int),
    "moe_bwd_dgrad": ([_p, _p, _p, _p, _p, _c_int, _c_i64, _c_i64, _c_i64, _p, _c_int, _p],
                      _c_int),
    "moe_bwd_wgrad": ([_p, _p, _p, _p, _p, _c_int, _c_i64, _c_i64, _c_i64, _p, _p], _c_int),
    "moe_fwd_grouped_gemm_mxfp8": ([_p, _p, _p, _p, _p, _c_int, _c_i64, _c_i64, _c_i64, _p,
                                    _c_int, _p], _c_int),
    "mxfp8_gather_rows": ([_p, _p, _c_int, _c_i64, _p, _p, _c_i64, _c_i64, _p, _p, _p], _c_int),
    "nvfp4_quantize_tile16": ([_p, _c_int, _c_i64, _c_i64, _c_i64, _p, _p, _p, _p], _c_int),
    "mxfp8_quantize_dual": ([_p, _c_int, _c_i64, _c_i64, _p, _p, _c_int, _c_i64, _p, _p, _p, _p,
                             _p], _c_int),
    "nvfp4_quantize_live": ([_p, _c_int, _c_i64, _c_i64, _p, _p, _p, _p, _p], _c_int),
    "moe_combine": ([_p, _c_int, _c_i64, _c_i64, _c_int, _c_i64, _p, _p, _p, _c_int, _p], _c_int),
    "moe_combine_bwd": ([_p, _c_int, _c_i64, _c_int, _c_i64, _p, _p, _p, _c_int, _c_i64, _p, _p,
                         _c_int, _p, _c_int, _p, _p], _c_int),
    "moe_padded_offsets": ([_p, _c_int, _c_int, _p, _p], _c_int),
    "nvfp4_quantize_sr": ([_p, _c_int, _c_i64, _c_i64, _c_u64, _c_u32, _p, _p, _p, _p], _c_int),
    "nvfp4_requant_sr": ([_p, _p, _p, _c_int, _c_i64, _c_i64, _c_i64, _p, _p, _c_int, _c_i64,
                          _c_int, _c_u64, _c_u32, _p, _p, _p, _p], _c_int),
    "nvfp4_quantize_sr_colwise": ([_p, _c_int, _c_i64, _c_i64, _p, _p, _c_int, _c_i64, _c_u64,
                                   _c_u32, _p, _p, _p, _p], _c_int),
    "moe_bwd_wgrad_nvfp4": ([_p, _p, _p, _p, _p, _p, _p, _c_int, _c_i64, _c_i64, _c_i64, _p, _p],
                            _c_int),
    "nvfp4moe_route_workspace_size": ([_c_i64, _c_int], _c_size),
    "moe_route": ([_p, _c_int, _c_i64, _c_int, _c_int, _c_int, _c_int, _c_f32, _p, _p, _p, _p, _p,
                   _p, _p, _c_size, _p], _c_int),
    "moe_balance_loss": ([_p, _p, _c_int, _c_int, _c_f32, _p, _p], _c_int),
    "moe_route_bwd": ([_p, _c_int, _c_i64, _c_int, _c_int, _c_int, _c_int, _c_f32, _p, _p, _p,
                       _c_f32, _p, _p, _p], _c_int),
    "nvfp4moe_grad_workspace_size": ([_p, _c_int], _c_size),
    "moe_grad_sumsq": ([_p, _p, _p, _c_int, _p, _p, _c_size, _p], _c_int),
    "moe_grad_clip": ([_p, _p, _p, _p, _c_int, _p, _c_f32, _p, _p], _c_int),
    "mxfp4_quantize": ([_p, _c_int, _c_i64, _c_i64, _p, _p, _p, _p], _c_int),
    "mxfp4_dequantize": ([_p, _p, _c_i64, _c_i64, _p, _c_int, _p], _c_int),
    "mxfp8_dequantize": ([_p, _p, _c_i64, _c_i64, _p, _c_int, _p], _c_int),
    "moe_group": ([_p, _c_i64, _c_int, _c_int, _c_int, _p, _p, _p, _p, _p, _p, _c_size, _p], _c_int),
    "moe_fwd_grouped_gemm_mxfp4": ([_p, _p, _c_i64, _p, _p, _p, _p, _c_int, _c_i64, _c_i64, _c_i64,
                                    _p, _c_int, _p], _c_int),
    "mxfp8_requant_sr_mxfp4": ([_p, _p, _c_i64, _c_i64, _p, _c_i64, _p, _p, _c_int, _c_i64, _c_u64,
                                _c_u32, _p, _p, _p], _c_int),
    "nvfp4moe_ffn_tokens_workspace_size": ([_c_i64, _c_int, _c_i64, _c_i64], _c_size),
    "moe_ffn_tokens": ([_p, _p, _c_int, _c_i64, _c_int, _c_int, _c_int, _c_int, _c_f32, _p, _p,
                        _c_int, _p, _p, _p, _p, _p, _p, _c_int, _c_int, _c_i64, _c_i64, _c_int,
                        _c_int, _p, _p, _p, _c_int, _p, _c_size, _p], _c_int),
}

_LIB = None
_TORCH = None


class Nvfp4moeError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: status {status} ({status_string(status)})")


def lib():
    """Load libnvfp4moe.so once; raise if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m precision_moe_numerics_nvfp4_amd.build` (or __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            f = getattr(L, name, None)
            if f is None:
                raise RuntimeError(
                    f"{LIB_PATH} lacks {name}: it is older than this package, build it again with "
                    "`python -m precision_moe_numerics_nvfp4_amd.build` (or __graft_entry__.build())")
            f.argtypes = args
            f.restype = res
        _LIB = L
    return _LIB


def abi_version():
    return lib().nvfp4moe_abi_version()


def status_string(status):
    return lib().nvfp4moe_status_string(int(status)).decode()


def _check(fn, status):
    if status != 0:
        raise Nvfp4moeError(fn, status)


def _torch():
    """torch, imported with the first call that needs it."""
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _dev(t, name, dtype=None, ndim=None):
    torch = _TORCH or _torch()
    if t.__class__ is torch.Tensor and t.is_cuda and t.is_contiguous() and \
            (dtype is None or t.dtype is dtype) and (ndim is None or t.dim() == ndim):
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor (got {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions (got {t.dim()})")
    return t


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream(t):
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _in_dtype(x):
    torch = _torch()
    if x.dtype == torch.float32:
        return NVFP4MOE_F32
    if x.dtype == torch.bfloat16:
        return NVFP4MOE_BF16
    raise ValueError(f"input must be float32 or bfloat16 (got {x.dtype})")


def _out_dtype(dtype):
    torch = _torch()
    if dtype == torch.float32:
        return NVFP4MOE_F32
    if dtype == torch.bfloat16:
        return NVFP4MOE_BF16
    raise ValueError(f"output dtype must be float32 or bfloat16 (got {dtype})")


def nvfp4_quantize(x, rows_per_group=None, codes=None, scales=None, outer=None):
    """x [rows, cols] float32|bfloat16 -> (codes [rows, cols/2] u8, scales
    [rows, cols/16] u8, outer f32 [rows] or [rows/rows_per_group])."""
    torch = _torch()
    _dev(x, "x", ndim=2)
    rows, cols = x.shape
    dev = x.device
    if codes is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=dev)
    n_outer = rows if rows_per_group is None else rows // max(int(rows_per_group), 1)
    if outer is None:
        outer = torch.empty((n_outer,), dtype=torch.float32, device=dev)
    mode = _OUTER_PER_ROW if rows_per_group is None else _OUTER_PER_GROUP
    st = lib().nvfp4_quantize(_ptr(x), _in_dtype(x), rows, cols, mode,
                              0 if rows_per_group is None else int(rows_per_group),
                              _ptr(codes), _ptr(scales), _ptr(outer), _stream(x))
    _check("nvfp4_quantize", st)
    return codes, scales, outer


def permute_workspace_size(T, k, n_local):
    return int(lib().nvfp4moe_permute_workspace_size(int(T), int(k), int(n_local)))


def moe_permute(topk_ids, e0, n_local, xq_codes, xq_scales, xq_outer, workspace=None, out=None):
    """Group routed (token, slot) pairs by local expert and gather NVFP4 rows.

    Returns a dict with offsets, padded_offsets (int64 [n_local+1]), row_token,
    row_slot (int32 [T*k]), pair_row (int32 [T, k], the row of each pair or
    -1) and codes/scales/outer of the permuted rows (capacity T*k rows; rows
    >= offsets[-1] are not written). An ``out`` dict without "pair_row" asks
    for no inverse map."""
    torch = _torch()
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    T, k = topk_ids.shape
    _dev(xq_codes, "xq_codes", torch.uint8, 2)
    _dev(xq_scales, "xq_scales", torch.uint8, 2)
    _dev(xq_outer, "xq_outer", torch.float32, 1)
    K = xq_codes.shape[1] * 2
    dev = topk_ids.device
    cap = T * k
    o = dict(out or {})
    if out is None:
        o["pair_row"] = torch.empty((T, k), dtype=torch.int32, device=dev)
    o.setdefault("offsets", torch.empty((n_local + 1,), dtype=torch.int64, device=dev))
    o.setdefault("padded_offsets", torch.empty((n_local + 1,), dtype=torch.int64, device=dev))
    o.setdefault("row_token", torch.empty((cap,), dtype=torch.int32, device=dev))
    o.setdefault("row_slot", torch.empty((cap,), dtype=torch.int32, device=dev))
    o.setdefault("codes", torch.empty((cap, K // 2), dtype=torch.uint8, device=dev))
    o.setdefault("scales", torch.empty((cap, K // 16), dtype=torch.uint8, device=dev))
    o.setdefault("outer", torch.empty((cap,), dtype=torch.float32, device=dev))
    ws_bytes = permute_workspace_size(T, k, n_local)
    if workspace is None:
        workspace = torch.empty((ws_bytes,), dtype=torch.uint8, device=dev)
    st = lib().moe_permute(_ptr(topk_ids), T, k, int(e0), int(n_local), _ptr(xq_codes),
                           _ptr(xq_scales), _ptr(xq_outer), K, _ptr(o["offsets"]),
                           _ptr(o["padded_offsets"]), _ptr(o["row_token"]), _ptr(o["row_slot"]),
                           _ptr(o.get("pair_row")), _ptr(o["codes"]), _ptr(o["scales"]), _ptr(o["outer"]),
                           _ptr(workspace), workspace.numel(), _stream(topk_ids))
    _check("moe_permute", st)
    return o


def moe_permute_noalloc(topk_ids, e0, n_local, xq_codes, xq_scales, xq_outer, out):
    """moe_permute through the entry point that allocates nothing: the
    library keeps the count table in its own per-GPU array (at most 4 MiB,
    see the header), and every output buffer comes from the caller in `out`
    (the dict moe_permute returns or takes; "pair_row" optional)."""
    torch = _torch()
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    T, k = topk_ids.shape
    _dev(xq_codes, "xq_codes", torch.uint8, 2)
    _dev(xq_scales, "xq_scales", torch.uint8, 2)
    _dev(xq_outer, "xq_outer", torch.float32, 1)
    K = xq_codes.shape[1] * 2
    for name in ("offsets", "padded_offsets", "row_token", "row_slot", "codes", "scales", "outer"):
        if name not in out:
            raise ValueError(f"moe_permute_noalloc: out lacks {name}")
    st = lib().moe_permute_noalloc(_ptr(topk_ids), T, k, int(e0), int(n_local), _ptr(xq_codes),
                                   _ptr(xq_scales), _ptr(xq_outer), K, _ptr(out["offsets"]),
                                   _ptr(out["padded_offsets"]), _ptr(out["row_token"]),
                                   _ptr(out["row_slot"]), _ptr(out.get("pair_row")),
                                   _ptr(out["codes"]), _ptr(out["scales"]), _ptr(out["outer"]),
                                   _stream(topk_ids))
    _check("moe_permute_noalloc", st)
    return out


def moe_fwd_grouped_gemm(a_codes, a_scales, a_outer, b_codes, b_scales, b_outer, offsets,
                         out_dtype=None, y=None):
    """y [m_cap, N] = grouped NVFP4 GEMM (see the header). b_* are [G*N, ...]
    or [G, N, ...]; offsets int64 [G+1] on the device."""
    torch = _torch()
    out_dtype = out_dtype or torch.float32
    _dev(a_codes, "a_codes", torch.uint8, 2)
    _dev(a_scales, "a_scales", torch.uint8, 2)
    _dev(a_outer, "a_outer", torch.float32, 1)
    _dev(b_codes, "b_codes", torch.uint8)
    _dev(b_scales, "b_scales", torch.uint8)
    _dev(b_outer, "b_outer", torch.float32, 1)
    _dev(offsets, "offsets", torch.int64, 1)
    m_cap, K = a_codes.shape[0], a_codes.shape[1] * 2
    G = b_outer.shape[0]
    N = b_codes.numel() // (G * (K // 2)) if G else 0
    if y is None:
        y = torch.empty((m_cap, N), dtype=out_dtype, device=a_codes.device)
    st = lib().moe_fwd_grouped_gemm(_ptr(a_codes), _ptr(a_scales), _ptr(a_outer), _ptr(b_codes),
                                    _ptr(b_scales), _ptr(b_outer), _ptr(offsets), G, m_cap, N, K,
                                    _ptr(y), _out_dtype(y.dtype), _stream(a_codes))
    _check("moe_fwd_grouped_gemm", st)
    return y


def mxfp8_requant_sr(codes, scales, outer, offsets, padded_offsets, P, seed, tag,
                     rows_per_group=None, out=None, out_e8=None):
    """Saved NVFP4 [rows, cols] -> MXFP8 with stochastic rounding, grouped
    transpose per offsets/padded_offsets: activations (per-row outer scales)
    [cols, P] (+ E8M0 [cols, P/32]); weights (rows_per_group) per-expert blocks
    [G * cols, rows_per_group] (+ [G * cols, rows_per_group/32]), P = G *
    rows_per_group."""
    torch = _torch()
    _dev(codes, "codes", torch.uint8, 2)
    _dev(scales, "scales", torch.uint8, 2)
    _dev(outer, "outer", torch.float32, 1)
    _dev(offsets, "offsets", torch.int64, 1)
    _dev(padded_offsets, "padded_offsets", torch.int64, 1)
    rows, cols = codes.shape[0], codes.shape[1] * 2
    G = offsets.shape[0] - 1
    dev = codes.device
    if rows_per_group is None:
        shape = (cols, P)
    else:
        if P != G * rows_per_group:
            raise ValueError("mxfp8_requant_sr: weights need P == G * rows_per_group")
        shape = (G * cols, rows_per_group)
    if out is None:
        out = torch.empty(shape, dtype=torch.uint8, device=dev)
    if out_e8 is None:
        out_e8 = torch.empty((shape[0], shape[1] // 32), dtype=torch.uint8, device=dev)
    if out.numel() < shape[0] * shape[1] or out_e8.numel() < shape[0] * (shape[1] // 32):
        raise ValueError("mxfp8_requant_sr: output buffers too small")
    mode = _OUTER_PER_ROW if rows_per_group is None else _OUTER_PER_GROUP
    st = lib().mxfp8_requant_sr(_ptr(codes), _ptr(scales), _ptr(outer), mode,
                                0 if rows_per_group is None else int(rows_per_group), rows, cols,
                                _ptr(offsets), _ptr(padded_offsets), G, int(P),
                                int(seed) & 0xFFFFFFFFFFFFFFFF, int(tag) & 0xFFFFFFFF,
                                _ptr(out), _ptr(out_e8), _stream(codes))
    _check("mxfp8_requant_sr", st)
    return out, out_e8


def mxfp8_quantize(x, orientation="rowwise", offsets=None, padded_offsets=None, P=0,
                   out=None, out_e8=None):
    """dY [rows, cols] float32|bfloat16 -> MXFP8 with round-to-nearest-even.
    'rowwise': [rows, cols] + [rows, cols/32]; 'colwise': grouped transpose
    [cols, P] + [cols, P/32]."""
    torch = _torch()
    _dev(x, "x", ndim=2)
    rows, cols = x.shape
    dev = x.device
    if orientation == "rowwise":
        if out is None:
            out = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
        if out_e8 is None:
            out_e8 = torch.empty((rows, cols // 32), dtype=torch.uint8, device=dev)
        st = lib().mxfp8_quantize(_ptr(x), _in_dtype(x), rows, cols, _ROWWISE, None, None, 0, 0,
                                  _ptr(out), _ptr(out_e8), _stream(x))
    elif orientation == "colwise":
        _dev(offsets, "offsets", torch.int64, 1)
        _dev(padded_offsets, "padded_offsets", torch.int64, 1)
        G = offsets.shape[0] - 1
        if out is None:
            out = torch.empty((cols, P), dtype=torch.uint8, device=dev)
        if out_e8 is None:
            out_e8 = torch.empty((cols, P // 32), dtype=torch.uint8, device=dev)
        st = lib().mxfp8_quantize(_ptr(x), _in_dtype(x), rows, cols, _COLWISE_GROUPED,
                                  _ptr(offsets), _ptr(padded_offsets), G, int(P), _ptr(out),
                                  _ptr(out_e8), _stream(x))
    else:
        raise ValueError("orientation must be 'rowwise' or 'colwise'")
    _check("mxfp8_quantize", st)
    return out, out_e8


def moe_bwd_dgrad(dy_e4m3, dy_e8m0, w_e4m3, w_e8m0, offsets, N, K, out_dtype=None, dx=None):
    """dX [m_cap, K] from dY8 [m_cap, N] and W8 [G*K, N] (MXFP8, each expert's
    transposed weight [K, N] contiguous, as mxfp8_requant_sr writes it)."""
    torch = _torch()
    out_dtype = out_dtype or torch.float32
    for t, n in ((dy_e4m3, "dy_e4m3"), (dy_e8m0, "dy_e8m0"), (w_e4m3, "w_e4m3"),
                 (w_e8m0, "w_e8m0")):
        _dev(t, n, torch.uint8, 2)
    _dev(offsets, "offsets", torch.int64, 1)
    m_cap = dy_e4m3.shape[0]
    G = offsets.shape[0] - 1
    if dx is None:
        dx = torch.empty((m_cap, K), dtype=out_dtype, device=dy_e4m3.device)
    st = lib().moe_bwd_dgrad(_ptr(dy_e4m3), _ptr(dy_e8m0), _ptr(w_e4m3), _ptr(w_e8m0),
                             _ptr(offsets), G, m_cap, int(N), int(K), _ptr(dx),
                             _out_dtype(dx.dtype), _stream(dy_e4m3))
    _check("moe_bwd_dgrad", st)
    return dx


def moe_bwd_wgrad(dyT_e4m3, dyT_e8m0, xT_e4m3, xT_e8m0, padded_offsets, N, K, dw=None):
    """dW [G, N, K] float32 from dYT8 [N, P] and XT8 [K, P] (MXFP8)."""
    torch = _torch()
    for t, n in ((dyT_e4m3, "dyT_e4m3"), (dyT_e8m0, "dyT_e8m0"), (xT_e4m3, "xT_e4m3"),
                 (xT_e8m0, "xT_e8m0")):
        _dev(t, n, torch.uint8, 2)
    _dev(padded_offsets, "padded_offsets", torch.int64, 1)
    G = padded_offsets.shape[0] - 1
    P = dyT_e4m3.shape[1]
    if dw is None:
        dw = torch.empty((G, N, K), dtype=torch.float32, device=dyT_e4m3.device)
    st = lib().moe_bwd_wgrad(_ptr(dyT_e4m3), _ptr(dyT_e8m0), _ptr(xT_e4m3), _ptr(xT_e8m0),
                             _ptr(padded_offsets), G, P, int(N), int(K), _ptr(dw),
                             _stream(dyT_e4m3))
    _check("moe_bwd_wgrad", st)
    return dw


def moe_fwd_grouped_gemm_mxfp8(x_e4m3, x_e8m0, w_e4m3, w_e8m0, offsets, out_dtype=None, y=None):
    """y [m_cap, N] from X8 [m_cap, K] and weights W8 [G*N, K] or [G, N, K] (MXFP8)."""
    torch = _torch()
    out_dtype = out_dtype or torch.float32
    _dev(x_e4m3, "x_e4m3", torch.uint8, 2)
    _dev(x_e8m0, "x_e8m0", torch.uint8, 2)
    _dev(w_e4m3, "w_e4m3", torch.uint8)
    _dev(w_e8m0, "w_e8m0", torch.uint8)
    _dev(offsets, "offsets", torch.int64, 1)
    m_cap, K = x_e4m3.shape
    G = offsets.shape[0] - 1
    N = (w_e4m3.numel() // K) // G if G else 0
    if w_e4m3.numel() != G * N * K or w_e8m0.numel() != G * N * (K // 32):
        raise ValueError("weights must hold G*N rows of K elements (and K/32 scales)")
    if y is None:
        y = torch.empty((m_cap, N), dtype=out_dtype, device=x_e4m3.device)
    st = lib().moe_fwd_grouped_gemm_mxfp8(_ptr(x_e4m3), _ptr(x_e8m0), _ptr(w_e4m3), _ptr(w_e8m0),
                                          _ptr(offsets), G, m_cap, N, K, _ptr(y),
                                          _out_dtype(y.dtype), _stream(x_e4m3))
    _check("moe_fwd_grouped_gemm_mxfp8", st)
    return y


def mxfp8_gather_rows(row_token, offsets, src_e4m3, src_e8m0, m_cap=None, out=None):
    """Rows of MXFP8 src [T, K] (+ [T, K/32]) in expert order: row r < offsets[-1]
    is src row row_token[r]. Returns (dst_e4m3 [m_cap, K], dst_e8m0 [m_cap, K/32])."""
    torch = _torch()
    _dev(row_token, "row_token", torch.int32, 1)
    _dev(offsets, "offsets", torch.int64, 1)
    _dev(src_e4m3, "src_e4m3", torch.uint8, 2)
    _dev(src_e8m0, "src_e8m0", torch.uint8, 2)
    T, K = src_e4m3.shape
    m_cap = row_token.shape[0] if m_cap is None else int(m_cap)
    if out is None:
        out = (torch.empty((m_cap, K), dtype=torch.uint8, device=src_e4m3.device),
               torch.empty((m_cap, K // 32), dtype=torch.uint8, device=src_e4m3.device))
    G = offsets.shape[0] - 1
    st = lib().mxfp8_gather_rows(_ptr(row_token), _ptr(offsets), G, m_cap, _ptr(src_e4m3),
                                 _ptr(src_e8m0), T, K, _ptr(out[0]), _ptr(out[1]),
                                 _stream(src_e4m3))
    _check("mxfp8_gather_rows", st)
    return out


def mxfp8_quantize_dual(x, offsets, padded_offsets, P, row_out=None, col_out=None):
    """dY [rows, cols] -> (row-wise MXFP8 [rows, cols] + [rows, cols/32] for the
    grouped rows, grouped column-wise [cols, P] + [cols, P/32]) in one pass."""
    torch = _torch()
    _dev(x, "x", ndim=2)
    _dev(offsets, "offsets", torch.int64, 1)
    _dev(padded_offsets, "padded_offsets", torch.int64, 1)
    rows, cols = x.shape
    dev = x.device
    if row_out is None:
        row_out = (torch.empty((rows, cols), dtype=torch.uint8, device=dev),
                   torch.empty((rows, cols // 32), dtype=torch.uint8, device=dev))
    if col_out is None:
        col_out = (torch.empty((cols, P), dtype=torch.uint8, device=dev),
                   torch.empty((cols, P // 32), dtype=torch.uint8, device=dev))
    G = offsets.shape[0] - 1
    st = lib().mxfp8_quantize_dual(_ptr(x), _in_dtype(x), rows, cols, _ptr(offsets),
                                   _ptr(padded_offsets), G, int(P), _ptr(row_out[0]),
                                   _ptr(row_out[1]), _ptr(col_out[0]), _ptr(col_out[1]), _stream(x))
    _check("mxfp8_quantize_dual", st)
    return row_out[0], row_out[1], col_out[0], col_out[1]


def nvfp4_quantize_tile16(x, rows_per_group=None, codes=None, scales=None, outer=None):
    """16x16-tile NVFP4 of x [rows, cols] (bf16|f32): (codes [rows, cols/2],
    scales [rows/16, cols/16], outer [rows/rows_per_group])."""
    torch = _torch()
    _dev(x, "x", ndim=2)
    rows, cols = x.shape
    rpg = rows if rows_per_group is None else int(rows_per_group)
    dev = x.device
    if codes is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((rows // 16, cols // 16), dtype=torch.uint8, device=dev)
    if outer is None:
        outer = torch.empty((max(rows // max(rpg, 1), 1),), dtype=torch.float32, device=dev)
    st = lib().nvfp4_quantize_tile16(_ptr(x), _in_dtype(x), rows, cols, rpg, _ptr(codes),
                                     _ptr(scales), _ptr(outer), _stream(x))
    _check("nvfp4_quantize_tile16", st)
    return codes, scales, outer


def nvfp4_quantize_live(x, offsets, codes=None, scales=None, outer=None):
    """Per-row NVFP4 of the routed rows r < offsets[-1] of x [m_cap, cols]
    (bf16|f32): (codes [m_cap, cols/2], scales [m_cap, cols/16], outer
    [m_cap]); later rows untouched."""
    torch = _torch()
    _dev(x, "x", ndim=2)
    _dev(offsets, "offsets", torch.int64, 1)
    rows, cols = x.shape
    dev = x.device
    if codes is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=dev)
    if outer is None:
        outer = torch.empty((rows,), dtype=torch.float32, device=dev)
    st = lib().nvfp4_quantize_live(_ptr(x), _in_dtype(x), rows, cols, _ptr(offsets[-1:]),
                                   _ptr(codes), _ptr(scales), _ptr(outer), _stream(x))
    _check("nvfp4_quantize_live", st)
    return codes, scales, outer


def moe_combine(y, pair_row, gate=None, out_dtype=None, out=None):
    """out [T, N] = sum_j gate[t, j] * y[pair_row[t, j]] (gate None: ones).
    y [m_cap, N] bf16|f32; pair_row int32 [T, k]; gate f32 [T, k]."""
    torch = _torch()
    _dev(y, "y", ndim=2)
    _dev(pair_row, "pair_row", torch.int32, 2)
    if gate is not None:
        _dev(gate, "gate", torch.float32, 2)
        if tuple(gate.shape) != tuple(pair_row.shape):
            raise ValueError("gate and pair_row must have the same shape")
    T, k = pair_row.shape
    N = y.shape[1]
    if out is None:
        out = torch.empty((T, N), dtype=out_dtype or y.dtype, device=y.device)
    _dev(out, "out", ndim=2)
    st = lib().moe_combine(_ptr(y), _in_dtype(y), y.shape[0], T, k, N, _ptr(pair_row),
                           _ptr(gate), _ptr(out), _out_dtype(out.dtype), _stream(y))
    _check("moe_combine", st)
    return out


def moe_combine_bwd(dout, row_token, row_slot, offsets, k, gate=None, y=None, dy=None,
                    dgate=None, dy_dtype=None, m_cap=None):
    """Backward of moe_combine for the routed rows: (dy [m_cap, N], dgate
    [T, k] or None). dout [T, N]; y [m_cap, N] (the forward's expert outputs)
    or None; rows >= offsets[-1] of dy and non-local dgate entries untouched."""
    torch = _torch()
    _dev(dout, "dout", ndim=2)
    _dev(row_token, "row_token", torch.int32, 1)
    _dev(row_slot, "row_slot", torch.int32, 1)
    _dev(offsets, "offsets", torch.int64, 1)
    T, N = dout.shape
    if m_cap is None:
        m_cap = row_token.shape[0] if dy is None else dy.shape[0]
    if dy is None:
        dy = torch.empty((m_cap, N), dtype=dy_dtype or dout.dtype, device=dout.device)
    _dev(dy, "dy", ndim=2)
    if gate is not None:
        _dev(gate, "gate", torch.float32, 2)
    if y is not None:
        _dev(y, "y", ndim=2)
        if dgate is None:
            dgate = torch.zeros((T, k), dtype=torch.float32, device=dout.device)
    G = offsets.shape[0] - 1
    st = lib().moe_combine_bwd(_ptr(dout), _in_dtype(dout), T, int(k), N, _ptr(row_token),
                               _ptr(row_slot), _ptr(offsets), G, int(m_cap), _ptr(gate), _ptr(y),
                               _in_dtype(y) if y is not None else NVFP4MOE_F32, _ptr(dy),
                               _out_dtype(dy.dtype), _ptr(dgate), _stream(dout))
    _check("moe_combine_bwd", st)
    return dy, dgate


# ------------------------------------------------------------ NVFP4 backward

def moe_padded_offsets(offsets, align=128, out=None):
    """Exclusive scan of the group lengths rounded up to ``align`` (int64 [G+1])."""
    torch = _torch()
    _dev(offsets, "offsets", torch.int64, 1)
    G = offsets.shape[0] - 1
    if out is None:
        out = torch.empty_like(offsets)
    st = lib().moe_padded_offsets(_ptr(offsets), G, int(align), _ptr(out), _stream(offsets))
    _check("moe_padded_offsets", st)
    return out


def nvfp4_quantize_sr(x, seed, tag, codes=None, scales=None, outer=None):
    """Row-wise NVFP4 of x [rows, cols] with stochastic rounding and rounded-up
    block scales: (codes [rows, cols/2], scales [rows, cols/16], outer [rows])."""
    torch = _torch()
    _dev(x, "x", ndim=2)
    rows, cols = x.shape
    dev = x.device
    if codes is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=dev)
    if outer is None:
        outer = torch.empty((rows,), dtype=torch.float32, device=dev)
    st = lib().nvfp4_quantize_sr(_ptr(x), _in_dtype(x), rows, cols, int(seed), int(tag),
                                 _ptr(codes), _ptr(scales), _ptr(outer), _stream(x))
    _check("nvfp4_quantize_sr", st)
    return codes, scales, outer


def nvfp4_requant_sr(codes, scales, outer, offsets, padded_offsets, P, seed, tag,
                     rows_per_group=None, per_group_layout=False, out=None):
    """Saved NVFP4 [rows, cols] -> grouped transpose -> NVFP4 with stochastic
    rounding, one outer scale per group. Transposed layout: (codes [cols, P/2],
    scales [cols, P/16], outer [G]); per-group layout (groups of one length L,
    P = G * L): (codes [G * cols, L/2], scales [G * cols, L/16], outer [G])."""
    torch = _torch()
    _dev(codes, "codes", torch.uint8, 2)
    _dev(scales, "scales", torch.uint8, 2)
    _dev(outer, "outer", torch.float32, 1)
    _dev(offsets, "offsets", torch.int64, 1)
    _dev(padded_offsets, "padded_offsets", torch.int64, 1)
    rows, cols = codes.shape[0], codes.shape[1] * 2
    G = offsets.shape[0] - 1
    dev = codes.device
    if out is None:
        if per_group_layout:
            L = P // max(G, 1)
            out = (torch.empty((G * cols, L // 2), dtype=torch.uint8, device=dev),
                   torch.empty((G * cols, L // 16), dtype=torch.uint8, device=dev),
                   torch.empty((G,), dtype=torch.float32, device=dev))
        else:
            out = (torch.empty((cols, P // 2), dtype=torch.uint8, device=dev),
                   torch.empty((cols, P // 16), dtype=torch.uint8, device=dev),
                   torch.empty((G,), dtype=torch.float32, device=dev))
    mode = _OUTER_PER_ROW if rows_per_group is None else _OUTER_PER_GROUP
    st = lib().nvfp4_requant_sr(_ptr(codes), _ptr(scales), _ptr(outer), mode,
                                0 if rows_per_group is None else int(rows_per_group), rows, cols,
                                _ptr(offsets), _ptr(padded_offsets), G, int(P),
                                _LAYOUT_PER_GROUP if per_group_layout else _LAYOUT_TRANSPOSED,
                                int(seed), int(tag), _ptr(out[0]), _ptr(out[1]), _ptr(out[2]),
                                _stream(codes))
    _check("nvfp4_requant_sr", st)
    return out


def nvfp4_quantize_sr_colwise(x, offsets, padded_offsets, P, seed, tag, out=None):
    """dY [rows, cols] -> grouped transpose [cols, P] -> NVFP4 with stochastic
    rounding, one outer scale per group: (codes [cols, P/2], scales
    [cols, P/16], outer [G])."""
    torch = _torch()
    _dev(x, "x", ndim=2)
    _dev(offsets, "offsets", torch.int64, 1)
    _dev(padded_offsets, "padded_offsets", torch.int64, 1)
    rows, cols = x.shape
    G = offsets.shape[0] - 1
    dev = x.device
    if out is None:
        out = (torch.empty((cols, P // 2), dtype=torch.uint8, device=dev),
               torch.empty((cols, P // 16), dtype=torch.uint8, device=dev),
               torch.empty((G,), dtype=torch.float32, device=dev))
    st = lib().nvfp4_quantize_sr_colwise(_ptr(x), _in_dtype(x), rows, cols, _ptr(offsets),
                                         _ptr(padded_offsets), G, int(P), int(seed), int(tag),
                                         _ptr(out[0]), _ptr(out[1]), _ptr(out[2]), _stream(x))
    _check("nvfp4_quantize_sr_colwise", st)
    return out


def moe_bwd_wgrad_nvfp4(dyT, xT, padded_offsets, N, K, dw=None):
    """dW [G, N, K] float32 from NVFP4 dYT [N, P] and XT [K, P], each given as
    (codes, scales, outer [G])."""
    torch = _torch()
    for t, n in ((dyT[0], "dyT codes"), (dyT[1], "dyT scales"), (xT[0], "xT codes"),
                 (xT[1], "xT scales")):
        _dev(t, n, torch.uint8, 2)
    _dev(dyT[2], "dyT outer", torch.float32, 1)
    _dev(xT[2], "xT outer", torch.float32, 1)
    _dev(padded_offsets, "padded_offsets", torch.int64, 1)
    G = padded_offsets.shape[0] - 1
    P = dyT[0].shape[1] * 2
    if dw is None:
        dw = torch.empty((G, N, K), dtype=torch.float32, device=dyT[0].device)
    st = lib().moe_bwd_wgrad_nvfp4(_ptr(dyT[0]), _ptr(dyT[1]), _ptr(dyT[2]), _ptr(xT[0]),
                                   _ptr(xT[1]), _ptr(xT[2]), _ptr(padded_offsets), G, P, int(N),
                                   int(K), _ptr(dw), _stream(dyT[0]))
    _check("moe_bwd_wgrad_nvfp4", st)
    return dw


# ------------------------------------------ routing and gradient clipping

def _launch(dev, name, *args):
    """Call the library with ``dev`` as the current device, on its current
    stream (the last argument of every call), and check the status."""
    torch = _TORCH or _torch()
    f = getattr(_LIB or lib(), name)
    stream = torch._C._cuda_getCurrentRawStream(dev.index)
    if torch._C._cuda_getDevice() == dev.index:
        st = f(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = f(*args, stream)
    if st:
        _check(name, st)


def _on(t, name, dtype, shape, dev):
    """The address of a tensor that goes with another one: its type, shape
    and device."""
    if t.__class__ is not (_TORCH or _torch()).Tensor or t.dtype is not dtype or not t.is_contiguous():
        _dev(t, name, dtype)
    if t.shape != shape or t.device != dev:
        raise ValueError(f"{name} must have shape {tuple(shape)} on {dev} "
                         f"(got {tuple(t.shape)} on {t.device})")
    return t.data_ptr()


def _buf(out, name, dtype, shape, dev):
    """The address of an output buffer: the caller's in the dict ``out``,
    checked, or a new one put there."""
    t = out.get(name)
    if t is None:
        t = out[name] = _torch().empty(shape, dtype=dtype, device=dev)
        return t.data_ptr()
    return _on(t, name, dtype, shape, dev)


def _workspace(t, need, dev):
    """(workspace, bytes): the caller's, or a new one (live until the call returns:
    torch hands its memory to later work of the same stream only)."""
    torch = _torch()
    if t is None:
        return (torch.empty((need,), dtype=torch.uint8, device=dev) if need else None), need
    _dev(t, "workspace", torch.uint8)
    if t.device != dev:
        raise ValueError(f"workspace must be on {dev} (got {t.device})")
    return t, t.numel()


def _score(score):
    if score not in _SCORES:
        raise ValueError(f"score must be 'softmax' or 'sigmoid' (got {score!r})")
    return _SCORES[score]


def _number(v, name, kind=float):
    """A host number of any type. A GPU tensor is refused: to read it the call
    would have to wait for the device (and could not be captured)."""
    if v.__class__ is kind:
        return v
    if isinstance(v, _torch().Tensor) and v.is_cuda:
        raise ValueError(f"{name} must be a host number (got a tensor on {v.device})")
    return kind(v)


def _route_sizes(fn, T, E, k):
    """The library's bounds, before an output of these sizes is made (and in
    whole numbers: 2^32 + 2 slots are not the two that a C int would hold)."""
    if E < 1 or k < 1:
        _check(fn, _EINVAL)
    if E > 1024 or k > 64 or k > E or T * k > 0x7FFFFFFF:
        _check(fn, _EUNSUPPORTED)


@functools.lru_cache(maxsize=256)
def route_workspace_size(T, E):
    return int(lib().nvfp4moe_route_workspace_size(int(T), int(E)))


def moe_route(logits, k, score="softmax", renorm=True, scale=1.0, bias=None, token_mask=None,
              stats=False, workspace=None, out=None):
    """Select k experts per token of logits [T, E] (bf16|f32; -inf closes an
    expert). Returns a dict with topk_ids int32 [T, k] (-1: no expert left),
    gate f32 [T, k], and with ``stats`` counts int64 [E+1] (pairs on each
    expert, then the tokens that have one) and prob_sum f32 [E].

    score 'softmax' or 'sigmoid'; renorm: gates divided by their sum; bias f32
    [E] ('sigmoid' only) shifts the choice, not the gates; token_mask bool or
    uint8 [T], False for padding; ``out`` may hold any of the results' buffers
    (others in it are left alone and not returned)."""
    torch = _torch()
    _dev(logits, "logits", ndim=2)
    T, E = logits.shape
    k = _number(k, "k", int)
    _route_sizes("moe_route", T, E, k)
    dev = logits.device
    names = ("topk_ids", "gate", "counts", "prob_sum") if stats else ("topk_ids", "gate")
    o = {} if out is None else {n: out[n] for n in names if n in out}
    ids = _buf(o, "topk_ids", torch.int32, (T, k), dev)
    gate = _buf(o, "gate", torch.float32, (T, k), dev)
    counts = prob_sum = ws = None
    ws_bytes = 0
    if stats:
        counts = _buf(o, "counts", torch.int64, (E + 1,), dev)
        prob_sum = _buf(o, "prob_sum", torch.float32, (E,), dev)
        ws, ws_bytes = _workspace(workspace, route_workspace_size(T, E), dev)
    if bias is not None:
        bias = _on(bias, "bias", torch.float32, (E,), dev)
    if token_mask is not None:
        if isinstance(token_mask, torch.Tensor) and token_mask.dtype == torch.bool:
            token_mask = token_mask.view(torch.uint8)
        token_mask = _on(token_mask, "token_mask", torch.uint8, (T,), dev)
    _launch(dev, "moe_route", logits.data_ptr(), _in_dtype(logits), T, E, k, _score(score),
            1 if renorm else 0, _number(scale, "scale"), bias, token_mask, ids, gate, counts, prob_sum,
            None if ws is None else ws.data_ptr(), ws_bytes)
    return o


def moe_balance_loss(counts, prob_sum, k, alpha, loss=None):
    """Balance loss f32 [1] of moe_route's statistics: alpha * E * sum_e
    counts[e] / (N k) * prob_sum[e] / N with N = counts[E]."""
    torch = _torch()
    _dev(prob_sum, "prob_sum", torch.float32, 1)
    dev, E = prob_sum.device, prob_sum.shape[0]
    k = _number(k, "k", int)
    _route_sizes("moe_balance_loss", 0, E, k)
    o = {"loss": loss}
    _launch(dev, "moe_balance_loss", _on(counts, "counts", torch.int64, (E + 1,), dev),
            prob_sum.data_ptr(), E, k, _number(alpha, "alpha"), _buf(o, "loss", torch.float32, (1,), dev))
    return o["loss"]


def moe_route_bwd(logits, topk_ids, dgate=None, score="softmax", renorm=True, scale=1.0,
                  counts=None, alpha=0.0, dloss=None, dlogits=None):
    """dlogits [T, E] (of the logits' type) from the gates' gradient dgate f32
    [T, k] (None: zero) and, when counts int64 [E+1] is given, the balance
    loss's: alpha as in moe_balance_loss, dloss f32 [1] on the device (None: 1)."""
    torch = _torch()
    _dev(logits, "logits", ndim=2)
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    T, E = logits.shape
    k = topk_ids.shape[1]
    _route_sizes("moe_route_bwd", T, E, k)
    dev = logits.device
    o = {"dlogits": dlogits}
    if dgate is not None:
        dgate = _on(dgate, "dgate", torch.float32, (T, k), dev)
    if counts is not None:
        counts = _on(counts, "counts", torch.int64, (E + 1,), dev)
    if dloss is not None:
        dloss = _on(dloss, "dloss", torch.float32, (1,), dev)
    _launch(dev, "moe_route_bwd", logits.data_ptr(), _in_dtype(logits), T, E, k, _score(score),
            1 if renorm else 0, _number(scale, "scale"), _on(topk_ids, "topk_ids", torch.int32, (T, k), dev),
            dgate, counts, _number(alpha, "alpha"), dloss, _buf(o, "dlogits", logits.dtype, (T, E), dev))
    return o["dlogits"]


@functools.lru_cache(maxsize=None)
def _tensors_lib():
    """libnvfp4moe_tensors.so, whose calls keep the interpreter's lock."""
    _torch()                                    # the libraries it is linked to
    if not os.path.exists(TENSORS_LIB_PATH):
        raise RuntimeError(
            f"{TENSORS_LIB_PATH} is missing: build it with "
            "`python -m precision_moe_numerics_nvfp4_amd.build` (or __graft_entry__.build())")
    L = ctypes.PyDLL(TENSORS_LIB_PATH)
    for f in (L.nvfp4moe_tensors_look, L.nvfp4moe_tensors_same):
        f.argtypes, f.restype = [ctypes.py_object, _p, _c_i64], _c_int
    return L


class GradList:
    """The gradients (or their clipped copies) of one device as the calls
    below take them: contiguous bf16|f32 tensors of any alignment that do not
    overlap. Made once of buffers that live on, it keeps the tensors and their
    memory; every call looks whether a tensor has other memory, another size,
    type or order since (``t.data = ...``, ``resize_``), and checks and takes
    the whole list anew where one has."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        self._look()

    def _look(self):
        torch = _torch()
        ts = self.tensors = list(self.tensors)
        n = len(ts)
        # before all else: what changes from here on is seen by the next call
        seen = (_c_i64 * (3 * n))()
        known = _tensors_lib().nvfp4moe_tensors_look(ts, seen, n)
        dev = None
        for i, t in enumerate(ts):
            if not (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous()):
                _dev(t, f"tensor {i}")
            if dev is None:
                dev = t.device
            elif t.device != dev:
                raise ValueError(f"tensor {i} is on {t.device}, the first on {dev}")
        # the storages stay alive: an address seen again is the same memory
        storages = [t.untyped_storage() for t in ts]
        starts, sizes = [t.data_ptr() for t in ts], [t.numel() for t in ts]
        codes = [_in_dtype(t) for t in ts]
        spans = sorted((p, p + m * (2 if c == NVFP4MOE_BF16 else 4))
                       for p, m, c in zip(starts, sizes, codes) if m)
        for (_, end), (start, _) in zip(spans, spans[1:]):
            if start < end:
                raise ValueError("tensors overlap (or one is listed twice)")
        if not known:
            raise ValueError("tensors without memory of their own")
        self.seen, self.device, self.spans, self.storages = seen, dev, spans, storages
        self.starts, self.sizes, self.types = starts, sizes, codes
        self.ptrs, self.numels, self.codes = (_p * n)(*starts), (_c_i64 * n)(*sizes), (_c_int * n)(*codes)
        self.workspace_size = int(lib().nvfp4moe_grad_workspace_size(self.numels, n))

    def __len__(self):
        return len(self.tensors)

    def current(self):
        if not _tensors_lib().nvfp4moe_tensors_same(self.tensors, self.seen, len(self.starts)):
            self._look()
        return self


def _grad_list(grads):
    return grads.current() if isinstance(grads, GradList) else GradList(grads)


def _overlap(a, b):
    """Whether any span of one list meets any of the other (each sorted, disjoint)."""
    if not a or not b or a[-1][1] <= b[0][0] or b[-1][1] <= a[0][0]:
        return False
    i = j = 0
    while i < len(a) and j < len(b):
        if a[i][0] < b[j][1] and b[j][0] < a[i][1]:
            return True
        if a[i][1] <= b[j][1]:
            i += 1
        else:
            j += 1
    return False


def grad_workspace_size(grads):
    """Bytes of workspace moe_grad_sumsq needs for a list (a GradList or tensors)."""
    return _grad_list(grads).workspace_size


def moe_grad_sumsq(grads, sumsq=None, workspace=None):
    """Sum of squares f64 [1] over a list of gradients (a GradList or tensors)."""
    torch = _torch()
    g = _grad_list(grads)
    dev = g.device
    if dev is None:
        if sumsq is None:
            raise ValueError("an empty list needs sumsq (which device?)")
        dev = sumsq.device
    o = {"sumsq": sumsq}
    ws, ws_bytes = _workspace(workspace, g.workspace_size, dev)
    _launch(dev, "moe_grad_sumsq", g.ptrs, g.codes, g.numels, len(g),
            _buf(o, "sumsq", torch.float64, (1,), dev), None if ws is None else ws.data_ptr(),
            ws_bytes)
    return o["sumsq"]


def moe_grad_clip(grads, sumsq, max_norm, outs=None, norm=None):
    """Scale a list of gradients by min(1, max_norm / (norm + 1e-6)), norm =
    sqrt(sumsq) of moe_grad_sumsq (or a sum of several ranks' values): in
    place, or into ``outs`` (same types and sizes, apart from the gradients).
    max_norm infinity leaves them as they are. Returns norm f32 [1], the norm
    before clipping."""
    torch = _torch()
    _dev(sumsq, "sumsq", torch.float64)
    g = _grad_list(grads)
    dev = sumsq.device
    o = g
    if outs is not None and outs is not grads:
        o = _grad_list(outs)
        if o.types != g.types or o.sizes != g.sizes:
            raise ValueError("outs must have the gradients' types and sizes")
        if o.starts != g.starts and _overlap(g.spans, o.spans):
            raise ValueError("outs must be the gradients themselves or apart from them")
    if not (g.device in (None, dev) and o.device in (None, dev)):
        raise ValueError(f"sumsq is on {dev}, the gradients or outs elsewhere")
    res = {"norm": norm}
    _launch(dev, "moe_grad_clip", g.ptrs, o.ptrs, g.codes, g.numels, len(g),
            _on(sumsq, "sumsq", torch.float64, (1,), dev), _number(max_norm, "max_norm"),
            _buf(res, "norm", torch.float32, (1,), dev))
    return res["norm"]


# ------------------------------------------ MXFP4, and the layer for a few tokens

def _c_size_of(v, name, bits=64):
    """A whole number that the C argument holds."""
    v = _number(v, name, int)
    if not -(1 << (bits - 1)) <= v < 1 << (bits - 1):
        raise ValueError(f"{name} is out of range (got {v})")
    return v


def _mxfp4_pair(codes, scales, name, dev):
    """Addresses, rows and columns of an MXFP4 tensor (any leading dimensions)."""
    u8 = (_TORCH or _torch()).uint8
    _dev(codes, name, u8)
    shape = codes.shape
    if len(shape) < 2:
        raise ValueError(f"{name} codes must have at least 2 dimensions (got {len(shape)})")
    half = shape[-1]
    rows = codes.numel() // half if half else 0
    if half % 16:
        raise ValueError(f"{name} codes must hold whole blocks of 32 (got {2 * half} columns)")
    if codes.device != dev:
        raise ValueError(f"{name} codes must be on {dev} (got {codes.device})")
    _dev(scales, name, u8)
    if scales.device != dev or scales.numel() != rows * (half // 16) or scales.shape[-1] != half // 16:
        raise ValueError(f"{name} scales must hold {half // 16} bytes for each of {rows} rows on {dev} "
                         f"(got {tuple(scales.shape)} on {scales.device})")
    return codes.data_ptr(), scales.data_ptr(), rows, 2 * half


def mxfp4_quantize(x, offsets=None, codes=None, scales=None):
    """x [rows, cols] float32|bfloat16 -> MXFP4 (codes [rows, cols/2] u8, scales
    [rows, cols/32] u8). With ``offsets`` (moe_group's) only the routed rows
    r < offsets[-1]; later rows of the outputs untouched."""
    torch = _TORCH or _torch()
    _dev(x, "x", ndim=2)
    rows, cols = x.shape
    dev, live = x.device, None
    if cols % 32:
        _check("mxfp4_quantize", _EUNSUPPORTED)
    if offsets is not None:
        _dev(offsets, "offsets", torch.int64, 1)
        if offsets.device != dev or offsets.numel() < 1:
            raise ValueError(f"offsets must hold a row count on {dev}")
        live = offsets.data_ptr() + 8 * (offsets.numel() - 1)
    o = dict(codes=codes, scales=scales)
    _launch(dev, "mxfp4_quantize", x.data_ptr(), _in_dtype(x), rows, cols, live,
            _buf(o, "codes", torch.uint8, (rows, cols // 2), dev),
            _buf(o, "scales", torch.uint8, (rows, cols // 32), dev))
    return o["codes"], o["scales"]


def _dequantize(fn, q, scales, rows, cols, dev, out_dtype, out):
    torch = _TORCH or _torch()
    o = {"out": out}
    dtype = out.dtype if out is not None else (out_dtype or torch.float32)
    code = _out_dtype(dtype)
    _launch(dev, fn, q, scales, rows, cols, _buf(o, "out", dtype, (rows, cols), dev), code)
    return o["out"]


def mxfp4_dequantize(codes, scales, out_dtype=None, out=None):
    """Values [rows, cols] (float32|bfloat16) of MXFP4 codes [rows, cols/2]."""
    _dev(codes, "codes", ndim=2)
    q, e, rows, cols = _mxfp4_pair(codes, scales, "mxfp4", codes.device)
    return _dequantize("mxfp4_dequantize", q, e, rows, cols, codes.device, out_dtype, out)


def mxfp8_dequantize(e4m3, e8m0, out_dtype=None, out=None):
    """Values [rows, cols] (float32|bfloat16) of MXFP8 elements [rows, cols]."""
    torch = _TORCH or _torch()
    _dev(e4m3, "e4m3", torch.uint8, 2)
    rows, cols = e4m3.shape
    if cols % 32:
        _check("mxfp8_dequantize", _EUNSUPPORTED)
    e = _on(e8m0, "e8m0", torch.uint8, (rows, cols // 32), e4m3.device)
    return _dequantize("mxfp8_dequantize", e4m3.data_ptr(), e, rows, cols, e4m3.device, out_dtype, out)


def moe_group(topk_ids, e0, n_local, workspace=None, out=None):
    """moe_permute's grouping without moving rows: a dict with offsets,
    padded_offsets (int64 [n_local+1]), row_token, row_slot (int32 [T*k]; rows
    >= offsets[-1] untouched) and pair_row (int32 [T, k]; an ``out`` dict
    without it asks for none)."""
    torch = _TORCH or _torch()
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    T, k = topk_ids.shape
    e0, n_local = _c_size_of(e0, "e0", 32), _c_size_of(n_local, "n_local", 32)
    if n_local < 1:
        _check("moe_group", _EINVAL)
    if n_local > 1024 or k > 64 or T * k > 0x7FFFFFFF:
        _check("moe_group", _EUNSUPPORTED)
    dev, i32, i64 = topk_ids.device, torch.int32, torch.int64
    o = dict(out or {})
    if out is None:
        o["pair_row"] = torch.empty((T, k), dtype=i32, device=dev)
    pair = o.get("pair_row")
    ws, ws_bytes = _workspace(workspace, permute_workspace_size(T, k, n_local), dev)
    _launch(dev, "moe_group", topk_ids.data_ptr(), T, k, e0, n_local,
            _buf(o, "offsets", i64, (n_local + 1,), dev), _buf(o, "padded_offsets", i64, (n_local + 1,), dev),
            _buf(o, "row_token", i32, (T * k,), dev), _buf(o, "row_slot", i32, (T * k,), dev),
            None if pair is None else _on(pair, "pair_row", i32, (T, k), dev), ws.data_ptr(), ws_bytes)
    return o


def _row_map(row_token, dev):
    """Address and length of a map from grouped rows to source rows."""
    _dev(row_token, "row_token", _torch().int32, 1)
    if row_token.device != dev:
        raise ValueError(f"row_token must be on {dev} (got {row_token.device})")
    return row_token.data_ptr(), row_token.shape[0]


def moe_fwd_grouped_gemm_mxfp4(a_codes, a_scales, b_codes, b_scales, offsets, row_token=None,
                               out_dtype=None, y=None):
    """y [m_cap, N] = grouped MXFP4 GEMM of activations [rows, K] with weights
    [G*N, K] or [G, N, K]; offsets int64 [G+1] on the device. With ``row_token``
    (int32 [m_cap], moe_group's) row r reads activation row row_token[r], else
    row r. Rows >= offsets[-1] of y are untouched."""
    torch = _TORCH or _torch()
    _dev(a_codes, "a codes", ndim=2)
    dev = a_codes.device
    ac, as_, rows, K = _mxfp4_pair(a_codes, a_scales, "a", dev)
    bc, bs, b_rows, b_cols = _mxfp4_pair(b_codes, b_scales, "b", dev)
    _dev(offsets, "offsets", torch.int64, 1)
    G = offsets.shape[0] - 1
    if offsets.device != dev or G < 0:
        raise ValueError(f"offsets must hold G + 1 row counts on {dev}")
    if b_cols != K or (b_rows % G if G else b_rows):
        raise ValueError(f"b must hold G = {G} weights of {K} columns (got {b_rows} rows of {b_cols})")
    N = b_rows // G if G else 0
    tok, m_cap = (None, rows) if row_token is None else _row_map(row_token, dev)
    o = {"y": y}
    dtype = y.dtype if y is not None else (out_dtype or torch.float32)
    code = _out_dtype(dtype)
    _launch(dev, "moe_fwd_grouped_gemm_mxfp4", ac, as_, rows, tok, bc, bs, offsets.data_ptr(), G, m_cap,
            N, K, _buf(o, "y", dtype, (m_cap, N), dev), code)
    return o["y"]


def mxfp8_requant_sr_mxfp4(codes, scales, offsets, padded_offsets, P, seed, tag, rows_per_group=None,
                           row_token=None, out=None, out_e8=None):
    """Saved MXFP4 [rows, cols] -> MXFP8 with stochastic rounding, grouped
    transpose, as mxfp8_requant_sr: activations [cols, P] (+ E8M0 [cols, P/32]),
    read through ``row_token`` where it is given; weights (rows_per_group)
    per-expert blocks [G * cols, rows_per_group], P = G * rows_per_group."""
    torch = _TORCH or _torch()
    _dev(codes, "codes", ndim=2)
    dev = codes.device
    q, e, rows, cols = _mxfp4_pair(codes, scales, "mxfp4", dev)
    _dev(offsets, "offsets", torch.int64, 1)
    G = offsets.shape[0] - 1
    if offsets.device != dev or G < 0:
        raise ValueError(f"offsets must hold G + 1 row counts on {dev}")
    P = _c_size_of(P, "P")
    if P < 0 or P % 32:
        _check("mxfp8_requant_sr_mxfp4", _EINVAL if P < 0 else _EUNSUPPORTED)
    tok, n = (None, rows) if row_token is None else _row_map(row_token, dev)
    if rows_per_group is None:
        rpg, shape = 0, (cols, P)
    else:
        rpg = _c_size_of(rows_per_group, "rows_per_group")
        if rpg < 1 or P != G * rpg or rows != P:
            raise ValueError("mxfp8_requant_sr_mxfp4: weights need P == rows == G * rows_per_group")
        if tok is not None:
            raise ValueError("mxfp8_requant_sr_mxfp4: row_token goes with activations only")
        if rpg % 32:
            _check("mxfp8_requant_sr_mxfp4", _EUNSUPPORTED)
        shape = (G * cols, rpg)
    o = dict(out=out, out_e8=out_e8)
    _launch(dev, "mxfp8_requant_sr_mxfp4", q, e, rows, cols, tok, rpg, offsets.data_ptr(),
            _on(padded_offsets, "padded_offsets", torch.int64, (G + 1,), dev), G, P,
            int(seed) & 0xFFFFFFFFFFFFFFFF, int(tag) & 0xFFFFFFFF,
            _buf(o, "out", torch.uint8, shape, dev),
            _buf(o, "out_e8", torch.uint8, (shape[0], shape[1] // 32), dev))
    return o["out"], o["out_e8"]


@functools.lru_cache(maxsize=256)
def ffn_tokens_workspace_size(T, k, K, F):
    return int(lib().nvfp4moe_ffn_tokens_workspace_size(int(T), int(k), int(K), int(F)))


def _weight(w, name, dev):
    """Parts of a 4-bit weight: MXFP4 (codes, scales) or NVFP4 (codes, scales,
    outer [n_local]), its addresses, rows and columns."""
    torch = _TORCH or _torch()
    if not isinstance(w, (tuple, list)) or len(w) not in _FORMATS:
        raise ValueError(f"{name} must be (codes, scales) in MXFP4 or (codes, scales, outer) in NVFP4")
    codes, scales = w[0], w[1]
    _dev(codes, name, torch.uint8)
    shape = codes.shape
    cols = 2 * shape[-1] if len(shape) >= 2 else 0
    if cols == 0 or codes.device != dev:
        raise ValueError(f"{name} codes must have rows of codes on {dev} "
                         f"(got {tuple(shape)} on {codes.device})")
    rows, block = codes.numel() // (cols // 2), 32 if len(w) == 2 else 16
    _dev(scales, name, torch.uint8)
    if cols % 32 or scales.numel() != rows * (cols // block) or scales.shape[-1] != cols // block or \
            scales.device != dev:
        raise ValueError(f"{name} scales must hold a byte for {block} codes of each of {rows} rows on {dev} "
                         f"(got {tuple(scales.shape)} on {scales.device})")
    outer = None
    if len(w) == 3:
        outer = w[2]
        _dev(outer, name, torch.float32, 1)
        if outer.device != dev:
            raise ValueError(f"{name} outer must be on {dev} (got {outer.device})")
        outer = outer.data_ptr()
    return codes.data_ptr(), scales.data_ptr(), outer, rows, cols


def moe_ffn_tokens(x, logits, k, w1, w2, act="silu", gated=False, score="softmax", renorm=True,
                   scale=1.0, bias=None, token_mask=None, e0=0, out_dtype=None, workspace=None,
                   out=None):
    """The whole expert layer for up to 64 tokens: x bf16 [T, K] and logits
    [T, E] (bf16|f32) -> a dict with out [T, K] (bf16, or ``out_dtype``
    float32), topk_ids int32 [T, k] and gate f32 [T, k] (moe_route's; its
    options too).

    w1 [n_local*F, K] (gated: [n_local*2F, K], an expert's first F rows go
    through ``act``, its last F multiply them) and w2 [n_local*K, F], each
    (codes, scales) in MXFP4 or (codes, scales, outer) in NVFP4, of the experts
    [e0, e0+n_local). act 'none', 'relu2' or 'silu'. ``out`` may hold any of the
    results' buffers; ``workspace`` ffn_tokens_workspace_size(T, k, K, F) bytes,
    of one call at a time."""
    torch = _TORCH or _torch()
    _dev(x, "x", torch.bfloat16, 2)
    T, K = x.shape
    dev = x.device
    _dev(logits, "logits", ndim=2)
    if logits.shape[0] != T or logits.device != dev:
        raise ValueError(f"logits must have {T} rows on {dev} (got {tuple(logits.shape)} on {logits.device})")
    E = logits.shape[1]
    k, e0 = _number(k, "k", int), _c_size_of(e0, "e0", 32)
    if act not in _ACTS:
        raise ValueError(f"act must be 'none', 'relu2' or 'silu' (got {act!r})")
    c1, s1, o1, rows1, cols1 = _weight(w1, "w1", dev)
    c2, s2, o2, rows2, F = _weight(w2, "w2", dev)
    if len(w1) != len(w2):
        raise ValueError("w1 and w2 must have the same format")
    n_local = rows2 // K if K else 0
    if cols1 != K or n_local * K != rows2 or rows1 != n_local * F * (2 if gated else 1):
        raise ValueError(f"w1 must be [n*{'2F' if gated else 'F'}, {K}] and w2 [n*{K}, F] "
                         f"(got [{rows1}, {cols1}] and [{rows2}, {F}])")
    if o1 is not None and (w1[2].shape[0] != n_local or w2[2].shape[0] != n_local):
        raise ValueError(f"outer scales must have shape ({n_local},)")
    if E < 1 or k < 1 or n_local < 1:
        _check("moe_ffn_tokens", _EINVAL)
    if T > 64 or k > 16 or T * k > 512 or k > E or E > 1024 or n_local > 1024:
        _check("moe_ffn_tokens", _EUNSUPPORTED)
    o = {} if out is None else {n: out[n] for n in ("out", "topk_ids", "gate") if n in out}
    dtype = o["out"].dtype if o.get("out") is not None else (out_dtype or torch.bfloat16)
    code = _out_dtype(dtype)
    y = _buf(o, "out", dtype, (T, K), dev)
    ids = _buf(o, "topk_ids", torch.int32, (T, k), dev)
    gate = _buf(o, "gate", torch.float32, (T, k), dev)
    if bias is not None:
        bias = _on(bias, "bias", torch.float32, (E,), dev)
    if token_mask is not None:
        if isinstance(token_mask, torch.Tensor) and token_mask.dtype == torch.bool:
            token_mask = token_mask.view(torch.uint8)
        token_mask = _on(token_mask, "token_mask", torch.uint8, (T,), dev)
    ws, ws_bytes = _workspace(workspace, ffn_tokens_workspace_size(T, k, K, F), dev)
    _launch(dev, "moe_ffn_tokens", x.data_ptr(), logits.data_ptr(), _in_dtype(logits), T, E, k,
            _score(score), 1 if renorm else 0, _number(scale, "scale"), bias, token_mask,
            _FORMATS[len(w1)], c1, s1, o1, c2, s2, o2, e0, n_local, K, F, _ACTS[act],
            1 if gated else 0, ids, gate, y, code, None if ws is None else ws.data_ptr(), ws_bytes)
    return o
