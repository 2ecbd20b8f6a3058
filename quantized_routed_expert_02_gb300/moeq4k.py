"""Python binding of the moeq4k C ABI (``libmoeq4k.so``).

Argument marshalling only: tensors become raw device pointers, the stream
defaults to PyTorch's current stream, and a non-OK status raises
``MoeError``.  Every step of the layer runs in the library's CUDA kernels;
there is no Python or CPU fallback.  Importing this module without the
built library raises immediately.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoeq4k.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m quantized_routed_expert_02_gb300.build` "
        "(or __graft_entry__.build()); the moeq4k layer has no fallback path")

_lib = ctypes.CDLL(LIB_PATH)

_P = ctypes.c_void_p
_I = ctypes.c_int
_S = ctypes.c_size_t

_SIGS = {
    "moe_status_str": ([ctypes.c_int], ctypes.c_char_p),
    "moe_version": ([], ctypes.c_int),
    "moe_workspace_bytes": ([_I, _I, _I, _I, _I], _S),
    "moe_workspace_bytes_host": ([_I, _I, _I, _I, _I], _S),
    "moe_layer_launch_count": ([_I, _I, _I, _I, _I], ctypes.c_int),
    "moe_workspace_init": ([_P, _S, _P], ctypes.c_int),
    "moe_router": ([_P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _S, _P], ctypes.c_int),
    "moe_permute": ([_P, _I, _I, _I, _P, _P, _P, _P, _S, _P], ctypes.c_int),
    "moe_ffn": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _S, _P], ctypes.c_int),
    "moe_layer": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _S, _P],
                  ctypes.c_int),
    "moe_layer_host": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _S, _P],
                       ctypes.c_int),
    "moe_layer_block": ([_P, _P, ctypes.c_float, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P,
                         _P, _I, _I, _P, _P, _P, _P, _S, _P], ctypes.c_int),
    "moe_quantize_q8k": ([_P, _I, _I, _P, _P, _P, _P], ctypes.c_int),
    "moe_ffn_q8k": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _S, _P], ctypes.c_int),
    "moe_layer_q8k": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _S, _P],
                      ctypes.c_int),
    "moe_layer_q8k_launch_count": ([_I, _I, _I, _I, _I], ctypes.c_int),
    "moe_ffn_q8k_codes": ([_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _S, _P],
                          ctypes.c_int),
    "moe_add_rmsnorm": ([_P, _I, _P, _P, ctypes.c_float, _I, _I, _P, _P, _I, _P, _P, _P, _P],
                        ctypes.c_int),
    "moe_rope_append": ([_P, _P, _P, _P, _I, _I, _I, _P, _P, ctypes.c_float, _P, _P, _P, _P, _P, _P,
                         _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _S, _P], ctypes.c_int),
    "moe_attention_workspace_bytes": ([_I, _I, _I], _S),
    "moe_attention_paged": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I,
                             ctypes.c_float, ctypes.c_float, _I, _P, _P, _P, _S, _P], ctypes.c_int),
    "moe_read_device_status": ([_P, _P, ctypes.POINTER(ctypes.c_int32)], ctypes.c_int),
    "moe_layer_noalloc": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P],
                          ctypes.c_int),
    "moe_debug_set_wait_limit": ([ctypes.c_ulonglong], None),
    "moe_debug_withhold_arrivals": ([_I], None),
}
for _name, (_args, _res) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _res

EXPORTS = tuple(_SIGS)

MOE_OK = 0
STATUS_NAMES = {i: _lib.moe_status_str(i).decode() for i in range(11)}


_F32, _F64, _I32, _I8 = torch.float32, torch.float64, torch.int32, torch.int8
MOE_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS_NAMES.get(code, code)}")


def _check(code: int, where: str) -> None:
    if code != MOE_OK:
        raise MoeError(code, where)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# The current stream's handle without building a Stream object (2.9 -> 0.3 us a call), where
# PyTorch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def status_str(code: int) -> str:
    return _lib.moe_status_str(int(code)).decode()


def version() -> int:
    return _lib.moe_version()


def moe_workspace_bytes(T, H, E, k, I) -> int:
    return _lib.moe_workspace_bytes(T, H, E, k, I)


def moe_workspace_bytes_host(T, H, E, k, I) -> int:
    return _lib.moe_workspace_bytes_host(T, H, E, k, I)


def moe_layer_launch_count(T, H, E, k, I) -> int:
    return _lib.moe_layer_launch_count(T, H, E, k, I)


def moe_layer_q8k_launch_count(T, H, E, k, I) -> int:
    return _lib.moe_layer_q8k_launch_count(T, H, E, k, I)


def alloc_workspace(T, H, E, k, I, device="cuda", host_staging=False) -> torch.Tensor:
    """A uint8 device workspace of the right size, initialised with
    moe_workspace_init (header and tag region zeroed)."""
    n = (moe_workspace_bytes_host if host_staging else moe_workspace_bytes)(T, H, E, k, I)
    if n == 0:
        raise MoeError(1, "moe_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    moe_workspace_init(ws)
    return ws


def moe_workspace_init(ws, stream=None) -> None:
    _check(_lib.moe_workspace_init(_ptr(ws), ws.numel(), _stream(stream)), "moe_workspace_init")


def moe_router(x, Wr, bias, k, idx, w, ws, stream=None) -> None:
    T, H = x.shape
    E = Wr.shape[0]
    _check(_lib.moe_router(_ptr(x), _ptr(Wr), _ptr(bias), T, H, E, k, _ptr(idx), _ptr(w),
                           _ptr(ws), ws.numel(), _stream(stream)), "moe_router")


def moe_permute(idx, E, counts, offs, perm, ws, stream=None) -> None:
    T, k = idx.shape
    _check(_lib.moe_permute(_ptr(idx), T, k, E, _ptr(counts), _ptr(offs), _ptr(perm),
                            _ptr(ws), ws.numel(), _stream(stream)), "moe_permute")


def moe_ffn(x, idx, w, gate, up, down, E, I, y, ws, stream=None) -> None:
    T, H = x.shape
    k = idx.shape[1]
    _check(_lib.moe_ffn(_ptr(x), _ptr(idx), _ptr(w), _ptr(gate), _ptr(up), _ptr(down),
                        T, H, E, k, I, _ptr(y), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_ffn")


def moe_layer(x, Wr, bias, gate, up, down, k, I, idx, w, y, ws, stream=None) -> None:
    T, H = x.shape
    E = Wr.shape[0]
    _check(_lib.moe_layer(_ptr(x), _ptr(Wr), _ptr(bias), _ptr(gate), _ptr(up), _ptr(down),
                          T, H, E, k, I, _ptr(idx), _ptr(w), _ptr(y), _ptr(ws), ws.numel(),
                          _stream(stream)), "moe_layer")


def moe_layer_block(hidden, norm_w, eps, Wr, bias, gate, up, down, k, I, idx, w, out, ws,
                    add_residual=True, capture_token=-1, cap_idx=None, cap_w=None, cap_ffn=None,
                    stream=None) -> None:
    """RMSNorm (``norm_w`` None: none) -> router -> expert FFN -> residual
    add; optional capture of one token's routing and pre-residual output."""
    T, H = hidden.shape
    E = Wr.shape[0]
    _check(_lib.moe_layer_block(_ptr(hidden), _ptr(norm_w), float(eps), _ptr(Wr), _ptr(bias),
                                _ptr(gate), _ptr(up), _ptr(down), T, H, E, k, I, _ptr(idx),
                                _ptr(w), _ptr(out), 1 if add_residual else 0, int(capture_token),
                                _ptr(cap_idx), _ptr(cap_w), _ptr(cap_ffn), _ptr(ws), ws.numel(),
                                _stream(stream)), "moe_layer_block")


def moe_layer_host(x_host, Wr, bias, gate, up, down, k, I, idx, w, y_host, ws,
                   stream=None) -> None:
    """``x_host`` / ``y_host``: CPU float32 tensors (pinned for async DMA)."""
    T, H = x_host.shape
    E = Wr.shape[0]
    _check(_lib.moe_layer_host(_ptr(x_host), _ptr(Wr), _ptr(bias), _ptr(gate), _ptr(up),
                               _ptr(down), T, H, E, k, I, _ptr(idx), _ptr(w), _ptr(y_host),
                               _ptr(ws), ws.numel(), _stream(stream)), "moe_layer_host")


def moe_layer_noalloc(x, Wr, bias, gate, up, down, k, I, idx, w, y, stream=None) -> None:
    """Single-token layer without a workspace (the library's fixed scratch)."""
    T, H = x.shape
    E = Wr.shape[0]
    _check(_lib.moe_layer_noalloc(_ptr(x), _ptr(Wr), _ptr(bias), _ptr(gate), _ptr(up), _ptr(down),
                                  T, H, E, k, I, _ptr(idx), _ptr(w), _ptr(y), _stream(stream)),
           "moe_layer_noalloc")


def moe_quantize_q8k(v, q, d, sums, stream=None) -> None:
    """Q8_K blocks of the fp32 rows ``v`` [rows, n]: int8 codes ``q`` [rows, n],
    fp32 scales ``d`` [rows, n/256], int32 sub-block sums ``sums`` [rows, n/32]."""
    rows, n = v.shape
    _check(_lib.moe_quantize_q8k(_ptr(v), rows, n, _ptr(q), _ptr(d), _ptr(sums), _stream(stream)),
           "moe_quantize_q8k")


def moe_ffn_q8k(x, idx, w, gate, up, down, E, I, y, ws, stream=None) -> None:
    T, H = x.shape
    k = idx.shape[1]
    _check(_lib.moe_ffn_q8k(_ptr(x), _ptr(idx), _ptr(w), _ptr(gate), _ptr(up), _ptr(down),
                            T, H, E, k, I, _ptr(y), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_ffn_q8k")


def moe_layer_q8k(x, Wr, bias, gate, up, down, k, I, idx, w, y, ws, stream=None) -> None:
    T, H = x.shape
    E = Wr.shape[0]
    _check(_lib.moe_layer_q8k(_ptr(x), _ptr(Wr), _ptr(bias), _ptr(gate), _ptr(up), _ptr(down),
                              T, H, E, k, I, _ptr(idx), _ptr(w), _ptr(y), _ptr(ws), ws.numel(),
                              _stream(stream)), "moe_layer_q8k")


def moe_ffn_q8k_codes(q, d, sums, idx, w, gate, up, down, E, I, y, ws, stream=None) -> None:
    """``moe_ffn_q8k`` on Q8_K rows: codes ``q`` [T, H], scales ``d``, sub-block sums ``sums``."""
    T, H = q.shape
    k = idx.shape[1]
    _check(_lib.moe_ffn_q8k_codes(_ptr(q), _ptr(d), _ptr(sums), _ptr(idx), _ptr(w), _ptr(gate),
                                  _ptr(up), _ptr(down), T, H, E, k, I, _ptr(y), _ptr(ws),
                                  ws.numel(), _stream(stream)), "moe_ffn_q8k_codes")


def _refuse(t, shape, dtype, name):
    """What is wrong with a tensor that is not a contiguous one of this shape and type."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: {t.dtype}, not {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, not {tuple(shape)}")
    raise ValueError(f"{name}: not contiguous")


def _tensor(t, shape, dtype, name):
    """The device pointer of a contiguous tensor of this shape and type.  The attention half
    takes many buffers whose sizes follow from one another, so the binding checks them before
    the library, which sees only pointers."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, shape, dtype, name)


def _dtype(t, name) -> int:
    code = MOE_DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: {t.dtype} is not one of float32, float16, bfloat16")
    return code


def moe_add_rmsnorm(x, residual, gamma, eps, sum_out=None, y=None, q8k=None, stream=None) -> None:
    """s = x + residual (None: s = x), y = RMSNorm(s) * gamma.  ``sum_out`` receives s, ``y`` the
    normed rows (fp32, fp16 or bf16), ``q8k`` = (q, d, sums) their Q8_K blocks."""
    rows = T, H = x.shape
    q = d = sums = None
    if q8k is not None:
        q = _tensor(q8k[0], rows, _I8, "q")
        d = _tensor(q8k[1], (T, H // 256), _F32, "d")
        sums = _tensor(q8k[2], (T, H // 32), _I32, "sums")
    code = _lib.moe_add_rmsnorm(
        _tensor(x, rows, x.dtype, "x"), _dtype(x, "x"),
        None if residual is None else _tensor(residual, rows, _F32, "residual"),
        _tensor(gamma, (H,), _F32, "gamma"), eps, T, H,
        None if sum_out is None else _tensor(sum_out, rows, _F32, "sum_out"),
        None if y is None else _tensor(y, rows, y.dtype, "y"), 0 if y is None else _dtype(y, "y"),
        q, d, sums, _stream(stream))
    if code:
        raise MoeError(code, "moe_add_rmsnorm")


def _batch(k_pages, v_pages, page_table, q_offs, kv_lens):
    """(pages, table, offsets, lengths) pointers, then B, max_pages, num_pages, page, Hkv, D."""
    cache = P, Hkv, page, D = k_pages.shape
    table = B, max_pages = page_table.shape
    t = k_pages.dtype
    return (_tensor(k_pages, cache, t, "k_pages"), _tensor(v_pages, cache, t, "v_pages"),
            _tensor(page_table, table, _I32, "page_table"), _tensor(q_offs, (B + 1,), _I32, "q_offs"),
            _tensor(kv_lens, (B,), _I32, "kv_lens"), B, max_pages, P, page, Hkv, D)


def moe_rope_append(qkv, pos, inv_freq, q_out, k_pages, v_pages, page_table, q_offs, kv_lens, ws,
                    axis=None, q_norm_w=None, k_norm_w=None, eps=1e-6, interleaved=False,
                    stream=None) -> None:
    """Rows ``qkv`` [N, (Hq + 2 Hkv) D] -> normed and rotated queries ``q_out`` [N, Hq, D], keys
    (normed, rotated) and values into the cache.  ``pos`` int32 [axes, N], ``inv_freq`` float64
    [rot / 2] radians per position, ``axis`` int32 [rot / 2]: the axis of each pair."""
    k, v, table, offs, lens, B, max_pages, P, page, Hkv, D = _batch(k_pages, v_pages, page_table,
                                                                    q_offs, kv_lens)
    out = N, Hq, _ = q_out.shape
    axes, half = pos.shape[0], inv_freq.shape[0]
    t = k_pages.dtype
    code = _lib.moe_rope_append(
        _tensor(qkv, (N, (Hq + 2 * Hkv) * D), t, "qkv"), _tensor(pos, (axes, N), _I32, "pos"),
        _tensor(inv_freq, (half,), _F64, "inv_freq"),
        None if axis is None else _tensor(axis, (half,), _I32, "axis"), axes, 2 * half,
        1 if interleaved else 0, None if q_norm_w is None else _tensor(q_norm_w, (D,), _F32, "q_norm_w"),
        None if k_norm_w is None else _tensor(k_norm_w, (D,), _F32, "k_norm_w"), eps,
        _tensor(q_out, out if out[2] == D else (N, Hq, D), t, "q_out"), k, v, table, offs, lens, N, B,
        max_pages, P, page, Hq, Hkv, D, _dtype(k_pages, "k_pages"), ws.data_ptr(), ws.numel(),
        _stream(stream))
    if code:
        raise MoeError(code, "moe_rope_append")


def moe_attention_workspace_bytes(Hq, Hkv, D) -> int:
    return _lib.moe_attention_workspace_bytes(Hq, Hkv, D)


def alloc_attention_workspace(Hq, Hkv, D, device="cuda") -> torch.Tensor:
    """A uint8 device workspace for moe_attention_paged (and moe_rope_append), initialised."""
    n = moe_attention_workspace_bytes(Hq, Hkv, D)
    if n == 0:
        raise MoeError(1, "moe_attention_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    moe_workspace_init(ws)
    return ws


def moe_attention_paged(q, k_pages, v_pages, page_table, q_offs, kv_lens, max_new, scale, out, ws,
                        lse=None, window=0, softcap=0.0, stream=None) -> None:
    """Attention of the new rows ``q`` [N, Hq, D] over each sequence's cached tokens -> ``out``
    [N, Hq, D], ``lse`` [N, Hq] (optional).  ``max_new``: the most new tokens of a sequence."""
    k, v, table, offs, lens, B, max_pages, P, page, Hkv, D = _batch(k_pages, v_pages, page_table,
                                                                    q_offs, kv_lens)
    N, Hq, _ = q.shape
    rows, t = (N, Hq, D), k_pages.dtype
    code = _lib.moe_attention_paged(
        _tensor(q, rows, t, "q"), k, v, table, offs, lens, N, B, max_new, max_pages, P, page, Hq, Hkv, D,
        _dtype(k_pages, "k_pages"), scale, softcap, window, _tensor(out, rows, t, "out"),
        None if lse is None else _tensor(lse, (N, Hq), _F32, "lse"), ws.data_ptr(), ws.numel(),
        _stream(stream))
    if code:
        raise MoeError(code, "moe_attention_paged")


def moe_read_device_status(ws, stream=None):
    """(status code, detail) of the workspace's sticky device status; syncs the stream."""
    detail = ctypes.c_int32(0)
    code = _lib.moe_read_device_status(_ptr(ws), _stream(stream), ctypes.byref(detail))
    return int(code), int(detail.value)


def moe_debug_set_wait_limit(ns: int) -> None:
    _lib.moe_debug_set_wait_limit(int(ns))


def moe_debug_withhold_arrivals(n: int) -> None:
    _lib.moe_debug_withhold_arrivals(int(n))
