"""Python binding of libwq (include/wq.h): argument marshalling only.

Every function here has the C entry point's name and arguments.  Tensor
arguments may be torch tensors (their device pointer is passed) or raw integer
device addresses.  `stream` defaults to torch's current HIP stream.  A status
other than WQ_OK raises WqError.  All computation happens in the HIP library;
if libwq.so is missing the import fails loudly -- there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libwq.so")

WQ_OK = 0
STATUS_NAMES = {0: "WQ_OK", 1: "WQ_ERR_INVALID_ARG", 2: "WQ_ERR_UNSUPPORTED", 3: "WQ_ERR_SHAPE",
                4: "WQ_ERR_ALIGNMENT", 5: "WQ_ERR_MIXED_FORMAT", 6: "WQ_ERR_WORKSPACE", 7: "WQ_ERR_HIP"}
WQ_NF4, WQ_NVFP4, WQ_Q4_0, WQ_Q8_0, WQ_Q4_1, WQ_Q5_0, WQ_Q4_K, WQ_Q6_K = 1, 2, 3, 4, 5, 6, 7, 8
WQ_BF16, WQ_F32 = 1, 2

EXPORTS = ("wq_status_str", "wq_packed_size", "wq_quantize", "wq_dequantize",
           "wq_workspace_size", "wq_matmul", "wq_matmul_noalloc", "wq_matmul_qkv",
           "wq_act_packed_size", "wq_quantize_act", "wq_w4a4_workspace_size", "wq_matmul_w4a4",
           "wq_cache_size", "wq_cache_write", "wq_cache_read", "wq_attn_workspace_size", "wq_attn")

# Format names accepted by the harness; aliases follow the NF4 option's names
# ("asr: add a 4-bit nf4 option for the Whisper engine": nf4, aliases 4bit, int4).
_FORMAT_NAMES = {"nf4": WQ_NF4, "4bit": WQ_NF4, "int4": WQ_NF4, "nvfp4": WQ_NVFP4,
                 "q4_0": WQ_Q4_0, "q8_0": WQ_Q8_0, "q4_1": WQ_Q4_1, "q5_0": WQ_Q5_0, "q4_k": WQ_Q4_K,
                 "q6_k": WQ_Q6_K}


def format_from_name(name: str) -> int:
    try:
        return _FORMAT_NAMES[name.strip().lower()]
    except KeyError:
        raise ValueError(f"unknown weight format {name!r}; expected one of {sorted(_FORMAT_NAMES)}") from None


class WqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


class wq_desc(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("block", ctypes.c_int32), ("n", ctypes.c_int64),
                ("k", ctypes.c_int64), ("dq_group", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class wq_packed(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class wq_cache_desc(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("page", ctypes.c_int32), ("pages", ctypes.c_int64), ("reserved", ctypes.c_int32)]


class wq_seqs(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("rows", ctypes.c_int32), ("row_start", ctypes.c_void_p),
                ("len", ctypes.c_void_p), ("table", ctypes.c_void_p), ("table_ld", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


def desc(fmt, n: int, k: int, dq: bool = False, block: int = 0) -> wq_desc:
    if isinstance(fmt, str):
        fmt = format_from_name(fmt)
    return wq_desc(int(fmt), int(block), int(n), int(k), 256 if dq else 0, 0)


def _int32(where: str, name: str, v) -> int:
    """v as a 32-bit argument: ctypes would pass its low bits."""
    v = int(v)
    if not -(1 << 31) <= v < 1 << 31:
        raise ValueError(f"{where}: {name} {v} does not fit 32 bits")
    return v


def cache_desc(fmt, head_dim: int, kv_heads: int, page: int, pages: int) -> wq_cache_desc:
    if isinstance(fmt, str):
        fmt = format_from_name(fmt)
    return wq_cache_desc(*(_int32("cache_desc", *a) for a in (("format", fmt), ("head_dim", head_dim), ("kv_heads", kv_heads), ("page", page))),
                         int(pages), 0)


def seqs(batch: int, rows: int, len, table=None, row_start=None, table_ld: int | None = None) -> wq_seqs:  # noqa: A002
    """The sequences of a cache or attention call.  `len`, `table` and `row_start` are int32 device tensors (contiguous;
    `table` [batch, pages per sequence]) or device addresses (a table's address needs `table_ld`); the result keeps
    tensors alive and passes their addresses."""
    for name, t, n in (("len", len, batch), ("table", table, None), ("row_start", row_start, batch + 1)):
        if t is None or isinstance(t, int):
            continue
        if str(t.dtype) != "torch.int32" or not t.is_contiguous():
            raise ValueError(f"seqs: {name} must be a contiguous int32 tensor, got {t.dtype}")
        if n is not None and t.numel() < n:
            raise ValueError(f"seqs: {name} has {t.numel()} entries; {n} are needed")
    if table is not None and not isinstance(table, int):
        if table.dim() != 2 or table.shape[0] < batch:
            raise ValueError(f"seqs: table must be [batch, pages per sequence], got {tuple(table.shape)}")
        if table_ld is not None and table_ld != table.shape[1]:
            raise ValueError(f"seqs: table has {table.shape[1]} entries per sequence, not {table_ld}")
        table_ld = table.shape[1]
    s = wq_seqs(_int32("seqs", "batch", batch), _int32("seqs", "rows", rows), _ptr(row_start), _ptr(len), _ptr(table),
                _int32("seqs", "table_ld", table_ld or 0), 0)
    s.tensors = (row_start, len, table)
    s.device = _device("seqs", *s.tensors)
    return s


def _device(where: str, *args):
    """The device index that the tensors among the arguments share (None if there are none)."""
    dev = None
    for t in args:
        if t is None or isinstance(t, int):
            continue
        d = t.get_device()
        if dev is None:
            dev = d
        elif d != dev:
            raise ValueError(f"{where}: tensors on devices {dev} and {d}")
    return dev


def _call_on(where: str, s: wq_seqs, tensors, stream, check: bool, fn, *args) -> int:
    """fn(*args, stream) with the tensors' device current: a launch goes to the current device, and the default stream
    is that device's."""
    dev = _device(where, *tensors)
    own = getattr(s, "device", None)
    if own is not None:
        if dev is not None and dev != own:
            raise ValueError(f"{where}: tensors on device {dev}, sequences on {own}")
        dev = own
    if dev is not None:
        global _torch
        if _torch is None:
            import torch
            _torch = torch
        if dev != _torch._C._cuda_getDevice():
            with _torch.cuda.device(dev):
                return _check(fn(*args, _stream(stream)), where, check)
        if stream is None:
            return _check(fn(*args, _torch._C._cuda_getCurrentRawStream(dev)), where, check)
    return _check(fn(*args, _stream(stream)), where, check)


_lib = None


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libwq.so not built ({LIB_PATH}); run `python -m block_quantized_bit_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        i64 = ctypes.c_int64
        pd = ctypes.POINTER(wq_desc)
        L.wq_status_str.restype = ctypes.c_char_p
        L.wq_status_str.argtypes = [ctypes.c_int]
        L.wq_packed_size.restype = ctypes.c_int
        L.wq_packed_size.argtypes = [pd, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]
        L.wq_quantize.restype = ctypes.c_int
        L.wq_quantize.argtypes = [pd, P, wq_packed, P]
        L.wq_dequantize.restype = ctypes.c_int
        L.wq_dequantize.argtypes = [pd, wq_packed, P, P]
        L.wq_workspace_size.restype = ctypes.c_int
        L.wq_workspace_size.argtypes = [pd, i64, ctypes.POINTER(ctypes.c_size_t)]
        L.wq_matmul.restype = ctypes.c_int
        L.wq_matmul.argtypes = [pd, i64, P, i64, wq_packed, P, P, ctypes.c_int32, i64, P, ctypes.c_size_t, P]
        L.wq_matmul_noalloc.restype = ctypes.c_int
        L.wq_matmul_noalloc.argtypes = [pd, i64, P, i64, wq_packed, P, P, ctypes.c_int32, i64, P]
        L.wq_matmul_qkv.restype = ctypes.c_int
        L.wq_matmul_qkv.argtypes = [pd, i64, P, i64, wq_packed, P, ctypes.c_int32, ctypes.POINTER(i64),
                                    ctypes.POINTER(P), ctypes.POINTER(i64), ctypes.c_int32, P, ctypes.c_size_t, P]
        L.wq_act_packed_size.restype = ctypes.c_int
        L.wq_act_packed_size.argtypes = [i64, i64, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]
        L.wq_quantize_act.restype = ctypes.c_int
        L.wq_quantize_act.argtypes = [i64, i64, P, i64, P, P, P]
        L.wq_w4a4_workspace_size.restype = ctypes.c_int
        L.wq_w4a4_workspace_size.argtypes = [pd, i64, ctypes.POINTER(ctypes.c_size_t)]
        L.wq_matmul_w4a4.restype = ctypes.c_int
        L.wq_matmul_w4a4.argtypes = [pd, i64, P, P, wq_packed, P, P, ctypes.c_int32, i64, P, ctypes.c_size_t, P]
        pc, ps, i32, sz = ctypes.POINTER(wq_cache_desc), ctypes.POINTER(wq_seqs), ctypes.c_int32, ctypes.c_size_t
        L.wq_cache_size.restype = ctypes.c_int
        L.wq_cache_size.argtypes = [pc, ctypes.POINTER(sz)]
        L.wq_cache_write.restype = ctypes.c_int
        L.wq_cache_write.argtypes = [pc, ps, P, i64, P, i64, i32, P, P]
        L.wq_cache_read.restype = ctypes.c_int
        L.wq_cache_read.argtypes = [pc, ps, P, P, i64, P, i64, i32, P]
        L.wq_attn_workspace_size.restype = ctypes.c_int
        L.wq_attn_workspace_size.argtypes = [pc, ps, i32, ctypes.POINTER(sz)]
        L.wq_attn.restype = ctypes.c_int
        L.wq_attn.argtypes = [pc, ps, i32, P, i64, P, ctypes.c_float, i32, i32, P, i64, P, sz, P]
        _lib = L
    return _lib


def _ptr(t):
    """Device address of a tensor argument.  A host tensor is refused here: the library
    hands its pointers to GPU kernels, which cannot read host memory."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"libwq takes device buffers; got a tensor on {getattr(t, 'device', type(t))}")
    return t.data_ptr()


_torch = None


def _stream(stream):
    if stream is None:
        global _torch
        if _torch is None:
            import torch
            _torch = torch
        return _torch._C._cuda_getCurrentRawStream(_torch.cuda.current_device())   # of torch.cuda.current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(st: int, where: str, check: bool) -> int:
    if check and st != WQ_OK:
        raise WqError(st, where)
    return st


def wq_status_str(status: int) -> str:
    return lib().wq_status_str(int(status)).decode()


def wq_packed_size(d: wq_desc):
    cb = ctypes.c_size_t()
    sb = ctypes.c_size_t()
    _check(lib().wq_packed_size(ctypes.byref(d), ctypes.byref(cb), ctypes.byref(sb)), "wq_packed_size", True)
    return cb.value, sb.value


def wq_quantize(d: wq_desc, w, codes, scales, stream=None, check=True) -> int:
    st = lib().wq_quantize(ctypes.byref(d), _ptr(w), wq_packed(_ptr(codes), _ptr(scales)), _stream(stream))
    return _check(st, "wq_quantize", check)


def wq_dequantize(d: wq_desc, codes, scales, w_out, stream=None, check=True) -> int:
    st = lib().wq_dequantize(ctypes.byref(d), wq_packed(_ptr(codes), _ptr(scales)), _ptr(w_out), _stream(stream))
    return _check(st, "wq_dequantize", check)


def wq_workspace_size(d: wq_desc, m: int) -> int:
    b = ctypes.c_size_t()
    _check(lib().wq_workspace_size(ctypes.byref(d), int(m), ctypes.byref(b)), "wq_workspace_size", True)
    return b.value


def wq_matmul(d: wq_desc, m: int, x, ldx: int, codes, scales, bias, y, ydt: int, ldy: int,
              ws=None, ws_bytes: int = 0, stream=None, check=True) -> int:
    st = lib().wq_matmul(ctypes.byref(d), int(m), _ptr(x), int(ldx), wq_packed(_ptr(codes), _ptr(scales)),
                         _ptr(bias), _ptr(y), int(ydt), int(ldy), _ptr(ws), int(ws_bytes), _stream(stream))
    return _check(st, "wq_matmul", check)


def wq_matmul_noalloc(d: wq_desc, m: int, x, ldx: int, codes, scales, bias, y, ydt: int, ldy: int,
                      stream=None, check=True) -> int:
    st = lib().wq_matmul_noalloc(ctypes.byref(d), int(m), _ptr(x), int(ldx), wq_packed(_ptr(codes), _ptr(scales)),
                                 _ptr(bias), _ptr(y), int(ydt), int(ldy), _stream(stream))
    return _check(st, "wq_matmul_noalloc", check)


def wq_matmul_qkv(d: wq_desc, m: int, x, ldx: int, codes, scales, bias, split_n, ys, ldys, ydt: int,
                  ws=None, ws_bytes: int = 0, stream=None, check=True) -> int:
    ns = len(split_n)
    if len(ys) != ns or len(ldys) != ns:
        raise ValueError(f"wq_matmul_qkv: {ns} splits but {len(ys)} outputs and {len(ldys)} leading dimensions")
    sn = (ctypes.c_int64 * ns)(*[int(v) for v in split_n])
    yp = (ctypes.c_void_p * len(ys))(*[_ptr(v) for v in ys])
    lp = (ctypes.c_int64 * len(ldys))(*[int(v) for v in ldys])
    st = lib().wq_matmul_qkv(ctypes.byref(d), int(m), _ptr(x), int(ldx), wq_packed(_ptr(codes), _ptr(scales)),
                             _ptr(bias), ns, sn, yp, lp, int(ydt), _ptr(ws), int(ws_bytes), _stream(stream))
    return _check(st, "wq_matmul_qkv", check)


def wq_act_packed_size(m: int, k: int):
    cb = ctypes.c_size_t()
    sb = ctypes.c_size_t()
    _check(lib().wq_act_packed_size(int(m), int(k), ctypes.byref(cb), ctypes.byref(sb)), "wq_act_packed_size", True)
    return cb.value, sb.value


def wq_quantize_act(m: int, k: int, x, ldx: int, codes, scales, stream=None, check=True) -> int:
    st = lib().wq_quantize_act(int(m), int(k), _ptr(x), int(ldx), _ptr(codes), _ptr(scales), _stream(stream))
    return _check(st, "wq_quantize_act", check)


def wq_w4a4_workspace_size(d: wq_desc, m: int) -> int:
    b = ctypes.c_size_t()
    _check(lib().wq_w4a4_workspace_size(ctypes.byref(d), int(m), ctypes.byref(b)), "wq_w4a4_workspace_size", True)
    return b.value


def wq_matmul_w4a4(d: wq_desc, m: int, xcodes, xscales, codes, scales, bias, y, ydt: int, ldy: int,
                   ws=None, ws_bytes: int = 0, stream=None, check=True) -> int:
    st = lib().wq_matmul_w4a4(ctypes.byref(d), int(m), _ptr(xcodes), _ptr(xscales),
                              wq_packed(_ptr(codes), _ptr(scales)), _ptr(bias), _ptr(y), int(ydt), int(ldy),
                              _ptr(ws), int(ws_bytes), _stream(stream))
    return _check(st, "wq_matmul_w4a4", check)


def wq_cache_size(d: wq_cache_desc) -> int:
    b = ctypes.c_size_t()
    _check(lib().wq_cache_size(ctypes.byref(d), ctypes.byref(b)), "wq_cache_size", True)
    return b.value


def wq_cache_write(d: wq_cache_desc, s: wq_seqs, k, ldk: int, v, ldv: int, xdt: int, cache, stream=None, check=True) -> int:
    return _call_on("wq_cache_write", s, (k, v, cache), stream, check, lib().wq_cache_write, ctypes.byref(d), ctypes.byref(s),
                    _ptr(k), ldk, _ptr(v), ldv, xdt, _ptr(cache))


def wq_cache_read(d: wq_cache_desc, s: wq_seqs, cache, k, ldk: int, v, ldv: int, ydt: int, stream=None, check=True) -> int:
    return _call_on("wq_cache_read", s, (cache, k, v), stream, check, lib().wq_cache_read, ctypes.byref(d), ctypes.byref(s),
                    _ptr(cache), _ptr(k), ldk, _ptr(v), ldv, ydt)


def wq_attn_workspace_size(d: wq_cache_desc, s: wq_seqs, q_heads: int) -> int:
    b = ctypes.c_size_t()
    _check(lib().wq_attn_workspace_size(ctypes.byref(d), ctypes.byref(s), _int32("wq_attn_workspace_size", "q_heads", q_heads), ctypes.byref(b)),
           "wq_attn_workspace_size", True)
    return b.value


def wq_attn(d: wq_cache_desc, s: wq_seqs, q_heads: int, q, ldq: int, cache, scale: float, causal, window: int, y, ldy: int,
            ws=None, ws_bytes: int = 0, stream=None, check=True) -> int:
    return _call_on("wq_attn", s, (q, cache, y, ws), stream, check, lib().wq_attn, ctypes.byref(d), ctypes.byref(s),
                    _int32("wq_attn", "q_heads", q_heads), _ptr(q), ldq, _ptr(cache), scale, _int32("wq_attn", "causal", causal),
                    _int32("wq_attn", "window", window), _ptr(y), ldy, _ptr(ws), ws_bytes)
