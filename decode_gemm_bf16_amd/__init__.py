"""Python binding of libuw.so, the lossless BF16 weight codec with fused
decode-into-matmul kernels for MI355X (gfx950).

Argument marshalling only: every step runs in the C++/HIP library declared in
``include/uw.h``.  PyTorch supplies device memory and streams.  Importing this
package loads the library and fails loudly if it has not been built
(``python decode_gemm_bf16_amd/build.py``); there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import functools
import operator
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libuw.so")

# enums and flags of uw.h
OK = 0
ERR_INVALID_ARG, ERR_SHAPE, ERR_OOM, ERR_HIP, ERR_FORMAT, ERR_UNSUPPORTED, ERR_NO_DEVICE, ERR_IO = 1, 2, 3, 4, 5, 6, 7, 8
P_AUTO, P1_FULL_DECODE, P2_EXP_DECODE, P3_PALETTE_TRANSCODE, P4_DIRECT_PALETTE, P5_PALETTE_DECODE = 0, 1, 2, 3, 4, 5
FMT_HUFFMAN, FMT_PALETTE, FMT_RAWAUX, ENC_HOST_ONLY = 0x1, 0x2, 0x4, 0x100
(STREAM_SM, STREAM_NIBBLES, STREAM_RAWMAP, STREAM_RAWBEFORE, STREAM_SIDE, STREAM_WORDS, STREAM_OFFSETS,
 STREAM_PALETTE, STREAM_LENGTHS) = range(9)

EXPORTED = [
    "uw_encode", "uw_decode", "uw_matmul", "uw_preprocess", "uw_set_streams", "uw_set_scratch", "uw_set_plan",
    "uw_set_variant", "uw_variant_name", "uw_variant_in_use", "uw_query", "uw_export", "uw_clone", "uw_save", "uw_load", "uw_upload", "uw_evict", "uw_grouped_matmul", "uw_free", "uw_last_error", "uw_silu_mul",
    "uw_mlp_forward", "uw_mlp_workspace_bytes", "uw_mlp_forward_noalloc", "uw_stack_forward", "uw_stack_workspace_bytes",
    "uw_route", "uw_group_rows_workspace_bytes", "uw_group_rows", "uw_dispatch_rows", "uw_combine_rows",
    "uw_moe_workspace_bytes", "uw_moe_forward", "uw_lora_create", "uw_lora_load", "uw_lora_free", "uw_lora_plan_bytes",
    "uw_lora_plan", "uw_lora_workspace_bytes", "uw_lora_apply", "uw_cache_write", "uw_attend_workspace_bytes", "uw_attend",
    "uw_cache_copy_pages", "uw_cache_keep", "uw_pages_create",
    "uw_pages_free", "uw_pages_left", "uw_pages_holders", "uw_pages_take", "uw_pages_share", "uw_pages_drop", "uw_pages_own",
    "uw_pages_compact", "uw_attention_workspace_bytes", "uw_attention_forward", "uw_stream_create", "uw_stream_destroy", "uw_device_cu_count", "uw_gemm_bf16", "uw_device_copy", "uw_device_read",
]

F32, BF16 = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1
LORA_MAX_RANK = 256  # UW_LORA_MAX_RANK


class UwError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"uw status {status}: {msg}")
        self.status = status


class Info(C.Structure):
    _fields_ = [
        ("rows", C.c_int64), ("cols", C.c_int64), ("formats", C.c_uint32), ("chunk", C.c_uint32),
        ("lmax", C.c_uint32), ("distinct_exponents", C.c_uint32), ("palette", C.c_uint8 * 16),
        ("code_lengths", C.c_uint8 * 256), ("raw_groups", C.c_uint64), ("groups", C.c_uint64),
        ("stream_bits", C.c_uint64), ("stream_words", C.c_uint64), ("bpw_palette", C.c_double),
        ("bpw_huffman", C.c_double), ("bpw_resident", C.c_double), ("resident_bytes", C.c_uint64),
        ("scratch_bytes", C.c_uint64 * 6), ("max_row_raw", C.c_uint32),
    ]


class RouteConfig(C.Structure):
    _fields_ = [
        ("experts", C.c_int32), ("top_k", C.c_int32), ("score", C.c_int32), ("groups", C.c_int32),
        ("top_groups", C.c_int32), ("group_score", C.c_int32), ("renormalise", C.c_int32), ("scale", C.c_float),
    ]


class CacheConfig(C.Structure):
    _fields_ = [("heads", C.c_int32), ("kv_heads", C.c_int32), ("dim", C.c_int32), ("page", C.c_int32),
                ("pages", C.c_int64)]


class Rotary(C.Structure):
    _fields_ = [("axes", C.c_int32), ("pairs", C.c_int32), ("adjacent", C.c_int32)]


class AttendConfig(C.Structure):
    _fields_ = [("scale", C.c_float), ("cap", C.c_float), ("window", C.c_int32)]


class AttentionBatch(C.Structure):
    _fields_ = ([(k, C.c_void_p) for k in ("positions", "freqs", "axis", "slots", "offsets", "lengths", "tables", "slopes",
                                           "prefix", "first", "mask")] +
                [(k, C.c_int64) for k in ("tokens", "seqs", "max_tokens", "max_length", "ldt", "max_pages")] +
                [("mask_words", C.c_int32)])


def _preload_runtime() -> None:
    """Load the HIP runtime that PyTorch ships before libuw.so, so that both
    resolve to one runtime (one process must not hold two HIP runtimes: they
    would not share devices, memory or streams)."""
    import importlib.util
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return
    tl = os.path.join(list(spec.submodule_search_locations)[0], "lib")
    for name in ("libamdhip64.so", "libhipblaslt.so"):
        path = os.path.join(tl, name)
        if os.path.exists(path):
            C.CDLL(path, mode=C.RTLD_GLOBAL)


def _load() -> C.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python decode_gemm_bf16_amd/build.py`")
    _preload_runtime()
    lib = C.CDLL(LIB_PATH)
    vp, i64, i32, u32, st = C.c_void_p, C.c_int64, C.c_int32, C.c_uint32, C.c_int
    sig = {
        "uw_encode": ([vp, i64, i64, u32, C.POINTER(vp)], st),
        "uw_decode": ([vp, vp], st),
        "uw_matmul": ([vp, vp, vp, i64, C.c_int], st),
        "uw_preprocess": ([vp, C.c_int], st),
        "uw_set_streams": ([vp, vp, vp], st),
        "uw_set_scratch": ([vp, vp, C.c_size_t], st),
        "uw_set_plan": ([vp, C.POINTER(i32), C.POINTER(i32), C.POINTER(i32), i32], st),
        "uw_set_variant": ([vp, i32], st),
        "uw_variant_name": ([i64, i32], C.c_char_p),
        "uw_variant_in_use": ([vp, i64, i32, C.POINTER(i32), C.c_char_p, C.c_size_t], st),
        "uw_query": ([vp, C.POINTER(Info)], st),
        "uw_export": ([vp, C.c_int, vp, C.c_size_t, C.POINTER(C.c_size_t)], st),
        "uw_clone": ([vp, C.POINTER(vp)], st),
        "uw_save": ([vp, C.c_char_p], st),
        "uw_load": ([C.c_char_p, u32, C.POINTER(vp)], st),
        "uw_upload": ([vp], st),
        "uw_evict": ([vp], st),
        "uw_grouped_matmul": ([C.POINTER(vp), i32, vp, C.POINTER(i64), vp, C.c_int], st),
        "uw_free": ([vp], None),
        "uw_last_error": ([], C.c_char_p),
        "uw_silu_mul": ([vp, vp, vp, i64, vp], st),
        "uw_mlp_forward": ([vp, vp, vp, C.POINTER(i32), vp, vp, i64, vp, C.c_size_t], st),
        "uw_mlp_workspace_bytes": ([i64, i64], C.c_size_t),
        "uw_mlp_forward_noalloc": ([vp, vp, vp, C.POINTER(i32), vp, vp, i64], st),
        "uw_stack_forward": ([C.POINTER(vp), C.POINTER(i32), i32, vp, vp, i64, i32, vp, C.c_size_t], st),
        "uw_stack_workspace_bytes": ([i64, i64, i64], C.c_size_t),
        "uw_route": ([vp, i32, i64, i64, vp, C.POINTER(RouteConfig), vp, vp, vp], st),
        "uw_group_rows_workspace_bytes": ([i64, i32], C.c_size_t),
        "uw_group_rows": ([vp, i64, i32, vp, vp, vp, vp, C.c_size_t, vp], st),
        "uw_dispatch_rows": ([vp, i64, vp, i64, i32, i64, vp, i64, vp], st),
        "uw_combine_rows": ([vp, i64, vp, vp, i64, i32, i64, vp, vp, i32, vp], st),
        "uw_moe_workspace_bytes": ([i64, i64, i64, i32, i32], C.c_size_t),
        "uw_moe_forward": ([C.POINTER(vp), C.POINTER(i32), vp, i32, i64, vp, C.POINTER(RouteConfig), vp, vp, vp, i64,
                            vp, C.c_size_t], st),
        "uw_lora_create": ([i64, i64, i32, i32, C.POINTER(vp)], st),
        "uw_lora_load": ([vp, i32, vp, vp, i32, C.c_float, vp], st),
        "uw_lora_free": ([vp], None),
        "uw_lora_plan_bytes": ([i64, i32], C.c_size_t),
        "uw_lora_plan": ([vp, i64, i32, vp, C.c_size_t, vp], st),
        "uw_lora_workspace_bytes": ([C.POINTER(vp), i32, i64], C.c_size_t),
        # (its five arrays are passed by address: one block of memory holds them)
        "uw_lora_apply": ([vp, i32, vp, C.c_size_t, vp, i64, vp, vp, vp, vp, i64, vp, C.c_size_t, vp], st),
        "uw_cache_write": ([C.POINTER(CacheConfig), C.POINTER(Rotary), vp, i64, vp, i64, vp, i64, i32, vp, vp, vp, vp, i64,
                            vp, i64, vp, vp, vp], st),
        "uw_attend_workspace_bytes": ([i64, i64, i32, i32, i32, i64, i64], C.c_size_t),
        "uw_attend": ([C.POINTER(CacheConfig), C.POINTER(AttendConfig), vp, i64, vp, vp, vp, vp, vp, i64, i64, vp, vp,
                       vp, vp, i32, i64, i64, i64, i64, vp, i64, i32, vp, vp, C.c_size_t, vp], st),
        "uw_cache_copy_pages": ([C.POINTER(CacheConfig), i64, vp, vp, vp, vp, i64, vp], st),
        "uw_cache_keep": ([C.POINTER(CacheConfig), i64, vp, vp, vp, i64, i64, vp, vp, i32, i64, vp, vp], st),
        "uw_pages_create": ([i64, C.POINTER(vp)], st),
        "uw_pages_free": ([vp], None),
        "uw_pages_left": ([vp], i64),
        "uw_pages_holders": ([vp, i32], i32),
        "uw_pages_take": ([vp, i64, vp], st),
        "uw_pages_share": ([vp, vp, i64], st),
        "uw_pages_drop": ([vp, vp, i64], st),
        "uw_pages_own": ([vp, i32, C.POINTER(i32)], st),
        "uw_pages_compact": ([vp, vp, vp, C.POINTER(i64)], st),
        "uw_attention_workspace_bytes": ([C.POINTER(CacheConfig), i64, i64, i64, i64], C.c_size_t),
        "uw_attention_forward": ([vp, vp, vp, vp, C.POINTER(i32), C.POINTER(CacheConfig), C.POINTER(Rotary),
                                  C.POINTER(AttendConfig), C.POINTER(AttentionBatch), vp, vp, vp, vp, vp, C.c_size_t], st),
        "uw_stream_create": ([i32, i32, C.POINTER(vp)], st),
        "uw_stream_destroy": ([vp], st),
        "uw_device_cu_count": ([], i32),
        "uw_gemm_bf16": ([vp, vp, vp, i64, i64, i64, vp], st),
        "uw_device_copy": ([vp, vp, C.c_size_t, vp], st),
        "uw_device_read": ([vp, vp, C.c_size_t, vp], st),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    return lib


_lib = _load()


def _check(status: int) -> None:
    if status != OK:
        raise UwError(status, _lib.uw_last_error().decode(errors="replace"))


def _ptr(t) -> int:
    """Device/host address of a torch tensor or numpy array (None -> 0)."""
    if t is None:
        return 0
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _stream_ptr(stream) -> int | None:
    if stream is None:
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream  # torch.cuda.Stream


def last_error() -> str:
    return _lib.uw_last_error().decode(errors="replace")


def variant_name(tokens: int, variant: int) -> str | None:
    r = _lib.uw_variant_name(tokens, variant)
    return r.decode() if r is not None else None


def variants(tokens: int) -> list[str]:
    out, i = [], 0
    while (n := variant_name(tokens, i)) is not None:
        out.append(n)
        i += 1
    return out


class Matrix:
    """An encoded weight matrix (an ``uw_handle``)."""

    def __init__(self, w_bits: np.ndarray, formats: int = FMT_HUFFMAN | FMT_PALETTE):
        w = np.ascontiguousarray(w_bits, dtype=np.uint16)
        if w.ndim != 2:
            raise ValueError("weight must be a 2-D array of bf16 bit patterns")
        h = C.c_void_p()
        _check(_lib.uw_encode(w.ctypes.data, w.shape[0], w.shape[1], formats, C.byref(h)))
        self._h = h
        self.rows, self.cols = w.shape
        self.formats = formats
        self._keep = []  # buffers whose lifetime the handle relies on (bound scratch)

    @property
    def handle(self) -> int:
        return self._h.value

    def free(self) -> None:
        if self._h:
            _lib.uw_free(self._h)
            self._h = C.c_void_p()

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass

    def clone(self) -> "Matrix":
        """A device copy of this matrix at a new address."""
        h = C.c_void_p()
        _check(_lib.uw_clone(self._h, C.byref(h)))
        m = Matrix.__new__(Matrix)
        m._h, m.rows, m.cols, m.formats, m._keep = h, self.rows, self.cols, self.formats, []
        return m

    def save(self, path: str) -> None:
        """Write the Huffman form to a bundle file (``uw_save``)."""
        _check(_lib.uw_save(self._h, os.fsencode(path)))

    @classmethod
    def load(cls, path: str, formats: int = FMT_HUFFMAN | FMT_PALETTE) -> "Matrix":
        """A matrix read from a bundle file; palette formats are transcoded on
        the device (``uw_load``)."""
        h = C.c_void_p()
        _check(_lib.uw_load(os.fsencode(path), formats, C.byref(h)))
        m = cls.__new__(cls)
        m._h, m.formats, m._keep = h, formats, []
        info = m.info()
        m.rows, m.cols = info["rows"], info["cols"]
        return m

    def upload(self) -> None:
        """Copy a host-only matrix's compressed streams to the device (``uw_upload``)."""
        _check(_lib.uw_upload(self._h))

    def evict(self) -> None:
        """Release the device copy of an uploaded matrix (``uw_evict``)."""
        _check(_lib.uw_evict(self._h))

    def decode(self, out) -> None:
        """bf16 W -> ``out`` (device tensor of rows*cols 16-bit elements)."""
        _check(_lib.uw_decode(self._h, _ptr(out)))

    def matmul(self, x, y, tokens: int | None = None, pipeline: int = P_AUTO) -> None:
        """y[tokens, rows] (float32, device) = x[tokens, cols] (bf16, device) @ W^T."""
        t = x.shape[0] if tokens is None else tokens
        _check(_lib.uw_matmul(self._h, _ptr(x), _ptr(y), t, pipeline))

    def preprocess(self, pipeline: int) -> None:
        _check(_lib.uw_preprocess(self._h, pipeline))

    def set_streams(self, main=None, side=None) -> None:
        _check(_lib.uw_set_streams(self._h, _stream_ptr(main), _stream_ptr(side)))

    def set_scratch(self, buf) -> None:
        nbytes = buf.numel() * buf.element_size()
        _check(_lib.uw_set_scratch(self._h, _ptr(buf), nbytes))
        self._keep = [buf]

    def set_plan(self, entries) -> None:
        """entries: iterable of (max_tokens, pipeline, variant)."""
        entries = list(entries)
        n = len(entries)
        arr = lambda i: (C.c_int32 * max(n, 1))(*[int(e[i]) for e in entries])
        _check(_lib.uw_set_plan(self._h, arr(0), arr(1), arr(2), n))

    def set_variant(self, variant: int) -> None:
        _check(_lib.uw_set_variant(self._h, variant))

    def variant_in_use(self, tokens: int, pipeline: int = 0) -> tuple[int, str]:
        """(pipeline, variant name) that matmul(..., tokens, pipeline) would run."""
        p = C.c_int32(0)
        buf = C.create_string_buffer(96)
        _check(_lib.uw_variant_in_use(self._h, tokens, pipeline, C.byref(p), buf, 96))
        return p.value, buf.value.decode()

    def info(self) -> dict:
        inf = Info()
        _check(_lib.uw_query(self._h, C.byref(inf)))
        d = {k: getattr(inf, k) for k, _ in Info._fields_}
        d["palette"] = list(inf.palette)
        d["code_lengths"] = list(inf.code_lengths)
        d["scratch_bytes"] = list(inf.scratch_bytes)
        return d

    def export(self, which: int) -> np.ndarray:
        n = C.c_size_t()
        _lib.uw_export(self._h, which, None, 0, C.byref(n))
        dtype = np.uint32 if which in (STREAM_RAWMAP, STREAM_RAWBEFORE, STREAM_WORDS, STREAM_OFFSETS) else np.uint8
        buf = np.empty(n.value // np.dtype(dtype).itemsize, dtype=dtype)
        _check(_lib.uw_export(self._h, which, buf.ctypes.data, buf.nbytes, C.byref(n)))
        return buf


def silu_mul(g, u, h, stream=None) -> None:
    _check(_lib.uw_silu_mul(_ptr(g), _ptr(u), _ptr(h), g.numel(), _stream_ptr(stream)))


def gemm_bf16(x, w, y, tokens: int, rows: int, cols: int, stream=None) -> None:
    """Uncompressed baseline through hipBLASLt: y = x @ w^T."""
    _check(_lib.uw_gemm_bf16(_ptr(x), _ptr(w), _ptr(y), tokens, rows, cols, _stream_ptr(stream)))


def device_copy(src, dst, nbytes: int, stream=None) -> None:
    _check(_lib.uw_device_copy(_ptr(src), _ptr(dst), nbytes, _stream_ptr(stream)))


def device_read(src, sink, nbytes: int, stream=None) -> None:
    """Read nbytes of src (HBM read ceiling); sink: >= 16 bytes of device memory."""
    _check(_lib.uw_device_read(_ptr(src), _ptr(sink), nbytes, _stream_ptr(stream)))


def mlp_workspace_bytes(tokens: int, inter: int) -> int:
    return _lib.uw_mlp_workspace_bytes(tokens, inter)


def mlp_forward(gate: Matrix, up: Matrix, down: Matrix, pipelines, x, y, tokens: int, work) -> None:
    p = (C.c_int32 * 3)(*pipelines)
    _check(_lib.uw_mlp_forward(gate._h, up._h, down._h, p, _ptr(x), _ptr(y), tokens, _ptr(work),
                               work.numel() * work.element_size()))


STATIC_WORKSPACE_BYTES = 32 << 20  # UW_STATIC_WORKSPACE_BYTES


def mlp_forward_noalloc(gate: Matrix, up: Matrix, down: Matrix, pipelines, x, y, tokens: int) -> None:
    """The SwiGLU layer with the library's fixed device workspace (no allocation;
    every projection must run the direct palette)."""
    p = (C.c_int32 * 3)(*pipelines)
    _check(_lib.uw_mlp_forward_noalloc(gate._h, up._h, down._h, p, _ptr(x), _ptr(y), tokens))


def stack_workspace_bytes(tokens: int, hidden: int, inter: int) -> int:
    return _lib.uw_stack_workspace_bytes(tokens, hidden, inter)


def stack_forward(mats, pipelines, x, y, tokens: int, work, overlap: bool = True) -> None:
    """mats: flat list [gate0, up0, down0, gate1, ...]."""
    n = len(mats)
    hs = (C.c_void_p * n)(*[m.handle for m in mats])
    p = (C.c_int32 * n)(*pipelines)
    _check(_lib.uw_stack_forward(hs, p, n // 3, _ptr(x), _ptr(y), tokens, int(bool(overlap)), _ptr(work),
                                 work.numel() * work.element_size()))


def stream_create(cu_first: int, cu_count: int) -> int:
    s = C.c_void_p()
    _check(_lib.uw_stream_create(cu_first, cu_count, C.byref(s)))
    return s.value


def stream_destroy(stream: int) -> None:
    _check(_lib.uw_stream_destroy(stream))


def device_cu_count() -> int:
    return int(_lib.uw_device_cu_count())


def bf16_tensor(bits: np.ndarray, device="cuda"):
    """A torch bfloat16 tensor holding exactly the given bf16 bit patterns."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(bits, dtype=np.uint16).view(np.int16))
    return t.to(device).view(torch.bfloat16)


def bits_of(t) -> np.ndarray:
    """bf16/int16 torch tensor -> numpy uint16 bit patterns (host copy)."""
    import torch
    return t.detach().view(torch.int16).cpu().numpy().view(np.uint16)


def grouped_matmul(experts, x, y, row_offsets, pipeline: int = P_AUTO) -> None:
    """y[o[e]:o[e+1]] = x[o[e]:o[e+1]] @ W_e^T for each expert e (``uw_grouped_matmul``)."""
    n = len(experts)
    hs = (C.c_void_p * n)(*[m.handle for m in experts])
    offs = (C.c_int64 * (n + 1))(*[int(v) for v in row_offsets])
    _check(_lib.uw_grouped_matmul(hs, n, _ptr(x), offs, _ptr(y), pipeline))


# ---- routing of tokens to experts and back, low-rank adapters ----
#
# These calls check what the C side cannot see of a tensor: its type, shape,
# strides and device.  A decode step calls them hundreds of times, on kernels
# of a few microseconds, so a check costs one attribute of the tensor each.

_torch = _Tensor = _f32 = _bf16 = _i32 = _i64 = _either = None


def _device() -> int:
    """The current GPU's index (-2 without one: no tensor's device has that index)."""
    global _torch, _Tensor, _f32, _bf16, _i32, _i64, _either
    if _torch is None:
        import torch
        _Tensor, _torch = torch.Tensor, torch
        _f32, _bf16, _i32, _i64 = (torch.float32,), (torch.bfloat16,), (torch.int32,), (torch.int64,)
        _either = _f32 + _bf16
    try:
        return _torch.cuda.current_device()
    except (RuntimeError, AssertionError):
        return -2


def _reject(t, name: str, dtypes, shape, rows: bool = False) -> None:
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d)[6:] for d in dtypes)}, not {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not (t.is_contiguous() or (rows and t.stride(1) == 1 and (t.stride(0) >= t.shape[1] or t.shape[0] == 1))):
        raise ValueError(f"{name} must be contiguous" + (" along its rows, which do not overlap" if rows else ""))
    raise ValueError(f"{name} must be on the current GPU, not {t.device}")


def _tensor(t, name: str, dtypes, shape, dev: int) -> int:
    """Address of ``t``: contiguous, of one of the types, this shape and device."""
    if not (isinstance(t, _Tensor) and t.dtype in dtypes and t.shape == shape and t.get_device() == dev
            and t.is_contiguous()):
        _reject(t, name, dtypes, shape)
    return t.data_ptr()


def _rows(t, name: str, dtypes, shape, dev: int) -> tuple[int, int]:
    """Address and row stride (elements) of a 2-D ``t`` whose rows are contiguous."""
    if isinstance(t, _Tensor) and t.dtype in dtypes and t.shape == shape and t.get_device() == dev:
        if t.is_contiguous():
            return t.data_ptr(), shape[1]
        st = t.stride()
        if shape[0] == 1 and st[1] == 1:
            return t.data_ptr(), shape[1]
        if st[1] == 1 and st[0] >= shape[1]:
            return t.data_ptr(), st[0]
    _reject(t, name, dtypes, shape, True)


def _shape2(t, name: str):
    """The shape of a 2-D tensor."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    s = t.shape
    if len(s) != 2:
        raise ValueError(f"{name} must have two dimensions, not {len(s)}")
    return s


def _bytes(t, name: str, dev: int) -> tuple[int, int]:
    """Address and size of a workspace tensor of any type and shape (None: 0, 0)."""
    if t is None:
        return 0, 0
    if not isinstance(t, _Tensor) or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and on the current GPU")
    return t.data_ptr(), t.nbytes


@functools.lru_cache(maxsize=64)
def _route_config(experts, top_k, score, groups, top_groups, group_score, renormalise, scale) -> RouteConfig:
    return RouteConfig(experts, top_k, score, groups, top_groups, group_score, int(bool(renormalise)), scale)


def route(logits, experts, weights, score: int = SCORE_SOFTMAX, bias=None, groups: int = 1, top_groups: int = 1,
          group_score: int = GROUP_MAX, renormalise: bool = True, scale: float = 1.0, stream=None) -> None:
    """Choose each token's experts (``uw_route``): logits [tokens, E] float32 or
    bfloat16 -> experts [tokens, top_k] int32 and weights [tokens, top_k] float32."""
    dev = _device()
    shape = t, e = _shape2(logits, "logits")
    lp, ld = _rows(logits, "logits", _either, shape, dev)
    out = _shape2(experts, "experts")
    k = out[1]
    cfg = _route_config(e, k, score, groups, top_groups, group_score, renormalise, scale)
    _check(_lib.uw_route(lp, F32 if logits.dtype == _f32[0] else BF16, ld, t,
                         None if bias is None else _tensor(bias, "bias", _f32, (e,), dev), cfg,
                         _tensor(experts, "experts", _i32, (t, k), dev), _tensor(weights, "weights", _f32, out, dev),
                         _stream_ptr(stream)))


def group_rows_workspace_bytes(n: int, groups: int) -> int:
    return _lib.uw_group_rows_workspace_bytes(n, groups)


def group_rows(index, groups: int, offsets, order, slot, work=None, stream=None) -> None:
    """Stable counting sort of index (int32, any shape, n entries) into groups
    (``uw_group_rows``): offsets [groups + 1], order [n] and slot (index's shape), int32."""
    dev = _device()
    shape = index.shape
    ip = _tensor(index, "index", _i32, shape, dev)
    n = index.numel()
    wp, wb = _bytes(work, "work", dev)
    _check(_lib.uw_group_rows(ip, n, groups, _tensor(offsets, "offsets", _i32, (groups + 1,), dev),
                              _tensor(order, "order", _i32, (n,), dev), _tensor(slot, "slot", _i32, shape, dev), wp, wb,
                              _stream_ptr(stream)))


def dispatch_rows(x, slot, xs, stream=None) -> None:
    """xs[slot[t, j]] = x[t] (``uw_dispatch_rows``): x [tokens, cols] bfloat16, slot
    [tokens, top_k] int32, xs [rows, cols] bfloat16."""
    dev = _device()
    shape = t, c = _shape2(x, "x")
    xp, ld = _rows(x, "x", _bf16, shape, dev)
    k = _shape2(slot, "slot")[1]
    rows = _shape2(xs, "xs")[0]
    _check(_lib.uw_dispatch_rows(xp, ld, _tensor(slot, "slot", _i32, (t, k), dev), t, k, c,
                                 _tensor(xs, "xs", _bf16, (rows, c), dev), rows, _stream_ptr(stream)))


def combine_rows(ys, slot, weights, y, base=None, stream=None) -> None:
    """y[t] = base[t] + sum_j weights[t, j] * ys[slot[t, j]] (``uw_combine_rows``): ys
    [rows, cols] float32, y [tokens, cols] float32 or bfloat16, base float32 or None."""
    dev = _device()
    shape = rows, c = _shape2(ys, "ys")
    yp = _tensor(ys, "ys", _f32, shape, dev)
    entries = t, k = _shape2(slot, "slot")
    _check(_lib.uw_combine_rows(yp, rows, _tensor(slot, "slot", _i32, entries, dev),
                                _tensor(weights, "weights", _f32, entries, dev), t, k, c,
                                None if base is None else _tensor(base, "base", _f32, (t, c), dev),
                                _tensor(y, "y", _either, (t, c), dev), F32 if y.dtype == _f32[0] else BF16,
                                _stream_ptr(stream)))


def moe_workspace_bytes(tokens: int, hidden: int, inter: int, experts: int, top_k: int) -> int:
    return _lib.uw_moe_workspace_bytes(tokens, hidden, inter, experts, top_k)


def moe_forward(mats, pipelines, logits, x, y, work, top_k: int, score: int = SCORE_SOFTMAX, bias=None, groups: int = 1,
                top_groups: int = 1, group_score: int = GROUP_MAX, renormalise: bool = True, scale: float = 1.0,
                base=None) -> None:
    """A layer of SwiGLU experts (``uw_moe_forward``) on the experts' main stream.
    mats: flat list [gate0, up0, down0, gate1, ...]; logits [tokens, E]."""
    n = len(mats)
    if n == 0 or n % 3:
        raise ValueError("mats must hold gate, up and down of each expert")
    dev = _device()
    t, hidden = _shape2(logits, "logits")[0], mats[0].cols
    lp, ld = _rows(logits, "logits", _either, (t, n // 3), dev)
    cfg = _route_config(n // 3, top_k, score, groups, top_groups, group_score, renormalise, scale)
    wp, wb = _bytes(work, "work", dev)
    _check(_lib.uw_moe_forward((C.c_void_p * n)(*[m.handle for m in mats]), (C.c_int32 * 3)(*pipelines), lp,
                               F32 if logits.dtype == _f32[0] else BF16, ld,
                               None if bias is None else _tensor(bias, "bias", _f32, (n // 3,), dev), cfg,
                               _tensor(x, "x", _bf16, (t, hidden), dev),
                               None if base is None else _tensor(base, "base", _f32, (t, hidden), dev),
                               _tensor(y, "y", _f32, (t, hidden), dev), t, wp, wb))


class Adapters:
    """Low-rank adapters of one projection in numbered slots (a ``uw_lora``)."""

    def __init__(self, slots: int, rows: int, cols: int, max_rank: int):
        h = C.c_void_p()
        self._h = h
        _check(_lib.uw_lora_create(rows, cols, slots, max_rank, C.byref(h)))
        self.slots, self.rows, self.cols, self.max_rank = slots, rows, cols, max_rank

    @property
    def handle(self) -> int:
        return self._h.value

    def load(self, slot: int, a, b, scale: float = 1.0, stream=None) -> None:
        """Copy A [rank, cols] and B [rows, rank] (bfloat16, on the GPU) into a slot (``uw_lora_load``)."""
        dev = _device()
        rank = _shape2(a, "a")[0]
        _check(_lib.uw_lora_load(self._h, slot, _tensor(a, "a", _bf16, (rank, self.cols), dev),
                                 _tensor(b, "b", _bf16, (self.rows, rank), dev), rank, scale, _stream_ptr(stream)))

    def clear(self, slot: int, stream=None) -> None:
        """Empty a slot: its tokens have no adapter."""
        _check(_lib.uw_lora_load(self._h, slot, None, None, 0, 0.0, _stream_ptr(stream)))

    def free(self) -> None:
        if self._h:
            _lib.uw_lora_free(self._h)
            self._h = C.c_void_p()

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


_LORA_BLOCK = [C.c_int64 * (5 * n) for n in range(5)]  # handles, bases, their strides, outputs, theirs


def lora_plan_bytes(tokens: int, slots: int) -> int:
    return _lib.uw_lora_plan_bytes(tokens, slots)


def lora_plan(index, slots: int, plan, stream=None) -> None:
    """Sort a batch's tokens by adapter slot (``uw_lora_plan``): index [tokens] int32."""
    dev = _device()
    n = index.numel()
    ip = _tensor(index, "index", _i32, (n,), dev)
    pp, pb = _bytes(plan, "plan", dev)
    _check(_lib.uw_lora_plan(ip, n, slots, pp, pb, _stream_ptr(stream)))


def lora_workspace_bytes(adapters, tokens: int) -> int:
    n = len(adapters)
    return _lib.uw_lora_workspace_bytes((C.c_void_p * n)(*[a.handle for a in adapters]), n, tokens)


def lora_apply(adapters, plan, x, ys, work, bases=None, stream=None) -> None:
    """ys[i] = bases[i] + scale * B (A x) per token for each projection's ``Adapters``
    (``uw_lora_apply``, 1 to 4 of them); bases None: in place, on top of what ys
    hold.  A base may be None by itself (zeros)."""
    n = len(adapters)
    if bases is None:
        bases = ys
    if not 1 <= n <= 4 or len(ys) != n or len(bases) != n:
        raise ValueError("adapters, ys and bases must have one length, 1 to 4")
    dev = _device()
    t = _shape2(x, "x")[0]
    xp, ldx = _rows(x, "x", _bf16, (t, adapters[0].cols), dev)
    hs, yp, ldy, bp, ldb = [], [], [], [], []
    for a, y, b in zip(adapters, ys, bases):
        hs.append(a._h.value or 0)
        shape = (t, a.rows)
        p, ld = _rows(y, "ys", _f32, shape, dev)
        yp.append(p)
        ldy.append(ld)
        if b is not y:
            p, ld = (0, 0) if b is None else _rows(b, "bases", _f32, shape, dev)
        bp.append(p)
        ldb.append(ld)
    pp, pb = _bytes(plan, "plan", dev)
    wp, wb = _bytes(work, "work", dev)
    block = _LORA_BLOCK[n](*hs, *bp, *ldb, *yp, *ldy)
    at, step = C.addressof(block), 8 * n
    _check(_lib.uw_lora_apply(at, n, pp, pb, xp, ldx, at + step, at + 2 * step, at + 3 * step, at + 4 * step, t, wp, wb,
                              _stream_ptr(stream)))


# ---- a paged cache of keys and values, and attention over it ----
#
# A layer's cache is two bfloat16 tensors kc and vc [pages, kv_heads, page, dim], all
# layers' [layers, pages, kv_heads, page, dim] (kc[l] is one layer's).  Within a page
# of a head the elements are in the order of the matrix operands (include/uw.h).


def _fits(v, bits: int = 32) -> bool:
    """Whether a whole number is one of so many bits (the C types cut others)."""
    return -(1 << (bits - 1)) <= operator.index(v) < 1 << (bits - 1)


def _attend_sizes(tokens, seqs, heads, kv_heads, dim, max_tokens, max_length) -> bool:
    """Whether the C types hold them (0 bytes are the answer to others)."""
    return all(_fits(v, 64) for v in (tokens, seqs, max_tokens, max_length)) and all(_fits(v) for v in (heads, kv_heads, dim))


def _page_list(pages) -> np.ndarray:
    a = np.asarray(pages)
    if a.size == 0:
        return np.empty(0, dtype=np.int32)
    if a.dtype.kind not in "iu":
        raise TypeError(f"pages must be whole numbers, not {a.dtype}")
    if not _fits(a.min()) or not _fits(a.max()):
        raise ValueError("a page's number must be that of one of the cache's pages")
    return np.ascontiguousarray(a, dtype=np.int32)


@functools.lru_cache(maxsize=256)
def _cache_config(heads, kv_heads, dim, page, pages) -> CacheConfig:
    return CacheConfig(heads, kv_heads, dim, page, pages)


@functools.lru_cache(maxsize=64)
def _attend_config(scale, cap, window) -> AttendConfig:
    c = AttendConfig(scale, cap, window)  # (its types cut what they cannot hold)
    if c.window != window:
        raise ValueError(f"window must be 0..2^31-1, not {window}")
    if cap and not c.cap:
        raise ValueError(f"cap must be 0 or a float32 above it, not {cap}")
    return c


@functools.lru_cache(maxsize=64)
def _rotary(axes, pairs, adjacent) -> Rotary:
    return Rotary(axes, pairs, int(bool(adjacent)))


def _cache_shape(kc, dims: int):
    if not isinstance(kc, _Tensor):
        raise TypeError("kc must be a torch tensor")
    s = kc.shape
    if len(s) != dims:
        raise ValueError(f"kc must have {dims} dimensions, not {len(s)}")
    return s


def _heads(cols: int, dim: int, name: str) -> int:
    if dim < 1 or cols % dim:
        raise ValueError(f"{name} must have a multiple of {dim} columns, not {cols}")
    return cols // dim


def cache_write(q, k, v, positions, freqs, slots, qr, kc, vc, axis=None, adjacent: bool = False, stream=None) -> None:
    """Turn q and k by their rotary positions, write k and v to the cache (``uw_cache_write``):
    q [tokens, heads * dim] (or None) -> qr, bfloat16; k, v [tokens, kv_heads * dim], all float32
    or all bfloat16; positions [axes, tokens] and slots [tokens] int32, freqs [pairs] float32,
    axis [pairs] int32 or None."""
    dev = _device()
    shape = pages, kv, page, dim = _cache_shape(kc, 4)
    t = _shape2(k, "k")[0]
    kind = (k.dtype,) if k.dtype in _either else _either
    kp, ldk = _rows(k, "k", kind, (t, kv * dim), dev)
    vp, ldv = _rows(v, "v", kind, (t, kv * dim), dev)
    heads = qp = ldq = op = ldo = 0
    if q is not None:
        rows = _shape2(q, "q")
        qp, ldq = _rows(q, "q", kind, (t, rows[1]), dev)
        heads = _heads(rows[1], dim, "q")
        op, ldo = _rows(qr, "qr", _bf16, (t, rows[1]), dev)
    axes = _shape2(positions, "positions")[0]
    pairs = freqs.numel()
    _check(_lib.uw_cache_write(_cache_config(heads, kv, dim, page, pages), _rotary(axes, pairs, adjacent), qp, ldq, kp,
                               ldk, vp, ldv, F32 if k.dtype == _f32[0] else BF16,
                               _tensor(positions, "positions", _i32, (axes, t), dev),
                               _tensor(freqs, "freqs", _f32, (pairs,), dev),
                               None if axis is None else _tensor(axis, "axis", _i32, (pairs,), dev),
                               _tensor(slots, "slots", _i32, (t,), dev), t, op, ldo,
                               _tensor(kc, "kc", _bf16, shape, dev), _tensor(vc, "vc", _bf16, shape, dev),
                               _stream_ptr(stream)))


def attend_workspace_bytes(tokens: int, seqs: int, heads: int, kv_heads: int, dim: int, max_tokens: int,
                           max_length: int) -> int:
    sizes = tokens, seqs, heads, kv_heads, dim, max_tokens, max_length
    return _lib.uw_attend_workspace_bytes(*sizes) if _attend_sizes(*sizes) else 0


def attend(q, kc, vc, offsets, lengths, tables, y, work=None, scale: float | None = None, cap: float = 0.0,
           window: int = 0, slopes=None, prefix=None, first=None, mask=None, lse=None, max_tokens: int | None = None,
           max_length: int | None = None, stream=None) -> None:
    """Attention of each sequence's new tokens over its pages (``uw_attend``): q [tokens,
    heads * dim] bfloat16 -> y bfloat16 or float32; offsets [seqs + 1], lengths [seqs] and tables
    [seqs, max_pages] int32; slopes [heads] float32, prefix [seqs] and first [tokens] int32, mask
    [tokens, words] int64, lse [tokens, heads] float32.  scale None: dim ** -0.5.  max_tokens and
    max_length (None: all tokens, the tables' reach) say what to lay the call out for; work is
    sized for the same numbers."""
    dev = _device()
    shape = pages, kv, page, dim = _cache_shape(kc, 4)
    rows = t, cols = _shape2(q, "q")
    heads = _heads(cols, dim, "q")
    config = _attend_config(dim ** -0.5 if scale is None else scale, cap, window)
    qp, ldq = _rows(q, "q", _bf16, rows, dev)
    yp, ldy = _rows(y, "y", _either, rows, dev)
    table = n, reach = _shape2(tables, "tables")
    tp, ldt = _rows(tables, "tables", _i32, table, dev)
    words = 0 if mask is None else _shape2(mask, "mask")[1]
    wp, wb = _bytes(work, "work", dev)
    _check(_lib.uw_attend(_cache_config(heads, kv, dim, page, pages), config, qp, ldq,
                          _tensor(kc, "kc", _bf16, shape, dev), _tensor(vc, "vc", _bf16, shape, dev),
                          _tensor(offsets, "offsets", _i32, (n + 1,), dev),
                          _tensor(lengths, "lengths", _i32, (n,), dev), tp, ldt, reach,
                          None if slopes is None else _tensor(slopes, "slopes", _f32, (heads,), dev),
                          None if prefix is None else _tensor(prefix, "prefix", _i32, (n,), dev),
                          None if first is None else _tensor(first, "first", _i32, (t,), dev),
                          None if mask is None else _tensor(mask, "mask", _i64, (t, words), dev), words, t, n,
                          t if max_tokens is None else max_tokens, reach * page if max_length is None else max_length,
                          yp, ldy, F32 if y.dtype == _f32[0] else BF16,
                          None if lse is None else _tensor(lse, "lse", _f32, (t, heads), dev), wp, wb,
                          _stream_ptr(stream)))


def cache_copy_pages(kc, vc, src, dst, stream=None) -> None:
    """Copy page src[i] to page dst[i] in all layers (``uw_cache_copy_pages``): kc, vc
    [layers, pages, kv_heads, page, dim], src and dst [n] int32."""
    dev = _device()
    shape = layers, pages, kv, page, dim = _cache_shape(kc, 5)
    n = src.numel()
    _check(_lib.uw_cache_copy_pages(_cache_config(0, kv, dim, page, pages), layers, _tensor(kc, "kc", _bf16, shape, dev),
                                    _tensor(vc, "vc", _bf16, shape, dev), _tensor(src, "src", _i32, (n,), dev),
                                    _tensor(dst, "dst", _i32, (n,), dev), n, _stream_ptr(stream)))


def cache_keep(kc, vc, tables, starts, kept, lengths, stream=None) -> None:
    """Move the rows of accepted drafted tokens to their places in all layers (``uw_cache_keep``):
    kc, vc [layers, pages, kv_heads, page, dim]; tables [seqs, max_pages], starts [seqs], kept
    [seqs, most] int32; lengths [seqs] int32 is written."""
    dev = _device()
    shape = layers, pages, kv, page, dim = _cache_shape(kc, 5)
    table = n, reach = _shape2(tables, "tables")
    tp, ldt = _rows(tables, "tables", _i32, table, dev)
    most = _shape2(kept, "kept")[1]
    _check(_lib.uw_cache_keep(_cache_config(0, kv, dim, page, pages), layers, _tensor(kc, "kc", _bf16, shape, dev),
                              _tensor(vc, "vc", _bf16, shape, dev), tp, ldt, reach,
                              _tensor(starts, "starts", _i32, (n,), dev), _tensor(kept, "kept", _i32, (n, most), dev),
                              most, n, _tensor(lengths, "lengths", _i32, (n,), dev), _stream_ptr(stream)))


class Pages:
    """The pages of a cache, counted on the host (a ``uw_pages``): lists of pages are
    int32 arrays.  The rows are copied by ``cache_copy_pages``."""

    def __init__(self, pages: int):
        h = C.c_void_p()
        self._h = h
        if not _fits(pages, 64):
            raise ValueError(f"pages must be 1..2^26, not {pages}")
        _check(_lib.uw_pages_create(pages, C.byref(h)))
        self.pages = pages

    @property
    def left(self) -> int:
        return _lib.uw_pages_left(self._h)

    def holders(self, page: int) -> int:
        return _lib.uw_pages_holders(self._h, page) if _fits(page) else 0

    def take(self, n: int) -> np.ndarray:
        """The n lowest free pages."""
        if not _fits(n, 64):
            raise ValueError(f"n must be 0..{self.pages}, not {n}")
        out = np.empty(min(max(n, 0), self.pages), dtype=np.int32)
        _check(_lib.uw_pages_take(self._h, n, out.ctypes.data))
        return out

    def share(self, pages) -> None:
        """A fork: each page is held once more."""
        a = _page_list(pages)
        _check(_lib.uw_pages_share(self._h, a.ctypes.data, a.size))

    def drop(self, pages) -> None:
        """Each page is held once less; free where nobody holds it."""
        a = _page_list(pages)
        _check(_lib.uw_pages_drop(self._h, a.ctypes.data, a.size))

    def own(self, page: int) -> int:
        """The page to write in place of ``page``: itself, or a new one to copy it to."""
        if not _fits(page):
            raise ValueError(f"page must be one of the {self.pages}, not {page}")
        out = C.c_int32()
        _check(_lib.uw_pages_own(self._h, page, C.byref(out)))
        return out.value

    def compact(self) -> tuple[np.ndarray, np.ndarray]:
        """(sources, destinations) of the moves that bring the used pages together."""
        src, dst, n = np.empty(self.pages, dtype=np.int32), np.empty(self.pages, dtype=np.int32), C.c_int64()
        _check(_lib.uw_pages_compact(self._h, src.ctypes.data, dst.ctypes.data, C.byref(n)))
        return src[:n.value].copy(), dst[:n.value].copy()

    def free(self) -> None:
        if self._h:
            _lib.uw_pages_free(self._h)
            self._h = C.c_void_p()

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def attention_workspace_bytes(tokens: int, seqs: int, heads: int, kv_heads: int, dim: int, max_tokens: int,
                              max_length: int) -> int:
    if not _attend_sizes(tokens, seqs, heads, kv_heads, dim, max_tokens, max_length):
        return 0
    return _lib.uw_attention_workspace_bytes(CacheConfig(heads, kv_heads, dim, 32, 1), tokens, seqs, max_tokens, max_length)


def attention_forward(q: Matrix, k: Matrix, v: Matrix, o: Matrix, pipelines, x, y, work, kc, vc, positions, freqs, slots,
                      offsets, lengths, tables, axis=None, adjacent: bool = False, scale: float | None = None,
                      cap: float = 0.0, window: int = 0, slopes=None, prefix=None, first=None, mask=None,
                      max_tokens: int | None = None, max_length: int | None = None) -> None:
    """An attention layer on compressed projections (``uw_attention_forward``), on the
    handles' main stream: x [tokens, hidden] bfloat16 -> y [tokens, hidden] float32; the
    others as in ``cache_write`` and ``attend``."""
    dev = _device()
    shape = pages, kv, page, dim = _cache_shape(kc, 4)
    rows = t, hidden = _shape2(x, "x")
    if hidden != q.cols:
        raise ValueError(f"x must have {q.cols} columns, not {hidden}")
    heads = _heads(q.rows, dim, "q's output")
    config = _attend_config(dim ** -0.5 if scale is None else scale, cap, window)
    axes = _shape2(positions, "positions")[0]
    pairs = freqs.numel()
    table = n, reach = _shape2(tables, "tables")
    tp, ldt = _rows(tables, "tables", _i32, table, dev)
    words = 0 if mask is None else _shape2(mask, "mask")[1]
    batch = AttentionBatch(
        _tensor(positions, "positions", _i32, (axes, t), dev), _tensor(freqs, "freqs", _f32, (pairs,), dev),
        None if axis is None else _tensor(axis, "axis", _i32, (pairs,), dev), _tensor(slots, "slots", _i32, (t,), dev),
        _tensor(offsets, "offsets", _i32, (n + 1,), dev), _tensor(lengths, "lengths", _i32, (n,), dev), tp,
        None if slopes is None else _tensor(slopes, "slopes", _f32, (heads,), dev),
        None if prefix is None else _tensor(prefix, "prefix", _i32, (n,), dev),
        None if first is None else _tensor(first, "first", _i32, (t,), dev),
        None if mask is None else _tensor(mask, "mask", _i64, (t, words), dev), t, n,
        t if max_tokens is None else max_tokens, reach * page if max_length is None else max_length, ldt, reach, words)
    wp, wb = _bytes(work, "work", dev)
    _check(_lib.uw_attention_forward(q._h, k._h, v._h, o._h, (C.c_int32 * 4)(*pipelines),
                                     _cache_config(heads, kv, dim, page, pages), _rotary(axes, pairs, adjacent), config, batch,
                                     _tensor(x, "x", _bf16, rows, dev), _tensor(kc, "kc", _bf16, shape, dev),
                                     _tensor(vc, "vc", _bf16, shape, dev), _tensor(y, "y", _f32, rows, dev), wp, wb))
