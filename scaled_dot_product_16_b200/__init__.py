"""Python binding of libattn.so: scaled-dot-product attention forward on B200 (sm_100a).

The operations (attn_fwd, attn_fwd_masked, attn_fwd_accumulate, attn_sparse_csr,
attn_sparse_csr_tc, attn_csr_plan_size, attn_csr_plan, attn_sparse_csr_tc_planned, attn_merge,
attn_fwd_sinks, attn_decode_workspace_size, attn_decode_paged, attn_cache_append, attn_cache_fork,
attn_cache_reserve, attn_cache_grow, attn_cache_evict, attn_cache_compact, attn_cache_copy,
attn_get_last_error) are the C-ABI calls declared in ``include/attn.h``; the functions here carry the same names and only marshal
arguments (tensor data pointers, sizes, the current CUDA stream) into them. Every step of the
computation runs in the library's CUDA kernels. There is no CPU path: if ``libattn.so`` is missing the first call raises.

PyTorch is used for device memory and streams only: pass CUDA tensors (contiguous, in the
layouts the header states) and preallocated outputs.
"""
from __future__ import annotations

import ctypes
import operator
import os
import threading
from typing import Optional

__all__ = [
    "attn_fwd", "attn_fwd_accumulate", "attn_sparse_csr", "attn_merge", "attn_get_last_error", "AttnError",
    "ATTN_BF16", "ATTN_F32", "ATTN_F16", "ATTN_BHSD", "ATTN_TND", "ATTN_MASK_NONE",
    "ATTN_MASK_CAUSAL_TOPLEFT", "ATTN_MASK_CAUSAL_BOTTOMRIGHT", "ATTN_MASK_BAND", "lib_path",
    "load_library", "attn_fwd_masked", "attn_sparse_csr_tc", "attn_csr_plan_size", "attn_csr_plan",
    "attn_sparse_csr_tc_planned", "attn_sparse_csr_tc_noalloc", "attn_fwd_sinks",
    "attn_decode_workspace_size", "attn_decode_paged", "attn_cache_append", "attn_cache_fork",
    "attn_cache_reserve", "attn_cache_grow", "attn_cache_evict", "attn_cache_compact", "attn_cache_copy", "ATTN_WINDOW_ALL",
]

(ATTN_OK, ATTN_ERR_INVALID, ATTN_ERR_UNSUPPORTED, ATTN_ERR_CUDA, ATTN_ERR_DATA, ATTN_ERR_TIMEOUT,
 ATTN_ERR_PAGES) = range(7)
ATTN_BF16, ATTN_F32, ATTN_F16 = 0, 1, 2
ATTN_BHSD, ATTN_TND = 0, 1
ATTN_MASK_NONE, ATTN_MASK_CAUSAL_TOPLEFT, ATTN_MASK_CAUSAL_BOTTOMRIGHT, ATTN_MASK_BAND = 0, 1, 2, 3
ATTN_WINDOW_ALL = 1 << 30  # window_tokens that keeps every key

_HERE = os.path.dirname(os.path.abspath(__file__))
_lock = threading.Lock()
_lib = None


class AttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_status_string(status)} (status {status})")


def lib_path() -> str:
    return os.path.join(_HERE, "libattn.so")


def load_library():
    """Load libattn.so (once). Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -m scaled_dot_product_16_b200.build`")
        lib = ctypes.CDLL(path)
        P, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
        lib.attn_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, I, I, I, P, P, P, P]
        lib.attn_fwd.restype = I
        lib.attn_fwd_accumulate.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, I, I, I, I, P, P, P, P]
        lib.attn_fwd_accumulate.restype = I
        lib.attn_fwd_masked.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, F, I, I64, I64, P, I64,
                                        I64, I, I, P, P, P, P]
        lib.attn_fwd_masked.restype = I
        lib.attn_sparse_csr.argtypes = [P, P, P, P, P, I, I, I, I, I64, P, P]
        lib.attn_sparse_csr_tc.argtypes = [P, P, P, P, P, I, I, I, I, I64, I, P, P]
        lib.attn_sparse_csr_tc.restype = I
        lib.attn_sparse_csr.restype = I
        lib.attn_csr_plan_size.argtypes = [I, I, I, I64, ctypes.POINTER(I64)]
        lib.attn_csr_plan_size.restype = I
        lib.attn_csr_plan.argtypes = [P, P, I, I, I, I64, P, I64, P]
        lib.attn_csr_plan.restype = I
        lib.attn_sparse_csr_tc_planned.argtypes = [P, P, P, P, I64, I, I, I, I, I64, I, P, P]
        lib.attn_sparse_csr_tc_planned.restype = I
        lib.attn_sparse_csr_tc_noalloc.argtypes = [P, P, P, P, P, I, I, I, I, I64, I, P, P]
        lib.attn_sparse_csr_tc_noalloc.restype = I
        lib.attn_merge.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, P, P, P, P, P]
        lib.attn_merge.restype = I
        lib.attn_fwd_sinks.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, I64, I64, I, I, P, P, P, P]
        lib.attn_fwd_sinks.restype = I
        lib.attn_decode_workspace_size.argtypes = [I, I, I, I, ctypes.POINTER(I64)]
        lib.attn_decode_workspace_size.restype = I
        lib.attn_decode_paged.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I64, F, I64, I64, I, I, P, I64,
                                          P, P, P, P]
        lib.attn_decode_paged.restype = I
        lib.attn_cache_append.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I64, I, I, P, P, P]
        lib.attn_cache_append.restype = I
        lib.attn_cache_fork.argtypes = [P, P, P, P, I, I, I, I, P, P, P, P]
        lib.attn_cache_fork.restype = I
        lib.attn_cache_reserve.argtypes = [P, P, P, P, I, I, I, I, P, P]
        lib.attn_cache_reserve.restype = I
        lib.attn_cache_grow.argtypes = [P, P, P, P, I, I, I, I, I, P, P, P]
        lib.attn_cache_grow.restype = I
        lib.attn_cache_evict.argtypes = [P, P, P, I, I, I, I, I64, I64, P]
        lib.attn_cache_evict.restype = I
        lib.attn_cache_compact.argtypes = [P, P, I, I, I, P, P, P, P, P, P]
        lib.attn_cache_compact.restype = I
        lib.attn_cache_copy.argtypes = [P, I, I, I64, I64, I, P, P, P]
        lib.attn_cache_copy.restype = I
        lib.attn_get_last_error.argtypes = [P, ctypes.POINTER(I)]
        lib.attn_get_last_error.restype = I
        lib.attn_status_string.argtypes = [I]
        lib.attn_status_string.restype = ctypes.c_char_p
        lib.attn_abi_version.argtypes = []
        lib.attn_abi_version.restype = I
        _lib = lib
        return lib


def _status_string(status: int) -> str:
    try:
        return load_library().attn_status_string(int(status)).decode()
    except Exception:  # pragma: no cover - only for messages
        return "unknown"


_ELEM = {ATTN_BF16: "bfloat16", ATTN_F32: "float32", ATTN_F16: "float16"}


def _dtype_name(x) -> str:
    return str(getattr(x, "dtype", "")).replace("torch.", "")


def _ptr(x, name: str = "tensor", numel: int = 0, dtype: Optional[str] = None) -> Optional[int]:
    """Device data pointer of a tensor argument (an int is passed through as a raw address and
    None as a null pointer). A tensor must be a dense CUDA tensor on the current device, of
    element type `dtype` (a torch dtype name) when given, holding at least `numel` elements:
    the library reads exactly the sizes it is given, so a smaller or differently typed tensor,
    or one on another GPU, would be read or written out of bounds."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if getattr(x, "is_cuda", True) is False:
        raise ValueError(f"{name} must be on a CUDA device")
    if hasattr(x, "is_contiguous") and not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and _dtype_name(x) != dtype:
        raise ValueError(f"{name} must be {dtype}, got {_dtype_name(x)}")
    if numel > 0 and x.numel() < numel:
        raise ValueError(f"{name} holds {x.numel()} elements; the sizes given need {numel}")
    dev = getattr(x, "device", None)
    if dev is not None and getattr(dev, "index", None) is not None:
        import torch
        cur = torch.cuda.current_device()
        if dev.index != cur:
            raise ValueError(f"{name} is on cuda:{dev.index} but the current device is cuda:{cur}")
    return int(x.data_ptr())


def _elem(dtype: int) -> Optional[str]:
    return _ELEM.get(int(dtype))


def _n(*xs) -> int:
    """Product of sizes, 0 if any is negative (the library then rejects the sizes itself)."""
    r = 1
    for x in xs:
        if int(x) < 0:
            return 0
        r *= int(x)
    return r


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _check(status: int, what: str) -> None:
    if status != ATTN_OK:
        raise AttnError(status, what)


def _fwd_sizes(B, Sq, Skv, Nq, Nkv, D, Dv, layout):
    """Element counts of q, k, v, out and one statistic array in attn_fwd's layouts."""
    if int(layout) == ATTN_TND:
        return _n(Sq, Nq, D), _n(Skv, Nkv, D), _n(Skv, Nkv, Dv), _n(Sq, Nq, Dv), _n(Sq, Nq)
    return (_n(B, Nq, Sq, D), _n(B, Nkv, Skv, D), _n(B, Nkv, Skv, Dv), _n(B, Nq, Sq, Dv),
            _n(B, Nq, Sq))


def _cu_ptr(cu, name: str, B: int):
    return _ptr(cu, name, _n(B), "int32")


def attn_fwd(q, k, v, *, cu_seqlens_q=None, cu_seqlens_kv=None, B: int, Sq: int, Skv: int,
             Nq: int, Nkv: int, D: int, scale: float, mask_mode: int, dtype: int, layout: int,
             out, softmax_max=None, softmax_sum=None, stream=None) -> None:
    """Fused attention forward (see ``attn_fwd`` in include/attn.h for layouts and limits)."""
    lib = load_library()
    nq, nk, nv, no, ns = _fwd_sizes(B, Sq, Skv, Nq, Nkv, D, D, layout)
    et = _elem(dtype)
    _check(lib.attn_fwd(_ptr(q, "q", nq, et), _ptr(k, "k", nk, et), _ptr(v, "v", nv, et),
                        _cu_ptr(cu_seqlens_q, "cu_seqlens_q", B), _cu_ptr(cu_seqlens_kv, "cu_seqlens_kv", B),
                        int(B), int(Sq), int(Skv), int(Nq), int(Nkv), int(D), float(scale),
                        int(mask_mode), int(dtype), int(layout), _ptr(out, "out", no, et),
                        _ptr(softmax_max, "softmax_max", ns, "float32"),
                        _ptr(softmax_sum, "softmax_sum", ns, "float32"), _stream(stream)), "attn_fwd")


def attn_fwd_accumulate(q, k, v, *, cu_seqlens_q=None, cu_seqlens_kv=None, B: int, Sq: int, Skv: int,
                        Nq: int, Nkv: int, D: int, scale: float, mask_mode: int, dtype: int,
                        layout: int, first: bool, acc_out, acc_max, acc_sum, stream=None) -> None:
    """attn_fwd over one chunk of keys, folded into a running accumulator in attn_merge's
    layouts (see ``attn_fwd_accumulate`` in include/attn.h)."""
    lib = load_library()
    nq, nk, nv, no, ns = _fwd_sizes(B, Sq, Skv, Nq, Nkv, D, D, layout)
    et = _elem(dtype)
    _check(lib.attn_fwd_accumulate(_ptr(q, "q", nq, et), _ptr(k, "k", nk, et), _ptr(v, "v", nv, et),
                                   _cu_ptr(cu_seqlens_q, "cu_seqlens_q", B),
                                   _cu_ptr(cu_seqlens_kv, "cu_seqlens_kv", B), int(B), int(Sq),
                                   int(Skv), int(Nq), int(Nkv), int(D), float(scale), int(mask_mode),
                                   int(dtype), int(layout), 1 if first else 0,
                                   _ptr(acc_out, "acc_out", no, et),
                                   _ptr(acc_max, "acc_max", 8 * ns, "float32"),
                                   _ptr(acc_sum, "acc_sum", 8 * ns, "float32"),
                                   _stream(stream)), "attn_fwd_accumulate")


def attn_fwd_masked(q, k, v, *, cu_seqlens_q=None, cu_seqlens_kv=None, B: int, Sq: int, Skv: int,
                    Nq: int, Nkv: int, Dqk: int, Dv: int, scale: float, mask_mode: int,
                    pre_tokens: int = 0, next_tokens: int = 0, atten_mask=None,
                    mask_batch_stride: int = 0, mask_row_stride: int = 0, dtype: int, layout: int,
                    out, softmax_max=None, softmax_sum=None, stream=None) -> None:
    """attn_fwd with a band, an optional uint8 mask (1 = excluded) and a value head size Dv
    (see ``attn_fwd_masked`` in include/attn.h)."""
    lib = load_library()
    nq, nk, nv, no, ns = _fwd_sizes(B, Sq, Skv, Nq, Nkv, Dqk, Dv, layout)
    et = _elem(dtype)
    nm = 0
    if int(layout) == ATTN_BHSD and _n(B, Sq, Skv) > 0:  # the last entry the mask is read at
        nm = max(0, (int(B) - 1) * int(mask_batch_stride) + (int(Sq) - 1) * int(mask_row_stride) + int(Skv))
    _check(lib.attn_fwd_masked(_ptr(q, "q", nq, et), _ptr(k, "k", nk, et), _ptr(v, "v", nv, et),
                               _cu_ptr(cu_seqlens_q, "cu_seqlens_q", B),
                               _cu_ptr(cu_seqlens_kv, "cu_seqlens_kv", B),
                               int(B), int(Sq), int(Skv), int(Nq), int(Nkv), int(Dqk), int(Dv),
                               float(scale), int(mask_mode), int(pre_tokens), int(next_tokens),
                               _ptr(atten_mask, "atten_mask", nm, "uint8"), int(mask_batch_stride),
                               int(mask_row_stride), int(dtype), int(layout), _ptr(out, "out", no, et),
                               _ptr(softmax_max, "softmax_max", ns, "float32"),
                               _ptr(softmax_sum, "softmax_sum", ns, "float32"), _stream(stream)),
           "attn_fwd_masked")


def attn_sparse_csr(q, k, v, csr_offset, csr_columns, *, B: int, H: int, S: int, D: int,
                    nnz_cap: int, out, stream=None) -> None:
    """CSR-sparse attention forward in float32 (see ``attn_sparse_csr`` in include/attn.h)."""
    lib = load_library()
    n = _n(B, H, S, D)
    _check(lib.attn_sparse_csr(_ptr(q, "q", n, "float32"), _ptr(k, "k", n, "float32"),
                               _ptr(v, "v", n, "float32"),
                               _ptr(csr_offset, "csr_offset", _n(B, H, int(S) + 1), "int32"),
                               _ptr(csr_columns, "csr_columns", _n(B, H, nnz_cap), "int32"),
                               int(B), int(H), int(S), int(D), int(nnz_cap), _ptr(out, "out", n, "float32"),
                               _stream(stream)), "attn_sparse_csr")


def attn_sparse_csr_tc(q, k, v, csr_offset, csr_columns, *, B: int, H: int, S: int, D: int,
                       nnz_cap: int, dtype: int, out, stream=None) -> None:
    """CSR-sparse attention forward in bf16/fp16 on the tensor cores (see
    ``attn_sparse_csr_tc`` in include/attn.h)."""
    lib = load_library()
    n = _n(B, H, S, D)
    et = _elem(dtype)
    _check(lib.attn_sparse_csr_tc(_ptr(q, "q", n, et), _ptr(k, "k", n, et), _ptr(v, "v", n, et),
                                  _ptr(csr_offset, "csr_offset", _n(B, H, int(S) + 1), "int32"),
                                  _ptr(csr_columns, "csr_columns", _n(B, H, nnz_cap), "int32"),
                                  int(B), int(H), int(S), int(D), int(nnz_cap), int(dtype),
                                  _ptr(out, "out", n, et), _stream(stream)), "attn_sparse_csr_tc")


def attn_csr_plan_size(*, B: int, H: int, S: int, nnz_cap: int) -> int:
    """Bytes of the plan of a CSR pattern of this shape (``attn_csr_plan_size`` in
    include/attn.h); allocate that many bytes (uint8, on the device) for attn_csr_plan."""
    lib = load_library()
    n = ctypes.c_int64(0)
    _check(lib.attn_csr_plan_size(int(B), int(H), int(S), int(nnz_cap), ctypes.byref(n)),
           "attn_csr_plan_size")
    return int(n.value)


def attn_csr_plan(csr_offset, csr_columns, *, B: int, H: int, S: int, nnz_cap: int, plan,
                  stream=None) -> None:
    """Build the plan of a CSR pattern into `plan` (a uint8 device tensor of at least
    attn_csr_plan_size bytes); see ``attn_csr_plan`` in include/attn.h."""
    lib = load_library()
    nb = attn_csr_plan_size(B=B, H=H, S=S, nnz_cap=nnz_cap)
    _check(lib.attn_csr_plan(_ptr(csr_offset, "csr_offset", _n(B, H, int(S) + 1), "int32"),
                             _ptr(csr_columns, "csr_columns", _n(B, H, nnz_cap), "int32"), int(B),
                             int(H), int(S), int(nnz_cap), _ptr(plan, "plan", nb, "uint8"),
                             int(plan.numel()) if plan is not None and not isinstance(plan, int) else nb,
                             _stream(stream)), "attn_csr_plan")


def attn_sparse_csr_tc_planned(q, k, v, plan, *, B: int, H: int, S: int, D: int, nnz_cap: int,
                               dtype: int, out, stream=None) -> None:
    """attn_sparse_csr_tc from a plan of the pattern (see ``attn_sparse_csr_tc_planned`` in
    include/attn.h)."""
    lib = load_library()
    n = _n(B, H, S, D)
    et = _elem(dtype)
    nb = attn_csr_plan_size(B=B, H=H, S=S, nnz_cap=nnz_cap)
    _check(lib.attn_sparse_csr_tc_planned(_ptr(q, "q", n, et), _ptr(k, "k", n, et), _ptr(v, "v", n, et),
                                          _ptr(plan, "plan", nb, "uint8"),
                                          int(plan.numel()) if plan is not None and not isinstance(plan, int) else nb,
                                          int(B), int(H), int(S), int(D), int(nnz_cap), int(dtype),
                                          _ptr(out, "out", n, et), _stream(stream)),
           "attn_sparse_csr_tc_planned")


def attn_sparse_csr_tc_noalloc(q, k, v, csr_offset, csr_columns, *, B: int, H: int, S: int, D: int,
                               nnz_cap: int, dtype: int, out, stream=None) -> None:
    """attn_sparse_csr_tc for callers that cannot allocate device memory: the library plans the
    pattern into its own fixed 48 MiB scratch array and runs the planned kernel (see
    ``attn_sparse_csr_tc_noalloc`` in include/attn.h; calls that overlap on the GPU race)."""
    lib = load_library()
    n = _n(B, H, S, D)
    et = _elem(dtype)
    _check(lib.attn_sparse_csr_tc_noalloc(_ptr(q, "q", n, et), _ptr(k, "k", n, et), _ptr(v, "v", n, et),
                                          _ptr(csr_offset, "csr_offset", _n(B, H, int(S) + 1), "int32"),
                                          _ptr(csr_columns, "csr_columns", _n(B, H, nnz_cap), "int32"),
                                          int(B), int(H), int(S), int(D), int(nnz_cap), int(dtype),
                                          _ptr(out, "out", n, et), _stream(stream)),
           "attn_sparse_csr_tc_noalloc")


def attn_merge(prev_out, prev_max, prev_sum, cur_out, cur_max, cur_sum, *, S: int, B: int, N: int,
               D: int, dtype: int, out, out_max, out_sum, layout: int = ATTN_BHSD,
               actual_seq_qlen=None, stream=None) -> None:
    """Merge two partial attention results (see ``attn_merge`` in include/attn.h)."""
    lib = load_library()
    et = _elem(dtype)
    if int(layout) == ATTN_TND:
        no, ns = _n(S, N, D), _n(S, N, 8)
    else:
        no, ns = _n(S, B, N, D), _n(B, N, S, 8)
    f = "float32"
    _check(lib.attn_merge(_ptr(prev_out, "prev_out", no, et), _ptr(prev_max, "prev_max", ns, f),
                          _ptr(prev_sum, "prev_sum", ns, f), _ptr(cur_out, "cur_out", no, et),
                          _ptr(cur_max, "cur_max", ns, f), _ptr(cur_sum, "cur_sum", ns, f), int(S),
                          int(B), int(N), int(D), int(dtype), int(layout),
                          _ptr(actual_seq_qlen, "actual_seq_qlen", _n(B), "int64"),
                          _ptr(out, "out", no, et), _ptr(out_max, "out_max", ns, f),
                          _ptr(out_sum, "out_sum", ns, f), _stream(stream)), "attn_merge")


# The serving calls are made once a layer and token, so what the binding adds to a call's latency
# counts: the checks of _ptr in the few attribute reads that a tensor in order needs, and _ptr itself,
# with its messages, for everything else.
_DEV = {}


def _tools():
    """What the fast checks need of torch: its tensor type, dtypes by code, device and raw stream getters."""
    import torch
    _DEV.update(tensor=torch.Tensor, elem={ATTN_BF16: torch.bfloat16, ATTN_F32: torch.float32, ATTN_F16: torch.float16},
                f32=torch.float32, i32=torch.int32, u8=torch.uint8, device=torch._C._cuda_getDevice,
                stream=torch._C._cuda_getCurrentRawStream)
    return _DEV


def _here() -> int:
    """The current CUDA device, or -1 where there is none (every tensor then goes through _ptr)."""
    try:
        return (_DEV or _tools())["device"]()
    except Exception:
        return -1


def _arg(x, name: str, numel: int, dt, dev: int) -> Optional[int]:
    """_ptr for a tensor that is expected to be in order: on device `dev`, dense, of torch dtype `dt`,
    with `numel` elements or more. (A tensor on the CPU is on device -1 too.)"""
    if (type(x) is _DEV["tensor"] and x.dtype is dt and x.get_device() == dev >= 0 and x.is_contiguous()
            and x.numel() >= numel):
        return x.data_ptr()
    return _ptr(x, name, max(numel, 0), str(dt).replace("torch.", "") if dt is not None else None)


def _plain(x):
    """A number of another library as one that ctypes takes."""
    if x is None or isinstance(x, (int, float)):
        return x
    return operator.index(x) if hasattr(x, "__index__") else float(x)


def _call(fn, *args) -> int:
    try:
        return fn(*args)
    except ctypes.ArgumentError:
        return fn(*[_plain(x) for x in args])


def _on(stream, dev: int) -> Optional[int]:
    """The stream to launch on, as _stream gives it."""
    if stream is None and dev >= 0:
        return _DEV["stream"](dev)
    return _stream(stream)


def attn_fwd_sinks(q, k, v, *, cu_seqlens_q=None, cu_seqlens_kv=None, B: int, Sq: int, Skv: int,
                   Nq: int, Nkv: int, D: int, scale: float, window_tokens: int, sink_tokens: int = 0,
                   dtype: int, layout: int, out, softmax_max=None, softmax_sum=None, stream=None) -> None:
    """attn_fwd through a sliding window of the newest keys and the first `sink_tokens` keys (see
    ``attn_fwd_sinks`` in include/attn.h)."""
    lib, dev = _lib or load_library(), _here()
    nq, nk, _, no, ns = _fwd_sizes(B, Sq, Skv, Nq, Nkv, D, D, layout)
    et, f32, i32 = _DEV["elem"].get(dtype), _DEV["f32"], _DEV["i32"]
    rc = _call(
        lib.attn_fwd_sinks,
        _arg(q, "q", nq, et, dev), _arg(k, "k", nk, et, dev), _arg(v, "v", nk, et, dev),
        None if cu_seqlens_q is None else _arg(cu_seqlens_q, "cu_seqlens_q", B, i32, dev),
        None if cu_seqlens_kv is None else _arg(cu_seqlens_kv, "cu_seqlens_kv", B, i32, dev), B, Sq, Skv, Nq, Nkv, D,
        scale, window_tokens, sink_tokens, dtype, layout, _arg(out, "out", no, et, dev),
        None if softmax_max is None else _arg(softmax_max, "softmax_max", ns, f32, dev),
        None if softmax_sum is None else _arg(softmax_sum, "softmax_sum", ns, f32, dev), _on(stream, dev))
    if rc:
        _check(rc, "attn_fwd_sinks")


def _pool(x, name: str, num_pages: int, page_elems: int, page_stride: int, dt, dev: int):
    """Device data pointer of a page pool. Its pages must be dense; the pool itself may be a view with
    gaps between the pages (one half of a [num_pages, 2, ...] tensor), whose distance must be
    `page_stride`."""
    stride = page_stride or page_elems
    if x is not None and not isinstance(x, int) and not x.is_contiguous():
        if x.dim() < 2 or not x[0].is_contiguous():
            raise ValueError(f"{name}: the elements of a page must be contiguous")
        if x.stride(0) != stride:
            raise ValueError(f"{name}: pages lie {x.stride(0)} elements apart, page_stride says {stride}")
        if x.shape[0] < num_pages or x[0].numel() < page_elems:
            raise ValueError(f"{name} holds {x.shape[0]} pages of {x[0].numel()} elements; the sizes given need "
                             f"{num_pages} of {page_elems}")
        return _arg(x[0], name, 0, dt, dev)
    return _arg(x, name, (num_pages - 1) * stride + page_elems if num_pages > 0 else 0, dt, dev)


def attn_decode_workspace_size(*, Nq: int, Nkv: int, D: int, dtype: int) -> int:
    """Bytes of the workspace of attn_decode_paged; allocate it with torch.zeros (uint8, on the device)."""
    lib = load_library()
    n = ctypes.c_int64(0)
    _check(lib.attn_decode_workspace_size(int(Nq), int(Nkv), int(D), int(dtype), ctypes.byref(n)),
           "attn_decode_workspace_size")
    return int(n.value)


def attn_decode_paged(q, k_cache, v_cache, page_table, seq_lens, *, B: int, Nq: int, Nkv: int, D: int,
                      num_pages: int, page_size: int, max_pages: int, page_stride: int = 0, scale: float,
                      window_tokens: int = ATTN_WINDOW_ALL, sink_tokens: int = 0, dtype: int, layout: int,
                      workspace, out, softmax_max=None, softmax_sum=None, stream=None) -> None:
    """Attention of one new token per row over a paged key/value cache (see ``attn_decode_paged`` in
    include/attn.h). `workspace` is a uint8 tensor of attn_decode_workspace_size bytes, zero-filled once."""
    lib, dev = _lib or load_library(), _here()
    et, f32, i32 = _DEV["elem"].get(dtype), _DEV["f32"], _DEV["i32"]
    nq, pe = B * Nq * D, page_size * Nkv * D
    ws = _arg(workspace, "workspace", 0, _DEV["u8"], dev)
    if workspace is None:
        ws_bytes = 0
    elif isinstance(workspace, int):
        ws_bytes = attn_decode_workspace_size(Nq=Nq, Nkv=Nkv, D=D, dtype=dtype)
    else:
        ws_bytes = workspace.numel()
    rc = _call(
        lib.attn_decode_paged,
        _arg(q, "q", nq, et, dev), _pool(k_cache, "k_cache", num_pages, pe, page_stride, et, dev),
        _pool(v_cache, "v_cache", num_pages, pe, page_stride, et, dev),
        _arg(page_table, "page_table", B * max_pages, i32, dev), _arg(seq_lens, "seq_lens", B, i32, dev), B, Nq, Nkv, D,
        num_pages, page_size, max_pages, page_stride, scale, window_tokens, sink_tokens, dtype, layout, ws, ws_bytes,
        _arg(out, "out", nq, et, dev),
        None if softmax_max is None else _arg(softmax_max, "softmax_max", B * Nq, f32, dev),
        None if softmax_sum is None else _arg(softmax_sum, "softmax_sum", B * Nq, f32, dev), _on(stream, dev))
    if rc:
        _check(rc, "attn_decode_paged")


def attn_cache_append(k, v, page_table, seq_lens, k_cache, v_cache, *, cu_seqlens=None, T: int, B: int,
                      Nkv: int, D: int, num_pages: int, page_size: int, max_pages: int, page_stride: int = 0,
                      dtype: int, layout: int, stream=None) -> None:
    """Write the keys and values of new tokens into a paged cache (see ``attn_cache_append`` in
    include/attn.h)."""
    lib, dev = _lib or load_library(), _here()
    et, i32 = _DEV["elem"].get(dtype), _DEV["i32"]
    nk, pe = T * Nkv * D, page_size * Nkv * D
    rc = _call(
        lib.attn_cache_append,
        _arg(k, "k", nk, et, dev), _arg(v, "v", nk, et, dev), _arg(page_table, "page_table", B * max_pages, i32, dev),
        _arg(seq_lens, "seq_lens", B, i32, dev),
        None if cu_seqlens is None else _arg(cu_seqlens, "cu_seqlens", B, i32, dev), T, B, Nkv, D, num_pages, page_size,
        max_pages, page_stride, dtype, layout, _pool(k_cache, "k_cache", num_pages, pe, page_stride, et, dev),
        _pool(v_cache, "v_cache", num_pages, pe, page_stride, et, dev), _on(stream, dev))
    if rc:
        _check(rc, "attn_cache_append")


def attn_cache_fork(page_table, src_rows, ref_count, page_table_out, ref_count_out, *, rows_in: int,
                    rows_out: int, max_pages: int, num_pages: int, seq_lens=None, seq_lens_out=None,
                    stream=None) -> None:
    """Rows of a page table take the pages of other rows: fork, reorder, free (see ``attn_cache_fork``
    in include/attn.h). The outputs may be the inputs."""
    lib, dev = _lib or load_library(), _here()
    i32 = _DEV["i32"]
    rc = _call(
        lib.attn_cache_fork,
        _arg(page_table, "page_table", rows_in * max_pages, i32, dev), _arg(src_rows, "src_rows", rows_out, i32, dev),
        _arg(ref_count, "ref_count", num_pages, i32, dev),
        None if seq_lens is None else _arg(seq_lens, "seq_lens", rows_in, i32, dev), rows_in, rows_out, max_pages,
        num_pages, _arg(page_table_out, "page_table_out", rows_out * max_pages, i32, dev),
        _arg(ref_count_out, "ref_count_out", num_pages, i32, dev),
        None if seq_lens_out is None else _arg(seq_lens_out, "seq_lens_out", rows_out, i32, dev), _on(stream, dev))
    if rc:
        _check(rc, "attn_cache_fork")


def attn_cache_reserve(page_table, ref_count, seq_lens, new_tokens, copies, *, B: int, max_pages: int,
                       num_pages: int, page_size: int, stream=None) -> None:
    """Give the rows pages of their own for their next tokens, in place (see ``attn_cache_reserve`` in
    include/attn.h). `new_tokens` may be None (one per row)."""
    lib, dev = _lib or load_library(), _here()
    i32 = _DEV["i32"]
    rc = _call(
        lib.attn_cache_reserve,
        _arg(page_table, "page_table", B * max_pages, i32, dev), _arg(ref_count, "ref_count", num_pages, i32, dev),
        _arg(seq_lens, "seq_lens", B, i32, dev),
        None if new_tokens is None else _arg(new_tokens, "new_tokens", B, i32, dev), B, max_pages, num_pages, page_size,
        _arg(copies, "copies", 2 * B, i32, dev), _on(stream, dev))
    if rc:
        _check(rc, "attn_cache_reserve")


def attn_cache_grow(page_table, ref_count, seq_lens, new_tokens, new_lens, copies, *, B: int, max_pages: int,
                    num_pages: int, page_size: int, live_only: bool = False, stream=None) -> None:
    """attn_cache_reserve that also adds the new tokens to the lengths, unless it is refused (see
    ``attn_cache_grow`` in include/attn.h). `new_tokens` may be None (one per row, or per row that is not empty)."""
    lib, dev = _lib or load_library(), _here()
    i32 = _DEV["i32"]
    rc = _call(
        lib.attn_cache_grow,
        _arg(page_table, "page_table", B * max_pages, i32, dev), _arg(ref_count, "ref_count", num_pages, i32, dev),
        _arg(seq_lens, "seq_lens", B, i32, dev),
        None if new_tokens is None else _arg(new_tokens, "new_tokens", B, i32, dev), int(live_only), B, max_pages,
        num_pages, page_size, _arg(copies, "copies", 2 * B, i32, dev), _arg(new_lens, "new_lens", B, i32, dev),
        _on(stream, dev))
    if rc:
        _check(rc, "attn_cache_grow")


def attn_cache_evict(page_table, ref_count, seq_lens, *, B: int, max_pages: int, num_pages: int, page_size: int,
                     window_tokens: int, sink_tokens: int = 0, stream=None) -> None:
    """Let go of pages that a window has left behind, in place (see ``attn_cache_evict`` in
    include/attn.h)."""
    lib, dev = _lib or load_library(), _here()
    i32 = _DEV["i32"]
    rc = _call(
        lib.attn_cache_evict,
        _arg(page_table, "page_table", B * max_pages, i32, dev), _arg(ref_count, "ref_count", num_pages, i32, dev),
        _arg(seq_lens, "seq_lens", B, i32, dev), B, max_pages, num_pages, page_size, window_tokens, sink_tokens,
        _on(stream, dev))
    if rc:
        _check(rc, "attn_cache_evict")


def attn_cache_compact(page_table, ref_count, page_table_out, ref_count_out, page_map, copies, live_pages, *,
                       rows: int, max_pages: int, num_pages: int, stream=None) -> None:
    """Plan the moves that bring all live pages to the front of the pool (see ``attn_cache_compact`` in
    include/attn.h). page_table_out and ref_count_out may be the inputs."""
    lib, dev = _lib or load_library(), _here()
    i32 = _DEV["i32"]
    rc = _call(
        lib.attn_cache_compact,
        _arg(page_table, "page_table", rows * max_pages, i32, dev), _arg(ref_count, "ref_count", num_pages, i32, dev),
        rows, max_pages, num_pages, _arg(page_table_out, "page_table_out", rows * max_pages, i32, dev),
        _arg(ref_count_out, "ref_count_out", num_pages, i32, dev), _arg(page_map, "page_map", num_pages, i32, dev),
        _arg(copies, "copies", 2 * (num_pages // 2), i32, dev), _arg(live_pages, "live_pages", 1, i32, dev),
        _on(stream, dev))
    if rc:
        _check(rc, "attn_cache_compact")


def attn_cache_copy(k_cache, v_cache, copies, *, n_copies: int, num_pages: int, page_elems: int,
                    page_stride: int = 0, dtype: int, stream=None) -> None:
    """Copy whole pages within a cache, as attn_cache_reserve and attn_cache_compact list them (see
    ``attn_cache_copy`` in include/attn.h)."""
    lib, dev = _lib or load_library(), _here()
    et = _DEV["elem"].get(dtype)
    rc = _call(
        lib.attn_cache_copy,
        _arg(copies, "copies", 2 * n_copies, _DEV["i32"], dev), n_copies, num_pages, page_elems,
        page_stride, dtype, _pool(k_cache, "k_cache", num_pages, page_elems, page_stride, et, dev),
        _pool(v_cache, "v_cache", num_pages, page_elems, page_stride, et, dev), _on(stream, dev))
    if rc:
        _check(rc, "attn_cache_copy")


def attn_get_last_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    lib = load_library()
    st = ctypes.c_int(0)
    _check(lib.attn_get_last_error(_stream(stream), ctypes.byref(st)), "attn_get_last_error")
    return int(st.value)
