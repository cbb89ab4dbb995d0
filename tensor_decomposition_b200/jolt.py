"""Python binding of the JoLT codec library (libjolt.so), argument marshalling only.

Every function has the name of the C entry point it calls (include/jolt.h). Tensors are
PyTorch CUDA tensors used as plain device memory; CUDA streams default to torch's current
stream. All computation happens in the library's CUDA kernels: if the library is missing
or fails to load, importing this module raises, there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libjolt.so")

JOLT_OK = 0
STATUS_NAMES = {0: "OK", 1: "INVALID_ARG", 2: "BUDGET_INFEASIBLE", 3: "OOM", 4: "CUDA",
                5: "NOT_CONVERGED", 6: "NONFINITE", 7: "TIMEOUT", 8: "CORRUPT_STREAM",
                9: "UNSUPPORTED"}
JOLT_BF16, JOLT_F32, JOLT_F16 = 0, 1, 2
JOLT_ENC_AUTO, JOLT_ENC_EXACT, JOLT_ENC_SKETCH = 0, 1, 2
JOLT_EIG_TRIDIAG, JOLT_EIG_JACOBI = 0, 1
JOLT_ROT_HAAR, JOLT_ROT_HADAMARD = 0, 1
JOLT_DBG_PI, JOLT_DBG_UT_F32, JOLT_DBG_UD_F32, JOLT_DBG_TABLE, JOLT_DBG_XX, JOLT_DBG_LAMBDA, \
    JOLT_DBG_OMEGA, JOLT_DBG_MEAS = range(8)
PART_NAMES = ("U_T", "U_D", "G", "scales", "codes")

EXPORTED = ["jolt_config_default", "jolt_plan", "jolt_plan_info", "jolt_encode", "jolt_decode",
            "jolt_rel_frob_error", "jolt_rel_frob_error_noalloc", "jolt_stream_status",
            "jolt_stream_info", "jolt_stream_to_host", "jolt_stream_from_host", "jolt_export_debug", "jolt_stream_destroy",
            "jolt_plan_destroy", "jolt_last_error", "jolt_profile_enable", "jolt_profile_report",
            "jolt_launch_count", "jolt_alloc_count", "jolt_selftest_gemm_bf16", "jolt_selftest_gemm_bf16_layout",
            "jolt_selftest_eig_dense", "jolt_selftest_eig_small", "jolt_attention", "jolt_attention_lse", "jolt_pages_create",
            "jolt_pages_status", "jolt_pages_destroy", "jolt_qk_norm_rope", "jolt_paged_append",
            "jolt_paged_attention"]


class JoltError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class Shape(ctypes.Structure):
    _fields_ = [("layers", ctypes.c_int32), ("heads", ctypes.c_int32), ("tokens", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("has_v", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class Config(ctypes.Structure):
    _fields_ = [("encoder", ctypes.c_int32), ("oversample", ctypes.c_int32),
                ("power_iters", ctypes.c_int32), ("rank_step", ctypes.c_int32),
                ("rt_max", ctypes.c_int32), ("bits_mask", ctypes.c_uint32),
                ("split_kv_budget", ctypes.c_int32), ("max_jacobi_sweeps", ctypes.c_int32),
                ("factors", ctypes.c_int32), ("measured_b", ctypes.c_int32), ("rotation", ctypes.c_int32),
                ("eig_solver", ctypes.c_int32)]


class PageShape(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int32), ("heads", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class BatchDesc(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("total_q", ctypes.c_int32), ("max_q", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m tensor_decomposition_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, u64, i32, st = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int32, ctypes.c_int
    i64, f32 = ctypes.c_int64, ctypes.c_float
    sig = {
        "jolt_config_default": (None, [ctypes.POINTER(Config)]),
        "jolt_plan": (st, [ctypes.POINTER(Shape), u64, i32, ctypes.POINTER(Config), ctypes.POINTER(vp)]),
        "jolt_plan_info": (st, [vp, ctypes.POINTER(i32), ctypes.POINTER(i32), ctypes.POINTER(i32),
                                ctypes.POINTER(u64)]),
        "jolt_encode": (st, [vp, vp, vp, u64, vp, ctypes.POINTER(vp)]),
        "jolt_decode": (st, [vp, vp, vp, vp]),
        "jolt_rel_frob_error": (st, [vp, vp, u64, i32, vp, ctypes.POINTER(ctypes.c_double)]),
        "jolt_rel_frob_error_noalloc": (st, [vp, vp, u64, i32, vp, ctypes.POINTER(ctypes.c_double)]),
        "jolt_stream_status": (st, [vp]),
        "jolt_stream_info": (st, [vp, ctypes.POINTER(u64), ctypes.POINTER(i32), ctypes.POINTER(ctypes.c_double)]),
        "jolt_stream_to_host": (st, [vp, vp, ctypes.POINTER(u64)]),
        "jolt_stream_from_host": (st, [vp, u64, vp, ctypes.POINTER(vp)]),
        "jolt_export_debug": (st, [vp, i32, i32, vp, ctypes.POINTER(u64)]),
        "jolt_stream_destroy": (None, [vp]),
        "jolt_plan_destroy": (None, [vp]),
        "jolt_last_error": (ctypes.c_char_p, []),
        "jolt_profile_enable": (st, [i32]),
        "jolt_profile_report": (st, [ctypes.c_char_p, ctypes.POINTER(u64)]),
        "jolt_launch_count": (u64, []),
        "jolt_alloc_count": (u64, []),
        "jolt_selftest_gemm_bf16": (st, [i32, i32, i32, vp, vp, vp, vp]),
        "jolt_selftest_gemm_bf16_layout": (st, [i32, i32, i32, vp, i32, vp, i32, vp, vp]),
        "jolt_selftest_eig_dense": (st, [i32, i32, i32, vp, vp, vp, vp]),
        "jolt_selftest_eig_small": (st, [i32, i32, vp, vp, vp, i32, vp]),
        "jolt_attention": (st, [vp, vp, i32, i32, ctypes.c_float, vp, vp]),
        "jolt_attention_lse": (st, [vp, i32, vp, i32, i32, ctypes.c_float, vp, vp, vp]),
        "jolt_pages_create": (st, [ctypes.POINTER(PageShape), vp, vp, vp, ctypes.POINTER(vp)]),
        "jolt_pages_status": (st, [vp, vp]),
        "jolt_pages_destroy": (None, [vp]),
        "jolt_qk_norm_rope": (st, [ctypes.c_char_p, vp]),
        "jolt_paged_append": (st, [vp, vp, ctypes.c_char_p, vp]),
        "jolt_paged_attention": (st, [vp, vp, ctypes.c_char_p, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_lib = _load()


def _check(status: int):
    if status != JOLT_OK:
        raise JoltError(status, _lib.jolt_last_error().decode())


def _stream_ptr(cuda_stream):
    if cuda_stream is None:   # the raw handle: making a torch Stream object takes 3 us
        import torch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if hasattr(cuda_stream, "cuda_stream"):
        return ctypes.c_void_p(cuda_stream.cuda_stream)
    return ctypes.c_void_p(int(cuda_stream))


def _dptr(t, dtype=None):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("expected a contiguous CUDA tensor")
    return ctypes.c_void_p(t.data_ptr())


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return JOLT_BF16
    if t.dtype == torch.float32:
        return JOLT_F32
    raise ValueError(f"unsupported dtype {t.dtype}")


def jolt_config_default() -> Config:
    c = Config()
    _lib.jolt_config_default(ctypes.byref(c))
    return c


class Plan:
    def __init__(self, handle, shape: Shape, budget: int, groups: int, cfg: Config):
        self.handle, self.shape, self.budget, self.groups, self.cfg = handle, shape, budget, groups, cfg

    def __del__(self):
        if getattr(self, "handle", None):
            _lib.jolt_plan_destroy(self.handle)
            self.handle = None


class Stream:
    def __init__(self, handle, plan=None, keep=(), layers=None):
        self.handle, self.plan, self._keep = handle, plan, keep
        self.layers = plan.shape.layers if plan is not None else layers

    def __del__(self):
        if getattr(self, "handle", None):
            _lib.jolt_stream_destroy(self.handle)
            self.handle = None


def jolt_plan(layers, heads, tokens, head_dim, has_v, dtype, byte_budget, num_groups, config=None) -> Plan:
    sh = Shape(layers, heads, tokens, head_dim, int(bool(has_v)), dtype)
    cfg = config if config is not None else jolt_config_default()
    h = ctypes.c_void_p()
    _check(_lib.jolt_plan(ctypes.byref(sh), int(byte_budget), int(num_groups), ctypes.byref(cfg), ctypes.byref(h)))
    return Plan(h, sh, int(byte_budget), int(num_groups), cfg)


def jolt_plan_info(plan: Plan) -> dict:
    r, l, e = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    w = ctypes.c_uint64()
    _check(_lib.jolt_plan_info(plan.handle, ctypes.byref(r), ctypes.byref(l), ctypes.byref(e), ctypes.byref(w)))
    return dict(rt_max=r.value, sketch_l=l.value, encoder=e.value, workspace_bytes=w.value)


def jolt_encode(plan: Plan, K, V, seed: int, cuda_stream=None) -> Stream:
    h = ctypes.c_void_p()
    _check(_lib.jolt_encode(plan.handle, _dptr(K), _dptr(V), int(seed) & (2 ** 64 - 1),
                            _stream_ptr(cuda_stream), ctypes.byref(h)))
    return Stream(h, plan)


def jolt_decode(stream: Stream, K_out, V_out=None, cuda_stream=None):
    _check(_lib.jolt_decode(stream.handle, _dptr(K_out), _dptr(V_out), _stream_ptr(cuda_stream)))


def jolt_rel_frob_error(ref, approx, cuda_stream=None) -> float:
    if ref.shape != approx.shape or ref.dtype != approx.dtype:
        raise ValueError("ref and approx must share shape and dtype")
    out = ctypes.c_double()
    _check(_lib.jolt_rel_frob_error(_dptr(ref), _dptr(approx), ref.numel(), _dtype_code(ref),
                                    _stream_ptr(cuda_stream), ctypes.byref(out)))
    return out.value


def jolt_rel_frob_error_noalloc(ref, approx, cuda_stream=None) -> float:
    if ref.shape != approx.shape or ref.dtype != approx.dtype:
        raise ValueError("ref and approx must share shape and dtype")
    out = ctypes.c_double()
    _check(_lib.jolt_rel_frob_error_noalloc(_dptr(ref), _dptr(approx), ref.numel(), _dtype_code(ref),
                                            _stream_ptr(cuda_stream), ctypes.byref(out)))
    return out.value


def jolt_stream_status(stream: Stream):
    _check(_lib.jolt_stream_status(stream.handle))


def jolt_stream_info(stream: Stream, groups: int) -> dict:
    bp = (ctypes.c_uint64 * 5)()
    al = (ctypes.c_int32 * (groups * 6))()
    lam = (ctypes.c_double * 2)()
    _check(_lib.jolt_stream_info(stream.handle, bp, al, lam))
    return dict(bytes_by_part=dict(zip(PART_NAMES, list(bp))),
                alloc=np.array(list(al), dtype=np.int64).reshape(groups, 2, 3), lambdas=list(lam))


def jolt_stream_to_host(stream: Stream) -> bytes:
    n = ctypes.c_uint64()
    _check(_lib.jolt_stream_to_host(stream.handle, None, ctypes.byref(n)))
    buf = ctypes.create_string_buffer(n.value)
    _check(_lib.jolt_stream_to_host(stream.handle, buf, ctypes.byref(n)))
    return buf.raw[: n.value]


def jolt_stream_from_host(data: bytes, cuda_stream=None) -> Stream:
    h = ctypes.c_void_p()
    buf = ctypes.create_string_buffer(data, len(data))
    _check(_lib.jolt_stream_from_host(buf, len(data), _stream_ptr(cuda_stream), ctypes.byref(h)))
    return Stream(h, layers=struct.unpack_from("<i", data, 16)[0])   # of the header that was just checked


def jolt_export_debug(stream: Stream, what: int, lt: int = 0) -> np.ndarray:
    n = ctypes.c_uint64()
    _check(_lib.jolt_export_debug(stream.handle, what, lt, None, ctypes.byref(n)))
    buf = ctypes.create_string_buffer(n.value)
    _check(_lib.jolt_export_debug(stream.handle, what, lt, buf, ctypes.byref(n)))
    raw = buf.raw[: n.value]
    if what in (JOLT_DBG_PI, JOLT_DBG_UT_F32, JOLT_DBG_UD_F32):
        return np.frombuffer(raw, dtype=np.float32).copy()
    if what == JOLT_DBG_OMEGA:
        return np.frombuffer(raw, dtype=np.uint16).copy()
    return np.frombuffer(raw, dtype=np.float64).copy()


def jolt_profile_enable(on: bool = True):
    _check(_lib.jolt_profile_enable(1 if on else 0))


def jolt_profile_report() -> dict:
    import json
    n = ctypes.c_uint64()
    _check(_lib.jolt_profile_report(None, ctypes.byref(n)))
    buf = ctypes.create_string_buffer(n.value)
    _check(_lib.jolt_profile_report(buf, ctypes.byref(n)))
    return json.loads(buf.value.decode())


def jolt_launch_count() -> int:
    return int(_lib.jolt_launch_count())


def jolt_alloc_count() -> int:
    return int(_lib.jolt_alloc_count())


def jolt_selftest_gemm_bf16(A, B, C, cuda_stream=None):
    """C = A B^T on the tensor cores; A [M][K], B [N][K] bf16, C [M][N] float32 (CUDA tensors)."""
    M, K = A.shape
    N = B.shape[0]
    _check(_lib.jolt_selftest_gemm_bf16(M, N, K, _dptr(A), _dptr(B), _dptr(C), _stream_ptr(cuda_stream)))


def jolt_selftest_gemm_bf16_layout(A, a_mn, B, b_mn, C, cuda_stream=None):
    """C = A B^T on the tensor cores with either operand stored transposed: A is [M][K] (a_mn
    false) or [K][M] (a_mn true), B is [N][K] or [K][N]; C [M][N] float32 (CUDA tensors)."""
    M, K = (A.shape[1], A.shape[0]) if a_mn else A.shape
    N = B.shape[1] if b_mn else B.shape[0]
    _check(_lib.jolt_selftest_gemm_bf16_layout(M, N, K, _dptr(A), int(bool(a_mn)), _dptr(B), int(bool(b_mn)),
                                               _dptr(C), _stream_ptr(cuda_stream)))


def jolt_selftest_eig_small(A, V, lam, solver=0, cuda_stream=None):
    """A: [batch][n][n] float64 CUDA tensor; V: [batch][n][n] and lam: [batch][n] float32 outputs."""
    _check(_lib.jolt_selftest_eig_small(int(A.shape[0]), int(A.shape[1]), _dptr(A), _dptr(V), _dptr(lam),
                                        int(solver), _stream_ptr(cuda_stream)))


def jolt_selftest_eig_dense(A, R, V, lam, cuda_stream=None):
    """A: [batch][n][n] float64 CUDA tensor; V: [batch][n][R] and lam: [batch][R] float64 outputs."""
    _check(_lib.jolt_selftest_eig_dense(int(A.shape[0]), int(A.shape[1]), int(R), _dptr(A), _dptr(V), _dptr(lam),
                                        _stream_ptr(cuda_stream)))


def _attention_tensors(Q, out, lse=None):
    """Bf16 queries and float32 results, rows of 128, on the current device: the library reads and writes them as
    these whatever they are."""
    import torch
    _here(Q.get_device(), torch)
    if Q.shape[-1] != 128:
        raise ValueError("the rows of Q must have 128 features")
    _array(Q, "Q", Q.shape, torch.bfloat16, Q.get_device())
    _array(out, "out", Q.shape, torch.float32, Q.get_device())
    _array(lse, "lse", Q.shape[:2], torch.float32, Q.get_device())


def jolt_attention(stream: Stream, Q, out, scale: float, cuda_stream=None):
    """Q: bf16 CUDA tensor [layers][q_heads][n][head_dim]; out: float32 CUDA tensor of the same shape."""
    if Q.dim() != 4 or tuple(out.shape) != tuple(Q.shape) or stream.layers not in (None, Q.shape[0]):
        raise ValueError("Q and out must be [layers][q_heads][n][head_dim] of the same shape")
    _attention_tensors(Q, out)
    _check(_lib.jolt_attention(stream.handle, _dptr(Q), int(Q.shape[1]), int(Q.shape[2]), float(scale), _dptr(out),
                               _stream_ptr(cuda_stream)))


def jolt_attention_lse(stream: Stream, layer: int, Q, out, lse, scale: float, cuda_stream=None):
    """Q: bf16 CUDA tensor [n][q_heads][head_dim] of one layer; out: float32, same shape; lse: float32 [n][q_heads].
    (The queries of fp16 pages have to be rounded to bf16 for it.)"""
    if Q.dim() != 3 or tuple(out.shape) != tuple(Q.shape) or tuple(lse.shape) != tuple(Q.shape[:2]):
        raise ValueError("Q and out must be [n][q_heads][head_dim] of the same shape and lse [n][q_heads]")
    _attention_tensors(Q, out, lse)
    _check(_lib.jolt_attention_lse(stream.handle, int(layer), _dptr(Q), int(Q.shape[1]), int(Q.shape[0]), float(scale),
                                   _dptr(out), _dptr(lse), _stream_ptr(cuda_stream)))


# ------------------------------------------------------------------ the growing cache
class Pages:
    """A page set (jolt_pages_create): keeps the page tensors alive. To be dropped after its calls have finished: what
    they report goes to the set that has its place then."""

    def __init__(self, handle, K_pages, V_pages):
        self.handle, self.K, self.V = handle.value, K_pages, V_pages
        self.heads, self.dtype, self.device = int(K_pages.shape[1]), K_pages.dtype, K_pages.get_device()

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:   # None while the interpreter shuts down
            _lib.jolt_pages_destroy(self.handle)
            self.handle = None


class Batch:
    """A batch description (jolt_batch): keeps its device arrays alive. Their contents may change
    between calls, their places may not."""

    def __init__(self, desc, keep):
        self.desc, self._keep = desc, keep
        self.ptr = ctypes.addressof(desc)
        self.total_q, self.device = desc.total_q, keep[0].get_device()


# The argument structs, packed: an argument a field through ctypes took 0.15 us each, a third of a small call.
_NORM_ROPE = struct.Struct("@PqqPPqqPqqPPqqPPiiiiiif")     # jolt_norm_rope
_NEW_ROWS = struct.Struct("@PqqPqqPPPiif")                 # jolt_new_rows
_QUERIES = struct.Struct("@PqqPPPPiif")                    # jolt_queries


def _row_dtype(t, torch):
    if t.dtype == torch.bfloat16:
        return JOLT_BF16
    if t.dtype == torch.float16:
        return JOLT_F16
    raise ValueError(f"unsupported dtype {t.dtype} (bf16 or f16)")


def _here(device, torch):
    """The tensors' device has to be the current one, as for every entry point."""
    if device < 0 or device != torch.cuda.current_device():
        raise ValueError(f"tensors are on device {device}, the current device is {torch.cuda.current_device()}")


def _raw_stream(cuda_stream, device, torch):
    return torch._C._cuda_getCurrentRawStream(device) if cuda_stream is None else _stream_ptr(cuda_stream)


def _rows(t, name, tokens, heads, dtype, device):
    """(pointer, token stride, head stride) of a [tokens][heads][128] tensor with contiguous rows."""
    if t.shape != (tokens, heads, 128) or t.dtype != dtype or t.get_device() != device:
        raise ValueError(f"{name} must be a CUDA tensor [{tokens}][{heads}][128] {dtype} on device {device}, "
                         f"got {tuple(t.shape)} {t.dtype} on {t.device}")
    ts, hs, one = t.stride()
    if one != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.data_ptr(), ts if tokens > 1 else 0, hs if heads > 1 else 0


def _array(t, name, shape, dtype, device):
    """Pointer of a contiguous array of the shape; 0 for None."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype != dtype or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor {list(shape)} on device {device}")
    return t.data_ptr()


def _rope(positions, inv_freq, tokens, device, torch):
    """(positions pointer, inv_freq pointer, rope_dim)."""
    if inv_freq is None:
        return 0, 0, 0
    n = inv_freq.shape[0]
    return (_array(positions, "positions", (tokens,), torch.int32, device),
            _array(inv_freq, "inv_freq", (n,), torch.float32, device), 2 * n)


def jolt_pages_create(K_pages, V_pages, cuda_stream=None) -> Pages:
    """K_pages, V_pages: contiguous bf16 or f16 CUDA tensors [num_pages][heads][page_size][128]."""
    if K_pages.dim() != 4 or V_pages.shape != K_pages.shape or V_pages.dtype != K_pages.dtype:
        raise ValueError("K_pages and V_pages must be [num_pages][heads][page_size][head_dim] of the same shape and type")
    import torch
    k, v = _dptr(K_pages), _dptr(V_pages)
    _here(K_pages.get_device(), torch)
    if V_pages.get_device() != K_pages.get_device():
        raise ValueError("K_pages and V_pages must be on one device")
    sh = PageShape(*K_pages.shape, _row_dtype(K_pages, torch))
    h = ctypes.c_void_p()
    _check(_lib.jolt_pages_create(ctypes.byref(sh), k, v, _stream_ptr(cuda_stream), ctypes.byref(h)))
    return Pages(h, K_pages, V_pages)


def jolt_pages_status(pages: Pages, cuda_stream=None):
    _check(_lib.jolt_pages_status(pages.handle, _stream_ptr(cuda_stream)))


def jolt_batch(q_start, kv_len, page_table, total_q: int, max_q: int) -> Batch:
    """q_start [num_seqs + 1], kv_len [num_seqs], page_table [num_seqs][max_pages]: int32 CUDA tensors.
    total_q: rows of the batch's tensors; max_q: the longest chunk that may occur."""
    import torch
    n, dev = int(kv_len.numel()), kv_len.get_device()
    if kv_len.dim() != 1 or page_table.dim() != 2 or dev < 0:
        raise ValueError("kv_len must be a CUDA tensor [num_seqs] and page_table [num_seqs][max_pages]")
    d = BatchDesc(n, int(total_q), int(max_q), int(page_table.shape[1]),
                  _array(q_start, "q_start", (n + 1,), torch.int32, dev),
                  _array(kv_len, "kv_len", (n,), torch.int32, dev),
                  _array(page_table, "page_table", (n, page_table.shape[1]), torch.int32, dev))
    return Batch(d, (q_start, kv_len, page_table))


def jolt_qk_norm_rope(Q, Q_out, K=None, K_out=None, positions=None, inv_freq=None, q_weight=None, k_weight=None,
                      eps=1e-6, interleaved=False, cuda_stream=None):
    """Q, Q_out: [tokens][q_heads][128], K, K_out: [tokens][k_heads][128] (bf16 or f16 CUDA tensors with
    contiguous rows, any token and head strides that are multiples of 8); an output may be its input."""
    import torch
    if Q.dim() != 3:
        raise ValueError("Q must be [tokens][q_heads][128]")
    if inv_freq is not None and positions is None:
        raise ValueError("inv_freq without positions")
    if (K is None) != (K_out is None):
        raise ValueError("K and K_out come together")
    t, dev, (n, hq, _) = Q.dtype, Q.get_device(), Q.shape
    _here(dev, torch)
    dt = _row_dtype(Q, torch)
    q, qo = _rows(Q, "Q", n, hq, t, dev), _rows(Q_out, "Q_out", n, hq, t, dev)
    hk, k, ko = 0, (0, 0, 0), (0, 0, 0)
    if K is not None:
        hk = K.shape[1]
        k, ko = _rows(K, "K", n, hk, t, dev), _rows(K_out, "K_out", n, hk, t, dev)
    pos, fr, rd = _rope(positions, inv_freq, n, dev, torch)
    st = _lib.jolt_qk_norm_rope(
        _NORM_ROPE.pack(*q, _array(q_weight, "q_weight", (128,), t, dev), *qo, *k,
                        _array(k_weight, "k_weight", (128,), t, dev), *ko, pos, fr, dt, n, hq, hk, rd,
                        1 if interleaved else 0, eps), _raw_stream(cuda_stream, dev, torch))
    if st:
        _check(st)


def jolt_paged_append(pages: Pages, batch: Batch, K, V, positions=None, inv_freq=None, k_weight=None, eps=1e-6,
                      interleaved=False, cuda_stream=None):
    """K, V: [total_q][heads][128] of the pages' type, contiguous rows, strides multiples of 8."""
    import torch
    n, h, t, dev = batch.total_q, pages.heads, pages.dtype, pages.device
    _here(dev, torch)
    if batch.device != dev:
        raise ValueError("the batch's arrays must be on the pages' device")
    pos, fr, rd = _rope(positions, inv_freq, n, dev, torch)
    st = _lib.jolt_paged_append(
        pages.handle, batch.ptr,
        _NEW_ROWS.pack(*_rows(K, "K", n, h, t, dev), *_rows(V, "V", n, h, t, dev),
                       _array(k_weight, "k_weight", (128,), t, dev), pos, fr, rd, 1 if interleaved else 0, eps),
        _raw_stream(cuda_stream, dev, torch))
    if st:
        _check(st)


def jolt_paged_attention(pages: Pages, batch: Batch, Q, out, scale: float, causal=True, lse=None, prefix_out=None,
                         prefix_lse=None, cuda_stream=None):
    """Q: [total_q][q_heads][128] of the pages' type with contiguous rows; out: contiguous, same shape and
    type; lse, prefix_lse: float32 [total_q][q_heads]; prefix_out: float32 [total_q][q_heads][128]."""
    import torch
    n, t, dev = batch.total_q, pages.dtype, pages.device
    if Q.dim() != 3:
        raise ValueError("Q must be [total_q][q_heads][128]")
    _here(dev, torch)
    if batch.device != dev:
        raise ValueError("the batch's arrays must be on the pages' device")
    hq, f32 = Q.shape[1], torch.float32
    st = _lib.jolt_paged_attention(
        pages.handle, batch.ptr,
        _QUERIES.pack(*_rows(Q, "Q", n, hq, t, dev), _array(prefix_out, "prefix_out", (n, hq, 128), f32, dev),
                      _array(prefix_lse, "prefix_lse", (n, hq), f32, dev), _array(out, "out", (n, hq, 128), t, dev),
                      _array(lse, "lse", (n, hq), f32, dev), hq, 1 if causal else 0, scale),
        _raw_stream(cuda_stream, dev, torch))
    if st:
        _check(st)
