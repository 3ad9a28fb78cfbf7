"""MI355X-native dense projection Y = X . W^T (+ bias) (-> GELU tanh).

A thin ctypes binding over ``libproj.so`` (C ABI declared in
``include/proj.h``).  Every step of the projection runs in the library's HIP
kernels; this module only turns torch tensors and streams into pointers and
sizes, and status codes into exceptions.  PyTorch provides device memory and
streams.  There is no fallback: if the library is not built, importing the
binding's entry points raises.

Names mirror the C ABI: ``proj_create``, ``proj_run``, ``proj_destroy``,
``proj_tune``, ``proj_get_plan``, ``proj_num_candidates``,
``proj_candidate_name``, ``proj_run_candidate``, ``proj_graph_capture``,
``proj_graph_launch``, ``proj_graph_destroy``, ``proj_status_string``, and
for fp32 weights held as a bf16 high/low pair ``proj_prepare_hilo``,
``proj_run_hilo``, ``proj_get_plan_hilo``, ``proj_num_candidates_hilo``,
``proj_candidate_name_hilo``, ``proj_run_candidate_hilo``, and for bf16
weights registered in the packed tile layout ``proj_packed_bytes``,
``proj_pack_weights``, ``proj_run_packed``, ``proj_get_plan_packed``,
``proj_num_candidates_packed``, ``proj_candidate_name_packed``,
``proj_run_candidate_packed``, the measured read floor
``proj_read_probe``, and ``proj_run_noalloc`` (proj_run with no device
allocation); for 4-bit weights with group scales ``proj_pack_codes``,
``proj_quantize_weights``, ``proj_run_quant``; and for the paged key-value
cache between a decoding step's projections ``proj_kv_append`` (with norms of
the query and key heads ``proj_kv_append_norm``) and ``proj_kv_attend`` (for a
batch behind one prefix ``proj_kv_attend_shared``) on a cache described once by
``kv_cache``; for 8-bit integers with a scale for each token and output
``proj_quantize_rows``, ``proj_run_int`` and, from bf16 tokens,
``proj_run_int_dynamic``.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libproj.so")

PROJ_OK = 0
PROJ_ERR_INVALID_ARG = 1
PROJ_ERR_UNSUPPORTED = 2
PROJ_ERR_HIP = 3
PROJ_ERR_NO_MEMORY = 4
PROJ_ERR_NOT_TUNED = 5
PROJ_ERR_DESTROYED = 6

EPI_NONE, EPI_BIAS, EPI_GELU_TANH, EPI_BIAS_GELU_TANH = 0, 1, 2, 3
OUT_F32, OUT_BF16 = 0, 1
KV_BF16, KV_FP8 = 0, 1

EXPORTS = ["proj_create", "proj_run", "proj_tune", "proj_destroy", "proj_status_string",
           "proj_last_error", "proj_get_plan", "proj_num_candidates", "proj_candidate_name",
           "proj_run_candidate", "proj_graph_capture", "proj_graph_launch", "proj_graph_destroy",
           "proj_prepare_hilo", "proj_run_hilo", "proj_get_plan_hilo", "proj_num_candidates_hilo",
           "proj_candidate_name_hilo", "proj_run_candidate_hilo", "proj_packed_bytes", "proj_pack_weights",
           "proj_run_packed", "proj_get_plan_packed", "proj_num_candidates_packed", "proj_candidate_name_packed",
           "proj_run_candidate_packed", "proj_read_probe", "proj_run_noalloc",
           "proj_pack_codes", "proj_quantize_weights", "proj_run_quant", "proj_kv_append", "proj_kv_attend",
           "proj_quantize_rows", "proj_run_int", "proj_run_int_dynamic", "proj_kv_append_norm", "proj_kv_attend_shared"]


class ProjError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s (status %d)%s" % (_status_text(status), status,
                                               ": " + message if message else ""))
        self.status = status


class _KvCache(ctypes.Structure):
    """proj_kv_cache of include/proj.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("pages", ctypes.c_int64),
                ("k_strides", ctypes.c_int64 * 3), ("v_strides", ctypes.c_int64 * 3), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libproj.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libproj.so is not built: run `python -m dense_linear_projection_amd._build` "
                           "(or __graft_entry__.build())")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, ci, st = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int
    run_args = [vp, vp, vp, vp, ci, i64, i64, i64, vp, ci, vp]
    sig = {
        "proj_create": ([ctypes.POINTER(vp), ci, ctypes.c_size_t], st),
        "proj_run": (run_args, st),
        "proj_tune": (run_args, st),
        "proj_destroy": ([vp], st),
        "proj_status_string": ([ci], ctypes.c_char_p),
        "proj_last_error": ([vp], ctypes.c_char_p),
        "proj_get_plan": ([vp, i64, i64, i64, ci, ci, ci, ctypes.c_char_p, ctypes.c_size_t], st),
        "proj_num_candidates": ([i64, i64, i64, ci, ci, ci], ci),
        "proj_candidate_name": ([i64, i64, i64, ci, ci, ci, ci, ctypes.c_char_p, ctypes.c_size_t], st),
        "proj_run_candidate": ([vp, ci, vp, vp, vp, ci, i64, i64, i64, vp, ci, vp], st),
        "proj_graph_capture": ([vp, ci, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp),
                                ctypes.POINTER(vp), ci, i64, i64, i64, ci, vp, ctypes.POINTER(vp)], st),
        "proj_graph_launch": ([vp, vp], st),
        "proj_graph_destroy": ([vp], st),
        "proj_prepare_hilo": ([vp, vp, i64, i64, vp, vp], st),
        "proj_run_hilo": (run_args, st),
        "proj_get_plan_hilo": ([vp, i64, i64, i64, ci, ci, ci, ctypes.c_char_p, ctypes.c_size_t], st),
        "proj_num_candidates_hilo": ([i64, i64, i64, ci, ci, ci], ci),
        "proj_candidate_name_hilo": ([i64, i64, i64, ci, ci, ci, ci, ctypes.c_char_p, ctypes.c_size_t], st),
        "proj_run_candidate_hilo": ([vp, ci, vp, vp, vp, ci, i64, i64, i64, vp, ci, vp], st),
        "proj_packed_bytes": ([i64, i64, ci], i64),
        "proj_pack_weights": ([vp, vp, i64, i64, ci, vp, vp], st),
        "proj_run_packed": ([vp, vp, vp, ci, vp, ci, i64, i64, i64, vp, ci, vp], st),
        "proj_get_plan_packed": ([vp, i64, i64, i64, ci, ci, ci, ci, ctypes.c_char_p, ctypes.c_size_t], st),
        "proj_num_candidates_packed": ([i64, i64, i64, ci, ci, ci, ci], ci),
        "proj_candidate_name_packed": ([i64, i64, i64, ci, ci, ci, ci, ci, ctypes.c_char_p, ctypes.c_size_t], st),
        "proj_run_candidate_packed": ([vp, ci, vp, vp, ci, vp, ci, i64, i64, i64, vp, ci, vp], st),
        "proj_read_probe": ([vp, vp, ctypes.c_size_t, vp], st),
        "proj_run_noalloc": (run_args, st),
        "proj_pack_codes": ([vp, vp, i64, i64, vp, vp], st),
        "proj_quantize_weights": ([vp, vp, i64, i64, ci, vp, vp, ci, vp, vp], st),
        "proj_run_quant": ([vp, vp, vp, vp, ci, vp, ci, vp, ci, i64, i64, i64, vp, ci, vp], st),
        "proj_kv_append": ([vp, vp, vp, i64, i64, ci, vp, i64, ci, ci, vp, vp, vp, vp], st),
        "proj_kv_attend": ([vp, vp, vp, i64, i64, ci, vp, i64, i64, vp, i64, i64, ctypes.c_float, vp, ci, vp, vp], st),
        "proj_quantize_rows": ([vp, vp, i64, i64, i64, vp, i64, vp, vp], st),
        "proj_run_int": ([vp, vp, vp, vp, vp, vp, ci, i64, i64, i64, vp, ci, vp], st),
        "proj_run_int_dynamic": ([vp, vp, i64, vp, vp, vp, ci, i64, i64, i64, vp, ci, vp], st),
        "proj_kv_append_norm": ([vp, vp, vp, i64, i64, ci, vp, vp, ci, ci, ctypes.c_float, vp, i64, ci, ci, vp, vp, vp, vp], st),
        "proj_kv_attend_shared": ([vp, vp, vp, i64, i64, ci, vp, i64, vp, i64, i64, vp, i64, i64, ctypes.c_float, vp, ci, vp,
                                   vp], st),
    }
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes, f.restype = args, res
    _lib = L
    return L


def _status_text(s: int) -> str:
    try:
        return lib().proj_status_string(int(s)).decode()
    except Exception:  # library not loadable: still describe the code
        return "status"


def _check(status: int, ctx=None) -> None:
    if status != PROJ_OK:
        msg = ""
        if ctx is not None:
            try:
                msg = lib().proj_last_error(ctx).decode()
            except Exception:
                msg = ""
        raise ProjError(status, msg)


# ------------------------------------------------------------- marshalling

def _ptr(t):
    """Device pointer of a tensor (or an int address, or None)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensor must be on a GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous (row-major)")
    return t.data_ptr()


_raw_stream = None  # device index -> current stream's handle


def _stream(stream):
    if stream is None:
        # the handle alone: building torch's stream object costs 2.7 us, most of a small call's checks
        global _raw_stream
        if _raw_stream is None:
            import torch
            get, dev = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
            _raw_stream = (lambda: get(dev())) if get and dev else lambda: torch.cuda.current_stream().cuda_stream
        return _raw_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _out_dtype(Y, out_dtype):
    if out_dtype is not None:
        return int(out_dtype)
    import torch
    if Y.dtype == torch.float32:
        return OUT_F32
    if Y.dtype == torch.bfloat16:
        return OUT_BF16
    raise ValueError("Y must be float32 or bfloat16")


def _check_operands(X, W, bias, Y):
    import torch
    for name, t in (("X", X), ("W", W), ("bias", bias)):
        if t is not None and not isinstance(t, int) and t.dtype != torch.bfloat16:
            raise ValueError("%s must be bfloat16" % name)
    if Y is not None and not isinstance(Y, int) and Y.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("Y must be float32 or bfloat16")


# ------------------------------------------------------------------ the ABI

DEFAULT_WORKSPACE_BYTES = 64 << 20


def proj_create(device: int = 0, max_workspace_bytes: int = DEFAULT_WORKSPACE_BYTES) -> int:
    """Create a context on `device` whose split-K workspace is
    max_workspace_bytes (plans whose fp32 partials need more are not used)."""
    h = ctypes.c_void_p()
    _check(lib().proj_create(ctypes.byref(h), int(device), int(max_workspace_bytes)))
    return h.value


def proj_destroy(ctx: int) -> None:
    _check(lib().proj_destroy(ctx))


def proj_status_string(status: int) -> str:
    return lib().proj_status_string(int(status)).decode()


def _shape(X, W, M, N, K):
    if M is None:
        M = X.shape[0]
    if N is None:
        N = W.shape[0]
    if K is None:
        K = X.shape[1] if X.dim() == 2 else 0
    return int(M), int(N), int(K)


def proj_run(ctx, X, W, bias, epilogue, Y, M=None, N=None, K=None, out_dtype=None, stream=None) -> None:
    """Enqueue Y = epilogue(X . W^T [+ bias]) on `stream` (default: torch's
    current stream).  X bf16 [M, K], W bf16 [N, K], bias bf16 [N] or None,
    Y float32 / bfloat16 [M, N]; all contiguous device tensors."""
    _check_operands(X, W, bias, Y)
    M, N, K = _shape(X, W, M, N, K)
    _check(lib().proj_run(ctx, _ptr(X), _ptr(W), _ptr(bias), int(epilogue), M, N, K, _ptr(Y),
                          _out_dtype(Y, out_dtype), _stream(stream)), ctx)


def proj_run_noalloc(ctx, X, W, bias, epilogue, Y, M=None, N=None, K=None, out_dtype=None, stream=None) -> None:
    """proj_run without any device allocation: split-K partials go to the
    library's static per-GPU scratch (2 MiB)."""
    _check_operands(X, W, bias, Y)
    M, N, K = _shape(X, W, M, N, K)
    _check(lib().proj_run_noalloc(ctx, _ptr(X), _ptr(W), _ptr(bias), int(epilogue), M, N, K, _ptr(Y),
                                  _out_dtype(Y, out_dtype), _stream(stream)), ctx)


def proj_tune(ctx, X, W, bias, epilogue, Y, M=None, N=None, K=None, out_dtype=None, stream=None) -> None:
    _check_operands(X, W, bias, Y)
    M, N, K = _shape(X, W, M, N, K)
    _check(lib().proj_tune(ctx, _ptr(X), _ptr(W), _ptr(bias), int(epilogue), M, N, K, _ptr(Y),
                           _out_dtype(Y, out_dtype), _stream(stream)), ctx)


def proj_get_plan(ctx, M, N, K, epilogue, out_dtype, aligned16=True) -> str:
    buf = ctypes.create_string_buffer(256)
    _check(lib().proj_get_plan(ctx, int(M), int(N), int(K), int(epilogue), int(out_dtype),
                               1 if aligned16 else 0, buf, 256), ctx)
    return buf.value.decode()


def proj_num_candidates(M, N, K, epilogue, out_dtype, aligned16=True) -> int:
    return int(lib().proj_num_candidates(int(M), int(N), int(K), int(epilogue), int(out_dtype),
                                         1 if aligned16 else 0))


def proj_candidate_name(M, N, K, epilogue, out_dtype, index, aligned16=True) -> str:
    buf = ctypes.create_string_buffer(256)
    _check(lib().proj_candidate_name(int(M), int(N), int(K), int(epilogue), int(out_dtype),
                                     1 if aligned16 else 0, int(index), buf, 256))
    return buf.value.decode()


def proj_run_candidate(ctx, index, X, W, bias, epilogue, Y, M=None, N=None, K=None, out_dtype=None,
                       stream=None) -> None:
    _check_operands(X, W, bias, Y)
    M, N, K = _shape(X, W, M, N, K)
    _check(lib().proj_run_candidate(ctx, int(index), _ptr(X), _ptr(W), _ptr(bias), int(epilogue), M, N, K,
                                    _ptr(Y), _out_dtype(Y, out_dtype), _stream(stream)), ctx)


# ---------------------------------------------- fp32 weights, high/low pair

def proj_prepare_hilo(ctx, W, Whl=None, stream=None):
    """Register fp32 weights W [N, K] (device float32 tensor) as the bf16
    pair Whl [N, 2K] = [H | L] (allocated here if not given); returns Whl."""
    import torch
    if W.dtype != torch.float32 or W.dim() != 2:
        raise ValueError("W must be a float32 [N, K] tensor")
    N, K = W.shape
    if Whl is None:
        Whl = torch.empty((N, 2 * K), dtype=torch.bfloat16, device=W.device)
    elif Whl.dtype != torch.bfloat16 or tuple(Whl.shape) != (N, 2 * K):
        raise ValueError("Whl must be bfloat16 [N, 2K]")
    _check(lib().proj_prepare_hilo(ctx, _ptr(W), int(N), int(K), _ptr(Whl), _stream(stream)), ctx)
    return Whl


def _shape_hilo(X, Whl, M, N, K):
    if M is None:
        M = X.shape[0]
    if N is None:
        N = Whl.shape[0]
    if K is None:
        K = X.shape[1]
    return int(M), int(N), int(K)


def proj_run_hilo(ctx, X, Whl, bias, epilogue, Y, M=None, N=None, K=None, out_dtype=None, stream=None) -> None:
    """Enqueue Y = epilogue(X . H^T + X . L^T [+ bias]) for X bf16 [M, K] and
    a registered pair Whl bf16 [N, 2K]."""
    _check_operands(X, Whl, bias, Y)
    M, N, K = _shape_hilo(X, Whl, M, N, K)
    _check(lib().proj_run_hilo(ctx, _ptr(X), _ptr(Whl), _ptr(bias), int(epilogue), M, N, K, _ptr(Y),
                               _out_dtype(Y, out_dtype), _stream(stream)), ctx)


def proj_get_plan_hilo(ctx, M, N, K, epilogue, out_dtype, aligned16=True) -> str:
    buf = ctypes.create_string_buffer(256)
    _check(lib().proj_get_plan_hilo(ctx, int(M), int(N), int(K), int(epilogue), int(out_dtype),
                                    1 if aligned16 else 0, buf, 256), ctx)
    return buf.value.decode()


def proj_num_candidates_hilo(M, N, K, epilogue, out_dtype, aligned16=True) -> int:
    return int(lib().proj_num_candidates_hilo(int(M), int(N), int(K), int(epilogue), int(out_dtype),
                                              1 if aligned16 else 0))


def proj_candidate_name_hilo(M, N, K, epilogue, out_dtype, index, aligned16=True) -> str:
    buf = ctypes.create_string_buffer(256)
    _check(lib().proj_candidate_name_hilo(int(M), int(N), int(K), int(epilogue), int(out_dtype),
                                          1 if aligned16 else 0, int(index), buf, 256))
    return buf.value.decode()


def proj_run_candidate_hilo(ctx, index, X, Whl, bias, epilogue, Y, M=None, N=None, K=None, out_dtype=None,
                            stream=None) -> None:
    _check_operands(X, Whl, bias, Y)
    M, N, K = _shape_hilo(X, Whl, M, N, K)
    _check(lib().proj_run_candidate_hilo(ctx, int(index), _ptr(X), _ptr(Whl), _ptr(bias), int(epilogue), M, N, K,
                                         _ptr(Y), _out_dtype(Y, out_dtype), _stream(stream)), ctx)


def proj_packed_bytes(N, K, tile16) -> int:
    """Bytes of the packed array for W [N, K] in tiles of 16 * tile16 rows
    (-1 if that packing is not offered)."""
    return int(lib().proj_packed_bytes(int(N), int(K), int(tile16)))


def proj_pack_weights(ctx, W, tile16, Wp=None, stream=None):
    """Pack bf16 W [N, K] into the tile layout (Wp allocated here if not
    given: a flat bf16 tensor of proj_packed_bytes / 2 elements); returns Wp."""
    import torch
    if W.dtype != torch.bfloat16 or W.dim() != 2:
        raise ValueError("W must be a bfloat16 [N, K] tensor")
    N, K = W.shape
    nbytes = proj_packed_bytes(N, K, tile16)
    if nbytes < 0:
        raise ValueError("no packing for N=%d K=%d tile16=%d" % (N, K, tile16))
    if Wp is None:
        Wp = torch.empty((nbytes // 2,), dtype=torch.bfloat16, device=W.device)
    elif Wp.dtype != torch.bfloat16 or Wp.numel() * 2 < nbytes:
        raise ValueError("Wp must be bfloat16 with at least %d bytes" % nbytes)
    _check(lib().proj_pack_weights(ctx, _ptr(W), int(N), int(K), int(tile16), _ptr(Wp), _stream(stream)), ctx)
    return Wp


def proj_run_packed(ctx, X, Wp, tile16, bias, epilogue, Y, N, M=None, K=None, out_dtype=None, stream=None) -> None:
    """Enqueue Y = epilogue(X . W^T [+ bias]) with W given packed (Wp from
    proj_pack_weights with the same tile16); N is W's row count."""
    _check_operands(X, Wp, bias, Y)
    M = int(X.shape[0] if M is None else M)
    K = int(X.shape[1] if K is None else K)
    _check(lib().proj_run_packed(ctx, _ptr(X), _ptr(Wp), int(tile16), _ptr(bias), int(epilogue), M, int(N), K,
                                 _ptr(Y), _out_dtype(Y, out_dtype), _stream(stream)), ctx)


def proj_get_plan_packed(ctx, M, N, K, tile16, epilogue, out_dtype, aligned16=True) -> str:
    buf = ctypes.create_string_buffer(256)
    _check(lib().proj_get_plan_packed(ctx, int(M), int(N), int(K), int(tile16), int(epilogue), int(out_dtype),
                                      1 if aligned16 else 0, buf, 256), ctx)
    return buf.value.decode()


def proj_num_candidates_packed(M, N, K, tile16, epilogue, out_dtype, aligned16=True) -> int:
    return int(lib().proj_num_candidates_packed(int(M), int(N), int(K), int(tile16), int(epilogue), int(out_dtype),
                                                1 if aligned16 else 0))


def proj_candidate_name_packed(M, N, K, tile16, epilogue, out_dtype, index, aligned16=True) -> str:
    buf = ctypes.create_string_buffer(256)
    _check(lib().proj_candidate_name_packed(int(M), int(N), int(K), int(tile16), int(epilogue), int(out_dtype),
                                            1 if aligned16 else 0, int(index), buf, 256))
    return buf.value.decode()


def proj_run_candidate_packed(ctx, index, X, Wp, tile16, bias, epilogue, Y, N, M=None, K=None, out_dtype=None,
                              stream=None) -> None:
    _check_operands(X, Wp, bias, Y)
    M = int(X.shape[0] if M is None else M)
    K = int(X.shape[1] if K is None else K)
    _check(lib().proj_run_candidate_packed(ctx, int(index), _ptr(X), _ptr(Wp), int(tile16), _ptr(bias),
                                           int(epilogue), M, int(N), K, _ptr(Y), _out_dtype(Y, out_dtype),
                                           _stream(stream)), ctx)


# ------------------------------------------- 4-bit weights, group scales

def _is_tensor(name, t, dtypes, shape=None):
    """Raise ValueError unless t is a device tensor of one of `dtypes` and, where given, of `shape`."""
    if not t.is_cuda:
        raise ValueError("%s must be on a GPU" % name)
    if t.dtype not in dtypes:
        raise ValueError("%s must be %s, got %s" % (name, " or ".join(map(str, dtypes)), t.dtype))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))


def _operand(name, t, dtypes, shape):
    """Pointer of a contiguous device tensor of one of `dtypes` and of `shape` (a tuple); ValueError for another."""
    if t.is_cuda and t.dtype in dtypes and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _is_tensor(name, t, dtypes, shape)
    raise ValueError("%s must be contiguous (row-major)" % name)


class _Types:
    """The operators' dtype tuples, made once torch is there."""

    def __init__(self):
        import torch
        self.f32 = torch.float32
        self.bf16, self.fp32, self.float = (torch.bfloat16,), (torch.float32,), (torch.bfloat16, torch.float32)
        self.u8, self.i8, self.i32, self.i64 = (torch.uint8,), (torch.int8,), (torch.int32,), (torch.int64,)


_types = None


def _dtypes():
    global _types
    if _types is None:
        _types = _Types()
    return _types


def _new(shapes_and_types, device, stream):
    """Tensors in the memory of `stream` (default: torch's current stream),
    which the allocator hands on only behind that stream's work."""
    import torch
    if stream is None:
        return [torch.empty(s, dtype=t, device=device) for s, t in shapes_and_types]
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return [torch.empty(s, dtype=t, device=device) for s, t in shapes_and_types]


def proj_pack_codes(ctx, q, codes=None, stream=None):
    """Lay out 4-bit codes given one to a byte (uint8 [N, K], K a multiple of
    8) as int32 words [N, K / 8] (allocated here if not given): of eight
    codes, code j sits at bits 4 * (j // 2) + 16 * (j % 2).  Returns them."""
    import torch
    _is_tensor("q", q, (torch.uint8,))
    if q.dim() != 2 or q.shape[1] % 8:
        raise ValueError("q must be uint8 [N, K] with K a multiple of 8")
    N, K = q.shape
    if codes is None:
        codes, = _new([((N, K // 8), torch.int32)], q.device, stream)
    _is_tensor("codes", codes, (torch.int32,), (N, K // 8))
    _check(lib().proj_pack_codes(ctx, _ptr(q), N, K, _ptr(codes), _stream(stream)), ctx)
    return codes


def proj_quantize_weights(ctx, W, group=128, zeros=True, scale_dtype=None, stream=None):
    """4-bit weights of bf16 W [N, K]: (codes int32 [N, K / 8], scales
    [N, G], zeros uint8 [N, G] or None), G = ceil(K / group).  With zeros=False every zero
    point is 8; scales are bf16 unless scale_dtype is torch.float32."""
    import torch
    _is_tensor("W", W, (torch.bfloat16,))
    if W.dim() != 2 or W.shape[1] % 8 or group not in (32, 64, 128):
        raise ValueError("W must be bfloat16 [N, K] with K a multiple of 8, group 32, 64 or 128")
    dt = torch.bfloat16 if scale_dtype is None else scale_dtype
    if dt not in (torch.bfloat16, torch.float32):
        raise ValueError("scale_dtype must be bfloat16 or float32")
    N, K = W.shape
    G = -(-K // group)
    codes, scales, z = _new([((N, K // 8), torch.int32), ((N, G), dt), ((N, G if zeros else 0), torch.uint8)], W.device, stream)
    if not zeros:
        z = None
    _check(lib().proj_quantize_weights(ctx, _ptr(W), N, K, int(group), _ptr(codes), _ptr(scales),
                                       OUT_F32 if dt == torch.float32 else OUT_BF16, _ptr(z), _stream(stream)), ctx)
    return codes, scales, z


def proj_run_quant(ctx, X, codes, scales, zeros, group, bias, epilogue, Y, stream=None) -> None:
    """Enqueue Y = epilogue(X . W^T [+ bias]) with 4-bit W[n, k] =
    scales[n, k // group] * (code[n, k] - zeros[n, k // group]) (zeros None:
    8).  X bf16 [M, K], codes int32 [N, K / 8], scales bf16 or float32 and
    zeros uint8 [N, ceil(K / group)], bias bf16 [N] or None, Y float32 /
    bfloat16 [M, N]; all contiguous device tensors.  X should start at a
    16-byte boundary: one that does not is right, but about 100 times slower
    with many rows."""
    T = _types or _dtypes()
    _is_tensor("X", X, T.bf16)
    _is_tensor("codes", codes, T.i32)
    if X.dim() != 2 or codes.dim() != 2 or group not in (32, 64, 128):
        raise ValueError("X [M, K] and codes [N, K / 8] must have two dimensions, group 32, 64 or 128")
    M, K = X.shape
    N, words = codes.shape
    if words * 8 != K:
        raise ValueError("codes of %d words to a row do not fit K = %d" % (words, K))
    G = -(-K // group)
    f32 = T.f32
    st = (_lib or lib()).proj_run_quant(
        ctx, _ptr(X), _ptr(codes), _operand("scales", scales, T.float, (N, G)), OUT_F32 if scales.dtype == f32 else OUT_BF16,
        None if zeros is None else _operand("zeros", zeros, T.u8, (N, G)), group,
        None if bias is None else _operand("bias", bias, T.bf16, (N,)), epilogue, M, N, K,
        _operand("Y", Y, T.float, (M, N)), OUT_F32 if Y.dtype == f32 else OUT_BF16, _stream(stream))
    if st:
        _check(st, ctx)


# ------------------------- 8-bit integers, a scale to each token and output

def proj_quantize_rows(ctx, X, q=None, scales=None, stream=None):
    """8-bit integers of bf16 rows X [M, K] (rows may be strided): (q int8
    [M, K rounded up to a multiple of 16], zero behind K, scales float32 [M]),
    allocated here unless given.  scales = max |row| / 127 and q = rint(127 x /
    max |row|): the tokens and the weights that proj_run_int takes."""
    T = _types or _dtypes()
    _is_tensor("X", X, T.bf16)
    if X.dim() != 2:
        raise ValueError("X must be [M, K]")
    M, K = X.shape
    padded = -(-K // 16) * 16
    if q is None or scales is None:
        made = _new([((M, padded), T.i8[0]), ((M,), T.f32)], X.device, stream)
        q, scales = made[0] if q is None else q, made[1] if scales is None else scales
    x, stride = _rows("X", X, K)
    _check((_lib or lib()).proj_quantize_rows(ctx, x, stride, M, K, _operand("q", q, T.i8, (M, padded)), padded,
                                              _operand("scales", scales, T.fp32, (M,)), _stream(stream)), ctx)
    return q, scales


def proj_run_int(ctx, X, x_scales, W, w_scales, bias, epilogue, Y, stream=None) -> None:
    """Enqueue Y = epilogue(x_scales[m] * w_scales[n] * sum_k X[m, k] W[n, k]
    [+ bias]): X int8 [M, K] and W int8 [N, K], K a multiple of 16 (as
    proj_quantize_rows pads them), x_scales and w_scales float32 [M] and [N],
    bias bf16 [N] or None, Y float32 / bfloat16 [M, N]; all contiguous device
    tensors, X and W starting at 16-byte boundaries."""
    T = _types or _dtypes()
    _is_tensor("X", X, T.i8)
    _is_tensor("W", W, T.i8)
    if X.dim() != 2 or W.dim() != 2:
        raise ValueError("X [M, K] and W [N, K] must have two dimensions")
    M, K = X.shape
    N = W.shape[0]
    st = (_lib or lib()).proj_run_int(
        ctx, _operand("X", X, T.i8, (M, K)), _operand("x_scales", x_scales, T.fp32, (M,)), _operand("W", W, T.i8, (N, K)),
        _operand("w_scales", w_scales, T.fp32, (N,)), None if bias is None else _operand("bias", bias, T.bf16, (N,)), epilogue,
        M, N, K, _operand("Y", Y, T.float, (M, N)), OUT_F32 if Y.dtype == T.f32 else OUT_BF16, _stream(stream))
    if st:
        _check(st, ctx)


def proj_run_int_dynamic(ctx, X, W, w_scales, bias, epilogue, Y, stream=None) -> None:
    """proj_run_int from bf16 tokens X [M, K] (rows may be strided), made
    integers row by row in the context's workspace; W int8 [N, K rounded up to a
    multiple of 16], zero behind K.  Tokens that meet several projections are
    made integers once with proj_quantize_rows instead."""
    T = _types or _dtypes()
    _is_tensor("X", X, T.bf16)
    _is_tensor("W", W, T.i8)
    if X.dim() != 2 or W.dim() != 2:
        raise ValueError("X [M, K] and W [N, K] must have two dimensions")
    M, K = X.shape
    N = W.shape[0]
    x, stride = _rows("X", X, K)
    st = (_lib or lib()).proj_run_int_dynamic(
        ctx, x, stride, _operand("W", W, T.i8, (N, -(-K // 16) * 16)), _operand("w_scales", w_scales, T.fp32, (N,)),
        None if bias is None else _operand("bias", bias, T.bf16, (N,)), epilogue, M, N, K, _operand("Y", Y, T.float, (M, N)),
        OUT_F32 if Y.dtype == T.f32 else OUT_BF16, _stream(stream))
    if st:
        _check(st, ctx)


# ------------------------------------------------- paged key-value cache

class kv_cache:
    """A paged cache in the caller's tensors k and v [pages, heads, page_size,
    head_dim], bfloat16 or float8_e4m3fn (values = stored * scale).  Any
    strides with a contiguous head: pages stored token-major are passed as
    `k.transpose(1, 2)`.  Built once and used by every call; it keeps k and v
    alive."""

    def __init__(self, k, v, k_scale: float = 1.0, v_scale: float = 1.0):
        import torch
        for name, t in (("k", k), ("v", v)):
            _is_tensor(name, t, (torch.bfloat16, torch.float8_e4m3fn))
            if t.dim() != 4 or (t.numel() and t.stride(3) != 1):
                raise ValueError("%s must be [pages, heads, page_size, head_dim] with contiguous heads" % name)
        if k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v differ in shape, dtype or device")
        self.k, self.v = k, v
        self.pages, self.heads, self.page_size, self.head_dim = k.shape
        s3 = ctypes.c_int64 * 3
        self._c = _KvCache(k.data_ptr(), v.data_ptr(), KV_FP8 if k.dtype == torch.float8_e4m3fn else KV_BF16, self.heads,
                           self.head_dim, self.page_size, self.pages, s3(*k.stride()[:3]), s3(*v.stride()[:3]),
                           float(k_scale), float(v_scale))
        self._p = ctypes.addressof(self._c)


def _rows(name, t, width):
    """Pointer and row stride (elements) of a tensor whose rows, of `width` elements, are contiguous."""
    if t.is_contiguous():
        return t.data_ptr(), width
    if not t[0].is_contiguous():
        raise ValueError("%s must have contiguous rows" % name)
    return t.data_ptr(), width if t.shape[0] == 1 else t.stride(0)


def _append_shape(cache, qkv, rope, q_heads, D):
    """(tokens, query heads, pointer and row stride of qkv)"""
    _is_tensor("qkv", qkv, D.bf16)
    if qkv.dim() != 2:
        raise ValueError("qkv must be [T, width]")
    T, width = qkv.shape
    heads = width // cache.head_dim - 2 * cache.heads
    if width % cache.head_dim or heads < 0 or (q_heads is not None and q_heads != heads):
        raise ValueError("qkv of width %d does not hold %s query and 2 * %d key-value heads of %d" %
                         (width, "any" if q_heads is None else q_heads, cache.heads, cache.head_dim))
    _is_tensor("rope", rope, D.fp32)
    if rope.dim() != 2:
        raise ValueError("rope must be [positions, rot]")
    return (T, heads) + _rows("qkv", qkv, width)


def proj_kv_append(ctx, cache, qkv, rope, positions, slots, q_out=None, q_heads=None, interleaved=False,
                   stream=None) -> None:
    """Enqueue one append: of qkv bf16 [T, (q_heads + 2 * heads) * head_dim]
    (rows may be strided) the query and key heads are rotated by the rows
    `positions` (int32 [T]) of rope float32 [positions, rot] (cosines, then
    sines); queries go to q_out bf16 [T, q_heads, head_dim] (None: dropped),
    keys and values into the cache's slots (int64 [T], page * page_size +
    place; negative: a padding token, not stored; two tokens with one slot: a
    mix of both)."""
    D = _types or _dtypes()
    T, heads, x, stride = _append_shape(cache, qkv, rope, q_heads, D)
    st = (_lib or lib()).proj_kv_append(
        ctx, cache._p, x, stride, T, heads, _ptr(rope), rope.shape[0], rope.shape[1], 1 if interleaved else 0,
        _operand("positions", positions, D.i32, (T,)), _operand("slots", slots, D.i64, (T,)),
        None if q_out is None else _operand("q_out", q_out, D.bf16, (T, heads, cache.head_dim)), _stream(stream))
    if st:
        _check(st, ctx)


def proj_kv_append_norm(ctx, cache, qkv, q_norm, k_norm, eps, rope, positions, slots, q_out=None, q_heads=None,
                        interleaved=False, stream=None) -> None:
    """proj_kv_append whose query and key heads are first divided by their root
    mean square: x / sqrt(mean(x^2) + eps) * w, with w = q_norm and k_norm
    (bfloat16 or float32, both of one type, [head_dim] or both of each head's own
    [q_heads, head_dim] and [heads, head_dim]; None: not normed)."""
    D = _types or _dtypes()
    T, heads, x, stride = _append_shape(cache, qkv, rope, q_heads, D)
    given = [(n, t, h) for n, t, h in (("q_norm", q_norm, heads), ("k_norm", k_norm, cache.heads)) if t is not None]
    per_head = bool(given) and given[0][1].dim() == 2
    f32 = bool(given) and given[0][1].dtype == D.f32
    for name, t, h in given:
        _operand(name, t, D.fp32 if f32 else D.bf16, (h, cache.head_dim) if per_head else (cache.head_dim,))
    st = (_lib or lib()).proj_kv_append_norm(
        ctx, cache._p, x, stride, T, heads, _ptr(q_norm), _ptr(k_norm), OUT_F32 if f32 else OUT_BF16, 1 if per_head else 0, eps,
        _ptr(rope), rope.shape[0], rope.shape[1], 1 if interleaved else 0, _operand("positions", positions, D.i32, (T,)),
        _operand("slots", slots, D.i64, (T,)),
        None if q_out is None else _operand("q_out", q_out, D.bf16, (T, heads, cache.head_dim)), _stream(stream))
    if st:
        _check(st, ctx)


def proj_kv_attend(ctx, cache, q, tables, lengths, scale, out, lse=None, window=0, max_len=None, stream=None) -> None:
    """Enqueue attention of one new token for each of B sequences: q bf16
    [B, q_heads, head_dim] (rows may be strided), tables int32 [B, width] the
    sequences' pages, lengths int32 [B] their tokens (0: a padding place, out
    0), the last `window` of them seen (0: all); out float32 / bfloat16
    [B, q_heads, head_dim], lse float32 [B, q_heads] or None.  max_len bounds
    the lengths (default: what the tables hold); a tight one gives a better
    split."""
    T = _types or _dtypes()
    _is_tensor("q", q, T.bf16)
    if q.dim() != 3 or q.shape[2] != cache.head_dim:
        raise ValueError("q must be [B, q_heads, %d]" % cache.head_dim)
    B, heads, D = q.shape
    _is_tensor("tables", tables, T.i32)
    if tables.dim() != 2 or tables.shape[0] != B:
        raise ValueError("tables must be [B, width]")
    tw = tables.shape[1]
    qp, stride = _rows("q", q, heads * D)
    tp, tstride = _rows("tables", tables, tw)
    st = (_lib or lib()).proj_kv_attend(
        ctx, cache._p, qp, stride, B, heads, tp, tstride, tw, _operand("lengths", lengths, T.i32, (B,)),
        tw * cache.page_size if max_len is None else max_len, window, scale, _operand("out", out, T.float, (B, heads, D)),
        OUT_F32 if out.dtype == T.f32 else OUT_BF16,
        None if lse is None else _operand("lse", lse, T.fp32, (B, heads)), _stream(stream))
    if st:
        _check(st, ctx)


def proj_kv_attend_shared(ctx, cache, q, prefix, prefix_len, tables, lengths, scale, out, lse=None, window=0, max_len=None,
                          stream=None) -> None:
    """proj_kv_attend for a batch whose sequences begin with the same prefix_len
    tokens, in the pages `prefix` (int32 [pages]); `tables` int32 [B, width] (rows
    may be strided) hold the pages of each sequence's own tokens, while lengths,
    window and max_len (default: the prefix and what the tables hold) count all of
    a sequence's tokens."""
    T = _types or _dtypes()
    _is_tensor("q", q, T.bf16)
    if q.dim() != 3 or q.shape[2] != cache.head_dim:
        raise ValueError("q must be [B, q_heads, %d]" % cache.head_dim)
    B, heads, D = q.shape
    _is_tensor("tables", tables, T.i32)
    if tables.dim() != 2 or tables.shape[0] != B:
        raise ValueError("tables must be [B, width]")
    _is_tensor("prefix", prefix, T.i32)
    if prefix.dim() != 1 or prefix_len < 0 or prefix.shape[0] * cache.page_size < prefix_len:
        raise ValueError("prefix must hold the pages of %d tokens" % prefix_len)
    tw = tables.shape[1]
    qp, stride = _rows("q", q, heads * D)
    tp, tstride = _rows("tables", tables, tw)
    st = (_lib or lib()).proj_kv_attend_shared(
        ctx, cache._p, qp, stride, B, heads, _operand("prefix", prefix, T.i32, prefix.shape), prefix_len, tp, tstride, tw,
        _operand("lengths", lengths, T.i32, (B,)), prefix_len + tw * cache.page_size if max_len is None else max_len, window,
        scale, _operand("out", out, T.float, (B, heads, D)), OUT_F32 if out.dtype == T.f32 else OUT_BF16,
        None if lse is None else _operand("lse", lse, T.fp32, (B, heads)), _stream(stream))
    if st:
        _check(st, ctx)


def proj_graph_capture(ctx, Xs, Ws, biases, Ys, epilogue, out_dtype=None, stream=None) -> int:
    """Capture len(Xs) calls (call i on Xs[i], Ws[i], biases[i], Ys[i]) into
    one instantiated HIP graph; returns its handle.  `stream` must not be the
    legacy default stream."""
    n = len(Xs)
    if not (len(Ws) == n and len(Ys) == n and (biases is None or len(biases) == n)):
        raise ValueError("buffer lists differ in length")
    for i in range(n):
        _check_operands(Xs[i], Ws[i], biases[i] if biases else None, Ys[i])
    M, N, K = _shape(Xs[0], Ws[0], None, None, None)
    arr = ctypes.c_void_p * n
    xs = arr(*[_ptr(t) for t in Xs])
    ws = arr(*[_ptr(t) for t in Ws])
    bs = arr(*[_ptr(t) for t in biases]) if biases else None
    ys = arr(*[_ptr(t) for t in Ys])
    g = ctypes.c_void_p()
    _check(lib().proj_graph_capture(ctx, n, xs, ws, bs, ys, int(epilogue), M, N, K,
                                    _out_dtype(Ys[0], out_dtype), _stream(stream), ctypes.byref(g)), ctx)
    return g.value


def proj_read_probe(ctx, buf, stream=None) -> None:
    """Enqueue one plain streaming read of the whole of tensor `buf` (its
    bytes a multiple of 16): the measured read floor to time beside
    proj_run on the same buffers."""
    nbytes = buf.numel() * buf.element_size()
    _check(lib().proj_read_probe(ctx, _ptr(buf), nbytes, _stream(stream)), ctx)


def proj_graph_launch(graph, stream=None) -> None:
    _check(lib().proj_graph_launch(graph, _stream(stream)))


def proj_graph_destroy(graph) -> None:
    _check(lib().proj_graph_destroy(graph))


# ------------------------------------------------------------ convenience

def project(ctx, X, W, bias=None, gelu=False, out_dtype=None, stream=None):
    """Allocate Y with torch and run the projection; returns Y."""
    import torch
    epi = (EPI_BIAS if bias is not None else EPI_NONE) | (EPI_GELU_TANH if gelu else 0)
    dt = torch.bfloat16 if out_dtype in (None, OUT_BF16, torch.bfloat16) else torch.float32
    Y = torch.empty((X.shape[0], W.shape[0]), dtype=dt, device=X.device)
    proj_run(ctx, X, W, bias, epi, Y, stream=stream)
    return Y
