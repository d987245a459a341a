"""GB300 (sm_103a) W8A8 mixture-of-experts expert layer, its router and its MXFP4 form.

Thin Python binding over the C ABI in ``include/moe_layer.h`` and
``include/moe_mxfp4.h`` (library
``_build/libmoe_layer.so``, built by ``moe_expert_layer_gb300.build``).  The
functions below carry the ABI's names and only marshal arguments: torch
tensors (device memory) become raw pointers, the stream defaults to torch's
current stream, and a non-zero status raises ``MoeError``.  Every stage of the
layer runs in the library's CUDA kernels; there is no other code path, and
importing the binding fails loudly when the library is missing.
"""
import ctypes
import os

from . import build as _build

LIB_PATH = _build.LIB_PATH

STATUS = {0: "MOE_OK", -1: "MOE_ERR_NULL", -2: "MOE_ERR_SHAPE", -3: "MOE_ERR_ALIGN",
          -4: "MOE_ERR_ARCH", -5: "MOE_ERR_WORKSPACE", -6: "MOE_ERR_LAUNCH",
          -8: "MOE_ERR_TIMEOUT"}

# every entry point declared in include/moe_layer.h and include/moe_mxfp4.h
EXPORTS = [
    "moe_status_string", "moe_layer_workspace_size", "moe_layer_fwd",
    "moe_layer_host_workspace_size", "moe_layer_fwd_host", "moe_workspace_status",
    "moe_workspace_clear_status", "moe_route_sort_workspace_size", "moe_route_sort",
    "moe_quant_tokens", "moe_quant_dispatch", "moe_front_reorder", "moe_gmm_workspace_size", "moe_gmm1",
    "moe_swiglu_quant", "moe_gmm1_swiglu", "moe_gmm2", "moe_combine_unpermute", "moe_route_sort_noalloc",
    "moe_selftest_wait_timeout", "moe_selftest_count_timeout",
    "moe_layer_graph_create", "moe_layer_graph_create_host", "moe_layer_graph_launch", "moe_layer_graph_destroy",
    "moe_layer_pipeline_workspace_size", "moe_layer_pipeline_create", "moe_layer_pipeline_submit",
    "moe_layer_pipeline_wait", "moe_layer_pipeline_destroy",
    "moe_weight_tiles_bytes", "moe_pack_weight_tiles",
    "moe_route_topk", "moe_mxfp4_scale_words", "moe_mxfp4_quant", "moe_mxfp4_dequant", "moe_mxfp4_weights_bytes",
    "moe_mxfp4_quant_weights", "moe_mxfp4_pack_weights", "moe_mxfp4_gmm_workspace_size", "moe_mxfp4_gmm",
    "moe_mxfp4_gmm_swiglu", "moe_mxfp4_layer_workspace_size", "moe_mxfp4_layer_fwd", "moe_selftest_mxfp4_tickets",
]

# weight layouts (moe_dims_t.weight_layout)
WEIGHTS_ROWS = 0
WEIGHTS_TILES = 1


class MoeError(RuntimeError):
    def __init__(self, fn, code):
        self.code = code
        super().__init__("%s failed: %s (%d)" % (fn, STATUS.get(code, "unknown"), code))


class moe_dims_t(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int32), ("K", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("topK", ctypes.c_int32), ("weight_layout", ctypes.c_int32)]


def dims(M, K, I, E, topK, weight_layout=WEIGHTS_ROWS):
    return moe_dims_t(M, K, I, E, topK, weight_layout)


_lib = None


def load_library(path=None):
    """Loads the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise ImportError("libmoe_layer.so not built (run moe_expert_layer_gb300.build.build())")
    lib = ctypes.CDLL(path)
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
    D = ctypes.POINTER(moe_dims_t)
    sigs = {
        "moe_status_string": ([i32], ctypes.c_char_p),
        "moe_layer_workspace_size": ([D], sz),
        "moe_layer_host_workspace_size": ([D], sz),
        "moe_layer_fwd": ([D] + [vp] * 9 + [sz, vp], i32),
        "moe_layer_fwd_host": ([D] + [vp] * 9 + [sz, vp], i32),
        "moe_layer_graph_create": ([D] + [vp] * 9 + [sz, vp, ctypes.POINTER(vp)], i32),
        "moe_layer_graph_create_host": ([D] + [vp] * 9 + [sz, vp, ctypes.POINTER(vp)], i32),
        "moe_layer_graph_launch": ([vp, vp], i32),
        "moe_layer_graph_destroy": ([vp], i32),
        "moe_layer_pipeline_workspace_size": ([D, i32], sz),
        "moe_layer_pipeline_create": ([D] + [vp] * 5 + [sz, i32, ctypes.POINTER(vp)], i32),
        "moe_layer_pipeline_submit": ([vp] * 5 + [ctypes.POINTER(ctypes.c_uint64)], i32),
        "moe_layer_pipeline_wait": ([vp, ctypes.c_uint64], i32),
        "moe_layer_pipeline_destroy": ([vp], i32),
        "moe_workspace_status": ([vp, ctypes.POINTER(i32), vp], i32),
        "moe_workspace_clear_status": ([vp, vp], i32),
        "moe_route_sort_workspace_size": ([D], sz),
        "moe_route_sort": ([D] + [vp] * 6 + [sz, vp], i32),
        "moe_quant_tokens": ([D] + [vp] * 7, i32),
        "moe_gmm_workspace_size": ([D], sz),
        "moe_quant_dispatch": ([D] + [vp] * 7, i32),
        "moe_front_reorder": ([D] + [vp] * 10 + [sz, vp], i32),
        "moe_gmm1": ([D] + [vp] * 8 + [sz, vp], i32),
        "moe_swiglu_quant": ([D] + [vp] * 10, i32),
        "moe_gmm1_swiglu": ([D] + [vp] * 13 + [sz, vp], i32),
        "moe_gmm2": ([D] + [vp] * 7 + [sz, vp], i32),
        "moe_combine_unpermute": ([D] + [vp] * 6, i32),
        "moe_route_sort_noalloc": ([D] + [vp] * 6, i32),
        "moe_selftest_wait_timeout": ([vp, ctypes.c_uint32, vp], i32),
        "moe_selftest_count_timeout": ([vp, vp, ctypes.c_uint32, vp], i32),
        "moe_weight_tiles_bytes": ([D, i32], sz),
        "moe_pack_weight_tiles": ([D, i32, vp, vp, vp], i32),
        "moe_route_topk": ([i32] * 3 + [vp, i32, ctypes.c_int64, vp, i32, i32, ctypes.c_float] + [vp] * 3, i32),
        "moe_mxfp4_scale_words": ([ctypes.c_int64, i32], sz),
        "moe_mxfp4_quant": ([i32, i32, vp, i32, ctypes.c_int64, vp, i32, i32] + [vp] * 3, i32),
        "moe_mxfp4_dequant": ([i32, i32, vp, vp, vp, i32, vp], i32),
        "moe_mxfp4_weights_bytes": ([i32] * 3, sz),
        "moe_mxfp4_quant_weights": ([i32] * 4 + [vp, i32, vp, vp], i32),
        "moe_mxfp4_pack_weights": ([i32] * 4 + [vp] * 4, i32),
        "moe_mxfp4_gmm_workspace_size": ([i32] * 4, sz),
        "moe_mxfp4_gmm": ([i32] * 4 + [vp] * 6 + [sz, vp], i32),
        "moe_mxfp4_gmm_swiglu": ([i32] * 4 + [vp] * 7 + [sz, vp], i32),
        "moe_mxfp4_layer_workspace_size": ([D], sz),
        "moe_mxfp4_layer_fwd": ([D] + [vp] * 7 + [sz, vp], i32),
        "moe_selftest_mxfp4_tickets": ([vp, vp], i32),
    }
    for name, (args, res) in sigs.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    _lib = lib
    return lib


def _p(t):
    """Raw pointer of a tensor (device or host), or None.  The ABI takes dense
    row-major arrays, so a tensor with any other strides (a transpose, a column
    slice, an expanded view) is refused rather than read with the wrong layout."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("the C ABI takes dense row-major arrays; got a tensor with shape %s and strides %s"
                         % (tuple(t.shape), tuple(t.stride())))
    return t.data_ptr()


_current_stream = None


def _find_current_stream():
    """A function that gives torch's current stream as a raw handle: straight from torch's core where
    it has it (the public call builds a Stream object each time, microseconds of a short call)."""
    import torch
    core = torch._C
    if hasattr(core, "_cuda_getCurrentRawStream") and hasattr(core, "_cuda_getDevice"):
        torch.cuda.current_stream()  # initialises CUDA
        return lambda: core._cuda_getCurrentRawStream(core._cuda_getDevice())
    return lambda: torch.cuda.current_stream().cuda_stream


def _stream(stream):
    global _current_stream
    if stream is None:
        if _current_stream is None:
            _current_stream = _find_current_stream()
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn, code):
    if code != 0:
        raise MoeError(fn, code)


def moe_layer_workspace_size(d):
    return load_library().moe_layer_workspace_size(ctypes.byref(d))


def moe_layer_host_workspace_size(d):
    return load_library().moe_layer_host_workspace_size(ctypes.byref(d))


def moe_route_sort_workspace_size(d):
    return load_library().moe_route_sort_workspace_size(ctypes.byref(d))


def moe_gmm_workspace_size(d):
    return load_library().moe_gmm_workspace_size(ctypes.byref(d))


def moe_weight_tiles_bytes(d, gemm):
    return load_library().moe_weight_tiles_bytes(ctypes.byref(d), gemm)


def moe_pack_weight_tiles(d, gemm, w, tiles, stream=None):
    _check("moe_pack_weight_tiles", load_library().moe_pack_weight_tiles(
        ctypes.byref(d), gemm, _p(w), _p(tiles), _stream(stream)))


def moe_layer_fwd(d, x, expert_idx, probs, w1, s1, w2, s2, out, workspace, stream=None):
    _check("moe_layer_fwd", load_library().moe_layer_fwd(
        ctypes.byref(d), _p(x), _p(expert_idx), _p(probs), _p(w1), _p(s1), _p(w2), _p(s2), _p(out),
        _p(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_layer_graph_create(d, x, expert_idx, probs, w1, s1, w2, s2, out, workspace, stream):
    """Records moe_layer_fwd on these buffers as a CUDA graph; returns the handle."""
    h = ctypes.c_void_p()
    _check("moe_layer_graph_create", load_library().moe_layer_graph_create(
        ctypes.byref(d), _p(x), _p(expert_idx), _p(probs), _p(w1), _p(s1), _p(w2), _p(s2), _p(out),
        _p(workspace), workspace.numel() * workspace.element_size(), _stream(stream), ctypes.byref(h)))
    return h


def moe_layer_graph_create_host(d, x_host, expert_idx_host, probs_host, w1, s1, w2, s2, out_host, workspace,
                                stream):
    """Records moe_layer_fwd_host (copies included, no synchronisation) as a CUDA graph."""
    h = ctypes.c_void_p()
    _check("moe_layer_graph_create_host", load_library().moe_layer_graph_create_host(
        ctypes.byref(d), _p(x_host), _p(expert_idx_host), _p(probs_host), _p(w1), _p(s1), _p(w2), _p(s2),
        _p(out_host), _p(workspace), workspace.numel() * workspace.element_size(), _stream(stream),
        ctypes.byref(h)))
    return h


def moe_layer_graph_launch(graph, stream=None):
    _check("moe_layer_graph_launch", load_library().moe_layer_graph_launch(graph, _stream(stream)))


def moe_layer_graph_destroy(graph):
    _check("moe_layer_graph_destroy", load_library().moe_layer_graph_destroy(graph))


def moe_layer_pipeline_workspace_size(d, depth):
    return load_library().moe_layer_pipeline_workspace_size(ctypes.byref(d), depth)


def moe_layer_pipeline_create(d, w1, s1, w2, s2, workspace, depth=2):
    """The pipelined host-memory executor; returns its handle."""
    h = ctypes.c_void_p()
    _check("moe_layer_pipeline_create", load_library().moe_layer_pipeline_create(
        ctypes.byref(d), _p(w1), _p(s1), _p(w2), _p(s2), _p(workspace),
        workspace.numel() * workspace.element_size(), depth, ctypes.byref(h)))
    return h


def moe_layer_pipeline_submit(pipeline, x_host, expert_idx_host, probs_host, out_host):
    """Enqueues one batch (host tensors); returns its ticket."""
    t = ctypes.c_uint64()
    _check("moe_layer_pipeline_submit", load_library().moe_layer_pipeline_submit(
        pipeline, _p(x_host), _p(expert_idx_host), _p(probs_host), _p(out_host), ctypes.byref(t)))
    return t.value


def moe_layer_pipeline_wait(pipeline, ticket):
    _check("moe_layer_pipeline_wait", load_library().moe_layer_pipeline_wait(pipeline, ticket))


def moe_layer_pipeline_destroy(pipeline):
    _check("moe_layer_pipeline_destroy", load_library().moe_layer_pipeline_destroy(pipeline))


def moe_layer_fwd_host(d, x_host, expert_idx_host, probs_host, w1, s1, w2, s2, out_host, workspace,
                       stream=None):
    _check("moe_layer_fwd_host", load_library().moe_layer_fwd_host(
        ctypes.byref(d), _p(x_host), _p(expert_idx_host), _p(probs_host), _p(w1), _p(s1), _p(w2),
        _p(s2), _p(out_host), _p(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def moe_workspace_status(workspace, stream=None):
    st = ctypes.c_int32(0)
    _check("moe_workspace_status",
           load_library().moe_workspace_status(_p(workspace), ctypes.byref(st), _stream(stream)))
    return st.value


def moe_workspace_clear_status(workspace, stream=None):
    _check("moe_workspace_clear_status",
           load_library().moe_workspace_clear_status(_p(workspace), _stream(stream)))


def moe_route_sort(d, expert_idx, sorted_src_route, expanded_row_idx, tokens_per_expert, cumsum,
                   workspace=None, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("moe_route_sort", load_library().moe_route_sort(
        ctypes.byref(d), _p(expert_idx), _p(sorted_src_route), _p(expanded_row_idx),
        _p(tokens_per_expert), _p(cumsum), _p(workspace), nbytes, _stream(stream)))


def moe_quant_tokens(d, x, expert_idx, xq_i8, xq_f16, pts1, a1_bounds, stream=None):
    _check("moe_quant_tokens", load_library().moe_quant_tokens(
        ctypes.byref(d), _p(x), _p(expert_idx), _p(xq_i8), _p(xq_f16), _p(pts1), _p(a1_bounds), _stream(stream)))


def moe_quant_dispatch(d, x, expert_idx, expanded_row_idx, a1_f16, pts1, a1_bounds, stream=None):
    _check("moe_quant_dispatch", load_library().moe_quant_dispatch(
        ctypes.byref(d), _p(x), _p(expert_idx), _p(expanded_row_idx), _p(a1_f16), _p(pts1), _p(a1_bounds),
        _stream(stream)))


def moe_front_reorder(d, x, expert_idx, sorted_src_route, expanded_row_idx, tokens_per_expert, cumsum, a1_f16,
                      pts1, a1_bounds, workspace=None, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("moe_front_reorder", load_library().moe_front_reorder(
        ctypes.byref(d), _p(x), _p(expert_idx), _p(sorted_src_route), _p(expanded_row_idx), _p(tokens_per_expert),
        _p(cumsum), _p(a1_f16), _p(pts1), _p(a1_bounds), _p(workspace), nbytes, _stream(stream)))


def moe_gmm1(d, a1_f16, sorted_src_route, cumsum, a1_bounds, w1, s1, c1, workspace, stream=None):
    _check("moe_gmm1", load_library().moe_gmm1(
        ctypes.byref(d), _p(a1_f16), _p(sorted_src_route), _p(cumsum), _p(a1_bounds), _p(w1), _p(s1), _p(c1),
        _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_swiglu_quant(d, c1, pts1, sorted_src_route, cumsum, expert_idx, q2_i8, q2_f16, pts2, q2_bounds,
                     stream=None):
    _check("moe_swiglu_quant", load_library().moe_swiglu_quant(
        ctypes.byref(d), _p(c1), _p(pts1), _p(sorted_src_route), _p(cumsum), _p(expert_idx), _p(q2_i8),
        _p(q2_f16), _p(pts2), _p(q2_bounds), _stream(stream)))


def moe_gmm1_swiglu(d, a1_f16, cumsum, a1_bounds, w1, s1, c1, pts1, sorted_src_route, expert_idx, q2_f16, pts2,
                    q2_bounds, workspace, stream=None):
    _check("moe_gmm1_swiglu", load_library().moe_gmm1_swiglu(
        ctypes.byref(d), _p(a1_f16), _p(cumsum), _p(a1_bounds), _p(w1), _p(s1), _p(c1), _p(pts1),
        _p(sorted_src_route), _p(expert_idx), _p(q2_f16), _p(pts2), _p(q2_bounds), _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_gmm2(d, q2_f16, cumsum, q2_bounds, w2, s2, c2, workspace, stream=None):
    _check("moe_gmm2", load_library().moe_gmm2(
        ctypes.byref(d), _p(q2_f16), _p(cumsum), _p(q2_bounds), _p(w2), _p(s2), _p(c2), _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_combine_unpermute(d, c2, pts2, expanded_row_idx, probs, out, stream=None):
    _check("moe_combine_unpermute", load_library().moe_combine_unpermute(
        ctypes.byref(d), _p(c2), _p(pts2), _p(expanded_row_idx), _p(probs), _p(out),
        _stream(stream)))


def moe_selftest_wait_timeout(status, limit_us, stream=None):
    """Runs the bounded-wait self-test; status (int32 device tensor) receives the code."""
    _check("moe_selftest_wait_timeout", load_library().moe_selftest_wait_timeout(
        _p(status), limit_us, _stream(stream)))


def moe_selftest_count_timeout(status, count, limit_us, stream=None):
    """Runs the bounded count-wait self-test; status and count are int32 device tensors."""
    _check("moe_selftest_count_timeout", load_library().moe_selftest_count_timeout(
        _p(status), _p(count), limit_us, _stream(stream)))


# Largest route count (M * topK) moe_route_sort_noalloc accepts (its fixed scratch).
ROUTE_SORT_NOALLOC_MAX_ROUTES = 524288

# Activation bounds arrays: int32 [E][BOUND_SEGMENTS], one entry per BOUND_SEGMENT-deep
# segment of the reduction dimension (include/moe_layer.h, "Activation bounds").
BOUND_SEGMENT = 1024
BOUND_SEGMENTS = 16


def moe_route_sort_noalloc(d, expert_idx, sorted_src_route, expanded_row_idx, tokens_per_expert,
                           cumsum, stream=None):
    """moe_route_sort without a workspace, for callers that cannot allocate device
    memory; its scratch is a fixed array inside the library (see the header)."""
    _check("moe_route_sort_noalloc", load_library().moe_route_sort_noalloc(
        ctypes.byref(d), _p(expert_idx), _p(sorted_src_route), _p(expanded_row_idx),
        _p(tokens_per_expert), _p(cumsum), _stream(stream)))


# ------------------------------------------------------------------- include/moe_mxfp4.h
# Element types and router scores (MOE_TYPE_*, MOE_SCORE_*).
TYPE_F32, TYPE_F16, TYPE_BF16 = 0, 1, 2
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
_TYPES = {"torch.float32": TYPE_F32, "torch.float16": TYPE_F16, "torch.bfloat16": TYPE_BF16}
_types = {}  # the same by torch.dtype, filled as they come (a lookup by name takes a microsecond)


def _type(t):
    k = _types.get(t.dtype)
    if k is None:
        if str(t.dtype) not in _TYPES:
            raise ValueError("float32, float16 or bfloat16 wanted; got %s" % t.dtype)
        k = _types[t.dtype] = _TYPES[str(t.dtype)]
    return k


def _rows(t):
    """Pointer and row stride (elements) of a 2-D tensor whose rows are dense."""
    shape, strides = t.shape, t.stride()
    if len(shape) != 2 or (strides[1] != 1 and shape[1] > 1):
        raise ValueError("a 2-D tensor with dense rows wanted; got shape %s, strides %s"
                         % (tuple(shape), tuple(strides)))
    return t.data_ptr(), strides[0] if shape[0] > 1 else shape[1]


def _sized(t, n, size, what):
    """Pointer of a dense array that has to hold n elements of `size` bytes."""
    if t.numel() < n or t.element_size() != size:
        raise ValueError("%s: %d elements of %d bytes wanted; got %d of %d"
                         % (what, n, size, t.numel(), t.element_size()))
    return _p(t)


class _Kind(set):
    """Element types that an array of a kind may have: given by name, filled as they come (torch.dtype)."""

    def __init__(self, name, *types):
        super().__init__()
        self.name, self.types = name, types

    def takes(self, dtype):
        if str(dtype) in self.types:
            self.add(dtype)
            return True
        return False


_BINARY16 = _Kind("binary16", "torch.float16", "torch.int16", "torch.uint16")  # also as its bits
_INT32 = _Kind("int32", "torch.int32", "torch.uint32")
_FLOAT32 = _Kind("float32", "torch.float32")


def _typed(t, n, kind, what):
    """Pointer of a dense array that has to hold n elements of a kind; raw pointers and None go on as they are."""
    if t is None or isinstance(t, int):
        return t
    if t.numel() < n or (t.dtype not in kind and not kind.takes(t.dtype)):
        raise ValueError("%s: %d elements of %s wanted; got %d of %s" % (what, n, kind.name, t.numel(), t.dtype))
    return _p(t)


def _nbytes(t):
    return t.numel() * t.element_size()


def _holding(t, n, what):
    """Pointer of a dense array of any type that has to hold n bytes."""
    if t is None or isinstance(t, int):
        return t
    if _nbytes(t) < n:
        raise ValueError("%s: %d bytes wanted; got %d" % (what, n, _nbytes(t)))
    return _p(t)


def moe_route_topk(logits, expert_idx, probs, bias=None, scoring=SCORE_SOFTMAX, renormalise=True, scale=1.0,
                   stream=None):
    """Routes of logits [M][E] (any row stride) into expert_idx, probs [M][topK]."""
    M, E = logits.shape
    topK = expert_idx.shape[1]
    p, stride = _rows(logits)
    _check("moe_route_topk", load_library().moe_route_topk(
        M, E, topK, p, _type(logits), stride, None if bias is None else _typed(bias, E, _FLOAT32, "bias"),
        scoring, 1 if renormalise else 0, scale, _typed(expert_idx, M * topK, _INT32, "expert_idx"),
        _typed(probs, M * topK, _FLOAT32, "probs"), _stream(stream)))


def moe_mxfp4_scale_words(rows, D):
    return load_library().moe_mxfp4_scale_words(rows, D)


def _scales(t, rows, D):
    return _sized(t, (D + 127) // 128 * ((rows + 3) // 4 * 4), 4, "scales")


def moe_mxfp4_quant(x, codes, scales, row_map=None, copies=1, stream=None):
    """MXFP4 rows of x [M][D] (any row stride): codes [rows][D / 2], scales of moe_mxfp4_scale_words(rows, D) words."""
    M, D = x.shape
    rows = codes.shape[0]
    p, stride = _rows(x)
    _check("moe_mxfp4_quant", load_library().moe_mxfp4_quant(
        M, D, p, _type(x), stride, None if row_map is None else _typed(row_map, M * copies, _INT32, "row_map"), copies,
        rows, _sized(codes, rows * D // 2, 1, "codes"), _scales(scales, rows, D), _stream(stream)))


def moe_mxfp4_dequant(codes, scales, out, stream=None):
    rows, D = out.shape
    _check("moe_mxfp4_dequant", load_library().moe_mxfp4_dequant(
        rows, D, _sized(codes, rows * D // 2, 1, "codes"), _scales(scales, rows, D), _p(out), _type(out),
        _stream(stream)))


def moe_mxfp4_weights_bytes(E, N, D):
    return load_library().moe_mxfp4_weights_bytes(E, N, D)


def _blocks(t, E, N, D):
    return _sized(t, max(1, moe_mxfp4_weights_bytes(E, N, D)), 1, "blocks")


def moe_mxfp4_quant_weights(w, blocks, gate_up=False, stream=None):
    """Weight blocks of w [E][N][D]."""
    E, N, D = w.shape
    _check("moe_mxfp4_quant_weights", load_library().moe_mxfp4_quant_weights(
        E, N, D, 1 if gate_up else 0, _p(w), _type(w), _blocks(blocks, E, N, D), _stream(stream)))


def moe_mxfp4_pack_weights(codes, scales, blocks, gate_up=False, stream=None):
    """Weight blocks of MXFP4 rows: codes [E][N][D / 2], scale bytes [E][N][D / 32]."""
    E, N, half = codes.shape
    _check("moe_mxfp4_pack_weights", load_library().moe_mxfp4_pack_weights(
        E, N, 2 * half, 1 if gate_up else 0, _sized(codes, E * N * half, 1, "codes"),
        _sized(scales, E * N * half // 16, 1, "scales"), _blocks(blocks, E, N, 2 * half), _stream(stream)))


def moe_mxfp4_gmm_workspace_size(R, E, N, D):
    return load_library().moe_mxfp4_gmm_workspace_size(R, E, N, D)


def moe_mxfp4_gmm(codes, scales, cumsum, w, c, workspace, stream=None):
    """c [R][N] (binary16) = rows of codes [R][D / 2] times their experts' blocks w."""
    R, N = c.shape
    E, D = cumsum.shape[0], 2 * codes.shape[1]
    _check("moe_mxfp4_gmm", load_library().moe_mxfp4_gmm(
        R, E, N, D, _sized(codes, R * D // 2, 1, "codes"), _scales(scales, R, D), _typed(cumsum, E, _INT32, "cumsum"),
        _blocks(w, E, N, D), _typed(c, R * N, _BINARY16, "c"), _p(workspace), _nbytes(workspace), _stream(stream)))


def moe_mxfp4_gmm_swiglu(codes, scales, cumsum, w, h_codes, h_scales, workspace, stream=None):
    """SwiGLU of the product with gate_up blocks w, as MXFP4 rows h_codes [R][I / 2], h_scales."""
    R, I = h_codes.shape[0], 2 * h_codes.shape[1]
    E, D = cumsum.shape[0], 2 * codes.shape[1]
    _check("moe_mxfp4_gmm_swiglu", load_library().moe_mxfp4_gmm_swiglu(
        R, E, I, D, _sized(codes, R * D // 2, 1, "codes"), _scales(scales, R, D), _typed(cumsum, E, _INT32, "cumsum"),
        _blocks(w, E, 2 * I, D), _sized(h_codes, R * I // 2, 1, "h_codes"), _scales(h_scales, R, I),
        _p(workspace), _nbytes(workspace), _stream(stream)))


def moe_mxfp4_layer_workspace_size(d):
    return load_library().moe_mxfp4_layer_workspace_size(ctypes.byref(d))


def moe_mxfp4_layer_fwd(d, x, expert_idx, probs, w1, w2, out, workspace, stream=None):
    """The expert layer of x [M][K] (binary16) on MXFP4 blocks w1 (gate_up) and w2, into out [M][K] (binary16)."""
    lib, R = load_library(), d.M * d.topK
    _check("moe_mxfp4_layer_fwd", lib.moe_mxfp4_layer_fwd(
        ctypes.byref(d), _typed(x, d.M * d.K, _BINARY16, "x"), _typed(expert_idx, R, _INT32, "expert_idx"),
        _typed(probs, R, _FLOAT32, "probs"), _holding(w1, lib.moe_mxfp4_weights_bytes(d.E, 2 * d.I, d.K), "w1"),
        _holding(w2, lib.moe_mxfp4_weights_bytes(d.E, d.K, d.I), "w2"), _typed(out, d.M * d.K, _BINARY16, "out"),
        _p(workspace), _nbytes(workspace), _stream(stream)))


def moe_selftest_mxfp4_tickets(answers, stream=None):
    """Runs the self-test of the few-token kernel's joint wait; answers: int32 device tensor [4]."""
    _check("moe_selftest_mxfp4_tickets", load_library().moe_selftest_mxfp4_tickets(_sized(answers, 4, 4, "answers"), _stream(stream)))
