"""Thin ctypes binding over libgemvfuse.so (the C ABI in include/gemvfuse.h).

Argument marshalling only: every computation runs in the library's CUDA kernels.
Arrays are passed as torch CUDA tensors (or raw integer device addresses); the
stream defaults to torch's current CUDA stream.  Importing this module loads the
library and raises ImportError if it has not been built -- there is no fallback.
"""

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgemvfuse.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libgemvfuse.so is not built (run __graft_entry__.build()): %s" % LIB_PATH)
_lib = ctypes.CDLL(LIB_PATH)

# enums (include/gemvfuse.h)
F32, F16, Q8_0, Q4_0, Q4_K = 0, 1, 2, 3, 4
EPI_NONE, EPI_SIGMOID, EPI_SILU, EPI_SILU_MUL, EPI_ADD = 0, 1, 2, 3, 4
EW_SIGMOID, EW_SILU, EW_MUL, EW_ADD = 1, 2, 3, 4
OK, ERR_INVALID, ERR_ALIAS, ERR_UNSUPPORTED, ERR_ALIGN, ERR_CUDA, ERR_TIMEOUT = 0, -1, -2, -3, -4, -5, -6
FLAG_PDL, FLAG_NO_SPLIT_K, FLAG_NO_TENSOR_CORES = 1, 2, 4
PATH_NONE, PATH_STREAM, PATH_GENERIC, PATH_TC = 0, 1, 2, 3

_vp, _i64, _i32, _u32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint32


class GfOpts(ctypes.Structure):
    _fields_ = [("ncols", _i64), ("fwht_signs", _vp), ("fwht_block", _i64), ("nsigns", _i64),
                ("view_ne", _i64 * 4), ("flags", _u32), ("fwht_workspace", _vp),
                ("rms_norm_weight", _vp), ("rms_norm_eps", ctypes.c_float)]


def _sig(name, args, res=_i32):
    f = getattr(_lib, name)
    f.argtypes = args
    f.restype = res
    return f


_gemv_fused = _sig("gemv_fused", [_vp, _i32, _vp, _i64, _i64, _i32, _vp, _vp, _vp])
_gemv_fused_ex = _sig("gemv_fused_ex", [_vp, _i32, _vp, _i64, _i64, _i32, _vp, _vp,
                                        ctypes.POINTER(GfOpts), _vp])
_gemv_glu = _sig("gemv_glu", [_vp, _vp, _i32, _vp, _i64, _i64, _vp, ctypes.POINTER(GfOpts), _vp])
_fwht_signed = _sig("fwht_signed", [_vp, _vp, _vp, _i64, _i64, _i64, _vp])
_gemv_fused_fwht_noalloc = _sig("gemv_fused_fwht_noalloc", [_vp, _i32, _vp, _i64, _i64, _i32, _vp, _vp, _i64,
                                                             _vp, _i64, _i64, _u32, _vp])
NOALLOC_MAX_WORKSPACE_FLOATS = 262144
_elementwise = _sig("gf_elementwise", [_i32, _vp, _vp, _i64, _vp, _i64, _vp])
_dequantize = _sig("gf_dequantize", [_vp, _i32, _i64, _i64, _vp, _vp])
_plan = _sig("gf_plan", [_vp, _i32, _vp, _i64, _i64, _i32, _vp, _vp, ctypes.POINTER(GfOpts),
                         ctypes.POINTER(_i64 * 8)])
_plan_glu = _sig("gf_plan_glu", [_vp, _vp, _i32, _vp, _i64, _i64, _vp, ctypes.POINTER(GfOpts),
                                 ctypes.POINTER(_i64 * 8)])
_device_status = _sig("gf_device_status", [_i32])
_selftest_wait = _sig("gf_selftest_wait_timeout", [_i64, _vp, _vp])
_status_string = _sig("gf_status_string", [_i32], ctypes.c_char_p)
_last_cuda_error = _sig("gf_last_cuda_error", [])
_version = _sig("gf_version", [])
_prepare = _sig("gf_prepare", [_vp, _i32, _vp, _i64, _i64, _i32, _vp, _vp, ctypes.POINTER(GfOpts),
                               ctypes.POINTER(_vp)])
_prepare_glu = _sig("gf_prepare_glu", [_vp, _vp, _i32, _vp, _i64, _i64, _vp, ctypes.POINTER(GfOpts),
                                       ctypes.POINTER(_vp)])
_launch_prepared = _sig("gf_launch_prepared", [ctypes.POINTER(_vp), _i32, _vp])
_free_prepared = _sig("gf_free_prepared", [_vp], None)


class MultiItem(ctypes.Structure):
    _fields_ = [("W", _vp), ("M", _i64), ("epilogue", _i32), ("aux", _vp), ("dst", _vp)]


MULTI_MAX = 4
_gemv_multi = _sig("gemv_multi", [ctypes.POINTER(MultiItem), _i32, _i32, _vp, _i64, ctypes.POINTER(GfOpts), _vp])
_prepare_multi = _sig("gf_prepare_multi", [ctypes.POINTER(MultiItem), _i32, _i32, _vp, _i64,
                                           ctypes.POINTER(GfOpts), ctypes.POINTER(_vp)])
_copy = _sig("gf_copy", [_vp, _vp, _i64, _u32, _vp])
_prepare_copy = _sig("gf_prepare_copy", [_vp, _vp, _i64, _u32, ctypes.POINTER(_vp)])
_graph_create = _sig("gf_graph_create", [ctypes.POINTER(_vp), _i32, ctypes.POINTER(_vp)])
_graph_launch = _sig("gf_graph_launch", [_vp, _vp])
_graph_free = _sig("gf_graph_free", [_vp], None)

SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1


class RouteOpts(ctypes.Structure):
    _fields_ = [("top_k", _i64), ("score", _i32), ("norm", _i32), ("scale", ctypes.c_float), ("bias", _vp),
                ("n_group", _i64), ("topk_group", _i64), ("group_top", _i32), ("ld", _i64), ("flags", _u32)]


class Experts(ctypes.Structure):
    _fields_ = [("W_gate", _vp), ("W_up", _vp), ("W_down", _vp), ("wtype", _i32), ("wtype_down", _i32), ("E", _i64),
                ("M", _i64), ("K", _i64), ("ids", _vp), ("weights", _vp), ("top_k", _i64), ("workspace", _vp),
                ("workspace_bytes", _i64), ("rms_norm_weight", _vp), ("rms_norm_eps", ctypes.c_float),
                ("flags", _u32)]


class Lora(ctypes.Structure):
    _fields_ = [("A", _vp), ("B", _vp), ("atype", _i32), ("n", _i64), ("rank", _i64), ("ids", _vp), ("scales", _vp),
                ("workspace", _vp), ("workspace_bytes", _i64)]


_route = _sig("gf_route", [_vp, _i64, _i64, ctypes.POINTER(RouteOpts), _vp, _vp, _vp])
_prepare_route = _sig("gf_prepare_route", [_vp, _i64, _i64, ctypes.POINTER(RouteOpts), _vp, _vp, ctypes.POINTER(_vp)])
_gemv_experts = _sig("gemv_experts", [ctypes.POINTER(Experts), _vp, _i64, _vp, _vp, _vp])
_prepare_experts = _sig("gf_prepare_experts", [ctypes.POINTER(Experts), _vp, _i64, _vp, _vp, ctypes.POINTER(_vp)])
_plan_experts = _sig("gf_plan_experts", [ctypes.POINTER(Experts), _vp, _i64, _vp, _vp, ctypes.POINTER(_i64 * 8)])
_plan_lora = _sig("gf_plan_lora", [_vp, _i32, _vp, _i64, _i64, _i32, _vp, _vp, ctypes.POINTER(Lora),
                                   ctypes.POINTER(GfOpts), ctypes.POINTER(_i64 * 8)])
_experts_workspace = _sig("gf_experts_workspace", [_i64] * 5, _i64)
_gemv_lora = _sig("gemv_lora", [_vp, _i32, _vp, _i64, _i64, _i32, _vp, _vp, ctypes.POINTER(Lora),
                                ctypes.POINTER(GfOpts), _vp])
_prepare_lora = _sig("gf_prepare_lora", [_vp, _i32, _vp, _i64, _i64, _i32, _vp, _vp, ctypes.POINTER(Lora),
                                         ctypes.POINTER(GfOpts), ctypes.POINTER(_vp)])
_lora_workspace = _sig("gf_lora_workspace", [_i64] * 5, _i64)

#: the raw C functions, for callers that want the status codes themselves
raw = _lib


class GemvFuseError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        msg = "%s: %s" % (what, status_string(status))
        if status == ERR_CUDA:
            msg += " (cudaError %d)" % _last_cuda_error()
        super().__init__(msg)


def status_string(status):
    return _status_string(int(status)).decode()


def version():
    return _version()


def _ptr(a):
    if a is None:
        return None
    if isinstance(a, int):
        return a
    return a.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(st, what):
    if st != OK:
        raise GemvFuseError(st, what)


def make_opts(ncols=1, fwht_signs=None, fwht_block=0, nsigns=None, view=None, pdl=False, fwht_workspace=None,
              rms_norm_weight=None, rms_norm_eps=0.0, split_k=True, tensor_cores=True):
    o = GfOpts()
    o.ncols = ncols
    o.fwht_signs = _ptr(fwht_signs)
    o.fwht_block = fwht_block
    if nsigns is None:
        nsigns = fwht_block if fwht_signs is not None and isinstance(fwht_signs, int) \
            else (fwht_signs.numel() if fwht_signs is not None else 0)
    o.nsigns = nsigns
    v = list(view or ())
    for i in range(4):
        o.view_ne[i] = v[i] if i < len(v) else 0
    o.flags = (FLAG_PDL if pdl else 0) | (0 if split_k else FLAG_NO_SPLIT_K) | \
        (0 if tensor_cores else FLAG_NO_TENSOR_CORES)
    o.fwht_workspace = _ptr(fwht_workspace)
    o.rms_norm_weight = _ptr(rms_norm_weight)
    o.rms_norm_eps = rms_norm_eps
    return o


def gemv_fused(W, wtype, x, M, K, epilogue, aux, dst, stream=None, check=True):
    st = _gemv_fused(_ptr(W), wtype, _ptr(x), M, K, epilogue, _ptr(aux), _ptr(dst), _stream(stream))
    if check:
        _check(st, "gemv_fused")
    return st


def gemv_fused_ex(W, wtype, x, M, K, epilogue, aux, dst, ncols=1, fwht_signs=None, fwht_block=0,
                  nsigns=None, view=None, pdl=False, fwht_workspace=None, rms_norm_weight=None,
                  rms_norm_eps=0.0, split_k=True, tensor_cores=True, stream=None, check=True):
    o = make_opts(ncols, fwht_signs, fwht_block, nsigns, view, pdl, fwht_workspace, rms_norm_weight,
                  rms_norm_eps, split_k, tensor_cores)
    st = _gemv_fused_ex(_ptr(W), wtype, _ptr(x), M, K, epilogue, _ptr(aux), _ptr(dst),
                        ctypes.byref(o), _stream(stream))
    if check:
        _check(st, "gemv_fused_ex")
    return st


def gemv_glu(W_gate, W_up, wtype, x, M, K, dst, ncols=1, fwht_signs=None, fwht_block=0, nsigns=None,
             view=None, pdl=False, fwht_workspace=None, rms_norm_weight=None, rms_norm_eps=0.0,
             split_k=True, stream=None, check=True):
    """dst = silu(W_gate x') * (W_up x') for each column (see include/gemvfuse.h)."""
    o = make_opts(ncols, fwht_signs, fwht_block, nsigns, view, pdl, fwht_workspace, rms_norm_weight,
                  rms_norm_eps, split_k)
    st = _gemv_glu(_ptr(W_gate), _ptr(W_up), wtype, _ptr(x), M, K, _ptr(dst), ctypes.byref(o), _stream(stream))
    if check:
        _check(st, "gemv_glu")
    return st


class Prepared:
    """A planned call (gf_prepare / gf_prepare_glu): launch() issues its kernels with no
    planning.  The buffers it was prepared with must stay allocated while it is used;
    the handle is released when the object is garbage-collected (or by close())."""

    def __init__(self, handle, keep):
        self._h = _vp(handle)
        self._keep = keep  # the options struct and tensors the handle points into

    @property
    def handle(self):
        return self._h

    def launch(self, stream=None, check=True):
        return launch_prepared([self], stream=stream, check=check)

    def close(self):
        if self._h is not None and self._h.value:
            _free_prepared(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def prepare(W, wtype, x, M, K, epilogue, aux, dst, ncols=1, fwht_signs=None, fwht_block=0, nsigns=None,
            view=None, pdl=False, fwht_workspace=None, rms_norm_weight=None, rms_norm_eps=0.0, split_k=True,
            tensor_cores=True, check=True):
    """gf_prepare: the call gemv_fused_ex(...) would make, planned once (see Prepared)."""
    o = make_opts(ncols, fwht_signs, fwht_block, nsigns, view, pdl, fwht_workspace, rms_norm_weight,
                  rms_norm_eps, split_k, tensor_cores)
    h = _vp()
    st = _prepare(_ptr(W), wtype, _ptr(x), M, K, epilogue, _ptr(aux), _ptr(dst), ctypes.byref(o), ctypes.byref(h))
    if check:
        _check(st, "gf_prepare")
    return Prepared(h.value, (W, x, aux, dst, fwht_signs, fwht_workspace, rms_norm_weight)) if st == OK else st


def prepare_glu(W_gate, W_up, wtype, x, M, K, dst, ncols=1, fwht_signs=None, fwht_block=0, nsigns=None,
                view=None, pdl=False, fwht_workspace=None, rms_norm_weight=None, rms_norm_eps=0.0, split_k=True,
                check=True):
    """gf_prepare_glu: the call gemv_glu(...) would make, planned once (see Prepared)."""
    o = make_opts(ncols, fwht_signs, fwht_block, nsigns, view, pdl, fwht_workspace, rms_norm_weight,
                  rms_norm_eps, split_k)
    h = _vp()
    st = _prepare_glu(_ptr(W_gate), _ptr(W_up), wtype, _ptr(x), M, K, _ptr(dst), ctypes.byref(o), ctypes.byref(h))
    if check:
        _check(st, "gf_prepare_glu")
    return Prepared(h.value, (W_gate, W_up, x, dst, fwht_signs, fwht_workspace, rms_norm_weight)) \
        if st == OK else st


def launch_prepared(calls, stream=None, check=True):
    """gf_launch_prepared: issue the prepared calls' kernels in order on `stream`."""
    arr = (_vp * max(1, len(calls)))(*[c.handle.value if isinstance(c, Prepared) else c for c in calls])
    st = _launch_prepared(arr, len(calls), _stream(stream))
    if check:
        _check(st, "gf_launch_prepared")
    return st


class Graph:
    """gf_graph_create: prepared calls recorded as one CUDA graph; launch() replays it."""

    def __init__(self, calls, check=True):
        arr = (_vp * max(1, len(calls)))(*[c.handle.value if isinstance(c, Prepared) else c for c in calls])
        h = _vp()
        st = _graph_create(arr, len(calls), ctypes.byref(h))
        if check:
            _check(st, "gf_graph_create")
        self.status = st
        self._h = h if st == OK else None
        self._keep = list(calls)

    def launch(self, stream=None, check=True):
        st = _graph_launch(self._h, _stream(stream))
        if check:
            _check(st, "gf_graph_launch")
        return st

    def close(self):
        if self._h is not None and self._h.value:
            _graph_free(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _multi_items(items):
    arr = (MultiItem * max(1, len(items)))()
    for i, (W, M, epi, aux, dst) in enumerate(items):
        arr[i].W, arr[i].M, arr[i].epilogue, arr[i].aux, arr[i].dst = _ptr(W), M, epi, _ptr(aux), _ptr(dst)
    return arr


def gemv_multi(items, wtype, x, K, ncols=1, fwht_signs=None, fwht_block=0, nsigns=None, pdl=False,
               fwht_workspace=None, rms_norm_weight=None, rms_norm_eps=0.0, stream=None, check=True):
    """dst_i = epilogue_i(W_i x') for items [(W, M, epilogue, aux, dst), ...] sharing x, in one
    pass (see include/gemvfuse.h)."""
    o = make_opts(ncols, fwht_signs, fwht_block, nsigns, None, pdl, fwht_workspace, rms_norm_weight, rms_norm_eps)
    st = _gemv_multi(_multi_items(items), len(items), wtype, _ptr(x), K, ctypes.byref(o), _stream(stream))
    if check:
        _check(st, "gemv_multi")
    return st


def prepare_multi(items, wtype, x, K, ncols=1, fwht_signs=None, fwht_block=0, nsigns=None, pdl=False,
                  fwht_workspace=None, rms_norm_weight=None, rms_norm_eps=0.0, check=True):
    """gf_prepare_multi: the call gemv_multi(...) would make, planned once (see Prepared)."""
    o = make_opts(ncols, fwht_signs, fwht_block, nsigns, None, pdl, fwht_workspace, rms_norm_weight, rms_norm_eps)
    h = _vp()
    st = _prepare_multi(_multi_items(items), len(items), wtype, _ptr(x), K, ctypes.byref(o), ctypes.byref(h))
    if check:
        _check(st, "gf_prepare_multi")
    return Prepared(h.value, (items, x, fwht_signs, fwht_workspace, rms_norm_weight)) if st == OK else st


def gemv_fused_fwht_noalloc(W, wtype, x, M, K, epilogue, aux, dst, ncols, fwht_signs, fwht_block, nsigns=None,
                            pdl=False, stream=None, check=True):
    """gemv_fused_ex with the signed-FWHT prologue, its workspace taken from the library's
    static device array (for callers that cannot allocate one); see include/gemvfuse.h."""
    if nsigns is None:
        nsigns = fwht_block if isinstance(fwht_signs, int) else fwht_signs.numel()
    st = _gemv_fused_fwht_noalloc(_ptr(W), wtype, _ptr(x), M, K, epilogue, _ptr(aux), _ptr(dst), ncols,
                                  _ptr(fwht_signs), fwht_block, nsigns, FLAG_PDL if pdl else 0, _stream(stream))
    if check:
        _check(st, "gemv_fused_fwht_noalloc")
    return st


def fwht_signed(x, signs, dst, n, block, nsigns=None, stream=None, check=True):
    if nsigns is None:
        nsigns = 0 if signs is None else (block if isinstance(signs, int) else signs.numel())
    st = _fwht_signed(_ptr(x), _ptr(signs), _ptr(dst), n, block, nsigns, _stream(stream))
    if check:
        _check(st, "fwht_signed")
    return st


def elementwise(op, a, b, dst, n, nb=None, stream=None, check=True):
    if nb is None:
        nb = n if b is None or isinstance(b, int) else b.numel()
    st = _elementwise(op, _ptr(a), _ptr(b), nb, _ptr(dst), n, _stream(stream))
    if check:
        _check(st, "gf_elementwise")
    return st


def dequantize(W, wtype, M, K, out, stream=None, check=True):
    st = _dequantize(_ptr(W), wtype, M, K, _ptr(out), _stream(stream))
    if check:
        _check(st, "gf_dequantize")
    return st


def plan(W, wtype, x, M, K, epilogue, aux, dst, **opts):
    """(path, info) without launching: path 1 = TMA-streamed, 2 = generic, <0 = error."""
    o = make_opts(**opts)
    info = (_i64 * 8)()
    path = _plan(_ptr(W), wtype, _ptr(x), M, K, epilogue, _ptr(aux), _ptr(dst), ctypes.byref(o),
                 ctypes.byref(info))
    return path, dict(zip(_PLAN_KEYS, list(info)))


_PLAN_KEYS = ("grid", "threads", "stage_rows", "stages", "k_chunk", "smem", "row_chunk", "split")


def plan_glu(W_gate, W_up, wtype, x, M, K, dst, **opts):
    """plan() for gemv_glu."""
    o = make_opts(**opts)
    info = (_i64 * 8)()
    path = _plan_glu(_ptr(W_gate), _ptr(W_up), wtype, _ptr(x), M, K, _ptr(dst), ctypes.byref(o),
                     ctypes.byref(info))
    return path, dict(zip(_PLAN_KEYS, list(info)))


def selftest_wait_timeout(limit_us, out, stream=None, check=True):
    """Run the bounded-wait failure self-test (see include/gemvfuse.h); out: device int32[4]."""
    st = _selftest_wait(int(limit_us), _ptr(out), _stream(stream))
    if check:
        _check(st, "gf_selftest_wait_timeout")
    return st


_repair_count = _sig("gf_repair_count", [_i32], _i64)


def repair_count(reset=False):
    """gf_repair_count: row chunks recomputed in fp32 by the integer-path kernels."""
    return _repair_count(1 if reset else 0)


def device_status(reset=False):
    return _device_status(1 if reset else 0)


def last_cuda_error():
    return _last_cuda_error()


def copy(dst, src, nbytes, pdl=False, stream=None, check=True):
    """gf_copy: nbytes from src to dst by a kernel (device memory, or host memory the
    device addresses, e.g. a pinned tensor)."""
    st = _copy(_ptr(dst), _ptr(src), nbytes, FLAG_PDL if pdl else 0, _stream(stream))
    if check:
        _check(st, "gf_copy")
    return st


def prepare_copy(dst, src, nbytes, pdl=False, check=True):
    """gf_prepare_copy: the copy gf_copy would launch, as a prepared call (a graph may hold
    it beside the GEMVs)."""
    h = _vp()
    st = _prepare_copy(_ptr(dst), _ptr(src), nbytes, FLAG_PDL if pdl else 0, ctypes.byref(h))
    if check:
        _check(st, "gf_prepare_copy")
    return Prepared(h.value, (dst, src)) if st == OK else st


# ---- products whose weights are chosen per column

def _nbytes(a, given):
    if given is not None:
        return given
    return 0 if a is None or isinstance(a, int) else a.numel() * a.element_size()


def _route_opts(top_k, score, bias, n_group, topk_group, group_top, norm, scale, ld, pdl):
    return RouteOpts(top_k, score, 1 if norm else 0, scale, _ptr(bias), n_group, topk_group, group_top, ld,
                     FLAG_PDL if pdl else 0)


def route(logits, T, E, top_k, ids, weights, score=SCORE_SOFTMAX, bias=None, n_group=1, topk_group=1, group_top=2,
          norm=True, scale=1.0, ld=0, pdl=False, stream=None, check=True):
    """gf_route: the top_k experts of each of T tokens and their weights (see include/gemvfuse.h)."""
    o = _route_opts(top_k, score, bias, n_group, topk_group, group_top, norm, scale, ld, pdl)
    st = _route(_ptr(logits), T, E, ctypes.byref(o), _ptr(ids), _ptr(weights), _stream(stream))
    if check:
        _check(st, "gf_route")
    return st


def prepare_route(logits, T, E, top_k, ids, weights, score=SCORE_SOFTMAX, bias=None, n_group=1, topk_group=1,
                  group_top=2, norm=True, scale=1.0, ld=0, pdl=False, check=True):
    """gf_prepare_route: the call route(...) would make, planned once (see Prepared)."""
    o = _route_opts(top_k, score, bias, n_group, topk_group, group_top, norm, scale, ld, pdl)
    h = _vp()
    st = _prepare_route(_ptr(logits), T, E, ctypes.byref(o), _ptr(ids), _ptr(weights), ctypes.byref(h))
    if check:
        _check(st, "gf_prepare_route")
    return Prepared(h.value, (logits, ids, weights, bias)) if st == OK else st


def experts_workspace(E, T, top_k, M, K):
    """Bytes of workspace gemv_experts needs for these sizes."""
    n = _experts_workspace(E, T, top_k, M, K)
    if n < 0:
        raise GemvFuseError(n, "gf_experts_workspace")
    return n


def _experts_struct(W_gate, W_up, wtype, W_down, wtype_down, E, M, K, ids, weights, top_k, workspace,
                    workspace_bytes, rms_norm_weight, rms_norm_eps, pdl, tensor_cores):
    return Experts(_ptr(W_gate), _ptr(W_up), _ptr(W_down), wtype, wtype_down, E, M, K, _ptr(ids), _ptr(weights),
                   top_k, _ptr(workspace), _nbytes(workspace, workspace_bytes), _ptr(rms_norm_weight), rms_norm_eps,
                   (FLAG_PDL if pdl else 0) | (0 if tensor_cores else FLAG_NO_TENSOR_CORES))


def gemv_experts(W_gate, W_up, wtype, W_down, wtype_down, E, x, M, K, ids, weights, T, top_k, aux, dst, workspace,
                 workspace_bytes=None, rms_norm_weight=None, rms_norm_eps=0.0, pdl=False, stream=None, check=True,
                 tensor_cores=True):
    """dst_t = aux_t + sum_j weights_tj Wd_e (silu(Wg_e x'_t) * (Wu_e x'_t)), e = ids_tj (see
    include/gemvfuse.h)."""
    ex = _experts_struct(W_gate, W_up, wtype, W_down, wtype_down, E, M, K, ids, weights, top_k, workspace,
                         workspace_bytes, rms_norm_weight, rms_norm_eps, pdl, tensor_cores)
    st = _gemv_experts(ctypes.byref(ex), _ptr(x), T, _ptr(aux), _ptr(dst), _stream(stream))
    if check:
        _check(st, "gemv_experts")
    return st


def prepare_experts(W_gate, W_up, wtype, W_down, wtype_down, E, x, M, K, ids, weights, T, top_k, aux, dst, workspace,
                    workspace_bytes=None, rms_norm_weight=None, rms_norm_eps=0.0, pdl=False, check=True,
                    tensor_cores=True):
    """gf_prepare_experts: the call gemv_experts(...) would make, planned once (see Prepared)."""
    ex = _experts_struct(W_gate, W_up, wtype, W_down, wtype_down, E, M, K, ids, weights, top_k, workspace,
                         workspace_bytes, rms_norm_weight, rms_norm_eps, pdl, tensor_cores)
    h = _vp()
    st = _prepare_experts(ctypes.byref(ex), _ptr(x), T, _ptr(aux), _ptr(dst), ctypes.byref(h))
    if check:
        _check(st, "gf_prepare_experts")
    return Prepared(h.value, (W_gate, W_up, W_down, x, ids, weights, aux, dst, workspace,
                              rms_norm_weight)) if st == OK else st


def plan_experts(W_gate, W_up, wtype, W_down, wtype_down, E, x, M, K, ids, weights, T, top_k, aux, dst, workspace,
                 workspace_bytes=None, rms_norm_weight=None, rms_norm_eps=0.0, pdl=False, tensor_cores=True):
    """gf_plan_experts: (path, info) of gemv_experts(...) without launching: path 0 = nothing to launch,
    2 = generic, 4 = tiled, <0 = error; info: columns of a group, whether gate and up, and down, run on
    the wide kernel."""
    ex = _experts_struct(W_gate, W_up, wtype, W_down, wtype_down, E, M, K, ids, weights, top_k, workspace,
                         workspace_bytes, rms_norm_weight, rms_norm_eps, pdl, tensor_cores)
    info = (_i64 * 8)()
    path = _plan_experts(ctypes.byref(ex), _ptr(x), T, _ptr(aux), _ptr(dst), ctypes.byref(info))
    return path, dict(cols=info[0], wide=bool(info[1]), wide_down=bool(info[2]))


def lora_workspace(ncols, M, K, rank, n):
    """Bytes of workspace gemv_lora needs for these sizes."""
    b = _lora_workspace(ncols, M, K, rank, n)
    if b < 0:
        raise GemvFuseError(b, "gf_lora_workspace")
    return b


def gemv_lora(W, wtype, x, M, K, epilogue, aux, dst, A, B, atype, n, rank, ids, scales, workspace,
              workspace_bytes=None, stream=None, check=True, **opts):
    """dst_c = tail(W x'_c + scales_a B_a (A_a x'_c), aux_c), a = ids_c; opts as make_opts (see
    include/gemvfuse.h)."""
    o = make_opts(**opts)
    lo = Lora(_ptr(A), _ptr(B), atype, n, rank, _ptr(ids), _ptr(scales), _ptr(workspace),
              _nbytes(workspace, workspace_bytes))
    st = _gemv_lora(_ptr(W), wtype, _ptr(x), M, K, epilogue, _ptr(aux), _ptr(dst), ctypes.byref(lo), ctypes.byref(o),
                    _stream(stream))
    if check:
        _check(st, "gemv_lora")
    return st


def prepare_lora(W, wtype, x, M, K, epilogue, aux, dst, A, B, atype, n, rank, ids, scales, workspace,
                 workspace_bytes=None, check=True, **opts):
    """gf_prepare_lora: the call gemv_lora(...) would make, planned once (see Prepared)."""
    o = make_opts(**opts)
    lo = Lora(_ptr(A), _ptr(B), atype, n, rank, _ptr(ids), _ptr(scales), _ptr(workspace),
              _nbytes(workspace, workspace_bytes))
    h = _vp()
    st = _prepare_lora(_ptr(W), wtype, _ptr(x), M, K, epilogue, _ptr(aux), _ptr(dst), ctypes.byref(lo),
                       ctypes.byref(o), ctypes.byref(h))
    if check:
        _check(st, "gf_prepare_lora")
    return Prepared(h.value, (W, x, aux, dst, A, B, ids, scales, workspace, opts)) if st == OK else st


def plan_lora(W, wtype, x, M, K, epilogue, aux, dst, A, B, atype, n, rank, ids, scales, workspace,
              workspace_bytes=None, **opts):
    """gf_plan_lora: (path, info) of the shared product of gemv_lora(...) without launching: plan()'s, or
    path 4 = tiled with info: columns of a group, whether it runs on the wide kernel."""
    o = make_opts(**opts)
    lo = Lora(_ptr(A), _ptr(B), atype, n, rank, _ptr(ids), _ptr(scales), _ptr(workspace),
              _nbytes(workspace, workspace_bytes))
    info = (_i64 * 8)()
    path = _plan_lora(_ptr(W), wtype, _ptr(x), M, K, epilogue, _ptr(aux), _ptr(dst), ctypes.byref(lo), ctypes.byref(o),
                      ctypes.byref(info))
    return path, dict(cols=info[0], wide=bool(info[1])) if path == 4 else dict(zip(_PLAN_KEYS, list(info)))


# ---- attention over an 8-bit cache

ROPE_HALVES, ROPE_PAIRS = 0, 1
ROPE_PLAIN, ROPE_LINEAR, ROPE_RAMP, ROPE_BANDS = 0, 1, 2, 3
CACHE_I8, CACHE_E4M3 = 0, 1


class RopeFreqs(ctypes.Structure):
    _fields_ = [("base", ctypes.c_double), ("kind", _i32), ("factor", ctypes.c_double), ("span", _i64),
                ("fast", ctypes.c_double), ("slow", ctypes.c_double), ("magnitude", ctypes.c_double), ("divisors", _vp)]


class RopeOpts(ctypes.Structure):
    _fields_ = [("table", _vp), ("n_rot", _i64), ("layout", _i32), ("type", _i32), ("ld", _i64), ("ld_dst", _i64),
                ("flags", _u32)]


class GfCache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("format", _i32), ("n_pages", _i64),
                ("heads", _i64), ("page", _i64), ("dim", _i64), ("block", _i64), ("table", _vp), ("n_seqs", _i64),
                ("table_ld", _i64)]


class StoreOpts(ctypes.Structure):
    _fields_ = [("type", _i32), ("ldk", _i64), ("ldv", _i64), ("rope", ctypes.POINTER(RopeOpts)), ("q", _vp),
                ("q_dst", _vp), ("q_heads", _i64), ("ldq", _i64), ("ld_q_dst", _i64), ("flags", _u32)]


class LoadOpts(ctypes.Structure):
    _fields_ = [("type", _i32), ("ldk", _i64), ("ldv", _i64), ("flags", _u32)]


class AttendOpts(ctypes.Structure):
    _fields_ = [("type", _i32), ("ldq", _i64), ("ld_dst", _i64), ("scale", ctypes.c_float), ("window", _i64),
                ("run", _i64), ("lse", _vp), ("workspace", _vp), ("workspace_bytes", _i64), ("flags", _u32)]


_cachep, _out = ctypes.POINTER(GfCache), ctypes.POINTER(_vp)
_rope_table_bytes = _sig("gf_rope_table_bytes", [_i64], _i64)
_rope_table = _sig("gf_rope_table", [_vp, _i64, ctypes.POINTER(RopeFreqs), _vp])
_rope = _sig("gf_rope", [_vp, _i64, _i64, _i64, _vp, ctypes.POINTER(RopeOpts), _vp, _vp])
_prepare_rope = _sig("gf_prepare_rope", [_vp, _i64, _i64, _i64, _vp, ctypes.POINTER(RopeOpts), _vp, _out])
_cache_store = _sig("gf_cache_store", [_cachep, _vp, _vp, _i64, _vp, _vp, ctypes.POINTER(StoreOpts), _vp])
_prepare_cache_store = _sig("gf_prepare_cache_store", [_cachep, _vp, _vp, _i64, _vp, _vp, ctypes.POINTER(StoreOpts), _out])
_cache_load = _sig("gf_cache_load", [_cachep, _i64, _vp, _vp, ctypes.POINTER(LoadOpts), _vp, _vp, _vp])
_prepare_cache_load = _sig("gf_prepare_cache_load", [_cachep, _i64, _vp, _vp, ctypes.POINTER(LoadOpts), _vp, _vp, _out])
_attend = _sig("gf_attend", [_cachep, _vp, _i64, _i64, _vp, _vp, ctypes.POINTER(AttendOpts), _vp, _vp])
_prepare_attend = _sig("gf_prepare_attend", [_cachep, _vp, _i64, _i64, _vp, _vp, ctypes.POINTER(AttendOpts), _vp, _out])
_attend_workspace = _sig("gf_attend_workspace", [_i64] * 5, _i64)


def rope_table_bytes(n_rot):
    """Bytes of the table that rope_table fills for n_rot rotated elements of a head."""
    n = _rope_table_bytes(n_rot)
    if n < 0:
        raise GemvFuseError(n, "gf_rope_table_bytes")
    return n


def rope_table(table, n_rot, base=10000.0, kind=ROPE_PLAIN, factor=1.0, span=0, fast=32.0, slow=1.0, magnitude=0.0,
               divisors=None, stream=None, check=True):
    """gf_rope_table: the frequencies of rotary positions, made once (see include/gemvfuse.h)."""
    f = RopeFreqs(base, kind, factor, span, fast, slow, magnitude, _ptr(divisors))
    st = _rope_table(_ptr(table), n_rot, ctypes.byref(f), _stream(stream))
    if check:
        _check(st, "gf_rope_table")
    return st


def rope(x, T, heads, dim, pos, table, dst, n_rot=0, layout=ROPE_HALVES, type=F32, ld=0, ld_dst=0, pdl=False, stream=None,
         check=True):
    """gf_rope: dst = x [T][heads][dim] rotated by the tokens' positions (see include/gemvfuse.h)."""
    o = RopeOpts(_ptr(table), n_rot, layout, type, ld, ld_dst, FLAG_PDL if pdl else 0)
    st = _rope(_ptr(x), T, heads, dim, _ptr(pos), ctypes.byref(o), _ptr(dst), _stream(stream))
    if check:
        _check(st, "gf_rope")
    return st


def prepare_rope(x, T, heads, dim, pos, table, dst, n_rot=0, layout=ROPE_HALVES, type=F32, ld=0, ld_dst=0, pdl=False,
                 check=True):
    """gf_prepare_rope: the call rope(...) would make, planned once (see Prepared)."""
    o = RopeOpts(_ptr(table), n_rot, layout, type, ld, ld_dst, FLAG_PDL if pdl else 0)
    h = _vp()
    st = _prepare_rope(_ptr(x), T, heads, dim, _ptr(pos), ctypes.byref(o), _ptr(dst), ctypes.byref(h))
    if check:
        _check(st, "gf_prepare_rope")
    return Prepared(h.value, (x, pos, table, dst)) if st == OK else st


class Cache:
    """The arrays of an 8-bit cache and their sizes (gf_cache, see include/gemvfuse.h); keeps them alive."""

    def __init__(self, k, v, k_scale, v_scale, format, n_pages, heads, page, dim, block, table, n_seqs, table_ld):
        self.keep = (k, v, k_scale, v_scale, table)
        self.struct = GfCache(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), format, n_pages, heads, page, dim, block,
                              _ptr(table), n_seqs, table_ld)


def _store_opts(type, ldk, ldv, rope, n_rot, layout, q, q_heads, ldq, q_dst, ld_q_dst, pdl):
    turn = None if rope is None else ctypes.pointer(RopeOpts(_ptr(rope), n_rot, layout, type, 0, 0, 0))
    return StoreOpts(type, ldk, ldv, turn, _ptr(q), _ptr(q_dst), q_heads, ldq, ld_q_dst, FLAG_PDL if pdl else 0)


def cache_store(cache, k, v, T, seq, pos, type=F32, ldk=0, ldv=0, rope=None, n_rot=0, layout=ROPE_HALVES, q=None, q_heads=0,
                ldq=0, q_dst=None, ld_q_dst=0, pdl=False, stream=None, check=True):
    """gf_cache_store: T tokens' keys and values quantised into the cache; with `rope` (a table) keys, and
    queries q into q_dst, are rotated first (see include/gemvfuse.h)."""
    o = _store_opts(type, ldk, ldv, rope, n_rot, layout, q, q_heads, ldq, q_dst, ld_q_dst, pdl)
    st = _cache_store(ctypes.byref(cache.struct), _ptr(k), _ptr(v), T, _ptr(seq), _ptr(pos), ctypes.byref(o),
                      _stream(stream))
    if check:
        _check(st, "gf_cache_store")
    return st


def prepare_cache_store(cache, k, v, T, seq, pos, type=F32, ldk=0, ldv=0, rope=None, n_rot=0, layout=ROPE_HALVES, q=None,
                        q_heads=0, ldq=0, q_dst=None, ld_q_dst=0, pdl=False, check=True):
    """gf_prepare_cache_store: the call cache_store(...) would make, planned once (see Prepared)."""
    o = _store_opts(type, ldk, ldv, rope, n_rot, layout, q, q_heads, ldq, q_dst, ld_q_dst, pdl)
    h = _vp()
    st = _prepare_cache_store(ctypes.byref(cache.struct), _ptr(k), _ptr(v), T, _ptr(seq), _ptr(pos), ctypes.byref(o),
                              ctypes.byref(h))
    if check:
        _check(st, "gf_prepare_cache_store")
    return Prepared(h.value, (cache, k, v, seq, pos, rope, q, q_dst)) if st == OK else st


def cache_load(cache, T, seq, pos, k, v, type=F32, ldk=0, ldv=0, pdl=False, stream=None, check=True):
    """gf_cache_load: T tokens' keys and values read back into k, v (see include/gemvfuse.h)."""
    o = LoadOpts(type, ldk, ldv, FLAG_PDL if pdl else 0)
    st = _cache_load(ctypes.byref(cache.struct), T, _ptr(seq), _ptr(pos), ctypes.byref(o), _ptr(k), _ptr(v),
                     _stream(stream))
    if check:
        _check(st, "gf_cache_load")
    return st


def prepare_cache_load(cache, T, seq, pos, k, v, type=F32, ldk=0, ldv=0, pdl=False, check=True):
    """gf_prepare_cache_load: the call cache_load(...) would make, planned once (see Prepared)."""
    o = LoadOpts(type, ldk, ldv, FLAG_PDL if pdl else 0)
    h = _vp()
    st = _prepare_cache_load(ctypes.byref(cache.struct), T, _ptr(seq), _ptr(pos), ctypes.byref(o), _ptr(k), _ptr(v),
                             ctypes.byref(h))
    if check:
        _check(st, "gf_prepare_cache_load")
    return Prepared(h.value, (cache, k, v, seq, pos)) if st == OK else st


def attend_workspace(T, q_heads, heads, dim, run=1):
    """Bytes of workspace attend needs for these sizes."""
    n = _attend_workspace(T, q_heads, heads, dim, run)
    if n < 0:
        raise GemvFuseError(n, "gf_attend_workspace")
    return n


def attend(cache, q, T, q_heads, seq, pos, dst, workspace, type=F32, ldq=0, ld_dst=0, scale=0.0, window=0, run=1, lse=None,
           workspace_bytes=None, pdl=False, stream=None, check=True):
    """gf_attend: attention of T tokens' queries over the cache (see include/gemvfuse.h)."""
    o = AttendOpts(type, ldq, ld_dst, scale, window, run, _ptr(lse), _ptr(workspace), _nbytes(workspace, workspace_bytes),
                   FLAG_PDL if pdl else 0)
    st = _attend(ctypes.byref(cache.struct), _ptr(q), T, q_heads, _ptr(seq), _ptr(pos), ctypes.byref(o), _ptr(dst),
                 _stream(stream))
    if check:
        _check(st, "gf_attend")
    return st


def prepare_attend(cache, q, T, q_heads, seq, pos, dst, workspace, type=F32, ldq=0, ld_dst=0, scale=0.0, window=0, run=1,
                   lse=None, workspace_bytes=None, pdl=False, check=True):
    """gf_prepare_attend: the call attend(...) would make, planned once (see Prepared)."""
    o = AttendOpts(type, ldq, ld_dst, scale, window, run, _ptr(lse), _ptr(workspace), _nbytes(workspace, workspace_bytes),
                   FLAG_PDL if pdl else 0)
    h = _vp()
    st = _prepare_attend(ctypes.byref(cache.struct), _ptr(q), T, q_heads, _ptr(seq), _ptr(pos), ctypes.byref(o),
                         _ptr(dst), ctypes.byref(h))
    if check:
        _check(st, "gf_prepare_attend")
    return Prepared(h.value, (cache, q, seq, pos, dst, workspace, lse)) if st == OK else st
