"""Python binding of libkd.so, the batched multi-session decode step for GB300.

Argument marshalling only: every function here has the name of the C entry
point it calls (include/kd.h), converts numpy arrays / torch tensors / streams
into pointers, and raises KdError on a non-zero status.  All the step's work
runs in the library's CUDA kernels; there is no fallback path.  PyTorch is used
only to hand over device memory and streams.
"""
from __future__ import annotations

import ctypes as C
import importlib.machinery
import importlib.util
import operator
import sys
from pathlib import Path

import numpy as np

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "libkd.so"
CALL_PATH = _PKG / ("_kdcall" + importlib.machinery.EXTENSION_SUFFIXES[0])

KD_MAX_BATCH = 16
KD_ATTN_NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024
KD_FLAG_NO_GRAPH = 1
KD_FLAG_SCHEDULE_STREAM = 2
KD_FLAG_SCHEDULE_GROUP = 4
KD_FLAG_FUSED_NORM = 32
KD_FLAG_UNFUSED = 64
KD_FLAG_KV_Q8_0 = 128
STATUS = {0: "KD_OK", -1: "KD_ERR_INVALID_ARG", -2: "KD_ERR_OOM", -3: "KD_ERR_CUDA",
          -4: "KD_ERR_NO_FREE_SLOT", -5: "KD_ERR_BAD_SESSION", -6: "KD_ERR_POSITION",
          -7: "KD_ERR_BATCH", -8: "KD_ERR_UNSUPPORTED", -9: "KD_ERR_DEVICE"}


class KdError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status
        self.name = STATUS.get(status, str(status))


class KdConfig(C.Structure):
    _fields_ = [("n_layers", C.c_int32), ("hidden", C.c_int32), ("n_heads", C.c_int32),
                ("n_kv_heads", C.c_int32), ("head_dim", C.c_int32), ("ffn", C.c_int32),
                ("vocab", C.c_int32), ("rope_theta", C.c_float), ("rms_eps", C.c_float),
                ("max_sessions", C.c_int32), ("max_ctx", C.c_int32), ("flags", C.c_int32)]


_vp = C.c_void_p
_vpp = C.POINTER(C.c_void_p)
_fp = C.POINTER(C.c_float)
_fpp = C.POINTER(_fp)


class KdWeights(C.Structure):
    _fields_ = [("tok_embd", _vp), ("output", _vp), ("output_norm", _fp),
                ("wq", _vpp), ("wk", _vpp), ("wv", _vpp), ("wo", _vpp),
                ("w_gate", _vpp), ("w_up", _vpp), ("w_down", _vpp),
                ("attn_norm", _fpp), ("ffn_norm", _fpp)]


KD_ROPE_MAX_DIM = 256
KD_ROPE_HALF, KD_ROPE_PAIRS = 0, 1
KD_ROPE_UNSCALED, KD_ROPE_LINEAR, KD_ROPE_BANDS, KD_ROPE_RAMP = 0, 1, 2, 3
KD_F32, KD_F16, KD_BF16 = 0, 1, 2
KD_PAGED_MAX_SEQS = 256
KD_PAGED_MAX_LEN = 1 << 30


class KdRopeConfig(C.Structure):
    _fields_ = [("head_dim", C.c_int32), ("rot_dim", C.c_int32), ("layout", C.c_int32), ("scaling", C.c_int32),
                ("original_ctx", C.c_int32), ("reserved", C.c_int32), ("theta", C.c_double), ("factor", C.c_double),
                ("low", C.c_double), ("high", C.c_double), ("magnitude", C.c_double)]


class KdRopeTable(C.Structure):
    _fields_ = [("head_dim", C.c_int32), ("rot_dim", C.c_int32), ("layout", C.c_int32), ("reserved", C.c_int32),
                ("magnitude", C.c_double), ("turns", C.c_uint64 * (KD_ROPE_MAX_DIM // 2))]


class KdSampleParams(C.Structure):
    _fields_ = [("temperature", C.c_float), ("reserved", C.c_uint32), ("seed", C.c_uint64), ("counter", C.c_uint64)]


def sample_params(temperatures, seeds, counters):
    """A host array of kd_sample_params from per-row temperatures, seeds and counters."""
    t = list(np.asarray(temperatures, dtype=np.float32).reshape(-1))
    arr = (KdSampleParams * len(t))()
    for i, (tt, sd, ct) in enumerate(zip(t, seeds, counters)):
        arr[i] = KdSampleParams(float(tt), 0, int(sd), int(ct))
    return arr


_lib = None


def lib():
    """Load libkd.so.  It must have been built (build.build()); nothing else will run."""
    global _lib
    if _lib is None:
        if not LIB_PATH.exists():
            raise ImportError(f"{LIB_PATH} is missing: build it with session_decode_step_gb300.build.build()")
        L = C.CDLL(str(LIB_PATH))
        i32, i32p = C.c_int32, C.POINTER(C.c_int32)
        sig = {
            "kd_model_load": [C.POINTER(KdConfig), C.POINTER(KdWeights), C.POINTER(_vp)],
            "kd_model_free": [_vp],
            "kd_session_bind": [_vp, i32p],
            "kd_session_free": [_vp, i32],
            "kd_session_load_kv": [_vp, i32, _vp, _vp, i32, _vp],
            "kd_session_length": [_vp, i32, i32p],
            "kd_decode_step": [_vp, i32p, i32p, i32p, i32, _vp, _vp, _vp],
            "kd_debug_capture_hidden": [_vp, _vp],
            "kd_debug_layer": [_vp, i32, i32p, i32p, i32, _vp, _vp, _vp],
            "kd_device_status": [_vp, i32p],
            "kd_debug_inject_wait_timeout": [_vp, i32],
            "kd_q8_matrix_status": [_vp, i32p],
            "kd_attn_device_status": [_vp, i32p, _vp],
            "kd_profile_enable": [_vp, i32],
            "kd_profile_read": [_vp, i32p, C.POINTER(C.c_double)],
            "kd_profile_timeline": [_vp, _vp, i32, i32p],
            "kd_q8_matrix_create": [_vp, i32, i32, C.POINTER(_vp)],
            "kd_q8_matrix_free": [_vp],
            "kd_mmvq": [_vp, _vp, i32, _vp, _vp],
            "kd_argmax": [_vp, i32, i32, _vp, _vp, _vp],
            "kd_sample": [_vp, i32, i32, _vp, _vp, _vp, _vp],
            "kd_decode_step_sampled": [_vp, i32p, i32p, i32p, i32, _vp, _vp, _vp, _vp],
            "kd_mmvq_schedule": [i32, i32, i32, i32p, i32p, i32p],
            "kd_attn_append_decode": [_vp, _vp, _vp, _vp, _vp, i32p, i32p, i32, i32, i32, i32, i32,
                                      i32, _vp, _vp, C.c_size_t, _vp],
            "kd_attn_append_decode_noalloc": [_vp, _vp, _vp, _vp, _vp, i32p, i32p, i32, i32, i32, i32, i32,
                                              i32, _vp, _vp],
            "kd_kv_q8_quantize": [_vp, C.c_int64, _vp, _vp, _vp],
            "kd_debug_fail_alloc": [i32, i32p],
            "kd_model_set_window": [_vp, i32, i32],
            "kd_session_reorder": [_vp, i32p, i32p, i32, _vp],
            "kd_session_fork": [_vp, i32, i32p, _vp],
            "kd_attn_window_append_decode": [_vp, _vp, _vp, _vp, _vp, i32p, i32p, i32, i32, i32, i32, i32, i32, i32, i32,
                                             _vp, _vp, C.c_size_t, _vp],
            "kd_attn_window_append_decode_q8": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, i32p, i32p, i32, i32, i32, i32, i32,
                                                i32, i32, _vp, _vp, C.c_size_t, _vp],
            "kd_beam_select": [_vp, C.c_int64, i32, i32, i32, _vp, _vp, i32, i32, _vp, _vp, _vp, _vp, _vp, C.c_size_t,
                               _vp],
            "kd_kv_reorder": [_vpp, i32p, i32, i32, i32, i32, i32, i32p, i32p, i32p, i32, i32, i32, _vp],
            "kd_debug_attn_paged_inject_wait_timeout": [i32],
            "kd_rope_plan": [C.POINTER(KdRopeConfig), C.POINTER(KdRopeTable)],
            "kd_rope": [_vp, _vp, i32, C.c_int64, _vp, i32, i32, _vp, C.c_int64, _vp],
            "kd_paged_append": [_vp, _vp, C.c_int64, _vp, C.c_int64, _vp, C.c_int64, i32, _vp, _vp, _vp, i32, i32p, i32p,
                                i32, i32, i32, i32, i32, i32, _vp, _vp, _vp],
            "kd_paged_append_q8": [_vp, _vp, C.c_int64, _vp, C.c_int64, _vp, C.c_int64, i32, _vp, _vp, _vp, _vp, _vp, i32,
                                   i32p, i32p, i32, i32, i32, i32, i32, _vp, _vp, _vp],
            "kd_attn_paged_decode": [_vp, _vp, _vp, _vp, i32, i32p, i32, i32p, i32p, i32, i32, i32, i32, i32, i32, _vp, _vp,
                                     C.c_size_t, _vp, _vp],
            "kd_attn_paged_decode_q8": [_vp, _vp, _vp, _vp, _vp, _vp, i32, i32p, i32, i32p, i32p, i32, i32, i32, i32, i32,
                                        _vp, _vp, C.c_size_t, _vp, _vp],
            "kd_attn_append_decode_q8": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, i32p, i32p, i32, i32, i32, i32, i32,
                                         _vp, _vp, C.c_size_t, _vp],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = C.c_int32
        L.kd_last_error.argtypes = []
        L.kd_last_error.restype = C.c_char_p
        L.kd_attn_workspace_bytes.argtypes = [i32, i32, i32, i32]
        L.kd_attn_workspace_bytes.restype = C.c_size_t
        L.kd_attn_window_workspace_bytes.argtypes = [i32] * 6
        L.kd_attn_window_workspace_bytes.restype = C.c_size_t
        L.kd_beam_workspace_bytes.argtypes = [i32] * 4
        L.kd_beam_workspace_bytes.restype = C.c_size_t
        L.kd_attn_paged_workspace_bytes.argtypes = [i32] * 4
        L.kd_attn_paged_workspace_bytes.restype = C.c_size_t
        L.kd_attn_paged_reads_once.argtypes = [i32] * 7
        L.kd_attn_paged_reads_once.restype = i32
        _lib = L
    return _lib


def kd_last_error() -> str:
    return lib().kd_last_error().decode()


def _check(status: int):
    if status != 0:
        raise KdError(status, kd_last_error())


def _ptr(obj):
    """Address of a numpy array, a torch tensor, an int, or None."""
    if obj is None:
        return None
    try:  # a torch tensor, the usual case, first
        if obj.is_contiguous():
            return obj.data_ptr()
    except AttributeError:
        pass
    else:
        raise ValueError("tensors passed to libkd must be contiguous")
    if isinstance(obj, int):
        return obj
    if isinstance(obj, np.ndarray):
        if not obj.flags["C_CONTIGUOUS"]:
            raise ValueError("arrays passed to libkd must be C-contiguous")
        return obj.ctypes.data
    raise TypeError(f"cannot take the address of {type(obj)}")


def _stream(stream):
    """The cudaStream_t of `stream`; None: the current stream of torch's current device (the default
    stream if torch, or its CUDA side, is not in use)."""
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream[0](_raw_stream[1]())
        torch = sys.modules.get("torch")
        if torch is None or not torch.cuda.is_initialized():
            return None
        return _current_raw_stream(torch)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_raw_stream = None  # (stream of a device, current device) of torch, once found


def _current_raw_stream(torch):
    # torch.cuda.current_stream() builds a Stream object (about 3 us); the raw handle is enough.
    global _raw_stream
    if _raw_stream is None:
        try:
            _raw_stream = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        except AttributeError:
            return torch.cuda.current_stream().cuda_stream
    stream, device = _raw_stream
    return stream(device())


def _i32(a, n=None):
    arr = np.ascontiguousarray(np.asarray(a, dtype=np.int32).reshape(-1))
    if n is not None and arr.size != n:
        raise ValueError(f"expected {n} entries, got {arr.size}")
    return arr


_I32P = C.POINTER(C.c_int32)


def _int(v, bits=32):
    v = operator.index(v)
    if not -1 << (bits - 1) <= v < 1 << (bits - 1):
        raise OverflowError(f"{v} does not fit {bits} bits")
    return v


class _CtypesCalls:
    """csrc/kd_py.c's calls through ctypes, with the same arguments, checks and errors and a few us more a
    call: where that module was not built for this interpreter."""

    @staticmethod
    def _window(fn, tensors, slots, positions, ints, out, workspace, stream):
        tensors = [_ptr(t) for t in tensors]
        slots = _i32(slots)
        positions = _i32(positions, slots.size)
        return fn(*tensors, slots.ctypes.data_as(_I32P), positions.ctypes.data_as(_I32P), slots.size, *map(_int, ints),
                  _ptr(out), _ptr(workspace), workspace.nbytes, _stream(stream))

    @classmethod
    def window(cls, q, k_new, v_new, k_cache, v_cache, slots, positions, *rest):
        *ints, out, workspace, stream = rest
        return cls._window(lib().kd_attn_window_append_decode, (q, k_new, v_new, k_cache, v_cache), slots, positions, ints,
                           out, workspace, stream)

    @classmethod
    def window_q8(cls, q, k_new, v_new, k_quants, k_scales, v_quants, v_scales, slots, positions, *rest):
        *ints, out, workspace, stream = rest
        return cls._window(lib().kd_attn_window_append_decode_q8, (q, k_new, v_new, k_quants, k_scales, v_quants, v_scales),
                           slots, positions, ints, out, workspace, stream)

    @staticmethod
    def beam(logits, ld, n_groups, n_beams, V, scores, done, eos, n_out, parents, tokens, scores_out, done_out, workspace,
             stream):
        return lib().kd_beam_select(_ptr(logits), _int(ld, 64), _int(n_groups), _int(n_beams), _int(V), _ptr(scores),
                                    _ptr(done), _int(eos), _int(n_out), _ptr(parents), _ptr(tokens), _ptr(scores_out),
                                    _ptr(done_out), _ptr(workspace), workspace.nbytes, _stream(stream))

    @staticmethod
    def reorder(planes, dst, src, lens, n_layers, n_slots, n_kv_heads, cap, window, sinks, stream):
        planes = list(planes)
        sizes = [_int(v) for v in (n_layers, n_slots, n_kv_heads, cap)]
        window, sinks = _int(window), _int(sinks)
        if min(sizes) < 1:
            raise ValueError("n_layers, n_slots, n_kv_heads and cap must be positive")
        rows = sizes[0] * sizes[1] * sizes[2] * sizes[3]
        base, width = [_ptr(t) for t in planes], [t.nbytes // rows for t in planes]
        if any(t.nbytes % rows or w >= 1 << 31 for t, w in zip(planes, width)):
            raise ValueError("a plane's size must be a whole number of bytes per row")
        dst = _i32(dst)
        src, lens = _i32(src, dst.size), _i32(lens, dst.size)
        return lib().kd_kv_reorder((C.c_void_p * len(base))(*base), (C.c_int32 * len(base))(*width), len(base), *sizes,
                                   *(a.ctypes.data_as(_I32P) for a in (dst, src, lens)), dst.size, window, sinks,
                                   _stream(stream))

    @staticmethod
    def rope(plan, x, positions, out, stream):
        px, ld, t, h, d, dtype = _heads(x, "x")
        po, ld_out, *shape, out_dtype = _heads(out, "out")
        if shape != [t, h, d] or out_dtype != dtype or (plan is not None and d != plan.head_dim):
            raise ValueError("x and out must be alike, in heads of the plan's head_dim")
        if positions.numel() != t or positions.dtype != sys.modules["torch"].int32:
            raise ValueError(f"expected {t} int32 positions")
        return lib().kd_rope(_plan(plan), px, dtype, ld, _ptr(positions), _int(t), _int(h), po, ld_out, _stream(stream))

    @staticmethod
    def append(plan, k_new, v_new, planes, table, starts, counts, n_heads, n_kv_heads, head_dim, n_pages, page_size, q, q_out,
               fault, stream):
        pk, k_ld, rows, h, d, dtype = _heads(k_new, "k_new")
        _check_planes(planes, n_kv_heads, head_dim, n_pages, page_size)
        pv, v_ld, *shape = _heads(v_new, "v_new")
        if shape != [rows, h, d, dtype] or (h, d) != (n_kv_heads, head_dim):
            raise ValueError("k_new and v_new must be alike: [rows][n_kv_heads][head_dim]")
        pq = po = None
        q_ld = 0
        if q is not None:
            pq, q_ld, *shape = _heads(q, "q")
            po, o_ld, *got = _heads(q_out, "q_out")
            if shape != [rows, n_heads, d, dtype] or got != [rows, n_heads, d, KD_F32] or o_ld != n_heads * d:
                raise ValueError("q must be [rows][n_heads][head_dim] of k_new's type, and q_out so in contiguous fp32")
        starts = _i32(starts)
        counts = _i32(counts, starts.size)
        table_ld = _table(table, starts.size)
        if min(counts, default=0) >= 0 and int(counts.sum(dtype=np.int64)) != rows:
            raise ValueError(f"{rows} new rows for counts of {int(counts.sum(dtype=np.int64))} in all")
        fn = lib().kd_paged_append if len(planes) == 2 else lib().kd_paged_append_q8
        shape = (_int(head_dim),) if len(planes) == 2 else ()
        return fn(_plan(plan), pk, k_ld, pv, v_ld, pq, q_ld, dtype, *map(_ptr, planes), _ptr(table), table_ld,
                  starts.ctypes.data_as(_I32P), counts.ctypes.data_as(_I32P), starts.size, _int(n_heads), _int(n_kv_heads),
                  *shape, _int(n_pages), _int(page_size), po, _ptr(fault), _stream(stream))

    @staticmethod
    def paged(q, planes, table, lens, group_rows, group_prefix, n_heads, n_kv_heads, head_dim, n_pages, page_size, out,
              workspace, fault, stream):
        lens = _i32(lens)
        table_ld = _table(table, lens.size)
        rows = _i32(() if group_rows is None else group_rows)
        prefix = _i32(() if group_prefix is None else group_prefix, rows.size)
        _check_size(q, 4 * lens.size * n_heads * head_dim, "q")
        _check_planes(planes, n_kv_heads, head_dim, n_pages, page_size)
        _check_size(out, 2 * lens.size * n_heads * head_dim, "out")
        fn = lib().kd_attn_paged_decode if len(planes) == 2 else lib().kd_attn_paged_decode_q8
        shape = (_int(head_dim),) if len(planes) == 2 else ()
        return fn(_ptr(q), *map(_ptr, planes), _ptr(table), table_ld, lens.ctypes.data_as(_I32P), lens.size,
                  rows.ctypes.data_as(_I32P), prefix.ctypes.data_as(_I32P), rows.size, _int(n_heads), _int(n_kv_heads),
                  *shape, _int(n_pages), _int(page_size), _ptr(out), _ptr(workspace), workspace.nbytes, _ptr(fault),
                  _stream(stream))


_dtypes = None


def _heads(x, what):
    """(address, row distance, rows, heads, head_dim, dtype) of a tensor [rows][heads][head_dim] whose heads lie
    one after another; rows may be further apart (a part of a fused projection)."""
    global _dtypes
    if _dtypes is None:
        torch = sys.modules["torch"]
        _dtypes = {torch.float32: KD_F32, torch.float16: KD_F16, torch.bfloat16: KD_BF16}
    if x.dim() == 3 and x.dtype in _dtypes:
        t, h, d = x.shape
        ld, sh, sd = x.stride()
        if (sd == 1 or d <= 1) and (sh == d or h <= 1):
            return x.data_ptr(), ld if t > 1 else max(ld, h * d), t, h, d, _dtypes[x.dtype]
    raise ValueError(f"{what} must be fp32, fp16 or bf16 [rows][heads][head_dim] with its heads one after another")


def _table(table, rows):
    """Row distance of a page table, an int32 tensor [sessions][pages]."""
    if table.dim() != 2 or table.dtype != sys.modules["torch"].int32 or table.shape[0] < rows:
        raise ValueError(f"the page table must be int32 [sessions][pages], with {rows} sessions or more")
    return _int(table.shape[1])


def _check_size(x, nbytes, what):
    if x is not None and not isinstance(x, int) and x.nbytes < nbytes:
        raise ValueError(f"{what} is smaller than the call's sizes")


def _check_planes(planes, n_kv_heads, head_dim, n_pages, page_size):
    for i, plane in enumerate(planes):
        width = 2 * head_dim if len(planes) == 2 else 8 if i & 1 else 128
        _check_size(plane, n_pages * n_kv_heads * page_size * width, "a plane of the cache")


def _plan(plan):
    return None if plan is None else C.addressof(plan)


_call = None


def _fast():
    """The marshalling module of the per-token calls (csrc/kd_py.c), beside libkd.so; ctypes without it."""
    global _call
    if _call is None:
        lib()
        call = _CtypesCalls
        if CALL_PATH.exists():  # by its path: another interpreter's module is never taken for this one's
            name = f"{__name__}._kdcall"
            spec = importlib.util.spec_from_file_location(name, CALL_PATH, loader=importlib.machinery.ExtensionFileLoader(
                name, str(CALL_PATH)))
            call = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(call)
            call.setup(_ptr, _i32, _stream)
        _call = call
    return _call


# ----------------------------------------------------------------- model ---
def make_config(shape, max_sessions: int, max_ctx: int, flags: int = 0) -> KdConfig:
    """A kd_config for a model shape (anything with the ModelShape fields)."""
    return KdConfig(shape.n_layers, shape.hidden, shape.n_heads, shape.n_kv_heads, shape.head_dim,
                    shape.ffn, shape.vocab, shape.rope_theta, shape.rms_eps, max_sessions, max_ctx,
                    flags)


def kd_model_load(cfg: KdConfig, weights: dict):
    """Load a model from host weights keyed like the synthetic generator's output."""
    L = cfg.n_layers

    def mats(name):
        return (_vp * L)(*[_ptr(weights[f"blk.{l}.{name}"]) for l in range(L)])

    keep = []  # arrays converted here must outlive the call

    def f32(a):
        a = np.ascontiguousarray(a, dtype=np.float32)
        keep.append(a)
        return C.cast(_ptr(a), _fp)

    def norms(name):
        return (_fp * L)(*[f32(weights[f"blk.{l}.{name}"]) for l in range(L)])
    w = KdWeights(_ptr(weights["tok_embd"]), _ptr(weights["output"]),
                  f32(weights["output_norm"]),
                  mats("attn_q"), mats("attn_k"), mats("attn_v"), mats("attn_output"),
                  mats("ffn_gate"), mats("ffn_up"), mats("ffn_down"),
                  norms("attn_norm"), norms("ffn_norm"))
    h = _vp()
    _check(lib().kd_model_load(C.byref(cfg), C.byref(w), C.byref(h)))
    return h


def kd_model_free(m):
    _check(lib().kd_model_free(m))


def kd_session_bind(m) -> int:
    out = C.c_int32()
    _check(lib().kd_session_bind(m, C.byref(out)))
    return out.value


def kd_session_free(m, session_id: int):
    _check(lib().kd_session_free(m, int(session_id)))


def kd_session_load_kv(m, session_id: int, k, v, length: int, stream=None):
    """k, v: [n_layers][n_kv][length][head_dim] fp16 (numpy uint16/float16 or a torch tensor)."""
    _check(lib().kd_session_load_kv(m, int(session_id), _ptr(k), _ptr(v), int(length), _stream(stream)))


def kd_session_length(m, session_id: int) -> int:
    out = C.c_int32()
    _check(lib().kd_session_length(m, int(session_id), C.byref(out)))
    return out.value


def kd_model_set_window(m, window: int, sinks: int = 0):
    """Sliding-window attention for the model's steps (window 0: every key again)."""
    _check(lib().kd_model_set_window(m, int(window), int(sinks)))


def kd_session_reorder(m, session_ids, parents, stream=None):
    """Session ids[i] becomes a copy of what session parents[i] was (-1: stays as it is), all at once."""
    ids = _i32(session_ids)
    par = _i32(parents, ids.size)
    i32p = C.POINTER(C.c_int32)
    _check(lib().kd_session_reorder(m, ids.ctypes.data_as(i32p), par.ctypes.data_as(i32p), ids.size, _stream(stream)))


def kd_session_fork(m, session_id: int, stream=None) -> int:
    """Bind a free slot as a copy of the session; returns its id."""
    out = C.c_int32()
    _check(lib().kd_session_fork(m, int(session_id), C.byref(out), _stream(stream)))
    return out.value


def kd_decode_step(m, session_ids, tokens, positions, logits_out=None, argmax_out=None, stream=None):
    """One batched step.  logits_out / argmax_out: device tensors (float32 [B][V], int32 [B]) or None."""
    ids = _i32(session_ids)
    B = ids.size
    tok, pos = _i32(tokens, B), _i32(positions, B)
    i32p = C.POINTER(C.c_int32)
    _check(lib().kd_decode_step(m, ids.ctypes.data_as(i32p), tok.ctypes.data_as(i32p),
                                pos.ctypes.data_as(i32p), B, _ptr(logits_out), _ptr(argmax_out),
                                _stream(stream)))


def kd_decode_step_sampled(m, session_ids, tokens, positions, params, logits_out=None, token_out=None, stream=None):
    """One batched step with device temperature sampling: params from sample_params(); token_out a
    device int32 [B] tensor (required)."""
    ids = _i32(session_ids)
    B = ids.size
    tok, pos = _i32(tokens, B), _i32(positions, B)
    if len(params) != B:
        raise ValueError(f"expected {B} sampling parameter rows, got {len(params)}")
    i32p = C.POINTER(C.c_int32)
    _check(lib().kd_decode_step_sampled(m, ids.ctypes.data_as(i32p), tok.ctypes.data_as(i32p),
                                        pos.ctypes.data_as(i32p), B, C.cast(params, _vp), _ptr(logits_out),
                                        _ptr(token_out), _stream(stream)))


def kd_debug_capture_hidden(m, buf):
    _check(lib().kd_debug_capture_hidden(m, _ptr(buf)))


def kd_debug_layer(m, layer: int, session_ids, positions, x_in, x_out, stream=None):
    ids = _i32(session_ids)
    pos = _i32(positions, ids.size)
    i32p = C.POINTER(C.c_int32)
    _check(lib().kd_debug_layer(m, int(layer), ids.ctypes.data_as(i32p), pos.ctypes.data_as(i32p), ids.size,
                                _ptr(x_in), _ptr(x_out), _stream(stream)))


def kd_device_status(m) -> int:
    out = C.c_int32()
    _check(lib().kd_device_status(m, C.byref(out)))
    return out.value


KERNEL_CLASSES = ("embed", "rmsnorm", "qkv", "attn_split", "attn_combine", "wo", "gate_up", "down",
                  "lm_head", "argmax")


def kd_debug_inject_wait_timeout(m, kernel_class: str):
    """Make one bounded wait of the next step's first `kernel_class` launch run out
    (a test of the device fault path; nothing faults or hangs)."""
    _check(lib().kd_debug_inject_wait_timeout(m, KERNEL_CLASSES.index(kernel_class)))


def kd_profile_enable(m, on: bool = True):
    _check(lib().kd_profile_enable(m, 1 if on else 0))


KD_TIMELINE_CTAS = 1024


def kd_profile_timeline(m, buf, max_launches: int = 0):
    """Turn the per-CTA timeline on (buf: device uint64 [max_launches][KD_TIMELINE_CTAS][4],
    zeroed) or off (buf None).  Returns the kernel class name of each launch index."""
    n = int(max_launches) if buf is not None else 0
    cls = (C.c_int32 * max(n, 1))()
    _check(lib().kd_profile_timeline(m, _ptr(buf), n, cls if n else None))
    return [KERNEL_CLASSES[c] if c >= 0 else None for c in cls[:n]]


def kd_profile_read(m) -> dict:
    """{kernel class: (launches, total ms)} since the previous read."""
    n = len(KERNEL_CLASSES)
    launches = (C.c_int32 * n)()
    ms = (C.c_double * n)()
    _check(lib().kd_profile_read(m, launches, ms))
    return {k: (launches[i], ms[i]) for i, k in enumerate(KERNEL_CLASSES)}


# -------------------------------------------------------------- op level ---
def kd_q8_matrix_create(q8_0: np.ndarray):
    """q8_0: canonical uint8 [rows][cols/32][34] in host memory."""
    rows, nb, _ = q8_0.shape
    h = _vp()
    _check(lib().kd_q8_matrix_create(_ptr(np.ascontiguousarray(q8_0)), rows, nb * 32, C.byref(h)))
    return h


def kd_q8_matrix_free(w):
    _check(lib().kd_q8_matrix_free(w))


def kd_mmvq(w, x, m: int, y, stream=None):
    _check(lib().kd_mmvq(w, _ptr(x), int(m), _ptr(y), _stream(stream)))


def kd_q8_matrix_status(w) -> int:
    out = C.c_int32()
    _check(lib().kd_q8_matrix_status(w, C.byref(out)))
    return out.value


KD_ARGMAX_WORKSPACE_BYTES = 256


def kd_mmvq_schedule(rows: int, cols: int, num_sms: int):
    """(mode, warps, share) the library picks for a rows x cols Q8_0 matrix on num_sms SMs
    (host only): mode 1 = group, 0 = stream."""
    mode, warps, share = C.c_int32(), C.c_int32(), C.c_int32()
    _check(lib().kd_mmvq_schedule(int(rows), int(cols), int(num_sms), C.byref(mode), C.byref(warps), C.byref(share)))
    return mode.value, warps.value, share.value


def kd_argmax(logits, B: int, V: int, out, workspace, stream=None):
    """logits: device fp32 [B][V]; out: device int32 [B]; workspace: KD_ARGMAX_WORKSPACE_BYTES of device memory."""
    _check(lib().kd_argmax(_ptr(logits), int(B), int(V), _ptr(out), _ptr(workspace), _stream(stream)))


KD_SAMPLE_WORKSPACE_BYTES = 1024


def kd_sample(logits, B: int, V: int, params, out, workspace, stream=None):
    """logits: device fp32 [B][V]; params: sample_params(...) of B rows; out: device int32 [B];
    workspace: KD_SAMPLE_WORKSPACE_BYTES of device memory."""
    if len(params) != B:
        raise ValueError(f"expected {B} sampling parameter rows, got {len(params)}")
    _check(lib().kd_sample(_ptr(logits), int(B), int(V), C.cast(params, _vp), _ptr(out), _ptr(workspace),
                           _stream(stream)))


def kd_attn_workspace_bytes(B: int, n_heads: int, head_dim: int, cap: int) -> int:
    return int(lib().kd_attn_workspace_bytes(B, n_heads, head_dim, cap))


def kd_attn_append_decode(q, k_new, v_new, k_cache, v_cache, slots, positions, n_heads, n_kv_heads,
                          head_dim, n_slots, cap, out, workspace, stream=None):
    sl = _i32(slots)
    B = sl.size
    ps = _i32(positions, B)
    i32p = C.POINTER(C.c_int32)
    nbytes = workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else workspace.nbytes
    _check(lib().kd_attn_append_decode(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                       sl.ctypes.data_as(i32p), ps.ctypes.data_as(i32p), B, n_heads,
                                       n_kv_heads, head_dim, n_slots, cap, _ptr(out), _ptr(workspace),
                                       nbytes, _stream(stream)))


def kd_debug_fail_alloc(nth: int) -> int:
    """Arm (nth >= 1) or disarm (0) the allocation-failure switch of the next
    kd_model_load; returns the number of allocations the last load made."""
    out = C.c_int32()
    _check(lib().kd_debug_fail_alloc(int(nth), C.byref(out)))
    return out.value


def kd_kv_q8_quantize(src, quants, scales, stream=None):
    """Rows of 128 fp32 values (device [rows][128]) into Q8_0 quants (uint8
    [rows][128], q + 128) and fp16 block scales ([rows][4], as int16/uint16 bits)."""
    rows = src.numel() // 128
    _check(lib().kd_kv_q8_quantize(_ptr(src), rows, _ptr(quants), _ptr(scales), _stream(stream)))


def kd_attn_append_decode_q8(q, k_new, v_new, k_quants, k_scales, v_quants, v_scales, slots, positions, n_heads,
                             n_kv_heads, n_slots, cap, out, workspace, stream=None):
    """kd_attn_append_decode over a Q8_0 cache of head_dim 128 (see include/kd.h)."""
    sl = _i32(slots)
    B = sl.size
    ps = _i32(positions, B)
    i32p = C.POINTER(C.c_int32)
    nbytes = workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else workspace.nbytes
    _check(lib().kd_attn_append_decode_q8(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_quants), _ptr(k_scales),
                                          _ptr(v_quants), _ptr(v_scales), sl.ctypes.data_as(i32p),
                                          ps.ctypes.data_as(i32p), B, n_heads, n_kv_heads, n_slots, cap, _ptr(out),
                                          _ptr(workspace), nbytes, _stream(stream)))


def kd_attn_window_workspace_bytes(B: int, n_heads: int, head_dim: int, cap: int, window: int, sinks: int) -> int:
    return int(lib().kd_attn_window_workspace_bytes(B, n_heads, head_dim, cap, window, sinks))


def kd_attn_window_append_decode(q, k_new, v_new, k_cache, v_cache, slots, positions, n_heads, n_kv_heads, head_dim,
                                 n_slots, cap, window, sinks, out, workspace, stream=None):
    """kd_attn_append_decode with a sliding window: row b attends t < sinks and t > positions[b] - window."""
    _check((_call or _fast()).window(q, k_new, v_new, k_cache, v_cache, slots, positions, n_heads, n_kv_heads, head_dim,
                                     n_slots, cap, window, sinks, out, workspace, stream))


def kd_attn_window_append_decode_q8(q, k_new, v_new, k_quants, k_scales, v_quants, v_scales, slots, positions, n_heads,
                                    n_kv_heads, n_slots, cap, window, sinks, out, workspace, stream=None):
    """kd_attn_window_append_decode over a Q8_0 cache of head_dim 128 (see include/kd.h)."""
    _check((_call or _fast()).window_q8(q, k_new, v_new, k_quants, k_scales, v_quants, v_scales, slots, positions, n_heads,
                                        n_kv_heads, n_slots, cap, window, sinks, out, workspace, stream))


KD_BEAM_MAX_BEAMS = 16
KD_BEAM_MAX_OUT = 32
KD_BEAM_MAX_VOCAB = 524288
KD_REORDER_MAX = 64


def kd_beam_workspace_bytes(n_groups: int, n_beams: int, V: int, n_out: int) -> int:
    return int(lib().kd_beam_workspace_bytes(n_groups, n_beams, V, n_out))


def kd_beam_select(logits, n_groups: int, n_beams: int, V: int, scores, n_out: int, parents_out, tokens_out, scores_out,
                   workspace, done=None, done_out=None, eos: int = -1, ld=None, stream=None):
    """Each group's n_out best (beam, token) continuations (see include/kd.h).  logits: device fp32
    [n_groups * n_beams] rows, `ld` (default V) apart; scores, done: device fp32 / int32 per row or None."""
    _check((_call or _fast()).beam(logits, V if ld is None else ld, n_groups, n_beams, V, scores, done, eos, n_out,
                                   parents_out, tokens_out, scores_out, done_out, workspace, stream))


def kd_kv_reorder(planes, dst, src, lens, n_layers: int, n_slots: int, n_kv_heads: int, cap: int, window: int = 0,
                  sinks: int = 0, stream=None):
    """Slot dst[i] becomes what slot src[i] was, all at once and in place.  planes: device tensors
    [n_layers][n_slots][n_kv_heads][cap][...], the trailing dimensions being a row's bytes."""
    _check((_call or _fast()).reorder(planes, dst, src, lens, n_layers, n_slots, n_kv_heads, cap, window, sinks, stream))


def kd_attn_device_status(workspace=None, stream=None) -> int:
    """Fault word of the last attention call given `workspace` (None: the last
    allocation-free call on the current device)."""
    out = C.c_int32()
    _check(lib().kd_attn_device_status(_ptr(workspace), C.byref(out), _stream(stream)))
    return out.value


def kd_attn_append_decode_noalloc(q, k_new, v_new, k_cache, v_cache, slots, positions, n_heads, n_kv_heads,
                                  head_dim, n_slots, cap, out, stream=None):
    """kd_attn_append_decode with its scratch in the library's fixed device array
    (no workspace argument, no allocation); see include/kd.h for the limits."""
    sl = _i32(slots)
    B = sl.size
    ps = _i32(positions, B)
    i32p = C.POINTER(C.c_int32)
    _check(lib().kd_attn_append_decode_noalloc(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                               sl.ctypes.data_as(i32p), ps.ctypes.data_as(i32p), B, n_heads,
                                               n_kv_heads, head_dim, n_slots, cap, _ptr(out), _stream(stream)))


# ---------------------------------------------------------- paged sessions ---
def kd_rope_plan(head_dim: int, theta: float, rot_dim=None, layout: int = KD_ROPE_HALF, scaling: int = KD_ROPE_UNSCALED,
                 factor: float = 1.0, low: float = 1.0, high: float = 4.0, original_ctx: int = 0,
                 magnitude: float = 1.0) -> KdRopeTable:
    """The table of a rotation (see include/kd.h), which the rotating calls take.  Host only."""
    cfg = KdRopeConfig(int(head_dim), int(head_dim if rot_dim is None else rot_dim), int(layout), int(scaling),
                       int(original_ctx), 0, float(theta), float(factor), float(low), float(high), float(magnitude))
    out = KdRopeTable()
    _check(lib().kd_rope_plan(C.byref(cfg), C.byref(out)))
    return out


def kd_rope(plan: KdRopeTable, x, positions, out, stream=None):
    """Rotate x [tokens][heads][head_dim] by positions (device int32 [tokens]) into out, which may be x."""
    _check((_call or _fast()).rope(plan, x, positions, out, stream))


def kd_paged_append(plan, k_new, v_new, k_pages, v_pages, table, starts, counts, n_kv_heads: int, head_dim: int,
                    n_pages: int, page_size: int, q=None, q_out=None, n_heads: int = 0, fault=None, stream=None):
    """Append k_new (rotated by `plan`; None: as it is) and v_new [rows][n_kv_heads][head_dim] to a paged fp16 cache:
    session b's counts[b] rows at positions starts[b] on; q [rows][n_heads][head_dim] rotated into q_out (fp32)."""
    _check((_call or _fast()).append(plan, k_new, v_new, (k_pages, v_pages), table, starts, counts, n_heads, n_kv_heads,
                                     head_dim, n_pages, page_size, q, q_out, fault, stream))


def kd_paged_append_q8(plan, k_new, v_new, k_quants, k_scales, v_quants, v_scales, table, starts, counts, n_kv_heads: int,
                       n_pages: int, page_size: int, q=None, q_out=None, n_heads: int = 0, fault=None, stream=None):
    """kd_paged_append to a Q8_0 cache of head_dim 128 (see include/kd.h)."""
    _check((_call or _fast()).append(plan, k_new, v_new, (k_quants, k_scales, v_quants, v_scales), table, starts, counts,
                                     n_heads, n_kv_heads, 128, n_pages, page_size, q, q_out, fault, stream))


def kd_attn_paged_workspace_bytes(B: int, n_heads: int, n_kv_heads: int, head_dim: int) -> int:
    return int(lib().kd_attn_paged_workspace_bytes(B, n_heads, n_kv_heads, head_dim))


def kd_attn_paged_reads_once(rows: int, prefix: int, n_heads: int, n_kv_heads: int, head_dim: int, page_size: int,
                             q8: bool = False) -> bool:
    """Whether the paged attention reads a group's shared prefix once for its sessions, or each session reads it."""
    return bool(lib().kd_attn_paged_reads_once(rows, prefix, n_heads, n_kv_heads, head_dim, page_size, q8))


def kd_attn_paged_decode(q, k_pages, v_pages, table, lens, n_heads: int, n_kv_heads: int, head_dim: int, n_pages: int,
                         page_size: int, out, workspace, group_rows=None, group_prefix=None, fault=None, stream=None):
    """Attention of one query per session over a paged fp16 cache: session b sees its first lens[b] keys.  Sessions in
    order form groups of group_rows[g], whose first group_prefix[g] keys are shared and read once (see include/kd.h)."""
    _check((_call or _fast()).paged(q, (k_pages, v_pages), table, lens, group_rows, group_prefix,
                                    n_heads, n_kv_heads, head_dim, n_pages, page_size, out, workspace, fault, stream))


def kd_attn_paged_decode_q8(q, k_quants, k_scales, v_quants, v_scales, table, lens, n_heads: int, n_kv_heads: int,
                            n_pages: int, page_size: int, out, workspace, group_rows=None, group_prefix=None, fault=None,
                            stream=None):
    """kd_attn_paged_decode over a Q8_0 cache of head_dim 128 (see include/kd.h)."""
    _check((_call or _fast()).paged(q, (k_quants, k_scales, v_quants, v_scales), table, lens,
                                    group_rows, group_prefix, n_heads, n_kv_heads, 128, n_pages, page_size, out, workspace,
                                    fault, stream))


def kd_debug_attn_paged_inject_wait_timeout(part: int):
    """The next call that reads a shared prefix once gives up waiting for its first tile's keys (0) or values (1)."""
    _check(lib().kd_debug_attn_paged_inject_wait_timeout(int(part)))
