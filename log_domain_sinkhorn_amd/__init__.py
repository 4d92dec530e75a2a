"""Python binding of the MI355X online log-domain Sinkhorn library.

Thin ctypes wrappers around the C ABI declared in ``include/sinkhorn.h``: the
functions here only marshal arguments (torch device tensors -> raw pointers,
the current HIP stream -> ``void*``) and turn status codes into exceptions.
Every step of the computation runs in the HIP kernels of ``libsinkhorn.so``.
PyTorch provides device memory and streams only.

The library must have been built (``python -m log_domain_sinkhorn_amd.build``);
every entry point raises ``ImportError`` without it: there is no CPU or
PyTorch fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from dataclasses import dataclass

import torch  # loads the HIP runtime the library links against
import torch.autograd.forward_ad as _forward_ad

__all__ = [
    "SinkhornError",
    "Schedule",
    "MultiscaleParams",
    "Problem",
    "mean_sqeuclid",
    "morton_order",
    "cross_attention",
    "cross_attention_grad",
    "attention_mass",
    "cache_evict",
    "rotary_frequencies",
    "rotate_heads",
    "rotate_heads_grad",
    "cache_append",
    "paged_attention",
    "lib",
    "LIB_PATH",
    "OK",
    "NOT_CONVERGED",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsinkhorn.so")

OK = 0
NOT_CONVERGED = 1
ERR_INVALID_ARG = -1
ERR_OOM = -2
ERR_HIP = -3
ERR_CAPACITY = -4
ERR_NONFINITE = -5
ERR_MASS = -6
ERR_UNSUPPORTED = -7

# kernel kinds for Problem.profile_enable (SINKHORN_PROF_* in sinkhorn.h)
PROF_DENSE = 1
PROF_SPARSE = 2
PROF_MATERIALIZE = 4
PROF_BARY = 8
PROF_DENSE_EXACT = 16

_p = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_f64 = ctypes.c_double


class _ScheduleC(ctypes.Structure):
    _fields_ = [
        ("eps_start", _f64),
        ("eps_target", _f64),
        ("eps_factor", _f64),
        ("iters_per_stage", _i32),
        ("fixed_iters", _i32),
        ("tol", _f64),
        ("max_iters", _i32),
        ("check_every", _i32),
    ]


class _ReportC(ctypes.Structure):
    _fields_ = [
        ("halfsteps", _i64),
        ("iters", _i64),
        ("final_iters", _i64),
        ("pairs_evaluated", _f64),
        ("row_l1", _f64),
        ("col_l1", _f64),
        ("seconds", _f64),
        ("stages", _i32),
        ("converged", _i32),
        ("history", ctypes.POINTER(_f64)),
        ("history_cap", _i32),
        ("history_len", _i32),
        ("seconds_per_halfstep", _f64),
        ("workspace_bytes", _i64),
        ("peak_extra_bytes", _i64),
    ]


class _MultiscaleParamsC(ctypes.Structure):
    _fields_ = [
        ("B", _i32),
        ("p_bits", _i32),
        ("eps", _f64),
        ("tol", _f64),
        ("delta_scale", _f64),
        ("coarse_eps_start", _f64),
        ("coarse_factor", _f64),
        ("coarse_iters_per_stage", _i32),
        ("coarse_tol", _f64),
        ("coarse_max", _i32),
        ("stall_window", _i32),
        ("stall_rel", _f64),
        ("max_fine", _i32),
        ("verify", _i32),
        ("adaptive", _i32),
        ("check_every", _i32),
        ("check_samples", _i32),
        ("check_samples_max", _i32),
        ("sample_seed", ctypes.c_uint64),
        ("warm_start", _i32),
    ]


class _MultiscaleReportC(ctypes.Structure):
    _fields_ = [
        ("coarse_iters", _i64),
        ("fine_updates", _i64),
        ("ncells_x", _i64),
        ("ncells_y", _i64),
        ("last_tiles", _i64),
        ("pairs_evaluated", _f64),
        ("R_A_row", _f64),
        ("R_A_col", _f64),
        ("omega", _f64),
        ("seconds_total", _f64),
        ("seconds_sort", _f64),
        ("seconds_coarse", _f64),
        ("seconds_lift", _f64),
        ("seconds_fine", _f64),
        ("certified", _i32),
        ("last_candidates", _i64),
        ("accepted_by_sample", _i32),
        ("checks", _i64),
        ("last_check_samples", _i64),
        ("last_check", _f64 * 4),
        ("peak_extra_bytes", _i64),
    ]


_i64x2 = _i64 * 2
_i64x3 = _i64 * 3


class _AttentionC(ctypes.Structure):
    _fields_ = [
        ("dtype", _i32),
        ("batch", _i32),
        ("heads_q", _i32),
        ("heads_kv", _i32),
        ("d", _i32),
        ("dv", _i32),
        ("len_q", _i64),
        ("len_k", _i64),
        ("scale", _f64),
        ("q_stride", _i64x3),
        ("k_stride", _i64x3),
        ("v_stride", _i64x3),
        ("out_stride", _i64x3),
        ("dout_stride", _i64x3),
        ("dq_stride", _i64x3),
        ("dk_stride", _i64x3),
        ("dv_stride", _i64x3),
        ("key_bias", _p),
        ("bias_stride", _i64x2),
        ("query_lengths", _p),
        ("key_lengths", _p),
    ]


class _CacheC(ctypes.Structure):
    _fields_ = [
        ("dtype", _i32),
        ("batch", _i32),
        ("heads", _i32),
        ("d", _i32),
        ("dv", _i32),
        ("len", _i64),
        ("keep", _i64),
        ("first", _i64),
        ("recent", _i64),
        ("k_stride", _i64x3),
        ("v_stride", _i64x3),
        ("k_out_stride", _i64x3),
        ("v_out_stride", _i64x3),
        ("key_lengths", _p),
    ]


class _RotationC(ctypes.Structure):
    _fields_ = [
        ("dtype", _i32),
        ("batch", _i32),
        ("heads_q", _i32),
        ("heads_kv", _i32),
        ("d", _i32),
        ("rotated", _i32),
        ("interleaved", _i32),
        ("norm", _i32),
        ("weight_dtype", _i32),
        ("len", _i64),
        ("gain", _f64),
        ("eps", _f64),
        ("q_stride", _i64x3),
        ("k_stride", _i64x3),
        ("q_out_stride", _i64x3),
        ("k_out_stride", _i64x3),
        ("dq_stride", _i64x3),
        ("dk_stride", _i64x3),
        ("frequencies", _p),
        ("positions", _p),
        ("position_stride", _i64),
        ("lengths", _p),
    ]


class _PagesC(ctypes.Structure):
    _fields_ = [
        ("page_size", _i32),
        ("table_len", _i32),
        ("pages", _i64),
        ("table_stride", _i64),
        ("k_stride", _i64x3),
        ("v_stride", _i64x3),
        ("dv", _i32),
        ("page_table", _p),
        ("lengths", _p),
    ]


def _packer(cls):
    """pack(*values) -> the bytes of a `cls`, arrays as their elements and pointers as
    integers (a third of the time that filling the fields takes)."""
    codes = {_i32: "i", _i64: "q", _f64: "d", _p: "P", _i64x2: "2q", _i64x3: "3q"}
    s = struct.Struct("@" + "".join(codes[t] for _, t in cls._fields_) + "0q")
    assert s.size == ctypes.sizeof(cls)

    def pack(*values):
        try:
            return s.pack(*values)
        except struct.error as e:
            raise ValueError(f"a size or stride is out of range ({e})") from None

    return pack


_pack_attention, _pack_rotation, _pack_pages = (_packer(c) for c in (_AttentionC, _RotationC, _PagesC))

# name -> argtypes (every entry point declared in include/sinkhorn.h)
_SIGS = {
    "sinkhorn_strerror": ([_i32], ctypes.c_char_p),
    "sinkhorn_last_error": ([], ctypes.c_char_p),
    "sinkhorn_mean_sqeuclid": ([_p, _p, _i64, _i64, _i32, _p, _p], _i32),
    "sinkhorn_init": ([_p, _p, _p, _p, _p, _i64, _i64, _i32, _f64, ctypes.c_uint32, _p], _i32),
    "sinkhorn_destroy": ([_p], _i32),
    "sinkhorn_problem_info": ([_p, _p, _p, _p, _p], _i32),
    "sinkhorn_device_memory": ([_p, _p, _p, _i32], _i32),
    "sinkhorn_halfstep_f": ([_p, _f64, _p, _p, _p, _p], _i32),
    "sinkhorn_halfstep_g": ([_p, _f64, _p, _p, _p, _p], _i32),
    "sinkhorn_marginal_residual": ([_p, _f64, _p, _p, _p, _p], _i32),
    "sinkhorn_solve": ([_p, _p, _p, _p, _p], _i32),
    "sinkhorn_materialize_rows": ([_p, _f64, _p, _p, _p, _i64, _p, _p], _i32),
    "sinkhorn_materialize_rows_noalloc": ([_p, _f64, _p, _p, _p, _i64, _p, _p], _i32),
    "sinkhorn_min_row": ([_p, _f64, _p, _p, _p], _i32),
    "sinkhorn_morton_order": ([_p, _p, _i64, _i64, _i32, _p, _p, _p, _p, _p], _i32),
    "sinkhorn_morton_sort": ([_p, _i32, _p, _p], _i32),
    "sinkhorn_block_screen": ([_p, _f64, _p, _p, _i32, _f64, _i32, _p, _p, _i64, _p], _i32),
    "sinkhorn_verify_tiles": ([_p, _f64, _p, _p, _i32, _f64, _p, _p, _p, _p, _p, _p, _p], _i32),
    "sinkhorn_sparse_halfstep_f": ([_p, _f64, _p, _i32, _p, _p, _p, _p, _p], _i32),
    "sinkhorn_sparse_halfstep_g": ([_p, _f64, _p, _i32, _p, _p, _p, _p, _p], _i32),
    "sinkhorn_barycentric": ([_p, _f64, _p, _p, _p, _p], _i32),
    "sinkhorn_sparsify": ([_p, _f64, _p, _p, ctypes.c_float, _i64, _p, _p, _p, _i64, _p], _i32),
    "sinkhorn_sparse_barycentric": ([_p, _f64, _p, _p, _i32, _p, _p, _p, _p], _i32),
    "sinkhorn_solve_multiscale": ([_p, _p, _p, _p, _p], _i32),
    "sinkhorn_sample_indices": ([_i64, _i32, ctypes.c_uint64, ctypes.c_uint64, _p, _p], _i32),
    "sinkhorn_sampled_residual": ([_p, _f64, _p, _p, _i32, _i32, ctypes.c_uint64, _p, _p], _i32),
    "sinkhorn_attention_workspace": ([_p, _i32, _p, _p, _p, _p, _p], _i32),
    "sinkhorn_cross_attention": ([_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _i64, _p], _i32),
    "sinkhorn_cross_attention_grad": ([_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _i64, _p], _i32),
    "sinkhorn_attention_mass": ([_p, _p, _p, _p, _p, _p, _p, _p, _i64, _p], _i32),
    "sinkhorn_cache_evict": ([_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _i64, _p], _i32),
    "sinkhorn_cache_workspace": ([_p, _p], _i32),
    "sinkhorn_rotary_frequencies": ([_i32, _f64, _f64, _f64, _f64, _f64, _p], _i32),
    "sinkhorn_rotate_heads": ([_p, _p, _p, _p, _p, _p, _p, _p], _i32),
    "sinkhorn_rotation_workspace": ([_p, _p], _i32),
    "sinkhorn_rotate_heads_grad": ([_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _i64, _p], _i32),
    "sinkhorn_cache_append": ([_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p], _i32),
    "sinkhorn_paged_workspace": ([_p, _p, _i64, _i64, _p], _i32),
    "sinkhorn_paged_attention": ([_p, _p, _i64, _i64, _p, _p, _p, _p, _p, _p, _i64, _p], _i32),
    "sinkhorn_profile_enable": ([_p, _i32], _i32),
    "sinkhorn_profile_read": ([_p, _p, _p, _p], _i32),
    "sinkhorn_probe_issue_rate": ([_i32, _i32, _p, _p, _p, _p], _i32),
}

EXPORTED = tuple(_SIGS)

_LIB = None


def lib() -> ctypes.CDLL:
    """The loaded library (raises ImportError if it was not built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing; build it with `python -m log_domain_sinkhorn_amd.build`"
            )
        handle = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
        _LIB = handle
    return _LIB


class SinkhornError(RuntimeError):
    def __init__(self, code: int, where: str):
        L = lib()
        detail = L.sinkhorn_last_error().decode()
        name = L.sinkhorn_strerror(code).decode()
        super().__init__(f"{where}: {name} ({code}){': ' + detail if detail else ''}")
        self.code = code


def _check(code: int, where: str) -> int:
    if code < 0:
        raise SinkhornError(code, where)
    return code


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _dev(t: torch.Tensor, dtype, name: str, shape=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


_increment_version = torch.autograd.graph.increment_version


def _changed(*outputs):
    """Tells autograd that a call wrote these tensors of the caller's (None: it had no such
    one): a graph that saved one before then refuses its backward pass, as it does after
    torch's own operations in place."""
    for t in outputs:
        if t is not None:
            _increment_version(t)


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


@dataclass
class Schedule:
    eps_start: float
    eps_target: float
    eps_factor: float = 0.5
    iters_per_stage: int = 10
    fixed_iters: int = 0
    tol: float = 1e-3
    max_iters: int = 10000
    check_every: int = 1

    def _c(self) -> _ScheduleC:
        return _ScheduleC(self.eps_start, self.eps_target, self.eps_factor, self.iters_per_stage,
                          self.fixed_iters, self.tol, self.max_iters, self.check_every)


@dataclass
class MultiscaleParams:
    B: int = 128
    p_bits: int = 0
    eps: float = 1e-4
    tol: float = 1e-2
    delta_scale: float = 1e-3
    coarse_eps_start: float = 1.0
    coarse_factor: float = 0.5
    coarse_iters_per_stage: int = 10
    coarse_tol: float = 1e-3
    coarse_max: int = 2048
    stall_window: int = 10
    stall_rel: float = 0.01
    max_fine: int = 8192
    verify: bool = False
    adaptive: bool = False
    check_every: int = 128
    check_samples: int = 1024
    check_samples_max: int = 8192
    sample_seed: int = 0
    warm_start: bool = False

    def _c(self) -> _MultiscaleParamsC:
        return _MultiscaleParamsC(self.B, self.p_bits, self.eps, self.tol, self.delta_scale,
                                  self.coarse_eps_start, self.coarse_factor,
                                  self.coarse_iters_per_stage, self.coarse_tol, self.coarse_max,
                                  self.stall_window, self.stall_rel, self.max_fine,
                                  int(bool(self.verify)), int(bool(self.adaptive)), self.check_every,
                                  self.check_samples, self.check_samples_max, self.sample_seed,
                                  int(bool(self.warm_start)))


def _struct_dict(s) -> dict:
    out = {}
    for name, _ in s._fields_:
        v = getattr(s, name)
        out[name] = list(v) if isinstance(v, ctypes.Array) else v
    return out


def sample_indices(count: int, k: int, seed: int, stream_id: int, device="cuda:0") -> torch.Tensor:
    """The sampled checks' indices as an int32 device tensor."""
    out = torch.empty(max(1, k), dtype=torch.int32, device=device)
    _check(lib().sinkhorn_sample_indices(int(count), int(k), int(seed), int(stream_id),
                                         _stream(torch.device(device)), _ptr(out)), "sample_indices")
    return out[:k]


def mean_sqeuclid(x: torch.Tensor, y: torch.Tensor) -> float:
    """Unweighted mean of ||x_i - y_j||^2 over all pairs (device fp64)."""
    _dev(x, torch.float32, "x")
    _dev(y, torch.float32, "y")
    out = _f64()
    _check(lib().sinkhorn_mean_sqeuclid(_ptr(x), _ptr(y), x.shape[0], y.shape[0], x.shape[1],
                                        _stream(x.device), ctypes.byref(out)), "mean_sqeuclid")
    return out.value


def morton_order(x: torch.Tensor, y: torch.Tensor):
    """(codes_x, perm_x, codes_y, perm_y): sorted Morton codes (int64 tensors
    holding the uint64 bits) and the original index of each sorted point."""
    _dev(x, torch.float32, "x")
    _dev(y, torch.float32, "y")
    n, d = x.shape
    m = y.shape[0]
    cx = torch.empty(n, dtype=torch.int64, device=x.device)
    cy = torch.empty(m, dtype=torch.int64, device=x.device)
    px = torch.empty(n, dtype=torch.int32, device=x.device)
    py = torch.empty(m, dtype=torch.int32, device=x.device)
    _check(lib().sinkhorn_morton_order(_ptr(x), _ptr(y), n, m, d, _stream(x.device), _ptr(cx),
                                       _ptr(px), _ptr(cy), _ptr(py)), "morton_order")
    return cx, px, cy, py


(PROBE_FMA_F32, PROBE_EXP_F32, PROBE_FMA_F64, PROBE_PAIR_F32, PROBE_PAIR_F32_NOEXP, PROBE_PAIR_F64,
 PROBE_SUB_F32, PROBE_FMAC_F32, PROBE_ADD_F64, PROBE_CVT_F32_F64, PROBE_PAIR_TILE_F32,
 PROBE_PAIR_SPLIT_F32, PROBE_PAIR_TILE_MFMA) = range(13)
FLAG_FP32_PAIRS = 1


def probe_issue_rate(kind: int, iters: int = 20000, device="cuda:0"):
    """(lane-instructions/s, pairs/s, kernel ms) of an issue-rate probe kernel."""
    rate, pairs, ms = _f64(), _f64(), _f64()
    with torch.cuda.device(device):
        _check(lib().sinkhorn_probe_issue_rate(int(kind), int(iters), _stream(device), ctypes.byref(rate),
                                               ctypes.byref(pairs), ctypes.byref(ms)), "probe_issue_rate")
    return rate.value, pairs.value, ms.value


def device_memory(reset: bool = False):
    """(current, peak, largest) device bytes the library holds, over all
    handles (``sinkhorn_device_memory``); reset=True then starts a new peak."""
    cur, peak, big = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check(lib().sinkhorn_device_memory(ctypes.byref(cur), ctypes.byref(peak), ctypes.byref(big),
                                        int(bool(reset))), "device_memory")
    return cur.value, peak.value, big.value


# ---------------------------------------------------------------- attention between two sets
_ATTN_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_ATTEND, _ATTEND_MASS, _ATTEND_GRAD, _ATTENTION_MASS = range(4)


def _head_tensor(t, name, dtype=None, shape=None):
    """A [batch, length, heads, width] tensor of one of the three element types
    with a contiguous last dimension (the other strides are free)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in _ATTN_DTYPES:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    has = t.shape
    if len(has) != 4:
        raise ValueError(f"{name} must be [batch, length, heads, width]")
    if shape is not None and has != shape:
        raise ValueError(f"{name} has shape {tuple(has)}, expected {tuple(shape)}")
    if t.stride(3) != 1 and has[3] > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return _ungraphed(t, name)


def _ungraphed(t, name):
    """No call here records a graph: a tensor whose gradient would be lost is refused."""
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires grad: these calls record no graph; detach it or use torch.no_grad(), "
                         "and take gradients from cross_attention_grad or rotate_heads_grad")
    # a tangent does not show in requires_grad; asked for only inside a dual level
    if getattr(_forward_ad, "_current_level", 0) >= 0 and _forward_ad.unpack_dual(t).tangent is not None:
        raise ValueError(f"{name} carries a tangent: these calls have no forward derivative; pass its primal")
    return t


def _written(t, name):
    """An output: no two of its elements may share memory."""
    span = 1
    for stride, size in sorted(zip(t.stride(), t.shape)):
        if size > 1:
            if stride < span:
                raise ValueError(f"{name} has overlapping elements")
            span = stride * size
    return t


def _plain(t, name, dtype, shape):
    """A contiguous side argument (not necessarily on the device yet)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _ungraphed(t, name)


def _same_device(first, others):
    """The device's index."""
    index = first.get_device()
    if index < 0:
        raise ValueError("the arguments must be device tensors")
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"the arguments are on different devices ({first.device}, {t.device})")
    return index


# the current stream's handle without a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(index, where, fn, *args):
    """fn(*args, current stream) with device `index` current."""
    if torch.cuda.current_device() == index:
        _check(fn(*args, _raw_stream(index)), where)
    else:
        with torch.cuda.device(index):
            _check(fn(*args, _raw_stream(index)), where)


def _at(t):
    return None if t is None else t.data_ptr()


def _strides3(t):
    """Element strides of batch, length and head (0 where there is one)."""
    s0, s1, s2, _ = t.stride()
    shape = t.shape
    if 1 in shape:
        return _i64x3(s0 if shape[0] > 1 else 0, s1 if shape[1] > 1 else 0, s2 if shape[2] > 1 else 0)
    return _i64x3(s0, s1, s2)


def _attention(q, k, v, scale, key_bias, query_lengths, key_lengths):
    _head_tensor(q, "q")
    B, lq, hq, d = q.shape
    _head_tensor(k, "k", q.dtype)
    _, lk, hkv, _ = k.shape
    if tuple(k.shape) != (B, lk, hkv, d):
        raise ValueError(f"k has shape {tuple(k.shape)}, expected ({B}, length, heads, {d})")
    dv = d
    if v is not None:
        _head_tensor(v, "v", q.dtype)
        dv = v.shape[3]
        if tuple(v.shape) != (B, lk, hkv, dv):
            raise ValueError(f"v has shape {tuple(v.shape)}, expected ({B}, {lk}, {hkv}, width)")
    if hkv < 1 or hq < 1 or hq % hkv:
        raise ValueError(f"{hq} query heads are no multiple of {hkv} key heads")
    a = _AttentionC(_ATTN_DTYPES[q.dtype], B, hq, hkv, d, dv, lq, lk,
                    1.0 / math.sqrt(max(d, 1)) if scale is None else float(scale), _strides3(q), _strides3(k))
    if v is not None:
        a.v_stride = _strides3(v)
    if key_bias is not None:
        if not isinstance(key_bias, torch.Tensor) or key_bias.dtype != torch.float32:
            raise TypeError("key_bias must be a float32 tensor")
        if key_bias.requires_grad and torch.is_grad_enabled():
            raise ValueError("key_bias is held fixed and takes no gradient")
        _ungraphed(key_bias, "key_bias")
        if tuple(key_bias.shape) not in ((B, lk), (B, hkv, lk)):
            raise ValueError(f"key_bias has shape {tuple(key_bias.shape)}, expected ({B}, {lk}) or ({B}, {hkv}, {lk})")
        if lk > 1 and key_bias.stride(-1) != 1:
            raise ValueError("the last dimension of key_bias must be contiguous")
        a.key_bias = key_bias.data_ptr()
        a.bias_stride = _i64x2(key_bias.stride(0), key_bias.stride(1) if key_bias.dim() == 3 else 0)
    if query_lengths is not None:
        a.query_lengths = _plain(query_lengths, "query_lengths", torch.int32, (B,)).data_ptr()
    if key_lengths is not None:
        a.key_lengths = _plain(key_lengths, "key_lengths", torch.int32, (B,)).data_ptr()
    return a


def _workspace(a, what, device, q, k, v=None, dout=None):
    n = _i64()
    _check(lib().sinkhorn_attention_workspace(ctypes.byref(a), what, _at(q), _at(k), _at(v), _at(dout),
                                              ctypes.byref(n)), "attention_workspace")
    return (torch.empty(n.value, dtype=torch.uint8, device=device) if n.value else None), n.value


def _mass_args(a, row_weight, mass_in, mass_out):
    B, hkv, lk = a.batch, a.heads_kv, a.len_k
    if row_weight is not None:
        _plain(row_weight, "row_weight", torch.float32, (B, a.len_q))
    if mass_in is not None:
        _plain(mass_in, "mass_in", torch.float32, (B, hkv, lk))
    if mass_out is not None:
        _plain(mass_out, "mass_out", torch.float32, (B, hkv, lk))


def cross_attention(q, k, v, *, scale=None, key_bias=None, query_lengths=None, key_lengths=None, row_weight=None,
                    mass_in=None, mass_out=None, out=None, lse=None):
    """(out, lse): softmax(scale q.k + key_bias) v for q [B, Lq, Hq, d] against
    k [B, Lk, Hkv, d] and v [B, Lk, Hkv, dv] (``sinkhorn_cross_attention``).

    out [B, Lq, Hq, dv] has q's type, lse [B, Hq, Lq] is float32. Query head h
    reads key head h // (Hq / Hkv). scale defaults to d ** -0.5. key_bias
    (float32, [B, Lk] or [B, Hkv, Lk]) is added to the scores; a key whose bias
    is <= -1e30 or whose index is >= key_lengths[b] (int32 [B]) takes no part. Rows
    without keys and rows >= query_lengths[b] give out = 0, lse = -inf.

    With mass_out (float32 [B, Hkv, Lk]) it also receives mass_in (same shape, may
    be mass_out; default 0) plus the weight each key gathered over rows and
    heads, rows weighted by row_weight (float32 [B, Lq], default 1).

    For the squared-Euclidean cost at eps, q = x, k = y, scale = 2 s / eps and
    key_bias = log b + (g - s |y|^2) / eps average v over the plan's rows.

    Outputs may lie between the rows of other arguments but share no element with
    them (mass_out with mass_in apart)."""
    a = _attention(q, k, v, scale, key_bias, query_lengths, key_lengths)
    B, lq, hq, _ = q.shape
    shape = (B, lq, hq, v.shape[3])
    if out is not None:
        _written(_head_tensor(out, "out", q.dtype, shape), "out")
    if lse is not None:
        _plain(lse, "lse", torch.float32, (B, hq, lq))
    if mass_out is None and (mass_in is not None or row_weight is not None):
        raise ValueError("mass_in and row_weight need mass_out")
    _mass_args(a, row_weight, mass_in, mass_out)
    index = _same_device(q, (k, v, key_bias, query_lengths, key_lengths, row_weight, mass_in, mass_out, out, lse))
    device = q.device
    given = out, lse, mass_out
    out = torch.empty(shape, dtype=q.dtype, device=device) if out is None else out
    lse = torch.empty((B, hq, lq), dtype=torch.float32, device=device) if lse is None else lse
    a.out_stride = _strides3(out)
    ws, n = _workspace(a, _ATTEND if mass_out is None else _ATTEND_MASS, device, q, k, v)
    _launch(index, "cross_attention", lib().sinkhorn_cross_attention, ctypes.byref(a), q.data_ptr(), k.data_ptr(),
            v.data_ptr(), out.data_ptr(), lse.data_ptr(), _at(row_weight), _at(mass_in), _at(mass_out), _at(ws), n)
    _changed(*given)
    return out, lse


def cross_attention_grad(dout, q, k, v, out, lse, *, scale=None, key_bias=None, query_lengths=None, key_lengths=None,
                         dq=None, dk=None, dv=None):
    """(dq, dk, dv) from dout, the gradient of out, and the out and lse that
    cross_attention returned for the same arguments
    (``sinkhorn_cross_attention_grad``). key_bias is held fixed."""
    a = _attention(q, k, v, scale, key_bias, query_lengths, key_lengths)
    B, lq, hq, _ = q.shape
    shape = (B, lq, hq, v.shape[3])
    _head_tensor(dout, "dout", q.dtype, shape)
    _head_tensor(out, "out", q.dtype, shape)
    _plain(lse, "lse", torch.float32, (B, hq, lq))
    for t, like, name in ((dq, q, "dq"), (dk, k, "dk"), (dv, v, "dv")):
        if t is not None:
            _written(_head_tensor(t, name, q.dtype, like.shape), name)
    index = _same_device(q, (k, v, key_bias, query_lengths, key_lengths, dout, out, lse, dq, dk, dv))
    device = q.device
    given = dq, dk, dv
    dq, dk, dv = (torch.empty(like.shape, dtype=q.dtype, device=device) if t is None else t
                  for t, like in ((dq, q), (dk, k), (dv, v)))
    a.out_stride, a.dout_stride = _strides3(out), _strides3(dout)
    a.dq_stride, a.dk_stride, a.dv_stride = _strides3(dq), _strides3(dk), _strides3(dv)
    ws, n = _workspace(a, _ATTEND_GRAD, device, q, k, v, dout)
    _launch(index, "cross_attention_grad", lib().sinkhorn_cross_attention_grad, ctypes.byref(a), q.data_ptr(),
            k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(),
            dv.data_ptr(), _at(ws), n)
    _changed(*given)
    return dq, dk, dv


def attention_mass(q, k, lse, *, scale=None, key_bias=None, query_lengths=None, key_lengths=None, row_weight=None,
                   mass_in=None, mass_out=None):
    """The weight each key gathers, [B, Hkv, Lk] float32, from the lse of a
    forward pass over the same arguments (``sinkhorn_attention_mass``): mass_in
    (default 0) plus the sum over rows and heads of row_weight exp(s - lse)."""
    a = _attention(q, k, None, scale, key_bias, query_lengths, key_lengths)
    _plain(lse, "lse", torch.float32, (a.batch, a.heads_q, a.len_q))
    _mass_args(a, row_weight, mass_in, mass_out)
    index = _same_device(q, (k, key_bias, query_lengths, key_lengths, lse, row_weight, mass_in, mass_out))
    given = mass_out
    if mass_out is None:
        mass_out = torch.empty((a.batch, a.heads_kv, a.len_k), dtype=torch.float32, device=q.device)
    ws, n = _workspace(a, _ATTENTION_MASS, q.device, q, k)
    _launch(index, "attention_mass", lib().sinkhorn_attention_mass, ctypes.byref(a), q.data_ptr(), k.data_ptr(),
            lse.data_ptr(), _at(row_weight), _at(mass_in), mass_out.data_ptr(), _at(ws), n)
    _changed(given)
    return mass_out


def cache_evict(k, v, mass, keep: int, *, key_lengths=None, first: int = 0, recent: int = 0, k_out=None, v_out=None,
                mass_out=None, index_out=None, lengths_out=None):
    """Prune a cache by gathered weight (``sinkhorn_cache_evict``): of the live
    keys of k [B, L, H, d], v [B, L, H, dv] keep the `first` first, the `recent`
    last and the heaviest others by mass [B, H, L] (float32), `keep` in all, in
    their order. Returns (k_out, v_out, mass_out, index_out, lengths_out): the
    kept rows [B, C, H, .] with C = min(keep, L), their weights and old positions
    [B, H, C] (0 and -1 behind the kept ones) and the counts [B] (int32). Rows of
    k_out and v_out behind the kept ones are left as they were (zero in buffers
    made here). Outputs share no element with k, v, mass or each other; they may be
    rows of the cache's own buffers behind its keys."""
    _head_tensor(k, "k")
    B, n, h, d = k.shape
    _head_tensor(v, "v", k.dtype)
    dv = v.shape[3]
    if tuple(v.shape) != (B, n, h, dv):
        raise ValueError(f"v has shape {tuple(v.shape)}, expected ({B}, {n}, {h}, width)")
    _plain(mass, "mass", torch.float32, (B, h, n))
    # as large as the C side takes them: a longer one means the same
    keep, first, recent = (max(-1, min(int(x), (1 << 63) - 1)) for x in (keep, first, recent))
    cap = min(keep, n)
    if keep < 1:
        raise ValueError("keep must be >= 1")
    if key_lengths is not None:
        _plain(key_lengths, "key_lengths", torch.int32, (B,))
    if k_out is not None:
        _written(_head_tensor(k_out, "k_out", k.dtype, (B, cap, h, d)), "k_out")
    if v_out is not None:
        _written(_head_tensor(v_out, "v_out", k.dtype, (B, cap, h, dv)), "v_out")
    if mass_out is not None:
        _plain(mass_out, "mass_out", torch.float32, (B, h, cap))
    if index_out is not None:
        _plain(index_out, "index_out", torch.int32, (B, h, cap))
    if lengths_out is not None:
        _plain(lengths_out, "lengths_out", torch.int32, (B,))
    index = _same_device(k, (v, mass, key_lengths, k_out, v_out, mass_out, index_out, lengths_out))
    device = k.device
    given = k_out, v_out, mass_out, index_out, lengths_out
    # without key_lengths every row of the outputs is written
    new = torch.empty if key_lengths is None else torch.zeros
    k_out = new((B, cap, h, d), dtype=k.dtype, device=device) if k_out is None else k_out
    v_out = new((B, cap, h, dv), dtype=k.dtype, device=device) if v_out is None else v_out
    if mass_out is None:
        mass_out = torch.empty((B, h, cap), dtype=torch.float32, device=device)
    if index_out is None:
        index_out = torch.empty((B, h, cap), dtype=torch.int32, device=device)
    if lengths_out is None:
        lengths_out = torch.empty(B, dtype=torch.int32, device=device)
    c = _CacheC(_ATTN_DTYPES[k.dtype], B, h, d, dv, n, keep, first, recent, _strides3(k), _strides3(v), _strides3(k_out),
                _strides3(v_out), _at(key_lengths))
    size = _i64()
    _check(lib().sinkhorn_cache_workspace(ctypes.byref(c), ctypes.byref(size)), "cache_workspace")
    ws = torch.empty(size.value, dtype=torch.uint8, device=device) if size.value else None
    _launch(index, "cache_evict", lib().sinkhorn_cache_evict, ctypes.byref(c), k.data_ptr(), v.data_ptr(),
            mass.data_ptr(), k_out.data_ptr(), v_out.data_ptr(), mass_out.data_ptr(), index_out.data_ptr(),
            lengths_out.data_ptr(), _at(ws), size.value)
    _changed(*given)
    return k_out, v_out, mass_out, index_out, lengths_out


# ---------------------------------------------------------------- decoding over a paged cache
def rotary_frequencies(rotated: int, base: float = 10000.0, *, factor: float = 1.0, original_length: float = 0.0,
                       low: float = 1.0, high: float = 32.0, device="cuda:0"):
    """Radians per position of each pair, float64 [rotated / 2] on `device`
    (``sinkhorn_rotary_frequencies``): base ** (-2 i / rotated), slowed down by
    `factor` for a context that much longer; with original_length only for pairs of
    few turns in it (all of it up to `low` turns, none from `high` on, linearly
    mixed in between)."""
    buf = (_f64 * max(1, int(rotated) // 2))()
    _check(lib().sinkhorn_rotary_frequencies(int(rotated), float(base), float(factor), float(original_length),
                                             float(low), float(high), buf), "rotary_frequencies")
    return torch.tensor(list(buf)[:int(rotated) // 2], dtype=torch.float64, device=device)


_NO_STRIDES = (0, 0, 0)


def _strides(t):
    """Element strides of batch, length and head (0 where there is one)."""
    s0, s1, s2, _ = t.stride()
    shape = t.shape
    if 1 in shape:
        return (s0 if shape[0] > 1 else 0, s1 if shape[1] > 1 else 0, s2 if shape[2] > 1 else 0)
    return s0, s1, s2


def _rotation(q, k, frequencies, interleaved, gain, norm_eps, q_weight, k_weight, positions, lengths):
    """What a call's description holds before its strides and behind them; q or k may be None."""
    one = k if q is None else q
    dtype = one.dtype
    B, n, heads_q, d = one.shape
    heads_kv = 0
    if q is None:
        heads_q, heads_kv = 0, heads_q
    elif k is not None:
        if k.dtype != dtype:
            raise TypeError(f"k must be {dtype}, got {k.dtype}")
        kb, kn, heads_kv, kd = k.shape
        if kb != B or kn != n or kd != d:
            raise ValueError(f"k has shape {tuple(k.shape)}, expected ({B}, {n}, heads, {d})")
    rotated = at = place = stride = norm = kind = count = 0
    eps = 0.0
    if frequencies is not None:
        if not isinstance(frequencies, torch.Tensor) or frequencies.dtype != torch.float64:
            raise TypeError("frequencies must be a float64 tensor")
        if frequencies.dim() != 1 or 2 * frequencies.shape[0] > d:
            raise ValueError(f"frequencies have shape {tuple(frequencies.shape)}, expected at most ({d // 2},)")
        if not frequencies.is_contiguous():
            raise ValueError("frequencies must be contiguous")
        rotated = 2 * _ungraphed(frequencies, "frequencies").shape[0]
        at = frequencies.data_ptr()
    elif positions is not None:
        raise ValueError("positions need frequencies")
    if norm_eps is not None:
        norm, eps = 1, float(norm_eps)
        of = None
        for w, t, name in ((q_weight, q, "q_weight"), (k_weight, k, "k_weight")):
            if w is None:
                continue
            if t is None:
                raise ValueError(f"{name} without its tensor")
            if of is None:
                of = dtype if isinstance(w, torch.Tensor) and w.dtype == dtype else torch.float32
                kind = _ATTN_DTYPES[of]
            _plain(w, name, of, (d,))
    elif q_weight is not None or k_weight is not None:
        raise ValueError("weights need norm_eps")
    if positions is not None:
        if not isinstance(positions, torch.Tensor) or positions.dtype != torch.int32:
            raise TypeError("positions must be an int32 tensor")
        if tuple(positions.shape) not in ((B, n), (n,)):
            raise ValueError(f"positions have shape {tuple(positions.shape)}, expected ({B}, {n}) or ({n},)")
        if n > 1 and positions.stride(-1) != 1:
            raise ValueError("the last dimension of positions must be contiguous")
        place = positions.data_ptr()
        stride = positions.stride(0) if positions.dim() == 2 and B > 1 else 0
    if lengths is not None:
        count = _plain(lengths, "lengths", torch.int32, (B,)).data_ptr()
    head = (_ATTN_DTYPES[dtype], B, heads_q, heads_kv, d, rotated, 1 if interleaved else 0, norm, kind, n, float(gain), eps)
    return head, (at, place, stride, count)


def _result(t, like, name):
    """An output like `like`: the caller's, or a new one."""
    if like is None:
        if t is not None:
            raise ValueError(f"{name} without its tensor")
        return None
    if t is None:
        return torch.empty_like(like, memory_format=torch.contiguous_format)
    return _written(_head_tensor(t, name, like.dtype, like.shape), name)


def rotate_heads(q, k=None, *, positions=None, frequencies=None, interleaved=False, gain=1.0, norm_eps=None,
                 q_weight=None, k_weight=None, lengths=None, q_out=None, k_out=None):
    """(q_out, k_out): the heads of q [B, L, Hq, d] and k [B, L, Hkv, d] normed and
    rotated to their positions, in one launch (``sinkhorn_rotate_heads``).

    With norm_eps each head is divided by sqrt(mean x^2 + norm_eps) and multiplied by
    its weight (q_weight, k_weight [d], float32 or of q's type; default 1). With
    frequencies (float64 [r / 2], see rotary_frequencies) its first r elements turn:
    pairs (i, i + r / 2), or (2 i, 2 i + 1) if interleaved, by positions frequencies[i],
    times gain. positions is int32 [B, L] or [L], default 0, 1, ... Rows >= lengths[b]
    (int32 [B]) give zeros. q_out may be q and k_out k; k may be None."""
    _head_tensor(q, "q")
    if k is not None:
        _head_tensor(k, "k")
    head, tail = _rotation(q, k, frequencies, interleaved, gain, norm_eps, q_weight, k_weight, positions, lengths)
    given = q_out, k_out
    q_out, k_out = _result(q_out, q, "q_out"), _result(k_out, k, "k_out")
    index = _same_device(q, (k, frequencies, q_weight, k_weight, positions, lengths, q_out, k_out))
    ks, ko = (_NO_STRIDES, _NO_STRIDES) if k is None else (_strides(k), _strides(k_out))
    r = _pack_rotation(*head, *_strides(q), *ks, *_strides(q_out), *ko, *_NO_STRIDES, *_NO_STRIDES, *tail)
    _launch(index, "rotate_heads", lib().sinkhorn_rotate_heads, r, q.data_ptr(), _at(k), _at(q_weight), _at(k_weight),
            q_out.data_ptr(), _at(k_out))
    _changed(*given)
    return q_out, k_out


def rotate_heads_grad(dq_out, dk_out=None, q=None, k=None, *, positions=None, frequencies=None, interleaved=False,
                      gain=1.0, norm_eps=None, q_weight=None, k_weight=None, lengths=None, dq=None, dk=None):
    """(dq, dk, dq_weight, dk_weight) from the gradients of rotate_heads' results
    for the same arguments (``sinkhorn_rotate_heads_grad``). q and k are needed with
    norm_eps only; the weights' gradients (float32 [d], also where the weight is
    left at 1) are None without it. dk_out and k may be None. dq may be dq_out and dk
    dk_out."""
    _head_tensor(dq_out, "dq_out")
    if dk_out is not None:
        _head_tensor(dk_out, "dk_out")
    head, tail = _rotation(dq_out, dk_out, frequencies, interleaved, gain, norm_eps, q_weight, k_weight, positions, lengths)
    norm = norm_eps is not None
    qs = ks = yk = dks = _NO_STRIDES
    if norm:
        if q is None or (k is None) != (dk_out is None):
            raise ValueError("the gradient of a norm needs q and k")
        qs = _strides(_head_tensor(q, "q", dq_out.dtype, dq_out.shape))
        if k is not None:
            ks = _strides(_head_tensor(k, "k", dk_out.dtype, dk_out.shape))
    given = dq, dk
    dq, dk = _result(dq, dq_out, "dq"), _result(dk, dk_out, "dk")
    index = _same_device(dq_out, (dk_out, q, k, frequencies, q_weight, k_weight, positions, lengths, dq, dk))
    if dk is not None:
        yk, dks = _strides(dk_out), _strides(dk)
    r = _pack_rotation(*head, *qs, *ks, *_strides(dq_out), *yk, *_strides(dq), *dks, *tail)
    wq = wk = ws = None
    n = 0
    if norm:
        device, d = dq_out.device, dq_out.shape[3]
        wq = torch.empty(d, dtype=torch.float32, device=device)
        wk = None if dk is None else torch.empty(d, dtype=torch.float32, device=device)
        size = _i64()
        _check(lib().sinkhorn_rotation_workspace(r, ctypes.byref(size)), "rotation_workspace")
        n = size.value
        ws = torch.empty(n, dtype=torch.uint8, device=device)
    _launch(index, "rotate_heads_grad", lib().sinkhorn_rotate_heads_grad, r, dq_out.data_ptr(), _at(dk_out), _at(q), _at(k),
            _at(q_weight), _at(k_weight), dq.data_ptr(), _at(dk), _at(wq), _at(wk), _at(ws), n)
    _changed(*given)
    return dq, dk, wq, wk


def _pages(dtype, B, heads, d, k_cache, v_cache, page_table, lengths, name):
    """The bytes that describe a paged cache of k [pages, page_size, heads, d] and v, v's width
    and the heads (None: k's)."""
    _head_tensor(k_cache, "k_cache", dtype)
    _head_tensor(v_cache, "v_cache", dtype)
    pages, size, kh, kd = k_cache.shape
    vp, vsize, vh, dv = v_cache.shape
    if heads is None:
        heads = kh
    if kh != heads or kd != d:
        raise ValueError(f"k_cache has shape {tuple(k_cache.shape)}, expected (pages, page_size, {heads}, {d})")
    if vp != pages or vsize != size or vh != heads:
        raise ValueError(f"v_cache has shape {tuple(v_cache.shape)}, expected ({pages}, {size}, {heads}, width)")
    if not isinstance(page_table, torch.Tensor) or page_table.dtype != torch.int32:
        raise TypeError("page_table must be an int32 tensor")
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError(f"page_table has shape {tuple(page_table.shape)}, expected ({B}, pages of a sequence)")
    row, one = page_table.stride()
    width = page_table.shape[1]
    if width > 1 and one != 1:
        raise ValueError("the last dimension of page_table must be contiguous")
    _plain(lengths, name, torch.int32, (B,))
    return _pack_pages(size, width, pages, row if B > 1 else 0, *_strides(k_cache), *_strides(v_cache), dv,
                       page_table.data_ptr(), lengths.data_ptr()), dv, heads


def cache_append(k, v, k_cache, v_cache, page_table, cache_lengths, *, new_lengths=None, positions=None,
                 frequencies=None, interleaved=False, gain=1.0, norm_eps=None, k_weight=None, q=None, q_weight=None,
                 q_out=None, lengths_out=None):
    """Append new tokens to a paged cache (``sinkhorn_cache_append``).

    The keys k [B, L, Hkv, d], normed and rotated as by rotate_heads (neither without
    norm_eps and frequencies), and the values v [B, L, Hkv, dv] of the first
    new_lengths[b] tokens (int32 [B], default L) go behind the cache_lengths[b] keys
    (int32 [B]) that sequence b has. k_cache [pages, page_size, Hkv, d] and v_cache
    [pages, page_size, Hkv, dv] hold key j in page page_table[b, j // page_size]
    (int32 [B, pages of a sequence]), slot j % page_size; page_size is a multiple of 8.
    A token's position is its place in the sequence, or positions (int32 [B, L] or
    [L]). With q [B, L, Hq, d] the tokens' queries are normed and rotated on the way.

    Returns (lengths_out, q_out): the keys in the cache now (int32 [B]) and the queries
    (None without q; zeros behind new_lengths). Tokens whose page is outside the cache
    or behind the table are not written. No two tokens may share a place."""
    _head_tensor(k, "k")
    B, n, h, d = k.shape
    _head_tensor(v, "v", k.dtype)
    vb, vn, vh, dv = v.shape
    if vb != B or vn != n or vh != h:
        raise ValueError(f"v has shape {tuple(v.shape)}, expected ({B}, {n}, {h}, width)")
    if q is not None:
        _head_tensor(q, "q", k.dtype)
        if q.shape[0] != B or q.shape[1] != n or q.shape[3] != d:
            raise ValueError(f"q has shape {tuple(q.shape)}, expected ({B}, {n}, heads, {d})")
    head, tail = _rotation(q, k, frequencies, interleaved, gain, norm_eps, q_weight, k_weight, positions, new_lengths)
    c, width, _ = _pages(k.dtype, B, h, d, k_cache, v_cache, page_table, cache_lengths, "cache_lengths")
    if dv != width:
        raise ValueError(f"v has shape {tuple(v.shape)}, expected ({B}, {n}, {h}, {width})")
    _written(k_cache, "k_cache")
    _written(v_cache, "v_cache")
    given = q_out, lengths_out
    if lengths_out is None:
        lengths_out = cache_lengths.new_empty(B)
    else:
        _plain(lengths_out, "lengths_out", torch.int32, (B,))
    q_out = _result(q_out, q, "q_out")
    index = _same_device(k, (v, q, k_cache, v_cache, page_table, cache_lengths, new_lengths, positions, frequencies,
                             k_weight, q_weight, q_out, lengths_out))
    qs, qo = (_NO_STRIDES, _NO_STRIDES) if q is None else (_strides(q), _strides(q_out))
    r = _pack_rotation(*head, *qs, *_strides(k), *qo, *_NO_STRIDES, *_NO_STRIDES, *_NO_STRIDES, *tail)
    _launch(index, "cache_append", lib().sinkhorn_cache_append, r, c, _at(q), k.data_ptr(), v.data_ptr(),
            _strides3(v), _at(q_weight), _at(k_weight), _at(q_out), k_cache.data_ptr(), v_cache.data_ptr(),
            lengths_out.data_ptr())
    _changed(k_cache, v_cache, *given)
    return lengths_out, q_out


def paged_attention(q, k_cache, v_cache, page_table, key_lengths, *, scale=None, query_lengths=None, first=0,
                    recent=None, out=None, lse=None):
    """(out, lse): causal attention of new tokens over the paged cache that they were
    appended to (``sinkhorn_paged_attention``).

    q [B, Lq, Hq, d] holds the queries of the last n = query_lengths[b] (int32 [B], default
    Lq) of the key_lengths[b] keys (int32 [B]) of sequence b; the cache is laid out as for
    cache_append, query head h reads key head h // (Hq / Hkv). The row at place p sees
    key j <= p, and with `recent` only its `recent` last keys (itself among them) and the
    `first` first of the sequence. scale defaults to d ** -0.5. out [B, Lq, Hq, dv] has q's
    type, lse [B, Hq, Lq] is float32; rows without keys, and rows >= query_lengths[b], give
    0 and -inf. Keys on pages outside the cache take no part. d and dv are multiples of 16
    bytes, as are the cache's strides."""
    _head_tensor(q, "q")
    B, lq, hq, d = q.shape
    c, dv, hkv = _pages(q.dtype, B, None, d, k_cache, v_cache, page_table, key_lengths, "key_lengths")
    if hkv < 1 or hq < 1 or hq % hkv:
        raise ValueError(f"{hq} query heads are no multiple of {hkv} key heads")
    count = 0 if query_lengths is None else _plain(query_lengths, "query_lengths", torch.int32, (B,)).data_ptr()
    if recent is None:
        recent = 0
        if first:
            raise ValueError("first needs recent")
    elif recent < 1:
        raise ValueError("recent must be >= 1")
    # as large as the C side takes them: a longer one means the same
    first, recent = max(-1, min(int(first), (1 << 63) - 1)), min(int(recent), (1 << 63) - 1)
    given = out, lse
    if out is not None:
        _written(_head_tensor(out, "out", q.dtype, (B, lq, hq, dv)), "out")
    elif dv == d:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        out = q.new_empty((B, lq, hq, dv))
    if lse is None:
        lse = torch.empty((B, hq, lq), dtype=torch.float32, device=q.device)
    else:
        _plain(lse, "lse", torch.float32, (B, hq, lq))
    index = _same_device(q, (k_cache, v_cache, page_table, key_lengths, query_lengths, out, lse))
    a = _pack_attention(_ATTN_DTYPES[q.dtype], B, hq, hkv, d, dv, lq, 0, 1.0 / math.sqrt(max(d, 1)) if scale is None else float(scale),
                        *_strides(q), *_NO_STRIDES, *_NO_STRIDES, *_strides(out), *(_NO_STRIDES * 4), 0, 0, 0, count, 0)
    size = _i64()
    _check(lib().sinkhorn_paged_workspace(a, c, first, recent, ctypes.byref(size)), "paged_workspace")
    n = size.value
    ws = torch.empty(n, dtype=torch.uint8, device=q.device) if n else None
    _launch(index, "paged_attention", lib().sinkhorn_paged_attention, a, c, first, recent, q.data_ptr(),
            k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), lse.data_ptr(), _at(ws), n)
    _changed(*given)
    return out, lse


class Problem:
    """A problem handle (``sinkhorn_init``) over device clouds x [n,d], y [m,d]."""

    def __init__(self, x, y, a=None, b=None, cost_scale: float = 1.0, flags: int = 0):
        _dev(x, torch.float32, "x")
        _dev(y, torch.float32, "y")
        if x.dim() != 2 or y.dim() != 2 or x.shape[1] != y.shape[1]:
            raise ValueError("x and y must be [n,d] and [m,d]")
        self.n, self.d = x.shape
        self.m = y.shape[0]
        if a is not None:
            _dev(a, torch.float32, "a", (self.n,))
        if b is not None:
            _dev(b, torch.float32, "b", (self.m,))
        self.device = x.device
        self.cost_scale = float(cost_scale)
        self.flags = int(flags)
        h = ctypes.c_void_p()
        _check(lib().sinkhorn_init(ctypes.byref(h), _ptr(x), _ptr(y), _ptr(a), _ptr(b), self.n,
                                   self.m, self.d, self.cost_scale, self.flags, _stream(self.device)),
               "init")
        self._h = h

    def close(self):
        if getattr(self, "_h", None):
            lib().sinkhorn_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def info(self):
        """(n, m, d, cost_scale) as the handle holds them (``sinkhorn_problem_info``)."""
        n, m, d, sc = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int32(), ctypes.c_double()
        _check(lib().sinkhorn_problem_info(self._h, ctypes.byref(n), ctypes.byref(m), ctypes.byref(d),
                                           ctypes.byref(sc)), "problem_info")
        return n.value, m.value, d.value, sc.value

    def _pot(self, t, k, name):
        return _dev(t, torch.float32, name, (k,))

    def _new(self, k):
        return torch.empty(k, dtype=torch.float32, device=self.device)

    def halfstep_f(self, eps, g, out=None, f_prev=None):
        """f = f-step(g). Returns (f, R_row of (f_prev, g) or None)."""
        self._pot(g, self.m, "g")
        out = self._new(self.n) if out is None else self._pot(out, self.n, "out")
        res = _f64() if f_prev is not None else None
        if f_prev is not None:
            self._pot(f_prev, self.n, "f_prev")
        _check(lib().sinkhorn_halfstep_f(self._h, float(eps), _ptr(g), _ptr(out), _ptr(f_prev),
                                         ctypes.byref(res) if res is not None else None), "halfstep_f")
        _changed(out)
        return out, (res.value if res is not None else None)

    def halfstep_g(self, eps, f, out=None, g_prev=None):
        """g = g-step(f). Returns (g, R_col of (f, g_prev) or None)."""
        self._pot(f, self.n, "f")
        out = self._new(self.m) if out is None else self._pot(out, self.m, "out")
        res = _f64() if g_prev is not None else None
        if g_prev is not None:
            self._pot(g_prev, self.m, "g_prev")
        _check(lib().sinkhorn_halfstep_g(self._h, float(eps), _ptr(f), _ptr(out), _ptr(g_prev),
                                         ctypes.byref(res) if res is not None else None), "halfstep_g")
        _changed(out)
        return out, (res.value if res is not None else None)

    def marginal_residual(self, eps, f, g):
        self._pot(f, self.n, "f")
        self._pot(g, self.m, "g")
        r, c = _f64(), _f64()
        _check(lib().sinkhorn_marginal_residual(self._h, float(eps), _ptr(f), _ptr(g),
                                                ctypes.byref(r), ctypes.byref(c)), "marginal_residual")
        return r.value, c.value

    def solve(self, sched: Schedule, f=None, g=None, history: int = 256):
        """Annealed dense solve. Returns (f, g, report dict); report['status']
        is OK or NOT_CONVERGED; report['history'] holds the row residuals of
        the last `history` checks at eps_target."""
        f = torch.zeros(self.n, dtype=torch.float32, device=self.device) if f is None else self._pot(f, self.n, "f")
        g = torch.zeros(self.m, dtype=torch.float32, device=self.device) if g is None else self._pot(g, self.m, "g")
        sc = sched._c()
        rep = _ReportC()
        buf = (_f64 * max(1, history))()
        rep.history = ctypes.cast(buf, ctypes.POINTER(_f64))
        rep.history_cap = int(history)
        st = _check(lib().sinkhorn_solve(self._h, ctypes.byref(sc), _ptr(f), _ptr(g), ctypes.byref(rep)),
                    "solve")
        _changed(f, g)
        out = _struct_dict(rep)
        out["history"] = list(buf[:min(rep.history_len, history)])
        out["status"] = st
        return f, g, out

    def materialize_rows(self, eps, f, g, rows, T=None, row_max=None):
        """T[r] = plan row rows[r] (fp32 [k, m]); row_max optional [k]."""
        self._pot(f, self.n, "f")
        self._pot(g, self.m, "g")
        _dev(rows, torch.int64, "rows")
        k = rows.shape[0]
        T = torch.empty((k, self.m), dtype=torch.float32, device=self.device) if T is None else \
            _dev(T, torch.float32, "T", (k, self.m))
        if row_max is not None:
            _dev(row_max, torch.float32, "row_max", (k,))
        _check(lib().sinkhorn_materialize_rows(self._h, float(eps), _ptr(f), _ptr(g), _ptr(rows), k,
                                               _ptr(T), _ptr(row_max)), "materialize_rows")
        _changed(T, row_max)
        return T, row_max

    def materialize_rows_noalloc(self, eps, f, g, rows, T, row_max=None):
        """materialize_rows into caller buffers with no allocation in the call
        (T [k, m] fp32 is required; k <= 4096, m <= 2^21 when d <= 8)."""
        self._pot(f, self.n, "f")
        self._pot(g, self.m, "g")
        _dev(rows, torch.int64, "rows")
        k = rows.shape[0]
        _dev(T, torch.float32, "T", (k, self.m))
        if row_max is not None:
            _dev(row_max, torch.float32, "row_max", (k,))
        _check(lib().sinkhorn_materialize_rows_noalloc(self._h, float(eps), _ptr(f), _ptr(g), _ptr(rows),
                                                       k, _ptr(T), _ptr(row_max)),
               "materialize_rows_noalloc")
        _changed(T, row_max)
        return T, row_max

    def min_row(self, eps, f, g) -> float:
        self._pot(f, self.n, "f")
        self._pot(g, self.m, "g")
        out = ctypes.c_float()
        _check(lib().sinkhorn_min_row(self._h, float(eps), _ptr(f), _ptr(g), ctypes.byref(out)),
               "min_row")
        return out.value

    def morton_sort(self, side: int):
        """(codes int64 holding the uint64 bits, perm int32) of side 0 (x) or 1 (y)."""
        count = self.n if side == 0 else self.m
        codes = torch.empty(count, dtype=torch.int64, device=self.device)
        perm = torch.empty(count, dtype=torch.int32, device=self.device)
        _check(lib().sinkhorn_morton_sort(self._h, int(side), _ptr(perm), _ptr(codes)), "morton_sort")
        return codes, perm

    def block_screen(self, eps, f, g, B, delta_rel, transpose=False, cap=None):
        """Admitted tiles as (ptr int64, idx int32) device tensors."""
        self._pot(f, self.n, "f")
        self._pot(g, self.m, "g")
        nb = (self.m + B - 1) // B if transpose else (self.n + B - 1) // B
        ptr = torch.empty(nb + 1, dtype=torch.int64, device=self.device)
        nnz = _i64()
        if cap is None:
            code = lib().sinkhorn_block_screen(self._h, float(eps), _ptr(f), _ptr(g), B,
                                               float(delta_rel), int(transpose), _ptr(ptr), None, 0,
                                               ctypes.byref(nnz))
            if code not in (OK, ERR_CAPACITY):
                _check(code, "block_screen")
            cap = nnz.value
        idx = torch.empty(max(1, cap), dtype=torch.int32, device=self.device)
        _check(lib().sinkhorn_block_screen(self._h, float(eps), _ptr(f), _ptr(g), B, float(delta_rel),
                                           int(transpose), _ptr(ptr), _ptr(idx), cap,
                                           ctypes.byref(nnz)), "block_screen")
        return ptr, idx[: nnz.value]

    def verify_tiles(self, eps, f, g, B, delta_rel, ptr, idx):
        """Verified tiles of a row-major candidate list: (vptr, vidx, tptr,
        tidx) device tensors, the kept tiles row-major and column-major."""
        self._pot(f, self.n, "f")
        self._pot(g, self.m, "g")
        nb = (self.n + B - 1) // B
        mb = (self.m + B - 1) // B
        _dev(ptr, torch.int64, "ptr", (nb + 1,))
        nnz = int(idx.shape[0])
        if nnz:
            _dev(idx, torch.int32, "idx")
        vptr = torch.empty(nb + 1, dtype=torch.int64, device=self.device)
        tptr = torch.empty(mb + 1, dtype=torch.int64, device=self.device)
        vidx = torch.empty(max(1, nnz), dtype=torch.int32, device=self.device)
        tidx = torch.empty(max(1, nnz), dtype=torch.int32, device=self.device)
        kept = _i64()
        _check(lib().sinkhorn_verify_tiles(self._h, float(eps), _ptr(f), _ptr(g), int(B),
                                           float(delta_rel), _ptr(ptr), _ptr(idx) if nnz else None,
                                           _ptr(vptr), _ptr(vidx), _ptr(tptr), _ptr(tidx),
                                           ctypes.byref(kept)), "verify_tiles")
        k = kept.value
        return vptr, vidx[:k], tptr, tidx[:k]

    def sparse_halfstep_f(self, eps, g, B, ptr, idx, out=None, f_prev=None):
        self._pot(g, self.m, "g")
        out = self._new(self.n) if out is None else self._pot(out, self.n, "out")
        res = _f64() if f_prev is not None else None
        _check(lib().sinkhorn_sparse_halfstep_f(self._h, float(eps), _ptr(g), B, _ptr(ptr), _ptr(idx),
                                                _ptr(out), _ptr(f_prev),
                                                ctypes.byref(res) if res is not None else None),
               "sparse_halfstep_f")
        _changed(out)
        return out, (res.value if res is not None else None)

    def sparse_halfstep_g(self, eps, f, B, ptr, idx, out=None, g_prev=None):
        self._pot(f, self.n, "f")
        out = self._new(self.m) if out is None else self._pot(out, self.m, "out")
        res = _f64() if g_prev is not None else None
        _check(lib().sinkhorn_sparse_halfstep_g(self._h, float(eps), _ptr(f), B, _ptr(ptr), _ptr(idx),
                                                _ptr(out), _ptr(g_prev),
                                                ctypes.byref(res) if res is not None else None),
               "sparse_halfstep_g")
        _changed(out)
        return out, (res.value if res is not None else None)

    def sparsify(self, eps, f, g, threshold: float, batch: int = 1024, cap=None):
        """(row_ptr, col, val): the plan entries >= threshold as CSR (int64,
        int32, fp32 device tensors). With cap=None the count is taken first
        (row_ptr only), then the entries are written into buffers of that size."""
        self._pot(f, self.n, "f")
        self._pot(g, self.m, "g")
        row_ptr = torch.empty(self.n + 1, dtype=torch.int64, device=self.device)
        nnz = _i64()
        if cap is None:
            _check(lib().sinkhorn_sparsify(self._h, float(eps), _ptr(f), _ptr(g), float(threshold), int(batch),
                                           _ptr(row_ptr), None, None, 0, ctypes.byref(nnz)), "sparsify")
            cap = nnz.value
        col = torch.empty(max(1, cap), dtype=torch.int32, device=self.device)
        val = torch.empty(max(1, cap), dtype=torch.float32, device=self.device)
        st = lib().sinkhorn_sparsify(self._h, float(eps), _ptr(f), _ptr(g), float(threshold), int(batch),
                                     _ptr(row_ptr), _ptr(col), _ptr(val), int(cap), ctypes.byref(nnz))
        if st != OK:
            raise SinkhornError(st, "sparsify")
        k = nnz.value
        return row_ptr, col[:k], val[:k]

    def barycentric(self, eps, g, f_hint=None, T=None, grad=None, want_T=True, want_grad=True):
        """(T, grad): barycentric projection of the plan rows and the source
        gradient 2 s a_i (x_i - T_i), [n, d] fp32 each (None when not wanted).
        f_hint, the f-step potential of g, only speeds up the loop."""
        self._pot(g, self.m, "g")
        if f_hint is not None:
            self._pot(f_hint, self.n, "f_hint")
        T, grad = self._bary_out(T, grad, want_T, want_grad)
        _check(lib().sinkhorn_barycentric(self._h, float(eps), _ptr(g), _ptr(f_hint), _ptr(T), _ptr(grad)),
               "barycentric")
        _changed(T, grad)
        return T, grad

    def sparse_barycentric(self, eps, g, B, ptr, idx, f_hint=None, T=None, grad=None, want_T=True,
                           want_grad=True):
        """The projection and gradient restricted to the admitted tiles."""
        self._pot(g, self.m, "g")
        if f_hint is not None:
            self._pot(f_hint, self.n, "f_hint")
        T, grad = self._bary_out(T, grad, want_T, want_grad)
        _check(lib().sinkhorn_sparse_barycentric(self._h, float(eps), _ptr(g), _ptr(f_hint), int(B), _ptr(ptr),
                                                 _ptr(idx), _ptr(T), _ptr(grad)), "sparse_barycentric")
        _changed(T, grad)
        return T, grad

    def _bary_out(self, T, grad, want_T, want_grad):
        shape = (self.n, self.d)
        if T is None and want_T:
            T = torch.empty(shape, dtype=torch.float32, device=self.device)
        elif T is not None:
            _dev(T, torch.float32, "T", shape)
        if grad is None and want_grad:
            grad = torch.empty(shape, dtype=torch.float32, device=self.device)
        elif grad is not None:
            _dev(grad, torch.float32, "grad", shape)
        return T, grad

    def profile_enable(self, kinds: int = PROF_DENSE):
        """Bracket every later launch of the selected kernel kinds (PROF_*
        bits; 0 stops) with HIP events on the library's stream."""
        _check(lib().sinkhorn_profile_enable(self._h, int(kinds)), "profile_enable")

    def profile_read(self):
        """(kernel_ms, launches, pairs) recorded since the last read (syncs)."""
        ms, n, pairs = _f64(), _i64(), _f64()
        _check(lib().sinkhorn_profile_read(self._h, ctypes.byref(ms), ctypes.byref(n), ctypes.byref(pairs)),
               "profile_read")
        return ms.value, n.value, pairs.value

    def sampled_residual(self, eps, f, g, side=0, k=1024, seed=0):
        """(estimate, standard error) of one side's L1 marginal residual from k
        drawn rows (side 0: x, side 1: y)."""
        self._pot(f, self.n, "f")
        self._pot(g, self.m, "g")
        est, se = _f64(), _f64()
        _check(lib().sinkhorn_sampled_residual(self._h, float(eps), _ptr(f), _ptr(g), int(side), int(k),
                                               int(seed), ctypes.byref(est), ctypes.byref(se)),
               "sampled_residual")
        return est.value, se.value

    def solve_multiscale(self, prm: MultiscaleParams, f=None, g=None):
        f = self._new(self.n) if f is None else self._pot(f, self.n, "f")
        g = self._new(self.m) if g is None else self._pot(g, self.m, "g")
        c = prm._c()
        rep = _MultiscaleReportC()
        st = _check(lib().sinkhorn_solve_multiscale(self._h, ctypes.byref(c), _ptr(f), _ptr(g),
                                                    ctypes.byref(rep)), "solve_multiscale")
        _changed(f, g)
        out = _struct_dict(rep)
        out["status"] = st
        return f, g, out

