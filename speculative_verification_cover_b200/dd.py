"""ctypes binding of libdd.so (include/dd.h), one Python function per C entry point.

Argument marshalling only: sizes are read off the tensors, pointers passed
as `data_ptr()`, the stream defaults to torch's current CUDA stream. Every
computation runs in libdd's CUDA kernels; there is no CPU fallback -- CPU
tensors, a missing library or a non-OK status raise.

With DD_CHECK_BOUNDS=1 in the environment (read when the library is first
loaded) the binding loads libdd_checked.so, the same library built with device
index checks (see dd_bounds_checked in include/dd.h).
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from dataclasses import dataclass, fields

import torch

from . import build

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdd.so")
CHECKED_LIB_PATH = os.path.join(_HERE, "libdd_checked.so")

DD_OK, DD_ERR_INVALID_ARG, DD_ERR_UNSUPPORTED, DD_ERR_CUDA, DD_ERR_TIMEOUT, DD_ERR_BOUNDS = range(6)
DD_F32, DD_BF16 = 0, 1
POLICIES = {"trust": 0, "kl": 1, "conf": 2, "cover": 3, "coupled": 4, "kl_stochastic": 5}
DD_NONE, DD_KEEP, DD_REPLACE, DD_REMASK, DD_COMMIT = 0, 1, 2, 3, 4
DD_MASK_TOKEN = -1

# Every symbol include/dd.h declares.
EXPORTED = (
    "dd_dualview_attention", "dd_dualview_attention_ex", "dd_dualview_attention_ex2",
    "dd_dualview_attention_workspace_size", "dd_verify_logits",
    "dd_verify_logits_workspace_size", "dd_verify_logits_static",
    "dd_coupled_gumbel", "dd_select_seeds", "dd_select_seeds_ex", "dd_decide",
    "dd_paged_attention", "dd_paged_attention_workspace_size", "dd_cache_evict",
    "dd_beam_select", "dd_beam_select_workspace_size", "dd_beam_reorder", "dd_paged_fork",
    "dd_status_string",
    "dd_get_device_error", "dd_set_spin_limit", "dd_selftest_bounded_wait",
    "dd_selftest_gumbel_screen", "dd_bounds_checked", "dd_selftest_bounds_check",
)


class DDError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")


class _RowStats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "lse_t", "lse_d", "conf_t", "p_sample_t", "entropy_t", "kl_dt",
        "argmax_t", "argmax_d", "sample_t", "sample_d")]


class _DecideParams(ctypes.Structure):
    _fields_ = [("policy", ctypes.c_int), ("tau_kl", ctypes.c_float),
                ("tau_conf", ctypes.c_float), ("temperature", ctypes.c_float),
                ("tau_commit", ctypes.c_float), ("min_commit", ctypes.c_int),
                ("seed", ctypes.c_uint64), ("step", ctypes.c_uint64)]


class _PagedCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("layer_stride", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("layers", ctypes.c_int), ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("Hkv", ctypes.c_int), ("d", ctypes.c_int), ("dtype", ctypes.c_int),
                ("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("max_pages", ctypes.c_int)]


class _RowState(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("row_bytes", ctypes.c_int64),
                ("src_stride", ctypes.c_int64), ("dst_stride", ctypes.c_int64)]


_lib = None


def lib_path() -> str:
    """The library lib() loads: the checked build when DD_CHECK_BOUNDS is set to
    anything but 0 or the empty string, libdd.so otherwise."""
    return CHECKED_LIB_PATH if os.environ.get("DD_CHECK_BOUNDS", "0") not in ("", "0") else LIB_PATH


def lib():
    """Load the library (once). Raises ImportError if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -m speculative_verification_cover_b200.build`")
    L = ctypes.CDLL(path)
    P, I, I64, U64, F, SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint64,
                             ctypes.c_float, ctypes.c_size_t)
    L.dd_dualview_attention.argtypes = [P] * 8 + [I] * 5 + [F, I, I] + [P] * 5 + [SZ, P]
    L.dd_dualview_attention.restype = I
    L.dd_dualview_attention_ex.argtypes = [P] * 8 + [I] * 5 + [F, I, I, I, F] + [P] * 5 + [SZ, P]
    L.dd_dualview_attention_ex.restype = I
    L.dd_dualview_attention_ex2.argtypes = [P] * 8 + [I] * 5 + [F, I, I, I, F] + [P] * 5 + [SZ, P, P]
    L.dd_dualview_attention_ex2.restype = I
    L.dd_dualview_attention_workspace_size.argtypes = [I] * 5
    L.dd_dualview_attention_workspace_size.restype = SZ
    L.dd_verify_logits.argtypes = [P, P, I, I, I, I, I64, I, F, U64, U64,
                                   ctypes.POINTER(_RowStats), P, SZ, P]
    L.dd_verify_logits.restype = I
    L.dd_verify_logits_static.argtypes = [P, P, I, I, I, I, I64, I, F, U64, U64,
                                          ctypes.POINTER(_RowStats), P]
    L.dd_verify_logits_static.restype = I
    L.dd_verify_logits_workspace_size.argtypes = [I, I, I, I]
    L.dd_verify_logits_workspace_size.restype = SZ
    L.dd_coupled_gumbel.argtypes = [U64, U64, I, I, I, I64, I, P, P]
    L.dd_coupled_gumbel.restype = I
    L.dd_select_seeds.argtypes = [P, I, I, P, P, P, I, I, I, P, P, P, P]
    L.dd_select_seeds.restype = I
    L.dd_select_seeds_ex.argtypes = [P, I, I, P, P, P, I, I, I, F, P, P, P, P, P]
    L.dd_select_seeds_ex.restype = I
    L.dd_decide.argtypes = [ctypes.POINTER(_DecideParams), P, P, P, ctypes.POINTER(_RowStats),
                            I, I, I, I, P, P, P, P]
    L.dd_decide.restype = I
    C = ctypes.POINTER(_PagedCache)
    L.dd_paged_attention.argtypes = [P, I64, P, P, I64, C, P, I, I, I, F, P, P, P, P, I64, P, SZ, P]
    L.dd_paged_attention.restype = I
    L.dd_paged_attention_workspace_size.argtypes = [I] * 6
    L.dd_paged_attention_workspace_size.restype = SZ
    L.dd_cache_evict.argtypes = [C, P, I, I, I, I, I, P, P, I64, P, P, P, P, P]
    L.dd_cache_evict.restype = I
    L.dd_beam_select.argtypes = [P, I, I, I, I, I64, P, P, I, P, P, P, P, P, SZ, P]
    L.dd_beam_select.restype = I
    L.dd_beam_select_workspace_size.argtypes = [I] * 4
    L.dd_beam_select_workspace_size.restype = SZ
    L.dd_beam_reorder.argtypes = [P, I, I, ctypes.POINTER(_RowState), I, P]
    L.dd_beam_reorder.restype = I
    L.dd_paged_fork.argtypes = [C, P, I, I, P, P, P, I64, P, P]
    L.dd_paged_fork.restype = I
    L.dd_status_string.argtypes = [I]
    L.dd_status_string.restype = ctypes.c_char_p
    L.dd_get_device_error.argtypes = [P]
    L.dd_get_device_error.restype = I
    L.dd_set_spin_limit.argtypes = [ctypes.c_uint32]
    L.dd_set_spin_limit.restype = ctypes.c_uint32
    L.dd_selftest_bounded_wait.argtypes = [ctypes.c_uint32, P]
    L.dd_selftest_bounded_wait.restype = I
    L.dd_selftest_gumbel_screen.argtypes = [P, P, P, P, I, ctypes.POINTER(F), P]
    L.dd_selftest_gumbel_screen.restype = I
    L.dd_bounds_checked.argtypes = []
    L.dd_bounds_checked.restype = I
    L.dd_selftest_bounds_check.argtypes = [I, I, ctypes.POINTER(I), P]
    L.dd_selftest_bounds_check.restype = I
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().dd_status_string(int(status)).decode()


def _check(fn, status):
    if status != DD_OK:
        raise DDError(fn, status)


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("libdd takes device memory: tensor is on the CPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _dtype_code(t):
    if t.dtype == torch.float32:
        return DD_F32
    if t.dtype == torch.bfloat16:
        return DD_BF16
    raise ValueError(f"unsupported dtype {t.dtype}")


@dataclass
class RowStats:
    """Per-row outputs of dd_verify_logits, each a [B, R] device tensor (or None)."""
    lse_t: torch.Tensor | None = None
    lse_d: torch.Tensor | None = None
    conf_t: torch.Tensor | None = None
    p_sample_t: torch.Tensor | None = None
    entropy_t: torch.Tensor | None = None
    kl_dt: torch.Tensor | None = None
    argmax_t: torch.Tensor | None = None
    argmax_d: torch.Tensor | None = None
    sample_t: torch.Tensor | None = None
    sample_d: torch.Tensor | None = None

    @classmethod
    def empty(cls, B, R, device="cuda"):
        f = dict(dtype=torch.float32, device=device)
        i = dict(dtype=torch.int32, device=device)
        return cls(*(torch.empty(B, R, **f) for _ in range(6)),
                   *(torch.empty(B, R, **i) for _ in range(4)))

    def _c(self):
        return _RowStats(*(_ptr(getattr(self, f.name)) for f in fields(self)))


def dd_dualview_attention_workspace_size(B, L, Hq, Hkv, d) -> int:
    return int(lib().dd_dualview_attention_workspace_size(B, L, Hq, Hkv, d))


def dd_dualview_attention(q, k_cur, v_cur, k_prev, v_prev, is_seed, is_masked, is_new,
                          out, lse, d_in=None, d_out=None, workspace=None, softmax_scale=0.0,
                          accumulate_stats=False, stream=None):
    """q [B,L,Hq,d]; k/v [B,L,Hkv,d]; masks [B,L] uint8; out like q; lse [B,Hq,L] fp32;
    d_in, d_out [B,L] fp32; workspace: uint8 device tensor of
    dd_dualview_attention_workspace_size(...) bytes."""
    B, L, Hq, d = q.shape
    Hkv = k_cur.shape[2]
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().dd_dualview_attention(
        _ptr(q), _ptr(k_cur), _ptr(v_cur), _ptr(k_prev), _ptr(v_prev), _ptr(is_seed),
        _ptr(is_masked), _ptr(is_new), B, L, Hq, Hkv, d, float(softmax_scale), _dtype_code(q),
        int(bool(accumulate_stats)), _ptr(out), _ptr(lse), _ptr(d_in), _ptr(d_out),
        _ptr(workspace), nbytes, _stream(stream))
    _check("dd_dualview_attention", st)


def dd_dualview_attention_ex(q, k_cur, v_cur, k_prev, v_prev, is_seed, is_masked, is_new,
                             out, lse, d_in=None, d_out=None, workspace=None, q_begin=0,
                             accumulate_stats=False, stats_weight=1.0, softmax_scale=0.0,
                             stream=None, prep_done=None):
    """One layer of a multi-layer pass with a prefix cache: query rows from q_begin on,
    this layer's d_in / d_out weighted by stats_weight (see include/dd.h). prep_done: a
    torch.cuda.Event recorded right after the mask preparation (dd_dualview_attention_ex2)."""
    B, L, Hq, d = q.shape
    Hkv = k_cur.shape[2]
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    args = (_ptr(q), _ptr(k_cur), _ptr(v_cur), _ptr(k_prev), _ptr(v_prev), _ptr(is_seed),
            _ptr(is_masked), _ptr(is_new), B, L, Hq, Hkv, d, float(softmax_scale), _dtype_code(q),
            int(q_begin), int(bool(accumulate_stats)), float(stats_weight), _ptr(out), _ptr(lse),
            _ptr(d_in), _ptr(d_out), _ptr(workspace), nbytes)
    if prep_done is None:
        st = lib().dd_dualview_attention_ex(*args, _stream(stream))
        _check("dd_dualview_attention_ex", st)
    else:
        if not prep_done.cuda_event:
            raise ValueError("prep_done has no CUDA event yet: record it once first")
        st = lib().dd_dualview_attention_ex2(*args, ctypes.c_void_p(prep_done.cuda_event),
                                             _stream(stream))
        _check("dd_dualview_attention_ex2", st)


def dd_verify_logits_workspace_size(B, R, V, dtype) -> int:
    code = dtype if isinstance(dtype, int) else _dtype_code(torch.empty(0, dtype=dtype))
    return int(lib().dd_verify_logits_workspace_size(B, R, V, code))


def dd_verify_logits(logits_t, logits_d, out: RowStats, pos_offset=0, temperature=0.0, seed=0,
                     step=0, workspace=None, stream=None):
    """logits [B,R,V]; a view narrowed from a wider [B,R,ld] buffer is accepted
    (the row stride ld is read from the tensor). out: RowStats of [B,R] tensors.
    workspace: uint8 device tensor of dd_verify_logits_workspace_size(...) bytes
    (allocated here with torch when not given)."""
    B, R, V = logits_t.shape
    if workspace is None:
        workspace = torch.empty(dd_verify_logits_workspace_size(B, R, V, logits_t.dtype),
                                dtype=torch.uint8, device=logits_t.device)
    if logits_t.stride(2) != 1 or logits_t.stride(0) != R * logits_t.stride(1):
        raise ValueError("logits must be [B,R,V] with unit vocabulary stride and packed rows")
    if logits_d.shape != logits_t.shape or logits_d.stride() != logits_t.stride():
        raise ValueError("verifier and drafter logits must have the same shape and strides")
    if not (logits_t.is_cuda and logits_d.is_cuda):
        raise ValueError("libdd takes device memory: logits are on the CPU")
    ld = logits_t.stride(1)
    st = lib().dd_verify_logits(
        ctypes.c_void_p(logits_t.data_ptr()), ctypes.c_void_p(logits_d.data_ptr()),
        _dtype_code(logits_t), B, R, V, ld, int(pos_offset), float(temperature),
        int(seed) & (2**64 - 1), int(step) & (2**64 - 1), ctypes.byref(out._c()),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check("dd_verify_logits", st)


def dd_verify_logits_static(logits_t, logits_d, out: RowStats, pos_offset=0, temperature=0.0,
                            seed=0, step=0, stream=None):
    """dd_verify_logits without a workspace: for callers that cannot allocate device
    memory, the partial states live in a fixed array inside libdd (see include/dd.h for
    its size limit and for why concurrent calls must not overlap)."""
    B, R, V = logits_t.shape
    if logits_t.stride(2) != 1 or logits_t.stride(0) != R * logits_t.stride(1):
        raise ValueError("logits must be [B,R,V] with unit vocabulary stride and packed rows")
    if logits_d.shape != logits_t.shape or logits_d.stride() != logits_t.stride():
        raise ValueError("verifier and drafter logits must have the same shape and strides")
    if not (logits_t.is_cuda and logits_d.is_cuda):
        raise ValueError("libdd takes device memory: logits are on the CPU")
    st = lib().dd_verify_logits_static(
        ctypes.c_void_p(logits_t.data_ptr()), ctypes.c_void_p(logits_d.data_ptr()),
        _dtype_code(logits_t), B, R, V, logits_t.stride(1), int(pos_offset), float(temperature),
        int(seed) & (2**64 - 1), int(step) & (2**64 - 1), ctypes.byref(out._c()), _stream(stream))
    _check("dd_verify_logits_static", st)


def dd_coupled_gumbel(g, seed=0, step=0, pos_offset=0, stream=None):
    """Fill g [B,R,V] fp32 with the shared Gumbel noise of dd_verify_logits."""
    B, R, V = g.shape
    st = lib().dd_coupled_gumbel(int(seed) & (2**64 - 1), int(step) & (2**64 - 1), B, R, V,
                                 g.stride(1), int(pos_offset), _ptr(g), _stream(stream))
    _check("dd_coupled_gumbel", st)


def dd_select_seeds(entropy, pos_offset, d_in, d_out, eligible, seeds, is_seed=None, score=None,
                    stream=None):
    """entropy [B,R]; d_in, d_out [B,L] fp32; eligible [B,L] u8; seeds [B,k] int32 out."""
    B, L = d_in.shape
    R = entropy.shape[1] if entropy is not None else 0
    k = seeds.shape[1] if seeds is not None else 0
    st = lib().dd_select_seeds(_ptr(entropy), R, int(pos_offset), _ptr(d_in), _ptr(d_out),
                               _ptr(eligible), B, L, k, _ptr(seeds), _ptr(is_seed), _ptr(score),
                               _stream(stream))
    _check("dd_select_seeds", st)


def dd_select_seeds_ex(entropy, pos_offset, d_in, d_out, eligible, seeds, is_seed=None,
                       score=None, count=None, min_score=float("-inf"), stream=None):
    """dd_select_seeds with an adaptive size: only scores >= min_score compete;
    count [B] int32 (optional) receives the number chosen per sequence."""
    B, L = d_in.shape
    R = entropy.shape[1] if entropy is not None else 0
    k = seeds.shape[1] if seeds is not None else 0
    st = lib().dd_select_seeds_ex(_ptr(entropy), R, int(pos_offset), _ptr(d_in), _ptr(d_out),
                                  _ptr(eligible), B, L, k, float(min_score), _ptr(seeds),
                                  _ptr(is_seed), _ptr(score), _ptr(count), _stream(stream))
    _check("dd_select_seeds_ex", st)


def dd_decide(policy, tokens, is_seed, eligible, stats: RowStats, pos_offset, decision,
              new_tokens, accepted=None, tau_kl=0.5, tau_conf=0.9, temperature=0.0,
              tau_commit=0.0, min_commit=0, seed=0, step=0, stream=None):
    """tokens [B,L] int32; stats from dd_verify_logits ([B,R]); decision [B,L] u8,
    new_tokens [B,L] int32, accepted [B] u8 outputs. tau_commit > 0 turns on dynamic
    threshold decoding of masked positions; seed / step key the draws of the
    stochastic KL policy."""
    B, L = tokens.shape
    ref = stats.argmax_t if stats.argmax_t is not None else stats.sample_t
    R = ref.shape[1]
    p = _DecideParams(POLICIES[policy] if isinstance(policy, str) else int(policy),
                      float(tau_kl), float(tau_conf), float(temperature), float(tau_commit),
                      int(min_commit), int(seed) & (2**64 - 1), int(step) & (2**64 - 1))
    st = lib().dd_decide(ctypes.byref(p), _ptr(tokens), _ptr(is_seed), _ptr(eligible),
                         ctypes.byref(stats._c()), B, L, R, int(pos_offset), _ptr(decision),
                         _ptr(new_tokens), _ptr(accepted), _stream(stream))
    _check("dd_decide", st)


# ------------------------------------------------------------------ cached decoding
# Every tensor of a call is checked here -- device, type, shape, layout -- before its
# address reaches the library; the call runs on that device, on `stream` (None: its
# current stream), and a workspace that is not given is allocated for that stream. A
# decode step makes many small calls, so a tensor's checks are one compiled call
# (csrc/dd_args.cpp), and what is wrong is looked for only once something is.
def _gpu(t, name):
    """Index of the device a call runs on: that of its first tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    gpu = t.get_device()
    if gpu < 0:
        raise ValueError(f"libdd takes device memory: {name} is on the CPU")
    return gpu


def _refuse(t, name, dtype, shape, gpu, rows):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.get_device() != gpu:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on cuda:{gpu}")
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous" + (" within a row" if rows else ""))


_host = None  # csrc/dd_args.cpp: the checks, and the library's calls without ctypes


def _load_host():
    """Load the binding's compiled part and give it the library's entry points."""
    global _host, _arg, _rows
    L = lib()
    path = build.args_path()
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -m speculative_verification_cover_b200.build`")
    spec = importlib.util.spec_from_file_location(__package__ + "._args", path)
    _args = importlib.util.module_from_spec(spec)
    _args.set_refuse(_refuse)
    for name in ("dd_paged_attention", "dd_cache_evict", "dd_beam_select", "dd_beam_reorder", "dd_paged_fork"):
        getattr(_args, "bind_" + name)(ctypes.cast(getattr(L, name), ctypes.c_void_p).value)
    _arg, _rows, _host = _args.arg, _args.rows, _args
    return _args


def _arg(t, name, dtype, shape, gpu):
    """Address of a contiguous tensor of the given type, shape and device."""
    _load_host()
    return _arg(t, name, dtype, shape, gpu)


def _rows(t, name, dtype, shape, gpu):
    """Address and row stride of a tensor whose rows (all dimensions but the first) are
    contiguous."""
    _load_host()
    return _rows(t, name, dtype, shape, gpu)


def _scratch(nbytes, gpu, stream):
    """Device scratch that the allocator reuses in the order of `stream`."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=f"cuda:{gpu}")
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), f"cuda:{gpu}")
    with torch.cuda.stream(s):
        return torch.empty(nbytes, dtype=torch.uint8, device=f"cuda:{gpu}")


def _workspace(t, gpu):
    """Address and bytes of a caller's workspace."""
    got = (_host or _load_host()).workspace(t, gpu)
    if got is not None:
        return got
    if not isinstance(t, torch.Tensor):
        raise TypeError("workspace: expected a torch.Tensor")
    if t.get_device() != gpu:
        raise ValueError(f"workspace is on {t.device}, the call's other tensors on cuda:{gpu}")
    raise ValueError("workspace must be contiguous")


def _call(name, gpu, stream, *args):
    """A library call on device `gpu` (made current only where it is not), on `stream`."""
    fn = getattr(_host or _load_host(), name)
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(gpu)
    else:
        s = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)
    if torch._C._cuda_getDevice() == gpu:
        st = fn(*args, s)
    else:
        with torch.cuda.device(gpu):
            st = fn(*args, s)
    if st:
        raise DDError(name, st)


def _overlaps(shape, stride):
    """Whether two elements of a tensor may be one (an expanded view, say)."""
    extent = 1
    for st, n in sorted((st, n) for n, st in zip(shape, stride) if n > 1):
        if st < extent:
            return True
        extent += st * (n - 1)
    return False


class PagedCache:
    """A paged K/V cache: k, v [pages, page_size, Hkv, d] or, for several layers that share
    page ids, [layers, pages, page_size, Hkv, d], and page_table [N, max_pages] int32.
    k and v have the same shape and strides, any strides with a unit last one (so a pool
    stored heads first is passed as its transposed view). A page id below 0 is a hole.
    Pools whose elements share memory (expanded views, one tensor as both k and v) are
    read only: calls that would write them are refused."""

    def __init__(self, k, v, page_table):
        gpu = _gpu(k, "k")
        if _gpu(v, "v") != gpu or _gpu(page_table, "page_table") != gpu:
            raise ValueError("k, v and page_table must be on one device")
        if k.dim() not in (4, 5) or v.shape != k.shape or v.stride() != k.stride():
            raise ValueError("k and v must be [pages, page_size, Hkv, d] or [layers, pages, "
                             "page_size, Hkv, d], of the same shape and strides")
        if v.dtype != k.dtype:
            raise ValueError("k and v must have the same dtype")
        if k.numel() == 0:
            raise ValueError("k and v must not be empty")
        if k.stride(-1) != 1:
            raise ValueError("k and v must have a unit stride over d")
        if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.numel() == 0:
            raise ValueError("page_table must be a non-empty [N, max_pages] int32 tensor")
        if page_table.stride(1) != 1 and page_table.shape[1] > 1:
            raise ValueError("page_table must be contiguous within a row")
        self.k, self.v, self.page_table, self.gpu, self.dtype = k, v, page_table, gpu, k.dtype
        *layers, self.n_pages, self.page_size, self.Hkv, self.d = k.shape
        self.layers = layers[0] if layers else 1
        self.N, self.max_pages = page_table.shape
        self.slots = self.max_pages * self.page_size  # what a table row has room for
        s = [st if n > 1 else 0 for n, st in zip(k.shape, k.stride())]
        self._c = _PagedCache(k.data_ptr(), v.data_ptr(), s[0] if layers else 0, *s[-4:-1],
                              self.layers, self.n_pages, self.page_size, self.Hkv, self.d,
                              _dtype_code(k), page_table.data_ptr(),
                              page_table.stride(0) if self.N > 1 else self.max_pages, self.max_pages)
        self._ref = ctypes.addressof(self._c)  # lives as long as the cache
        self.read_only = k.data_ptr() == v.data_ptr() or _overlaps(k.shape, k.stride())

    def layer(self, i):
        """One layer's cache of a several-layer one (the same memory and page table)."""
        if self.k.dim() != 5:
            raise ValueError("the cache has a single layer")
        return PagedCache(self.k[i], self.v[i], self.page_table)

    def with_table(self, page_table):
        """The same pools under another page table (dd_paged_fork's, say)."""
        return PagedCache(self.k, self.v, page_table)

    def _fits(self, n, gpu):
        if n != self.N:
            raise ValueError(f"the page table has {self.N} rows, the call {n} sequences")
        if gpu != self.gpu:
            raise ValueError(f"the cache is on cuda:{self.gpu}, the call's tensors on cuda:{gpu}")

    def _written(self):
        if self.read_only:
            raise ValueError("elements of k and v share memory: the cache can only be read")


def dd_paged_attention_workspace_size(B, Hq, Hkv, d, max_len, with_mass=False) -> int:
    return int(lib().dd_paged_attention_workspace_size(B, Hq, Hkv, d, max_len, int(bool(with_mass))))


def dd_paged_attention(q, cache: PagedCache, lengths, out, lse=None, k_new=None, v_new=None,
                       mass=None, mass_out=None, max_len=None, workspace=None, softmax_scale=0.0,
                       stream=None):
    """Attention of one new token per sequence over a paged cache. q [B,Hq,d] (its rows may
    be a slice of wider ones); lengths [B] int32; out [B,Hq,d]; lse [B,Hq] fp32;
    k_new, v_new [B,Hkv,d]: appended at slot lengths - 1 first; mass (None: zero),
    mass_out [B,M] fp32 with M >= max_len: the attention mass per slot, added up. max_len:
    bound on lengths (None: the smaller of M and what the page table has room for)."""
    gpu = _gpu(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, d]")
    shape = q.shape
    B, Hq, d = shape
    Hkv, dtype = cache.Hkv, cache.dtype
    cache._fits(B, gpu)
    if d != cache.d or Hq % Hkv:
        raise ValueError(f"q {tuple(shape)} does not fit a cache of {Hkv} heads of {cache.d}")
    qp, qs = _rows(q, "q", dtype, shape, gpu)
    op = _arg(out, "out", dtype, shape, gpu)
    np_ = _arg(lengths, "lengths", torch.int32, (B,), gpu)
    lp = None if lse is None else _arg(lse, "lse", torch.float32, (B, Hq), gpu)
    kp = vp = None
    ns = 0
    if k_new is not None or v_new is not None:
        cache._written()
        kp, ns = _rows(k_new, "k_new", dtype, (B, Hkv, d), gpu)
        vp, vs = _rows(v_new, "v_new", dtype, (B, Hkv, d), gpu)
        if ns != vs and B > 1:
            raise ValueError("k_new and v_new must have the same strides")
    mi = mo = None
    ms = 0
    if mass_out is not None:
        rows = (B, mass_out.shape[-1])
        mo, ms = _rows(mass_out, "mass_out", torch.float32, rows, gpu)
        if mass is not None:
            mi, vs = _rows(mass, "mass", torch.float32, rows, gpu)
            if ms != vs and B > 1:
                raise ValueError("mass and mass_out must have the same strides")
        if B == 1:
            ms = rows[1]
        if max_len is None:
            max_len = min(cache.slots, rows[1])
        elif max_len > rows[1]:  # the library sees the row stride alone, which may be larger
            raise DDError("dd_paged_attention", DD_ERR_INVALID_ARG)
    elif mass is not None:
        raise ValueError("mass without mass_out")
    max_len = cache.slots if max_len is None else int(max_len)
    if workspace is None:
        workspace = _scratch(dd_paged_attention_workspace_size(B, Hq, Hkv, d, max_len, mo is not None), gpu,
                             stream)
    wp, wb = _workspace(workspace, gpu)
    _call("dd_paged_attention", gpu, stream, qp, qs, kp, vp, ns, cache._ref, np_, B, Hq, max_len,
          softmax_scale, op, lp, mi, mo, ms, wp, wb)


def dd_cache_evict(cache: PagedCache, lengths, mass, pos, budget, mass_out, pos_out, lengths_out,
                   sink=0, recent=0, src=None, max_len=None, stream=None):
    """Bring every sequence down to `budget` slots by accumulated mass. mass, mass_out
    [N,M] fp32, pos, pos_out, src (optional output: each new slot's old one) [N,M] int32,
    M >= max_len; lengths, lengths_out [N] int32; outputs are other tensors than inputs.
    max_len: bound on lengths (None: the smaller of M and what the page table has room for)."""
    gpu = _gpu(mass, "mass")
    if mass.dim() != 2:
        raise ValueError("mass must be [N, M]")
    shape = mass.shape
    N, M = shape
    cache._fits(N, gpu)
    cache._written()
    max_len = min(M, cache.slots) if max_len is None else int(max_len)
    i32, f32 = torch.int32, torch.float32
    mi = _arg(mass, "mass", f32, shape, gpu)
    pi = _arg(pos, "pos", i32, shape, gpu)
    mo = _arg(mass_out, "mass_out", f32, shape, gpu)
    po = _arg(pos_out, "pos_out", i32, shape, gpu)
    sp = None if src is None else _arg(src, "src", i32, shape, gpu)
    ln = _arg(lengths, "lengths", i32, (N,), gpu)
    lo = _arg(lengths_out, "lengths_out", i32, (N,), gpu)
    _call("dd_cache_evict", gpu, stream, cache._ref, ln, N, max_len, int(budget), int(sink), int(recent),
          mi, pi, M, mo, po, sp, lo)


def dd_beam_select_workspace_size(B, K, V, dtype) -> int:
    code = dtype if isinstance(dtype, int) else _dtype_code(torch.empty(0, dtype=dtype))
    return int(lib().dd_beam_select_workspace_size(B, K, V, code))


def dd_beam_select(logits, score, parent, token, score_out, done=None, done_out=None, eos=-1,
                   workspace=None, stream=None):
    """One step of beam search: logits [B,K,V] (a view narrowed from a wider [B,K,ld] buffer is
    accepted), score, score_out [B,K] fp32, parent, token [B,K] int32, done, done_out [B,K]
    uint8. Outputs are other tensors than inputs."""
    gpu = _gpu(logits, "logits")
    if logits.dim() != 3:
        raise ValueError("logits must be [B, K, V]")
    B, K, V = logits.shape
    per_b, ld, unit = logits.stride()
    if K == 1:
        ld = per_b if B > 1 else -(-V // 8) * 8
    if (V > 1 and unit != 1) or (B > 1 and per_b != K * ld):
        raise ValueError("logits must be [B,K,V] with unit vocabulary stride and packed rows")
    i32, f32, bk = torch.int32, torch.float32, (B, K)
    sp = _arg(score, "score", f32, bk, gpu)
    so = _arg(score_out, "score_out", f32, bk, gpu)
    pp = _arg(parent, "parent", i32, bk, gpu)
    tp = _arg(token, "token", i32, bk, gpu)
    dp = None if done is None else _arg(done, "done", torch.uint8, bk, gpu)
    do = None if done_out is None else _arg(done_out, "done_out", torch.uint8, bk, gpu)
    code = _dtype_code(logits)
    if workspace is None:
        workspace = _scratch(lib().dd_beam_select_workspace_size(B, K, V, code), gpu, stream)
    wp, wb = _workspace(workspace, gpu)
    _call("dd_beam_select", gpu, stream, logits.data_ptr(), code, B, K, V, ld, sp, dp, int(eos), pp, tp, so,
          do, wp, wb)


def dd_beam_reorder(parent, states, stream=None):
    """States follow their parents: parent [B,K] int32; states: up to 8 pairs (src, dst) of
    tensors [B*K, ...] or [B,K,...], contiguous, of the same shape and dtype."""
    gpu = _gpu(parent, "parent")
    if parent.dim() != 2:
        raise ValueError("parent must be [B, K]")
    B, K = parent.shape
    n = B * K
    rows = []
    for src, dst in states:
        shape = src.shape
        sp = _arg(src, "src", src.dtype, shape, gpu)
        dp = _arg(dst, "dst", src.dtype, shape, gpu)
        if len(shape) < 1 or shape[0] != n and (len(shape) < 2 or shape[0] != B or shape[1] != K):
            raise ValueError(f"a state must be [B*K, ...] or [B, K, ...], got {tuple(shape)}")
        size = src.nbytes
        if sp < dp + size and dp < sp + size:
            raise ValueError("src and dst of a state must not overlap")
        rows += (sp, dp, size // n if n else 0)
    _call("dd_beam_reorder", gpu, stream, _arg(parent, "parent", torch.int32, (B, K), gpu), B, K, rows)


def dd_paged_fork(cache: PagedCache, parent, lengths, fresh, table_out, lengths_out, stream=None):
    """The beams' caches follow their parents: parent [B,K] int32; lengths, fresh, lengths_out
    [B*K] int32; table_out [B*K, max_pages] int32. Full pages are shared; page fresh[n], with
    the filled rows of a partly filled last page, is where beam n goes on. Outputs are other
    tensors than inputs."""
    gpu = _gpu(parent, "parent")
    if parent.dim() != 2:
        raise ValueError("parent must be [B, K]")
    B, K = parent.shape
    n = B * K
    cache._fits(n, gpu)
    cache._written()
    i32 = torch.int32
    pp = _arg(parent, "parent", i32, (B, K), gpu)
    lp = _arg(lengths, "lengths", i32, (n,), gpu)
    fp = _arg(fresh, "fresh", i32, (n,), gpu)
    lo = _arg(lengths_out, "lengths_out", i32, (n,), gpu)
    to, ts = _rows(table_out, "table_out", i32, (n, cache.max_pages), gpu)
    _call("dd_paged_fork", gpu, stream, cache._ref, pp, B, K, lp, fp, to, ts if n > 1 else cache.max_pages, lo)


def dd_get_device_error(stream=None) -> int:
    """Synchronise the stream; return and clear the device error word."""
    return int(lib().dd_get_device_error(_stream(stream)))


def dd_set_spin_limit(limit: int) -> int:
    return int(lib().dd_set_spin_limit(int(limit)))


def dd_selftest_bounded_wait(spin_limit: int, stream=None):
    _check("dd_selftest_bounded_wait", lib().dd_selftest_bounded_wait(int(spin_limit),
                                                                      _stream(stream)))


def dd_selftest_gumbel_screen(g_req, stream=None):
    """The library's fp32 noise and screen j of every noise level (2^23 each), the
    screen limit of each requested level g_req (fp32 device tensor), and the
    constant above which the noise is skipped outright."""
    dev = g_req.device
    g = torch.empty(1 << 23, dtype=torch.float32, device=dev)
    j = torch.empty(1 << 23, dtype=torch.float32, device=dev)
    limit = torch.empty_like(g_req)
    gmax = ctypes.c_float(0.0)
    _check("dd_selftest_gumbel_screen", lib().dd_selftest_gumbel_screen(
        _ptr(g), _ptr(j), _ptr(g_req), _ptr(limit), g_req.numel(), ctypes.byref(gmax),
        _stream(stream)))
    return g, j, limit, float(gmax.value)


def dd_bounds_checked() -> bool:
    """True when the loaded library is the checked build."""
    return bool(lib().dd_bounds_checked())


def dd_selftest_bounds_check(n: int, index: int, stream=None) -> int:
    """One checked read of element `index` of a 64-int library array (element i
    holds 3*i + 1) limited to its first n: the value, or -1 when the check skipped
    the read (dd_get_device_error then returns DD_ERR_BOUNDS)."""
    v = ctypes.c_int(0)
    _check("dd_selftest_bounds_check",
           lib().dd_selftest_bounds_check(int(n), int(index), ctypes.byref(v), _stream(stream)))
    return int(v.value)
