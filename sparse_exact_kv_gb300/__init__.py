"""Python binding of liblola.so, the GB300 LoLA hybrid-attention library.

Argument marshalling only: every step of the method runs in the library's CUDA kernels.
The functions carry the C ABI's names (include/lola.h) and take torch tensors for the
device buffers; torch provides device memory and streams, nothing else.

If the shared library is missing or fails to load, importing this package raises: there
is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.machinery
import importlib.util
import os
import warnings

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblola.so")

LOLA_OK = 0
LOLA_ERR_INVALID_ARG = -1
LOLA_ERR_UNSUPPORTED = -2
LOLA_ERR_WORKSPACE = -3
LOLA_ERR_CUDA = -4
LOLA_ERR_DEVICE = -5
LOLA_F32 = 0
LOLA_BF16 = 1
LOLA_READ_HIDE_STATE = 1
LOLA_READ_HIDE_CACHE = 2
LOLA_ALLOC_TOKEN = 0
LOLA_ALLOC_CHUNK = 1
LOLA_SCORE_SRE = 0
LOLA_SCORE_KERNEL_SQ = 1
LOLA_SCORE_KERNEL_ABS = 2
LOLA_SCORE_KERNEL_RATIO = 3
LOLA_SCORE_ATTENTION = 4
LOLA_PAIRS_HALVES = 0
LOLA_PAIRS_NEIGHBOURS = 1
PAIRS = {"halves": 0, "neighbours": 1}
LOLA_ATTN_BAD_OFFSETS = 1
LOLA_ATTN_BAD_PAGE = 2
LOLA_ATTN_TIMEOUT = 4
SCORES = {"sre": 0, "kernel_sq": 1, "kernel_abs": 2, "kernel_ratio": 3, "attention": 4}

# every symbol include/lola.h declares
EXPORTS = ("lola_version", "lola_status_string", "lola_last_cuda_error", "lola_check_config",
           "lola_state_layout_of", "lola_state_bytes", "lola_prefill_workspace_bytes", "lola_state_init",
           "lola_prefill", "lola_decode_step", "lola_read_status", "lola_kernel_timing", "lola_kernel_time",
           "lola_kernel_name", "lola_prefill_noalloc", "lola_selftest_bounded_wait", "lola_sre_map",
           "lola_sre_map_relative", "lola_hola_workspace_bytes", "lola_hola_prefill", "lola_hola_status",
           "lola_attn_prefill", "lola_paged_slot", "lola_paged_append", "lola_paged_prefill",
           "lola_paged_decode_workspace_bytes",
           "lola_paged_decode", "lola_attn_status", "lola_selftest_attn_wait")
# size of the fixed scratch array behind lola_prefill_noalloc (include/lola.h)
LOLA_NOALLOC_SCRATCH_BYTES = 32 << 20
KERNELS = ("state_init", "phi", "select", "output", "decode", "phi_q", "hola_prep", "hola_state", "hola_cache",
           "hola_read", "attn", "append", "paged")


class lola_config(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hh", ctypes.c_int32), ("d_k", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("D", ctypes.c_int32), ("eta", ctypes.c_int32),
                ("lambda_", ctypes.c_int32), ("chunk", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("read_mask", ctypes.c_int32), ("alloc", ctypes.c_int32), ("score", ctypes.c_int32)]


class lola_hola_config(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hh", ctypes.c_int32), ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("w", ctypes.c_int32), ("chunk", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class lola_attn_config(ctypes.Structure):
    _fields_ = [("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class lola_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row", ctypes.c_int64), ("head", ctypes.c_int64)]


class lola_paged_kv(ctypes.Structure):
    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("n_pages", ctypes.c_int32), ("page", ctypes.c_int32),
                ("n_seq", ctypes.c_int32), ("width", ctypes.c_int32), ("table_stride", ctypes.c_int64),
                ("table", ctypes.c_void_p), ("kv_len", ctypes.c_void_p)]


class lola_state_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("head_bytes", "H", "s", "win_pos", "win_k", "win_v", "win_phi", "c_pos", "c_k", "c_v", "c_phi",
                 "c_N", "c_z", "ev", "tok_phi")]


class LolaError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = _lib.lola_status_string(status).decode()
        if status == LOLA_ERR_CUDA:
            msg += ": " + _lib.lola_last_cuda_error().decode()
        super().__init__(f"{where}: {msg} ({status})")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                          "(or python -m sparse_exact_kv_gb300._build)")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    C = ctypes.POINTER(lola_config)
    HC = ctypes.POINTER(lola_hola_config)
    AC = ctypes.POINTER(lola_attn_config)
    PK = ctypes.POINTER(lola_paged_kv)
    R = ctypes.POINTER(lola_rows)
    sig = {
        "lola_version": ([], ctypes.c_int32),
        "lola_status_string": ([ctypes.c_int32], ctypes.c_char_p),
        "lola_last_cuda_error": ([], ctypes.c_char_p),
        "lola_check_config": ([C], ctypes.c_int32),
        "lola_state_layout_of": ([C, ctypes.POINTER(lola_state_layout)], ctypes.c_int32),
        "lola_state_bytes": ([C], ctypes.c_size_t),
        "lola_prefill_workspace_bytes": ([C, ctypes.c_int32], ctypes.c_size_t),
        "lola_state_init": ([C, P, P], ctypes.c_int32),
        "lola_prefill": ([C, ctypes.c_int32, P, P, P, P, ctypes.c_int64, P, P, P, P, ctypes.c_size_t, P],
                         ctypes.c_int32),
        "lola_decode_step": ([C, P, P, ctypes.c_int64, P, P, P, P, P, P], ctypes.c_int32),
        "lola_read_status": ([C, P, P, P], ctypes.c_int32),
        "lola_kernel_timing": ([ctypes.c_int32], ctypes.c_int32),
        "lola_kernel_time": ([ctypes.c_int32, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)],
                             ctypes.c_int32),
        "lola_kernel_name": ([ctypes.c_int32], ctypes.c_char_p),
        "lola_prefill_noalloc": ([C, ctypes.c_int32, P, P, P, P, ctypes.c_int64, P, P, P, P], ctypes.c_int32),
        "lola_selftest_bounded_wait": ([ctypes.c_int64, ctypes.POINTER(ctypes.c_int64), P], ctypes.c_int32),
        "lola_sre_map": ([C, ctypes.c_int32, P, P, ctypes.c_size_t, P, P], ctypes.c_int32),
        "lola_sre_map_relative": ([C, ctypes.c_int32, P, P, ctypes.c_size_t, P, P, P], ctypes.c_int32),
        "lola_hola_workspace_bytes": ([HC, ctypes.c_int32], ctypes.c_int64),
        "lola_hola_prefill": ([HC, ctypes.c_int32] + [P] * 14 + [ctypes.c_size_t, P], ctypes.c_int32),
        "lola_hola_status": ([HC, ctypes.c_int32, P, P, P], ctypes.c_int32),
        "lola_attn_prefill": ([AC] + [ctypes.c_int32] * 3 + [P, P, R, R, R, R, P, P], ctypes.c_int32),
        "lola_paged_slot": ([AC, PK, ctypes.c_int32, ctypes.c_int32, ctypes.c_int64], ctypes.c_int64),
        "lola_paged_prefill": ([AC, PK, ctypes.c_int32, ctypes.c_int32, P, R, R, P, P], ctypes.c_int32),
        "lola_paged_append": ([AC, PK, ctypes.c_int32, P, R, R, R, R, P, ctypes.c_int32, ctypes.c_int32, P, P],
                              ctypes.c_int32),
        "lola_paged_decode_workspace_bytes": ([AC], ctypes.c_int64),
        "lola_paged_decode": ([AC, PK, R, R, P, P, ctypes.c_size_t, P], ctypes.c_int32),
        "lola_selftest_attn_wait": ([ctypes.c_int32], ctypes.c_int32),
        "lola_attn_status": ([ctypes.POINTER(ctypes.c_int32), P], ctypes.c_int32),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    return lib


_lib = _load()


class _Declines:
    """In the marshalling module's place: every call takes its Python form."""
    prefill = prefill_paged = decode = append = staticmethod(lambda *args: NotImplemented)


def _marshalling(path):
    """The marshalling module of that file, which links liblola.so and torch; _Declines if it is not there or does
    not load (another torch than the one it was compiled against: nothing but speed depends on it)."""
    try:
        loader = importlib.machinery.ExtensionFileLoader("_lola_py", path)
        return importlib.util.module_from_spec(importlib.util.spec_from_file_location("_lola_py", path, loader=loader))
    except (ImportError, OSError):
        return _Declines


_PYMOD = os.path.join(os.path.dirname(os.path.abspath(__file__)), f"_lola_py-{torch.__version__}.so")
_fast = _marshalling(_PYMOD)


def make_config(B, Hh, d_k, d_v, D, eta, lam, chunk, dtype, read_mask=0, alloc=LOLA_ALLOC_TOKEN,
                score=LOLA_SCORE_SRE) -> lola_config:
    """``read_mask``: LOLA_READ_HIDE_STATE | LOLA_READ_HIDE_CACHE, memories left out of every
    query's read (the memory and the decisions are unchanged).  ``alloc``: LOLA_ALLOC_TOKEN
    (the per-token rule) or LOLA_ALLOC_CHUNK (chunk-granular allocation).  ``score``:
    LOLA_SCORE_SRE (the self-recall error) or one of the query-dependent scores of the scoring
    ablation (a LOLA_SCORE_* value or its name in SCORES)."""
    dt = dtype if isinstance(dtype, int) else {"f32": LOLA_F32, "bf16": LOLA_BF16,
                                               torch.float32: LOLA_F32, torch.bfloat16: LOLA_BF16}[dtype]
    sc = SCORES[score] if isinstance(score, str) else int(score)
    return lola_config(B, Hh, d_k, d_v, D, eta, lam, chunk, dt, read_mask, alloc, sc)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if isinstance(stream, int):          # a raw cudaStream_t (0: the legacy default stream)
        return ctypes.c_void_p(stream)
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status, where):
    if status != LOLA_OK:
        raise LolaError(status, where)


def lola_version() -> int:
    return _lib.lola_version()


def lola_status_string(status: int) -> str:
    return _lib.lola_status_string(status).decode()


def lola_check_config(cfg: lola_config) -> int:
    return _lib.lola_check_config(ctypes.byref(cfg))


def lola_state_layout_of(cfg: lola_config) -> lola_state_layout:
    out = lola_state_layout()
    _check(_lib.lola_state_layout_of(ctypes.byref(cfg), ctypes.byref(out)), "lola_state_layout_of")
    return out


def lola_state_bytes(cfg: lola_config) -> int:
    return _lib.lola_state_bytes(ctypes.byref(cfg))


def lola_prefill_workspace_bytes(cfg: lola_config, n: int) -> int:
    return _lib.lola_prefill_workspace_bytes(ctypes.byref(cfg), n)


def lola_state_init(cfg: lola_config, state: torch.Tensor, stream=None) -> None:
    _check(_lib.lola_state_init(ctypes.byref(cfg), _ptr(state), _stream(stream)), "lola_state_init")


def lola_prefill(cfg: lola_config, n: int, Q, K, V, W, w_head_stride: int, Y, state, write_pos, workspace,
                 stream=None) -> None:
    """Enqueue lola_prefill on ``stream`` (default: torch's current stream)."""
    _check(_lib.lola_prefill(ctypes.byref(cfg), n, _ptr(Q), _ptr(K), _ptr(V), _ptr(W), w_head_stride, _ptr(Y),
                             _ptr(state), _ptr(write_pos), _ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream(stream)), "lola_prefill")


def lola_prefill_noalloc(cfg: lola_config, n: int, Q, K, V, W, w_head_stride: int, Y, state, write_pos=None,
                         stream=None) -> None:
    """lola_prefill without a workspace: its scratch is the library's fixed device array
    (LOLA_NOALLOC_SCRATCH_BYTES), for callers that cannot allocate device memory."""
    _check(_lib.lola_prefill_noalloc(ctypes.byref(cfg), n, _ptr(Q), _ptr(K), _ptr(V), _ptr(W), w_head_stride,
                                     _ptr(Y), _ptr(state), _ptr(write_pos), _stream(stream)),
           "lola_prefill_noalloc")


def lola_decode_step(cfg: lola_config, state, W, w_head_stride: int, q, k, v, y, written_pos=None,
                     stream=None) -> None:
    _check(_lib.lola_decode_step(ctypes.byref(cfg), _ptr(state), _ptr(W), w_head_stride, _ptr(q), _ptr(k),
                                 _ptr(v), _ptr(y), _ptr(written_pos), _stream(stream)), "lola_decode_step")


def lola_read_status(cfg: lola_config, state, stream=None):
    """Synchronises the stream and returns (status, per-head status words as a list)."""
    BH = cfg.B * cfg.Hh
    buf = (ctypes.c_int32 * BH)()
    st = _lib.lola_read_status(ctypes.byref(cfg), _ptr(state), buf, _stream(stream))
    return st, list(buf)


def lola_kernel_timing(enable: bool) -> None:
    _check(_lib.lola_kernel_timing(1 if enable else 0), "lola_kernel_timing")


def lola_kernel_time(kernel) -> tuple[float, int]:
    """(total device ms, launches) of a kernel id or name since timing was enabled."""
    kid = KERNELS.index(kernel) if isinstance(kernel, str) else int(kernel)
    ms, cnt = ctypes.c_double(), ctypes.c_int64()
    _check(_lib.lola_kernel_time(kid, ctypes.byref(ms), ctypes.byref(cnt)), "lola_kernel_time")
    return ms.value, cnt.value


def lola_kernel_name(kid: int) -> str:
    return _lib.lola_kernel_name(kid).decode()


def lola_sre_map(cfg: lola_config, n: int, V, workspace, out, stream=None) -> None:
    """SRE of every key held by each snapshot of the last prefill in ``workspace`` (section
    4.4): ``out`` float32 [B, Hh, nck, n]."""
    _check(_lib.lola_sre_map(ctypes.byref(cfg), n, _ptr(V), _ptr(workspace), workspace.numel() * workspace.element_size(),
                             _ptr(out), _stream(stream)), "lola_sre_map")


def lola_sre_map_relative(cfg: lola_config, n: int, V, workspace, out, base, stream=None) -> None:
    """The relative SRE map (appendix G, Eq. 26): ``out`` float32 [B, Hh, nck, n] = the map
    minus each held key's SRE at first write, ``base`` float32 [B, Hh, n] = that SRE."""
    _check(_lib.lola_sre_map_relative(ctypes.byref(cfg), n, _ptr(V), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _ptr(out), _ptr(base),
                                      _stream(stream)), "lola_sre_map_relative")


def lola_selftest_bounded_wait(limit_ns: int, stream=None):
    """Runs the kernels' bounded mbarrier wait on a barrier nothing completes; returns
    (status, nanoseconds waited): LOLA_ERR_DEVICE when the wait gave up as designed."""
    ns = ctypes.c_int64(0)
    st = _lib.lola_selftest_bounded_wait(int(limit_ns), ctypes.byref(ns), _stream(stream))
    return st, ns.value


# ---------------------------------------------------------------------------------------
# The write-magnitude exact cache on a gated delta-rule state (include/lola.h)
# ---------------------------------------------------------------------------------------

def make_hola_config(B, Hh, d, w, chunk, dtype=LOLA_BF16) -> lola_hola_config:
    return lola_hola_config(B, Hh, d, d, w, chunk, dtype)


def lola_hola_workspace_bytes(cfg: lola_hola_config, n: int) -> int:
    b = _lib.lola_hola_workspace_bytes(ctypes.byref(cfg), n)
    if b < 0:
        raise LolaError(int(b), "lola_hola_workspace_bytes")
    return int(b)


def lola_hola_prefill(cfg: lola_hola_config, n: int, Q, K, V, alpha, beta, gamma_q, gamma_k, sink, gate, Y,
                      workspace, S_out=None, scores=None, cache=None, stream=None) -> None:
    _check(_lib.lola_hola_prefill(ctypes.byref(cfg), n, _ptr(Q), _ptr(K), _ptr(V), _ptr(alpha), _ptr(beta),
                                  _ptr(gamma_q), _ptr(gamma_k), _ptr(sink), _ptr(gate), _ptr(Y), _ptr(S_out),
                                  _ptr(scores), _ptr(cache), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream)),
           "lola_hola_prefill")


def lola_hola_status(cfg: lola_hola_config, n: int, workspace, stream=None):
    """Synchronises the stream and returns (status, per-head status words as a list)."""
    buf = (ctypes.c_int32 * (cfg.B * cfg.Hh))()
    st = _lib.lola_hola_status(ctypes.byref(cfg), n, _ptr(workspace), buf, _stream(stream))
    return st, list(buf)


# ---------------------------------------------------------------------------------------
# Exact softmax attention: packed prompts and a paged key-value cache (include/lola.h)
# ---------------------------------------------------------------------------------------

def make_attn_config(Hq, Hkv, d, dtype, scale=None) -> lola_attn_config:
    """``scale``: the logit scale, None for 1 / sqrt(d)."""
    if scale is not None and ctypes.c_float(scale).value == 0:
        raise ValueError("scale: want a positive number, or None for 1 / sqrt(d)")      # (0 is None's form in C)
    dt = dtype if isinstance(dtype, int) else {"f32": LOLA_F32, "bf16": LOLA_BF16,
                                               torch.float32: LOLA_F32, torch.bfloat16: LOLA_BF16}[dtype]
    return lola_attn_config(Hq, Hkv, d, dt, 0.0 if scale is None else scale)


def _rows(t):
    """lola_rows of a [rows, heads, d] tensor (a size-1 axis' stride is made a packed one)."""
    if t is None:
        return None
    n, h, d = t.shape
    row, head, one = t.stride()
    if one != 1:
        raise ValueError("the head width must be the contiguous axis")
    if h == 1:
        head = d
    if n == 1:
        row = h * head
    return lola_rows(t.data_ptr(), row, head)


def _addr(t):
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _index_of(dev):
    """The index of ``dev``, which has to be the current CUDA device."""
    i = dev.index
    if i is None or dev.type != "cuda" or i != torch._C._cuda_getDevice():
        raise ValueError(f"tensors are on {dev}, not on the current CUDA device")
    return i


def _stream_of(stream, index):
    """The cudaStream_t of ``stream``; None: torch's current stream of device ``index`` (looked up
    without making a Stream object, 3 us a call)."""
    if stream is None:
        return _raw_stream(index) if _raw_stream else torch.cuda.current_stream(index).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _table_stride(table):
    """The rows' stride (one row's is any; rows that overlap, as an expanded table's do, are refused by
    the library)."""
    n, width = table.shape
    return width if n == 1 else table.stride(0)


def _paged(k_pool, v_pool, kv_len, table):
    pages, _, page, _ = k_pool.shape
    n, width = table.shape
    return lola_paged_kv(k_pool.data_ptr(), v_pool.data_ptr(), pages, page, n, width, _table_stride(table),
                         table.data_ptr(), kv_len.data_ptr())


def lola_attn_prefill(cfg: lola_attn_config, Q, K, V, O, cu_q, cu_k=None, lse=None, stream=None) -> None:
    """Q, O: [total_q, Hq, d]; K, V: [total_k, Hkv, d]; cu_q, cu_k: int32 [n_seq + 1] on the device."""
    st = _lib.lola_attn_prefill(cfg, cu_q.shape[0] - 1, Q.shape[0], K.shape[0], cu_q.data_ptr(), _addr(cu_k), _rows(Q),
                                _rows(K), _rows(V), _rows(O), _addr(lse), _stream_of(stream, Q.get_device()))
    if st:
        raise LolaError(st, "lola_attn_prefill")


def lola_paged_slot(cfg: lola_attn_config, kv: lola_paged_kv, seq: int, head: int, pos: int) -> int:
    """Element offset of a token's row in the pools, or -1 (``kv`` with host pointers)."""
    return _lib.lola_paged_slot(ctypes.byref(cfg), ctypes.byref(kv), seq, head, pos)


def lola_paged_append(cfg: lola_attn_config, kv: lola_paged_kv, K, V, cu_new=None, Q=None, QO=None, inv_freq=None,
                      pairs=LOLA_PAIRS_HALVES, positions=None, stream=None) -> None:
    """K, V: [n, Hkv, d]; Q, QO: [n, Hq, d]; inv_freq: float32 [rot / 2]."""
    rot = 0 if inv_freq is None else 2 * inv_freq.shape[0]
    st = _lib.lola_paged_append(cfg, kv, K.shape[0], _addr(cu_new), _rows(K), _rows(V), _rows(Q), _rows(QO),
                                _addr(inv_freq), rot, pairs, _addr(positions), _stream_of(stream, K.get_device()))
    if st:
        raise LolaError(st, "lola_paged_append")


def lola_paged_prefill(cfg: lola_attn_config, kv: lola_paged_kv, Q, O, cu_q, total_k=0, lse=None, stream=None) -> None:
    """Q, O: [total_q, Hq, d]; cu_q: int32 [n_seq + 1]; total_k: the tokens of all sequences, if known."""
    st = _lib.lola_paged_prefill(cfg, kv, Q.shape[0], total_k, cu_q.data_ptr(), _rows(Q), _rows(O), _addr(lse),
                                 _stream_of(stream, Q.get_device()))
    if st:
        raise LolaError(st, "lola_paged_prefill")


def lola_paged_decode_workspace_bytes(cfg: lola_attn_config) -> int:
    b = _lib.lola_paged_decode_workspace_bytes(ctypes.byref(cfg))
    if b < 0:
        raise LolaError(int(b), "lola_paged_decode_workspace_bytes")
    return int(b)


def lola_paged_decode(cfg: lola_attn_config, kv: lola_paged_kv, Q, O, workspace, lse=None, stream=None) -> None:
    """Q, O: [n_seq, Hq, d]; lse: float32 [n_seq, Hq]."""
    st = _lib.lola_paged_decode(cfg, kv, _rows(Q), _rows(O), _addr(lse), workspace.data_ptr(), workspace.nbytes,
                                _stream_of(stream, Q.get_device()))
    if st:
        raise LolaError(st, "lola_paged_decode")


def lola_selftest_attn_wait(block: int) -> None:
    """The block of keys at which every third CTA of the exact-attention kernels gives up; -1: none."""
    _check(_lib.lola_selftest_attn_wait(int(block)), "lola_selftest_attn_wait")


def lola_attn_status(stream=None):
    """Synchronises the stream; (status, LOLA_ATTN_* bits of the device since the last call)."""
    bits = ctypes.c_int32(0)
    st = _lib.lola_attn_status(ctypes.byref(bits), _stream(stream))
    return st, bits.value


# ---------------------------------------------------------------------------------------
# Convenience: buffers allocated through torch, then the C ABI
# ---------------------------------------------------------------------------------------

@functools.lru_cache(maxsize=256)
def _attn_plan(Hq, Hkv, d, dtype, scale):
    """The config of a kind of layer, the decode step's workspace bytes (checks the config), and both as the
    marshalling module takes them (the config by its address: a layer holds on to it)."""
    cfg = make_attn_config(Hq, Hkv, d, dtype, scale)
    size = lola_paged_decode_workspace_bytes(cfg)
    return cfg, size, (ctypes.addressof(cfg), size)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


class ExactAttention:
    """One layer's exact softmax attention: packed prompts, and single tokens over a paged cache.

    ``k_pool``, ``v_pool``: [n_pages, Hkv, page, d] (``allocate`` makes them); a layer that only
    runs ``prefill`` needs none.  Outputs and the decode step's workspace are allocated through
    torch on the call's stream, so calls on several streams do not share any.  Shapes, types and
    devices are checked here, strides and alignment by the library; all tensors are on the current
    CUDA device.  A batch of no sequences is refused.  For serving: outputs carry no gradient, also
    of inputs that require one."""

    __slots__ = ("cfg", "Hq", "Hkv", "d", "dtype", "k_pool", "v_pool", "_ws", "_plan")

    def __init__(self, Hq, Hkv, d, dtype=torch.bfloat16, k_pool=None, v_pool=None, scale=None):
        if _fast is _Declines:
            warnings.warn(f"{os.path.basename(_PYMOD)}, the marshalling module of ExactAttention for this torch, is missing or does "
                          "not load: calls take their slower Python form (rebuild the package)", RuntimeWarning, stacklevel=2)
        self.cfg, self._ws, self._plan = _attn_plan(Hq, Hkv, d, dtype, scale)
        self.Hq, self.Hkv, self.d, self.dtype = Hq, Hkv, d, dtype
        self.k_pool, self.v_pool = k_pool, v_pool
        if k_pool is not None or v_pool is not None:
            self._check_pools()

    def _check_pools(self):
        k, v = self.k_pool, self.v_pool
        _need(k is not None and v is not None, "k_pool and v_pool come together")
        shape = k.shape
        _need(len(shape) == 4 and shape[1] == self.Hkv and shape[3] == self.d and k.dtype == self.dtype and k.is_contiguous(),
              "pools are contiguous [n_pages, Hkv, page, d] of the layer's dtype")
        _need(v.shape == shape and v.dtype == self.dtype and v.is_contiguous() and v.device == k.device,
              "k_pool and v_pool differ in shape, type or device")

    def __reduce__(self):
        # (``_plan`` is the address of this object's ``cfg``: a copy, or another process' object, is made anew)
        return type(self), (self.Hq, self.Hkv, self.d, self.dtype, self.k_pool, self.v_pool, self.cfg.scale or None)

    @classmethod
    def allocate(cls, Hq, Hkv, d, n_pages, page=64, dtype=torch.bfloat16, device="cuda", scale=None):
        pool = lambda: torch.zeros(n_pages, Hkv, page, d, dtype=dtype, device=device)  # noqa: E731
        return cls(Hq, Hkv, d, dtype, pool(), pool(), scale)

    def _heads(self, t, heads, n, dev, what):
        """lola_rows of t, which has to be [n, heads, d] of the layer's type on ``dev``."""
        if t.shape != (n, heads, self.d) or t.dtype != self.dtype or t.device != dev:
            raise ValueError(f"{what}: want [{n}, {heads}, {self.d}] {self.dtype} on {dev}")
        row, head, one = t.stride()
        if one != 1 or n < 2 or heads < 2:
            return _rows(t)
        return lola_rows(t.data_ptr(), row, head)

    @staticmethod
    def _vector(t, n, dev, what, dtype=torch.int32):
        if t.shape != (n,) or t.dtype != dtype or t.device != dev or not t.is_contiguous():
            raise ValueError(f"{what}: want a contiguous {dtype} [{n}] on {dev}")

    @staticmethod
    def _lse(t, shape, dev):
        if not (t.shape == shape and t.dtype == torch.float32 and t.device == dev and t.is_contiguous()):
            raise ValueError(f"lse: want a contiguous float32 {list(shape)} on {dev}")

    @staticmethod
    def _empty(shape, dtype, dev, stream):
        """torch.empty on the call's stream, so that torch reuses the memory in its order."""
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=dev)
        with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=dev) if isinstance(stream, int) else stream):
            return torch.empty(shape, dtype=dtype, device=dev)

    def _like(self, q, stream):
        """A fresh output of q's shape, and its lola_rows."""
        if stream is None:
            out = torch.empty_like(q)            # (a third of the time of torch.empty)
        else:
            out = self._empty(q.shape, q.dtype, q.device, stream)
        return out, _rows(out)

    def prefill(self, q, k, v, cu_q, cu_k=None, out=None, lse=None, stream=None):
        """Causal attention over packed prompts: q [total_q, Hq, d], k, v [total_k, Hkv, d] (any row
        and head strides), cu_q, cu_k int32 [n_seq + 1].  Returns out [total_q, Hq, d]; ``lse``
        float32 [Hq, total_q] receives the log normalisers.  A fresh ``out`` is not initialised
        outside the sequences."""
        if out is None and lse is None and stream is None:
            out = _fast.prefill(self._plan, q, k, v, cu_q, cu_k)
            if out is not NotImplemented:
                return out
            out = None
        dev, n, m, n1 = q.device, q.shape[0], k.shape[0], cu_q.shape[0]
        rq = self._heads(q, self.Hq, n, dev, "q")
        rk = self._heads(k, self.Hkv, m, dev, "k")
        rv = self._heads(v, self.Hkv, m, dev, "v")
        self._vector(cu_q, n1, dev, "cu_q")
        if cu_k is not None:
            self._vector(cu_k, n1, dev, "cu_k")
        if lse is not None:
            self._lse(lse, (self.Hq, n), dev)
        if out is not None:
            ro = self._heads(out, self.Hq, n, dev, "out")
        index = _index_of(dev)
        if out is None:
            out, ro = self._like(q, stream)
        st = _lib.lola_attn_prefill(self.cfg, n1 - 1, n, m, cu_q.data_ptr(), _addr(cu_k), rq, rk, rv, ro, _addr(lse),
                                    _stream_of(stream, index))
        if st:
            raise LolaError(st, "lola_attn_prefill")
        return out

    def _cache(self, kv_len, table):
        pool = self.k_pool
        if pool is None:
            raise ValueError("this layer has no key-value pools")
        self._check_pools()                        # (they may be others than the constructor saw)
        dev, (n, width), one = pool.device, table.shape, table.stride(1)
        self._vector(kv_len, n, dev, "kv_len")
        if table.dtype != torch.int32 or table.device != dev or (one != 1 and width != 1):
            raise ValueError(f"table: want int32 [{n}, width] on {dev}, rows contiguous")
        pages, _, page, _ = pool.shape
        return lola_paged_kv(pool.data_ptr(), self.v_pool.data_ptr(), pages, page, n, width,
                             _table_stride(table), table.data_ptr(), kv_len.data_ptr()), dev, n, _index_of(dev)

    def append(self, k, v, kv_len, table, cu_new=None, q=None, inv_freq=None, q_out=None, pairs="halves",
               positions=None, stream=None):
        """Appends k, v [n, Hkv, d] to the cache and returns the rotated q (None without q).

        ``kv_len`` int32 [n_seq] counts the new tokens in; ``table`` int32 [n_seq, width]; ``cu_new``
        int32 [n_seq + 1] the rows of each sequence's new tokens (None: one each); ``inv_freq``
        float32 [rot / 2] radians per position (None: no rotation); ``pairs`` the channel pairs of
        the rotation, "halves" or "neighbours"; ``positions`` int32 [n] in place of the tokens'
        indexes.  ``q_out`` may be q itself; rows outside the sequences, and of sequences without
        tokens, are left as they were in it (a fresh one is not initialised there)."""
        if q_out is None and positions is None and stream is None:
            r = _fast.append(self._plan, self.k_pool, self.v_pool, k, v, kv_len, table, cu_new, q, inv_freq, PAIRS[pairs])
            if r is not NotImplemented:
                return r
        kv, dev, n_seq, index = self._cache(kv_len, table)
        n = k.shape[0]
        rk = self._heads(k, self.Hkv, n, dev, "k")
        rv = self._heads(v, self.Hkv, n, dev, "v")
        rq = ro = freq = None
        rot = 0
        if cu_new is not None:
            self._vector(cu_new, n_seq + 1, dev, "cu_new")
        if inv_freq is not None:
            rot = 2 * inv_freq.shape[0]
            self._vector(inv_freq, rot // 2, dev, "inv_freq", torch.float32)
            freq = inv_freq.data_ptr()
        if positions is not None:
            self._vector(positions, n, dev, "positions")
        if q is not None:
            rq = self._heads(q, self.Hq, n, dev, "q")
            if q_out is not None:
                ro = self._heads(q_out, self.Hq, n, dev, "q_out")
            else:
                q_out, ro = self._like(q, stream)
        elif q_out is not None:
            raise ValueError("q_out without q")
        st = _lib.lola_paged_append(self.cfg, kv, n, _addr(cu_new), rk, rv, rq, ro, freq, rot, PAIRS[pairs],
                                    _addr(positions), _stream_of(stream, index))
        if st:
            raise LolaError(st, "lola_paged_append")
        return q_out

    def prefill_paged(self, q, cu_q, kv_len, table, total_k=0, out=None, lse=None, stream=None):
        """Causal attention of packed prompts, or later pieces of them, over the cache: q [total_q, Hq, d]
        with the rows cu_q int32 [n_seq + 1] of each sequence, whose kv_len tokens (the queries' own
        included, appended before) are read from their pages.  ``total_k``: the sum of kv_len where it
        is known (it only helps to choose the kernel's form).  Returns out [total_q, Hq, d]; ``lse`` as
        in ``prefill``."""
        if out is None and lse is None and stream is None:
            out = _fast.prefill_paged(self._plan, self.k_pool, self.v_pool, q, cu_q, kv_len, table, total_k)
            if out is not NotImplemented:
                return out
            out = None
        kv, dev, n_seq, index = self._cache(kv_len, table)
        n = q.shape[0]
        rq = self._heads(q, self.Hq, n, dev, "q")
        self._vector(cu_q, n_seq + 1, dev, "cu_q")
        if lse is not None:
            self._lse(lse, (self.Hq, n), dev)
        if out is not None:
            ro = self._heads(out, self.Hq, n, dev, "out")
        else:
            out, ro = self._like(q, stream)
        st = _lib.lola_paged_prefill(self.cfg, kv, n, total_k, cu_q.data_ptr(), rq, ro, _addr(lse), _stream_of(stream, index))
        if st:
            raise LolaError(st, "lola_paged_prefill")
        return out

    def decode_step(self, q, kv_len, table, out=None, lse=None, workspace=None, stream=None):
        """One query token per sequence, q [n_seq, Hq, d], over its kv_len cached tokens; returns out
        [n_seq, Hq, d].  ``lse`` float32 [n_seq, Hq].  ``workspace``: a buffer of
        lola_paged_decode_workspace_bytes; by default one is allocated for the call."""
        if out is None and lse is None and workspace is None and stream is None:
            out = _fast.decode(self._plan, self.k_pool, self.v_pool, q, kv_len, table)
            if out is not NotImplemented:
                return out
            out = None
        kv, dev, n, index = self._cache(kv_len, table)
        rq = self._heads(q, self.Hq, n, dev, "q")
        if lse is not None:
            self._lse(lse, (n, self.Hq), dev)
        if out is not None:
            ro = self._heads(out, self.Hq, n, dev, "out")
        else:
            out, ro = self._like(q, stream)
        size = self._ws
        if workspace is None:
            workspace = self._empty(size, torch.uint8, dev, stream)
        else:
            size = workspace.nbytes
            if workspace.device != dev or not workspace.is_contiguous():
                raise ValueError(f"workspace: want a contiguous buffer on {dev}")
        st = _lib.lola_paged_decode(self.cfg, kv, rq, ro, _addr(lse), workspace.data_ptr(), size,
                                    _stream_of(stream, index))
        if st:
            raise LolaError(st, "lola_paged_decode")
        return out


class Lola:
    """One layer's LoLA memory for B x Hh heads: owns the state and the prefill workspace."""

    def __init__(self, B, Hh, d, D, eta, lam, chunk=64, dtype=torch.bfloat16, device="cuda", read_mask=0,
                 alloc=LOLA_ALLOC_TOKEN, score=LOLA_SCORE_SRE):
        self.cfg = make_config(B, Hh, d, d, D, eta, lam, chunk, dtype, read_mask, alloc, score)
        _check(lola_check_config(self.cfg), "config")
        self.dtype = dtype
        self.device = torch.device(device)
        self.state = torch.empty(lola_state_bytes(self.cfg), dtype=torch.uint8, device=self.device)
        self.workspace = None
        lola_state_init(self.cfg, self.state)

    def layout(self) -> lola_state_layout:
        return lola_state_layout_of(self.cfg)

    def workspace_for(self, n: int) -> torch.Tensor:
        need = lola_prefill_workspace_bytes(self.cfg, n)
        if self.workspace is None or self.workspace.numel() < need:
            self.workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
        return self.workspace

    def prefill(self, Q, K, V, W, Y=None, write_pos=None, stream=None):
        """Q, K, V: [B, Hh, n, d] device tensors of the config's dtype; W: [D/2, d] float32."""
        n = Q.shape[2]
        if Y is None:
            Y = torch.empty_like(V)
        ws = self.workspace_for(n)
        lola_prefill(self.cfg, n, Q, K, V, W, 0, Y, self.state, write_pos, ws, stream)
        return Y

    def decode_step(self, q, k, v, W, y=None, written_pos=None, stream=None):
        """q, k, v: [B, Hh, d] device tensors; returns y [B, Hh, d]."""
        if y is None:
            y = torch.empty_like(v)
        lola_decode_step(self.cfg, self.state, W, 0, q, k, v, y, written_pos, stream)
        return y

    def read_state(self):
        """Host copies of every head's memory: dict of numpy arrays (H, s, window, cache)."""
        import numpy as np
        L = self.layout()
        c = self.cfg
        raw = self.state.view(c.B * c.Hh, L.head_bytes).cpu().numpy()
        io = np.uint16 if c.dtype == LOLA_BF16 else np.float32
        isz = 2 if c.dtype == LOLA_BF16 else 4

        def f(off, count, dt, size):
            return np.ascontiguousarray(raw[:, off: off + count * size]).view(dt)

        BH = c.B * c.Hh
        hdr = f(0, 16, np.int32, 4)
        return dict(t=hdr[:, 0], n_cache=hdr[:, 1], n_written=hdr[:, 2], status=hdr[:, 3],
                    H=f(L.H, c.D * c.d_v, np.float32, 4).reshape(BH, c.D, c.d_v),
                    s=f(L.s, c.D, np.float32, 4),
                    win_pos=f(L.win_pos, c.eta, np.int32, 4),
                    win_k=f(L.win_k, c.eta * c.d_k, io, isz).reshape(BH, c.eta, c.d_k),
                    win_v=f(L.win_v, c.eta * c.d_v, io, isz).reshape(BH, c.eta, c.d_v),
                    win_phi=f(L.win_phi, c.eta * c.D, np.float32, 4).reshape(BH, c.eta, c.D),
                    c_pos=f(L.c_pos, c.lambda_, np.int32, 4),
                    c_k=f(L.c_k, c.lambda_ * c.d_k, io, isz).reshape(BH, c.lambda_, c.d_k),
                    c_v=f(L.c_v, c.lambda_ * c.d_v, io, isz).reshape(BH, c.lambda_, c.d_v),
                    c_phi=f(L.c_phi, c.lambda_ * c.D, np.float32, 4).reshape(BH, c.lambda_, c.D),
                    c_N=f(L.c_N, c.lambda_ * c.d_v, np.float32, 4).reshape(BH, c.lambda_, c.d_v),
                    c_z=f(L.c_z, c.lambda_, np.float32, 4),
                    ev=f(L.ev, c.d_v + 1, np.float32, 4))
