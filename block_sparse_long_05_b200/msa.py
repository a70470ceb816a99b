"""Python binding of libmsa (the C ABI in include/msa.h), by ctypes; the paged-cache
calls, which are short, through a compiled module (csrc_torch/binding.cpp).

Argument marshalling only: every step of the MSA hot path runs in the CUDA
kernels behind the C ABI.  torch supplies device memory and the current CUDA
stream.  If libmsa.so is missing, every call raises: there is no CPU path.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmsa.so")

STATUS = {
    0: "MSA_OK",
    1: "MSA_ERR_INVALID_ARG",
    2: "MSA_ERR_UNSUPPORTED",
    3: "MSA_ERR_WORKSPACE",
    4: "MSA_ERR_CUDA",
    5: "MSA_ERR_TIMEOUT",
    6: "MSA_ERR_BAD_IDS",
}

EXPORTED = ("msa_workspace_size", "msa_index_topk", "msa_select_invert", "msa_sparse_attn",
            "msa_index_topk_ev", "msa_sparse_attn_ev", "msa_device_status", "msa_status_string",
            "msa_selftest_umma", "msa_sparse_attn_decode_noalloc", "msa_index_topk_paged",
            "msa_sparse_attn_paged", "msa_index_topk_i8", "msa_index_topk_i8_ev",
            "msa_workspace_size_kv_group", "msa_cache_workspace_size", "msa_kv_append",
            "msa_kv_append_i8", "msa_kv_gather", "msa_kv_gather_i8", "msa_attn_paged",
            "msa_attn_paged_i8", "msa_sparse_attn_paged_i8", "msa_attn_paged_kernels")

MAX_STAGES = 4


class StageEvents(ctypes.Structure):
    """msa_stage_events: cudaEvent_t handles recorded around each stage."""
    _fields_ = [("start", ctypes.c_void_p * MAX_STAGES), ("stop", ctypes.c_void_p * MAX_STAGES)]


def _event_handle(ev) -> int:
    """Raw cudaEvent_t of a torch.cuda.Event (created on first record)."""
    if ev.cuda_event == 0:
        ev.record()
    return ev.cuda_event


def _stage_events(events):
    """events: {stage: (start torch.cuda.Event, stop torch.cuda.Event)} or None."""
    if not events:
        return None
    se = StageEvents()
    for i, (a, b) in events.items():
        se.start[i] = _event_handle(a) if a is not None else None
        se.stop[i] = _event_handle(b) if b is not None else None
    return ctypes.byref(se)


class MSAError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} returned {STATUS.get(code, code)} ({code})")
        self.code = code


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libmsa.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m block_sparse_long_05_b200.build` (needs nvcc, sm_100a)")
    lib = ctypes.CDLL(path)
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.msa_workspace_size.argtypes = [I, I, I, I, I, I, I, I, I]
    lib.msa_workspace_size.restype = Z
    lib.msa_workspace_size_kv_group.argtypes = [I, I, I, I, I, I, I, I, I, I]
    lib.msa_workspace_size_kv_group.restype = Z
    lib.msa_index_topk.argtypes = [P, P, P, I, I, I, I, I, I, P, Z, P]
    lib.msa_index_topk.restype = I
    lib.msa_select_invert.argtypes = [P, P, P, I, I, I, I, I, P, Z, P]
    lib.msa_select_invert.restype = I
    lib.msa_sparse_attn.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, I, P, Z, P]
    lib.msa_sparse_attn.restype = I
    lib.msa_device_status.argtypes = [P, P]
    lib.msa_device_status.restype = I
    lib.msa_status_string.argtypes = [I]
    lib.msa_status_string.restype = ctypes.c_char_p
    lib.msa_index_topk_ev.argtypes = [P, P, P, I, I, I, I, I, I, P, Z, P, P]
    lib.msa_index_topk_ev.restype = I
    lib.msa_index_topk_i8.argtypes = [P, P, P, I, I, I, I, I, I, P, Z, P]
    lib.msa_index_topk_i8.restype = I
    lib.msa_index_topk_i8_ev.argtypes = [P, P, P, I, I, I, I, I, I, P, Z, P, P]
    lib.msa_index_topk_i8_ev.restype = I
    lib.msa_sparse_attn_ev.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, I, P, Z, P, P]
    lib.msa_sparse_attn_ev.restype = I
    lib.msa_sparse_attn_decode_noalloc.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, P, P]
    lib.msa_sparse_attn_decode_noalloc.restype = I
    lib.msa_index_topk_paged.argtypes = [P, P, P, I, I, P, I, I, I, I, I, P, Z, P]
    lib.msa_index_topk_paged.restype = I
    lib.msa_sparse_attn_paged.argtypes = [P, P, P, P, I, I, P, P, P, I, I, I, I, I, I, I, P, Z, P]
    lib.msa_sparse_attn_paged.restype = I
    L = ctypes.c_int64
    lib.msa_cache_workspace_size.argtypes = [I, I, I]
    lib.msa_cache_workspace_size.restype = Z
    step = [P, I, I, P, P]  # page_table, page_stride, num_pages, cu, kv_len
    lib.msa_kv_append.argtypes = [P, L, P, L, P, L, P, P, P, *step, I, I, I, I, I, I, P, Z, P]
    lib.msa_kv_append_i8.argtypes = [P, L, P, L, P, L, P, P, P, P, P, *step, I, I, I, I, I, I, P, Z,
                                     P]
    lib.msa_kv_gather.argtypes = [P, P, *step, P, P, I, I, I, I, I, P, Z, P]
    lib.msa_kv_gather_i8.argtypes = [P, P, P, P, *step, P, P, I, I, I, I, I, P, Z, P]
    lib.msa_attn_paged.argtypes = [P, L, P, P, *step, P, P, I, I, I, I, I, I, I, I, I, P, Z, P]
    lib.msa_attn_paged_i8.argtypes = [P, L, P, P, P, P, *step, P, P, I, I, I, I, I, I, I, I, I, P, Z,
                                      P]
    lib.msa_sparse_attn_paged_i8.argtypes = [P, P, P, P, P, P, I, I, P, P, P, I, I, I, I, I, I, I, P,
                                             Z, P]
    for f in ("kv_append", "kv_append_i8", "kv_gather", "kv_gather_i8", "attn_paged",
              "attn_paged_i8", "sparse_attn_paged_i8"):
        getattr(lib, "msa_" + f).restype = I
    lib.msa_attn_paged_kernels.argtypes = [I] * 9
    lib.msa_attn_paged_kernels.restype = I
    lib.msa_selftest_umma.argtypes = [P, P, P, I, I, I, P, P]
    lib.msa_selftest_umma.restype = I
    _lib = lib
    return lib


def _check(fn: str, code: int):
    if code != 0:
        raise MSAError(fn, code)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev(t: torch.Tensor, dtype, name: str) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def workspace_size(Bt, n_q, T, Hq, Hkv, d, d_idx, block, K, kv_group=None) -> int:
    """Workspace bytes: the minimum (msa_workspace_size), or with kv_group
    the size for prefill attention passes of kv_group kv heads each
    (kv_group = Hkv: one pass over all heads)."""
    lib = load_library()
    if kv_group is None:
        return int(lib.msa_workspace_size(Bt, n_q, T, Hq, Hkv, d, d_idx, block, K))
    return int(lib.msa_workspace_size_kv_group(Bt, n_q, T, Hq, Hkv, d, d_idx, block, K, kv_group))


HEADER_BYTES = 2304  # MSA_WORKSPACE_HEADER_BYTES


class Workspace:
    """Device scratch for the calls (its header zeroed at creation)."""

    def __init__(self, nbytes: int, device=None):
        if nbytes <= 0:
            raise ValueError("workspace size must be positive (unsupported shape?)")
        self.buf = torch.empty(nbytes + 256, dtype=torch.uint8, device=device or "cuda")
        off = (-self.buf.data_ptr()) % 256
        self.view = self.buf[off:off + nbytes]
        self.view[:HEADER_BYTES].zero_()
        self.nbytes = nbytes
        self.ptr = self.view.data_ptr()
        self.device_index = self.view.get_device()

    @classmethod
    def for_shape(cls, Bt, n_q, T, Hq, Hkv, d, d_idx, block, K, device=None,
                  kv_group=None) -> "Workspace":
        return cls(workspace_size(Bt, n_q, T, Hq, Hkv, d, d_idx, block, K, kv_group), device)

    @classmethod
    def for_cache(cls, Hq, Hkv, d, device=None) -> "Workspace":
        """Workspace of the paged-cache calls (kv_append .. sparse_attn_paged_i8)."""
        return cls(int(load_library().msa_cache_workspace_size(Hq, Hkv, d)), device)


def index_topk(q_idx: torch.Tensor, k_idx: torch.Tensor, block: int, K: int, ws: Workspace,
               ids: torch.Tensor | None = None, stream=None, events=None) -> torch.Tensor:
    """q_idx [Bt, n_q, d_idx], k_idx [Bt, T, d_idx] bf16 -> ids [Bt, n_q, K] int32.
    events: optional {stage: (start, stop)} torch.cuda.Event pairs (msa_index_topk_ev)."""
    _dev(q_idx, torch.bfloat16, "q_idx")
    _dev(k_idx, torch.bfloat16, "k_idx")
    Bt, n_q, d_idx = q_idx.shape
    T = k_idx.shape[1]
    if k_idx.shape != (Bt, T, d_idx):
        raise ValueError(f"k_idx shape {tuple(k_idx.shape)} does not match q_idx")
    if ids is None:
        ids = torch.empty((Bt, n_q, K), dtype=torch.int32, device=q_idx.device)
    _dev(ids, torch.int32, "ids")
    lib = load_library()
    _check("msa_index_topk", lib.msa_index_topk_ev(q_idx.data_ptr(), k_idx.data_ptr(),
                                                   ids.data_ptr(), Bt, n_q, T, d_idx, block, K,
                                                   ws.ptr, ws.nbytes, _stream(stream),
                                                   _stage_events(events)))
    return ids


def index_topk_i8(q_idx: torch.Tensor, k_idx: torch.Tensor, block: int, K: int, ws: Workspace,
                  ids: torch.Tensor | None = None, stream=None, events=None) -> torch.Tensor:
    """Index branch on signed 8-bit index keys (msa_index_topk_i8):
    q_idx [Bt, n_q, d_idx], k_idx [Bt, T, d_idx] int8 -> ids [Bt, n_q, K] int32,
    the same selection msa_index_topk makes on the same integer values."""
    _dev(q_idx, torch.int8, "q_idx")
    _dev(k_idx, torch.int8, "k_idx")
    Bt, n_q, d_idx = q_idx.shape
    T = k_idx.shape[1]
    if k_idx.shape != (Bt, T, d_idx):
        raise ValueError(f"k_idx shape {tuple(k_idx.shape)} does not match q_idx")
    if ids is None:
        ids = torch.empty((Bt, n_q, K), dtype=torch.int32, device=q_idx.device)
    _dev(ids, torch.int32, "ids")
    lib = load_library()
    _check("msa_index_topk_i8", lib.msa_index_topk_i8_ev(q_idx.data_ptr(), k_idx.data_ptr(),
                                                         ids.data_ptr(), Bt, n_q, T, d_idx, block,
                                                         K, ws.ptr, ws.nbytes, _stream(stream),
                                                         _stage_events(events)))
    return ids


def select_invert(ids: torch.Tensor, T: int, block: int, ws: Workspace, stream=None):
    """ids [Bt, n_q, K] int32 -> (row_ptr [Bt*N+1], entries [Bt*n_q*K]) int32 (CSR)."""
    _dev(ids, torch.int32, "ids")
    Bt, n_q, K = ids.shape
    N = (T + block - 1) // block
    row_ptr = torch.empty(Bt * N + 1, dtype=torch.int32, device=ids.device)
    entries = torch.empty(max(Bt * n_q * K, 1), dtype=torch.int32, device=ids.device)
    lib = load_library()
    _check("msa_select_invert", lib.msa_select_invert(ids.data_ptr(), row_ptr.data_ptr(),
                                                      entries.data_ptr(), Bt, n_q, T, block, K,
                                                      ws.ptr, ws.nbytes, _stream(stream)))
    return row_ptr, entries


def sparse_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, ids: torch.Tensor, block: int,
                ws: Workspace, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                stream=None, events=None):
    """q [Bt, n_q, Hq, d], k/v [Bt, T, Hkv, d] bf16, ids [Bt, n_q, K] int32
    -> (out [Bt, n_q, Hq, d] fp32, lse [Bt, n_q, Hq] fp32).
    events: optional {stage: (start, stop)} torch.cuda.Event pairs (msa_sparse_attn_ev)."""
    _dev(q, torch.bfloat16, "q")
    _dev(k, torch.bfloat16, "k")
    _dev(v, torch.bfloat16, "v")
    _dev(ids, torch.int32, "ids")
    Bt, n_q, Hq, d = q.shape
    T, Hkv = k.shape[1], k.shape[2]
    if k.shape != (Bt, T, Hkv, d) or v.shape != k.shape:
        raise ValueError("k/v shapes do not match q")
    K = ids.shape[-1]
    if ids.shape != (Bt, n_q, K):
        raise ValueError("ids shape does not match q")
    if out is None:
        out = torch.empty((Bt, n_q, Hq, d), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((Bt, n_q, Hq), dtype=torch.float32, device=q.device)
    _dev(out, torch.float32, "out")
    _dev(lse, torch.float32, "lse")
    lib = load_library()
    _check("msa_sparse_attn", lib.msa_sparse_attn_ev(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                                     ids.data_ptr(), out.data_ptr(),
                                                     lse.data_ptr(), Bt, n_q, T, Hq, Hkv, d,
                                                     block, K, ws.ptr, ws.nbytes,
                                                     _stream(stream), _stage_events(events)))
    return out, lse


def index_topk_paged(q_idx: torch.Tensor, k_idx_pages: torch.Tensor, page_table: torch.Tensor,
                     T: int, K: int, ws: Workspace, ids: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Decode index branch over paged index keys (msa_index_topk_paged):
    q_idx [Bt, 1, d_idx], k_idx_pages [num_pages, block, d_idx] bf16,
    page_table [Bt, page_stride] int32 -> ids [Bt, 1, K] int32."""
    _dev(q_idx, torch.bfloat16, "q_idx")
    _dev(k_idx_pages, torch.bfloat16, "k_idx_pages")
    _dev(page_table, torch.int32, "page_table")
    Bt, n_q, d_idx = q_idx.shape
    num_pages, block, d2 = k_idx_pages.shape
    if n_q != 1 or d2 != d_idx or page_table.dim() != 2 or page_table.shape[0] != Bt:
        raise ValueError("paged index: q_idx [Bt, 1, d_idx], k_idx_pages [pages, block, d_idx], "
                         "page_table [Bt, stride]")
    if ids is None:
        ids = torch.empty((Bt, 1, K), dtype=torch.int32, device=q_idx.device)
    _dev(ids, torch.int32, "ids")
    _check("msa_index_topk_paged", load_library().msa_index_topk_paged(
        q_idx.data_ptr(), k_idx_pages.data_ptr(), page_table.data_ptr(), page_table.shape[1],
        num_pages, ids.data_ptr(), Bt, T, d_idx, block, K, ws.ptr, ws.nbytes, _stream(stream)))
    return ids


def sparse_attn_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                      page_table: torch.Tensor, T: int, ids: torch.Tensor, ws: Workspace,
                      out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                      stream=None):
    """Decode sparse branch over paged K/V (msa_sparse_attn_paged): q [Bt, 1, Hq, d],
    k_pages/v_pages [num_pages, block, Hkv, d] bf16, page_table [Bt, page_stride]
    int32, ids [Bt, 1, K] -> (out [Bt, 1, Hq, d], lse [Bt, 1, Hq]) fp32."""
    for t, name in ((q, "q"), (k_pages, "k_pages"), (v_pages, "v_pages")):
        _dev(t, torch.bfloat16, name)
    _dev(page_table, torch.int32, "page_table")
    _dev(ids, torch.int32, "ids")
    Bt, n_q, Hq, d = q.shape
    num_pages, block, Hkv, d2 = k_pages.shape
    K = ids.shape[-1]
    if n_q != 1 or d2 != d or v_pages.shape != k_pages.shape or ids.shape != (Bt, 1, K) or \
            page_table.dim() != 2 or page_table.shape[0] != Bt:
        raise ValueError("paged attention: shapes do not match")
    if out is None:
        out = torch.empty((Bt, 1, Hq, d), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((Bt, 1, Hq), dtype=torch.float32, device=q.device)
    _dev(out, torch.float32, "out")
    _dev(lse, torch.float32, "lse")
    _check("msa_sparse_attn_paged", load_library().msa_sparse_attn_paged(
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
        page_table.shape[1], num_pages, ids.data_ptr(), out.data_ptr(), lse.data_ptr(), Bt, T, Hq,
        Hkv, d, block, K, ws.ptr, ws.nbytes, _stream(stream)))
    return out, lse


def sparse_attn_decode_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                               ids: torch.Tensor, block: int, out: torch.Tensor | None = None,
                               lse: torch.Tensor | None = None, status: torch.Tensor | None = None,
                               stream=None):
    """Decode attention (n_q = 1) whose scratch is the library's static device
    array (msa_sparse_attn_decode_noalloc): no workspace is passed and the
    library allocates nothing.  q [Bt, 1, Hq, d], k/v [Bt, T, Hkv, d] bf16,
    ids [Bt, 1, K] int32 -> (out [Bt, 1, Hq, d], lse [Bt, 1, Hq]) fp32.
    status: optional int32 CUDA tensor of one element that receives error bits."""
    _dev(q, torch.bfloat16, "q")
    _dev(k, torch.bfloat16, "k")
    _dev(v, torch.bfloat16, "v")
    _dev(ids, torch.int32, "ids")
    Bt, n_q, Hq, d = q.shape
    if n_q != 1:
        raise ValueError("the no-allocation entry point serves decode steps (n_q == 1)")
    T, Hkv = k.shape[1], k.shape[2]
    K = ids.shape[-1]
    if out is None:
        out = torch.empty((Bt, 1, Hq, d), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((Bt, 1, Hq), dtype=torch.float32, device=q.device)
    sp = 0
    if status is not None:
        _dev(status, torch.int32, "status")
        sp = status.data_ptr()
    lib = load_library()
    _check("msa_sparse_attn_decode_noalloc",
           lib.msa_sparse_attn_decode_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                              ids.data_ptr(), out.data_ptr(), lse.data_ptr(), Bt,
                                              T, Hq, Hkv, d, block, K, sp or None,
                                              _stream(stream)))
    return out, lse


BINDING_PATH = os.path.join(_HERE, "_msa_torch.so")
_fast = None


def load_binding(path: str = BINDING_PATH):
    """Load the compiled binding of the paged-cache calls (raises if it has not been
    built).  It checks the tensors against the workspace's device, makes the outputs
    that are not given, and calls libmsa on that device and its current stream."""
    global _fast
    if _fast is not None:
        return _fast
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m block_sparse_long_05_b200.build`")
    lib = load_library()
    spec = importlib.util.spec_from_file_location("_msa_torch", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.bind(*(ctypes.cast(getattr(lib, "msa_" + f), ctypes.c_void_p).value for f in (
        "kv_append", "kv_append_i8", "kv_gather", "kv_gather_i8", "attn_paged", "attn_paged_i8",
        "sparse_attn_paged_i8")))
    _fast = mod
    return mod


def kv_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
              page_table: torch.Tensor, cu: torch.Tensor, kv_len: torch.Tensor, ws: Workspace,
              k_idx: torch.Tensor | None = None, k_idx_pages: torch.Tensor | None = None,
              stream=None) -> None:
    """A step's new rows into the pages (msa_kv_append): k, v [total, Hkv, d] bf16 (rows
    may be strided), k_pages / v_pages [num_pages, block, Hkv, d] bf16, page_table
    [Bt, page_stride], cu [Bt + 1], kv_len [Bt] int32; optionally the index keys k_idx
    [total, d_idx] into k_idx_pages [num_pages, block, d_idx]."""
    r = (_fast or load_binding()).append(ws.ptr, ws.nbytes, ws.device_index, stream, False, k, v,
                                         k_pages, v_pages, None, None, page_table, cu, kv_len,
                                         k_idx, k_idx_pages)
    if r is not None:
        raise MSAError("msa_kv_append", r)


def kv_append_i8(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                 k_scales: torch.Tensor, v_scales: torch.Tensor, page_table: torch.Tensor,
                 cu: torch.Tensor, kv_len: torch.Tensor, ws: Workspace,
                 k_idx: torch.Tensor | None = None, k_idx_pages: torch.Tensor | None = None,
                 stream=None) -> None:
    """kv_append into int8 pages with a scale per (token, kv head) row
    (msa_kv_append_i8): k_scales / v_scales [num_pages, Hkv, block] fp32."""
    r = (_fast or load_binding()).append(ws.ptr, ws.nbytes, ws.device_index, stream, True, k, v,
                                         k_pages, v_pages, k_scales, v_scales, page_table, cu,
                                         kv_len, k_idx, k_idx_pages)
    if r is not None:
        raise MSAError("msa_kv_append_i8", r)


def kv_gather(k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
              cu: torch.Tensor, kv_len: torch.Tensor, total: int, ws: Workspace,
              k: torch.Tensor | None = None, v: torch.Tensor | None = None, stream=None):
    """Cached rows of a step's positions as packed bf16 (msa_kv_gather):
    -> (k, v) [total, Hkv, d].  Rows behind cu[Bt] are left as they were."""
    r = (_fast or load_binding()).gather(ws.ptr, ws.nbytes, ws.device_index, stream, False, total,
                                         k_pages, v_pages, None, None, page_table, cu, kv_len, k, v)
    if r.__class__ is int:
        raise MSAError("msa_kv_gather", r)
    return r


def kv_gather_i8(k_pages: torch.Tensor, v_pages: torch.Tensor, k_scales: torch.Tensor,
                 v_scales: torch.Tensor, page_table: torch.Tensor, cu: torch.Tensor,
                 kv_len: torch.Tensor, total: int, ws: Workspace, k: torch.Tensor | None = None,
                 v: torch.Tensor | None = None, stream=None):
    """kv_gather from int8 pages (msa_kv_gather_i8): code * scale, rounded once."""
    r = (_fast or load_binding()).gather(ws.ptr, ws.nbytes, ws.device_index, stream, True, total,
                                         k_pages, v_pages, k_scales, v_scales, page_table, cu,
                                         kv_len, k, v)
    if r.__class__ is int:
        raise MSAError("msa_kv_gather_i8", r)
    return r


def attn_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
               page_table: torch.Tensor, cu: torch.Tensor, kv_len: torch.Tensor, ws: Workspace,
               window: int = 0, sinks: int = 0, max_q: int | None = None,
               out: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None):
    """Attention of a step's rows over their cached contexts (msa_attn_paged): q
    [total, Hq, d] bf16 (rows may be strided) over k_pages / v_pages
    [num_pages, block, Hkv, d] bf16 -> (out [total, Hq, d] bf16, lse [total, Hq] fp32).
    window > 0: each query sees the last `window` keys and the first `sinks` ones.
    max_q: the largest number of rows of one sequence, if known.  It chooses kernels: a
    decode step (max_q=1) without it takes up to 1.8 times as long."""
    r = (_fast or load_binding()).attend(ws.ptr, ws.nbytes, ws.device_index, stream, False, q,
                                         k_pages, v_pages, None, None, page_table, cu, kv_len,
                                         window, sinks, max_q, out, lse)
    if r.__class__ is int:
        raise MSAError("msa_attn_paged", r)
    return r


def attn_paged_i8(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                  k_scales: torch.Tensor, v_scales: torch.Tensor, page_table: torch.Tensor,
                  cu: torch.Tensor, kv_len: torch.Tensor, ws: Workspace, window: int = 0,
                  sinks: int = 0, max_q: int | None = None, out: torch.Tensor | None = None,
                  lse: torch.Tensor | None = None, stream=None):
    """attn_paged over int8 pages with their scales (msa_attn_paged_i8)."""
    r = (_fast or load_binding()).attend(ws.ptr, ws.nbytes, ws.device_index, stream, True, q,
                                         k_pages, v_pages, k_scales, v_scales, page_table, cu,
                                         kv_len, window, sinks, max_q, out, lse)
    if r.__class__ is int:
        raise MSAError("msa_attn_paged_i8", r)
    return r


def attn_paged_kernels(Bt: int, total: int, Hq: int, Hkv: int, block: int, page_stride: int,
                       window: int = 0, sinks: int = 0, max_q: int | None = None) -> tuple[str, ...]:
    """The kernels that attn_paged and attn_paged_i8 launch for a step of these sizes
    (msa_attn_paged_kernels): "split", "chunk", both, or none."""
    m = load_library().msa_attn_paged_kernels(Bt, total, max_q or 0, Hq, Hkv, block, page_stride,
                                              window, sinks)
    return tuple(name for bit, name in ((1, "split"), (2, "chunk")) if m & bit)


def sparse_attn_paged_i8(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                         k_scales: torch.Tensor, v_scales: torch.Tensor, page_table: torch.Tensor,
                         T: int, ids: torch.Tensor, ws: Workspace, out: torch.Tensor | None = None,
                         lse: torch.Tensor | None = None, stream=None):
    """Decode sparse branch over int8 pages (msa_sparse_attn_paged_i8): q [Bt, 1, Hq, d]
    bf16, ids [Bt, 1, K] int32 -> (out [Bt, 1, Hq, d] bf16, lse [Bt, 1, Hq] fp32).  ws is
    a cache workspace (Workspace.for_cache)."""
    r = (_fast or load_binding()).sparse(ws.ptr, ws.nbytes, ws.device_index, stream, q, k_pages,
                                         v_pages, k_scales, v_scales, page_table, T, ids, out, lse)
    if r.__class__ is int:
        raise MSAError("msa_sparse_attn_paged_i8", r)
    return r


def device_status(ws: Workspace, stream=None) -> int:
    """Synchronise the stream, read and clear the workspace's device status."""
    return int(load_library().msa_device_status(ws.ptr, _stream(stream)))


def status_string(code: int) -> str:
    return load_library().msa_status_string(int(code)).decode()


def selftest_umma(A: torch.Tensor, B: torch.Tensor, b_mn_major: bool, a_tmem: bool = False,
                  stream=None):
    """C[128, N] = A[128, Kd] @ B with B as [N, Kd] (K-major) or [Kd, N] (MN-major);
    a_tmem: the MMA reads A from tensor memory."""
    _dev(A, torch.bfloat16, "A")
    _dev(B, torch.bfloat16, "B")
    Kd = A.shape[1]
    N = B.shape[1] if b_mn_major else B.shape[0]
    C = torch.empty((128, N), dtype=torch.float32, device=A.device)
    status = torch.zeros(1, dtype=torch.int32, device=A.device)
    lib = load_library()
    flags = int(b_mn_major) | (2 if a_tmem else 0)
    _check("msa_selftest_umma", lib.msa_selftest_umma(A.data_ptr(), B.data_ptr(), C.data_ptr(), N,
                                                      Kd, flags, status.data_ptr(),
                                                      _stream(stream)))
    return C, status
