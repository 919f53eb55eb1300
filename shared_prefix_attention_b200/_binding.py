"""ctypes binding of libpsa.  Argument marshalling only: every step of the
attention path runs in the library's CUDA kernels; PyTorch supplies device
memory and the current stream.  There is no CPU fallback -- if the library
is missing, importing a call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Sequence

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpsa.so")
# The same library built with device-side bounds checks (PSA_DEBUG): an index
# taken from caller data outside its buffer is reported as PSA_ERR_BOUNDS
# through the status word instead of being followed.
DEBUG_LIB_PATH = os.path.join(_HERE, "libpsa_debug.so")

PSA_OK = 0
PSA_ERR_INVALID_ARG = 1
PSA_ERR_UNSUPPORTED = 2
PSA_ERR_WORKSPACE = 3
PSA_ERR_CUDA = 4
PSA_ERR_TIMEOUT = 5
PSA_ERR_CAPACITY = 6
PSA_ERR_BOUNDS = 7
PSA_BF16 = 0
PSA_F32 = 1

# Every symbol include/psa.h declares.
EXPORTS = [
    "psa_version", "psa_status_string", "psa_spec_flat", "psa_build_spec",
    "psa_build_schedule", "psa_prefill_tiles", "psa_prefill_workspace_size",
    "psa_prefill_fwd", "psa_verify_auto_splits", "psa_verify_workspace_size",
    "psa_verify_fwd", "psa_verify_fwd_noalloc", "psa_sparse_latent_fwd", "psa_read_status",
    "psa_wait_selftest", "psa_verify_shared_auto_splits", "psa_verify_shared_fwd",
    "psa_verify_shared_tree_fwd",
    "psa_verify_fp8_fwd", "psa_transpose_spec", "psa_prefill_bwd_tiles",
    "psa_prefill_bwd_workspace_size", "psa_prefill_bwd", "psa_verify_tree_fwd",
    "psa_verify_extend_fwd", "psa_qk_norm_rope_fwd", "psa_qk_norm_rope_bwd_workspace_size",
    "psa_qk_norm_rope_bwd", "psa_cache_append", "psa_cache_read", "psa_build_chunk_plan",
    "psa_chunk_workspace_size", "psa_chunk_fwd",
]


class PsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class Segment(ctypes.Structure):
    _fields_ = [("len", ctypes.c_int32), ("parent", ctypes.c_int32)]


class Rect(ctypes.Structure):
    _fields_ = [("q0", ctypes.c_int32), ("q1", ctypes.c_int32), ("k0", ctypes.c_int32),
                ("k1", ctypes.c_int32), ("causal", ctypes.c_int32)]


class VerifyFeatures(ctypes.Structure):
    _fields_ = [("has_custom_mask", ctypes.c_int32), ("is_causal", ctypes.c_int32),
                ("sliding_window", ctypes.c_int32), ("has_sinks", ctypes.c_int32),
                ("logit_cap", ctypes.c_float), ("xai_temperature_len", ctypes.c_int32),
                ("ragged_extend", ctypes.c_int32)]


class KvScales(ctypes.Structure):
    """psa_kv_scales: per-tensor scales of an e4m3 KV cache."""
    _fields_ = [("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class NormRope(ctypes.Structure):
    """psa_norm_rope: the norm and rotation of query and key rows."""
    _fields_ = [("positions", ctypes.c_void_p), ("cos_sin", ctypes.c_void_p),
                ("n_positions", ctypes.c_int64), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("weight_dtype", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class ChunkInfo(ctypes.Structure):
    """psa_chunk_info: what a chunk plan was built for."""
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("window", ctypes.c_int32),
                ("n_rows", ctypes.c_int32), ("n_ctas", ctypes.c_int32),
                ("n_units", ctypes.c_int32), ("n_joins", ctypes.c_int32),
                ("max_join_rows", ctypes.c_int32), ("all_twin", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("n_keys", ctypes.c_int64),
                ("part_rows", ctypes.c_int64), ("len", ctypes.c_int64)]


_lib = None


def lib():
    """The loaded libpsa (raises if it has not been built)."""
    global _lib
    if _lib is None:
        _lib = load(LIB_PATH)
    return _lib


class use_library:
    """Context manager: the binding's calls go to the library at ``path``
    (e.g. DEBUG_LIB_PATH) inside the block, and back to the previous one
    after it."""

    def __init__(self, path: str):
        self.path = path

    def __enter__(self):
        global _lib
        self.saved = _lib
        _lib = load(self.path)
        return _lib

    def __exit__(self, *exc):
        global _lib
        _lib = self.saved
        return False


_loaded: dict = {}


def load(path: str):
    """Load a build of libpsa and declare its C signatures (cached per path;
    raises if the file is missing)."""
    if path in _loaded:
        return _loaded[path]
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m shared_prefix_attention_b200.build`")
    L = ctypes.CDLL(path)
    P, I32, I64, SZ, F = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t,
                          ctypes.c_float)
    sig = {
        "psa_version": ([], ctypes.c_int),
        "psa_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "psa_spec_flat": ([I32, I32, I32, P, I32, P], ctypes.c_int),
        "psa_build_spec": ([P, I32, P, I32, P], ctypes.c_int),
        "psa_build_schedule": ([P, I32, P, I32, I32, I32, P, I64, P], ctypes.c_int),
        "psa_prefill_tiles": ([I32, P, P], ctypes.c_int),
        "psa_prefill_workspace_size": ([ctypes.c_int, I32, I32, I32, I32], SZ),
        "psa_prefill_fwd": ([P, P, P, P, P, ctypes.c_int, I32, I32, I32, I32, F, P, I64, P, SZ,
                             P, P], ctypes.c_int),
        "psa_verify_auto_splits": ([I32, I64, I32, I32], I32),
        "psa_verify_workspace_size": ([I32, I32, I32, I32, I32], SZ),
        "psa_verify_fwd": ([P, P, P, P, P, I64, P, I64, P, P, P, I32, I32, I32, I32, I32, F, I32,
                            P, P, SZ, P, P], ctypes.c_int),
        "psa_verify_fwd_noalloc": ([P, P, P, P, P, I64, P, I64, P, P, P, I32, I32, I32, I32, I32,
                                    F, I32, P, P, P], ctypes.c_int),
        "psa_sparse_latent_fwd": ([P, P, P, P, P, I32, I32, I32, I32, I32, F, P, P],
                                  ctypes.c_int),
        "psa_read_status": ([P, P, P], ctypes.c_int),
        "psa_wait_selftest": ([I32, P, P], ctypes.c_int),
        "psa_verify_shared_auto_splits": ([I32, I32, I32, I32, I64], I32),
        "psa_transpose_spec": ([P, I32, P], ctypes.c_int),
        "psa_prefill_bwd_tiles": ([I32, P, P], ctypes.c_int),
        "psa_verify_tree_fwd": ([P, P, P, P, P, I64, P, I64, P, P, P, P, I32, I32, I32, I32, I32,
                                 F, I32, P, P, SZ, P, P], ctypes.c_int),
        "psa_verify_extend_fwd": ([P, P, P, P, P, I64, P, I32, I32, P, I64, P, P, P, P, P, P,
                                   I32, I32, I32, I32, F, I32, P, P, SZ, P, P], ctypes.c_int),
        "psa_prefill_bwd_workspace_size": ([I32, I32], SZ),
        "psa_prefill_bwd": ([P, P, P, P, P, P, P, P, P, I32, I32, I32, I32, F, P, I64, P, I64, P,
                             SZ, P, P], ctypes.c_int),
        "psa_verify_fp8_fwd": ([P, P, P, P, P, I64, P, I64, P, F, F, P, P, I32, I32, I32, I32,
                                I32, F, I32, P, P, SZ, P, P], ctypes.c_int),
        "psa_verify_shared_tree_fwd": ([P, P, P, P, P, I64, P, P, P, I32, I32, I32, I32, I32, F,
                                        I32, P, ctypes.c_size_t, P, P], ctypes.c_int),
        "psa_verify_shared_fwd": ([P, P, P, P, P, I64, P, P, I32, I32, I32, I32, I32, F, I32, P,
                                   ctypes.c_size_t, P, P], ctypes.c_int),
        "psa_qk_norm_rope_fwd": ([P, I64, P, I64, ctypes.c_int, I32, I32, I32, I32, P, P, P, P,
                                  P], ctypes.c_int),
        "psa_qk_norm_rope_bwd_workspace_size": ([I32], SZ),
        "psa_qk_norm_rope_bwd": ([P, I64, P, I64, P, P, ctypes.c_int, I32, I32, I32, I32, P, P,
                                  I64, P, I64, P, P, P, SZ, P, P], ctypes.c_int),
        "psa_cache_append": ([P, I64, P, I64, P, I64, I32, I32, I32, I32, P, P, P, I64, P, P, P,
                              P, P], ctypes.c_int),
        "psa_cache_read": ([P, P, I64, P, I64, I32, I32, P, P, P, P, P], ctypes.c_int),
        "psa_build_chunk_plan": ([P, P, I32, I32, I32, I32, I32, I32, P, I64, P], ctypes.c_int),
        "psa_chunk_workspace_size": ([P], SZ),
        "psa_chunk_fwd": ([P, P, P, I64, P, P, P, P, I32, F, F, P, P, P, SZ, P, P], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _loaded[path] = L
    return L


def status_string(status: int) -> str:
    return lib().psa_status_string(int(status)).decode()


def _check(rc: int, where: str):
    if rc != PSA_OK:
        raise PsaError(rc, where)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data_as(ctypes.c_void_p)
    return ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _require_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("psa kernels take CUDA tensors; there is no CPU path")
        if t is not None and not t.is_contiguous():
            raise ValueError("psa kernels take contiguous tensors")


# ---------------------------------------------------------------- host spec

def spec_flat(P: int, N: int, S: int) -> list[tuple[int, int]]:
    n = ctypes.c_int32(0)
    lib().psa_spec_flat(P, N, S, None, 0, ctypes.byref(n))
    arr = (Segment * max(1, n.value))()
    _check(lib().psa_spec_flat(P, N, S, arr, n.value, ctypes.byref(n)), "psa_spec_flat")
    return [(arr[i].len, arr[i].parent) for i in range(n.value)]


def build_spec(segments: Sequence[tuple[int, int]]) -> np.ndarray:
    """Rectangles [n, 5] int32 (q0, q1, k0, k1, causal) for a segment forest."""
    segs = (Segment * max(1, len(segments)))(*[Segment(int(a), int(b)) for a, b in segments])
    n = ctypes.c_int32(0)
    rc = lib().psa_build_spec(segs, len(segments), None, 0, ctypes.byref(n))
    if rc not in (PSA_OK, PSA_ERR_CAPACITY):
        _check(rc, "psa_build_spec")
    out = np.zeros((max(1, n.value), 5), dtype=np.int32)
    _check(lib().psa_build_spec(segs, len(segments), _ptr(out), n.value, ctypes.byref(n)),
           "psa_build_spec")
    return out[:n.value]


def prefill_tiles(head_dim: int) -> tuple[int, int]:
    m, n = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(lib().psa_prefill_tiles(head_dim, ctypes.byref(m), ctypes.byref(n)),
           "psa_prefill_tiles")
    return m.value, n.value


def build_schedule(rects: np.ndarray, cu_seqlens: Sequence[int], tile_m: int,
                   tile_n: int) -> np.ndarray:
    """Tile schedule (host int32 array) for :func:`prefill`."""
    rects = np.ascontiguousarray(rects, dtype=np.int32)
    cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int32))
    n = ctypes.c_int64(0)
    ng = len(cu) - 1
    rc = lib().psa_build_schedule(_ptr(rects), len(rects), _ptr(cu), ng, tile_m, tile_n, None, 0,
                                  ctypes.byref(n))
    if rc not in (PSA_OK, PSA_ERR_CAPACITY):
        _check(rc, "psa_build_schedule")
    out = np.zeros(n.value, dtype=np.int32)
    _check(lib().psa_build_schedule(_ptr(rects), len(rects), _ptr(cu), ng, tile_m, tile_n,
                                    _ptr(out), n.value, ctypes.byref(n)), "psa_build_schedule")
    return out


def transpose_spec(rects: np.ndarray) -> np.ndarray:
    """Rectangles with rows and columns swapped (keys become rows)."""
    rects = np.ascontiguousarray(rects, dtype=np.int32)
    out = np.zeros_like(rects)
    _check(lib().psa_transpose_spec(_ptr(rects), len(rects), _ptr(out)), "psa_transpose_spec")
    return out


def plan_prefill(segments, cu_seqlens, head_dim: int, device="cuda") -> torch.Tensor:
    """Spec + schedule for a segment forest, uploaded to ``device``."""
    tm, tn = prefill_tiles(head_dim)
    sched = build_schedule(build_spec(segments), cu_seqlens, tm, tn)
    return torch.from_numpy(sched).to(device)


# ---------------------------------------------------------------- kernels

def prefill(q, k, v, schedule: torch.Tensor, scale: float, out=None, lse=None,
            workspace=None, status=None):
    """O [T, Hq, d] (q's dtype) and LSE [T, Hq] fp32 over the flat layout."""
    _require_cuda(q, k, v, schedule, out, lse, workspace)
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    dtype = {torch.bfloat16: PSA_BF16, torch.float32: PSA_F32}[q.dtype]
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device) if lse is None else lse
    if workspace is None:
        nbytes = lib().psa_prefill_workspace_size(dtype, T, Hq, Hkv, d)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    rc = lib().psa_prefill_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), dtype, T, Hq,
                               Hkv, d, float(scale), _ptr(schedule), schedule.numel(),
                               _ptr(workspace), workspace.numel(), _word(status, q.device),
                               _stream(q.device))
    _check(rc, "psa_prefill_fwd")
    return out, lse


def verify_workspace_size(B: int, Ld: int, Hq: int, head_dim: int, nsplit: int) -> int:
    return int(lib().psa_verify_workspace_size(B, Ld, Hq, head_dim, nsplit))


def verify_auto_splits(B: int, max_prefix_len: int, Hkv: int, head_dim: int) -> int:
    return int(lib().psa_verify_auto_splits(B, max_prefix_len, Hkv, head_dim))


def verify(q_draft, k_draft, v_draft, k_cache, v_cache, kv_indptr: torch.Tensor,
           max_prefix_len: int, scale: float, Ld: int, nsplit: int = 0, out=None, lse=None,
           workspace=None, status=None, features: VerifyFeatures | None = None,
           kv_indices=None):
    """Split-KV verify.  kv_indptr: device int32 [B+1] prefix offsets."""
    _require_cuda(q_draft, k_draft, v_draft, k_cache, v_cache, kv_indptr, out, lse, workspace,
                  kv_indices)
    BL, Hq, d = q_draft.shape
    Hkv = k_cache.shape[1]
    B = BL // Ld
    if nsplit == 0:
        nsplit = verify_auto_splits(B, max_prefix_len, Hkv, d)
    out = torch.empty_like(q_draft) if out is None else out
    lse = torch.empty((BL, Hq), dtype=torch.float32, device=q_draft.device) if lse is None else lse
    if workspace is None:
        workspace = torch.empty(max(256, verify_workspace_size(B, Ld, Hq, d, nsplit)),
                                dtype=torch.uint8, device=q_draft.device)
    rc = lib().psa_verify_fwd(_ptr(q_draft), _ptr(k_draft), _ptr(v_draft), _ptr(k_cache),
                              _ptr(v_cache), k_cache.shape[0], _ptr(kv_indptr),
                              int(max_prefix_len), _ptr(kv_indices), _ptr(out), _ptr(lse), B,
                              Ld, Hq, Hkv, d, float(scale), nsplit,
                              ctypes.byref(features) if features is not None else None,
                              _ptr(workspace), workspace.numel(), _word(status, q_draft.device),
                              _stream(q_draft.device))
    _check(rc, "psa_verify_fwd")
    return out, lse


def verify_noalloc(q_draft, k_draft, v_draft, k_cache, v_cache, kv_indptr: torch.Tensor,
                   max_prefix_len: int, scale: float, Ld: int, nsplit: int = 0, out=None,
                   lse=None, status=None):
    """Split-KV verify through psa_verify_fwd_noalloc: the library's fixed
    device scratch replaces the workspace (for callers that cannot allocate
    device memory at the call site).  Outputs are allocated here only for
    convenience; pass ``out`` / ``lse`` to avoid that too."""
    _require_cuda(q_draft, k_draft, v_draft, k_cache, v_cache, kv_indptr, out, lse)
    BL, Hq, d = q_draft.shape
    Hkv = k_cache.shape[1]
    if Ld <= 0 or BL % Ld != 0:
        raise ValueError(f"verify_noalloc: {BL} draft rows are not a whole number of "
                         f"requests of {Ld} drafts")
    B = BL // Ld
    out = torch.empty_like(q_draft) if out is None else out
    lse = torch.empty((BL, Hq), dtype=torch.float32, device=q_draft.device) if lse is None else lse
    rc = lib().psa_verify_fwd_noalloc(_ptr(q_draft), _ptr(k_draft), _ptr(v_draft),
                                      _ptr(k_cache), _ptr(v_cache), k_cache.shape[0],
                                      _ptr(kv_indptr), int(max_prefix_len), None, _ptr(out),
                                      _ptr(lse), B, Ld, Hq, Hkv, d, float(scale), nsplit, None,
                                      _word(status, q_draft.device), _stream(q_draft.device))
    _check(rc, "psa_verify_fwd_noalloc")
    return out, lse


def sparse_latent(q, latent, idx, scale: float, out=None, lse=None, status=None):
    """Shared-latent sparse attention: O [T, H, dl] bf16, LSE [T, H] fp32."""
    _require_cuda(q, latent, idx, out, lse)
    T, H, dl = q.shape
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((T, H), dtype=torch.float32, device=q.device) if lse is None else lse
    rc = lib().psa_sparse_latent_fwd(_ptr(q), _ptr(latent), _ptr(idx), _ptr(out), _ptr(lse), T,
                                     latent.shape[0], H, dl, idx.shape[1], float(scale),
                                     _word(status, q.device), _stream(q.device))
    _check(rc, "psa_sparse_latent_fwd")
    return out, lse


def read_status(status: torch.Tensor) -> int:
    v = ctypes.c_int32(0)
    _check(lib().psa_read_status(_ptr(status), ctypes.byref(v), _stream(status.device)),
           "psa_read_status")
    return v.value


def wait_selftest(status: torch.Tensor, arrive: bool) -> None:
    """Launches the library's bounded-wait self-test on ``status``'s device:
    with ``arrive`` the wait completes at once, without it the wait gives up
    after the library's budget and writes PSA_ERR_TIMEOUT to ``status``."""
    _check(lib().psa_wait_selftest(1 if arrive else 0, _ptr(status), _stream(status.device)),
           "psa_wait_selftest")


def verify_shared_auto_splits(B: int, Ld: int, Hq: int, Hkv: int, prefix_len: int) -> int:
    return int(lib().psa_verify_shared_auto_splits(B, Ld, Hq, Hkv, int(prefix_len)))


def verify_shared(q_draft, k_draft, v_draft, k_prefix, v_prefix, scale: float, Ld: int,
                  nsplit: int = 0, out=None, lse=None, workspace=None, status=None,
                  draft_mask=None):
    """Verify against one prefix shared by every request: O [B*Ld, Hq, d]
    bf16 and LSE [B*Ld, Hq] fp32; k_prefix/v_prefix [L, Hkv, d].  With
    draft_mask (device uint8 [B*Ld, Ld]) the draft block is that tree mask."""
    _require_cuda(q_draft, k_draft, v_draft, k_prefix, v_prefix, out, lse, workspace,
                  draft_mask)
    BL, Hq, d = q_draft.shape
    Hkv = k_draft.shape[1]
    B = BL // Ld
    L = k_prefix.shape[0]
    ns = nsplit or verify_shared_auto_splits(B, Ld, Hq, Hkv, L)
    out = torch.empty_like(q_draft) if out is None else out
    lse = torch.empty((BL, Hq), dtype=torch.float32, device=q_draft.device) if lse is None else lse
    if workspace is None:
        workspace = torch.empty(max(verify_workspace_size(B, Ld, Hq, d, ns), 256),
                                dtype=torch.uint8, device=q_draft.device)
    kp, vp = (_ptr(k_prefix) if L else None), (_ptr(v_prefix) if L else None)
    if draft_mask is None:
        rc = lib().psa_verify_shared_fwd(_ptr(q_draft), _ptr(k_draft), _ptr(v_draft), kp, vp, L,
                                         _ptr(out), _ptr(lse), B, Ld, Hq, Hkv, d, float(scale), ns,
                                         _ptr(workspace), workspace.numel(),
                                         _word(status, q_draft.device), _stream(q_draft.device))
        _check(rc, "psa_verify_shared_fwd")
    else:
        rc = lib().psa_verify_shared_tree_fwd(_ptr(q_draft), _ptr(k_draft), _ptr(v_draft), kp, vp,
                                              L, _ptr(draft_mask), _ptr(out), _ptr(lse), B, Ld,
                                              Hq, Hkv, d, float(scale), ns, _ptr(workspace),
                                              workspace.numel(), _word(status, q_draft.device),
                                              _stream(q_draft.device))
        _check(rc, "psa_verify_shared_tree_fwd")
    return out, lse


def verify_fp8(q_draft, k_draft, v_draft, k_cache8, v_cache8, k_scale: float, v_scale: float,
               kv_indptr: torch.Tensor, max_prefix_len: int, scale: float, Ld: int,
               nsplit: int = 0, out=None, lse=None, workspace=None, status=None,
               kv_indices=None):
    """Split-KV verify over an e4m3 prefix cache (uint8 or float8_e4m3fn
    tensors [Ntok, Hkv, d]) standing for k_scale * e4m3 and v_scale * e4m3;
    kv_indices: optional token-granular page table (device int32)."""
    _require_cuda(q_draft, k_draft, v_draft, k_cache8, v_cache8, kv_indptr, out, lse,
                  workspace, kv_indices)
    BL, Hq, d = q_draft.shape
    Hkv = k_draft.shape[1]
    B = BL // Ld
    ns = nsplit or verify_auto_splits(B, max_prefix_len, Hkv, d)
    out = torch.empty_like(q_draft) if out is None else out
    lse = torch.empty((BL, Hq), dtype=torch.float32, device=q_draft.device) if lse is None else lse
    if workspace is None:
        workspace = torch.empty(max(verify_workspace_size(B, Ld, Hq, d, ns), 256),
                                dtype=torch.uint8, device=q_draft.device)
    rc = lib().psa_verify_fp8_fwd(_ptr(q_draft), _ptr(k_draft), _ptr(v_draft), _ptr(k_cache8),
                                  _ptr(v_cache8), k_cache8.shape[0], _ptr(kv_indptr),
                                  int(max_prefix_len), _ptr(kv_indices), float(k_scale),
                                  float(v_scale),
                                  _ptr(out), _ptr(lse), B, Ld, Hq, Hkv, d, float(scale), ns, None,
                                  _ptr(workspace), workspace.numel(), _word(status, q_draft.device),
                                  _stream(q_draft.device))
    _check(rc, "psa_verify_fp8_fwd")
    return out, lse


def prefill_bwd_tiles(head_dim: int):
    tm, tn = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(lib().psa_prefill_bwd_tiles(head_dim, ctypes.byref(tm), ctypes.byref(tn)),
           "psa_prefill_bwd_tiles")
    return tm.value, tn.value


def plan_prefill_bwd(segments, cu_seqlens, head_dim: int, device="cuda"):
    """The two backward schedules (row-major for dQ, key-major for dK / dV)
    for a segment forest, uploaded to ``device``."""
    tm, tn = prefill_bwd_tiles(head_dim)
    spec = build_spec(segments)
    sq = build_schedule(spec, cu_seqlens, tm, tn)
    skv = build_schedule(transpose_spec(spec), cu_seqlens, tm, tn)
    return torch.from_numpy(sq).to(device), torch.from_numpy(skv).to(device)


def prefill_bwd(q, k, v, o, lse, dout, schedules, scale: float, dq=None, dk=None, dv=None,
                workspace=None, status=None):
    """Gradients (dq, dk, dv) of the prefill output for upstream gradient
    ``dout``; ``schedules`` from :func:`plan_prefill_bwd`."""
    sq, skv = schedules
    _require_cuda(q, k, v, o, lse, dout, sq, skv, dq, dk, dv, workspace)
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        workspace = torch.empty(max(int(lib().psa_prefill_bwd_workspace_size(T, Hq)), 256),
                                dtype=torch.uint8, device=q.device)
    rc = lib().psa_prefill_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout),
                               _ptr(dq), _ptr(dk), _ptr(dv), T, Hq, Hkv, d, float(scale),
                               _ptr(sq), sq.numel(), _ptr(skv), skv.numel(), _ptr(workspace),
                               workspace.numel(), _word(status, q.device), _stream(q.device))
    _check(rc, "psa_prefill_bwd")
    return dq, dk, dv


def verify_tree(q_draft, k_draft, v_draft, k_cache, v_cache, kv_indptr: torch.Tensor,
                max_prefix_len: int, draft_mask: torch.Tensor, scale: float, Ld: int,
                nsplit: int = 0, out=None, lse=None, workspace=None, status=None,
                kv_indices=None):
    """Split-KV verify with a custom draft mask (device uint8 [B*Ld, Ld])."""
    _require_cuda(q_draft, k_draft, v_draft, k_cache, v_cache, kv_indptr, draft_mask, out,
                  lse, workspace, kv_indices)
    BL, Hq, d = q_draft.shape
    Hkv = k_draft.shape[1]
    B = BL // Ld
    ns = nsplit or verify_auto_splits(B, max_prefix_len, Hkv, d)
    out = torch.empty_like(q_draft) if out is None else out
    lse = torch.empty((BL, Hq), dtype=torch.float32, device=q_draft.device) if lse is None else lse
    if workspace is None:
        workspace = torch.empty(max(verify_workspace_size(B, Ld, Hq, d, ns), 256),
                                dtype=torch.uint8, device=q_draft.device)
    feat = VerifyFeatures(1, 1, -1, 0, 0.0, -1, 0)
    rc = lib().psa_verify_tree_fwd(_ptr(q_draft), _ptr(k_draft), _ptr(v_draft), _ptr(k_cache),
                                   _ptr(v_cache), k_cache.shape[0], _ptr(kv_indptr),
                                   int(max_prefix_len), _ptr(kv_indices), _ptr(draft_mask),
                                   _ptr(out),
                                   _ptr(lse), B, Ld, Hq, Hkv, d, float(scale), ns,
                                   ctypes.byref(feat), _ptr(workspace), workspace.numel(),
                                   _word(status, q_draft.device), _stream(q_draft.device))
    _check(rc, "psa_verify_tree_fwd")
    return out, lse


def verify_extend(q_draft, k_draft, v_draft, k_cache, v_cache, qo_indptr: torch.Tensor,
                  max_draft_len: int, kv_indptr: torch.Tensor, max_prefix_len: int,
                  scale: float, kv_indices=None, draft_mask=None, mask_indptr=None,
                  nsplit: int = 0, out=None, lse=None, workspace=None, status=None,
                  k_scale: float | None = None, v_scale: float | None = None):
    """Verify in the extend form: ragged draft counts (qo_indptr, device int32
    [B+1]), an optional page table (kv_indices: prefix position t is cache row
    kv_indices[t]) and optional per-request tree masks (flat device uint8,
    request b's Lb x Lb block at mask_indptr[b]).  With k_scale / v_scale the
    caches hold e4m3 bytes standing for k_scale * e4m3 and v_scale * e4m3."""
    _require_cuda(q_draft, k_draft, v_draft, k_cache, v_cache, qo_indptr, kv_indptr, out,
                  lse, workspace, kv_indices, draft_mask, mask_indptr)
    NR, Hq, d = q_draft.shape
    Hkv = k_draft.shape[1]
    B = qo_indptr.numel() - 1
    ns = nsplit or verify_auto_splits(B, max_prefix_len, Hkv, d)
    out = torch.empty_like(q_draft) if out is None else out
    lse = torch.empty((NR, Hq), dtype=torch.float32, device=q_draft.device) if lse is None else lse
    if workspace is None:
        workspace = torch.empty(max(verify_workspace_size(1, NR, Hq, d, ns), 256),
                                dtype=torch.uint8, device=q_draft.device)
    feat = VerifyFeatures(int(draft_mask is not None), 1, -1, 0, 0.0, -1, 1)
    sc = None
    if k_scale is not None or v_scale is not None:
        sc = ctypes.byref(KvScales(float(k_scale), float(v_scale)))
    rc = lib().psa_verify_extend_fwd(_ptr(q_draft), _ptr(k_draft), _ptr(v_draft),
                                     _ptr(k_cache), _ptr(v_cache), k_cache.shape[0],
                                     _ptr(qo_indptr), NR, int(max_draft_len), _ptr(kv_indptr),
                                     int(max_prefix_len), _ptr(kv_indices), _ptr(draft_mask),
                                     _ptr(mask_indptr), sc, _ptr(out), _ptr(lse), B, Hq, Hkv, d,
                                     float(scale), ns, ctypes.byref(feat), _ptr(workspace),
                                     workspace.numel(), _word(status, q_draft.device),
                                     _stream(q_draft.device))
    _check(rc, "psa_verify_extend_fwd")
    return out, lse


# ---------------------------------------------------------------- around a layer's attention

# Short forms of torch.cuda.current_device() and current_stream().cuda_stream:
# a decoding step's calls take a few microseconds on the GPU, so every
# microsecond of the host's part counts.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(name: str, device, *args):
    """Calls ``name`` on ``device``'s current stream, with ``device`` current
    (launches and tensor maps belong to the current device's context)."""
    fn = getattr(_lib or lib(), name)
    index = device.index
    if index == _current_device():
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, _raw_stream(index))
    if rc != PSA_OK:
        raise PsaError(rc, name)


def _addr(t):
    return None if t is None else t.data_ptr()


def _word(status, device):
    """Address of the status word."""
    if status is None:
        return None
    if status.dtype is not _I32 or status.device != device or status.numel() < 1:
        raise ValueError(f"status: an int32 tensor on {device} is needed")
    return status.data_ptr()


def _scratch(workspace, device):
    """A caller's workspace: dense bytes."""
    if workspace.dtype is not torch.uint8 or workspace.device != device \
            or not workspace.is_contiguous():
        raise ValueError(f"workspace: a contiguous uint8 tensor on {device} is needed")


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


# Small calls cost what these checks cost: each property of a tensor is asked
# for once (about 0.1 us), and in the order that needs the fewest.
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_WEIGHT_DTYPES = {_BF16: PSA_BF16, _F32: PSA_F32}


def _dense(t, shape, dtype, device, name: str):
    """A contiguous CUDA tensor of this shape, dtype and device."""
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor {tuple(shape)} on {device} is "
                         f"needed, not {t.dtype} {tuple(t.shape)} on {t.device}")
    return t


def _rows(t, dtype, device, name: str):
    """[T, H, d] with dense heads, tokens any distance apart: (T, H, d, token stride)."""
    shape = t.shape
    if len(shape) != 3 or t.dtype is not dtype or t.device != device or not t.is_cuda:
        raise ValueError(f"{name}: a {dtype} CUDA tensor [T, H, d] is needed on {device}")
    T, H, d = shape
    st, sh, sd = t.stride()
    if (sh != d and H > 1) or sd != 1:
        raise ValueError(f"{name}: the heads of a token have to be dense")
    return T, H, d, st if T > 1 else H * d


def _norm_rope(T: int, d: int, device, positions, cos_sin, q_weight, k_weight, eps, interleaved):
    """The psa_norm_rope of these arguments (the tensors are the caller's)."""
    pos = cs = qw = kw = None
    n_pos = rot = wdt = 0
    if cos_sin is not None:
        if positions is None:
            raise ValueError("a rotation (cos_sin) needs positions")
        shape = cos_sin.shape
        if len(shape) != 2:
            raise ValueError("cos_sin: [positions, rot_dim] is needed")
        n_pos, rot = shape
        if n_pos == 0:
            raise ValueError("cos_sin: at least one position is needed")
        pos = _dense(positions, (T,), _I32, device, "positions").data_ptr()
        cs = _dense(cos_sin, shape, _F32, device, "cos_sin").data_ptr()
    if q_weight is not None or k_weight is not None:
        dtype = (k_weight if q_weight is None else q_weight).dtype
        wdt = _WEIGHT_DTYPES.get(dtype)
        if wdt is None:
            raise ValueError("q_weight, k_weight: bf16 or fp32 is needed")
        if q_weight is not None:
            qw = _dense(q_weight, (d,), dtype, device, "q_weight").data_ptr()
        if k_weight is not None:
            if k_weight.dtype is not dtype:
                raise ValueError("q_weight and k_weight have to be of one dtype")
            kw = _dense(k_weight, (d,), dtype, device, "k_weight").data_ptr()
    return ctypes.byref(NormRope(pos, cs, n_pos, rot, bool(interleaved), qw, kw, wdt, eps))


def qk_norm_rope(q, k, positions, cos_sin, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, q_out=None, k_out=None, status=None):
    """RMS norm of every query and key head (where a weight [d] is given) and
    the position rotation, in one pass: dense (q_out, k_out).

    q [T, Hq, d] and k [T, Hkv, d], bf16 or fp32, may be slices of one
    projection's output (dense heads, any token stride of whole 16 bytes).
    positions: device int32 [T]; cos_sin: device fp32 [n_positions, rot_dim],
    rot_dim/2 cosines then rot_dim/2 sines of every position (None: no
    rotation).  Pairs are (i, i + rot_dim/2), or (2i, 2i + 1) with
    ``interleaved``; elements behind rot_dim pass through.  q_out and k_out may
    be q and k themselves (dense ones); other overlaps are refused."""
    dtype, dev = q.dtype, q.device
    code = _WEIGHT_DTYPES.get(dtype)
    _need(code is not None, "q: bf16 or fp32 is needed")
    T, Hq, d, qs = _rows(q, dtype, dev, "q")
    Tk, Hkv, dk, ks = _rows(k, dtype, dev, "k")
    _need(Tk == T and dk == d, "q and k have to agree in tokens and head size")
    how = _norm_rope(T, d, dev, positions, cos_sin, q_weight, k_weight, eps, interleaved)
    q_out = (torch.empty_like(q) if q_out is None
             else _dense(q_out, (T, Hq, d), dtype, dev, "q_out"))
    k_out = (torch.empty_like(k) if k_out is None
             else _dense(k_out, (T, Hkv, d), dtype, dev, "k_out"))
    _launch("psa_qk_norm_rope_fwd", dev, q.data_ptr(), qs, k.data_ptr(), ks, code, T, Hq, Hkv, d,
            how, q_out.data_ptr(), k_out.data_ptr(), _word(status, dev))
    return q_out, k_out


def qk_norm_rope_bwd(q, k, dq_out, dk_out, positions, cos_sin, q_weight=None, k_weight=None,
                     eps: float = 1e-6, interleaved: bool = False, dq=None, dk=None,
                     workspace=None, status=None):
    """Gradients of :func:`qk_norm_rope` for the upstream gradients dq_out and
    dk_out of its outputs: (dq, dk, dq_weight, dk_weight), the weights' in fp32
    and None where there is no weight.  dq and dk may be given as slices of
    one gradient tensor (dense heads, any token stride of whole 16 bytes), or
    be the upstream gradients or the inputs themselves."""
    dtype, dev = q.dtype, q.device
    code = _WEIGHT_DTYPES.get(dtype)
    _need(code is not None, "q: bf16 or fp32 is needed")
    T, Hq, d, qs = _rows(q, dtype, dev, "q")
    Tk, Hkv, hd, ks = _rows(k, dtype, dev, "k")
    _need(Tk == T and hd == d, "q and k have to agree in tokens and head size")
    _dense(dq_out, (T, Hq, d), dtype, dev, "dq_out")
    _dense(dk_out, (T, Hkv, d), dtype, dev, "dk_out")
    how = _norm_rope(T, d, dev, positions, cos_sin, q_weight, k_weight, eps, interleaved)
    dqs, dks = Hq * d, Hkv * d
    if dq is None:
        dq = torch.empty_like(dq_out)
    else:
        _need(dq.shape == q.shape, "dq has to be shaped as q")
        dqs = _rows(dq, dtype, dev, "dq")[3]
    if dk is None:
        dk = torch.empty_like(dk_out)
    else:
        _need(dk.shape == k.shape, "dk has to be shaped as k")
        dks = _rows(dk, dtype, dev, "dk")[3]
    dqw = None if q_weight is None else torch.empty_like(q_weight, dtype=_F32)
    dkw = None if k_weight is None else torch.empty_like(k_weight, dtype=_F32)
    if workspace is None:
        workspace = q.new_empty(lib().psa_qk_norm_rope_bwd_workspace_size(d), dtype=torch.uint8)
    else:
        _scratch(workspace, dev)
    _launch("psa_qk_norm_rope_bwd", dev, q.data_ptr(), qs, k.data_ptr(), ks, dq_out.data_ptr(),
            dk_out.data_ptr(), code, T, Hq, Hkv, d, how,
            dq.data_ptr(), dqs, dk.data_ptr(), dks, _addr(dqw), _addr(dkw), workspace.data_ptr(),
            workspace.numel(), _word(status, dev))
    return dq, dk, dqw, dkw


_E4M3_DTYPES = (torch.float8_e4m3fn, torch.uint8)


def _caches(k_cache, v_cache, k_scale, v_scale, device):
    """(tokens, heads, d, scales or None) of a pair of cache tensors."""
    sc = None
    if k_scale is not None or v_scale is not None:
        if k_scale is None or v_scale is None:
            raise ValueError("an e4m3 cache needs both k_scale and v_scale")
        sc = ctypes.byref(KvScales(k_scale, v_scale))
        ok = k_cache.dtype in _E4M3_DTYPES and v_cache.dtype in _E4M3_DTYPES
    else:
        ok = k_cache.dtype is _BF16 and v_cache.dtype is _BF16
    shape = k_cache.shape
    if (not ok or len(shape) != 3 or v_cache.shape != shape or not k_cache.is_contiguous()
            or not v_cache.is_contiguous() or not k_cache.is_cuda or k_cache.device != device
            or v_cache.device != device):
        raise ValueError(f"k_cache, v_cache: contiguous tensors [tokens, Hkv, d] on {device} are "
                         "needed, shaped alike, bf16 or (with k_scale and v_scale) e4m3 bytes")
    return (*shape, sc)


def cache_append(q, k, v, k_cache, v_cache, slots, positions=None, cos_sin=None, q_weight=None,
                 k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                 k_scale: float | None = None, v_scale: float | None = None, q_out=None,
                 status=None):
    """The serving form of :func:`qk_norm_rope`: returns the queries (dense
    bf16 [T, Hq, d]; None for q = None) and writes the tokens' keys, normed and
    rotated, and values to the cache rows ``slots`` (device int32 [T]; a
    negative slot is padding: nothing of that token is cached).  With k_scale /
    v_scale the caches hold e4m3 codes of x / scale, saturated at +-448.
    Two tokens may not share a row."""
    dev = k_cache.device
    ntok, Hkv, d, sc = _caches(k_cache, v_cache, k_scale, v_scale, dev)
    T, Hk, dk, ks = _rows(k, _BF16, dev, "k")
    Tv, Hv, dv, vs = _rows(v, _BF16, dev, "v")
    _need((Hk, dk) == (Hkv, d) and (Tv, Hv, dv) == (T, Hkv, d),
          "k and v have to agree with the caches in heads and head size")
    Hq, qs = 0, 0
    if q is not None:
        Tq, Hq, dq, qs = _rows(q, _BF16, dev, "q")
        _need(Tq == T and dq == d, "q, k and v have to agree in tokens and head size")
        q_out = (torch.empty_like(q) if q_out is None
                 else _dense(q_out, (T, Hq, d), _BF16, dev, "q_out"))
    _dense(slots, (T,), _I32, dev, "slots")
    how = _norm_rope(T, d, dev, positions, cos_sin, q_weight, k_weight, eps, interleaved)
    _launch("psa_cache_append", dev, _addr(q), qs, k.data_ptr(), ks, v.data_ptr(), vs, T, Hq, Hkv,
            d, how, k_cache.data_ptr(), v_cache.data_ptr(), ntok, slots.data_ptr(),
            sc, _addr(q_out) if q is not None else None, _word(status, dev))
    return q_out if q is not None else None


def cache_read(k_cache, v_cache, rows, k_scale: float | None = None,
               v_scale: float | None = None, k=None, v=None, status=None):
    """Cache rows ``rows`` (device int32 [n], e.g. a slice of a page table)
    as dense bf16 (k, v) [n, Hkv, d]; e4m3 caches are scaled back."""
    dev = k_cache.device
    ntok, Hkv, d, sc = _caches(k_cache, v_cache, k_scale, v_scale, dev)
    n = rows.numel()
    _dense(rows, (n,), _I32, dev, "rows")
    k = (k_cache.new_empty((n, Hkv, d), dtype=_BF16) if k is None
         else _dense(k, (n, Hkv, d), _BF16, dev, "k"))
    v = (torch.empty_like(k) if v is None
         else _dense(v, (n, Hkv, d), _BF16, dev, "v"))
    _launch("psa_cache_read", dev, k_cache.data_ptr(), v_cache.data_ptr(), ntok, rows.data_ptr(),
            n, Hkv, d, sc, k.data_ptr(), v.data_ptr(), _word(status, dev))
    return k, v


class ChunkPlan:
    """The work plan of :func:`chunk` for given lengths: the device copy of the
    lists, and what a call needs to know of them (``info``,
    ``workspace_bytes``).  One plan serves any number of calls, all layers of a
    step among them.  Its sizes are part of a launch: a captured call replays
    with its plan's lengths, other lengths need a plan and a capture of their
    own."""

    def __init__(self, info: ChunkInfo, data: torch.Tensor, workspace_bytes: int):
        if data.dtype is not _I32 or data.numel() < info.len or not data.is_contiguous():
            raise ValueError(f"a chunk plan of {info.len} contiguous int32 words is needed")
        self.info, self.data, self.workspace_bytes = info, data, workspace_bytes
        # read once: a ctypes field costs a call's time
        self._ref = ctypes.byref(info)
        self._shape = (info.Hq, info.Hkv, info.head_dim, info.n_keys)


_INT32_MAX = 2**31 - 1


def _int32s(x, name: str):
    """x as int32 values, none of them changed on the way."""
    given = np.asarray(x)
    try:
        with np.errstate(invalid="ignore"):
            out = given.astype(np.int32)
        same = (out == given).all()
    except OverflowError:
        same = False
    if not same:
        raise ValueError(f"{name}: whole numbers of 32 bits are needed")
    return out


def build_chunk_plan(qo_lens, kv_lens, Hq: int, Hkv: int, head_dim: int, window: int = 0,
                     n_ctas: int = 148):
    """(plan as a host int32 array, ChunkInfo) for ``n_ctas`` work lists."""
    ql = np.ascontiguousarray(_int32s(qo_lens, "qo_lens"))
    kl = np.ascontiguousarray(_int32s(kv_lens, "kv_lens"))
    _need(ql.ndim == 1 and ql.shape == kl.shape, "one query and one key length per request")
    # a window beyond every key is no window
    Hq, Hkv, head_dim, window, n_ctas = _int32s(
        [Hq, Hkv, head_dim, min(window, _INT32_MAX), n_ctas],
        "Hq, Hkv, head_dim, window, n_ctas").tolist()
    info = ChunkInfo()
    out = np.zeros(4096, dtype=np.int32)
    while True:
        rc = lib().psa_build_chunk_plan(_ptr(ql), _ptr(kl), len(ql), Hq, Hkv, head_dim,
                                        window, n_ctas, _ptr(out), len(out),
                                        ctypes.byref(info))
        if rc == PSA_ERR_CAPACITY and info.len > len(out):
            out = np.zeros(info.len, dtype=np.int32)
            continue
        _check(rc, "psa_build_chunk_plan")
        return out[:info.len], info


def plan_chunk(qo_lens, kv_lens, Hq: int, Hkv: int, head_dim: int, window: int = 0,
               device="cuda") -> ChunkPlan:
    """Work plan for :func:`chunk`: request b has qo_lens[b] new tokens and
    kv_lens[b] cached keys, the new tokens' own included (host lists).
    window > 0: a token sees its last ``window`` keys only, itself included."""
    device = torch.device(device)
    sms = torch.cuda.get_device_properties(device).multi_processor_count
    data, info = build_chunk_plan(qo_lens, kv_lens, Hq, Hkv, head_dim, window, sms)
    return ChunkPlan(info, torch.from_numpy(data).to(device),
                     int(lib().psa_chunk_workspace_size(ctypes.byref(info))))


def chunk(q, k_cache, v_cache, plan: ChunkPlan, scale: float, kv_indices=None,
          logit_cap: float = 0.0, k_scale: float | None = None, v_scale: float | None = None,
          out=None, lse=None, workspace=None, status=None):
    """Attention of each request's new tokens over its cached keys: O [T, Hq, d]
    bf16 and LSE [T, Hq] fp32.

    q [T, Hq, d] bf16 holds the plan's new tokens request by request (rows
    behind them are left alone); the caches [tokens, Hkv, d], bf16 or (with
    k_scale / v_scale) e4m3, hold the new tokens' keys already
    (:func:`cache_append`).  kv_indices: device int32 page table, key position
    t (flat over the requests) is cache row kv_indices[t]; without it the
    positions are the cache's first rows.  logit_cap c > 0: logits become
    c tanh(logit / c)."""
    dev = q.device
    Hq, Hkv, d, n_keys = plan._shape
    ntok, Hc, dc, sc = _caches(k_cache, v_cache, k_scale, v_scale, dev)
    T = q.shape[0]
    _dense(q, (T, Hq, d), torch.bfloat16, dev, "q")
    if Hc != Hkv or dc != d:
        raise ValueError("the caches do not fit the plan's heads")
    if plan.data.device != dev:
        raise ValueError("the plan is on another device")
    if kv_indices is not None:
        n = kv_indices.numel()
        if n < n_keys:
            raise ValueError(f"kv_indices: {n_keys} entries are needed")
        _dense(kv_indices, (n,), torch.int32, dev, "kv_indices")
    out = (torch.empty_like(q) if out is None
           else _dense(out, (T, Hq, d), torch.bfloat16, dev, "out"))
    lse = (q.new_empty((T, Hq), dtype=torch.float32) if lse is None
           else _dense(lse, (T, Hq), torch.float32, dev, "lse"))
    if workspace is None:
        workspace = q.new_empty(plan.workspace_bytes, dtype=torch.uint8)
    else:
        _scratch(workspace, dev)
    _launch("psa_chunk_fwd", dev, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), ntok,
            _addr(kv_indices), sc, out.data_ptr(), lse.data_ptr(), T, scale, logit_cap, plan._ref,
            plan.data.data_ptr(), workspace.data_ptr(), workspace.numel(), _word(status, dev))
    return out, lse
