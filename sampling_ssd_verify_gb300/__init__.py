"""GB300 (sm_103a) speculative-decoding sampling path: thin Python binding.

Every step of the path runs in the CUDA kernels of ``libssd.so`` (built from
``csrc/`` by :func:`build`); this module only marshals PyTorch tensors into
the C ABI declared in ``include/ssd.h`` (device pointers, the current CUDA
stream, workspace buffers) and raises on error codes.  There is no CPU
fallback: without the library, or without a GPU, every call raises.

Entry points (same names as the C ABI):
  verify, topf_bonus, saguaro_sample, cache_build, cache_build_guesses,
  cache_lookup, fanout, plus verify_host (host tensors in, host results out,
  copies included); around a round: process_logits (penalties, biases and
  grammar masks), page_plan (pages, slots and positions of a paged cache),
  prefix_attention (attention of rows that share prefixes), tree_attention
  (of drafts, as a tree or chain, over the cache and one another), append_path
  (accepted drafts' keys and values into the cache) and fork_rows (rows of the
  block tables continued, forked and freed).

Sources (page title, section):
  [SSD-note] "论文阅读：Speculative Speculative Decoding — 消除推测解码的最后一个顺序瓶颈"
  [SD-7.3]   "7.3 Speculative Decoding：投机采样加速"
"""

from __future__ import annotations

import ctypes
import os
import struct

import numpy as np

from . import _build

__all__ = [
    "SSDError", "build", "lib", "verify", "verify_round", "verify_host", "topf_bonus",
    "saguaro_sample", "tree_verify",
    "cache_bytes", "cache_build", "cache_build_guesses", "cache_lookup", "fanout",
    "process_logits", "page_plan", "prefix_attention", "tree_attention", "append_path",
    "fork_rows", "MASKED_LOGIT",
    "DEV_BAD_TOKEN", "DEV_ZERO_RESIDUAL", "DEV_TIMEOUT", "DEV_TABLE_FULL", "DEV_DUPLICATE_KEY",
    "DEV_BAD_TEMPERATURE", "DEV_BAD_FANOUT", "DEV_BAD_PENALTY", "DEV_BAD_LENGTH",
    "DEV_NO_PAGES", "DEV_BAD_PAGE",
]

DEV_BAD_TOKEN = 0x1
DEV_ZERO_RESIDUAL = 0x2
DEV_TIMEOUT = 0x4
DEV_TABLE_FULL = 0x8
DEV_DUPLICATE_KEY = 0x10
DEV_BAD_TEMPERATURE = 0x20
DEV_BAD_FANOUT = 0x40
DEV_BAD_PENALTY = 0x80
DEV_BAD_LENGTH = 0x100
DEV_NO_PAGES = 0x200
DEV_BAD_PAGE = 0x400

MASKED_LOGIT = -1048576.0  # what a token outside the grammar gets: -2^20

SSD_BF16, SSD_F32, SSD_F16 = 0, 1, 2
_ERR_WORKSPACE = 5
_lib = None


class SSDError(RuntimeError):
    pass


class _Logits(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("pad_", ctypes.c_int32),
                ("row_stride", ctypes.c_int64)]


class _LogitRules(ctypes.Structure):
    _fields_ = [("history", ctypes.c_void_p), ("history_stride", ctypes.c_int64),
                ("history_max", ctypes.c_int32), ("n_bias", ctypes.c_int32),
                ("history_len", ctypes.c_void_p), ("prompt_len", ctypes.c_void_p),
                ("draft_tokens", ctypes.c_void_p), ("draft_stride", ctypes.c_int64),
                ("parent", ctypes.c_char_p), ("repetition", ctypes.c_void_p),
                ("frequency", ctypes.c_void_p), ("presence", ctypes.c_void_p),
                ("bias_ids", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("mask", ctypes.c_void_p), ("mask_seq_stride", ctypes.c_int64),
                ("mask_row_stride", ctypes.c_int64), ("fill", ctypes.c_float),
                ("pad_", ctypes.c_int32)]


class _Paged(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _Attention(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("R", ctypes.c_int32), ("Hq", ctypes.c_int32),
                ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32), ("G", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("q_row_stride", ctypes.c_int64),
                ("q_head_stride", ctypes.c_int64), ("k", _Paged), ("v", _Paged),
                ("prefix_tables", ctypes.c_void_p), ("prefix_len", ctypes.c_void_p),
                ("group_off", ctypes.c_void_p), ("tables", ctypes.c_void_p),
                ("lens", ctypes.c_void_p), ("prefix_table_stride", ctypes.c_int64),
                ("table_stride", ctypes.c_int64), ("prefix_cols", ctypes.c_int32),
                ("cols", ctypes.c_int32), ("out", ctypes.c_void_p),
                ("out_row_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
                ("lse", ctypes.c_void_p), ("scale", ctypes.c_float), ("pad_", ctypes.c_int32)]


_vp = ctypes.c_void_p
_i = ctypes.c_int
_sz = ctypes.c_size_t
_LP = ctypes.POINTER(_Logits)

_SIGS = {
    "ssd_status_string": ([_i], ctypes.c_char_p),
    "ssd_version": ([], _i),
    "ssd_verify_workspace_size": ([_i, _i, _i, _i], _sz),
    "ssd_verify_skipped_bytes": ([_vp, _sz, _i, _i, _i, _i, _i, _vp, _vp], _i),
    "ssd_verify": ([_LP, _LP, _i, _i, _i, _i, ctypes.c_float, _vp, _vp, ctypes.c_uint32, _vp,
                    ctypes.c_float, _vp, _vp, _vp, _vp, _vp, _i, _vp, _sz, _vp, _vp], _i),
    "ssd_verify_ck": ([_LP, _LP, _i, _i, _i, _i, ctypes.c_float, _vp, _vp, ctypes.c_uint32, _vp,
                       _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _sz, _vp, _vp], _i),
    "ssd_verify_ex": ([_LP, _LP, _i, _i, _i, _i, _vp, _vp, _vp, ctypes.c_uint32, _vp,
                       _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _sz, _vp, _vp], _i),
    "ssd_verify_round": ([_LP, _LP, _i, _i, _i, _i, ctypes.c_float, _vp, _vp, ctypes.c_uint32,
                          _vp, ctypes.c_float, _vp, _vp, _vp, _vp, _vp, _i, _vp, _sz, _vp, _vp,
                          _vp, _sz, _vp, _vp], _i),
    "ssd_topf_workspace_size": ([_i, _i, _i], _sz),
    "ssd_topf_bonus": ([_LP, _i, _i, _i, ctypes.c_float, _vp, _i, _vp, _i, _vp, _vp, _vp, _sz,
                        _vp, _vp], _i),
    "ssd_saguaro_workspace_size": ([_i, _i], _sz),
    "ssd_saguaro_sample": ([_LP, _i, _i, ctypes.c_float, ctypes.c_float, _vp, _i, _vp, _i,
                            ctypes.c_uint32, _vp, _vp, _vp, _vp, _sz, _vp, _vp], _i),
    "ssd_tree_workspace_size": ([_i, _i, _i], _sz),
    "ssd_tree_verify": ([_LP, _LP, _i, _i, _i, ctypes.c_float, _vp, _vp, _vp, ctypes.c_uint32,
                         _vp, _vp, _i, _vp, _vp, _vp, _sz, _vp, _vp], _i),
    "ssd_cache_bytes": ([_i], _sz),
    "ssd_cache_build": ([_vp, _sz, _vp, _vp, _vp, _vp, _i, _vp, _vp], _i),
    "ssd_cache_build_guesses": ([_vp, _sz, _vp, _i, _i, _i, _vp, _vp], _i),
    "ssd_cache_lookup": ([_vp, _sz, _vp, _vp, _i, _vp, _vp, _vp], _i),
    "ssd_fanout": ([_i, _i, ctypes.c_double, ctypes.c_double, _vp], _i),
    "ssd_process_logits": ([_LP, _LP, _i, _i, _i, ctypes.POINTER(_LogitRules), _vp, _vp, _vp],
                           _i),
    "ssd_page_plan": ([_vp, _vp, _vp, _i, _vp, ctypes.c_int64, _i, _vp, _i, _vp, _i, _i] +
                      [_vp] * 10, _i),
    "ssd_prefix_attention_workspace_size": ([ctypes.POINTER(_Attention)], _sz),
    "ssd_prefix_attention": ([ctypes.POINTER(_Attention), _vp, _sz, _vp, _vp], _i),
    "ssd_tree_attention_workspace_size": ([_vp], _sz),
    "ssd_tree_attention": ([_vp, _vp, _sz, _vp, _vp], _i),
    "ssd_append_path": ([_vp, _vp, _vp], _i),
    "ssd_fork_rows_workspace_size": ([_vp], _sz),
    "ssd_fork_rows": ([_vp, _vp, _sz, _vp, _vp], _i),
}


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libssd.so for sm_103a (see ``_build.py``)."""
    return _build.build(force=force, verbose=verbose)


def lib_path() -> str:
    return _build.LIB_PATH


def lib():
    """Load libssd.so (it must have been built; nothing falls back)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_build.LIB_PATH):
            raise SSDError(f"{_build.LIB_PATH} is missing: build it with "
                           "sampling_ssd_verify_gb300.build()")
        L = ctypes.CDLL(_build.LIB_PATH)
        for name, (args, res) in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _check(status: int, what: str):
    if status != 0:
        msg = lib().ssd_status_string(status).decode()
        raise SSDError(f"{what}: {msg} (status {status})")


# ---- tensor marshalling ---------------------------------------------------------------
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dev_ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise SSDError("expected a CUDA tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _on_current(dev):
    """The library launches on the current GPU: tensors of another are refused."""
    now = _torch()._C._cuda_getDevice()
    if dev != now:
        raise SSDError(f"the tensors are on cuda:{dev}, the current GPU is cuda:{now}: make the "
                       f"call within torch.cuda.device({dev})")


def _logits(t, nrows_inner=None):
    """Describe a [..., R, V] tensor whose rows are evenly spaced."""
    torch = _torch()
    if not t.is_cuda:
        raise SSDError("logits must be on the GPU")
    _on_current(t.get_device())
    if t.dtype == torch.bfloat16:
        dt = SSD_BF16
    elif t.dtype == torch.float32:
        dt = SSD_F32
    else:
        raise SSDError(f"unsupported logits dtype {t.dtype}")
    if t.stride(-1) != 1:
        raise SSDError("logit rows must be contiguous over the vocabulary")
    rs = t.stride(-2) if t.dim() >= 2 else t.shape[-1]
    for d in range(t.dim() - 2):
        if t.stride(d) != rs * int(np.prod(t.shape[d + 1:-1])):
            raise SSDError("logit rows must be evenly spaced")
    return _Logits(ctypes.c_void_p(t.data_ptr()), dt, 0, rs)


def _workspace(nbytes, device):
    torch = _torch()
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _i32(t):
    torch = _torch()
    if t.dtype != torch.int32 or not t.is_contiguous():
        raise SSDError("expected a contiguous int32 tensor")
    return t


def _u64_seeds(seeds, device):
    torch = _torch()
    if isinstance(seeds, np.ndarray):
        seeds = torch.from_numpy(seeds.astype(np.uint64).view(np.int64)).to(device)
    if seeds.dtype not in (torch.int64, getattr(torch, "uint64", torch.int64)):
        raise SSDError("seeds must be 64-bit")
    return seeds.contiguous()


# ---- entry points ------------------------------------------------------------------------
def verify(target, draft, draft_tokens, seeds, round_, fanout=None, C=1.0, T=1.0,
           guesses=True, guess_q=True, resid_mass=True, workspace=None, dev_status=None,
           stream=None, out=None):
    """ssd_verify on device tensors.

    target [B, K+1, V], draft [B, Kq, V] (bf16 or fp32, same dtype),
    draft_tokens int32 [B, K], seeds 64-bit [B], fanout: sequence of Kq ints.
    C: the Saguaro factor, or a sequence of K factors, one per draft position
    (ssd_verify_ck).  T: the temperature (0: greedy), or one per sequence --
    a device float32 tensor [B] or anything numpy reads (ssd_verify_ex).
    Returns a dict of device tensors: accept_len, bonus, resid_mass, guesses,
    guess_q (the optional ones only when requested).
    """
    torch = _torch()
    B, K1, V = target.shape
    K = K1 - 1
    Kq = draft.shape[-2]
    dev = target.device
    F = np.zeros(Kq, dtype=np.int32) if fanout is None else np.ascontiguousarray(fanout,
                                                                                  dtype=np.int32)
    if len(F) != Kq:
        raise SSDError("fanout must have Kq entries")
    Fmax = max(1, int(F.max()) if len(F) else 1)
    o = out if out is not None else {}
    if "accept_len" not in o:
        o["accept_len"] = torch.empty(B, dtype=torch.int32, device=dev)
        o["bonus"] = torch.empty(B, dtype=torch.int32, device=dev)
        if resid_mass:
            o["resid_mass"] = torch.empty(B, dtype=torch.float32, device=dev)
        if guesses:
            o["guesses"] = torch.empty((B, Kq, Fmax), dtype=torch.int32, device=dev)
            if guess_q:
                o["guess_q"] = torch.empty((B, Kq, Fmax), dtype=torch.float32, device=dev)
    L = lib()
    wsb = L.ssd_verify_workspace_size(B, K, Kq, V)
    if wsb == 0:
        raise SSDError("invalid verify shape")
    ws = workspace if workspace is not None else _workspace(wsb, dev)
    tl, dl = _logits(target), _logits(draft)
    if np.ndim(T) > 0:
        Tr = T if hasattr(T, "is_cuda") else torch.as_tensor(np.asarray(T, dtype=np.float32),
                                                              device=dev)
        if Tr.shape != (B,) or Tr.dtype != torch.float32 or not Tr.is_cuda:
            raise SSDError("per-sequence T must be float32 [B] on the device")
        Tr = Tr.contiguous()
        Cv = None if np.ndim(C) == 0 and float(C) == 1.0 else \
            np.ascontiguousarray(np.broadcast_to(np.asarray(C, dtype=np.float32), (K,)))
        st = L.ssd_verify_ex(ctypes.byref(tl), ctypes.byref(dl), B, K, Kq, V, _dev_ptr(Tr),
                             _dev_ptr(_i32(draft_tokens)), _dev_ptr(_u64_seeds(seeds, dev)),
                             int(round_) & 0xFFFFFFFF, F.ctypes.data_as(ctypes.c_void_p),
                             None if Cv is None else Cv.ctypes.data_as(ctypes.c_void_p),
                             _dev_ptr(o["accept_len"]), _dev_ptr(o["bonus"]),
                             _dev_ptr(o.get("resid_mass")), _dev_ptr(o.get("guesses")),
                             _dev_ptr(o.get("guess_q")), Fmax, _dev_ptr(ws), ws.numel(),
                             _dev_ptr(dev_status), _stream(stream))
        _check(st, "ssd_verify_ex")
        return o
    if np.ndim(C) == 0:
        fn, c_arg, name = L.ssd_verify, float(C), "ssd_verify"
    else:
        Cv = np.ascontiguousarray(C, dtype=np.float32)
        if Cv.shape != (K,):
            raise SSDError("C must be a scalar or have one entry per draft position")
        fn, c_arg, name = L.ssd_verify_ck, Cv.ctypes.data_as(ctypes.c_void_p), "ssd_verify_ck"
    st = fn(ctypes.byref(tl), ctypes.byref(dl), B, K, Kq, V, float(T),
            _dev_ptr(_i32(draft_tokens)), _dev_ptr(_u64_seeds(seeds, dev)),
            int(round_) & 0xFFFFFFFF, F.ctypes.data_as(ctypes.c_void_p), c_arg,
            _dev_ptr(o["accept_len"]), _dev_ptr(o["bonus"]),
            _dev_ptr(o.get("resid_mass")), _dev_ptr(o.get("guesses")),
            _dev_ptr(o.get("guess_q")), Fmax, _dev_ptr(ws), ws.numel(),
            _dev_ptr(dev_status), _stream(stream))
    _check(st, name)
    return o


def verify_round(target, draft, draft_tokens, seeds, round_, fanout, C=1.0, T=1.0,
                 guess_q=True, resid_mass=True, table=None, workspace=None, dev_status=None,
                 stream=None, out=None):
    """ssd_verify_round: verify, the round's outcome cache and its lookup in
    one launch.  Returns verify's outputs (guesses always) plus ``branch``
    [B] and ``all_hit`` [1] (device tensors) and the ``table`` used."""
    torch = _torch()
    B, K1, V = target.shape
    K = K1 - 1
    Kq = draft.shape[-2]
    dev = target.device
    F = np.ascontiguousarray(fanout, dtype=np.int32)
    if len(F) != Kq:
        raise SSDError("fanout must have Kq entries")
    Fmax = max(1, int(F.max()))
    o = out if out is not None else {}
    if "accept_len" not in o:
        o["accept_len"] = torch.empty(B, dtype=torch.int32, device=dev)
        o["bonus"] = torch.empty(B, dtype=torch.int32, device=dev)
        if resid_mass:
            o["resid_mass"] = torch.empty(B, dtype=torch.float32, device=dev)
        o["guesses"] = torch.empty((B, Kq, Fmax), dtype=torch.int32, device=dev)
        if guess_q:
            o["guess_q"] = torch.empty((B, Kq, Fmax), dtype=torch.float32, device=dev)
        o["branch"] = torch.empty(B, dtype=torch.int32, device=dev)
        o["all_hit"] = torch.empty(1, dtype=torch.int32, device=dev)
    if table is None:
        table = o.get("table")
    if table is None:
        table = torch.empty(cache_bytes(B * Kq * Fmax), dtype=torch.uint8, device=dev)
    o["table"] = table
    L = lib()
    wsb = L.ssd_verify_workspace_size(B, K, Kq, V)
    if wsb == 0:
        raise SSDError("invalid verify shape")
    ws = workspace if workspace is not None else _workspace(wsb, dev)
    tl, dl = _logits(target), _logits(draft)
    st = L.ssd_verify_round(ctypes.byref(tl), ctypes.byref(dl), B, K, Kq, V, float(T),
                            _dev_ptr(_i32(draft_tokens)), _dev_ptr(_u64_seeds(seeds, dev)),
                            int(round_) & 0xFFFFFFFF, F.ctypes.data_as(ctypes.c_void_p), float(C),
                            _dev_ptr(o["accept_len"]), _dev_ptr(o["bonus"]),
                            _dev_ptr(o.get("resid_mass")), _dev_ptr(o["guesses"]),
                            _dev_ptr(o.get("guess_q")), Fmax, _dev_ptr(table), table.numel(),
                            _dev_ptr(o["branch"]), _dev_ptr(o["all_hit"]), _dev_ptr(ws), ws.numel(),
                            _dev_ptr(dev_status), _stream(stream))
    _check(st, "ssd_verify_round")
    return o


def verify_skipped_bytes(workspace, target, K, Kq, stream=None):
    """ssd_verify_skipped_bytes: the bytes of target rows the last verify
    call on `workspace` (target [B, K+1, V]) did not read, as a Python int
    (synchronises the stream)."""
    torch = _torch()
    B, V = target.shape[0], target.shape[-1]
    dt = SSD_BF16 if target.dtype == torch.bfloat16 else SSD_F32
    out = torch.zeros(1, dtype=torch.int64, device=workspace.device)
    st = lib().ssd_verify_skipped_bytes(_dev_ptr(workspace), workspace.numel(), B, K, Kq, V, dt,
                                        _dev_ptr(out), _stream(stream))
    _check(st, "ssd_verify_skipped_bytes")
    return int(out.item())


def verify_host(target, draft, draft_tokens, seeds, round_, fanout=None, C=1.0, T=1.0,
                device="cuda", guesses=True, workspace=None, dev_buffers=None):
    """End-to-end call with HOST tensors: copies the inputs to the GPU, runs
    ssd_verify and copies the results back (pinned host memory makes the
    copies asynchronous).  Returns a dict of CPU tensors."""
    torch = _torch()
    db = dev_buffers if dev_buffers is not None else {}
    for name, t in (("target", target), ("draft", draft), ("tokens", draft_tokens),
                    ("seeds", seeds)):
        if name not in db:
            db[name] = torch.empty(t.shape, dtype=t.dtype, device=device)
        db[name].copy_(t, non_blocking=True)
    o = verify(db["target"], db["draft"], db["tokens"], db["seeds"], round_, fanout, C, T,
               guesses=guesses, workspace=workspace, out=db.get("out"))
    db["out"] = o
    host = {k: torch.empty(v.shape, dtype=v.dtype, pin_memory=True) for k, v in o.items()}
    for k, v in o.items():
        host[k].copy_(v, non_blocking=True)
    torch.cuda.current_stream().synchronize()
    return host


def topf_bonus(draft, fanout, T=1.0, draft_tokens=None, K=None, Fmax=None, guess_q=True,
               workspace=None, dev_status=None, stream=None):
    """ssd_topf_bonus: guesses [B, Kq, Fmax] (+ guess_q) for draft [B, Kq, V]."""
    torch = _torch()
    B, Kq, V = draft.shape
    dev = draft.device
    F = np.ascontiguousarray(fanout, dtype=np.int32)
    Fmax = max(1, int(F.max())) if Fmax is None else int(Fmax)
    g = torch.empty((B, Kq, Fmax), dtype=torch.int32, device=dev)
    gq = torch.empty((B, Kq, Fmax), dtype=torch.float32, device=dev) if guess_q else None
    L = lib()
    ws = workspace if workspace is not None else _workspace(L.ssd_topf_workspace_size(B, Kq, V),
                                                            dev)
    Kt = 0 if draft_tokens is None else (draft_tokens.shape[-1] if K is None else int(K))
    dl = _logits(draft)
    st = L.ssd_topf_bonus(ctypes.byref(dl), B, Kq, V, float(T),
                          _dev_ptr(None if draft_tokens is None else _i32(draft_tokens)), Kt,
                          F.ctypes.data_as(ctypes.c_void_p), Fmax, _dev_ptr(g), _dev_ptr(gq),
                          _dev_ptr(ws), ws.numel(), _dev_ptr(dev_status), _stream(stream))
    _check(st, "ssd_topf_bonus")
    return {"guesses": g, "guess_q": gq}


def saguaro_sample(rows, T, C, F, seeds, j, round_, guesses=True, qprime=True, workspace=None,
                   dev_status=None, stream=None, out=None, Fmax=None):
    """ssd_saguaro_sample over branch rows [R, V]: token, qprime, guesses.

    F: one fan-out for every row (an int), or one per row -- a device int32
    tensor [R] (then Fmax, the largest, must be given) or anything numpy
    reads (uploaded here).  guesses are [R, Fmax], -1 padded."""
    torch = _torch()
    R, V = rows.shape[-2], rows.shape[-1]
    dev = rows.device
    F_row = None
    if np.ndim(F) == 0 and not hasattr(F, "is_cuda"):
        Fm = int(F)
    elif hasattr(F, "is_cuda"):
        if Fmax is None:
            raise SSDError("a device F tensor needs Fmax")
        F_row, Fm = _i32(F), int(Fmax)
    else:
        Fa = np.ascontiguousarray(F, dtype=np.int32)
        if Fa.shape != (R,):
            raise SSDError("per-row F must have R entries")
        Fm = int(Fa.max()) if Fmax is None else int(Fmax)
        F_row = torch.from_numpy(Fa).to(dev)
    if F_row is not None and F_row.shape != (R,):
        raise SSDError("per-row F must have R entries")
    o = out if out is not None else {}
    if "token" not in o:
        o["token"] = torch.empty(R, dtype=torch.int32, device=dev)
        if qprime:
            o["qprime"] = torch.empty(R, dtype=torch.float32, device=dev)
        if guesses and Fm > 0:
            o["guesses"] = torch.empty((R, Fm), dtype=torch.int32, device=dev)
    L = lib()
    ws = workspace if workspace is not None else _workspace(L.ssd_saguaro_workspace_size(R, V),
                                                            dev)
    rl = _logits(rows)
    st = L.ssd_saguaro_sample(ctypes.byref(rl), R, V, float(T), float(C), _dev_ptr(F_row), Fm,
                              _dev_ptr(_u64_seeds(seeds, dev)), int(j),
                              int(round_) & 0xFFFFFFFF, _dev_ptr(o["token"]),
                              _dev_ptr(o.get("qprime")), _dev_ptr(o.get("guesses")),
                              _dev_ptr(ws), ws.numel(), _dev_ptr(dev_status), _stream(stream))
    _check(st, "ssd_saguaro_sample")
    return o


def tree_verify(target, draft, parent, tokens, seeds, round_, T=1.0, workspace=None,
                dev_status=None, stream=None, out=None):
    """ssd_tree_verify: target, draft [B, N, V] (row u of a tree: p_u / q_u at
    node u), parent: N ints (parent[0] = -1, parent[u] < u), tokens int32
    [B, N] on the device.  Returns accept_len [B], path [B, depth], bonus
    [B] and resid_mass [B] (device tensors)."""
    torch = _torch()
    B, N, V = target.shape
    dev = target.device
    par = np.ascontiguousarray(parent, dtype=np.int32)
    if par.shape != (N,):
        raise SSDError("parent must have N entries")
    depth = np.zeros(N, dtype=np.int64)
    for u in range(1, N):
        if not 0 <= par[u] < u:
            raise SSDError("parent[u] must lie in [0, u)")
        depth[u] = depth[par[u]] + 1
    Dmax = max(1, int(depth.max()))
    o = out if out is not None else {}
    if "accept_len" not in o:
        o["accept_len"] = torch.empty(B, dtype=torch.int32, device=dev)
        o["path"] = torch.empty((B, Dmax), dtype=torch.int32, device=dev)
        o["bonus"] = torch.empty(B, dtype=torch.int32, device=dev)
        o["resid_mass"] = torch.empty(B, dtype=torch.float32, device=dev)
    L = lib()
    wsb = L.ssd_tree_workspace_size(B, N, V)
    if wsb == 0:
        raise SSDError("invalid tree shape")
    ws = workspace if workspace is not None else _workspace(wsb, dev)
    tl, dl = _logits(target), _logits(draft)
    st = L.ssd_tree_verify(ctypes.byref(tl), ctypes.byref(dl), B, N, V, float(T),
                           par.ctypes.data_as(ctypes.c_void_p), _dev_ptr(_i32(tokens)),
                           _dev_ptr(_u64_seeds(seeds, dev)), int(round_) & 0xFFFFFFFF,
                           _dev_ptr(o["accept_len"]), _dev_ptr(o["path"]), Dmax,
                           _dev_ptr(o["bonus"]), _dev_ptr(o["resid_mass"]), _dev_ptr(ws),
                           ws.numel(), _dev_ptr(dev_status), _stream(stream))
    _check(st, "ssd_tree_verify")
    return o


def cache_bytes(n_keys: int) -> int:
    return int(lib().ssd_cache_bytes(int(n_keys)))


def cache_build(row, k, t, branch, table=None, dev_status=None, stream=None):
    torch = _torch()
    n = row.numel()
    if row.is_cuda:
        _on_current(row.get_device())
    if table is None:
        table = torch.empty(cache_bytes(n), dtype=torch.uint8, device=row.device)
    st = lib().ssd_cache_build(_dev_ptr(table), table.numel(), _dev_ptr(_i32(row)),
                               _dev_ptr(_i32(k)), _dev_ptr(_i32(t)), _dev_ptr(_i32(branch)), n,
                               _dev_ptr(dev_status), _stream(stream))
    _check(st, "ssd_cache_build")
    return table


def cache_build_guesses(guesses, table=None, dev_status=None, stream=None):
    torch = _torch()
    B, Kq, Fmax = guesses.shape
    if guesses.is_cuda:
        _on_current(guesses.get_device())
    if table is None:
        table = torch.empty(cache_bytes(B * Kq * Fmax), dtype=torch.uint8, device=guesses.device)
    st = lib().ssd_cache_build_guesses(_dev_ptr(table), table.numel(), _dev_ptr(_i32(guesses)),
                                       B, Kq, Fmax, _dev_ptr(dev_status), _stream(stream))
    _check(st, "ssd_cache_build_guesses")
    return table


def cache_lookup(table, accept_len, bonus, out=None, stream=None):
    torch = _torch()
    B = accept_len.numel()
    if accept_len.is_cuda:
        _on_current(accept_len.get_device())
    o = out if out is not None else {
        "branch": torch.empty(B, dtype=torch.int32, device=accept_len.device),
        "all_hit": torch.empty(1, dtype=torch.int32, device=accept_len.device)}
    st = lib().ssd_cache_lookup(_dev_ptr(table), table.numel(), _dev_ptr(_i32(accept_len)),
                                _dev_ptr(_i32(bonus)), B, _dev_ptr(o["branch"]),
                                _dev_ptr(o["all_hit"]), _stream(stream))
    _check(st, "ssd_cache_lookup")
    return o


def fanout(K: int, budget: int, a: float = 0.7, r: float = 1.0) -> np.ndarray:
    """Geometric fan-out F_0..F_K (host helper of the library)."""
    F = np.zeros(K + 1, dtype=np.int32)
    _check(lib().ssd_fanout(int(K), int(budget), float(a), float(r),
                            F.ctypes.data_as(ctypes.c_void_p)), "ssd_fanout")
    return F


# ---- around a round ---------------------------------------------------------------------
# Calls of a few microseconds on the device: their checks are kept few and
# cheap (a tensor's type, device, shape and layout, each asked for once).
def _tensor(t, name, dtype, shape, dev):
    """Address of a contiguous tensor of that type and shape on GPU `dev`."""
    if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    raise SSDError(f"{name}: expected a contiguous {dtype} tensor {tuple(shape)} on cuda:{dev}, "
                   f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _rows2d(t, name, rows, i32, dev):
    """Address, row stride and columns of an int32 [rows, n] tensor with
    contiguous rows that do not overlap."""
    shape = t.shape
    if t.dtype is not i32 or t.get_device() != dev or len(shape) != 2 or shape[0] != rows:
        raise SSDError(f"{name}: expected an int32 tensor of {rows} rows on cuda:{dev}, "
                       f"got {t.dtype} {tuple(shape)} on {t.device}")
    n = shape[1]
    if t.is_contiguous():
        return t.data_ptr(), n, n
    if (n > 1 and t.stride(1) != 1) or (rows > 1 and t.stride(0) < n):
        raise SSDError(f"{name}: rows must be contiguous and must not overlap")
    return t.data_ptr(), max(t.stride(0), n), n


def _rows3d(t):
    """ssd_logits of a [B, N, V] tensor whose rows are evenly spaced."""
    return _Logits(t.data_ptr(), SSD_BF16 if t.element_size() == 2 else SSD_F32, 0,
                   t.shape[2]) if t.is_contiguous() else _logits(t)


def _use_stream(stream, dev, tensors):
    """The stream's handle; memory taken from the current stream's pool is
    not given out again before `stream` is done with it."""
    torch = _torch()
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream != torch.cuda.current_stream(dev):
        for t in tensors:
            t.record_stream(stream)
    return stream.cuda_stream


def _without(o, name):
    """The call's results: `o`, but for an earlier call's that this one was not asked for."""
    return {k: v for k, v in o.items() if k != name}


def process_logits(logits, history=None, history_len=None, prompt_len=None, draft_tokens=None,
                   parent=None, repetition=None, presence=None, frequency=None, bias_ids=None,
                   bias=None, mask=None, fill=MASKED_LOGIT, allowed=False, dev_status=None,
                   stream=None, out=None):
    """ssd_process_logits: penalties, biases and a grammar on logits [B, N, V].

    history int32 [B, H] with history_len [B] (its first prompt_len [B] tokens
    count for the repetition penalty alone).  draft_tokens int32 [B, N-1], or
    [B, N] with an entry for node 0 that is not looked at; parent: N ints (a
    chain when None).  repetition, presence, frequency: float32 [B].  bias_ids
    int32 [B, n] (negative: padding), bias float32 [B, n].  mask int32 words
    [B or 1, N or 1, ceil(V / 32)], bit v % 32 of word v / 32 set where token v
    is allowed; others get `fill`.
    Returns a dict: ``logits`` [B, N, V], new unless `out` has it (it may be
    the input itself), and with allowed=True ``allowed`` int32 [B, N], the
    number of tokens that the mask allows."""
    torch = _torch()
    i32, f32 = torch.int32, torch.float32
    shape = logits.shape
    dev = logits.get_device()
    if len(shape) != 3 or dev < 0 or logits.dtype not in (torch.bfloat16, f32):
        raise SSDError("expected bfloat16 or float32 logits [B, N, V] on the GPU")
    _on_current(dev)
    B, N, V = shape
    o = out if out is not None else {}
    z = o.get("logits")
    if z is None:
        z = o["logits"] = torch.empty(shape, dtype=logits.dtype, device=logits.device)
    elif z.shape != shape or z.dtype is not logits.dtype or z.get_device() != dev:
        raise SSDError("out logits must have the input's shape, type and device")
    count = None
    if allowed:
        if "allowed" not in o:
            o["allowed"] = torch.empty((B, N), dtype=i32, device=logits.device)
        count = _tensor(o["allowed"], "allowed", i32, (B, N), dev)
    row = (B,)
    h = h_stride = h_max = h_len = p_len = 0
    if history is not None:
        if history_len is None:
            raise SSDError("history needs history_len")
        h, h_stride, h_max = _rows2d(history, "history", B, i32, dev)
        h_len = _tensor(history_len, "history_len", i32, row, dev)
        if prompt_len is not None:
            p_len = _tensor(prompt_len, "prompt_len", i32, row, dev)
    drafts = d_stride = 0
    if draft_tokens is not None and N > 1:
        drafts, d_stride, n = _rows2d(draft_tokens, "draft_tokens", B, i32, dev)
        if n != N - 1 and n != N:
            raise SSDError("draft_tokens must have N - 1 or N columns")
        drafts += 4 * (n - N + 1)
    if parent is not None:
        if len(parent) != N:
            raise SSDError("parent must have N entries")
        parent = np.asarray(parent, dtype=np.int32).tobytes()
    rep = 0 if repetition is None else _tensor(repetition, "repetition", f32, row, dev)
    freq = 0 if frequency is None else _tensor(frequency, "frequency", f32, row, dev)
    pres = 0 if presence is None else _tensor(presence, "presence", f32, row, dev)
    n_bias = ids = values = 0
    if bias_ids is not None and bias is not None:
        ids, stride, n_bias = _rows2d(bias_ids, "bias_ids", B, i32, dev)
        if stride != n_bias and B > 1:
            raise SSDError("bias_ids must be contiguous")
        values = _tensor(bias, "bias", f32, (B, n_bias), dev)
    elif bias_ids is not bias:
        raise SSDError("bias_ids and bias go together")
    m = m_seq = m_row = 0
    if mask is not None:
        W = (V + 31) // 32
        ms = mask.shape
        if mask.dtype is not i32 or mask.get_device() != dev or len(ms) != 3 or ms[2] != W or \
                ms[0] not in (1, B) or ms[1] not in (1, N) or (W > 1 and mask.stride(2) != 1):
            raise SSDError("mask: expected int32 words [B or 1, N or 1, ceil(V / 32)]")
        m, strides = mask.data_ptr(), mask.stride()
        m_seq = strides[0] if ms[0] > 1 else 0
        m_row = strides[1] if ms[1] > 1 else 0
    r = _LogitRules(h, h_stride, h_max, n_bias, h_len, p_len, drafts, d_stride, parent, rep, freq,
                    pres, ids, values, m, m_seq, m_row, fill, 0)
    st = lib().ssd_process_logits(_rows3d(logits), _rows3d(z), B, N, V, r, count,
                                  _dev_ptr(dev_status), _use_stream(stream, dev, o.values()))
    if st:
        _check(st, "ssd_process_logits")
    return o if allowed or "allowed" not in o else _without(o, "allowed")


_PLAN = ("positions", "owner", "cu", "kv_len", "held", "served", "free_count")
_PLAN_NAMES = {"slots", *_PLAN}


def _plan_views(torch, B, T, device):
    """page_plan's outputs: the slots, and the others in one buffer, each on a
    64-byte boundary."""
    counts = (T, T, B + 1, B, B, B, 1)
    base = torch.empty(sum(n + 15 & ~15 for n in counts), dtype=torch.int32, device=device)
    views, at = {"slots": torch.empty(T, dtype=torch.int64, device=device)}, 0
    for name, n in zip(_PLAN, counts):
        views[name] = base[at:at + n]
        at += n + 15 & ~15
    return views


def _plan_pointers(o, B, T, i32, dev):
    """Addresses of page_plan's outputs but the slots: views of one buffer, one
    after the other.  That they are is told by the buffer's memory (a view made
    in inference mode knows no base)."""
    cu = o.get("cu")
    if cu is None or "slots" not in o:
        raise SSDError("out: expected all outputs of an earlier call")
    if cu.dtype is not i32 or cu.get_device() != dev or cu.numel() != B + 1:
        raise SSDError("out: expected the dict of an earlier call with these sizes")
    memory = cu.untyped_storage()
    first = at = memory.data_ptr()
    ptrs = []
    for name, n in zip(_PLAN, (T, T, B + 1, B, B, B, 1)):
        if name not in o or n and o[name].data_ptr() != at:
            raise SSDError(f"out: {name} is not that of an earlier call with these sizes")
        ptrs.append(at)
        at += (n + 15 & ~15) * 4
    if at - first > memory.nbytes():
        raise SSDError("out: expected the dict of an earlier call with these sizes")
    return ptrs


def page_plan(lens, new, held, tables, free_pages, free_count, page_size, max_rows,
              dev_status=None, stream=None, out=None):
    """ssd_page_plan: the pages of a paged key/value cache after a round, and
    where the next tokens go.

    lens, new, held int32 [B]: tokens in the cache, tokens to append, pages
    held; tables int32 [B, W] and the stack free_pages int32 [n] with
    free_count int32 [1] (entries of both are written, free_count is not).
    Returns a dict of device tensors: slots int64, positions and owner int32
    [max_rows]; cu int32 [B + 1]; kv_len, held, served int32 [B]; free_count
    int32 [1].  `out`: the dict of an earlier call, to use its tensors again
    (not while one of them is this call's input).
    What it gives back is free whoever else holds it: rows with pages that they
    share end through fork_rows, and do not fall below the tokens shared."""
    torch = _torch()
    i32 = torch.int32
    dev = lens.get_device()
    if dev < 0 or lens.dim() != 1:
        raise SSDError("expected lengths [B] on the GPU")
    _on_current(dev)
    B, T = lens.shape[0], int(max_rows)
    if T < 0:
        raise SSDError("max_rows must not be negative")
    row, one = (B,), (1,)
    o = out if out is not None else {}
    if "cu" not in o and _PLAN_NAMES.isdisjoint(o):
        o.update(_plan_views(torch, B, T, lens.device))
    ptrs = _plan_pointers(o, B, T, i32, dev)
    table, stride, cols = _rows2d(tables, "tables", B, i32, dev)
    st = lib().ssd_page_plan(
        _tensor(lens, "lens", i32, row, dev), _tensor(new, "new", i32, row, dev),
        _tensor(held, "held", i32, row, dev), B, table, stride, cols,
        _tensor(free_pages, "free_pages", i32, free_pages.shape, dev), free_pages.numel(),
        _tensor(free_count, "free_count", i32, one, dev), int(page_size), T,
        _tensor(o["slots"], "slots", torch.int64, (T,), dev), *ptrs, _dev_ptr(dev_status),
        _use_stream(stream, dev, (o["cu"], o["slots"])))
    if st:
        _check(st, "ssd_page_plan")
    return o


def prefix_attention(q, k_cache, v_cache, prefix_tables, prefix_len, group_off, tables=None,
                     lens=None, scale=None, lse=True, workspace=None, dev_status=None,
                     stream=None, out=None):
    """ssd_prefix_attention: one query token per row, q [R, Hq, D] (bf16 or
    fp16), over caches [pages, page_size, Hkv, D] of its type (any strides
    with a contiguous head dimension).

    Rows group_off[g] .. group_off[g+1] (int32 [G+1]) read the first
    prefix_len[g] (int32 [G]) tokens of pages prefix_tables[g, :] (int32
    [G, W]), and each row the first lens[r] (int32 [R]) tokens of its own
    pages tables[r, :] (int32 [R, W']).  scale: 1 / sqrt(D) when None.
    Returns a dict: ``out`` [R, Hq, D] and, unless lse=False, ``lse`` float32
    [R, Hq].  `out`: the dict of an earlier call of these shapes, to use its
    tensors and workspace again, or one with some of them; what is absent is
    added, and a workspace that is too small (more groups, wider tables) replaced:
    a captured graph needs a dict of its own."""
    torch = _torch()
    i32 = torch.int32
    qs, ks, dt = q.shape, k_cache.shape, q.dtype
    if len(qs) != 3 or len(ks) != 4 or v_cache.shape != ks or ks[3] != qs[2]:
        raise SSDError("expected q [R, Hq, D] and caches [pages, page_size, Hkv, D]")
    R, Hq, D = qs
    code = SSD_BF16 if dt is torch.bfloat16 else SSD_F16 if dt is torch.float16 else -1
    if code < 0 or k_cache.dtype is not dt or v_cache.dtype is not dt:
        raise SSDError("q and the caches must share bfloat16 or float16")
    dev = q.get_device()
    if dev < 0 or k_cache.get_device() != dev or v_cache.get_device() != dev:
        raise SSDError("q and the caches must be on one GPU")
    _on_current(dev)
    o = out if out is not None else {}
    y = o.get("out")
    if y is None:
        y = o["out"] = torch.empty(qs, dtype=dt, device=q.device)
    elif y.shape != qs or y.dtype is not dt or y.get_device() != dev:
        raise SSDError("out must have q's shape, type and device")
    if lse and o.get("lse") is None:
        o["lse"] = torch.empty((R, Hq), dtype=torch.float32, device=q.device)
    q_at, k_at, v_at, y_at = q.stride(), k_cache.stride(), v_cache.stride(), y.stride()
    if q_at[2] != 1 or k_at[3] != 1 or v_at[3] != 1 or y_at[2] != 1:
        raise SSDError("the head dimension must be contiguous")
    G = prefix_len.numel()
    pt, pt_stride, pt_cols = _rows2d(prefix_tables, "prefix_tables", G, i32, dev)
    t = t_stride = t_cols = n = 0
    if tables is not None and lens is not None:
        t, t_stride, t_cols = _rows2d(tables, "tables", R, i32, dev)
        n = _tensor(lens, "lens", i32, (R,), dev)
    elif tables is not lens:
        raise SSDError("tables and lens go together")
    a = _Attention(code, R, Hq, ks[2], D, G, ks[0], ks[1], q.data_ptr(), q_at[0], q_at[1],
                   (k_cache.data_ptr(), k_at[0], k_at[1], k_at[2]),
                   (v_cache.data_ptr(), v_at[0], v_at[1], v_at[2]), pt,
                   _tensor(prefix_len, "prefix_len", i32, (G,), dev),
                   _tensor(group_off, "group_off", i32, (G + 1,), dev), t, n, pt_stride, t_stride,
                   pt_cols, t_cols, y.data_ptr(), y_at[0], y_at[1],
                   _tensor(o["lse"], "lse", torch.float32, (R, Hq), dev) if lse else 0,
                   D ** -0.5 if scale is None else scale, 0)
    L = lib()
    ws = workspace if workspace is not None else o.get("workspace")
    if ws is None:
        ws = o["workspace"] = _workspace(L.ssd_prefix_attention_workspace_size(a), q.device)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise SSDError("the workspace must be a contiguous tensor on q's GPU")
    handle = _use_stream(stream, dev, (*o.values(), ws))
    st = L.ssd_prefix_attention(a, ws.data_ptr(), ws.numel() * ws.element_size(),
                                _dev_ptr(dev_status), handle)
    if st == _ERR_WORKSPACE and workspace is None:
        # the rows are as before, but not the groups or tables; nothing has been launched
        ws = o["workspace"] = _workspace(L.ssd_prefix_attention_workspace_size(a), q.device)
        handle = _use_stream(stream, dev, (ws,))
        st = L.ssd_prefix_attention(a, ws.data_ptr(), ws.numel(), _dev_ptr(dev_status), handle)
    if st:
        _check(st, "ssd_prefix_attention")
    return o if lse or "lse" not in o else _without(o, "lse")


# The descriptors of the calls below are packed as the C structs lie in memory (ctypes takes
# several times as long to fill one): ssd_tree_attn, ssd_append, ssd_fork.
_PACK_TREE = struct.Struct("@8i" + "Q3q" + "Q3q" * 4 + "QQqQ" + "Q3q" + "Qif").pack
_PACK_APPEND = struct.Struct("@10i" + "Q4q" * 4 + "4Qq").pack
_PACK_FORK = struct.Struct("@10i" + "4Qq3Q" + "Q4q" * 2 + "6Q").pack
_UNPACKED = (struct.error, OverflowError)  # sizes beyond 32 bits, a scale beyond float32
_parents = {}  # trees by their bytes: the library reads them by address


def _parent_address(parent, N):
    try:
        par = np.asarray(parent, dtype=np.int32)
        good = par.shape == (N,) and (par is parent or par.tolist() == (
            parent.tolist() if hasattr(parent, "tolist") else list(parent)))
    except (TypeError, ValueError, OverflowError):
        good = False
    if not good:
        raise SSDError("parent must have N entries, whole numbers of 32 bits")
    key = par.tobytes()
    kept = _parents.get(key)
    if kept is None:
        if len(_parents) >= 256:
            _parents.clear()
        kept = _parents[key] = ctypes.create_string_buffer(key, max(len(key), 1))
    return ctypes.addressof(kept), kept


def _launch(fn, size, name, a, o, workspace, dev, device, dev_status, stream):
    """Call `fn` with a workspace of the dict's, which is made, or replaced when it is too
    small; `size` gives its bytes."""
    ws = workspace if workspace is not None else o.get("workspace")
    if ws is None:
        ws = o["workspace"] = _workspace(size(a), device)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise SSDError(f"the workspace must be a contiguous tensor on cuda:{dev}")
    status = None if dev_status is None else _dev_ptr(dev_status)
    if stream is None:
        handle = _torch_module._C._cuda_getCurrentRawStream(dev)
    else:
        handle = _use_stream(stream, dev, (*o.values(), ws))
    st = fn(a, ws.data_ptr(), ws.numel() * ws.element_size(), status, handle)
    if st == _ERR_WORKSPACE and workspace is None:  # nothing has been launched
        ws = o["workspace"] = _workspace(size(a), device)
        handle = _use_stream(stream, dev, (ws,))
        st = fn(a, ws.data_ptr(), ws.numel(), status, handle)
    if st:
        _check(st, name)


def tree_attention(q, k, v, k_cache, v_cache, tables, lens, parent=None, scale=None, lse=True,
                   workspace=None, dev_status=None, stream=None, out=None):
    """ssd_tree_attention: drafted nodes of a sequence over its cache and one another.

    q [B, N, Hq, D] and the nodes' k, v [B, N, Hkv, D] (bf16 or fp16, any strides with a
    contiguous head dimension, so pieces of one projection too); caches [pages, page_size, Hkv,
    D] of that type; tables int32 [B, W], lens int32 [B]: tokens in the cache, without the nodes.
    parent: N ints as in tree_verify (a chain when None): node u attends to the cache and to the
    nodes on its path, itself included.  N = 1: one token per sequence.  scale: 1 / sqrt(D) when
    None.
    Returns a dict: ``out`` [B, N, Hq, D] and, unless lse=False, ``lse`` float32 [B, N, Hq].
    `out`: as in prefix_attention; a captured graph needs a dict of its own."""
    torch = _torch()
    i32 = torch.int32
    qs, ks, cs, dt = q.shape, k.shape, k_cache.shape, q.dtype
    try:
        B, N, Hq, D = qs
        kB, kN, Hkv, kD = ks
        pages, page_size, cH, cD = cs
        fits = kB == B and kN == N and kD == D and cH == Hkv and cD == D
    except ValueError:
        fits = False
    if not fits or v.shape != ks or v_cache.shape != cs:
        raise SSDError("expected q [B, N, Hq, D], k and v [B, N, Hkv, D] and caches [pages, "
                       "page_size, Hkv, D]")
    code = SSD_BF16 if dt is torch.bfloat16 else SSD_F16 if dt is torch.float16 else -1
    dev = q.get_device()
    if code < 0 or k.dtype is not dt or v.dtype is not dt or k_cache.dtype is not dt or \
            v_cache.dtype is not dt:
        raise SSDError("q, the nodes and the caches must share bfloat16 or float16")
    if dev < 0 or k.get_device() != dev or v.get_device() != dev or \
            k_cache.get_device() != dev or v_cache.get_device() != dev:
        raise SSDError("q, the nodes and the caches must be on one GPU")
    if torch._C._cuda_getDevice() != dev:
        _on_current(dev)
    o = out if out is not None else {}
    y = o.get("out")
    if y is None:
        y = o["out"] = torch.empty(qs, dtype=dt, device=q.device)
    elif y.shape != qs or y.dtype is not dt or y.get_device() != dev:
        raise SSDError("out must have q's shape, type and device")
    at = 0
    if lse:
        z = o.get("lse")
        if z is None:
            z = o["lse"] = torch.empty((B, N, Hq), dtype=torch.float32, device=q.device)
        at = _tensor(z, "lse", torch.float32, (B, N, Hq), dev)
    qa, ya, ka, va, kc, vc = (q.stride(), y.stride(), k.stride(), v.stride(), k_cache.stride(),
                              v_cache.stride())
    if qa[3] != 1 or ya[3] != 1 or ka[3] != 1 or va[3] != 1 or kc[3] != 1 or vc[3] != 1:
        raise SSDError("the head dimension must be contiguous")
    tree, kept = (0, None) if parent is None else _parent_address(parent, N)
    table, stride, cols = _rows2d(tables, "tables", B, i32, dev)
    try:
        a = _PACK_TREE(code, B, N, Hq, Hkv, D, pages, page_size, q.data_ptr(), qa[0], qa[1], qa[2],
                       k.data_ptr(), ka[0], ka[1], ka[2], v.data_ptr(), va[0], va[1], va[2],
                       k_cache.data_ptr(), kc[0], kc[1], kc[2], v_cache.data_ptr(), vc[0], vc[1],
                       vc[2], table, _tensor(lens, "lens", i32, (B,), dev), stride, tree,
                       y.data_ptr(), ya[0], ya[1], ya[2], at, cols,
                       D ** -0.5 if scale is None else scale)
    except _UNPACKED as e:
        raise SSDError(f"ssd_tree_attention: {e}") from None
    L = lib()
    _launch(L.ssd_tree_attention, L.ssd_tree_attention_workspace_size, "ssd_tree_attention", a, o,
            workspace, dev, q.device, dev_status, stream)
    return o if lse or "lse" not in o else _without(o, "lse")


def _layers(t, name, dev):
    """The shape [L, X, Y, H, D] of a tensor, its bytes of an element, and ssd_layers of it (its
    address, strides in bytes); [X, Y, H, D] is one layer."""
    shape = t.shape
    n, es = len(shape), t.element_size()
    if n == 5 and t.get_device() == dev:
        s0, s1, s2, s3, s4 = t.stride()
    elif n == 4 and t.get_device() == dev:
        s1, s2, s3, s4 = t.stride()
        s0, shape = 0, (1, *shape)
    else:
        raise SSDError(f"{name}: expected a tensor of 4 dimensions, or 5 with the layers, on "
                       f"cuda:{dev}")
    if s4 != 1 or shape[4] * es % 16 != 0:
        raise SSDError(f"{name}: a head must be contiguous, and a multiple of 16 bytes")
    return shape, es, (t.data_ptr(), s0 * es, s1 * es, s2 * es, s3 * es)


def _like(t, other, layers, name, dev):
    """ssd_layers of a tensor of `other`'s shape and type, whose own are `layers`."""
    if t.stride() == other.stride() and t.get_device() == dev:
        return (t.data_ptr(), *layers[1:])
    return _layers(t, name, dev)[2]


_NO_LAYERS = (0, 0, 0, 0, 0)


def append_path(k, v, k_cache, v_cache, slots, owner, cu, path=None, dev_status=None,
                stream=None):
    """ssd_append_path: accepted nodes' keys and values into the caches of all layers.

    k, v [L, B, N, H, D] and caches [L, pages, page_size, H, D], or without the first dimension
    for one layer; any one type, any strides with contiguous heads of a multiple of 16 bytes;
    v and v_cache may both be None.  slots int64 [T], owner int32 [T] and cu int32 [B + 1] are
    page_plan's for the accepted tokens: row t of sequence b = owner[t] takes the node at place
    t - cu[b] of its path: node 0, then path[b, 0], path[b, 1], .. (int32 [B, n], tree_verify's;
    None: a chain).  Rows with a negative slot are passed over.  The caches are written in place
    and do not overlap the nodes.  Returns None."""
    torch = _torch()
    i32 = torch.int32
    dev, dt = k_cache.get_device(), k_cache.dtype
    if dev < 0:
        raise SSDError("expected caches on the GPU")
    if torch._C._cuda_getDevice() != dev:
        _on_current(dev)
    (L, B, N, H, D), es, kl = _layers(k, "k", dev)
    (cL, pages, page_size, cH, cD), _, cl = _layers(k_cache, "k_cache", dev)
    if L != cL or H != cH or D != cD or k.dtype is not dt:
        raise SSDError("nodes and caches must share the layers, heads and type")
    vl = wl = _NO_LAYERS
    if v is not None and v_cache is not None:
        if v.shape != k.shape or v_cache.shape != k_cache.shape or v.dtype is not dt or \
                v_cache.dtype is not dt:
            raise SSDError("v and v_cache must have the shapes and type of k and k_cache")
        vl, wl = _like(v, k, kl, "v", dev), _like(v_cache, k_cache, cl, "v_cache", dev)
    elif v is not v_cache:
        raise SSDError("v and v_cache go together")
    row = slots.shape
    if len(row) != 1:
        raise SSDError("expected slots [T]")
    at = _tensor(cu, "cu", i32, (B + 1,), dev)
    p = p_stride = p_cols = 0
    if path is not None:
        p, p_stride, p_cols = _rows2d(path, "path", B, i32, dev)
        p = p or at  # one of no columns has no memory, but no address would mean a chain
    try:
        a = _PACK_APPEND(L, B, N, H, D * es, pages, page_size, row[0], p_cols, 0, *kl, *vl, *cl,
                         *wl, _tensor(slots, "slots", torch.int64, row, dev),
                         _tensor(owner, "owner", i32, row, dev), at, p, p_stride)
    except _UNPACKED as e:
        raise SSDError(f"ssd_append_path: {e}") from None
    st = lib().ssd_append_path(a, None if dev_status is None else _dev_ptr(dev_status),
                               torch._C._cuda_getCurrentRawStream(dev) if stream is None
                               else stream.cuda_stream)
    if st:
        _check(st, "ssd_append_path")


_FORK = ("tables", "lens", "held", "served", "shares", "free_count")


def _fork_views(torch, counts, cols, device):
    """fork_rows' outputs: in one buffer, each on a 64-byte boundary."""
    base = torch.empty(sum(n + 15 & ~15 for n in counts), dtype=torch.int32, device=device)
    views, at = {}, 0
    for name, n in zip(_FORK, counts):
        views[name] = base[at:at + n]
        at += n + 15 & ~15
    views["tables"] = views["tables"].view(-1, cols)
    return views


def _fork_pointers(o, counts, i32, dev):
    """Addresses of fork_rows' outputs: views of one buffer, one after the other.  Their sizes
    are looked at too: others may take the same places."""
    t = o.get("tables")
    if t is None or t.dtype is not i32 or t.get_device() != dev or t.shape[0] != counts[1] or \
            not t.is_contiguous():
        raise SSDError("out: expected the dict of an earlier call with these sizes")
    memory = t.untyped_storage()
    first = at = memory.data_ptr()
    ptrs = []
    get = o.get
    for name, n in zip(_FORK, counts):
        t = get(name)
        if t is None or t.data_ptr() != at or t.numel() != n:
            raise SSDError(f"out: {name} is not that of an earlier call with these sizes")
        ptrs.append(at)
        at += (n + 15 & ~15) * 4
    if at - first > memory.nbytes():
        raise SSDError("out: expected the dict of an earlier call with these sizes")
    return ptrs


def fork_rows(src, lens, held, tables, shares, free_pages, free_count, page_size, k_cache=None,
              v_cache=None, workspace=None, dev_status=None, stream=None, out=None):
    """ssd_fork_rows: rows of the block tables continued, forked and freed.

    src int32 [B]: the old row that each new one continues (-1: none); lens, held int32 [S] and
    tables int32 [S, W] of the old rows; shares int32 [pages]: rows that hold a page beside the
    first; the stack free_pages int32 [n] with free_count int32 [1] (entries past it are
    written).  Old rows that nobody continues give their pages back; the first row that
    continues one keeps its pages, the others share the full ones and get a copy of the tokens
    of the last in a page from the stack.  k_cache, v_cache [L, pages, page_size, H, D] (or of
    one layer) hold those tokens (None: nothing is copied; v_cache alone may be None too).
    page_plan does not know shares: rows with shared pages end here alone, and their lengths
    never fall below the tokens that they share.
    Returns a dict of device tensors: tables [B, W], lens, held, served [B], shares [pages],
    free_count [1], all int32.  `out`: the dict of an earlier call of these sizes, to use its
    tensors and workspace again (not while one of them is this call's input)."""
    torch = _torch()
    i32 = torch.int32
    dev = src.get_device()
    row, old, pool, stack = src.shape, lens.shape, shares.shape, free_pages.shape
    if dev < 0 or not len(row) == len(old) == len(pool) == len(stack) == 1:
        raise SSDError("expected src [B], lens [S], shares [pages] and free_pages [n] on the GPU")
    if torch._C._cuda_getDevice() != dev:
        _on_current(dev)
    B, S, pages = row[0], old[0], pool[0]
    table, stride, cols = _rows2d(tables, "tables", S, i32, dev)
    kl = vl = _NO_LAYERS
    L = H = size = 0
    if k_cache is not None:
        ks, es, kl = _layers(k_cache, "k_cache", dev)
        L, H, size = ks[0], ks[3], ks[4] * es
        if ks[1] != pages or ks[2] != page_size:
            raise SSDError("the caches must have one page for each entry of shares, of page_size "
                           "tokens")
        if v_cache is not None:
            if v_cache.shape != k_cache.shape or v_cache.dtype is not k_cache.dtype:
                raise SSDError("the caches must have one shape and type")
            vl = _like(v_cache, k_cache, kl, "v_cache", dev)
    elif v_cache is not None:
        raise SSDError("v_cache goes with k_cache")
    o = out if out is not None else {}
    counts = (B * cols, B, B, B, pages, 1)
    if "tables" not in o and _FORK_NAMES.isdisjoint(o):
        if cols < 1:
            raise SSDError("the tables must have columns")
        o.update(_fork_views(torch, counts, cols, src.device))
    ptrs = _fork_pointers(o, counts, i32, dev)
    try:
        a = _PACK_FORK(S, B, cols, int(page_size), pages, stack[0], L, H, size, 0,
                       _tensor(src, "src", i32, row, dev), _tensor(lens, "lens", i32, old, dev),
                       _tensor(held, "held", i32, old, dev), table, stride,
                       _tensor(shares, "shares", i32, pool, dev),
                       _tensor(free_pages, "free_pages", i32, stack, dev),
                       _tensor(free_count, "free_count", i32, (1,), dev), *kl, *vl, *ptrs)
    except _UNPACKED as e:
        raise SSDError(f"ssd_fork_rows: {e}") from None
    f = lib()
    _launch(f.ssd_fork_rows, f.ssd_fork_rows_workspace_size, "ssd_fork_rows", a, o, workspace, dev,
            src.device, dev_status, stream)
    return o


_FORK_NAMES = set(_FORK)
