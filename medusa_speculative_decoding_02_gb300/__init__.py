"""Thin Python binding over libmedusa_gb300.so (ctypes).

Every step of the Medusa decoding step runs in the library's CUDA kernels;
this module only turns torch tensors into device pointers, sizes and the
current CUDA stream, allocates outputs and workspaces with torch, and raises
``MedusaError`` on a non-OK status.  There is no CPU or PyTorch fallback: if
the compiled library is missing, importing the calls fails loudly.

Public calls (same names as the C ABI in include/medusa.h):
    heads, heads_lm, heads_sample, heads_noalloc, build_tree, build_tree_static, tree_attention, evaluate_posterior,
    speculative_posterior, commit_kv, evaluate_posterior_commit, qk_norm_rope, qk_norm_rope_append,
    tree_attention_window, kv4_append, kv4_unpack, commit_kv4, tree_attention_kv4, paged_append,
    commit_paged, chunk_attention_paged, tree_attention_paged, token_logprobs
plus workspace-size queries, device-status helpers, launch_count,
``StepExecutor`` (medusa_step_create / medusa_step_run: the whole step, input
copies included, issued by one native call), and ``StepGraph``, which
captures a whole decoding step (copies and calls) into a CUDA graph once and
replays it per step.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmedusa_gb300.so")

F32, BF16 = 0, 1
GREEDY, TYPICAL = 0, 1
WS_HEADER = 256
STEP_GRAPH = 1
MAX_TOP_S = 16
MAX_TREE_ROWS = 256

STATUS = {0: "MEDUSA_OK", 1: "MEDUSA_ERR_INVALID_ARG", 2: "MEDUSA_ERR_UNSUPPORTED",
          3: "MEDUSA_ERR_WORKSPACE", 4: "MEDUSA_ERR_CUDA", 5: "MEDUSA_ERR_TIMEOUT",
          6: "MEDUSA_ERR_DEVICE_CHECK"}
DEVICE_STATUS = {0: "ok", 1: "bad token", 2: "bad parent", 3: "bad prefix", 4: "bad score",
                 5: "bad depth", 6: "timeout", 7: "bad path", 8: "bad cache",
                 9: "drain timeout", 10: "bad page"}

EXPORTS = ("medusa_status_string", "medusa_last_error", "medusa_launch_count",
           "medusa_wait_budget", "medusa_set_wait_budget",
           "medusa_read_device_status", "medusa_clear_device_status",
           "medusa_heads_workspace_size", "medusa_heads",
           "medusa_heads_lm_workspace_size", "medusa_heads_lm",
           "medusa_build_tree_workspace_size", "medusa_build_tree", "medusa_build_tree_static",
           "medusa_tree_attention_workspace_size", "medusa_tree_attention",
           "medusa_posterior_workspace_size", "medusa_evaluate_posterior",
           "medusa_evaluate_posterior_commit", "medusa_commit_kv", "medusa_heads_sample",
           "medusa_speculative_workspace_size", "medusa_speculative_posterior",
           "medusa_step_desc_size", "medusa_step_create", "medusa_step_run",
           "medusa_step_wait", "medusa_step_destroy",
           "medusa_qk_norm_rope", "medusa_qk_norm_rope_append",
           "medusa_tree_attention_window_workspace_size", "medusa_tree_attention_window",
           "medusa_kv4_row_bytes", "medusa_kv4_append", "medusa_kv4_unpack", "medusa_commit_kv4",
           "medusa_tree_attention_kv4_workspace_size", "medusa_tree_attention_kv4",
           "medusa_paged_append", "medusa_commit_paged", "medusa_paged_attention_workspace_size",
           "medusa_chunk_attention_paged", "medusa_tree_attention_paged", "medusa_token_logprobs")


class _Copy(ctypes.Structure):
    """medusa_copy"""
    _fields_ = [("dst", ctypes.c_void_p), ("src", ctypes.c_void_p), ("bytes", ctypes.c_size_t)]


class _StepDesc(ctypes.Structure):
    """medusa_step_desc, field for field (checked against medusa_step_desc_size)."""
    _P, _I, _F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float
    _fields_ = [("early", _P), ("n_early", _I), ("late", _P), ("n_late", _I), ("dtype", _I),
                ("h", _P), ("W1", _P), ("b1", _P), ("W2", _P),
                ("B", _I), ("d", _I), ("V", _I), ("K", _I), ("top_s", _I),
                ("topk_ids", _P), ("topk_logp", _P),
                ("root", _P), ("s_host", _P), ("n", _I), ("prefix_len", _P),
                ("tokens", _P), ("parent", _P), ("depth", _P), ("pos_id", _P), ("anc_mask", _P),
                ("paths", _P), ("n_leaf", _P),
                ("q", _P), ("k_cache", _P), ("v_cache", _P), ("P_max", _I), ("H", _I), ("dh", _I),
                ("scale", _F), ("attn_out", _P),
                ("logits", _P), ("mode", _I), ("eps", _F), ("delta", _F), ("temperature", _F),
                ("accept_len", _P), ("path", _P), ("path_tokens", _P), ("next_token", _P),
                ("accept", _P), ("new_prefix_len", _P), ("ws", _P), ("ws_bytes", ctypes.c_size_t),
                ("flags", _I)]


class MedusaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmedusa_gb300.so (built by ``build.build()``); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'` (needs nvcc, sm_103a)")
    L = ctypes.CDLL(LIB_PATH)
    P, I, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    U64, I64 = ctypes.c_uint64, ctypes.c_int64
    sig = {
        "medusa_status_string": ([I], ctypes.c_char_p),
        "medusa_last_error": ([], ctypes.c_char_p),
        "medusa_launch_count": ([], ctypes.c_uint64),
        "medusa_wait_budget": ([], ctypes.c_uint32),
        "medusa_set_wait_budget": ([ctypes.c_uint32], None),
        "medusa_read_device_status": ([P, P, P], I),
        "medusa_clear_device_status": ([P, P], I),
        "medusa_heads_workspace_size": ([I, I, I, I, I], S),
        "medusa_heads": ([I, P, P, P, P, I, I, I, I, I, P, P, P, S, P], I),
        "medusa_heads_lm_workspace_size": ([I, I, I, I, I], S),
        "medusa_heads_lm": ([I, P, P, P, P, P, I, I, I, I, I, P, P, P, P, P, S, P], I),
        "medusa_build_tree_workspace_size": ([I, I, I, I], S),
        "medusa_build_tree": ([P, P, P, I, I, P, I, I, P, P, P, P, P, P, P, P, P, S, P], I),
        "medusa_build_tree_static": ([P, P, P, I, I, P, I, I, P, P, P, P, P, P, P, P, P, S, P], I),
        "medusa_tree_attention_workspace_size": ([I, I, I, I, I, I], S),
        "medusa_tree_attention": ([I, P, P, P, P, I, P, I, I, I, I, F, P, P, S, P], I),
        "medusa_posterior_workspace_size": ([I, I], S),
        "medusa_evaluate_posterior": ([I, P, P, P, P, I, I, I, I, I, F, F, F, P, P, P, P, P, P, S, P], I),
        "medusa_evaluate_posterior_commit": ([I, P, P, P, P, I, I, I, I, I, F, F, F, P, P, P, P, P,
                                              P, P, P, I, I, P, P, S, P], I),
        "medusa_commit_kv": ([I, P, P, P, P, P, I, I, I, I, I, P, P, S, P], I),
        "medusa_heads_sample": ([I, P, P, P, P, I, I, I, I, F, U64, U64, P, P, P, S, P], I),
        "medusa_speculative_workspace_size": ([I, I], S),
        "medusa_speculative_posterior": ([I, P, P, P, I, I, I, F, U64, U64, P, P, P, P, P, S, P],
                                         I),
        "medusa_step_desc_size": ([], S),
        "medusa_step_create": ([ctypes.POINTER(_StepDesc), ctypes.POINTER(P)], I),
        "medusa_step_run": ([P, P, I], I),
        "medusa_step_wait": ([P, P], I),
        "medusa_step_destroy": ([P], None),
        "medusa_qk_norm_rope": ([I, P, P, I64, I64, P, P, F, I, P, P, I, I, P, I, I, I, I, I, P, P,
                                 P], I),
        "medusa_qk_norm_rope_append": ([I, P, P, P, I64, I64, I64, P, P, F, I, P, P, I, I, P, P, P, P,
                                        I, I, I, I, I, I, P, P, S, P], I),
        "medusa_kv4_row_bytes": ([I, I], S),
        "medusa_kv4_append": ([I, P, P, I64, I64, P, P, P, I, P, I, I, I, I, P, S, P], I),
        "medusa_kv4_unpack": ([I, P, P, P, I, P, I, I, I, I, P, P, P, S, P], I),
        "medusa_commit_kv4": ([P, P, P, P, P, I, I, I, I, I, P, P, S, P], I),
        "medusa_paged_append": ([I, P, P, I64, I64, P, P, I, I, P, I, P, I, P, I, I, I, I, P, S, P], I),
        "medusa_commit_paged": ([I, P, P, I, I, P, I, P, I, P, P, I, I, I, I, I, P, P, S, P], I),
        "medusa_paged_attention_workspace_size": ([I] * 7, S),
        "medusa_token_logprobs": ([I, P, I64, P, I, I, I, F, P, P, P, P, P, P, S, P], I),
    }
    for kind in ("chunk", "tree"):
        sig[f"medusa_{kind}_attention_paged"] = ([I, P, P, P, I, I, P, I, P, I, P, I, I, I, I, I, F, P,
                                                  P, S, P], I)
    for kind in ("window", "kv4"):
        sig[f"medusa_tree_attention_{kind}_workspace_size"] = ([I] * 9, S)
        sig[f"medusa_tree_attention_{kind}"] = ([I, P, P, P, P, I, P, P, I, I, I, I, I, I, I, F, P, P,
                                                 S, P], I)
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def _check(rc: int):
    if rc != 0:
        msg = lib().medusa_last_error().decode(errors="replace")
        raise MedusaError(rc, msg)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _need(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _result_ptr(t: Optional[torch.Tensor], name: str):
    """Pointer of a posterior output: a CUDA tensor, or a pinned CPU tensor
    that the kernel writes directly (no copy back)."""
    if t is None:
        return None
    if not (t.is_cuda or t.is_pinned()):
        raise ValueError(f"{name} must be a CUDA tensor or pinned host memory")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _ptr(t)


def launch_count() -> int:
    return int(lib().medusa_launch_count())


def wait_budget() -> int:
    """Poll limit of the bounded device waits (fault injection: 0 makes
    them time out at once and set the "timeout" device status)."""
    return int(lib().medusa_wait_budget())


def set_wait_budget(polls: int) -> None:
    lib().medusa_set_wait_budget(int(polls))


def new_workspace(nbytes: int, device=None) -> torch.Tensor:
    """Zeroed device workspace (the status word must start at 0)."""
    n = (max(int(nbytes), WS_HEADER) + 255) // 256 * 256
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def read_device_status(ws: torch.Tensor, stream=None) -> int:
    out = ctypes.c_int32(0)
    _check(lib().medusa_read_device_status(_ptr(ws), ctypes.byref(out), _stream(stream)))
    return int(out.value)


def clear_device_status(ws: torch.Tensor, stream=None):
    _check(lib().medusa_clear_device_status(_ptr(ws), _stream(stream)))


# ------------------------------------------------------------------ heads ---

def heads_workspace_size(B: int, K: int, d: int, V: int, top_s: int) -> int:
    return int(lib().medusa_heads_workspace_size(B, K, d, V, top_s))


def heads(h, W1, b1, W2, top_s: int, ws=None, out=None, stream=None):
    """Top-s token ids [B,K,s] (int32) and log-probs (fp32) of the K heads."""
    for t, n in ((h, "h"), (W1, "W1"), (W2, "W2")):
        _need(t, n)
    if b1 is not None:
        _need(b1, "b1")
    B, d = h.shape
    K, V = W2.shape[0], W2.shape[1]
    if ws is None:
        ws = new_workspace(heads_workspace_size(B, K, d, V, top_s), h.device)
    if out is None:
        out = (torch.empty((B, K, top_s), dtype=torch.int32, device=h.device),
               torch.empty((B, K, top_s), dtype=torch.float32, device=h.device))
    ids, logp = out
    _check(lib().medusa_heads(_dtype(h), _ptr(h), _ptr(W1), _ptr(b1), _ptr(W2), B, d, V, K, top_s,
                              _ptr(ids), _ptr(logp), _ptr(ws), ws.numel(), _stream(stream)))
    return ids, logp


def heads_lm_workspace_size(B: int, K: int, d: int, V: int, top_s: int) -> int:
    return int(lib().medusa_heads_lm_workspace_size(B, K, d, V, top_s))


def heads_lm(h, W_lm, W1, b1, W2, top_s: int, ws=None, out=None, stream=None):
    """The LM head and the Medusa heads in one weight pass.  Returns
    (root int32 [B], root_logp fp32 [B], topk_ids int32 [B,K,top_s],
    topk_logp fp32 [B,K,top_s])."""
    for t, name in ((h, "h"), (W_lm, "W_lm"), (W1, "W1"), (W2, "W2")):
        _need(t, name)
    B, d = h.shape
    K, V = W2.shape[0], W2.shape[1]
    dev = h.device
    if ws is None:
        ws = new_workspace(heads_lm_workspace_size(B, K, d, V, top_s), dev)
    if out is None:
        out = (torch.empty((B,), dtype=torch.int32, device=dev),
               torch.empty((B,), dtype=torch.float32, device=dev),
               torch.empty((B, K, top_s), dtype=torch.int32, device=dev),
               torch.empty((B, K, top_s), dtype=torch.float32, device=dev))
    root, root_logp, ids, logp = out
    _check(lib().medusa_heads_lm(_dtype(h), _ptr(h), _ptr(W_lm), _ptr(W1), _ptr(b1), _ptr(W2), B, d,
                                 V, K, int(top_s), _ptr(root), _ptr(root_logp), _ptr(ids),
                                 _ptr(logp), _ptr(ws), ws.numel(), _stream(stream)))
    return root, root_logp, ids, logp


def heads_noalloc(h, W1, b1, W2, top_s: int, out=None, stream=None):
    """medusa_heads with the library's own 4 MiB device scratch: for callers
    that cannot allocate device memory when they run the heads.  Calls that
    overlap on the GPU share the scratch and must be serialised."""
    for t, n in ((h, "h"), (W1, "W1"), (W2, "W2")):
        _need(t, n)
    fn = lib().medusa_heads_noalloc
    P, I = ctypes.c_void_p, ctypes.c_int
    fn.argtypes = [I, P, P, P, P, I, I, I, I, I, P, P, P]
    fn.restype = I
    B, d = h.shape
    K, V = W2.shape[0], W2.shape[1]
    if out is None:
        out = (torch.empty((B, K, top_s), dtype=torch.int32, device=h.device),
               torch.empty((B, K, top_s), dtype=torch.float32, device=h.device))
    ids, logp = out
    _check(fn(_dtype(h), _ptr(h), _ptr(W1), _ptr(b1), _ptr(W2), B, d, V, K, top_s, _ptr(ids),
              _ptr(logp), _stream(stream)))
    return ids, logp


# ------------------------------------------------------------------- tree ---

@dataclass
class Tree:
    tokens: torch.Tensor
    parent: torch.Tensor
    depth: torch.Tensor
    pos_id: torch.Tensor
    anc_mask: torch.Tensor
    paths: torch.Tensor
    n_leaf: torch.Tensor

    @staticmethod
    def empty(B: int, n: int, K: int, device) -> "Tree":
        R = n + 1
        W = (R + 63) // 64
        i32 = dict(dtype=torch.int32, device=device)
        return Tree(torch.empty((B, R), **i32), torch.empty((B, R), **i32),
                    torch.empty((B, R), **i32), torch.empty((B, R), **i32),
                    torch.empty((B, R, W), dtype=torch.int64, device=device),
                    torch.empty((B, n, K + 1), **i32), torch.empty((B,), **i32))


def build_tree_workspace_size(B: int, K: int, top_s: int, n: int) -> int:
    return int(lib().medusa_build_tree_workspace_size(B, K, top_s, n))


def build_tree(root, topk_ids, topk_logp, s: Sequence[int], n: int, prefix_len=None, ws=None,
               out: Optional[Tree] = None, stream=None) -> Tree:
    """Budgeted candidate tree (canonical order) from the heads' top-s lists."""
    for t, nm in ((root, "root"), (topk_ids, "topk_ids"), (topk_logp, "topk_logp")):
        _need(t, nm)
    B, K, S = topk_ids.shape
    s_host = (ctypes.c_int32 * K)(*[int(x) for x in s])
    if ws is None:
        ws = new_workspace(build_tree_workspace_size(B, K, S, n), root.device)
    t = out or Tree.empty(B, n, K, root.device)
    _check(lib().medusa_build_tree(_ptr(root), _ptr(topk_ids), _ptr(topk_logp), B, K, s_host, S, n,
                                   _ptr(prefix_len), _ptr(t.tokens), _ptr(t.parent), _ptr(t.depth),
                                   _ptr(t.pos_id), _ptr(t.anc_mask), _ptr(t.paths), _ptr(t.n_leaf),
                                   _ptr(ws), ws.numel(), _stream(stream)))
    return t


def build_tree_static(root, topk_ids, log_a, s: Sequence[int], n: int, prefix_len=None, ws=None,
                      out: Optional[Tree] = None, stream=None) -> Tree:
    """Candidate tree whose shape comes from a calibrated table log_a [K, top_s]
    (shared by every sequence); tokens from each sequence's top-s lists."""
    for t, nm in ((root, "root"), (topk_ids, "topk_ids"), (log_a, "log_a")):
        _need(t, nm)
    B, K, S = topk_ids.shape
    if tuple(log_a.shape) != (K, S) or log_a.dtype != torch.float32:
        raise ValueError(f"log_a must be float32 [{K}, {S}], got {log_a.dtype} {tuple(log_a.shape)}")
    s_host = (ctypes.c_int32 * K)(*[int(x) for x in s])
    if ws is None:
        ws = new_workspace(build_tree_workspace_size(B, K, S, n), root.device)
    t = out or Tree.empty(B, n, K, root.device)
    _check(lib().medusa_build_tree_static(_ptr(root), _ptr(topk_ids), _ptr(log_a), B, K, s_host, S,
                                          n, _ptr(prefix_len), _ptr(t.tokens), _ptr(t.parent),
                                          _ptr(t.depth), _ptr(t.pos_id), _ptr(t.anc_mask),
                                          _ptr(t.paths), _ptr(t.n_leaf), _ptr(ws), ws.numel(),
                                          _stream(stream)))
    return t


# -------------------------------------------------------------- attention ---

def tree_attention_workspace_size(dtype: int, B: int, R: int, H: int, dh: int, P_max: int) -> int:
    return int(lib().medusa_tree_attention_workspace_size(dtype, B, R, H, dh, P_max))


def cache_pointers(caches: Sequence[torch.Tensor], device) -> torch.Tensor:
    """Device array of the per-sequence cache base pointers."""
    for c in caches:
        _need(c, "cache")
    return torch.tensor([c.data_ptr() for c in caches], dtype=torch.int64, device=device)


def tree_attention(q, k_ptrs, v_ptrs, prefix_len, P_max: int, anc_mask, scale=None, out=None,
                   ws=None, stream=None):
    """Tree-masked attention.  q [B,R,H,dh]; k_ptrs/v_ptrs: int64 device arrays of
    per-sequence cache pointers (see cache_pointers); prefix_len int32 [B]."""
    _need(q, "q")
    B, R, H, dh = q.shape
    dt = _dtype(q)
    if scale is None:
        scale = 1.0 / math.sqrt(dh)
    if ws is None:
        ws = new_workspace(tree_attention_workspace_size(dt, B, R, H, dh, P_max), q.device)
    if out is None:
        out = torch.empty_like(q)
    _check(lib().medusa_tree_attention(dt, _ptr(q), _ptr(k_ptrs), _ptr(v_ptrs), _ptr(prefix_len),
                                       int(P_max), _ptr(anc_mask), B, R, H, dh, float(scale),
                                       _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
    return out


# -------------------------------------------------------------- posterior ---

@dataclass
class Posterior:
    accept_len: torch.Tensor
    path: torch.Tensor
    path_tokens: torch.Tensor
    next_token: torch.Tensor
    accept: Optional[torch.Tensor]

    @staticmethod
    def empty(B: int, R: int, K: int, device, with_accept: bool = True) -> "Posterior":
        i32 = dict(dtype=torch.int32, device=device)
        return Posterior(torch.empty((B,), **i32), torch.empty((B, K + 1), **i32),
                         torch.empty((B, K + 1), **i32), torch.empty((B,), **i32),
                         torch.empty((B, R), **i32) if with_accept else None)

    @staticmethod
    def pinned(B: int, R: int, K: int, with_accept: bool = True) -> "Posterior":
        """Results in page-locked host memory: the posterior kernel writes
        them there directly; read them after the stream has synchronised."""
        i32 = dict(dtype=torch.int32)
        mk = lambda shape: torch.empty(shape, **i32).pin_memory()
        return Posterior(mk((B,)), mk((B, K + 1)), mk((B, K + 1)), mk((B,)),
                         mk((B, R)) if with_accept else None)


def posterior_workspace_size(B: int, R: int) -> int:
    return int(lib().medusa_posterior_workspace_size(B, R))


def evaluate_posterior(logits, tokens, parent, depth, K: int, mode: int = GREEDY, eps=0.09,
                       delta=0.3, temperature=1.0, ws=None, out: Optional[Posterior] = None,
                       with_accept: bool = True, stream=None) -> Posterior:
    """Acceptance + longest accepted path.  logits [B,R,V] bf16 or fp32."""
    _need(logits, "logits")
    B, R, V = logits.shape
    if ws is None:
        ws = new_workspace(posterior_workspace_size(B, R), logits.device)
    o = out or Posterior.empty(B, R, K, logits.device, with_accept)
    _check(lib().medusa_evaluate_posterior(_dtype(logits), _ptr(logits), _ptr(tokens), _ptr(parent),
                                           _ptr(depth), B, R, V, K, int(mode), float(eps),
                                           float(delta), float(temperature),
                                           _result_ptr(o.accept_len, "accept_len"),
                                           _result_ptr(o.path, "path"),
                                           _result_ptr(o.path_tokens, "path_tokens"),
                                           _result_ptr(o.next_token, "next_token"),
                                           _result_ptr(o.accept, "accept"), _ptr(ws), ws.numel(),
                                           _stream(stream)))
    return o


def evaluate_posterior_commit(logits, tokens, parent, depth, K: int, k_ptrs, v_ptrs, prefix_len,
                              H: int, dh: int, new_prefix_len=None, mode: int = GREEDY, eps=0.09,
                              delta=0.3, temperature=1.0, ws=None,
                              out: Optional[Posterior] = None, with_accept: bool = True,
                              stream=None):
    """evaluate_posterior, then the commit of commit_kv in the same kernel.
    The caches hold logits.dtype elements.  Returns (Posterior, new_prefix_len)."""
    _need(logits, "logits")
    B, R, V = logits.shape
    if ws is None:
        ws = new_workspace(posterior_workspace_size(B, R), logits.device)
    o = out or Posterior.empty(B, R, K, logits.device, with_accept)
    if new_prefix_len is None:
        new_prefix_len = torch.empty((B,), dtype=torch.int32, device=logits.device)
    _check(lib().medusa_evaluate_posterior_commit(
        _dtype(logits), _ptr(logits), _ptr(tokens), _ptr(parent), _ptr(depth), B, R, V, K,
        int(mode), float(eps), float(delta), float(temperature),
        _result_ptr(o.accept_len, "accept_len"), _result_ptr(o.path, "path"),
        _result_ptr(o.path_tokens, "path_tokens"), _result_ptr(o.next_token, "next_token"),
        _result_ptr(o.accept, "accept"), _ptr(k_ptrs), _ptr(v_ptrs),
        _ptr(prefix_len), int(H), int(dh), _ptr(new_prefix_len), _ptr(ws), ws.numel(),
        _stream(stream)))
    return o, new_prefix_len


# ----------------------------------------------------------------- commit ---

def commit_kv(dtype: int, k_ptrs, v_ptrs, prefix_len, path, accept_len, R: int, H: int, dh: int,
              new_prefix_len=None, ws=None, stream=None):
    """Move the accepted path's K/V rows into slots P_b..P_b+L (in place in the
    caches behind k_ptrs/v_ptrs); return new_prefix_len = P_b + L + 1."""
    B, K1 = path.shape
    dev = path.device
    if ws is None:
        ws = new_workspace(WS_HEADER, dev)
    if new_prefix_len is None:
        new_prefix_len = torch.empty((B,), dtype=torch.int32, device=dev)
    _check(lib().medusa_commit_kv(int(dtype), _ptr(k_ptrs), _ptr(v_ptrs), _ptr(prefix_len),
                                  _ptr(path), _ptr(accept_len), B, K1 - 1, int(R), int(H), int(dh),
                                  _ptr(new_prefix_len), _ptr(ws), ws.numel(), _stream(stream)))
    return new_prefix_len


# --------------------------------------------------------------- sampling ---

def heads_sample(h, W1, b1, W2, temperature: float, seed: int, step: int, ws=None, out=None,
                 stream=None):
    """One draft per head sampled from softmax(logits / T) (Gumbel-max with the
    library's Philox streams).  Returns (drafts int32 [B,K], draft_logits fp32
    [B,K,V])."""
    for t, name in ((h, "h"), (W1, "W1"), (W2, "W2")):
        _need(t, name)
    B, d = h.shape
    K, V = W2.shape[0], W2.shape[1]
    dev = h.device
    if ws is None:
        ws = new_workspace(heads_workspace_size(B, K, d, V, 1), dev)
    if out is None:
        out = (torch.empty((B, K), dtype=torch.int32, device=dev),
               torch.empty((B, K, V), dtype=torch.float32, device=dev))
    drafts, dl = out
    _check(lib().medusa_heads_sample(_dtype(h), _ptr(h), _ptr(W1), _ptr(b1), _ptr(W2), B, d, V, K,
                                     float(temperature), int(seed), int(step), _ptr(drafts),
                                     _ptr(dl), _ptr(ws), ws.numel(), _stream(stream)))
    return drafts, dl


@dataclass
class Speculative:
    accept_len: torch.Tensor
    path_tokens: torch.Tensor
    next_token: torch.Tensor
    accept: Optional[torch.Tensor]


def speculative_workspace_size(B: int, K: int) -> int:
    return int(lib().medusa_speculative_workspace_size(B, K))


def speculative_posterior(logits, tokens, draft_logits, temperature: float, seed: int, step: int,
                          ws=None, out: Optional[Speculative] = None, with_accept: bool = True,
                          stream=None) -> Speculative:
    """Exact speculative sampling on a chain: logits [B,K+1,V], tokens [B,K+1]
    (root then drafts), draft_logits fp32 [B,K,V]."""
    _need(logits, "logits")
    B, R, V = logits.shape
    K = R - 1
    dev = logits.device
    if ws is None:
        ws = new_workspace(speculative_workspace_size(B, K), dev)
    if out is None:
        i32 = dict(dtype=torch.int32, device=dev)
        out = Speculative(torch.empty((B,), **i32), torch.empty((B, K + 1), **i32),
                          torch.empty((B,), **i32),
                          torch.empty((B, K), **i32) if with_accept else None)
    _check(lib().medusa_speculative_posterior(
        _dtype(logits), _ptr(logits), _ptr(tokens), _ptr(draft_logits), B, V, K,
        float(temperature), int(seed), int(step), _ptr(out.accept_len), _ptr(out.path_tokens),
        _ptr(out.next_token), _ptr(out.accept), _ptr(ws), ws.numel(), _stream(stream)))
    return out


# ------------------------------------------- rotation, 4-bit cache, windows ---
#
# These calls run in a few microseconds on the GPU, so their checks are one
# short function per tensor, and the current stream is taken as its handle.

_INT = torch.int32
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _launch_on(ref: torch.Tensor, stream):
    """(device index, stream handle) of a call whose tensors must all be on the
    current device."""
    dev = ref.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError("tensors must be on the current CUDA device")
    if stream is not None:
        return dev, stream.cuda_stream
    return dev, _raw_stream(dev) if _raw_stream else torch.cuda.current_stream().cuda_stream


def _vec(t, n: int, dtype, dev: int, name: str):
    """Address of an array argument: n dense elements of dtype on device dev."""
    if t.dtype is not dtype or t.get_device() != dev or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous {dtype} elements on the same device, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _dense(t, shape, dtype, dev: int, name: str):
    """Address of a dense tensor argument of the given shape."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a dense {dtype} tensor of {tuple(shape)} on the same device, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _ints(*values):
    """Refuses integers past 32 bits, which the foreign call would take modulo 2^32."""
    for x in values:
        if not -0x80000000 <= x <= 0x7fffffff:
            raise ValueError(f"{x} does not fit in 32 bits")


def _ws_args(ws, dev: int):
    if ws.get_device() != dev or ws.dtype is not torch.uint8 or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous uint8 tensor on the same device")
    return ws.data_ptr(), ws.numel()


def _rows(t: torch.Tensor, name: str):
    """Row stride in elements of [B,R,heads,dh] rows: heads and dh dense, all
    rows evenly apart (a dense tensor, or a slice of a wider projection)."""
    shape = t.shape
    if len(shape) != 4:
        raise ValueError(f"{name} must be [B,R,heads,dh]")
    B, R, H, dh = shape
    if t.is_contiguous():
        return H * dh
    s = t.stride()
    if s[3] != 1 or (H > 1 and s[2] != dh) or (B > 1 and R > 1 and s[0] != R * s[1]):
        raise ValueError(f"{name}: heads must be dense and rows evenly apart")
    return s[1] if R > 1 else s[0] if B > 1 else H * dh


def _issue_on(stream):
    """Allocations belong to the stream that uses them, so that their memory is
    not handed out again while that stream still works on it."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _scratch(nbytes: int, device, stream):
    """A workspace made on the launch stream with the status word at 0 (the rest
    needs no clearing)."""
    with _issue_on(stream):
        t = torch.empty((max(int(nbytes), WS_HEADER) + 255) // 256 * 256, dtype=torch.uint8,
                        device=device)
        t[:WS_HEADER].zero_()
    return t


def _new(stream, like: torch.Tensor, shape=None, dtype=None):
    """An output tensor made on the launch stream."""
    shape, dtype = like.shape if shape is None else shape, dtype or like.dtype
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _rope_args(q, k, q_weight, k_weight, dev):
    qs, ks = q.shape, k.shape
    if k.dtype is not q.dtype or k.get_device() != dev or len(ks) != 4 or len(qs) != 4 \
            or ks[0] != qs[0] or ks[1] != qs[1] or ks[3] != qs[3]:
        raise ValueError("q must be [B,R,H,dh] and k [B,R,Hkv,dh] of the same dtype and device")
    dh = qs[3]
    return (None if q_weight is None else _vec(q_weight, dh, q.dtype, dev, "q_weight"),
            None if k_weight is None else _vec(k_weight, dh, q.dtype, dev, "k_weight"))


def qk_norm_rope(q, k, pos, inv_freq, q_weight=None, k_weight=None, eps: float = 1e-6,
                 norm: bool = True, interleaved: bool = False, n_rows=None, out=None, stream=None):
    """Per-head RMS norms of q [B,R,H,dh] and k [B,R,Hkv,dh] and their rotation to
    the positions ``pos`` (int32 [B,R], e.g. ``Tree.pos_id``), in one pass.
    ``inv_freq`` (fp32 [rot/2]) holds radians per position; ``norm=False``
    rotates only.  q and k may be slices of one wider projection.  Rows
    i >= n_rows[b] are left alone.  Returns (q_out, k_out), ``out`` if given
    (it may be (q, k))."""
    dt = _dtype(q)
    dev, st = _launch_on(q, stream)
    qw, kw = _rope_args(q, k, q_weight, k_weight, dev)
    B, R, H, dh = q.shape
    half = inv_freq.numel()
    if out is None:
        out = (_new(stream, q), _new(stream, k))
    _check(lib().medusa_qk_norm_rope(
        dt, q.data_ptr(), k.data_ptr(), _rows(q, "q"), _rows(k, "k"), qw, kw, eps, 1 if norm else 0,
        _vec(pos, B * R, _INT, dev, "pos"), _vec(inv_freq, half, torch.float32, dev, "inv_freq"),
        2 * half, 1 if interleaved else 0,
        None if n_rows is None else _vec(n_rows, B, _INT, dev, "n_rows"), B, R, H, k.shape[2], dh,
        _dense(out[0], q.shape, q.dtype, dev, "q_out"), _dense(out[1], k.shape, q.dtype, dev, "k_out"),
        st))
    return out


def qk_norm_rope_append(q, k, v, pos, inv_freq, k_ptrs, v_ptrs, prefix_len, P_max: int,
                        q_weight=None, k_weight=None, eps: float = 1e-6, norm: bool = True,
                        interleaved: bool = False, n_rows=None, out=None, ws=None, stream=None):
    """qk_norm_rope with the finished K rows, and the V rows, written into cache
    slots prefix_len[b] + i of the caches behind k_ptrs / v_ptrs
    ([>= P_max+R, Hkv, dh]).  Returns q_out."""
    dt = _dtype(q)
    dev, st = _launch_on(q, stream)
    qw, kw = _rope_args(q, k, q_weight, k_weight, dev)
    if v.dtype is not k.dtype or v.shape != k.shape or v.get_device() != dev:
        raise ValueError("v must have k's shape, dtype and device")
    _ints(P_max)
    B, R, H, dh = q.shape
    half = inv_freq.numel()
    if out is None:
        out = _new(stream, q)
    if ws is None:
        ws = _scratch(WS_HEADER, q.device, stream)
    ws_ptr, ws_n = _ws_args(ws, dev)
    _check(lib().medusa_qk_norm_rope_append(
        dt, q.data_ptr(), k.data_ptr(), v.data_ptr(), _rows(q, "q"), _rows(k, "k"), _rows(v, "v"), qw,
        kw, eps, 1 if norm else 0, _vec(pos, B * R, _INT, dev, "pos"),
        _vec(inv_freq, half, torch.float32, dev, "inv_freq"), 2 * half, 1 if interleaved else 0,
        None if n_rows is None else _vec(n_rows, B, _INT, dev, "n_rows"),
        _vec(k_ptrs, B, torch.int64, dev, "k_ptrs"), _vec(v_ptrs, B, torch.int64, dev, "v_ptrs"),
        _vec(prefix_len, B, _INT, dev, "prefix_len"), P_max, B, R, H, k.shape[2], dh,
        _dense(out, q.shape, q.dtype, dev, "out"), ws_ptr, ws_n, st))
    return out


def kv4_row_bytes(Hkv: int, dh: int) -> int:
    """Bytes of one slot of a 4-bit cache (one of K and V)."""
    _ints(Hkv, dh)
    return int(lib().medusa_kv4_row_bytes(int(Hkv), int(dh)))


def kv4_cache(slots: int, Hkv: int, dh: int, device=None) -> torch.Tensor:
    """A zeroed 4-bit cache of one sequence: uint8 [slots, row bytes]."""
    n = kv4_row_bytes(Hkv, dh)
    if n == 0:
        raise ValueError(f"Hkv={Hkv}, dh={dh}: dh must be 64 or 128, Hkv in 1..1024")
    return torch.zeros((slots, n), dtype=torch.uint8, device=device or "cuda")


def kv4_append(k, v, k_ptrs, v_ptrs, prefix_len, P_max: int, n_rows=None, ws=None, stream=None):
    """Rows k, v [B,R,Hkv,dh] into slots prefix_len[b] + i of the 4-bit caches behind
    k_ptrs / v_ptrs (see kv4_cache, at least P_max + R slots each).  Rows
    i >= n_rows[b] are left alone."""
    dt = _dtype(k)
    dev, st = _launch_on(k, stream)
    if v.dtype is not k.dtype or v.shape != k.shape or v.get_device() != dev:
        raise ValueError("v must have k's shape, dtype and device")
    _ints(P_max)
    ks, vs = _rows(k, "k"), _rows(v, "v")
    B, R, Hkv, dh = k.shape
    if ws is None:
        ws = _scratch(WS_HEADER, k.device, stream)
    ws_ptr, ws_n = _ws_args(ws, dev)
    _check(lib().medusa_kv4_append(
        dt, k.data_ptr(), v.data_ptr(), ks, vs, _vec(k_ptrs, B, torch.int64, dev, "k_ptrs"),
        _vec(v_ptrs, B, torch.int64, dev, "v_ptrs"), _vec(prefix_len, B, _INT, dev, "prefix_len"), P_max,
        None if n_rows is None else _vec(n_rows, B, _INT, dev, "n_rows"), B, R, Hkv, dh, ws_ptr, ws_n,
        st))


def kv4_unpack(k_ptrs, v_ptrs, prefix_len, P_max: int, R: int, Hkv: int, dh: int,
               dtype=torch.bfloat16, n_rows=None, out=None, ws=None, stream=None):
    """The values of slots prefix_len[b] + i, i < R, of 4-bit caches: (k, v)
    [B,R,Hkv,dh].  Rows i >= n_rows[b] are left as ``out`` has them."""
    dev, st = _launch_on(k_ptrs, stream)
    _ints(P_max, R, Hkv, dh)
    B = k_ptrs.numel()
    shape = (B, R, Hkv, dh)
    if out is None:
        out = (_new(stream, k_ptrs, shape, dtype), _new(stream, k_ptrs, shape, dtype))
    ko, vo = out
    if ws is None:
        ws = _scratch(WS_HEADER, k_ptrs.device, stream)
    ws_ptr, ws_n = _ws_args(ws, dev)
    _check(lib().medusa_kv4_unpack(
        _dtype(ko), _vec(k_ptrs, B, torch.int64, dev, "k_ptrs"),
        _vec(v_ptrs, B, torch.int64, dev, "v_ptrs"), _vec(prefix_len, B, _INT, dev, "prefix_len"), P_max,
        None if n_rows is None else _vec(n_rows, B, _INT, dev, "n_rows"), B, R, Hkv, dh,
        _dense(ko, shape, ko.dtype, dev, "k_out"), _dense(vo, shape, ko.dtype, dev, "v_out"), ws_ptr,
        ws_n, st))
    return out


def commit_kv4(k_ptrs, v_ptrs, prefix_len, path, accept_len, R: int, Hkv: int, dh: int,
               new_prefix_len=None, ws=None, stream=None):
    """commit_kv on 4-bit caches, which must have P_b + R slots; returns
    new_prefix_len = P_b + L + 1."""
    dev, st = _launch_on(path, stream)
    _ints(R, Hkv, dh)
    B, K1 = path.shape
    if new_prefix_len is None:
        new_prefix_len = _new(stream, prefix_len)
    if ws is None:
        ws = _scratch(WS_HEADER, path.device, stream)
    ws_ptr, ws_n = _ws_args(ws, dev)
    _check(lib().medusa_commit_kv4(
        _vec(k_ptrs, B, torch.int64, dev, "k_ptrs"), _vec(v_ptrs, B, torch.int64, dev, "v_ptrs"),
        _vec(prefix_len, B, _INT, dev, "prefix_len"), _vec(path, B * K1, _INT, dev, "path"),
        _vec(accept_len, B, _INT, dev, "accept_len"), B, K1 - 1, R, Hkv, dh,
        _vec(new_prefix_len, B, _INT, dev, "new_prefix_len"), ws_ptr, ws_n, st))
    return new_prefix_len


def tree_attention_window_workspace_size(dtype: int, B: int, R: int, H: int, Hkv: int, dh: int,
                                         P_max: int, window: int = 0, sinks: int = 0,
                                         kv4: bool = False) -> int:
    """Workspace of tree_attention_window, or with kv4 of tree_attention_kv4."""
    _ints(B, R, H, Hkv, dh, P_max, window, sinks)
    fn = (lib().medusa_tree_attention_kv4_workspace_size if kv4
          else lib().medusa_tree_attention_window_workspace_size)
    return int(fn(dtype, B, R, H, Hkv, dh, int(P_max), int(window), int(sinks)))


def _cache_attention(kv4, q, k_ptrs, v_ptrs, prefix_len, P_max, anc_mask, Hkv, depth, window, sinks,
                     scale, out, ws, stream):
    dt = _dtype(q)
    dev, st = _launch_on(q, stream)
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    B, R, H, dh = q.shape
    if Hkv is None:
        Hkv = H
    _ints(P_max, window, sinks, Hkv)
    if out is None:
        out = _new(stream, q)
    if ws is None:
        ws = _scratch(tree_attention_window_workspace_size(dt, B, R, H, Hkv, dh, P_max, window, sinks,
                                                           kv4), q.device, stream)
    ws_ptr, ws_n = _ws_args(ws, dev)
    fn = lib().medusa_tree_attention_kv4 if kv4 else lib().medusa_tree_attention_window
    _check(fn(dt, q.data_ptr(), _vec(k_ptrs, B, torch.int64, dev, "k_ptrs"),
              _vec(v_ptrs, B, torch.int64, dev, "v_ptrs"),
              _vec(prefix_len, B, _INT, dev, "prefix_len"), P_max,
              _vec(anc_mask, B * R * ((R + 63) // 64), torch.int64, dev, "anc_mask"),
              None if depth is None else _vec(depth, B * R, _INT, dev, "depth"), window, sinks, B, R, H,
              Hkv, dh, dh ** -0.5 if scale is None else scale,
              _dense(out, q.shape, q.dtype, dev, "out"), ws_ptr, ws_n, st))
    return out


def tree_attention_window(q, k_ptrs, v_ptrs, prefix_len, P_max: int, anc_mask, Hkv=None, depth=None,
                          window: int = 0, sinks: int = 0, scale=None, out=None, ws=None,
                          stream=None):
    """Tree attention in which a row sees the last ``window`` positions up to its
    own and the first ``sinks`` ones (window 0: everything); ``depth`` is
    Tree.depth.  q [B,R,H,dh]; caches [>= P_b+R, Hkv, dh], query head h reads
    KV head h // (H // Hkv)."""
    return _cache_attention(False, q, k_ptrs, v_ptrs, prefix_len, P_max, anc_mask, Hkv, depth, window,
                            sinks, scale, out, ws, stream)


def tree_attention_kv4(q, k_ptrs, v_ptrs, prefix_len, P_max: int, anc_mask, Hkv=None, depth=None,
                       window: int = 0, sinks: int = 0, scale=None, out=None, ws=None, stream=None):
    """tree_attention_window over 4-bit caches (kv4_cache, kv4_append)."""
    return _cache_attention(True, q, k_ptrs, v_ptrs, prefix_len, P_max, anc_mask, Hkv, depth, window,
                            sinks, scale, out, ws, stream)


# ------------------------------------------ paged cache, log probabilities ---

def _pages(k_pages, v_pages, page_table, B: int, Hkv: int, dh: int, dtype, dev: int):
    """The cache arguments of a call on pages."""
    ks, ts = k_pages.shape, page_table.shape
    if len(ks) != 4 or ks[2] != Hkv or ks[3] != dh:
        raise ValueError(f"the pools must be [pages,page,{Hkv},{dh}], got {tuple(ks)}")
    if len(ts) != 2 or ts[0] != B:
        raise ValueError(f"page_table must be [{B},pages], got {tuple(ts)}")
    _ints(ks[0], ts[1])
    return (_dense(k_pages, ks, dtype, dev, "k_pages"), _dense(v_pages, ks, dtype, dev, "v_pages"), ks[0],
            ks[1], _vec(page_table, B * ts[1], _INT, dev, "page_table"), ts[1])


def _pool_heads(k_pages):
    """(Hkv, dh) of a pool."""
    if len(k_pages.shape) != 4:
        raise ValueError("the pools must be [pages,page,Hkv,dh]")
    return k_pages.shape[2:]


def paged_append(k, v, k_pages, v_pages, page_table, prefix_len, P_max: int, n_rows=None, ws=None,
                 stream=None):
    """Rows k, v [B,R,Hkv,dh] into slots prefix_len[b] + i of a cache in pages: pools
    [pages,page,Hkv,dh], slot j of sequence b in row j % page of page
    page_table[b, j // page].  Rows i >= n_rows[b] are left alone."""
    dt = _dtype(k)
    dev, st = _launch_on(k, stream)
    if v.dtype is not k.dtype or v.shape != k.shape or v.get_device() != dev:
        raise ValueError("v must have k's shape, dtype and device")
    _ints(P_max)
    ks, vs = _rows(k, "k"), _rows(v, "v")
    B, R, Hkv, dh = k.shape
    cache = _pages(k_pages, v_pages, page_table, B, Hkv, dh, k.dtype, dev)
    if ws is None:
        ws = _scratch(WS_HEADER, k.device, stream)
    ws_ptr, ws_n = _ws_args(ws, dev)
    _check(lib().medusa_paged_append(
        dt, k.data_ptr(), v.data_ptr(), ks, vs, *cache, _vec(prefix_len, B, _INT, dev, "prefix_len"), P_max,
        None if n_rows is None else _vec(n_rows, B, _INT, dev, "n_rows"), B, R, Hkv, dh, ws_ptr, ws_n,
        st))


def commit_paged(k_pages, v_pages, page_table, prefix_len, P_max: int, path, accept_len, R: int,
                 new_prefix_len=None, ws=None, stream=None):
    """commit_kv on a cache in pages; returns new_prefix_len = P_b + L + 1."""
    dt = _dtype(k_pages)
    dev, st = _launch_on(path, stream)
    _ints(P_max, R)
    if len(path.shape) != 2:
        raise ValueError("path must be [B,K+1]")
    B, K1 = path.shape
    Hkv, dh = _pool_heads(k_pages)
    cache = _pages(k_pages, v_pages, page_table, B, Hkv, dh, k_pages.dtype, dev)
    if new_prefix_len is None:
        new_prefix_len = _new(stream, prefix_len)
    if ws is None:
        ws = _scratch(WS_HEADER, path.device, stream)
    ws_ptr, ws_n = _ws_args(ws, dev)
    _check(lib().medusa_commit_paged(
        dt, *cache, _vec(prefix_len, B, _INT, dev, "prefix_len"), P_max,
        _vec(path, B * K1, _INT, dev, "path"), _vec(accept_len, B, _INT, dev, "accept_len"), B, K1 - 1, R,
        Hkv, dh, _vec(new_prefix_len, B, _INT, dev, "new_prefix_len"), ws_ptr, ws_n, st))
    return new_prefix_len


def paged_attention_workspace_size(dtype: int, B: int, R: int, H: int, Hkv: int, dh: int,
                                   P_max: int) -> int:
    """Workspace of chunk_attention_paged and of tree_attention_paged."""
    _ints(B, R, H, Hkv, dh, P_max)
    return int(lib().medusa_paged_attention_workspace_size(dtype, B, R, H, Hkv, dh, int(P_max)))


def _paged_attention(fn, q, k_pages, v_pages, page_table, prefix_len, P_max, last, scale, out, ws, stream,
                     dt, dev, st):
    if len(q.shape) != 4 or not q.is_contiguous():
        raise ValueError("q must be a contiguous [B,R,H,dh]")
    B, R, H, dh = q.shape
    Hkv = _pool_heads(k_pages)[0]
    _ints(P_max)
    cache = _pages(k_pages, v_pages, page_table, B, Hkv, dh, q.dtype, dev)
    if out is None:
        out = _new(stream, q)
    if ws is None:
        ws = _scratch(paged_attention_workspace_size(dt, B, R, H, Hkv, dh, P_max), q.device, stream)
    ws_ptr, ws_n = _ws_args(ws, dev)
    _check(fn(dt, q.data_ptr(), *cache, _vec(prefix_len, B, _INT, dev, "prefix_len"), P_max, last, B, R, H,
              Hkv, dh, dh ** -0.5 if scale is None else scale, _dense(out, q.shape, q.dtype, dev, "out"),
              ws_ptr, ws_n, st))
    return out


def chunk_attention_paged(q, k_pages, v_pages, page_table, prefix_len, P_max: int, n_rows=None,
                          scale=None, out=None, ws=None, stream=None):
    """Attention of a chunk of new tokens over a cache in pages (see paged_append),
    which holds their K and V already: row i of q [B,R,H,dh] sees slots
    0 .. prefix_len[b] + i.  A piece of a prompt, or with R = 1 plain decoding.
    Rows i >= n_rows[b] are left as ``out`` has them."""
    dt = _dtype(q)
    dev, st = _launch_on(q, stream)
    last = None if n_rows is None else _vec(n_rows, q.shape[0], _INT, dev, "n_rows")
    return _paged_attention(lib().medusa_chunk_attention_paged, q, k_pages, v_pages, page_table, prefix_len,
                            P_max, last, scale, out, ws, stream, dt, dev, st)


def tree_attention_paged(q, k_pages, v_pages, page_table, prefix_len, P_max: int, anc_mask, scale=None,
                         out=None, ws=None, stream=None):
    """tree_attention over a cache in pages (see paged_append); query head h reads KV
    head h // (H // Hkv)."""
    dt = _dtype(q)
    dev, st = _launch_on(q, stream)
    B, R = q.shape[:2]
    mask = _vec(anc_mask, B * R * ((R + 63) // 64), torch.int64, dev, "anc_mask")
    return _paged_attention(lib().medusa_tree_attention_paged, q, k_pages, v_pages, page_table, prefix_len,
                            P_max, mask, scale, out, ws, stream, dt, dev, st)


@dataclass
class TokenLogprobs:
    logp: torch.Tensor      # fp32 [...]
    entropy: torch.Tensor   # fp32 [...], nats
    rank: torch.Tensor      # int32 [...]
    top_ids: torch.Tensor   # int32 [..., top]
    top_logp: torch.Tensor  # fp32 [..., top]


def _logprob_outputs(shape, top: int, device) -> TokenLogprobs:
    f32, empty, more = torch.float32, torch.empty, (*shape, top)
    return TokenLogprobs(empty(shape, dtype=f32, device=device), empty(shape, dtype=f32, device=device),
                         empty(shape, dtype=_INT, device=device), empty(more, dtype=_INT, device=device),
                         empty(more, dtype=f32, device=device))


def token_logprobs(logits, tokens, top: int = 0, temperature: float = 1.0,
                   out: Optional[TokenLogprobs] = None, ws=None, stream=None) -> TokenLogprobs:
    """ln p of the given tokens under softmax(logits / temperature), their ranks (0: the
    argmax), each row's entropy and its ``top`` most probable tokens, in one pass
    over the logits [..., V] (rows evenly apart); tokens int32 [...], -1 for none."""
    dt = _dtype(logits)
    dev, st = _launch_on(logits, stream)
    if not logits.shape:
        raise ValueError("logits must be [...,V]")
    shape, V = logits.shape[:-1], logits.shape[-1]
    N = tokens.numel()
    if tokens.shape != shape:
        raise ValueError(f"tokens must be {tuple(shape)}, got {tuple(tokens.shape)}")
    _ints(N, V, top)
    step = _row_step(logits, "logits")
    if out is None:
        if stream is None:
            out = _logprob_outputs(shape, top, logits.device)
        else:
            with torch.cuda.stream(stream):
                out = _logprob_outputs(shape, top, logits.device)
        outs = [t.data_ptr() for t in (out.logp, out.entropy, out.rank, out.top_ids, out.top_logp)]
    else:
        f32 = torch.float32
        outs = [_vec(out.logp, N, f32, dev, "logp"), _vec(out.entropy, N, f32, dev, "entropy"),
                _vec(out.rank, N, _INT, dev, "rank")]
        outs += [_vec(out.top_ids, N * top, _INT, dev, "top_ids"),
                 _vec(out.top_logp, N * top, f32, dev, "top_logp")] if top else [None, None]
    if ws is None:
        ws = _scratch(WS_HEADER, logits.device, stream)
    ws_ptr, ws_n = _ws_args(ws, dev)
    _check(lib().medusa_token_logprobs(dt, logits.data_ptr(), step, _vec(tokens, N, _INT, dev, "tokens"), N, V,
                                       top, temperature, *outs, ws_ptr, ws_n, st))
    return out


def _row_step(t: torch.Tensor, name: str) -> int:
    """Elements between the rows of a tensor whose last dimension is dense and whose
    rows are evenly apart."""
    V = t.shape[-1]
    if t.is_contiguous():
        return V
    s, n = t.stride(), t.shape
    if s[-1] != 1 and V > 1:
        raise ValueError(f"{name}: the last dimension must be dense")
    step = None  # of the innermost dimension that has more than one row
    rows = 1
    for d in range(len(n) - 2, -1, -1):
        if n[d] == 1:
            continue
        if step is None:
            step = s[d]
        elif s[d] != step * rows:
            raise ValueError(f"{name}: rows must be evenly apart")
        rows *= n[d]
    return V if step is None else step


# ------------------------------------------------------------- step graph ---

class StepGraph:
    """A decoding step captured once into a CUDA graph and replayed.

    ``fn`` issues the step on the current stream: copies of the step's
    inputs from pinned host buffers, the library calls (heads, tree,
    attention, posterior, ...), and the results' way back to the host: copies
    into pinned buffers, or a posterior whose outputs are pinned host memory
    (``Posterior.pinned``), which its kernel writes directly.  Every buffer it touches must stay allocated and at the
    same address while the graph lives; new inputs are written into the same
    pinned host buffers before each ``replay``.  The launches keep their
    programmatic-dependent-launch edges inside the graph.
    """

    def __init__(self, fn, warmup: int = 2):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(warmup):
                fn()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            fn()
        torch.cuda.synchronize()

    def replay(self):
        self.graph.replay()


# ---------------------------------------------------------- step executor ---

def _copy_pair(dst: torch.Tensor, src: torch.Tensor, name: str):
    _need(dst, f"{name} destination")
    if not (src.is_cuda or src.is_pinned()):
        raise ValueError(f"{name} source must be pinned host memory or a CUDA tensor")
    if not src.is_contiguous():
        raise ValueError(f"{name} source must be contiguous")
    nb = dst.numel() * dst.element_size()
    if src.numel() * src.element_size() != nb or nb == 0:
        raise ValueError(f"{name}: source and destination sizes differ or are empty")
    return _Copy(dst.data_ptr(), src.data_ptr(), nb)


class StepExecutor:
    """One decoding step issued by one native call (medusa_step_run).

    The executor holds the step's buffers (the descriptor of
    medusa_step_create): ``early`` and ``late`` are lists of (device
    destination, pinned-host or device source) tensor pairs copied at the
    start of every run -- early ones before the heads on the caller's stream,
    late ones on the executor's side stream during the heads pass.  Then
    heads, tree, attention and posterior (with the fused commit when
    ``new_prefix_len`` is given) run as the separate calls do.  Every tensor
    must keep its address while the executor lives; write new inputs into
    the same host buffers before each ``run``.  With ``graph=True`` the
    sequence is captured once at construction as a CUDA graph and each run
    is one graph launch.
    """

    def __init__(self, *, h, W1, b1, W2, top_s: int, topk: tuple, root, s: Sequence[int], n: int,
                 prefix_len, tree: "Tree", q, k_ptrs, v_ptrs, P_max: int, attn_out, logits,
                 post: "Posterior", K: int, mode: int = GREEDY, eps=0.09, delta=0.3,
                 temperature=1.0, ws=None, early=(), late=(), new_prefix_len=None, scale=None,
                 graph: bool = False):
        L = lib()
        if ctypes.sizeof(_StepDesc) != L.medusa_step_desc_size():
            raise MedusaError(1, "medusa_step_desc layout differs from the binding's")
        for t, nm in ((h, "h"), (W1, "W1"), (W2, "W2"), (root, "root"), (prefix_len, "prefix_len"),
                      (q, "q"), (attn_out, "attn_out"), (logits, "logits"), (k_ptrs, "k_ptrs"),
                      (v_ptrs, "v_ptrs")):
            _need(t, nm)
        B, d = h.shape
        V = W2.shape[1]
        H, dh = q.shape[2], q.shape[3]
        ids, logp = topk
        if ws is None:
            R = n + 1
            need = max(heads_workspace_size(B, K, d, V, top_s),
                       build_tree_workspace_size(B, K, top_s, n),
                       tree_attention_workspace_size(_dtype(q), B, R, H, dh, P_max),
                       posterior_workspace_size(B, R))
            ws = new_workspace(need, h.device)
        self._early = (_Copy * max(1, len(early)))(
            *[_copy_pair(a, b, f"early[{i}]") for i, (a, b) in enumerate(early)])
        self._late = (_Copy * max(1, len(late)))(
            *[_copy_pair(a, b, f"late[{i}]") for i, (a, b) in enumerate(late)])
        self._s = (ctypes.c_int32 * K)(*[int(x) for x in s])
        pv = lambda t: None if t is None else t.data_ptr()
        res = lambda t, nm: None if t is None else _result_ptr(t, nm).value
        desc = _StepDesc(
            early=ctypes.addressof(self._early), n_early=len(early),
            late=ctypes.addressof(self._late), n_late=len(late), dtype=_dtype(h),
            h=pv(h), W1=pv(W1), b1=pv(b1), W2=pv(W2), B=B, d=d, V=V, K=K, top_s=int(top_s),
            topk_ids=pv(ids), topk_logp=pv(logp), root=pv(root),
            s_host=ctypes.addressof(self._s), n=int(n), prefix_len=pv(prefix_len),
            tokens=pv(tree.tokens), parent=pv(tree.parent), depth=pv(tree.depth),
            pos_id=pv(tree.pos_id), anc_mask=pv(tree.anc_mask), paths=pv(tree.paths),
            n_leaf=pv(tree.n_leaf), q=pv(q), k_cache=pv(k_ptrs), v_cache=pv(v_ptrs),
            P_max=int(P_max), H=H, dh=dh,
            scale=float(1.0 / math.sqrt(dh) if scale is None else scale), attn_out=pv(attn_out),
            logits=pv(logits), mode=int(mode), eps=float(eps), delta=float(delta),
            temperature=float(temperature),
            accept_len=res(post.accept_len, "accept_len"), path=res(post.path, "path"),
            path_tokens=res(post.path_tokens, "path_tokens"),
            next_token=res(post.next_token, "next_token"), accept=res(post.accept, "accept"),
            new_prefix_len=pv(new_prefix_len), ws=pv(ws), ws_bytes=ws.numel(),
            flags=STEP_GRAPH if graph else 0)
        # every buffer the descriptor names stays referenced while the executor lives
        self._keep = (h, W1, b1, W2, ids, logp, root, prefix_len, tree, q, k_ptrs, v_ptrs,
                      attn_out, logits, post, new_prefix_len, ws, tuple(early), tuple(late))
        self.ws = ws
        handle = ctypes.c_void_p()
        _check(L.medusa_step_create(ctypes.byref(desc), ctypes.byref(handle)))
        self._handle = handle
        self._h = handle.value  # plain integers keep the per-step call short
        self._run = L.medusa_step_run

    def run(self, stream=None, synchronize: bool = True):
        """Issue one step on ``stream`` (the current stream by default); with
        ``synchronize`` wait for it, so results in pinned memory are ready."""
        if self._handle is None:
            raise MedusaError(1, "StepExecutor is closed")
        s = (torch.cuda.current_stream() if stream is None else stream).cuda_stream
        rc = self._run(self._h, s, 1 if synchronize else 0)
        if rc:
            _check(rc)

    def wait(self, stream=None):
        """Wait for every step issued so far (the wait of ``run``)."""
        if self._handle is None:
            raise MedusaError(1, "StepExecutor is closed")
        s = (torch.cuda.current_stream() if stream is None else stream).cuda_stream
        _check(lib().medusa_step_wait(self._h, s))

    def close(self):
        if getattr(self, "_handle", None) is not None:
            lib().medusa_step_destroy(self._handle)
            self._handle = None
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
