"""Thin ctypes binding of libtv (the C ABI in include/tv.h), with the same call names.

Only argument marshalling happens here: torch tensors supply device pointers, shapes,
strides and the current CUDA stream; every step of the computation runs in the library's
CUDA kernels.  There is no CPU fallback: if libtv.so has not been built, or a call fails,
this module raises.

    build_visibility(parent, anc, depth, dense_mask=None, status=None)
    rope_neox(x, out, prefix_len, depth, base=10000.0, cache=None)
    verify_prologue(parent, prefix_len, q_pe_in, q_pe_out, kpe_tree, ckv_tree, c_kv, k_pe, ...)
    verify_attn(q_latent, q_pe, c_kv, k_pe, prefix_len, anc, out, lse, scale, ...)
    build_tree(logprobs, cand_tokens, budget, parent, tokens, root=None, depth=None, ...)
    tree_accept(logits, parent, tokens, accept_len, path, new_tokens, target=None, ...)
    compact_kv(c_kv, k_pe, cache, prefix_len, path, accept_len, new_prefix_len, ...)
    tree_sample(logits, parent, tokens, uniforms, accept_len, path, new_tokens, ...)
    pages_reserve(pool, length, new_length, copies, ...), pages_fork(pool, fork_from, length),
    pages_release(pool, keep), pages_compact(pool, moves, n_moves),
    pages_copy(c_kv, k_pe, page_size, copies, ...)
    prefill_attn(q_nope, q_pe, w_kv, c_kv, k_pe, q_start, prefix_len, out, scale, ...)
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtv.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "tv.h")

TV_OK, TV_ERR_INVALID_ARG, TV_ERR_INVALID_TREE, TV_ERR_UNSUPPORTED = 0, -1, -2, -3
TV_ERR_CUDA, TV_ERR_TIMEOUT, TV_ERR_WORKSPACE, TV_ERR_BOUNDS = -4, -5, -6, -7
TV_ERR_NO_PAGES = -8
TV_F32, TV_BF16 = 0, 1
PATH_AUTO, PATH_SIMT, PATH_TCGEN05 = 0, 1, 2
PAGED_AUTO, PAGED_STEP_MAPS, PAGED_GATHER = 0, 1, 2
MASK_TREE, MASK_CAUSAL = 0, 1
DRAFT_BY_DEPTH, DRAFT_BY_NODE = 0, 1


class TVError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"{msg} (status {code})")
        self.status = code


class CacheLayout(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("page_size", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("kv_stride_b", ctypes.c_int64),
                ("num_rows", ctypes.c_int64)]


class AttnArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("Q", ctypes.c_int32),
        ("d_latent", ctypes.c_int32), ("d_rope", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("q_dt", ctypes.c_int), ("kv_dt", ctypes.c_int),
        ("q_latent", ctypes.c_void_p), ("q_pe", ctypes.c_void_p),
        ("c_kv", ctypes.c_void_p), ("k_pe", ctypes.c_void_p),
        ("ckv_row_stride", ctypes.c_int64), ("kpe_row_stride", ctypes.c_int64),
        ("cache", CacheLayout),
        ("prefix_len", ctypes.c_void_p),
        ("max_prefix_len", ctypes.c_int32),
        ("anc", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("status", ctypes.c_void_p),
        ("path", ctypes.c_int32),
        ("num_splits", ctypes.c_int32),
        ("paged_view", ctypes.c_int32),
        ("mask_mode", ctypes.c_int32),
        ("overlap_prev", ctypes.c_int32),
    ]


class PrologueArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("B", ctypes.c_int32), ("Q", ctypes.c_int32), ("H", ctypes.c_int32),
        ("d_latent", ctypes.c_int32), ("d_rope", ctypes.c_int32),
        ("parent", ctypes.c_void_p), ("prefix_len", ctypes.c_void_p),
        ("q_pe_in", ctypes.c_void_p), ("q_pe_out", ctypes.c_void_p), ("q_dt", ctypes.c_int),
        ("kpe_tree", ctypes.c_void_p), ("ckv_tree", ctypes.c_void_p),
        ("c_kv", ctypes.c_void_p), ("k_pe", ctypes.c_void_p), ("kv_dt", ctypes.c_int),
        ("ckv_row_stride", ctypes.c_int64), ("kpe_row_stride", ctypes.c_int64),
        ("cache", CacheLayout),
        ("anc", ctypes.c_void_p), ("depth", ctypes.c_void_p),
        ("rope_base", ctypes.c_double),
        ("status", ctypes.c_void_p),
    ]


class SampleArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("B", ctypes.c_int32), ("Q", ctypes.c_int32),
        ("vocab", ctypes.c_int64),
        ("logits", ctypes.c_void_p), ("logits_dt", ctypes.c_int),
        ("logits_row_stride", ctypes.c_int64),
        ("temperature", ctypes.c_void_p),
        ("parent", ctypes.c_void_p), ("tokens", ctypes.c_void_p),
        ("uniforms", ctypes.c_void_p),
        ("draft_probs", ctypes.c_void_p), ("draft_row_stride", ctypes.c_int64),
        ("draft_rows", ctypes.c_int32), ("draft_mode", ctypes.c_int32),
        ("accept_len", ctypes.c_void_p), ("path", ctypes.c_void_p),
        ("new_tokens", ctypes.c_void_p),
        ("status", ctypes.c_void_p),
    ]


class PrefillArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("T", ctypes.c_int32),
        ("d_latent", ctypes.c_int32), ("d_nope", ctypes.c_int32),
        ("d_rope", ctypes.c_int32), ("d_v", ctypes.c_int32),
        ("scale", ctypes.c_float), ("dt", ctypes.c_int),
        ("q_nope", ctypes.c_void_p), ("q_pe", ctypes.c_void_p), ("w_kv", ctypes.c_void_p),
        ("c_kv", ctypes.c_void_p), ("k_pe", ctypes.c_void_p),
        ("ckv_row_stride", ctypes.c_int64), ("kpe_row_stride", ctypes.c_int64),
        ("cache", CacheLayout),
        ("q_start", ctypes.c_void_p), ("prefix_len", ctypes.c_void_p),
        ("max_q_len", ctypes.c_int32), ("max_kv_len", ctypes.c_int32),
        ("total_kv", ctypes.c_int64),
        ("out", ctypes.c_void_p), ("status", ctypes.c_void_p),
    ]


class PagePool(ctypes.Structure):
    _fields_ = [
        ("page_table", ctypes.c_void_p), ("n_pages", ctypes.c_void_p),
        ("refcount", ctypes.c_void_p),
        ("rows", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
    ]


_lib = None


def load():
    """Open libtv.so (built by speculative_decoding_tree_04_gb300.build); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libtv.so is not built ({LIB_PATH}); run "
                           "`python -m speculative_decoding_tree_04_gb300.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, i64, dbl = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_double
    lib.tv_build_visibility.argtypes = [P, i32, i32, P, P, P, P, P]
    lib.tv_rope_neox.argtypes = [P, i32, i64, i64, P, i32, i64, i64, ctypes.POINTER(CacheLayout),
                                 i32, i32, i32, i32, P, P, dbl, P]
    lib.tv_verify_attn_workspace_size.argtypes = [ctypes.POINTER(AttnArgs)]
    lib.tv_verify_attn_workspace_size.restype = ctypes.c_size_t
    lib.tv_verify_attn_path.argtypes = [ctypes.POINTER(AttnArgs)]
    lib.tv_verify_attn_launches.argtypes = [ctypes.POINTER(AttnArgs)]
    lib.tv_verify_attn.argtypes = [ctypes.POINTER(AttnArgs), P, ctypes.c_size_t, P]
    lib.tv_verify_attn_noalloc.argtypes = [ctypes.POINTER(AttnArgs), P]
    lib.tv_noalloc_scratch_bytes.restype = ctypes.c_size_t
    lib.tv_status_string.argtypes = [i32]
    lib.tv_status_string.restype = ctypes.c_char_p
    lib.tv_last_error.restype = ctypes.c_char_p
    lib.tv_version.restype = ctypes.c_int
    lib.tv_testing_set_wait_fault.argtypes = [i32, ctypes.c_uint64, P]
    lib.tv_testing_set_prompt_fault.argtypes = [i32, i32, ctypes.c_uint64, P]
    lib.tv_build_tree.argtypes = [P, P, P, i32, i32, i32, i32, P, P, P, P, P, P]
    lib.tv_verify_prologue.argtypes = [ctypes.POINTER(PrologueArgs), P]
    lib.tv_tree_accept_workspace_size.argtypes = [i32, i32, i64]
    lib.tv_tree_accept_workspace_size.restype = ctypes.c_size_t
    lib.tv_tree_accept.argtypes = [P, i32, i64, i64, P, P, i32, i32, P, P, P, P, P, P,
                                   ctypes.c_size_t, P]
    lib.tv_compact_kv.argtypes = [P, P, i32, i64, i64, i32, i32, ctypes.POINTER(CacheLayout),
                                  P, P, P, i32, i32, P, P, P]
    lib.tv_tree_sample.argtypes = [ctypes.POINTER(SampleArgs), P]
    POOL, sz = ctypes.POINTER(PagePool), ctypes.c_size_t
    lib.tv_pages_workspace_size.argtypes = [POOL]
    lib.tv_pages_workspace_size.restype = sz
    lib.tv_pages_reserve.argtypes = [POOL, P, P, P, P, P, sz, P]
    lib.tv_pages_fork.argtypes = [POOL, P, P, P, P]
    lib.tv_pages_release.argtypes = [POOL, P, P, P]
    lib.tv_pages_compact.argtypes = [POOL, P, P, P, P, sz, P]
    lib.tv_pages_copy.argtypes = [P, P, i32, i64, i64, i32, i32, i32, i64, i64, i32, i64, P, P,
                                  i32, P, P]
    lib.tv_prefill_attn_workspace_size.argtypes = [ctypes.POINTER(PrefillArgs)]
    lib.tv_prefill_attn_workspace_size.restype = sz
    lib.tv_prefill_attn.argtypes = [ctypes.POINTER(PrefillArgs), P, sz, P]
    _lib = lib
    return lib


def header_functions(paths=None):
    """Names of the functions the headers under include/ declare (for symbol checks)."""
    if paths is None:
        inc = os.path.dirname(HEADER)
        paths = sorted(os.path.join(inc, f) for f in os.listdir(inc) if f.endswith(".h"))
    names = set()
    for path in ([paths] if isinstance(paths, str) else paths):
        with open(path) as f:
            text = f.read()
        text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
        names |= set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(tv_\w+)\s*\(", text, re.M))
    return sorted(names)


def _check(rc, what):
    if rc != TV_OK:
        lib = load()
        raise TVError(rc, f"{what}: {lib.tv_last_error().decode()}")


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return TV_F32
    if t.dtype == torch.bfloat16:
        return TV_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("libtv takes CUDA tensors only")


def build_visibility(parent, anc, depth, dense_mask=None, status=None, stream=None):
    """parent [B,Q] int32 -> anc [B,Q] int64 (bit patterns of uint64), depth [B,Q] int32."""
    _need_cuda(parent, anc, depth, dense_mask, status)
    assert parent.dtype == torch.int32 and anc.dtype in (torch.int64, torch.uint64)
    assert parent.is_contiguous() and anc.is_contiguous() and depth.is_contiguous()
    B, Q = parent.shape
    rc = load().tv_build_visibility(_ptr(parent), B, Q, _ptr(anc), _ptr(depth),
                                    _ptr(dense_mask), _ptr(status), _stream(stream))
    _check(rc, "tv_build_visibility")


def make_cache(page_table=None, page_size=64, kv_stride_b=0, num_rows=0) -> CacheLayout:
    """Cache geometry; num_rows = rows of the c_kv / k_pe arrays (0 = unknown)."""
    if page_table is not None:
        _need_cuda(page_table)
        assert page_table.dtype == torch.int32 and page_table.is_contiguous()
        return CacheLayout(page_table.data_ptr(), page_size, page_table.shape[1], 0, num_rows)
    return CacheLayout(None, page_size, 0, kv_stride_b, num_rows)


def rope_neox(x, out, prefix_len, depth, base=10000.0, cache: CacheLayout | None = None,
              stream=None):
    """NeoX RoPE on x [B,Q,H,D] (or [B,Q,D] for one head) into out; depth None means row
    i sits at position prefix_len + i (a chain, as in prefill).

    Without ``cache`` out has x's shape (in place allowed).  With ``cache`` out is a cache
    array [rows, D] (row stride out.stride(0)) and row (b, i) goes to the cache slot of
    logical key prefix_len[b] + i.
    """
    _need_cuda(x, out, prefix_len, depth)
    x4 = x if x.dim() == 4 else x.unsqueeze(2)
    B, Q, NH, D = x4.shape
    if x4.stride(-1) != 1 or out.stride(-1) != 1:
        raise ValueError("innermost dimension must be contiguous")
    isr, ish = x4.stride(1), x4.stride(2)
    if x4.stride(0) != Q * isr:
        raise ValueError("x rows must be uniformly strided over (B, Q)")
    if cache is None:
        o4 = out if out.dim() == 4 else out.unsqueeze(2)
        if o4.stride(0) != Q * o4.stride(1):
            raise ValueError("out rows must be uniformly strided over (B, Q)")
        osr, osh = o4.stride(1), o4.stride(2)
        cp = None
    else:
        osr, osh = out.stride(0), D
        cp = ctypes.byref(cache)
    rc = load().tv_rope_neox(_ptr(x), _dt(x), isr, ish, _ptr(out), _dt(out), osr, osh, cp,
                             B, Q, NH, D, _ptr(prefix_len), _ptr(depth), float(base),
                             _stream(stream))
    _check(rc, "tv_rope_neox")


def attn_args(q_latent, q_pe, c_kv, k_pe, prefix_len, anc, out, lse, scale, max_prefix_len,
              page_table=None, page_size=64, kv_stride_b=0, status=None, path=PATH_AUTO,
              num_splits=0, paged_view=PAGED_AUTO, mask_mode=MASK_TREE,
              overlap_prev=0) -> AttnArgs:
    _need_cuda(q_latent, q_pe, c_kv, k_pe, prefix_len, anc, out, lse, page_table, status)
    B, Q, H, DL = q_latent.shape
    DR = q_pe.shape[-1]
    for t in (q_latent, q_pe, prefix_len, anc, out, lse):
        if t is not None and not t.is_contiguous():
            raise ValueError("q_latent, q_pe, prefix_len, anc, out, lse must be contiguous")
    if c_kv.stride(-1) != 1 or k_pe.stride(-1) != 1:
        raise ValueError("cache rows must be contiguous")
    a = AttnArgs()
    a.struct_size = ctypes.sizeof(AttnArgs)
    a.B, a.H, a.Q, a.d_latent, a.d_rope = B, H, Q, DL, DR
    a.scale = float(scale)
    a.q_dt, a.kv_dt = _dt(q_latent), _dt(c_kv)
    a.q_latent, a.q_pe = q_latent.data_ptr(), q_pe.data_ptr()
    a.c_kv, a.k_pe = c_kv.data_ptr(), k_pe.data_ptr()
    a.ckv_row_stride, a.kpe_row_stride = c_kv.stride(0), k_pe.stride(0)
    a.cache = make_cache(page_table, page_size, kv_stride_b,
                         min(c_kv.shape[0], k_pe.shape[0]))
    a.prefix_len = prefix_len.data_ptr()
    a.max_prefix_len = int(max_prefix_len)
    a.anc = None if anc is None else anc.data_ptr()
    a.out, a.lse = out.data_ptr(), lse.data_ptr()
    a.status = None if status is None else status.data_ptr()
    a.path, a.num_splits, a.paged_view = int(path), int(num_splits), int(paged_view)
    a.mask_mode = int(mask_mode)
    a.overlap_prev = int(overlap_prev)
    return a


def workspace_size(a: AttnArgs) -> int:
    return int(load().tv_verify_attn_workspace_size(ctypes.byref(a)))


def attn_launches(a: AttnArgs) -> int:
    """Kernels one tv_verify_attn call with these arguments enqueues."""
    rc = load().tv_verify_attn_launches(ctypes.byref(a))
    if rc < 0:
        _check(rc, "tv_verify_attn_launches")
    return rc


def chosen_path(a: AttnArgs) -> int:
    rc = load().tv_verify_attn_path(ctypes.byref(a))
    if rc < 0:
        _check(rc, "tv_verify_attn_path")
    return rc


_ws_cache: dict = {}


def verify_attn_noalloc(a: AttnArgs, stream=None):
    """tv_verify_attn_noalloc on prepared arguments: the CUDA-core kernel with its split
    scratch in the library's fixed device array (no workspace, no allocation)."""
    rc = load().tv_verify_attn_noalloc(ctypes.byref(a), _stream(stream))
    _check(rc, "tv_verify_attn_noalloc")


def noalloc_scratch_bytes() -> int:
    return int(load().tv_noalloc_scratch_bytes())


def verify_attn(q_latent, q_pe, c_kv, k_pe, prefix_len, anc, out, lse, scale, max_prefix_len,
                page_table=None, page_size=64, kv_stride_b=0, status=None, path=PATH_AUTO,
                num_splits=0, workspace=None, stream=None, paged_view=PAGED_AUTO,
                mask_mode=MASK_TREE, overlap_prev=0):
    """Tree-verify attention; out [B,Q,H,DL] and lse [B,Q,H] (float32) are written.

    ``workspace`` (a CUDA uint8 tensor) is allocated through torch and cached per device
    when not given.  ``overlap_prev=1`` declares that the call queued just before this one
    writes neither prefix_len nor the page table (tv_attn_args.overlap_prev)."""
    a = attn_args(q_latent, q_pe, c_kv, k_pe, prefix_len, anc, out, lse, scale,
                  max_prefix_len, page_table, page_size, kv_stride_b, status, path, num_splits,
                  paged_view, mask_mode, overlap_prev)
    need = workspace_size(a)
    if workspace is None and need > 0:
        key = q_latent.device
        ws = _ws_cache.get(key)
        if ws is None or ws.numel() < need:
            ws = torch.empty(need, dtype=torch.uint8, device=q_latent.device)
            _ws_cache[key] = ws
        workspace = ws
    wptr = None if workspace is None else ctypes.c_void_p(workspace.data_ptr())
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().tv_verify_attn(ctypes.byref(a), wptr, wbytes, _stream(stream))
    _check(rc, "tv_verify_attn")
    return a


def accept_workspace_size(B: int, Q: int, vocab: int) -> int:
    return int(load().tv_tree_accept_workspace_size(B, Q, vocab))


def tree_accept(logits, parent, tokens, accept_len, path, new_tokens, target=None,
                status=None, workspace=None, stream=None):
    """Greedy acceptance: logits [B,Q,V] (float32 or bf16, rows contiguous) -> accept_len
    [B], path [B,Q], new_tokens [B,Q] (and target [B,Q] if given), all int32.  The
    workspace (argmax keys) is allocated through torch and cached when not given."""
    _need_cuda(logits, parent, tokens, accept_len, path, new_tokens, target, status)
    B, Q, V = logits.shape
    if logits.stride(2) != 1 or logits.stride(0) != Q * logits.stride(1):
        raise ValueError("logits rows must be contiguous and uniformly strided over (B, Q)")
    for t in (parent, tokens, accept_len, path, new_tokens):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError("parent, tokens and the outputs must be contiguous int32")
    need = accept_workspace_size(B, Q, V)
    if workspace is None and need > 0:
        key = ("accept", logits.device)
        ws = _ws_cache.get(key)
        if ws is None or ws.numel() < need:
            ws = torch.empty(need, dtype=torch.uint8, device=logits.device)
            _ws_cache[key] = ws
        workspace = ws
    wptr = None if workspace is None else ctypes.c_void_p(workspace.data_ptr())
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().tv_tree_accept(_ptr(logits), _dt(logits), V, logits.stride(1), _ptr(parent),
                               _ptr(tokens), B, Q, _ptr(target), _ptr(accept_len), _ptr(path),
                               _ptr(new_tokens), _ptr(status), wptr, wbytes, _stream(stream))
    _check(rc, "tv_tree_accept")


def compact_kv(c_kv, k_pe, cache: CacheLayout, prefix_len, path, accept_len, new_prefix_len,
               status=None, stream=None):
    """Post-verify compaction of the cache arrays c_kv [rows, DL] and k_pe [rows, DR] (in
    place) under ``cache`` (with num_rows set); new_prefix_len [B] int32 is written."""
    _need_cuda(c_kv, k_pe, prefix_len, path, accept_len, new_prefix_len, status)
    if c_kv.stride(-1) != 1 or k_pe.stride(-1) != 1:
        raise ValueError("cache rows must be contiguous")
    B, Q = path.shape
    rc = load().tv_compact_kv(_ptr(c_kv), _ptr(k_pe), _dt(c_kv), c_kv.stride(0), k_pe.stride(0),
                              c_kv.shape[1], k_pe.shape[1], ctypes.byref(cache),
                              _ptr(prefix_len), _ptr(path), _ptr(accept_len), B, Q,
                              _ptr(new_prefix_len), _ptr(status), _stream(stream))
    _check(rc, "tv_compact_kv")


def build_tree(logprobs, cand_tokens, budget, parent, tokens, root=None, depth=None, score=None,
               status=None, stream=None):
    """Best-first draft tree: logprobs [B,L,K] float32 (descending over K), cand_tokens
    [B,L,K] int32 -> parent, tokens [B, budget+1] int32 (depth, score optional)."""
    _need_cuda(logprobs, cand_tokens, root, parent, tokens, depth, score, status)
    B, L, K = logprobs.shape
    for t in (logprobs, cand_tokens, parent, tokens):
        if not t.is_contiguous():
            raise ValueError("tv_build_tree takes contiguous tensors")
    if logprobs.dtype != torch.float32 or cand_tokens.dtype != torch.int32:
        raise ValueError("logprobs must be float32 and cand_tokens int32")
    rc = load().tv_build_tree(_ptr(logprobs), _ptr(cand_tokens), _ptr(root), B, L, K,
                              int(budget), _ptr(parent), _ptr(tokens), _ptr(depth), _ptr(score),
                              _ptr(status), _stream(stream))
    _check(rc, "tv_build_tree")


def verify_prologue(parent, prefix_len, q_pe_in, q_pe_out, kpe_tree, ckv_tree, c_kv, k_pe,
                    cache: CacheLayout, anc, depth, base=10000.0, status=None, stream=None):
    """tv_verify_prologue: visibility, RoPE of q_pe (into q_pe_out, may be q_pe_in), RoPE of
    the draft keys into their cache slots and the append of the draft latent rows
    (ckv_tree may be None), in one launch."""
    _need_cuda(parent, prefix_len, q_pe_in, q_pe_out, kpe_tree, ckv_tree, c_kv, k_pe, anc,
               depth, status)
    B, Q, H, DR = q_pe_in.shape
    for t in (parent, prefix_len, q_pe_in, q_pe_out, kpe_tree, anc, depth):
        if not t.is_contiguous():
            raise ValueError("tv_verify_prologue takes contiguous tensors")
    a = PrologueArgs()
    a.struct_size = ctypes.sizeof(PrologueArgs)
    a.B, a.Q, a.H, a.d_rope = B, Q, H, DR
    a.d_latent = c_kv.shape[1]
    a.parent, a.prefix_len = parent.data_ptr(), prefix_len.data_ptr()
    a.q_pe_in, a.q_pe_out, a.q_dt = q_pe_in.data_ptr(), q_pe_out.data_ptr(), _dt(q_pe_in)
    a.kpe_tree = kpe_tree.data_ptr()
    a.ckv_tree = None if ckv_tree is None else ckv_tree.data_ptr()
    a.c_kv, a.k_pe, a.kv_dt = c_kv.data_ptr(), k_pe.data_ptr(), _dt(k_pe)
    a.ckv_row_stride, a.kpe_row_stride = c_kv.stride(0), k_pe.stride(0)
    a.cache = cache
    a.anc, a.depth = anc.data_ptr(), depth.data_ptr()
    a.rope_base = float(base)
    a.status = None if status is None else status.data_ptr()
    rc = load().tv_verify_prologue(ctypes.byref(a), _stream(stream))
    _check(rc, "tv_verify_prologue")


def _on_device(*ts):
    """Check that every tensor given lives on one CUDA device, and return its index."""
    dev = None
    for t in ts:
        if t is not None:
            d = t.get_device()
            if d != dev:
                if d < 0:
                    raise ValueError("libtv takes CUDA tensors only")
                if dev is not None:
                    raise ValueError(f"tensors on cuda:{dev} and cuda:{d}")
                dev = d
    return dev


def _raw_stream(dev, stream):
    """Handle of the stream to launch on (default: the tensors' device's current one)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device.index != dev:
        raise ValueError(f"tensors on cuda:{dev}, stream on {stream.device}")
    return stream.cuda_stream


def _call(dev, name, *args):
    """One library call with the tensors' device current; raises on a failure."""
    fn = getattr(_lib or load(), name)
    if torch._C._cuda_getDevice() == dev:
        rc = fn(*args)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args)
    if rc != TV_OK:
        _check(rc, name)


def _scratch(kind, dev, stream, handle, size_of, x):
    """Workspace of size_of(x) bytes for one call on the stream: one buffer per device, stream
    and kind of call, grown when needed.  During a capture the buffer is the graph's own:
    graphs that share one could replay at the same time, and it must outlive them."""
    if stream is not None or torch._C._cuda_getDevice() != dev:
        # both the size and the allocation are the device's and the stream's: a block that the
        # current stream has just given up may still be read by work queued there
        with torch.cuda.device(dev), torch.cuda.stream(stream):
            return _scratch(kind, dev, None, handle, size_of, x)
    need = max(1, size_of(x))
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(need, dtype=torch.uint8, device=f"cuda:{dev}")
    key = (kind, dev, handle)
    ws = _ws_cache.get(key)
    if ws is None or ws.numel() < need:
        ws = _ws_cache[key] = torch.empty(need, dtype=torch.uint8, device=f"cuda:{dev}")
    return ws


def _i32(name, t, shape):
    if t.shape != shape or t.dtype is not torch.int32 or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 of shape {tuple(shape)}")


def _row_stride(name, t):
    """Elements between the rows of a [B, rows, V] tensor whose rows lie evenly spaced."""
    B, n, V = t.shape
    if t.numel() and t.stride(2) != 1 and V > 1:
        raise ValueError(f"{name} rows must be contiguous")
    if n == 1:
        return t.stride(0) if B > 1 else V
    if B > 1 and t.stride(0) != n * t.stride(1):
        raise ValueError(f"{name} rows must be evenly spaced over its first two dimensions")
    return t.stride(1)


def _status_arg(status):
    if status is None:
        return None
    if status.dtype is not torch.int32 or status.numel() < 1:
        raise ValueError("status must be an int32 tensor")
    return status.data_ptr()


def tree_sample(logits, parent, tokens, uniforms, accept_len, path, new_tokens,
                temperature=None, draft_probs=None, draft_mode=DRAFT_BY_DEPTH, status=None,
                stream=None):
    """Sampled acceptance: logits [B,Q,V] (float32 or bf16), a draft tree parent and tokens
    [B,Q] int32, uniforms [B,Q] float32 -> accept_len [B], path and new_tokens [B,Q] int32.

    temperature [B] float32 (0 = greedy).  draft_probs [B,R,V] float32: the distributions
    the children were drawn from, by depth or by node (draft_mode); None when the candidates
    were chosen without chance."""
    dev = _on_device(logits, parent, tokens, uniforms, accept_len, path, new_tokens,
                     temperature, draft_probs, status)
    B, Q, V = logits.shape
    l_stride = _row_stride("logits", logits)
    for name, t, shape in (("parent", parent, (B, Q)), ("tokens", tokens, (B, Q)),
                           ("accept_len", accept_len, (B,)), ("path", path, (B, Q)),
                           ("new_tokens", new_tokens, (B, Q))):
        _i32(name, t, shape)
    for name, t, shape in (("uniforms", uniforms, (B, Q)), ("temperature", temperature, (B,))):
        if t is not None and (t.shape != shape or t.dtype is not torch.float32 or
                              not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous float32 of shape {shape}")
    probs, p_stride, p_rows = None, 0, 0
    if draft_probs is not None:
        d = draft_probs
        if d.dtype is not torch.float32 or d.dim() != 3 or d.shape[0] != B or d.shape[2] != V:
            raise ValueError("draft_probs must be float32 [B, rows, V]")
        probs, p_stride, p_rows = d.data_ptr(), _row_stride("draft_probs", d), d.shape[1]
    a = SampleArgs(ctypes.sizeof(SampleArgs), B, Q, V, logits.data_ptr(), _dt(logits), l_stride,
                   None if temperature is None else temperature.data_ptr(),
                   parent.data_ptr(), tokens.data_ptr(), uniforms.data_ptr(), probs, p_stride,
                   p_rows, int(draft_mode), accept_len.data_ptr(), path.data_ptr(),
                   new_tokens.data_ptr(), _status_arg(status))
    _call(dev, "tv_tree_sample", ctypes.byref(a), _raw_stream(dev, stream))


def make_page_pool(refcount, page_table, n_pages, page_size) -> PagePool:
    """A pool over refcount [pages], page_table [rows, max_pages] and n_pages [rows] int32
    (empty: 0, -1 and 0); the tensors are kept alive by it and changed in place."""
    dev = _on_device(refcount, page_table, n_pages)
    rows, most = page_table.shape
    _i32("refcount", refcount, (refcount.numel(),))
    _i32("page_table", page_table, (rows, most))
    _i32("n_pages", n_pages, (rows,))
    p = PagePool(page_table.data_ptr(), n_pages.data_ptr(), refcount.data_ptr(), rows, most,
                 refcount.numel(), int(page_size))
    p.tensors, p.device, p.row_shape = (refcount, page_table, n_pages), dev, (rows,)
    return p


def pages_workspace_size(pool: PagePool) -> int:
    return int(load().tv_pages_workspace_size(ctypes.byref(pool)))


def _pool_call(name, pool, per_row, others, status, stream, workspace=None, scratch=False):
    """Marshal one pool call: per-row int32 arguments, other device arguments, status."""
    dev = _on_device(*per_row.values(), *others, status, workspace)
    if dev != pool.device:
        raise ValueError(f"pool on cuda:{pool.device}, arguments on cuda:{dev}")
    for what, t in per_row.items():
        _i32(what, t, pool.row_shape)
    args = [t.data_ptr() for t in per_row.values()]
    args += [t.data_ptr() for t in others]
    args.append(_status_arg(status))
    handle = _raw_stream(dev, stream)
    if scratch:
        if workspace is None:
            workspace = _scratch("pages", dev, stream, handle, pages_workspace_size, pool)
        args += [workspace.data_ptr(), workspace.numel() * workspace.element_size()]
    _call(dev, name, ctypes.byref(pool), *args, handle)


def pages_reserve(pool: PagePool, length, new_length, copies, status=None, workspace=None,
                  stream=None):
    """Give every row the pages of keys length .. new_length-1 for itself; copies [rows,3]
    int32 becomes the list pages_copy takes."""
    _i32("copies", copies, (pool.rows, 3))
    _pool_call("tv_pages_reserve", pool, {"length": length, "new_length": new_length},
               (copies,), status, stream, workspace, True)


def pages_fork(pool: PagePool, fork_from, length, status=None, stream=None):
    """Row r shares the pages of the first length[r] keys of row fork_from[r] (-1: none)."""
    _pool_call("tv_pages_fork", pool, {"fork_from": fork_from, "length": length}, (), status,
               stream)


def pages_release(pool: PagePool, keep, status=None, stream=None):
    """Row r keeps the pages of its first keep[r] keys (negative: left alone)."""
    _pool_call("tv_pages_release", pool, {"keep": keep}, (), status, stream)


def pages_compact(pool: PagePool, moves, n_moves, status=None, workspace=None, stream=None):
    """Move the pages in use to the front of the pool: tables and counts now, the cache's
    rows by pages_copy with moves [num_pages,3] and count=n_moves [1] (int32)."""
    _i32("moves", moves, (pool.num_pages, 3))
    _i32("n_moves", n_moves, (1,))
    _pool_call("tv_pages_compact", pool, {}, (moves, n_moves), status, stream, workspace, True)


def pages_copy(c_kv, k_pe, page_size, copies, count=None, status=None, stream=None):
    """Copy the listed pages' rows in c_kv [rows, DL] and k_pe [rows, DR], or in every layer
    of [layers, rows, DL] and [layers, rows, DR].  copies [n,3] int32 as pages_reserve or
    pages_compact wrote it; count [1]: only its first count entries."""
    dev = _on_device(c_kv, k_pe, copies, count, status)
    c3 = c_kv if c_kv.dim() == 3 else c_kv.unsqueeze(0)
    k3 = k_pe if k_pe.dim() == 3 else k_pe.unsqueeze(0)
    if c3.shape[:2] != k3.shape[:2] or c_kv.dtype != k_pe.dtype:
        raise ValueError("c_kv and k_pe must have the same layers, rows and dtype")
    if c3.stride(2) != 1 or k3.stride(2) != 1:
        raise ValueError("cache rows must be contiguous")
    n = copies.shape[0]
    _i32("copies", copies, (n, 3))
    if count is not None:
        _i32("count", count, (1,))
    layers, rows, DL = c3.shape
    _call(dev, "tv_pages_copy", c_kv.data_ptr(), k_pe.data_ptr(), _dt(c_kv), c3.stride(1),
          k3.stride(1), DL, k3.shape[2], layers, c3.stride(0), k3.stride(0), int(page_size), rows,
          copies.data_ptr(), None if count is None else count.data_ptr(), n, _status_arg(status),
          _raw_stream(dev, stream))


def prefill_args(q_nope, q_pe, w_kv, c_kv, k_pe, q_start, prefix_len, out, scale, max_q_len,
                 max_kv_len, total_kv, page_table=None, page_size=64, kv_stride_b=0,
                 status=None) -> PrefillArgs:
    T, H, DN = q_nope.shape
    B, DR, DL = prefix_len.shape[0], q_pe.shape[2], w_kv.shape[2]
    DV = w_kv.shape[1] - DN
    dt = q_nope.dtype
    for name, t, shape in (("q_nope", q_nope, (T, H, DN)), ("q_pe", q_pe, (T, H, DR)),
                           ("w_kv", w_kv, (H, DN + DV, DL)), ("out", out, (T, H, DV))):
        if t.shape != shape or t.dtype is not dt or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous {dt} of shape {shape}")
    for name, t, d in (("c_kv", c_kv, DL), ("k_pe", k_pe, DR)):
        if t.dim() != 2 or t.shape[1] != d or t.stride(1) != 1 or t.dtype is not dt:
            raise ValueError(f"{name} must be rows of {d} contiguous {dt}")
    _i32("q_start", q_start, (B + 1,))
    _i32("prefix_len", prefix_len, (B,))
    rows = min(c_kv.shape[0], k_pe.shape[0])
    if page_table is not None:
        _i32("page_table", page_table, (B, page_table.shape[1]))
        cache = CacheLayout(page_table.data_ptr(), page_size, page_table.shape[1], 0, rows)
    else:
        cache = CacheLayout(None, page_size, 0, kv_stride_b, rows)
    return PrefillArgs(ctypes.sizeof(PrefillArgs), B, H, T, DL, DN, DR, DV, float(scale),
                       _dt(q_nope), q_nope.data_ptr(), q_pe.data_ptr(), w_kv.data_ptr(),
                       c_kv.data_ptr(), k_pe.data_ptr(), c_kv.stride(0), k_pe.stride(0), cache,
                       q_start.data_ptr(), prefix_len.data_ptr(), int(max_q_len),
                       int(max_kv_len), int(total_kv), out.data_ptr(), _status_arg(status))


def prefill_workspace_size(a: PrefillArgs) -> int:
    return int(load().tv_prefill_attn_workspace_size(ctypes.byref(a)))


def prefill_attn(q_nope, q_pe, w_kv, c_kv, k_pe, q_start, prefix_len, out, scale, max_q_len,
                 max_kv_len, total_kv, page_table=None, page_size=64, kv_stride_b=0,
                 status=None, workspace=None, stream=None):
    """Causal attention of packed prompts in the expanded form: q_nope [T,H,128], q_pe
    [T,H,64], w_kv [H,256,DL], cache rows c_kv [rows,DL] and k_pe [rows,64], q_start [B+1]
    and prefix_len [B] int32 -> out [T,H,128] (all bf16).  max_q_len, max_kv_len and
    total_kv bound a sequence's queries, its keys, and all sequences' keys together."""
    dev = _on_device(q_nope, q_pe, w_kv, c_kv, k_pe, q_start, prefix_len, out, page_table,
                     status, workspace)
    a = prefill_args(q_nope, q_pe, w_kv, c_kv, k_pe, q_start, prefix_len, out, scale, max_q_len,
                     max_kv_len, total_kv, page_table, page_size, kv_stride_b, status)
    handle = _raw_stream(dev, stream)
    if workspace is None:
        workspace = _scratch("prefill", dev, stream, handle, prefill_workspace_size, a)
    _call(dev, "tv_prefill_attn", ctypes.byref(a), workspace.data_ptr(),
          workspace.numel() * workspace.element_size(), handle)
