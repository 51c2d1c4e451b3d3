"""Thin ctypes binding of libddt.so (``include/ddt.h``).

Argument marshalling only: torch tensors become device pointers, the current
torch stream becomes the ``cudaStream_t``; every step of the verify path runs
in the library's kernels.  There is no fallback: if the shared library is
missing or fails to load, importing this module raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch

from . import _build

DL, DR, D = 512, 64, 576
_BF16, _I32 = torch.bfloat16, torch.int32
MAX_DEPTH, MAX_TOPK, MAX_Q_LEN, MAX_SPLITS = 7, 16, 128, 128

STATUS = {0: "DDT_OK", 1: "DDT_ERR_INVALID_ARG", 2: "DDT_ERR_UNSUPPORTED", 3: "DDT_ERR_WORKSPACE",
          4: "DDT_ERR_CUDA", 5: "DDT_ERR_DEVICE_CHECK", 6: "DDT_ERR_TIMEOUT"}


class DDTError(RuntimeError):
    def __init__(self, fn, status, detail=""):
        self.status = status
        super().__init__(f"{fn}: {STATUS.get(status, status)}{(' ' + detail) if detail else ''}")


# The calls that go through ddt_call_words, in the order of its numbers: their
# arguments are packed into one buffer, which costs a fifth of what ctypes takes
# for the 12 to 29 of them.
_IN_WORDS = dict.fromkeys(("ddt_gqa_norm_rope_append", "ddt_gqa_verify_attn", "ddt_cache_copy", "ddt_cache_commit",
                           "ddt_cache_compact", "ddt_gqa_chunk_attn", "ddt_gqa_chunk_weights",
                           "ddt_cache_evict"))


def _call(name, *args):
    """The call with its arguments (a null pointer is 0)."""
    st = lib.ddt_call_words(_IN_WORDS[name](*args))
    if st != 0:
        raise DDTError(name, st)


def _load():
    path = _build.LIB
    if not os.path.exists(path):
        raise ImportError(f"libddt.so not built at {path}; run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    P, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                            ctypes.c_size_t)
    sig = {
        "ddt_abi_version": ([], i32),
        "ddt_status_string": ([i32], ctypes.c_char_p),
        "ddt_build_tree": ([P, P, P, P, P, i32, i32, i32, P, P, P, P], i32),
        "ddt_mask_indptr": ([P, P, i32, P], i32),
        "ddt_compile_visibility": ([P, P, P, P, i32, i32, P, P], i32),
        "ddt_build_tree_visibility": ([P, P, P, P, P, P, P, i32, i32, i32, P, P, P, P, P], i32),
        "ddt_build_chain_visibility": ([P, P, P, i32, P, P, P, P], i32),
        "ddt_verify_attn_num_splits": ([i32, i32, i32, i32, i32], i32),
        "ddt_verify_attn_launched_splits": ([i32, i32], i32),
        "ddt_verify_attn_noalloc_splits": ([i32, i32, i32, i32, i32, i32], i32),
        "ddt_verify_attn_workspace_size": ([i32, i32, i32], sz),
        "ddt_verify_attn": ([P, P, i64, P, P, P, P, P, i32, i32, i32, i32, i32, f32, i32, P, P, P,
                             sz, P], i32),
        "ddt_verify_attn_noalloc": ([P, P, i64, P, P, P, P, P, i32, i32, i32, i32, i32, f32, i32, P,
                                     P, P], i32),
        "ddt_accept": ([P, P, P, P, i32, i32, P, P, P, P, P], i32),
        "ddt_commit_kv": ([P, i64, P, P, P, P, P, i32, i32, P, P], i32),
        "ddt_tree_links": ([P, P, i32, P, P, P, P], i32),
        "ddt_accept_sampled": ([P, P, P, P, P, i32, P, P, P, P, i32, i32, i32, P, P, P, P, P],
                               i32),
        "ddt_gqa_norm_rope_append": ([P, i64, P, i64, P, i64, P, P, f32, P, i64, i32, i32, P, P, P, P,
                                      i32, i32, i32, i32, i32, i32, P, P, P, i64, i64, P], i32),
        "ddt_gqa_verify_attn_num_ctas": ([i32, i32, i32, i32, i32, i32], i32),
        "ddt_gqa_verify_attn_workspace_size": ([i32, i32, i32, i32, i32, i32], sz),
        "ddt_gqa_verify_attn": ([P, P, P, i64, i64, P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32,
                                 i32, i32, f32, i32, P, P, P, sz, P], i32),
        "ddt_cache_copy": ([P, i64, i64, P, i64, i64, i32, i64, P, P, i32, P], i32),
        "ddt_cache_commit": ([P, i64, i64, i32, i64, P, P, P, P, P, i32, i32, i32, P, P], i32),
        "ddt_cache_compact_workspace_size": ([i64], sz),
        "ddt_cache_compact": ([P, i64, i64, i32, i64, P, i32, P, P, P, sz, P], i32),
        "ddt_gqa_chunk_attn_num_ctas": ([i32, i32, i32, i32, i32, i32], i32),
        "ddt_gqa_chunk_attn_workspace_size": ([i32, i32, i32, i32, i32], sz),
        "ddt_gqa_chunk_attn": ([P, P, P, i64, i64, P, P, P, i32, i32, i32, i32, i32, i32, i32, i32, f32,
                                f32, P, i32, P, i32, P, P, P, sz, P], i32),
        "ddt_gqa_chunk_weights_num_ctas": ([i32, i32], i32),
        "ddt_gqa_chunk_weights_workspace_size": ([i32], sz),
        "ddt_gqa_chunk_weights": ([P, P, i64, i64, P, P, P, P, i32, i32, i32, i32, i32, i32, i32, i32, f32,
                                   f32, P, i32, P, i32, P, P, i32, f32, i32, P, P, sz, P], i32),
        "ddt_cache_evict": ([P, P, P, P, i32, i32, i32, i32, i32, P, i32, P, P, P, i32, P], i32),
        "ddt_call_words": ([ctypes.c_char_p], i32),
        "ddt_get_error": ([P, P], i32),
        "ddt_selftest_wait_timeout": ([ctypes.c_uint32, P], i32),
        "ddt_verify_step": ([P, P], i32),
        "ddt_prefill_step": ([P, P], i32),
        "ddt_step_graph_create": ([P, P], i32),
        "ddt_step_graph_create_io": ([P, P, P, sz, P, P, sz, P], i32),
        "ddt_step_graph_launch": ([P, P], i32),
        "ddt_step_graph_destroy": ([P], i32),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    for i, name in enumerate(_IN_WORDS):
        args = sig[name][0]
        pack = struct.Struct("=qq" + "".join("d" if a is f32 else "q" for a in args)).pack
        _IN_WORDS[name] = functools.partial(pack, i, len(args))
    return lib


lib = _load()


class StepArgs(ctypes.Structure):
    """ddt_step_args of include/ddt.h, field for field."""
    _P, _i32 = ctypes.c_void_p, ctypes.c_int32
    _fields_ = [
        ("topk_logp", _P), ("topk_ids", _P), ("root_id", _P), ("budget", _P),
        ("max_depth", _i32), ("topk", _i32),
        ("batch", _i32), ("total_q", _i32), ("max_q_len", _i32), ("max_kv_len", _i32),
        ("total_mask_words", _i32),
        ("qo_indptr", _P), ("kv_indptr", _P), ("prefix_len", _P), ("mask_indptr", _P),
        ("q", _P), ("kv_pool", _P), ("pool_rows", ctypes.c_int64), ("kv_indices", _P),
        ("num_heads", _i32), ("scale", ctypes.c_float), ("num_splits", _i32),
        ("workspace", _P), ("workspace_bytes", ctypes.c_size_t),
        ("target_argmax", _P),
        ("node_token", _P), ("parent", _P), ("depth", _P), ("mask", _P), ("out", _P), ("lse", _P),
        ("accept_len", _P), ("accepted_nodes", _P), ("commit_tokens", _P), ("bonus", _P),
        ("commit_kv", _i32), ("new_len", _P),
    ]


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn, st):
    if st != 0:
        raise DDTError(fn, st)


def _dev(t, dtype, name):
    if not (t.is_cuda and t.dtype == dtype and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")
    return t


def abi_version() -> int:
    return lib.ddt_abi_version()


def ddt_build_tree(topk_logp, topk_ids, root_id, budget, qo_indptr, node_token, parent, depth,
                   stream=None):
    B, max_depth, K = topk_logp.shape
    _dev(topk_logp, torch.float32, "topk_logp")
    for n, t in (("topk_ids", topk_ids), ("root_id", root_id), ("budget", budget),
                 ("qo_indptr", qo_indptr), ("node_token", node_token), ("parent", parent),
                 ("depth", depth)):
        _dev(t, torch.int32, n)
    _check("ddt_build_tree", lib.ddt_build_tree(
        _p(topk_logp), _p(topk_ids), _p(root_id), _p(budget), _p(qo_indptr), B, max_depth, K,
        _p(node_token), _p(parent), _p(depth), _stream(stream)))


def ddt_mask_indptr(qo_indptr_host, prefix_len_host):
    """Host helper: int32 word offsets of the bit-packed mask (CPU tensors in/out)."""
    qo = qo_indptr_host.to(torch.int32).contiguous().cpu()
    pl = prefix_len_host.to(torch.int32).contiguous().cpu()
    out = torch.empty(pl.numel() + 1, dtype=torch.int32)
    _check("ddt_mask_indptr", lib.ddt_mask_indptr(_p(qo), _p(pl), pl.numel(), _p(out)))
    return out


def ddt_compile_visibility(parent, qo_indptr, prefix_len, mask_indptr, mask, stream=None):
    for n, t in (("parent", parent), ("qo_indptr", qo_indptr), ("prefix_len", prefix_len),
                 ("mask_indptr", mask_indptr)):
        _dev(t, torch.int32, n)
    if not (mask.is_cuda and mask.dtype in (torch.int32, torch.uint32) and mask.is_contiguous()):
        raise ValueError("mask must be a contiguous CUDA 32-bit tensor")
    B = prefix_len.numel()
    _check("ddt_compile_visibility", lib.ddt_compile_visibility(
        _p(parent), _p(qo_indptr), _p(prefix_len), _p(mask_indptr), B, mask.numel(), _p(mask),
        _stream(stream)))


def ddt_build_chain_visibility(qo_indptr, prefix_len, mask_indptr, parent, depth, mask,
                               stream=None):
    """A prefill chunk's chain (parent[i] = i - 1, depth[i] = i) and its causal mask."""
    for n, t in (("qo_indptr", qo_indptr), ("prefix_len", prefix_len), ("mask_indptr", mask_indptr),
                 ("parent", parent), ("depth", depth)):
        _dev(t, torch.int32, n)
    if not (mask.is_cuda and mask.dtype in (torch.int32, torch.uint32) and mask.is_contiguous()):
        raise ValueError("mask must be a contiguous CUDA 32-bit tensor")
    B = prefix_len.numel()
    if qo_indptr.numel() != B + 1 or mask_indptr.numel() != B + 1:
        raise ValueError("qo_indptr and mask_indptr must hold batch + 1 offsets")
    if parent.numel() != depth.numel():
        raise ValueError("parent and depth must have the same length")
    _check("ddt_build_chain_visibility", lib.ddt_build_chain_visibility(
        _p(qo_indptr), _p(prefix_len), _p(mask_indptr), B, _p(parent), _p(depth), _p(mask),
        _stream(stream)))


def ddt_build_tree_visibility(topk_logp, topk_ids, root_id, budget, qo_indptr, prefix_len,
                              mask_indptr, node_token, parent, depth, mask, stream=None):
    """ddt_build_tree and ddt_compile_visibility in one launch (same outputs)."""
    B, max_depth, K = topk_logp.shape
    _dev(topk_logp, torch.float32, "topk_logp")
    for n, t in (("topk_ids", topk_ids), ("root_id", root_id), ("budget", budget),
                 ("qo_indptr", qo_indptr), ("prefix_len", prefix_len), ("mask_indptr", mask_indptr),
                 ("node_token", node_token), ("parent", parent), ("depth", depth)):
        _dev(t, torch.int32, n)
    if not (mask.is_cuda and mask.dtype in (torch.int32, torch.uint32) and mask.is_contiguous()):
        raise ValueError("mask must be a contiguous CUDA 32-bit tensor")
    _check("ddt_build_tree_visibility", lib.ddt_build_tree_visibility(
        _p(topk_logp), _p(topk_ids), _p(root_id), _p(budget), _p(qo_indptr), _p(prefix_len),
        _p(mask_indptr), B, max_depth, K, _p(node_token), _p(parent), _p(depth), _p(mask),
        _stream(stream)))


def ddt_verify_attn_num_splits(batch, num_heads, max_q_len, max_kv_len, num_sms=0):
    return lib.ddt_verify_attn_num_splits(batch, num_heads, max_q_len, max_kv_len, num_sms)


def ddt_verify_attn_launched_splits(max_kv_len, num_splits):
    """Splits a ddt_verify_attn call with num_splits (>= 1) launches (the
    requested count rounded to whole 64-column tiles)."""
    return lib.ddt_verify_attn_launched_splits(int(max_kv_len), int(num_splits))


def ddt_verify_attn_noalloc_splits(batch, num_heads, total_q, max_q_len, max_kv_len, num_splits=0):
    """Splits a ddt_verify_attn_noalloc call with these sizes launches."""
    return lib.ddt_verify_attn_noalloc_splits(int(batch), int(num_heads), int(total_q),
                                              int(max_q_len), int(max_kv_len), int(num_splits))


def ddt_verify_attn_workspace_size(total_q, num_heads, num_splits):
    return lib.ddt_verify_attn_workspace_size(total_q, num_heads, num_splits)


def _attn_args(q, kv_pool, kv_indices, kv_indptr, qo_indptr, mask, mask_indptr, out, lse,
               max_q_len, max_kv_len):
    """The checks both attention entry points need (the C ABI cannot see tensor
    shapes): dtypes, contiguity, 576-wide rows, out [total_q, H, 512], lse
    [total_q, H]; returns (total_q, H, batch, max_q_len, max_kv_len)."""
    _dev(q, torch.bfloat16, "q")
    _dev(kv_pool, torch.bfloat16, "kv_pool")
    _dev(out, torch.float32, "out")
    for n, t in (("kv_indices", kv_indices), ("kv_indptr", kv_indptr), ("qo_indptr", qo_indptr),
                 ("mask_indptr", mask_indptr)):
        _dev(t, torch.int32, n)
    if not (mask.is_cuda and mask.dtype in (torch.int32, torch.uint32) and mask.is_contiguous()):
        raise ValueError("mask must be a contiguous CUDA 32-bit tensor")
    if q.dim() != 3 or kv_pool.dim() != 2:
        raise ValueError("q must be [total_q, H, 576] and kv_pool [pool_rows, 576]")
    total_q, H, d = q.shape
    if d != D or kv_pool.shape[-1] != D or tuple(out.shape) != (total_q, H, DL):
        raise ValueError("q/kv_pool rows must be 576 wide and out [total_q, H, 512]")
    if lse is not None:
        _dev(lse, torch.float32, "lse")
        if tuple(lse.shape) != (total_q, H):
            raise ValueError("lse must be [total_q, H]")
    B = qo_indptr.numel() - 1
    if kv_indptr.numel() != B + 1 or mask_indptr.numel() != B + 1:
        raise ValueError("qo_indptr, kv_indptr and mask_indptr must all hold batch + 1 entries")
    if max_q_len is None or max_kv_len is None:
        qo = qo_indptr.cpu()
        kv = kv_indptr.cpu()
        max_q_len = int((qo[1:] - qo[:-1]).max())
        max_kv_len = int((kv[1:] - kv[:-1]).max())
    return total_q, H, B, int(max_q_len), int(max_kv_len)


def ddt_verify_attn(q, kv_pool, kv_indices, kv_indptr, qo_indptr, mask, mask_indptr, scale,
                    out, lse=None, max_q_len=None, max_kv_len=None, num_splits=0,
                    workspace=None, stream=None):
    """q: [total_q, H, 576] bf16; kv_pool: [pool_rows, 576] bf16; out: [total_q, H, 512] f32.

    max_q_len / max_kv_len are host-side bounds used to size the grid; when
    omitted they are read from the indptrs (a device->host copy)."""
    total_q, H, B, max_q_len, max_kv_len = _attn_args(q, kv_pool, kv_indices, kv_indptr, qo_indptr,
                                                      mask, mask_indptr, out, lse, max_q_len,
                                                      max_kv_len)
    if workspace is None:
        splits = num_splits or ddt_verify_attn_num_splits(B, H, max_q_len, max_kv_len)
        nbytes = ddt_verify_attn_workspace_size(total_q, H, splits)
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device) if nbytes else None
        num_splits = splits
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("ddt_verify_attn", lib.ddt_verify_attn(
        _p(q), _p(kv_pool), kv_pool.shape[0], _p(kv_indices), _p(kv_indptr), _p(qo_indptr),
        _p(mask), _p(mask_indptr), B, H, total_q, int(max_q_len), int(max_kv_len), float(scale),
        int(num_splits), _p(out), _p(lse), _p(workspace), ws_bytes, _stream(stream)))


NOALLOC_SCRATCH_BYTES = 32 << 20


def ddt_verify_attn_noalloc(q, kv_pool, kv_indices, kv_indptr, qo_indptr, mask, mask_indptr,
                            scale, out, lse=None, max_q_len=None, max_kv_len=None, num_splits=0,
                            stream=None):
    """ddt_verify_attn for callers that cannot allocate device memory (a
    pre-reserved engine pool, a host without an allocator, a loop where a
    device-synchronising cudaMalloc is not allowed): the split scratch is a
    fixed 32 MiB array inside libddt.so, so neither this wrapper nor the call
    allocates on the device.  Calls overlapping on the GPU race on that
    array.  num_splits = 0 takes the library's choice among the counts that
    fit the array; an explicit count that needs more scratch than the array
    holds raises DDTError(DDT_ERR_WORKSPACE)."""
    total_q, H, B, max_q_len, max_kv_len = _attn_args(q, kv_pool, kv_indices, kv_indptr, qo_indptr,
                                                      mask, mask_indptr, out, lse, max_q_len,
                                                      max_kv_len)
    _check("ddt_verify_attn_noalloc", lib.ddt_verify_attn_noalloc(
        _p(q), _p(kv_pool), kv_pool.shape[0], _p(kv_indices), _p(kv_indptr), _p(qo_indptr),
        _p(mask), _p(mask_indptr), B, H, total_q, int(max_q_len), int(max_kv_len), float(scale),
        int(num_splits), _p(out), _p(lse), _stream(stream)))


def ddt_accept(node_token, parent, qo_indptr, target_argmax, max_depth, accept_len,
               accepted_nodes, commit_tokens, bonus, stream=None):
    for n, t in (("node_token", node_token), ("parent", parent), ("qo_indptr", qo_indptr),
                 ("target_argmax", target_argmax), ("accept_len", accept_len),
                 ("accepted_nodes", accepted_nodes), ("commit_tokens", commit_tokens),
                 ("bonus", bonus)):
        _dev(t, torch.int32, n)
    B = qo_indptr.numel() - 1
    _check("ddt_accept", lib.ddt_accept(
        _p(node_token), _p(parent), _p(qo_indptr), _p(target_argmax), B, int(max_depth),
        _p(accept_len), _p(accepted_nodes), _p(commit_tokens), _p(bonus), _stream(stream)))


def ddt_commit_kv(kv_pool, kv_indices, kv_indptr, qo_indptr, accept_len, accepted_nodes, max_depth,
                  new_len=None, stream=None):
    """KV commit: gathers each request's accepted latents into positions
    P .. P + accept_len - 1 of its sequence, in place in kv_pool."""
    _dev(kv_pool, torch.bfloat16, "kv_pool")
    for n, t in (("kv_indices", kv_indices), ("kv_indptr", kv_indptr), ("qo_indptr", qo_indptr),
                 ("accept_len", accept_len), ("accepted_nodes", accepted_nodes)):
        _dev(t, torch.int32, n)
    if new_len is not None:
        _dev(new_len, torch.int32, "new_len")
    B = qo_indptr.numel() - 1
    _check("ddt_commit_kv", lib.ddt_commit_kv(
        _p(kv_pool), kv_pool.shape[0], _p(kv_indices), _p(kv_indptr), _p(qo_indptr),
        _p(accept_len), _p(accepted_nodes), B, int(max_depth), _p(new_len), _stream(stream)))


def ddt_verify_step(args: StepArgs, stream=None):
    """One verify step in one call (tree + mask, attention, accept, optional commit)."""
    _check("ddt_verify_step", lib.ddt_verify_step(ctypes.byref(args), _stream(stream)))


def ddt_prefill_step(args: StepArgs, stream=None):
    """One prefill chunk in one call (causal chain + mask, attention)."""
    _check("ddt_prefill_step", lib.ddt_prefill_step(ctypes.byref(args), _stream(stream)))


class StepGraph:
    """A library-owned CUDA graph of one ddt_verify_step; the tensors behind
    `args` must outlive it."""

    def __init__(self, args: StepArgs, keep_alive=(), io=None):
        """io = (h_in, d_in, h_out, d_out): pinned host and device uint8 buffers;
        the graph then copies h_in -> d_in before the step and d_out -> h_out
        after it (ddt_step_graph_create_io)."""
        self._keep = (args, tuple(keep_alive), io)
        h = ctypes.c_void_p()
        if io is None:
            _check("ddt_step_graph_create",
                   lib.ddt_step_graph_create(ctypes.byref(args), ctypes.byref(h)))
        else:
            h_in, d_in, h_out, d_out = io
            for t, dev, n in ((h_in, False, "h_in"), (d_in, True, "d_in"), (h_out, False, "h_out"),
                              (d_out, True, "d_out")):
                if t.is_cuda != dev or not t.is_contiguous() or (not dev and not t.is_pinned()):
                    raise ValueError(f"{n} must be a contiguous {'CUDA' if dev else 'pinned host'} "
                                     "tensor")
            nin = h_in.numel() * h_in.element_size()
            nout = h_out.numel() * h_out.element_size()
            if nin > d_in.numel() * d_in.element_size() or nout > d_out.numel() * d_out.element_size():
                raise ValueError("a host buffer is larger than its device buffer")
            _check("ddt_step_graph_create_io", lib.ddt_step_graph_create_io(
                ctypes.byref(args), _p(h_in), _p(d_in), nin, _p(h_out), _p(d_out), nout,
                ctypes.byref(h)))
        self._h = h

    def launch(self, stream=None):
        _check("ddt_step_graph_launch", lib.ddt_step_graph_launch(self._h, _stream(stream)))

    def close(self):
        if self._h:
            _check("ddt_step_graph_destroy", lib.ddt_step_graph_destroy(self._h))
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def ddt_tree_links(parent, qo_indptr, first_child, next_sibling, retrieve_index, stream=None):
    """The tree as (first_child, next_sibling, retrieve_index) links."""
    for n, t in (("parent", parent), ("qo_indptr", qo_indptr), ("first_child", first_child),
                 ("next_sibling", next_sibling), ("retrieve_index", retrieve_index)):
        _dev(t, torch.int32, n)
    _check("ddt_tree_links", lib.ddt_tree_links(
        _p(parent), _p(qo_indptr), qo_indptr.numel() - 1, _p(first_child), _p(next_sibling),
        _p(retrieve_index), _stream(stream)))


def ddt_accept_sampled(node_token, first_child, next_sibling, qo_indptr, target_logits,
                       temperature, top_k, coins, max_depth, accept_len, accepted_nodes,
                       commit_tokens, bonus, stream=None, top_p=None):
    """Sampling accept: tree rejection sampling with temperature, top-k and top-p.
    target_logits float32 [rows, vocab]; temperature float32 [B]; top_k int32 [B];
    coins float32 [rows, coin_stride] uniform in [0, 1); top_p float32 [B] or None."""
    _dev(target_logits, torch.float32, "target_logits")
    _dev(temperature, torch.float32, "temperature")
    _dev(coins, torch.float32, "coins")
    for n, t in (("node_token", node_token), ("first_child", first_child),
                 ("next_sibling", next_sibling), ("qo_indptr", qo_indptr), ("top_k", top_k),
                 ("accept_len", accept_len), ("accepted_nodes", accepted_nodes),
                 ("commit_tokens", commit_tokens), ("bonus", bonus)):
        _dev(t, torch.int32, n)
    B = qo_indptr.numel() - 1
    if top_p is not None:
        _dev(top_p, torch.float32, "top_p")
        if top_p.numel() != B:
            raise ValueError("top_p must hold one value per request")
    if temperature.numel() != B or top_k.numel() != B:
        raise ValueError("temperature and top_k must hold one value per request")
    _check("ddt_accept_sampled", lib.ddt_accept_sampled(
        _p(node_token), _p(first_child), _p(next_sibling), _p(qo_indptr), _p(target_logits),
        target_logits.shape[1], _p(temperature), _p(top_k), _p(top_p), _p(coins), coins.shape[1], B,
        int(max_depth), _p(accept_len), _p(accepted_nodes), _p(commit_tokens), _p(bonus),
        _stream(stream)))


# ---------------------------------------------------------------- grouped-query layers, cache rows
def _on_device(first, name):
    """The CUDA device a call runs on: its first tensor's, which has to be the current one."""
    dev = first.device
    if dev.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {dev}, which is not the current device")
    return dev


def _like(t, dtype, dev, name):
    if t.dtype is not dtype or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on {dev}")
    return t.data_ptr()


def _mask_ptr(mask, dev):
    if mask.dtype not in (torch.int32, torch.uint32) or mask.device != dev or not mask.is_contiguous():
        raise ValueError(f"mask must be a contiguous 32-bit tensor on {dev}")
    return mask.data_ptr()


def _heads(t, dev, name, heads=None):
    """Pointer, row stride, rows, heads and head_dim of a [rows, heads, head_dim] bf16 tensor
    whose rows are contiguous (the rows themselves may be apart)."""
    shape = t.shape
    if t.dtype is not _BF16 or t.device != dev or len(shape) != 3:
        raise ValueError(f"{name} must be a [rows, heads, head_dim] bfloat16 tensor on {dev}")
    n, h, d = shape
    sn, sh, sd = t.stride()
    if (sd != 1 and d > 1) or (sh != d and h > 1):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    if heads is not None and (h, d) != heads:
        raise ValueError(f"{name} must have {heads[0]} heads of {heads[1]} values")
    return t.data_ptr(), (sn if n > 1 else h * d), n, h, d


def _pools(k_pool, v_pool, dev):
    kp, stride, rows, G, D = _heads(k_pool, dev, "k_pool")
    vp, vstride, vrows, _, _ = _heads(v_pool, dev, "v_pool", (G, D))
    if vrows != rows or vstride != stride:
        raise ValueError("k_pool and v_pool must have the same rows at the same stride")
    return kp, vp, stride, rows, G, D


def _raw_stream(stream, dev):
    # the raw handle of the current stream without a Stream object around it
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev.index)


def _scratch(nbytes, dev, stream):
    """A workspace of one call: the caching allocator may give its memory away again once the
    call's own stream is past it, so it is allocated on that stream."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)


def ddt_gqa_norm_rope_append(q, k, v, q_weight, k_weight, eps, cos_sin, depth, qo_indptr, kv_indices,
                             kv_indptr, q_out, k_pool, v_pool, interleaved=False, stream=None):
    """Norm, rotation and cache append of a grouped-query layer in one pass.

    q [total_q, H, D], k and v [total_q, G, D] bf16 (rows contiguous; slices of one projection
    will do); q_weight / k_weight bf16 [D] or None (no norm); cos_sin float32 [max_pos, rope_dim]
    (cosines, then sines) or None (no rotation); depth int32 [total_q] or None (a chain);
    q_out [total_q, H, D] contiguous, may be q; k_pool, v_pool [pool_rows, G, D]."""
    dev = _on_device(q, "q")
    qp, qs, total_q, H, D = _heads(q, dev, "q")
    kp, ks, nk, G, _ = _heads(k, dev, "k")
    vp, vs, nv, _, _ = _heads(v, dev, "v", (G, D))
    kpp, vpp, stride, rows, Gp, Dp = _pools(k_pool, v_pool, dev)
    if nk != total_q or nv != total_q or k.shape[2] != D or (Gp, Dp) != (G, D):
        raise ValueError("q, k, v and the pools must agree in tokens, K/V heads and head_dim")
    if q_out.shape != (total_q, H, D):
        raise ValueError("q_out must have q's shape")
    for n, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and w.numel() != D:
            raise ValueError(f"{n} must hold head_dim values")
    max_pos, rope_dim = 0, 0
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [max_pos, rope_dim]")
        max_pos, rope_dim = cos_sin.shape
    B = qo_indptr.numel() - 1
    if kv_indptr.numel() != B + 1:
        raise ValueError("qo_indptr and kv_indptr must both hold batch + 1 entries")
    if depth is not None and depth.numel() < total_q:
        raise ValueError("depth must hold an entry per token")
    if total_q == 0 or B == 0:
        return
    i32, bf16 = _I32, _BF16
    _call(
        "ddt_gqa_norm_rope_append", qp, qs, kp, ks, vp, vs,
        0 if q_weight is None else _like(q_weight, bf16, dev, "q_weight"),
        0 if k_weight is None else _like(k_weight, bf16, dev, "k_weight"), eps,
        0 if cos_sin is None else _like(cos_sin, torch.float32, dev, "cos_sin"), max_pos, rope_dim,
        int(bool(interleaved)), 0 if depth is None else _like(depth, i32, dev, "depth"),
        _like(qo_indptr, i32, dev, "qo_indptr"), _like(kv_indices, i32, dev, "kv_indices"),
        _like(kv_indptr, i32, dev, "kv_indptr"), B, total_q, kv_indices.numel(), H, G, D,
        _like(q_out, bf16, dev, "q_out"), kpp, vpp, stride, rows, _raw_stream(stream, dev))


def ddt_gqa_verify_attn_num_ctas(batch, num_heads, num_kv_heads, max_q_len, max_kv_len, num_sms=0):
    return lib.ddt_gqa_verify_attn_num_ctas(batch, num_heads, num_kv_heads, max_q_len, max_kv_len, num_sms)


def ddt_gqa_verify_attn_workspace_size(batch, num_heads, num_kv_heads, head_dim, max_q_len, num_ctas):
    return lib.ddt_gqa_verify_attn_workspace_size(batch, num_heads, num_kv_heads, head_dim, max_q_len, num_ctas)


def ddt_gqa_verify_attn(q, k_pool, v_pool, kv_indices, kv_indptr, qo_indptr, mask, mask_indptr, scale,
                        out, lse=None, max_q_len=None, max_kv_len=None, num_ctas=0, workspace=None,
                        stream=None):
    """Tree-verify attention over grouped-query rows.  q, out: [total_q, H, D] bf16; k_pool, v_pool:
    [pool_rows, G, D] bf16 (rows may be apart: slices of one [pool_rows, 2, G, D] pool will do);
    lse: float32 [total_q, H] or None.

    max_q_len / max_kv_len are host-side bounds; when omitted they are read from the indptrs (a
    device->host copy).  num_ctas: the CTAs that the cached columns are dealt to (0 = choose, within
    what `workspace` holds); without a workspace, the count's workspace is allocated here."""
    dev = _on_device(q, "q")
    qp, qs, total_q, H, D = _heads(q, dev, "q")
    kp, vp, stride, rows, G, Dp = _pools(k_pool, v_pool, dev)
    if Dp != D:
        raise ValueError("q and the pools must have the same head_dim")
    if qs != H * D:
        raise ValueError("q must be contiguous")
    if out.shape != (total_q, H, D):
        raise ValueError("out must have q's shape")
    if lse is not None and lse.shape != (total_q, H):
        raise ValueError("lse must be [total_q, H]")
    B = qo_indptr.numel() - 1
    if kv_indptr.numel() != B + 1 or mask_indptr.numel() != B + 1:
        raise ValueError("qo_indptr, kv_indptr and mask_indptr must all hold batch + 1 entries")
    if total_q == 0 or B == 0:
        return
    if max_q_len is None or max_kv_len is None:
        with torch.cuda.stream(stream):   # behind what writes them there
            max_q_len = int((qo_indptr[1:] - qo_indptr[:-1]).max())
            max_kv_len = int((kv_indptr[1:] - kv_indptr[:-1]).max())
    if workspace is None:
        ctas = num_ctas or lib.ddt_gqa_verify_attn_num_ctas(B, H, G, max_q_len, max_kv_len, 0)
        nbytes = lib.ddt_gqa_verify_attn_workspace_size(B, H, G, D, max_q_len, ctas)
        if nbytes:
            workspace = _scratch(nbytes, dev, stream)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    ws, ws_bytes = (0, 0) if workspace is None else (workspace.data_ptr(),
                                                     workspace.numel() * workspace.element_size())
    i32, bf16 = _I32, _BF16
    _call(
        "ddt_gqa_verify_attn", qp, kp, vp, stride, rows, _like(kv_indices, i32, dev, "kv_indices"),
        _like(kv_indptr, i32, dev, "kv_indptr"), _like(qo_indptr, i32, dev, "qo_indptr"),
        _mask_ptr(mask, dev), _like(mask_indptr, i32, dev, "mask_indptr"), B, H, G, D, total_q,
        kv_indices.numel(), mask.numel(), max_q_len, max_kv_len, scale, num_ctas,
        _like(out, bf16, dev, "out"), 0 if lse is None else _like(lse, torch.float32, dev, "lse"),
        ws, ws_bytes, _raw_stream(stream, dev))


def _slab(t, dev, name):
    """Pointer, bytes between pools, rows, pools and row bytes of a [pools, rows, ...] tensor whose
    pools are contiguous (the pools themselves may be apart)."""
    shape, es = t.shape, t.element_size()
    if len(shape) < 3 or t.device != dev:
        raise ValueError(f"{name} must be a [pools, rows, ...] tensor on {dev}")
    if t.is_contiguous() and 0 not in shape:
        pools, rows = shape[0], shape[1]
        row = t.numel() // (pools * rows) * es
        return t.data_ptr(), rows * row, rows, pools, row
    strides = t.stride()
    size = 1   # values of the dimensions walked so far, innermost first
    for n, s in zip(shape[:1:-1], strides[:1:-1]):
        if n != 1 and s != size:
            raise ValueError(f"{name}: every pool must be contiguous")
        size *= n
    pools, rows = shape[0], shape[1]
    if pools == 0 or rows == 0 or size == 0 or (rows != 1 and strides[1] != size):
        raise ValueError(f"{name}: every pool must be contiguous and hold a row")
    row = size * es
    return t.data_ptr(), (strides[0] * es if pools > 1 else rows * row), rows, pools, row


def ddt_cache_copy(src_pool, dst_pool, src, dst, stream=None):
    """Row dst[i] of every dst pool <- row src[i] of the same src pool.  src_pool, dst_pool:
    [pools, rows, ...] (one pool per layer, or one for K and one for V per layer; may be the same
    tensor); src, dst: int32 [n]."""
    dev = _on_device(src_pool, "src_pool")
    sp, sgap, srows, pools, row = _slab(src_pool, dev, "src_pool")
    dp, dgap, drows = sp, sgap, srows
    if dst_pool is not src_pool:
        dp, dgap, drows, dpools, drow = _slab(dst_pool, dev, "dst_pool")
        if dpools != pools or drow != row or src_pool.dtype != dst_pool.dtype:
            raise ValueError("src_pool and dst_pool must agree in pools, row and type")
    n = src.numel()
    if dst.numel() != n:
        raise ValueError("src and dst must have the same length")
    if n == 0:
        return
    _call(
        "ddt_cache_copy", sp, sgap, srows, dp, dgap, drows, pools, row, _like(src, _I32, dev, "src"),
        _like(dst, _I32, dev, "dst"), n, _raw_stream(stream, dev))


def ddt_cache_commit(pool, kv_indices, kv_indptr, qo_indptr, accept_len, accepted_nodes, max_depth,
                     new_len=None, stream=None):
    """KV commit in every pool of a [pools, rows, ...] tensor: each request's accepted rows gathered
    into positions P .. P + accept_len - 1 of its sequence, in place."""
    dev = _on_device(pool, "pool")
    pp, gap, rows, pools, row = _slab(pool, dev, "pool")
    B = qo_indptr.numel() - 1
    if kv_indptr.numel() != B + 1 or accept_len.numel() != B or accepted_nodes.numel() != B * (max_depth + 1):
        raise ValueError("kv_indptr, accept_len and accepted_nodes must match the batch and max_depth")
    if new_len is not None and new_len.numel() != B:
        raise ValueError("new_len must hold one value per request")
    if B == 0:
        return
    i32 = _I32
    _call(
        "ddt_cache_commit", pp, gap, rows, pools, row, _like(kv_indices, i32, dev, "kv_indices"),
        _like(kv_indptr, i32, dev, "kv_indptr"), _like(qo_indptr, i32, dev, "qo_indptr"),
        _like(accept_len, i32, dev, "accept_len"), _like(accepted_nodes, i32, dev, "accepted_nodes"),
        B, kv_indices.numel(), max_depth, 0 if new_len is None else _like(new_len, i32, dev, "new_len"),
        _raw_stream(stream, dev))


def ddt_cache_compact_workspace_size(pool_rows):
    return lib.ddt_cache_compact_workspace_size(pool_rows)


def ddt_cache_compact(pool, kv_indices, new_indices, live, workspace=None, stream=None):
    """The rows named by kv_indices moved to the front of every pool of a [pools, rows, ...] tensor;
    new_indices (may be kv_indices) receives their numbers, live (int32 [1]) how many they are."""
    dev = _on_device(pool, "pool")
    pp, gap, rows, pools, row = _slab(pool, dev, "pool")
    if new_indices.numel() != kv_indices.numel() or live.numel() != 1:
        raise ValueError("new_indices must have kv_indices' length, live one entry")
    if workspace is None:
        workspace = _scratch(max(1, lib.ddt_cache_compact_workspace_size(rows)), dev, stream)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    i32 = _I32
    _call(
        "ddt_cache_compact", pp, gap, rows, pools, row, _like(kv_indices, i32, dev, "kv_indices"), kv_indices.numel(),
        _like(new_indices, i32, dev, "new_indices"), _like(live, i32, dev, "live"), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _raw_stream(stream, dev))


# ---------------------------------------------------------------- chunks
MAX_CHUNK = 1 << 20


def _bounds(qo_indptr, kv_indptr, max_q_len, max_kv_len, stream):
    """Host-side bounds; read on the call's stream (behind what writes the offsets) where not given."""
    if max_q_len is None or max_kv_len is None:
        with torch.cuda.stream(stream):
            max_q_len = int((qo_indptr[1:] - qo_indptr[:-1]).max())
            max_kv_len = int((kv_indptr[1:] - kv_indptr[:-1]).max())
    return max_q_len, max_kv_len


def _scores(slopes, full_len, H, B, dev):
    """Pointers of what the chunk calls' scores and visibility take."""
    if slopes is not None and slopes.numel() != H:
        raise ValueError("slopes must hold a value per head")
    if full_len is not None and full_len.numel() != B:
        raise ValueError("full_len must hold a value per request")
    return (0 if slopes is None else _like(slopes, torch.float32, dev, "slopes"),
            0 if full_len is None else _like(full_len, _I32, dev, "full_len"))


def _workspace(workspace, nbytes, dev, stream):
    """Pointer and bytes of the caller's workspace, or of one allocated here (returned to be kept)."""
    if workspace is None:
        if not nbytes:
            return None, 0, 0
        workspace = _scratch(nbytes, dev, stream)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def ddt_gqa_chunk_attn_num_ctas(batch, num_heads, num_kv_heads, max_q_len, max_kv_len, num_sms=0):
    return lib.ddt_gqa_chunk_attn_num_ctas(batch, num_heads, num_kv_heads, max_q_len, max_kv_len, num_sms)


def ddt_gqa_chunk_attn_workspace_size(num_heads, num_kv_heads, head_dim, max_q_len, num_ctas):
    return lib.ddt_gqa_chunk_attn_workspace_size(num_heads, num_kv_heads, head_dim, max_q_len, num_ctas)


def ddt_gqa_chunk_attn(q, k_pool, v_pool, kv_indices, kv_indptr, qo_indptr, scale, out, lse=None,
                       max_q_len=None, max_kv_len=None, score_cap=0.0, slopes=None, window=0, full_len=None,
                       num_ctas=0, workspace=None, stream=None):
    """Attention of a chunk of new tokens of any length over grouped-query rows.  q, out: [total_q, H, D]
    bf16; k_pool, v_pool: [pool_rows, G, D] bf16; lse: float32 [total_q, H] or None.

    Token i of a request is at position p = kv_len - q_len + i and sees the columns j < full_len[b]
    (int32 [batch] or None) and p - window < j <= p (window 0: all up to p).  Scores are capped to
    score_cap * tanh(z / score_cap) where score_cap > 0, then reduced by slopes[h] * |p - j| (float32 [H] or
    None).  The other arguments are those of ddt_gqa_verify_attn."""
    dev = _on_device(q, "q")
    qp, qs, total_q, H, D = _heads(q, dev, "q")
    kp, vp, stride, rows, G, Dp = _pools(k_pool, v_pool, dev)
    if Dp != D:
        raise ValueError("q and the pools must have the same head_dim")
    if qs != H * D:
        raise ValueError("q must be contiguous")
    if out.shape != (total_q, H, D):
        raise ValueError("out must have q's shape")
    if lse is not None and lse.shape != (total_q, H):
        raise ValueError("lse must be [total_q, H]")
    B = qo_indptr.numel() - 1
    if kv_indptr.numel() != B + 1:
        raise ValueError("qo_indptr and kv_indptr must both hold batch + 1 entries")
    slopes_p, full_p = _scores(slopes, full_len, H, B, dev)
    if total_q == 0 or B == 0:
        return
    max_q_len, max_kv_len = _bounds(qo_indptr, kv_indptr, max_q_len, max_kv_len, stream)
    nbytes = 0
    if workspace is None:
        ctas = num_ctas or lib.ddt_gqa_chunk_attn_num_ctas(B, H, G, max_q_len, max_kv_len, 0)
        nbytes = lib.ddt_gqa_chunk_attn_workspace_size(H, G, D, max_q_len, ctas)
    workspace, ws, ws_bytes = _workspace(workspace, nbytes, dev, stream)
    i32 = _I32
    _call(
        "ddt_gqa_chunk_attn", qp, kp, vp, stride, rows, _like(kv_indices, i32, dev, "kv_indices"),
        _like(kv_indptr, i32, dev, "kv_indptr"), _like(qo_indptr, i32, dev, "qo_indptr"), B, H, G, D, total_q,
        kv_indices.numel(), max_q_len, max_kv_len, scale, score_cap, slopes_p, window, full_p, num_ctas,
        _like(out, _BF16, dev, "out"), 0 if lse is None else _like(lse, torch.float32, dev, "lse"),
        ws, ws_bytes, _raw_stream(stream, dev))


def ddt_gqa_chunk_weights_num_ctas(batch, num_sms=0):
    return lib.ddt_gqa_chunk_weights_num_ctas(batch, num_sms)


def ddt_gqa_chunk_weights_workspace_size(num_ctas):
    return lib.ddt_gqa_chunk_weights_workspace_size(num_ctas)


def ddt_gqa_chunk_weights(q, k_pool, lse, kv_indices, kv_indptr, qo_indptr, scale, weights, prev=None,
                          prev_indptr=None, decay=1.0, last_rows=0, max_q_len=None, max_kv_len=None, score_cap=0.0,
                          slopes=None, window=0, full_len=None, num_ctas=0, workspace=None, stream=None):
    """How much attention every column received from a chunk: weights (float32, an entry per entry of
    kv_indices) = decay * prev + the sum over heads and tokens of the softmax's weights, given the chunk
    attention's arguments and its lse (float32 [total_q, H]).

    last_rows: only that many last tokens of a request count (0: all).  prev: float32 sums of earlier
    steps, of each request's first columns by prev_indptr (int32 [batch + 1]; None: laid out as weights,
    and then maybe weights itself: the layers of a step add up)."""
    dev = _on_device(q, "q")
    qp, qs, total_q, H, D = _heads(q, dev, "q")
    kp, stride, rows, G, Dp = _heads(k_pool, dev, "k_pool")
    if Dp != D:
        raise ValueError("q and k_pool must have the same head_dim")
    if qs != H * D:
        raise ValueError("q must be contiguous")
    if lse.shape != (total_q, H):
        raise ValueError("lse must be [total_q, H]")
    if weights.numel() != kv_indices.numel():
        raise ValueError("weights must hold a value per entry of kv_indices")
    B = qo_indptr.numel() - 1
    if kv_indptr.numel() != B + 1 or (prev_indptr is not None and prev_indptr.numel() != B + 1):
        raise ValueError("qo_indptr, kv_indptr and prev_indptr must all hold batch + 1 entries")
    if prev is not None and prev_indptr is None and prev.numel() != weights.numel():
        raise ValueError("prev must be laid out as weights, or come with prev_indptr")
    slopes_p, full_p = _scores(slopes, full_len, H, B, dev)
    if kv_indices.numel() == 0 or B == 0:
        return
    max_q_len, max_kv_len = _bounds(qo_indptr, kv_indptr, max_q_len, max_kv_len, stream)
    nbytes = 0
    if workspace is None:
        nbytes = lib.ddt_gqa_chunk_weights_workspace_size(num_ctas or lib.ddt_gqa_chunk_weights_num_ctas(B, 0))
    workspace, ws, ws_bytes = _workspace(workspace, nbytes, dev, stream)
    i32, f32 = _I32, torch.float32
    _call(
        "ddt_gqa_chunk_weights", qp, kp, stride, rows, _like(lse, f32, dev, "lse"),
        _like(kv_indices, i32, dev, "kv_indices"), _like(kv_indptr, i32, dev, "kv_indptr"),
        _like(qo_indptr, i32, dev, "qo_indptr"), B, H, G, D, total_q, kv_indices.numel(), max_q_len, max_kv_len, scale,
        score_cap, slopes_p, window, full_p, last_rows, 0 if prev is None else _like(prev, f32, dev, "prev"),
        0 if prev is None or prev_indptr is None else _like(prev_indptr, i32, dev, "prev_indptr"),
        0 if prev is None else prev.numel(), decay, num_ctas, _like(weights, f32, dev, "weights"), ws, ws_bytes,
        _raw_stream(stream, dev))


def ddt_cache_evict(weights, kv_indices, kv_indptr, budget, new_indices, new_indptr, new_weights=None,
                    evicted=None, sinks=0, recent=0, max_kv_len=None, stream=None):
    """Per request the budget[b] (int32 [batch]) columns with the largest weights stay, its first `sinks`
    and last `recent` ones before all others, in their order: new_indices (int32), new_weights (float32,
    as long, or None) and new_indptr (int32 [batch + 1], from 0 on); evicted (int32 or None) gets the slots
    of the others.  new_indices and evicted hold what the budgets give, or more."""
    dev = _on_device(weights, "weights")
    B = kv_indptr.numel() - 1
    if weights.numel() != kv_indices.numel():
        raise ValueError("weights must hold a value per entry of kv_indices")
    if budget.numel() != B or new_indptr.numel() != B + 1:
        raise ValueError("budget must hold a value per request, new_indptr batch + 1 entries")
    if new_weights is not None and new_weights.numel() != new_indices.numel():
        raise ValueError("new_weights must be as long as new_indices")
    if B <= 0:
        with torch.cuda.stream(stream):
            new_indptr.zero_()   # the call itself writes nothing then
        return
    if max_kv_len is None:
        with torch.cuda.stream(stream):   # behind what writes them there
            max_kv_len = int((kv_indptr[1:] - kv_indptr[:-1]).max())
    i32, f32 = _I32, torch.float32
    _call(
        "ddt_cache_evict", _like(weights, f32, dev, "weights"), _like(kv_indices, i32, dev, "kv_indices"),
        _like(kv_indptr, i32, dev, "kv_indptr"), _like(budget, i32, dev, "budget"), B, kv_indices.numel(), max_kv_len,
        sinks, recent, _like(new_indices, i32, dev, "new_indices"), new_indices.numel(),
        _like(new_indptr, i32, dev, "new_indptr"),
        0 if new_weights is None else _like(new_weights, f32, dev, "new_weights"),
        0 if evicted is None else _like(evicted, i32, dev, "evicted"), 0 if evicted is None else evicted.numel(),
        _raw_stream(stream, dev))


def ddt_get_error(stream=None):
    """Returns (status, device_error_bits) and clears the device error word."""
    word = ctypes.c_uint32(0)
    st = lib.ddt_get_error(_stream(stream), ctypes.byref(word))
    return st, word.value


def ddt_selftest_wait_timeout(poll_limit=1 << 12, stream=None):
    """Launch the bounded-wait failure check: a kernel waiting on a barrier
    nobody arrives on gives up after `poll_limit` polls and latches the timeout
    bit (read it with ddt_get_error)."""
    _check("ddt_selftest_wait_timeout", lib.ddt_selftest_wait_timeout(int(poll_limit), _stream(stream)))
