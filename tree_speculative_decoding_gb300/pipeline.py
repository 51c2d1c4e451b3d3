"""One DDTree verify step on the GPU through the C ABI.

``VerifyStep`` owns the device buffers of one batch and runs the four stages
in order on one stream: ddt_build_tree -> ddt_compile_visibility ->
ddt_verify_attn -> ddt_accept (the per-iteration data flow of "The Oracle
Drafter", section "The Engine Interface Design", with the mask and positions
built on the device instead of the host).  By default the first two run as
one launch (ddt_build_tree_visibility); ``fused_tree_mask=False`` calls them
separately.  It only allocates and calls the binding; all arithmetic runs in
libddt.so.
"""
from __future__ import annotations

import numpy as np
import torch

from . import ddt


def _i32(a, device):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(device)


def _bf16(a, device):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.uint16).view(np.int16)).view(
        torch.bfloat16).to(device)


class _Arena:
    """One contiguous device buffer holding several tensors at 256-byte-aligned
    offsets.  Each entry is (name, dtype, data or shape): numpy data (uint16
    holding bf16 bits for bfloat16) is copied in, a shape is left uninitialised."""

    def __init__(self, entries, device):
        layout, off = [], 0
        for name, dtype, src in entries:
            shape = tuple(src) if isinstance(src, tuple) else tuple(np.shape(src))
            nbytes = int(np.prod(shape, dtype=np.int64)) * torch.empty((), dtype=dtype).element_size()
            layout.append((name, dtype, shape, off, nbytes, None if isinstance(src, tuple) else src))
            off += (nbytes + 255) // 256 * 256
        self.buf = torch.empty(max(off, 256), dtype=torch.uint8, device=device)
        self.offsets = {name: o for name, _, _, o, _, _ in layout}
        self.views = {}
        for name, dtype, shape, o, nbytes, src in layout:
            v = self.buf[o:o + nbytes].view(dtype).view(shape)
            if src is not None:
                if dtype == torch.bfloat16:
                    host = torch.from_numpy(np.ascontiguousarray(src, np.uint16).view(np.int16)).view(torch.bfloat16)
                else:
                    host = torch.from_numpy(np.ascontiguousarray(src)).to(dtype)
                v.copy_(host.reshape(shape))
            self.views[name] = v


class VerifyStep:
    """Device-resident inputs and outputs of one verify step for a Workload."""

    def __init__(self, wl, device="cuda", target_argmax=None, num_splits=0, fused_tree_mask=True):
        self.wl = wl
        self.fused_tree_mask = fused_tree_mask
        self.device = torch.device(device)
        dev = self.device
        self.B, self.H = wl.B, wl.H
        self.total_q = wl.total_q
        self.max_q_len = int(wl.q_len.max())
        self.max_kv_len = int(wl.kv_len.max())
        mip = ddt.ddt_mask_indptr(torch.from_numpy(wl.qo_indptr.astype(np.int32)),
                                  torch.from_numpy(wl.prefix_len.astype(np.int32)))
        self.mask_indptr_host = mip
        self.total_words = int(mip[-1])
        argmax = wl.argmax_random if target_argmax is None else target_argmax
        T, W = self.total_q, wl.max_depth + 1
        # Per-step inputs in one device buffer and the step's results in another,
        # so that a host round trip is one copy each way.
        self.inputs = _Arena([
            ("topk_logp", torch.float32, np.ascontiguousarray(wl.topk_logp, np.float32)),
            ("topk_ids", torch.int32, wl.topk_ids), ("root_id", torch.int32, wl.root_id),
            ("budget", torch.int32, wl.budget), ("qo_indptr", torch.int32, wl.qo_indptr),
            ("kv_indptr", torch.int32, wl.kv_indptr), ("kv_indices", torch.int32, wl.kv_indices),
            ("prefix_len", torch.int32, wl.prefix_len), ("mask_indptr", torch.int32, mip.numpy()),
            ("target_argmax", torch.int32, argmax),
            ("q", torch.bfloat16, wl.q)], dev)
        for name, t in self.inputs.views.items():
            setattr(self, name, t)
        # The accept results come first: they are what a host reads back every
        # step (results_bytes from the start of the buffer); the attention output
        # and its lse follow, for a caller that wants them on the host too.
        self.outputs = _Arena([
            ("accept_len", torch.int32, (self.B,)), ("accepted_nodes", torch.int32, (self.B, W)),
            ("commit_tokens", torch.int32, (self.B, W)), ("bonus", torch.int32, (self.B,)),
            ("new_len", torch.int32, (self.B,)),
            ("out", torch.float32, (T, self.H, ddt.DL)), ("lse", torch.float32, (T, self.H))], dev)
        for name, t in self.outputs.views.items():
            setattr(self, name, t)
        self.results_bytes = self.outputs.offsets["out"]
        self.kv_pool = _bf16(wl.kv_pool, dev)  # the resident cache, not a per-step input
        self.node_token = torch.empty(T, dtype=torch.int32, device=dev)
        self.parent = torch.empty(T, dtype=torch.int32, device=dev)
        self.depth = torch.empty(T, dtype=torch.int32, device=dev)
        self.mask = torch.empty(self.total_words, dtype=torch.int32, device=dev)

        self.num_splits = num_splits or ddt.ddt_verify_attn_num_splits(
            self.B, self.H, self.max_q_len, self.max_kv_len)
        # what the attention launches: the requested count rounded to whole kv tiles
        self.launched_splits = ddt.ddt_verify_attn_launched_splits(self.max_kv_len, self.num_splits)
        nbytes = ddt.ddt_verify_attn_workspace_size(T, self.H, self.num_splits)
        self.workspace = (torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None)

    # -- stages -------------------------------------------------------------
    def build_tree(self, stream=None):
        ddt.ddt_build_tree(self.topk_logp, self.topk_ids, self.root_id, self.budget,
                           self.qo_indptr, self.node_token, self.parent, self.depth, stream)

    def compile_visibility(self, stream=None):
        ddt.ddt_compile_visibility(self.parent, self.qo_indptr, self.prefix_len, self.mask_indptr,
                                   self.mask, stream)

    def build_chain_visibility(self, stream=None):
        """Replaces the tree by a chain, parent[i] = i - 1 (depth i) within each
        request, and writes its mask, which is causal over the request's q_len
        new tokens (ddt_build_chain_visibility, one launch).  Engine page, "The
        Core Design Problem: A Unified Forward Pass": prefill, decode and tree
        verify are one forward that differs only in its mask, so verify_attn
        after it is a prefill chunk after the prefix."""
        ddt.ddt_build_chain_visibility(self.qo_indptr, self.prefix_len, self.mask_indptr,
                                       self.parent, self.depth, self.mask, stream)

    def run_prefill(self, stream=None):
        """A prefill chunk as one C call (ddt_prefill_step): chain + causal
        mask, then the attention."""
        ddt.ddt_prefill_step(self.step_args(), stream)

    def build_tree_visibility(self, stream=None):
        ddt.ddt_build_tree_visibility(self.topk_logp, self.topk_ids, self.root_id, self.budget,
                                      self.qo_indptr, self.prefix_len, self.mask_indptr,
                                      self.node_token, self.parent, self.depth, self.mask, stream)

    def verify_attn(self, stream=None):
        ddt.ddt_verify_attn(self.q, self.kv_pool, self.kv_indices, self.kv_indptr, self.qo_indptr,
                            self.mask, self.mask_indptr, self.wl.scale, self.out, self.lse,
                            max_q_len=self.max_q_len, max_kv_len=self.max_kv_len,
                            num_splits=self.num_splits, workspace=self.workspace, stream=stream)

    def accept(self, stream=None):
        ddt.ddt_accept(self.node_token, self.parent, self.qo_indptr, self.target_argmax,
                       self.wl.max_depth, self.accept_len, self.accepted_nodes,
                       self.commit_tokens, self.bonus, stream)

    def commit_kv(self, stream=None):
        """The step after accept: the accepted latents move to the positions after
        the prefix, in place in kv_pool; new_len = prefix + accept_len."""
        ddt.ddt_commit_kv(self.kv_pool, self.kv_indices, self.kv_indptr, self.qo_indptr,
                          self.accept_len, self.accepted_nodes, self.wl.max_depth, self.new_len,
                          stream)

    def step_args(self, commit_kv=False):
        """The step's buffers as one ddt_step_args (for ddt_verify_step and StepGraph)."""
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        a = ddt.StepArgs()
        a.topk_logp, a.topk_ids, a.root_id, a.budget = (p(self.topk_logp), p(self.topk_ids),
                                                        p(self.root_id), p(self.budget))
        a.max_depth, a.topk = self.wl.max_depth, self.wl.K
        a.batch, a.total_q, a.max_q_len, a.max_kv_len = self.B, self.total_q, self.max_q_len, self.max_kv_len
        a.total_mask_words = self.total_words
        a.qo_indptr, a.kv_indptr = p(self.qo_indptr), p(self.kv_indptr)
        a.prefix_len, a.mask_indptr = p(self.prefix_len), p(self.mask_indptr)
        a.q, a.kv_pool, a.pool_rows, a.kv_indices = (p(self.q), p(self.kv_pool), self.kv_pool.shape[0],
                                                     p(self.kv_indices))
        a.num_heads, a.scale, a.num_splits = self.H, self.wl.scale, self.num_splits
        a.workspace = p(self.workspace)
        a.workspace_bytes = 0 if self.workspace is None else self.workspace.numel()
        a.target_argmax = p(self.target_argmax)
        a.node_token, a.parent, a.depth, a.mask = p(self.node_token), p(self.parent), p(self.depth), p(self.mask)
        a.out, a.lse = p(self.out), p(self.lse)
        a.accept_len, a.accepted_nodes = p(self.accept_len), p(self.accepted_nodes)
        a.commit_tokens, a.bonus = p(self.commit_tokens), p(self.bonus)
        a.commit_kv, a.new_len = int(bool(commit_kv)), p(self.new_len)
        return a

    def run_one_call(self, stream=None, commit_kv=False):
        """The step as a single C call (ddt_verify_step)."""
        ddt.ddt_verify_step(self.step_args(commit_kv), stream)

    def step_graph(self, commit_kv=False, host_io=None):
        """A library-owned CUDA graph of the step (ddt_step_graph_*).  host_io =
        (h_in, h_out), pinned host buffers: the graph then copies h_in into the
        inputs before the step and the first len(h_out) bytes of the outputs
        into h_out after it (ddt_step_graph_create_io).  h_out of results_bytes
        brings back the accept results alone; of the whole output buffer, the
        attention output and lse as well."""
        io = None
        if host_io is not None:
            io = (host_io[0], self.inputs.buf, host_io[1], self.outputs.buf)
        return ddt.StepGraph(self.step_args(commit_kv), keep_alive=(self,), io=io)

    @property
    def launches_per_step(self):
        """Kernels one run() or run_one_call() launches: tree + mask (two launches
        for run() with fused_tree_mask=False), attention partial (+ combine when
        it splits), accept."""
        attn = 2 if self.launched_splits > 1 else 1
        return (1 if self.fused_tree_mask else 2) + attn + 1

    def run(self, stream=None):
        if self.fused_tree_mask:
            self.build_tree_visibility(stream)
        else:
            self.build_tree(stream)
            self.compile_visibility(stream)
        self.verify_attn(stream)
        self.accept(stream)

    def check_device_errors(self):
        st, bits = ddt.ddt_get_error()
        if st != 0:
            raise ddt.DDTError("device check", st, f"bits=0x{bits:x}")


class GqaVerifyStep:
    """One verify step of a stack of grouped-query layers for a Workload's requests, trees and
    slots (its latent pool and queries are not used).

    The model runs between the calls: ``build_tree_visibility`` once, then per layer ``layer`` on
    the projections' q, k and v (norm and rotation, the cache rows of the new tokens, the tree
    attention: its result is what the output projection reads), then ``accept`` on the target's
    tokens and ``commit``, which moves the accepted rows of every layer at once.  ``kv`` is the
    cache: [2 * num_layers, rows, num_kv_heads, head_dim], layer l's K pool at 2 l, its V pool at
    2 l + 1.  ``compact`` moves the rows in use to the front of all of them.

    A token is rotated by its request's cached tokens and its depth.  Where rows have left the cache (a
    GqaChunkStep's ``evict``) that is too little: ``position`` (int32 per new token, on the device: its
    depth and what has left its request) then takes the depth's place in the rotation."""

    def __init__(self, wl, num_layers, num_heads, num_kv_heads, head_dim, cos_sin=None, eps=1e-6,
                 interleaved=False, scale=None, device="cuda", position=None):
        self.wl, self.num_layers = wl, num_layers
        self.device = dev = torch.device(device)
        self.B, self.total_q = wl.B, wl.total_q
        self.max_q_len, self.max_kv_len = int(wl.q_len.max()), int(wl.kv_len.max())
        self.cos_sin, self.eps, self.interleaved, self.position = cos_sin, float(eps), interleaved, position
        self.scale = head_dim ** -0.5 if scale is None else float(scale)
        mip = ddt.ddt_mask_indptr(torch.from_numpy(wl.qo_indptr.astype(np.int32)),
                                  torch.from_numpy(wl.prefix_len.astype(np.int32)))
        T, W, i32 = self.total_q, wl.max_depth + 1, torch.int32
        self.topk_logp = torch.from_numpy(np.ascontiguousarray(wl.topk_logp, np.float32)).to(dev)
        for name in ("topk_ids", "root_id", "budget", "qo_indptr", "kv_indptr", "kv_indices", "prefix_len"):
            setattr(self, name, _i32(getattr(wl, name), dev))
        self.mask_indptr = mip.to(dev)
        empty = lambda *shape, dtype=i32: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
        self.node_token, self.parent, self.depth = empty(T), empty(T), empty(T)
        self.mask = empty(int(mip[-1]))
        self.accept_len, self.bonus, self.new_len, self.live = empty(self.B), empty(self.B), empty(self.B), empty(1)
        self.accepted_nodes, self.commit_tokens = empty(self.B, W), empty(self.B, W)
        self.kv = torch.zeros((2 * num_layers, wl.pool_rows, num_kv_heads, head_dim), dtype=torch.bfloat16, device=dev)
        self.q = empty(T, num_heads, head_dim, dtype=torch.bfloat16)  # normed and rotated
        self.out = torch.empty_like(self.q)
        ctas = ddt.ddt_gqa_verify_attn_num_ctas(self.B, num_heads, num_kv_heads, self.max_q_len, self.max_kv_len)
        nbytes = ddt.ddt_gqa_verify_attn_workspace_size(self.B, num_heads, num_kv_heads, head_dim, self.max_q_len, ctas)
        # the layers' attention and the compaction use it one after another
        self.workspace = empty(max(nbytes, ddt.ddt_cache_compact_workspace_size(wl.pool_rows)), dtype=torch.uint8)

    def build_tree_visibility(self, stream=None):
        ddt.ddt_build_tree_visibility(self.topk_logp, self.topk_ids, self.root_id, self.budget,
                                      self.qo_indptr, self.prefix_len, self.mask_indptr,
                                      self.node_token, self.parent, self.depth, self.mask, stream)

    def build_chain_visibility(self, stream=None):
        """A causal chain in place of the tree: the layers then run a prefill chunk or a decode."""
        ddt.ddt_build_chain_visibility(self.qo_indptr, self.prefix_len, self.mask_indptr,
                                       self.parent, self.depth, self.mask, stream)

    def layer(self, index, q, k, v, q_weight=None, k_weight=None, stream=None):
        """Layer `index` between its projections: q [total_q, heads, head_dim], k and v [total_q,
        K/V heads, head_dim] bf16; returns the attention's output, good until the next layer."""
        k_pool, v_pool = self.kv[2 * index], self.kv[2 * index + 1]
        place = self.depth if self.position is None else self.position
        ddt.ddt_gqa_norm_rope_append(q, k, v, q_weight, k_weight, self.eps, self.cos_sin, place,
                                     self.qo_indptr, self.kv_indices, self.kv_indptr, self.q, k_pool, v_pool,
                                     interleaved=self.interleaved, stream=stream)
        ddt.ddt_gqa_verify_attn(self.q, k_pool, v_pool, self.kv_indices, self.kv_indptr, self.qo_indptr, self.mask,
                                self.mask_indptr, self.scale, self.out, max_q_len=self.max_q_len,
                                max_kv_len=self.max_kv_len, workspace=self.workspace, stream=stream)
        return self.out

    def accept(self, target_argmax, stream=None):
        ddt.ddt_accept(self.node_token, self.parent, self.qo_indptr, target_argmax, self.wl.max_depth,
                       self.accept_len, self.accepted_nodes, self.commit_tokens, self.bonus, stream)

    def commit(self, stream=None):
        """The accepted rows of every layer to the positions after the prefix; new_len = prefix +
        accept_len."""
        ddt.ddt_cache_commit(self.kv, self.kv_indices, self.kv_indptr, self.qo_indptr, self.accept_len,
                             self.accepted_nodes, self.wl.max_depth, self.new_len, stream)

    def copy(self, src, dst, stream=None):
        """Rows src of every layer to rows dst: a request forked or moved."""
        ddt.ddt_cache_copy(self.kv, self.kv, src, dst, stream)

    def compact(self, stream=None):
        """The rows that kv_indices names to the front of every pool; kv_indices becomes their new
        numbers, live their count.  After a commit it still names the step's rejected nodes: their
        rows are free once the caller has written the next step's slots over them."""
        ddt.ddt_cache_compact(self.kv, self.kv_indices, self.kv_indices, self.live, self.workspace, stream)

    check_device_errors = VerifyStep.check_device_errors


class GqaChunkStep:
    """One chunk of new tokens per request (a prompt, a part of one, or a single token) through a stack
    of grouped-query layers, on a cache that may be a GqaVerifyStep's, and what keeps that cache within
    a budget.

    ``kv`` is the cache, [2 * num_layers, rows, num_kv_heads, head_dim] (layer l's K pool at 2 l, its V
    pool at 2 l + 1); ``kv_indices`` (int32, on the device) has per request the slots of its prefix_len
    cached tokens, then those of its q_len new ones (host arrays).  Per layer ``layer`` takes the
    projections' q, k and v and returns what the output projection reads; score_cap, slopes, window and
    full_len are the layer's (``ddt.ddt_gqa_chunk_attn``), given here for all of them or to ``layer``.

    With ``observe`` (given here for all layers or to ``layer``) the step also sums what every column
    receives, over the layers that are observed, from all of the chunk's tokens or from the last
    ``last_rows`` of them, on top of decay * prev (the step before's: the weights and offsets that its
    ``evict`` returned).  ``evict`` then cuts every request down to its budget.
    Positions count columns: where rows have left the cache, ``position`` (int32 per new token, on the
    device: its place behind the cached columns, so i + what has left) keeps the rotation's."""

    def __init__(self, kv, kv_indices, prefix_len, q_len, num_heads, cos_sin=None, eps=1e-6, interleaved=False,
                 scale=None, score_cap=0.0, slopes=None, window=0, full_len=None, position=None, observe=False,
                 last_rows=0, prev=None, prev_indptr=None, decay=1.0):
        self.kv, self.kv_indices, self.device = kv, kv_indices, kv.device
        dev, G, D = kv.device, kv.shape[2], kv.shape[3]
        self.prefix_len, self.q_len = np.asarray(prefix_len, np.int64), np.asarray(q_len, np.int64)
        self.kv_len = self.prefix_len + self.q_len
        self.B, self.num_layers = len(self.q_len), kv.shape[0] // 2
        offsets = lambda n: np.concatenate([[0], np.cumsum(n)])  # noqa: E731
        self.qo_indptr, self.kv_indptr = _i32(offsets(self.q_len), dev), _i32(offsets(self.kv_len), dev)
        self.total_q, self.total_kv = int(self.q_len.sum()), int(self.kv_len.sum())
        if kv_indices.numel() != self.total_kv:
            raise ValueError("kv_indices must hold prefix_len + q_len slots per request")
        self.max_q_len, self.max_kv_len = int(self.q_len.max(initial=0)), int(self.kv_len.max(initial=0))
        self.cos_sin, self.eps, self.interleaved, self.position = cos_sin, float(eps), interleaved, position
        self.scale = D ** -0.5 if scale is None else float(scale)
        self.scores = dict(score_cap=score_cap, slopes=slopes, window=window, full_len=full_len)
        self.observe, self.last_rows = observe, last_rows
        self.prev, self.prev_indptr, self.decay = prev, prev_indptr, decay
        empty = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
        self.q = empty(self.total_q, num_heads, D, dtype=torch.bfloat16)  # normed and rotated
        self.out = torch.empty_like(self.q)
        self.lse = empty(self.total_q, num_heads, dtype=torch.float32)
        self._weights = empty(self.total_kv, dtype=torch.float32)
        self._observed = None   # the lowest layer that was observed: it starts the sums
        self._given = False     # the weights were handed out before any was
        self.live = empty(1, dtype=torch.int32)
        ctas = ddt.ddt_gqa_chunk_attn_num_ctas(self.B, num_heads, G, self.max_q_len, self.max_kv_len)
        # the layers' calls and the compaction use it one after another
        self.workspace = empty(max(ddt.ddt_gqa_chunk_attn_workspace_size(num_heads, G, D, max(1, self.max_q_len), ctas),
                                   ddt.ddt_gqa_chunk_weights_workspace_size(ddt.ddt_gqa_chunk_weights_num_ctas(self.B)),
                                   ddt.ddt_cache_compact_workspace_size(kv.shape[1]), 256), dtype=torch.uint8)

    @property
    def weights(self):
        """The sums, float32 by kv_indptr.  A step that observes nothing evicts by what is put here."""
        self._given = True
        return self._weights

    @weights.setter
    def weights(self, sums):
        self._weights, self._given = sums, True

    def layer(self, index, q, k, v, q_weight=None, k_weight=None, stream=None, observe=None, **scores):
        """Layer `index` between its projections: q [total_q, heads, head_dim], k and v [total_q,
        K/V heads, head_dim] bf16; returns the attention's output, good until the next layer.  Layers
        run in order; the lowest one that is observed starts the sums, with the earlier ones."""
        observe = self.observe if observe is None else observe
        k_pool, v_pool = self.kv[2 * index], self.kv[2 * index + 1]
        how = dict(self.scores, max_q_len=self.max_q_len, max_kv_len=self.max_kv_len, workspace=self.workspace, stream=stream, **scores)
        ddt.ddt_gqa_norm_rope_append(q, k, v, q_weight, k_weight, self.eps, self.cos_sin, self.position,
                                     self.qo_indptr, self.kv_indices, self.kv_indptr, self.q, k_pool, v_pool,
                                     interleaved=self.interleaved, stream=stream)
        ddt.ddt_gqa_chunk_attn(self.q, k_pool, v_pool, self.kv_indices, self.kv_indptr, self.qo_indptr, self.scale,
                               self.out, self.lse if observe else None, **how)
        if observe:
            starts = self._observed is None or index <= self._observed
            before = (self.prev, self.prev_indptr, self.decay) if starts else (self._weights, None, 1.0)
            ddt.ddt_gqa_chunk_weights(self.q, k_pool, self.lse, self.kv_indices, self.kv_indptr, self.qo_indptr, self.scale,
                                      self._weights, prev=before[0], prev_indptr=before[1], decay=before[2],
                                      last_rows=self.last_rows, **how)
            if starts:
                self._observed = index
        return self.out

    def evict(self, budget, sinks=0, recent=0, stream=None):
        """Every request down to budget (host array) columns: its first `sinks` and last `recent` ones and
        those that received most.  Returns (kv_indices, kv_indptr, weights, evicted) of what is left: slots,
        offsets and sums, on the device (of the call's stream), and the slots that left; new_len has the
        lengths on the host.  The budgets come from the host: a graph takes ``ddt.ddt_cache_evict``."""
        if self._observed is None and not self._given:
            raise ValueError("nothing to evict by: no layer was observed, nor were weights given")
        with torch.cuda.stream(stream):
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("evict cannot be captured: it copies its budgets from the host")
        self.new_len = np.minimum(self.kv_len, np.maximum(np.asarray(budget, np.int64), 0))
        kept = int(self.new_len.sum())
        new = lambda n, dtype=torch.int32: torch.empty(n, dtype=dtype, device=self.device)  # noqa: E731
        # on the call's stream: it may still need the budgets' memory when this returns
        with torch.cuda.stream(stream):
            left = new(kept), new(self.B + 1), new(kept, torch.float32), new(self.total_kv - kept)
            budgets = torch.from_numpy(self.new_len.astype(np.int32)).pin_memory().to(self.device, non_blocking=True)
            ddt.ddt_cache_evict(self._weights, self.kv_indices, self.kv_indptr, budgets, left[0], left[1], left[2], left[3],
                                sinks=sinks, recent=recent, max_kv_len=self.max_kv_len)
        return left

    def compact(self, kv_indices, stream=None):
        """The rows that kv_indices names to the front of every pool, their new numbers into kv_indices, their
        count into live."""
        ddt.ddt_cache_compact(self.kv, kv_indices, kv_indices, self.live, self.workspace, stream)

    check_device_errors = VerifyStep.check_device_errors
