"""Drafted (speculative) decode steps over a paged latent cache, with every
length, page and tree on the GPU.

``StepPlan`` owns what all layers of a model share: the pages each sequence
holds, the free list, the block table, and one step's row offsets, slots,
positions and ancestor masks (mla_step_plan).  ``TreeDecodeStep`` owns one
layer's pool and buffers and runs

    mla_cache_append_slots -> mla_absorb_q -> mla_decode_tree -> mla_out_uv

for the planned rows; ``StepPlan.commit`` keeps an accepted path of each
sequence's drafted rows in every layer (mla_cache_commit).  Nothing reads a
length on the host, so a whole step, from the plan to the commit, can be
recorded as one CUDA graph and replayed while sequences grow, finish and come.

A step's rows are ragged: sequence b brings ``new_counts[b]`` of them (0: it
sits this step out), a drafted tree with ``parents``, or a run of tokens (a
prompt, or a single token) without.  A finished sequence gives its pages back
in the first plan that finds ``seq_lens[b]`` and ``new_counts[b]`` zero.
"""
from __future__ import annotations

import functools
import math

import numpy as np

from . import (D_C, D_NOPE, D_R, D_ROW, D_V, MLA_DEVERR_CAPACITY, MLA_E4M3, MLA_F32, PAGE, mla_absorb_q,
               mla_cache_append_slots, mla_cache_commit, mla_decode_tree, mla_decode_tree_workspace_bytes, mla_out_uv,
               mla_rope_table, mla_step_plan)
from .step import _DT, _torch_dtype


def _need(name, t, cuda, dtype, n):
    """Raise unless a kernel (on the GPU: cuda) can read n numbers of t: the calls take its address and the plan's
    sizes, nothing else.  (Integer addresses pass, as in the calls.  A layer makes five of these, 0.4 us each.)"""
    if isinstance(t, int) or (t.dtype is dtype and t.is_cuda is cuda and t.numel() >= n and t.is_contiguous()):
        return
    if t.dtype is not dtype or t.numel() < n:
        raise ValueError(f"{name}: need {n} numbers of {dtype}, got {t.dtype} {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_pinned():
        raise ValueError(f"{name} is on {t.device}, the plan is not")


def _on_the_plan_s_device(method):
    """The calls work on the current device: make it the plan's one meanwhile (0.3 us where it is)."""
    @functools.wraps(method)
    def call(self, *args, **kwargs):
        plan = self if isinstance(self, StepPlan) else self.plan
        cuda = plan.torch.cuda
        if plan.index is None or plan.index == cuda.current_device():
            return method(self, *args, **kwargs)
        with cuda.device(plan.index):
            return method(self, *args, **kwargs)
    return call


class StepPlan:
    """The bookkeeping of `batch` sequences over a pool of `num_pages` pages.

    max_pages: pages a sequence may hold; max_rows: new rows of one step, all
    sequences together; max_nodes: rows of one sequence's drafted tree, and of
    every other sequence's in a step with trees (a longer prompt waits for a
    step without)."""

    def __init__(self, *, batch, num_pages, max_pages, max_rows, max_nodes=64, device="cuda"):
        import torch
        self.torch = torch
        self.batch, self.num_pages, self.max_pages = int(batch), int(num_pages), int(max_pages)
        self.max_rows, self.mask_words = int(max_rows), -(-int(max_nodes) // 64)
        self.device = torch.device(device)
        self.cuda = self.device.type == "cuda"

        def ints(*shape, fill=0):
            return torch.full(shape, fill, dtype=torch.int32, device=self.device)

        self.seq_lens = ints(self.batch)                  # cached rows, drafts not counted
        self.held = ints(self.batch)                      # pages of each sequence
        self.free_pages = torch.arange(self.num_pages - 1, -1, -1, dtype=torch.int32, device=self.device)
        self.free_count = ints(1, fill=self.num_pages)
        self.block_table = ints(self.batch, self.max_pages, fill=-1)
        # one step's plan
        self.row_start, self.kv_lens = ints(self.batch + 1), ints(self.batch)
        self.seq_ids, self.slots = ints(self.max_rows, fill=-1), ints(self.max_rows, fill=-1)
        self.positions = ints(self.max_rows)
        self.tree_mask = torch.zeros((self.max_rows, self.mask_words), dtype=torch.int64, device=self.device)
        self.is_tree = False
        self.err = ints(1)
        self.index = self.err.device.index if self.cuda else None

    @_on_the_plan_s_device
    def plan(self, new_counts, parents=None, stream=None):
        """Lay out a step: int32 new_counts [batch] rows per sequence; parents
        int32 [max_rows] (each row's parent within its sequence's rows, -1 for
        a root) for drafted trees, or None for runs of tokens."""
        _need("new_counts", new_counts, self.cuda, self.torch.int32, self.batch)
        if parents is not None:
            _need("parents", parents, self.cuda, self.torch.int32, self.max_rows)
        self.is_tree = parents is not None
        mla_step_plan(self.seq_lens, new_counts, parents, self.batch, self.max_rows, self.mask_words, self.held,
                      self.held, self.free_pages, self.free_count, self.free_count, self.block_table, self.max_pages,
                      PAGE, self.num_pages, self.row_start, self.kv_lens, self.seq_ids, self.positions, self.slots,
                      self.tree_mask if self.is_tree else None, self.err, stream)

    @_on_the_plan_s_device
    def commit(self, layers, accept_counts, accept_nodes, stream=None):
        """Keep accept_counts[b] rows of each sequence's new ones, those of the
        ascending path accept_nodes[row_start[b]:], in every layer's cache;
        seq_lens then counts them."""
        if not layers:
            raise ValueError("commit needs the layers whose caches hold the step's rows")
        _need("accept_counts", accept_counts, self.cuda, self.torch.int32, self.batch)
        _need("accept_nodes", accept_nodes, self.cuda, self.torch.int32, self.max_rows)
        for i, layer in enumerate(layers):
            last = i == len(layers) - 1
            mla_cache_commit(self.kv_lens, self.row_start, self.batch, self.max_rows, accept_counts, accept_nodes,
                             self.block_table, self.max_pages, PAGE, layer.cache, layer.cache_scale,
                             layer.cache_dtype, self.num_pages, self.seq_lens if last else None, self.err, stream)

    @_on_the_plan_s_device
    def keep_all(self, stream=None):
        """Every planned row stays (a prompt, a single token): seq_lens = kv_lens."""
        if stream is None:
            self.seq_lens.copy_(self.kv_lens)
            return
        if isinstance(stream, int):
            stream = self.torch.cuda.ExternalStream(stream, device=self.err.device)
        with self.torch.cuda.stream(stream):
            self.seq_lens.copy_(self.kv_lens)

    def check(self):
        """Read the error word (this waits for the GPU), clear it and raise if a
        plan did not fit, an index was out of range or a wait ran out."""
        flags = int(self.err.item())
        if flags:
            self.err.zero_()
            what = "a plan did not fit" if flags & MLA_DEVERR_CAPACITY else "bad indices or a device wait that ran out"
            raise RuntimeError(f"drafted step: device error word {flags:#x} ({what})")


class TreeDecodeStep:
    """One layer's cache and buffers for the rows a StepPlan lays out.

    dtype: "bf16" or "f32" (queries, weights); cache_dtype: "bf16" or "e4m3"
    with bf16, "f32" with f32."""

    def __init__(self, plan: StepPlan, *, n_heads, dtype="bf16", cache_dtype="bf16", max_pos=None, theta=10000.0,
                 eps=1e-6, norm_gain=None, softmax_scale=None):
        import torch
        if (dtype, cache_dtype) not in (("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")):
            raise ValueError(f"unsupported dtype, cache_dtype: {dtype}, {cache_dtype}")
        self.plan = plan
        self.n_heads = int(n_heads)
        self.dtype, self.cache_dtype = _DT[dtype], _DT[cache_dtype]
        dev = plan.err.device
        self.eps = float(eps)
        self.softmax_scale = float(softmax_scale if softmax_scale is not None else 1.0 / math.sqrt(192.0))
        self.max_pos = int(max_pos if max_pos is not None else plan.max_pages * PAGE)
        cos = np.empty((self.max_pos, D_R // 2), np.float32)
        sin = np.empty_like(cos)
        mla_rope_table(theta, self.max_pos, cos, sin)
        self.rope_cos, self.rope_sin = torch.from_numpy(cos).to(dev), torch.from_numpy(sin).to(dev)
        self.norm_gain = None if norm_gain is None else torch.as_tensor(np.asarray(norm_gain, np.float32)).to(dev)
        # zero-filled: the attention reads whole pages
        self.cache = torch.zeros((plan.num_pages, D_ROW // 64, PAGE, 64), dtype=_torch_dtype(self.cache_dtype),
                                 device=dev)
        self.cache_scale = (torch.zeros((plan.num_pages, PAGE), dtype=torch.float32, device=dev)
                            if self.cache_dtype == MLA_E4M3 else None)
        rows, qdt = plan.max_rows, torch.float32 if self.dtype == MLA_F32 else torch.bfloat16
        # zero-filled: rows behind a step's last one are projected along with the others
        self.q_abs = torch.zeros((rows, self.n_heads, D_ROW), dtype=qdt, device=dev)
        self.o_lat = torch.zeros((rows, self.n_heads, D_C), dtype=qdt, device=dev)
        self.lse = torch.zeros((rows, self.n_heads), dtype=torch.float32, device=dev)
        self.out = torch.zeros((rows, self.n_heads, D_V), dtype=qdt, device=dev)
        self.workspace = torch.empty(mla_decode_tree_workspace_bytes(self.cache_dtype, rows, self.n_heads),
                                     dtype=torch.uint8, device=dev)

    @_on_the_plan_s_device
    def append(self, kv_a, stream=None):
        """Cache rows of the planned tokens: kv_a [max_rows, 576] (rows behind the
        step's last one are skipped)."""
        p = self.plan
        f32 = kv_a.dtype is p.torch.float32
        _need("kv_a", kv_a, p.cuda, kv_a.dtype if f32 else p.torch.bfloat16, p.max_rows * D_ROW)
        mla_cache_append_slots(kv_a, MLA_F32 if f32 else _DT["bf16"], p.max_rows, p.slots,
                               p.positions, self.norm_gain, self.eps, self.rope_cos, self.rope_sin, self.max_pos,
                               self.cache, self.cache_scale, self.cache_dtype, p.num_pages, p.err, stream)

    @_on_the_plan_s_device
    def absorb(self, q_nope, q_pe, w_uk, stream=None):
        """q_abs = [W_UK^T q_nope; q_pe], q_nope [max_rows, H, 128], q_pe [max_rows, H, 64] rotated to the rows'
        `plan.positions`, w_uk [H, 128, 512], all of `dtype`."""
        cuda, dt, vecs = self.plan.cuda, self.q_abs.dtype, self.plan.max_rows * self.n_heads
        _need("q_nope", q_nope, cuda, dt, vecs * D_NOPE)
        _need("q_pe", q_pe, cuda, dt, vecs * D_R)
        _need("w_uk", w_uk, cuda, dt, self.n_heads * D_NOPE * D_C)
        mla_absorb_q(q_nope, q_pe, w_uk, self.q_abs, self.plan.max_rows, self.n_heads, self.dtype, stream)

    @_on_the_plan_s_device
    def attend(self, stream=None):
        p = self.plan
        mla_decode_tree(self.q_abs, self.dtype, self.cache, self.cache_scale, self.cache_dtype, p.num_pages,
                        p.block_table, p.max_pages, PAGE, p.kv_lens, p.row_start, p.batch, p.max_rows, self.n_heads,
                        p.tree_mask if p.is_tree else None, p.mask_words, self.softmax_scale, self.workspace,
                        self.o_lat, self.dtype, self.lse, p.err, stream)

    @_on_the_plan_s_device
    def project_out(self, w_uv, stream=None):
        """`out` = W_UV o_lat; w_uv [H, 128, 512] of `dtype`."""
        _need("w_uv", w_uv, self.plan.cuda, self.o_lat.dtype, self.n_heads * D_V * D_C)
        mla_out_uv(self.o_lat, w_uv, self.out, self.plan.max_rows, self.n_heads, self.dtype, stream)

    def run(self, kv_a, q_nope, q_pe, w_uk, w_uv, stream=None):
        """Append the planned rows and attend; returns `out` [max_rows, H, 128]."""
        self.append(kv_a, stream)
        self.absorb(q_nope, q_pe, w_uk, stream)
        self.attend(stream)
        self.project_out(w_uv, stream)
        return self.out
