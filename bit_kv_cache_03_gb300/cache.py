"""Device buffers of one attention layer's NVFP4 paged cache, allocated by PyTorch.

PyTorch provides memory and streams only; every computation goes through the C ABI.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from . import (_capturing, kv_nvfp4_append, kv_nvfp4_append_slots, kv_nvfp4_decode_attn,
               kv_nvfp4_decode_attn_weights, kv_nvfp4_decode_step, kv_nvfp4_decode_step_host,
               kv_nvfp4_evict_compact, kv_nvfp4_evict_select, kv_nvfp4_plan,
               kv_nvfp4_plan_workspace_bytes, kv_nvfp4_pool_bytes, kv_nvfp4_rope_table_init,
               kv_nvfp4_weights_workspace_bytes, make_layout)


class PagedNVFP4Cache:
    """Page pool, block table, RoPE table and status word for one layer on one GPU."""

    def __init__(self, num_pages, block_table, max_pos, num_q_heads=24, num_kv_heads=4,
                 rot_dim=32, theta=1e7, pos_scale=1.0, device="cuda"):
        self.layout = make_layout(num_q_heads, num_kv_heads, 128, 64, rot_dim)
        self.device = torch.device(device)
        self.num_pages = int(num_pages)
        self.pool = torch.empty(kv_nvfp4_pool_bytes(self.layout, self.num_pages),
                                dtype=torch.uint8, device=self.device)
        bt = np.ascontiguousarray(block_table, np.int32)
        self.num_seqs, self.max_pages = bt.shape
        self.block_table = torch.from_numpy(bt).to(self.device)
        self.max_pos = int(max_pos)
        self.rot_dim = rot_dim
        self.rope = torch.empty(max(1, self.max_pos * rot_dim), dtype=torch.float32,
                                device=self.device)
        if rot_dim > 0:
            kv_nvfp4_rope_table_init(self.rope, self.max_pos, rot_dim, theta, pos_scale)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.workspace = None
        self.weights_workspace = None
        self.plan_info = None
        self._captured = []

    # -- fused quantize-append --------------------------------------------------------------
    def append(self, k, v, seq_ids, positions, q=None, q_codes=None, q_scales=None, stream=None,
               slots=None):
        """slots: int32 cache slots of the tokens where they differ from the positions (behind an
        eviction)."""
        T = int(k.shape[0])
        if slots is not None:
            self._check_current()
            if slots.dtype != torch.int32 or not slots.is_contiguous() or slots.numel() != T or \
                    slots.device != self.pool.device:
                raise ValueError("slots must be device int32, one per token")
            kv_nvfp4_append_slots(self.layout, q, k, v, seq_ids, slots, positions, T, self.rope,
                                  self.max_pos, self.block_table, self.num_seqs, self.max_pages,
                                  self.num_pages, self.pool, q_codes, q_scales, self.status, stream)
            return
        kv_nvfp4_append(self.layout, q, k, v, seq_ids, positions, T, self.rope, self.max_pos,
                        self.block_table, self.num_seqs, self.max_pages, self.num_pages,
                        self.pool, q_codes, q_scales, self.status, stream)

    def quantized_q_buffers(self, T):
        H = self.layout.num_q_heads
        return (torch.empty(T * H * 64, dtype=torch.uint8, device=self.device),
                torch.empty(T * H * 8, dtype=torch.uint8, device=self.device))

    # -- split-K plan + attention -----------------------------------------------------------
    def plan(self, seq_lens, q_len, causal=True, chunk_tokens=1024, stream=None):
        """Builds the work list of the next attention calls (seq_lens include the new tokens), on
        `stream`, behind the calls that use the last one."""
        need = kv_nvfp4_plan_workspace_bytes(self.layout, seq_lens, q_len, causal, chunk_tokens)
        if self.workspace is None or self.workspace.numel() < need:
            self._enlarge("workspace", need, stream)
        self.plan_info = kv_nvfp4_plan(self.layout, seq_lens, q_len, causal, chunk_tokens,
                                       self.workspace, self.workspace.numel(), stream)
        return self.plan_info

    def attend(self, q_codes, q_scales, out, sm_scale=None, stream=None):
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(128)
        self._hold_captured(stream)
        kv_nvfp4_decode_attn(self.layout, self.plan_info, self.workspace, q_codes, q_scales,
                             sm_scale, self.pool, self.num_pages, self.block_table, self.max_pages,
                             out, self.status, stream)

    # -- attention that accounts for each key's weight, and eviction by it -----------------------
    def weight_accounts(self):
        """Zeroed accounts [num_seqs, num_kv_heads, slots] for attend_weights and evict, for every slot
        of the block table (evict is sized by their width: accounts no wider than the longest sequence
        will be also do, and are faster to choose from when there are many sequences)."""
        return torch.zeros(self.num_seqs, self.layout.num_kv_heads, self.max_pages * 64,
                           dtype=torch.float32, device=self.device)

    def attend_weights(self, q_codes, q_scales, out, weights, weights_in=None, sm_scale=None,
                       stream=None):
        """attend() with a bf16 `out`, adding every key's attention weight to `weights` (or writing
        weights_in plus them). On the plan of the last plan(), whose workspace and this call's belong
        to one call at a time: a call on another stream has to be ordered behind the one before it.
        With at most 8 query rows per KV head this call's workspace takes 4 bytes per row and cached
        token of every KV head. A captured call replays on the plan that it was captured with: a later
        plan() that fits the same workspace overwrites it."""
        self._check_accounts(weights, weights_in)
        if self.plan_info is None:
            raise ValueError("attend_weights needs a plan()")
        if self.plan_info.num_seqs > self.num_seqs:
            raise ValueError("the plan has more sequences than the cache")
        if weights_in is not None and weights_in.shape != weights.shape:
            raise ValueError("weights_in must have the shape of weights")
        rows = self.plan_info.num_seqs * self.plan_info.q_len * self.layout.num_q_heads
        if out.dtype != torch.bfloat16 or not out.is_contiguous() or out.numel() != rows * 128 or \
                out.device != weights.device:
            raise ValueError("out must be a contiguous device bfloat16 [rows, num_q_heads, 128]")
        for x, each in ((q_codes, 64), (q_scales, 8)):
            if x.device != weights.device or not x.is_contiguous() or x.nbytes < rows * each:
                raise ValueError("q_codes and q_scales must be contiguous, on the device, and hold "
                                 "64 and 8 bytes per row of the plan")
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(128)
        need = kv_nvfp4_weights_workspace_bytes(self.layout, self.plan_info)
        if self.weights_workspace is None or self.weights_workspace.numel() < need:
            self._enlarge("weights_workspace", need, stream)
        self._hold_captured(stream)
        kv_nvfp4_decode_attn_weights(
            self.layout, self.plan_info, self.workspace, self.weights_workspace,
            self.weights_workspace.numel(), q_codes, q_scales, sm_scale, self.pool, self.num_pages,
            self.block_table, self.max_pages, out, weights if weights_in is None else weights_in,
            weights, weights.shape[2], self.status, stream)

    def evict(self, weights, seq_lens, keep, index, sink=0, recent=0, stream=None):
        """Keeps min(seq_len, keep) tokens of each sequence by accumulated weight, the first `sink`
        and the last `recent` ahead of the others, and compacts the cache and the weights to them
        in place. Tokens so protected rank by slot alone: a keep below sink + recent drops the newest of
        them, the last token first. seq_lens, keep: device int32 [num_seqs]; index: device int32
        [num_seqs, num_kv_heads, n] (every KV head keeps its own tokens) or [num_seqs, 1, n] (one
        set for all), n at least the largest kept count; receives the kept slots, ascending. A sequence
        holds min(seq_len, keep) tokens afterwards; its next ones go behind them with append(slots=...)
        under their own positions (decode_step takes the position from the slot, which is no longer
        right). No page may belong to two sequences."""
        self._check_accounts(weights)
        for x in (seq_lens, keep):
            if x.dtype != torch.int32 or not x.is_contiguous() or x.numel() != self.num_seqs or \
                    x.device != weights.device:
                raise ValueError("seq_lens and keep must be device int32 [num_seqs]")
        if index.dtype != torch.int32 or not index.is_contiguous() or index.dim() != 3 or \
                index.shape[0] != self.num_seqs or index.device != weights.device or \
                index.shape[1] not in (1, self.layout.num_kv_heads):
            raise ValueError("index must be a contiguous device int32 "
                             "[num_seqs, num_kv_heads or 1, n]")
        per_head = index.shape[1] != 1
        kv_nvfp4_evict_select(self.layout, weights, weights.shape[2], seq_lens, keep, self.num_seqs,
                              per_head, sink, recent, index, index.shape[2], self.status, stream)
        kv_nvfp4_evict_compact(self.layout, index, index.shape[2], per_head, seq_lens, keep,
                               self.num_seqs, self.block_table, self.max_pages, self.num_pages,
                               self.pool, None, 0, weights, weights.shape[2], self.status, stream)

    def _enlarge(self, name, need, stream):
        """Replaces a workspace by one of `need` bytes, from the allocator's memory of the stream that
        works in it. The old one may be another stream's memory, which takes it back the moment it is
        dropped: the allocator is told to wait for this call's stream, behind which the calls that used
        it lie. What was outgrown once gets a sixteenth more: a sequence's need grows with every page."""
        with self._on(stream):
            old = getattr(self, name)
            if old is not None:
                old.record_stream(torch.cuda.current_stream())
                need += need // 16
            old = None
            setattr(self, name, None)  # before the new one is made: the two need not fit together
            setattr(self, name, torch.empty(max(need, 256), dtype=torch.uint8, device=self.device))

    def _hold_captured(self, stream):
        """A graph replays a captured call on the workspaces that the call had: they live as long as the
        cache does, outgrown or not."""
        if torch.cuda.is_current_stream_capturing() if stream is None else _capturing(stream):
            self._captured += [b for b in (self.workspace, self.weights_workspace)
                               if b is not None and all(b is not x for x in self._captured)]

    @staticmethod
    def _on(stream):
        return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int)
                                 else stream)

    def _check_current(self):
        # a launch goes to the current device; with the buffers of another one it would fault
        if self.pool.device.index != torch.cuda.current_device():
            raise ValueError("the cache's device is not the current one")

    def _check_accounts(self, *tensors):
        self._check_current()
        for w in tensors:
            if w is not None and (w.device != self.pool.device or w.dtype != torch.float32 or
                                  not w.is_contiguous() or w.dim() != 3 or
                                  tuple(w.shape[:2]) != (self.num_seqs, self.layout.num_kv_heads)):
                raise ValueError("weights must be a contiguous device float32 "
                                 "[num_seqs, num_kv_heads, slots]")

    # -- append of the step's new tokens + attention, one launch ------------------------------
    def decode_step(self, q, k, v, out, q_codes=None, q_scales=None, sm_scale=None, stream=None):
        """New tokens of every sequence (sequence-major rows, at the last q_len positions of the
        lengths given to the last plan) appended and attended in one kernel launch. The positions are
        the slots too: not for a cache that evict() compacted, whose tokens have other positions."""
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(128)
        self._hold_captured(stream)
        kv_nvfp4_decode_step(self.layout, self.plan_info, self.workspace, q, k, v, self.rope,
                             self.max_pos, self.block_table, self.max_pages, self.num_pages,
                             self.pool, q_codes, q_scales, sm_scale, out, self.status, stream)

    # -- one decode step from host buffers -------------------------------------------------------
    def decode_step_host(self, seq_lens, q_len, h_q, h_k, h_v, d_q, d_k, d_v, d_out, h_out,
                         causal=True, chunk_tokens=1024, sm_scale=None, stream=None):
        """Plan, host-to-device copies of the new tokens, the fused step and the device-to-host
        copy of the output, enqueued by one library call (the workspace must already be large
        enough: call plan() once with the same shape first)."""
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(128)
        kv_nvfp4_decode_step_host(self.layout, seq_lens, q_len, causal, chunk_tokens,
                                  self.workspace, self.workspace.numel(), h_q, h_k, h_v, d_q, d_k,
                                  d_v, self.rope, self.max_pos, self.block_table, self.max_pages,
                                  self.num_pages, self.pool, sm_scale, d_out, h_out, self.status,
                                  stream)
