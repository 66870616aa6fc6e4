"""The target model's steps through the entry points, with their buffers.

A convenience for callers that hold torch tensors.  ``VerifyStep`` owns the
outputs and the workspaces of one verification step and issues, in stream order,
tree_mask_build -> tree_verify_attention -> tree_accept -> kv_compact, with
tree_logits_process before and token_counts_update after tree_accept where the
rows are to be sampled with penalties, biases, a grammar or a temperature.
``ChunkStep`` is the same for a chunk of prompt or plainly decoded tokens:
chunk_kv_append -> chunk_attention.  Each runs eagerly (``run``) or as a captured
CUDA graph (``capture``, then replay).  Marshalling only; the arithmetic is in the
CUDA library.
"""
from __future__ import annotations

import torch

from . import (GREEDY, GREEDY_MASKED, STOCHASTIC, chunk_attention, chunk_attention_workspace,
               chunk_kv_append, kv_compact, token_counts_update, tree_accept,
               tree_accept_workspace, tree_logits_process, tree_mask_build, tree_verify_attention,
               tree_verify_attention_workspace)


def _capture(run, step_args) -> "torch.cuda.CUDAGraph":
    """One eager step, which takes the library's one-time host set-up (function attributes,
    occupancy queries) so that none of it is recorded, then the recording."""
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run(**step_args, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(**step_args, stream=torch.cuda.current_stream())
    return graph


class ChunkStep:
    """Chunks of prompts, or single decoded tokens, of up to B sequences with T rows in all:
    rotates the queries and keys by ``rope``, appends K/V to the paged cache and attends.  The
    attention is in ``out``, the rotated queries in ``q``.  A sequence that st_append refuses has
    its rows of the step before in ``q``, and nothing of worth in ``out``, whatever st_attn says."""

    def __init__(self, *, T, B, Hq, Hkv, d, dtype, rope=None, scale=0.0, softcap=0.0, window=0,
                 device="cuda"):
        dev = torch.device(device)
        self.rope = rope
        self.attn_args = dict(scale=scale, softcap=softcap, window=window)
        self.q = torch.zeros((T, Hq, d), dtype=dtype, device=dev)
        self.out = torch.zeros((T, Hq, d), dtype=dtype, device=dev)
        self.st_append = torch.zeros(B, dtype=torch.int32, device=dev)
        self.st_attn = torch.zeros(B, dtype=torch.int32, device=dev)
        ws = chunk_attention_workspace(T, B, Hq, Hkv, d, dtype)
        self.workspace = torch.zeros(max(ws, 256), dtype=torch.uint8, device=dev)

    def run(self, *, q, k, v, k_cache, v_cache, block_table, q_start, prefix_lens, positions=None,
            stream=None):
        chunk_kv_append(q, k, v, k_cache, v_cache, block_table, q_start, prefix_lens,
                        self.st_append, q_out=self.q, rope=self.rope, positions=positions,
                        stream=stream)
        chunk_attention(self.q, k_cache, v_cache, block_table, q_start, prefix_lens, self.out,
                        self.st_attn, self.workspace, stream=stream, **self.attn_args)

    def capture(self, **step_args) -> "torch.cuda.CUDAGraph":
        """Records one step into a CUDA graph (see VerifyStep.capture).  q_start, prefix_lens
        and the block table are read on the device: a captured step serves any split of its T
        rows written into the same tensors."""
        return _capture(self.run, step_args)


class VerifyStep:
    """process: the target rows are raw, and ``run`` takes ``sampling`` (see there)."""

    def __init__(self, *, B, N, Hq, Hkv, d, max_blocks, bs, dtype, max_path, V=1,
                 mode=GREEDY, process=False, device="cuda"):
        self.B, self.N, self.Hq, self.Hkv, self.d = B, N, Hq, Hkv, d
        self.max_path = max_path
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.mask = torch.zeros((B, N), dtype=torch.int64, device=dev)
        self.depth = torch.zeros((B, N), **i32)
        self.st_mask = torch.zeros(B, **i32)
        self.out = torch.zeros((B, N, Hq, d), dtype=dtype, device=dev)
        self.st_attn = torch.zeros(B, **i32)
        self.accept_len = torch.zeros(B, **i32)
        self.path = torch.zeros((B, max_path), **i32)
        self.out_tokens = torch.zeros((B, max_path), **i32)
        self.st_accept = torch.zeros(B, **i32)
        self.new_lens = torch.zeros(B, **i32)
        self.src_slots = torch.zeros((B, max_path), dtype=torch.int64, device=dev)
        self.dst_slots = torch.zeros((B, max_path), dtype=torch.int64, device=dev)
        self.st_compact = torch.zeros(B, **i32)
        ws = tree_verify_attention_workspace(B, N, Hq, Hkv, d, max_blocks, bs, dtype)
        self.workspace = torch.zeros(max(ws, 256), dtype=torch.uint8, device=dev)
        aws = tree_accept_workspace(mode, B, N, V)
        self.accept_workspace = torch.zeros(max(aws, 256), dtype=torch.uint8, device=dev)
        self.target = None
        if process:
            self.target = torch.zeros((B, N, V), dtype=torch.float32, device=dev)
            self.st_process = torch.zeros(B, **i32)
            self.st_counts = torch.zeros(B, **i32)

    def mask_build(self, parents, stream=None, node_counts=None):
        tree_mask_build(parents, self.mask, self.depth, self.st_mask, stream=stream,
                        node_counts=node_counts)

    def attention(self, q, k_cache, v_cache, block_table, prefix_lens, stream=None,
                  node_counts=None):
        tree_verify_attention(q, k_cache, v_cache, block_table, prefix_lens, self.mask, self.out,
                              self.st_attn, self.workspace, stream=stream,
                              node_counts=node_counts)

    def process(self, mode, logits, draft_tokens, sampling, stream=None, node_counts=None):
        tree_logits_process(logits, self.target, self.st_process, probs=mode == STOCHASTIC,
                            mask=self.mask, draft_tokens=draft_tokens, stream=stream,
                            node_counts=node_counts, **sampling)

    def accept(self, mode, parents, draft_tokens, target, draft_probs=None, seed=0, offset=0,
               stream=None, node_counts=None):
        tree_accept(mode, parents, draft_tokens, target, draft_probs, self.accept_len, self.path,
                    self.out_tokens, self.st_accept, seed=seed, offset=offset,
                    workspace=self.accept_workspace, stream=stream, node_counts=node_counts)

    def compact(self, k_cache, v_cache, block_table, prefix_lens, stream=None):
        kv_compact(k_cache, v_cache, block_table, prefix_lens, self.path, self.accept_len,
                   self.new_lens, self.st_compact, src_slots=self.src_slots,
                   dst_slots=self.dst_slots, stream=stream)

    def run(self, *, parents, q, k_cache, v_cache, block_table, prefix_lens, draft_tokens, target,
            draft_probs=None, mode=GREEDY, seed=0, offset=0, stream=None, node_counts=None,
            sampling=None):
        """node_counts (int32 [B] on the device, or None): each sequence's tree is its
        first node_counts[b] node slots; read on the device, so a captured step serves
        any count vector written into the same tensor.
        sampling (or None: target is what tree_accept reads): tree_logits_process's counts,
        bias, grammar, repetition, frequency, presence and temperature, those that are wanted;
        target is then the target model's raw rows, float32 or bfloat16, and the tokens that
        the step emits are added to counts.  A sequence that cannot be processed, or whose
        grammar leaves nothing where a token is to be chosen, emits none (st_process,
        st_accept; out_tokens -1): its counts stay, and its cache keeps the root."""
        if sampling is not None and self.target is None:
            raise ValueError("sampling needs a step made with process=True")
        self.mask_build(parents, stream, node_counts)
        self.attention(q, k_cache, v_cache, block_table, prefix_lens, stream, node_counts)
        if sampling is not None:
            self.process(mode, target, draft_tokens, sampling, stream, node_counts)
            target = self.target
            if mode == GREEDY:
                mode = GREEDY_MASKED
        self.accept(mode, parents, draft_tokens, target, draft_probs, seed, offset, stream,
                    node_counts)
        if sampling is not None and sampling.get("counts") is not None:
            token_counts_update(sampling["counts"], self.out_tokens, self.st_counts,
                                stream=stream)
        self.compact(k_cache, v_cache, block_table, prefix_lens, stream)

    def capture(self, **step_args) -> "torch.cuda.CUDAGraph":
        """Records one step (the four launches of ``run`` with these tensors) into
        a CUDA graph; ``graph.replay()`` then re-issues it with one launch.  The
        graph keeps the tensors' addresses and the host-side choices of this call
        (schedule, tensor descriptors): refill the same input tensors in place
        between replays and keep the shapes.  One eager step first takes the
        library's one-time host set-up (function attributes, occupancy queries),
        so none of it is recorded; the caches are mutated by that step like by
        any other (compaction), and so are the token counts."""
        return _capture(self.run, step_args)


__all__ = ["ChunkStep", "VerifyStep", "GREEDY", "STOCHASTIC"]
