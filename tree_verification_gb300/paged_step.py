"""One hybrid-tree verify step over a paged KV cache, with preallocated buffers.

``PagedVerifyStep`` is ``step.VerifyStep`` for a ``paged.PagedCache``: the
step's rows go to their pages, queries and keys are rotated on the way, and
the accepted rows stay where compaction puts them.  On one CUDA stream:

    reserve (pages for Kmax rows, copy on write)  ->  graft_build_tree  ->  plan
    ->  per layer: append (rotary positions by depth, K and V into pages), attend (tree mask)
    ->  graft_accept_compact without layers (acceptance alone)  ->  compact  ->  M update

Sequences fork and leave between steps with the cache's own calls; ``active``
([n_seqs] bool on the device, all True at first) says which the next steps
verify.  An idle slot (a sequence that left, or one whose prompt is still
being appended in chunks) keeps its pages, rows and length and adds nothing to
M; its acc_len is 0, and what else the step leaves of it means nothing (its
rows of O are left alone).  Its inputs may be anything, except that its root
token has to be one and its drafter logits finite (its target logits too,
where the step samples).

A sequence for which there were not pages enough (GRAFT_STATUS_CACHE_OVERFLOW)
keeps its rows and its length where its accepted rows do not fit the pages
that it holds alone: what ``acc`` says of it did not reach the cache.

Every buffer is fixed, so a step can be captured once in a CUDA graph and
replayed; run it once before capturing (the handle's buffers grow then).
"""
from __future__ import annotations

import math
from typing import Callable, Optional, Sequence

import torch

from . import binding as gb
from .paged import PagedCache


class PagedVerifyStep:
    """Buffers of one step for all sequences of ``cache`` (its n_seqs is the batch).

    inv_freq, interleaved and factor describe the rotary positions (graft_rope_append; inv_freq None: none).
    m_policy, temperature and seed are VerifyStep's.
    """

    def __init__(self, cfg: gb.GraftConfig, cache: PagedCache, Hq: int, inv_freq: Optional[torch.Tensor] = None,
                 interleaved: bool = False, factor: float = 1.0, m_policy: str = "tree", temperature: float = 0.0,
                 seed: int = 0):
        if m_policy not in ("tree", "emitted", "both"):
            raise ValueError("m_policy must be 'tree', 'emitted' or 'both'")
        if Hq % cache.Hkv:
            raise ValueError("Hq must be a multiple of the cache's KV heads")
        cache._tables()
        self.cfg, self.cache, self.Hq = cfg, cache, Hq
        self.inv_freq, self.interleaved, self.factor = inv_freq, interleaved, float(factor)
        self.m_policy, self.temperature, self.seed = m_policy, float(temperature), int(seed)
        self.B = B = cache.n_seqs
        self.device = dev = cache.device
        self.n_layers = len(cache.K)
        K = cfg.Kmax
        i32 = dict(dtype=torch.int32, device=dev)
        self.tree = dict(tok=torch.empty(B, K, **i32), parent=torch.empty(B, K, **i32),
                         depth=torch.empty(B, K, **i32), pos=torch.empty(B, K, **i32),
                         mask=torch.empty(B, K, dtype=torch.int64, device=dev), stage=torch.empty(B, **i32))
        self.acc = dict(argmax=torch.empty(B, K, **i32), acc_len=torch.empty(B, **i32), path=torch.empty(B, K, **i32),
                        out_tok=torch.empty(B, K, **i32), bonus=torch.empty(B, **i32))
        self.status = cache.status  # one word for the step's calls and the cache's
        u8 = dict(dtype=torch.uint8, device=dev)
        with torch.cuda.device(dev):  # (sizes that go by the device)
            self.ws_tree = torch.zeros(max(1, gb.graft_build_tree_workspace_size(cfg, B)), **u8)
            self.ws_acc = torch.empty(max(1, gb.graft_accept_compact_workspace_size(B, K, cfg.V)), **u8)
            self.ws_upd = torch.empty(max(1, gb.graft_update_M_workspace_size(B * K)), **u8)
            self.ws_emit = torch.empty(max(1, gb.graft_update_M_emitted_workspace_size(B, K)), **u8)
            self.ws_smp = torch.empty(max(1, gb.graft_sample_tokens_workspace_size(B, K, cfg.V)), **u8)
        self.q_start = (torch.arange(B + 1, **i32) * K).contiguous()
        self.rows = torch.full((B,), K, **i32)
        self.active = torch.ones(B, dtype=torch.bool, device=dev)
        self._src = torch.empty(B, K, **i32)  # tree tokens for M, -1 (no pair) in idle slots
        self._none = torch.full((), gb.EMPTY_TOKEN, **i32)
        self._no_layers = torch.empty(0, dtype=torch.int64, device=dev)
        self._lengths = torch.empty(B, **i32)  # the acceptance's copy (0 in idle slots): compaction advances the cache's own
        self.O = torch.zeros(B, K, Hq, gb.HEAD_DIM, dtype=cache.dtype, device=dev)
        self.Qr = torch.empty_like(self.O)
        self.scale = 1.0 / math.sqrt(gb.HEAD_DIM)
        self.graph: Optional[torch.cuda.CUDAGraph] = None

    def run(self, draft_logits, root_tok, M_succ, M_cnt, Q: Sequence[torch.Tensor], K: Sequence[torch.Tensor],
            V: Sequence[torch.Tensor], target_logits, attended: Optional[Callable[[int, torch.Tensor], None]] = None,
            inputs_ready: Optional[Callable[[object], None]] = None) -> None:
        """Enqueue one step on the current stream of the cache's device (asynchronous).

        Q, K, V: per layer, [B * Kmax][heads][128] rows before rotation (they may be columns of one matrix).
        ``attended`` is called with (layer, O) after each layer's attention is enqueued (O is overwritten by the
        next layer); ``inputs_ready`` as in VerifyStep.run ("tree", each layer's index, "accept").
        """
        with torch.cuda.device(self.device):  # (the calls that are not the handle's go by the current device)
            self._run(draft_logits, root_tok, M_succ, M_cnt, Q, K, V, target_logits, attended, inputs_ready)

    def _run(self, draft_logits, root_tok, M_succ, M_cnt, Q, K, V, target_logits, attended, inputs_ready) -> None:
        c, B, Kmax = self.cache, self.B, self.cfg.Kmax
        ready = inputs_ready if inputs_ready is not None else (lambda _: None)
        ready("tree")
        on, part = self.active, c._with(self.active)
        c.reserve(self.rows, active=part)
        gb.graft_build_tree(self.cfg, draft_logits, root_tok, M_succ, c.lengths, out=self.tree, status=self.status,
                            ws=self.ws_tree)
        c.plan(self.q_start, B * Kmax, self.Hq, Kmax, tree=True, active=part)
        pos, mask = self.tree["pos"].view(-1), self.tree["mask"].view(-1)
        q, o = self.Qr.view(B * Kmax, self.Hq, gb.HEAD_DIM), self.O.view(B * Kmax, self.Hq, gb.HEAD_DIM)
        for layer in range(self.n_layers):
            ready(layer)
            c.append(layer, Q[layer], K[layer], V[layer], self.q_start, inv_freq=self.inv_freq,
                     interleaved=self.interleaved, positions=pos, factor=self.factor, out=q, active=part)
            c.attend(layer, q, self.scale, mask=mask, out=o)
            if attended is not None:
                attended(layer, self.O)
        ready("accept")
        torch.mul(c.lengths, on, out=self._lengths)
        tables = [self._no_layers] * 4
        args = (self.tree["tok"], self.tree["parent"], self.tree["depth"], *tables, 0, c.Hkv,
                c.max_pages * c.page_rows, self._lengths)
        if self.temperature > 0.0:
            gb.graft_sample_tokens(target_logits, self.tree["pos"], self.temperature, self.seed,
                                   sampled=self.acc["argmax"], ws=self.ws_smp)
            gb.graft_accept_compact(None, *args, out=self.acc, status=self.status, ws=self.ws_acc,
                                    argmax=self.acc["argmax"], V=self.cfg.V)
        else:
            gb.graft_accept_compact(target_logits, *args, out=self.acc, status=self.status, ws=self.ws_acc)
        self.acc["acc_len"].mul_(on)
        c.compact(self.acc["path"], self.acc["acc_len"], active=part)
        if self.m_policy in ("tree", "both"):
            torch.where(on[:, None], self.tree["tok"], self._none, out=self._src)
            gb.graft_update_M(M_succ, M_cnt, self._src.view(-1), self.acc["argmax"].view(-1), status=self.status,
                              ws=self.ws_upd)
        if self.m_policy in ("emitted", "both"):
            gb.graft_update_M_emitted(M_succ, M_cnt, self.tree["tok"], self.acc["out_tok"], self.acc["acc_len"],
                                      status=self.status, ws=self.ws_emit)

    def capture(self, *args, **kw) -> torch.cuda.CUDAGraph:
        """Capture run(*args) into a CUDA graph (the arguments' storage is baked in).

        The step runs once outside the capture first, on the cache and M as they are: restore them afterwards if
        that step is not wanted."""
        with torch.cuda.device(self.device):
            g = torch.cuda.CUDAGraph()
            s = torch.cuda.Stream(device=self.device)
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                self.run(*args, **kw)
            torch.cuda.current_stream().wait_stream(s)
            torch.cuda.synchronize(self.device)
            with torch.cuda.graph(g):
                self.run(*args, **kw)
        self.graph = g
        return g
