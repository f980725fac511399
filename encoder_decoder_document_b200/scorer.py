"""One query against a ragged batch of documents: the four scoring steps chained.

``FBNLScorer`` owns the decoder weights (device, bf16) and reusable device
buffers, and runs, on one stream:

  kalm_ragged_offsets -> kalm_chunk_pool (document cache) -> kalm_cross_kv_proj
  (all layers at once) -> kalm_broadcast_rows (the query's decoder input for
  every document) -> per layer: kalm_linear (Q | K_self | V_self),
  kalm_merged_attention, kalm_linear (output projection + residual) ->
  kalm_yes_no_score.

With norm weights (``DeviceWeights.w_norm_pre`` and the fields after it) every
block reads kalm_rms_norm / kalm_norm_residual outputs instead of the plain
residual stream.  Documents that many queries name can live in a
``DocumentCache`` (``new_cache``, ``cache_put``): ``rerank_cached`` scores any of
them, the attention reading their cross K/V in 8 bits
(kalm_merged_attention_cache).

Python only sequences the calls and owns the buffers; every step runs in the
CUDA kernels of libkalm.  ``capture()`` records the whole sequence in a CUDA
graph so a query costs one graph launch.  ``rerank()`` is the user-facing call:
host inputs in, the best-first list out ("KaLM-Reranker-V1-Nano - MLX",
"Usage": rerank returns {index, relevance_score} entries, highest first;
"KaLM-Reranker-V1-Small-Q4_K_M-GGUF", "Score a pair": larger margins rank first).
"""
from __future__ import annotations

import dataclasses
from typing import Optional

import numpy as np
import torch

from . import (kalm_broadcast_rows, kalm_check_device_errors, kalm_chunk_pool, kalm_cross_kv_proj,
               kalm_device_check, kalm_linear, kalm_merged_attention_out_proj, kalm_attention_out_proj_sync_len,
               kalm_merged_attention, kalm_ragged_offsets, kalm_yes_no_score, kalm_attention_items,
               kalm_attention_schedule, kalm_linear_rope, kalm_rope_table, kalm_linear_chain,
               kalm_linear_chain_rope, kalm_linear_chain_sync_len, kalm_merged_attention_cache,
               kalm_merged_attention_cache_rows, kalm_norm_residual, kalm_rms_norm)
from .document_cache import CacheView, DocumentCache

HEAD_DIM = 256
# the pages' runtime limits ("Runtime boundaries"): passages of at most 1,024 encoder
# tokens, a query budget of 512 tokens
MAX_DOC_TOKENS = 1024
MAX_QUERY_TOKENS = 512


def bf16_from_bits(bits: np.ndarray, device="cuda") -> torch.Tensor:
    """uint16 bf16 bit patterns (host) -> bf16 device tensor (bit-exact)."""
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16))
    return t.to(device).view(torch.bfloat16)


@dataclasses.dataclass
class DeviceWeights:
    w_qkv: torch.Tensor       # [L][(n_q + 2 n_kv) D][H]
    w_o: torch.Tensor         # [L][H][n_q D]
    w_kv_cross: torch.Tensor  # [L][2 n_kv D][H]
    w_yes: torch.Tensor       # [H]
    w_no: torch.Tensor        # [H]
    # the norms around the blocks (None: the plain residual stack)
    w_norm_pre: Optional[torch.Tensor] = None    # [L][H], before each block's Q|K|V projection
    w_norm_post: Optional[torch.Tensor] = None   # [L][H], of each block's output
    gate: Optional[torch.Tensor] = None          # [L][H], times the (normed) block output
    w_norm_final: Optional[torch.Tensor] = None  # [H], before the readout
    norm_eps: float = 1e-6
    norm_weight_offset: float = 0.0              # 1.0 for checkpoints that store the weights minus one
    residual_scale: float = 1.0                  # of the residual stream at each block's sum

    @classmethod
    def from_bits(cls, w, device="cuda") -> "DeviceWeights":
        return cls(bf16_from_bits(w.w_qkv, device), bf16_from_bits(w.w_o, device),
                   bf16_from_bits(w.w_kv_cross, device), bf16_from_bits(w.w_yes, device),
                   bf16_from_bits(w.w_no, device))


CACHE_PUT_BYTES = 1 << 30  # bf16 cross K/V that cache_put holds at a time

# What prepare(), use_slot() and capture() keep of one query shape.
_PREPARED = ("_shape", "n_docs", "total_tokens", "total_pooled", "lq", "slots", "slot", "enc", "doc_len", "x0", "tok_off",
             "pool_off", "q_off", "zero_off", "one_doc_off", "pooled", "kv_cross", "qkv", "o", "x", "h", "y", "h0", "result",
             "yes", "no", "margin", "score", "order", "sync", "chain_sync", "graph", "graphs", "graphs_decode", "graph_inst")


class FBNLScorer:
    """Scores one query's documents.  With ``prune`` (the default) work that
    cannot reach the score is skipped, exactly: the first layer's Q/K/V are
    computed once for the query's common decoder input (every document starts
    from it), and the last layer computes attention only for the query tile that
    holds each document's final row and the output projection only for that row
    (the readout reads nothing else)."""

    def __init__(self, weights: DeviceWeights, n_q: int, n_kv: int, chunk: int = 4, head_dim: int = HEAD_DIM,
                 prune: bool = True, rope_theta: Optional[float] = None, fused_out: bool = False,
                 chain: bool = True):
        kalm_device_check()
        self.w = weights
        self.L, qkv_rows, self.H = weights.w_qkv.shape
        self.n_q, self.n_kv, self.D, self.chunk = n_q, n_kv, head_dim, chunk
        assert qkv_rows == (n_q + 2 * n_kv) * head_dim
        self.scale = head_dim ** -0.5
        self.prune = prune
        self.norms = weights.w_norm_pre is not None
        if not self.norms and (weights.w_norm_post is not None or weights.gate is not None or
                               weights.w_norm_final is not None or weights.residual_scale != 1.0):
            raise ValueError("w_norm_post, gate, w_norm_final and residual_scale need w_norm_pre")
        if self.norms and fused_out:
            raise ValueError("fused_out adds the residual in its projection: it does not go with norms")
        self.rope_theta = rope_theta  # rotary base for the decoder's self Q/K, or None (no rotation)
        # attention and output projection of every layer but the pruned last one in one
        # launch (kalm_merged_attention_out_proj)
        self.fused_out = fused_out
        # each layer's output projection and the next layer's Q|K|V projection in one launch
        # (kalm_linear_chain, or kalm_linear_chain_rope with rotation), in the pruned stack
        # without the fused layer
        self.chain = chain and prune and not fused_out and not self.norms
        self.view: Optional[CacheView] = None  # documents of a DocumentCache being scored
        self._qkv_ready = -1  # layer whose Q|K|V the last chained launch produced
        # the rotary angles' (cos, sin), built once for this base
        self.rope_tab = kalm_rope_table(rope_theta, head_dim) if rope_theta is not None else None
        self._shape = None
        self.graph: Optional[torch.cuda.CUDAGraph] = None
        self.graphs = None
        self.graphs_decode = None
        self.graph_inst = None
        self._cached_set: dict = {}  # the buffers of queries over a DocumentCache, while this query's own are in place
        # optional per-launch timing: (label, event) recorded after every entry-point call
        self.marks: Optional[list] = None
        self.launches = 0  # kernel launches issued by the last forward()
        self.side: Optional[torch.cuda.Stream] = None  # second stream for work beside the pooling
        self._side_pending = False  # the broadcast of X is on the second stream, not yet joined

    # ------------------------------------------------------------------ buffers
    def prepare(self, n_docs: int, total_tokens: int, total_pooled: int, lq: int, device="cuda") -> None:
        """Allocate the device buffers for one query shape (re-used across calls)."""
        shape = (n_docs, total_tokens, total_pooled, lq)
        if self._shape == shape:
            return
        # until every buffer is there: a failed allocation leaves nothing half prepared, and no graph over freed buffers
        self._shape = self.graph = self.graphs = self.graphs_decode = None
        D, H, L = self.D, self.H, self.L
        rows = n_docs * lq
        kw = dict(device=device)
        self.n_docs, self.total_tokens, self.total_pooled, self.lq = shape
        # two input slots, so the next query's inputs can be copied while this one runs; until then, and until their
        # offsets are computed, the documents are empty (a step on memory's leftovers could walk any length)
        self.slots = [dict(enc=torch.empty(max(total_tokens, 1), H, dtype=torch.bfloat16, **kw),
                           doc_len=torch.zeros(n_docs, dtype=torch.int32, **kw),
                           x0=torch.zeros(lq, H, dtype=torch.bfloat16, **kw)) for _ in range(2)]
        self.use_slot(0)
        self.tok_off = torch.zeros(n_docs + 1, dtype=torch.int64, **kw)
        self.pool_off = torch.zeros(n_docs + 1, dtype=torch.int64, **kw)
        # every document of a query has the query's Lq decoder rows, so their offsets belong
        # to the shape and are fixed here once (document d's rows start at d * Lq)
        self.q_off = torch.arange(n_docs + 1, dtype=torch.int64, **kw) * lq
        self.zero_off = torch.zeros(n_docs, dtype=torch.int64, **kw)
        self.one_doc_off = torch.tensor([0, lq], dtype=torch.int64, **kw)  # the query's common rows
        self.pooled = torch.empty(max(total_pooled, 1), H, dtype=torch.bfloat16, **kw)
        self.kv_cross = torch.empty(max(total_pooled, 1), L * 2 * self.n_kv * D, dtype=torch.bfloat16, **kw)
        self.qkv = torch.empty(rows, (self.n_q + 2 * self.n_kv) * D, dtype=torch.bfloat16, **kw)
        self.o = torch.empty(rows, self.n_q * D, dtype=torch.bfloat16, **kw)
        self.x = torch.empty(rows, H, dtype=torch.bfloat16, **kw)
        if self.norms:  # a block's normed input (and that of the query's common rows), and its output
            self.h, self.y = (torch.empty(rows, H, dtype=torch.bfloat16, **kw) for _ in range(2))
            self.h0 = torch.empty(lq, H, dtype=torch.bfloat16, **kw)
        # (yes, no, margin, score) rows of one buffer: one device->host copy per query
        self.result = torch.empty(4, n_docs, dtype=torch.float32, **kw)
        # work order of the full-layer attention launches (same costs in every layer); in index order until scheduled
        self.order = torch.arange(max(kalm_attention_items(n_docs, lq, self.n_q, self.n_kv), 1), dtype=torch.int32,
                                  **kw)
        self.yes, self.no, self.margin, self.score = self.result[0], self.result[1], self.result[2], self.result[3]
        # the fused layer's per-document counters (zero before a launch, left zero by it)
        self.sync = torch.zeros(max(kalm_attention_out_proj_sync_len(n_docs, lq, H), 1), dtype=torch.int32, **kw)
        # the chained projections' per-row-block counters (zero before a launch, left zero by it)
        self.chain_sync = torch.zeros(max(kalm_linear_chain_sync_len(rows), 1), dtype=torch.int32, **kw)
        self._shape = shape

    def use_slot(self, i: int) -> None:
        """Point the input buffers at slot i (for the next forward() or capture)."""
        self.slot = i
        self.enc, self.doc_len, self.x0 = (self.slots[i][k] for k in ("enc", "doc_len", "x0"))

    def _exchange(self, other: dict) -> dict:
        """Put another prepared set in place (empty: none yet) and return the one that was."""
        mine = {k: self.__dict__.pop(k) for k in _PREPARED if k in self.__dict__}
        if mine["graph_inst"] is not None:  # the marks are its events
            mine["marks"], self.marks = self.marks, None
        self.__dict__.update(dict(_shape=None, graph=None, graphs=None, graphs_decode=None, graph_inst=None) | other)
        return mine

    # ------------------------------------------------------------------ steps
    def _mark(self, label: str) -> None:
        self.launches += 1
        if self.marks is not None:
            ev = torch.cuda.Event(enable_timing=True, external=True)
            ev.record()
            self.marks.append((label, ev))

    def pool(self, side: Optional[torch.cuda.Stream] = None) -> None:
        """Offsets, attention work order, pooled document cache.  With a ``side`` stream
        the work order and the query input broadcast (both need only the offsets) run
        there, beside the pooling and the cross projection; the caller joins it."""
        self.view = None  # the documents are this query's own
        kalm_ragged_offsets(self.doc_len, self.tok_off, self.pool_off, self.chunk)
        self._mark("offsets")
        if side is not None:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                kalm_attention_schedule(self.q_off, self.pool_off, self.lq, self.n_q, self.n_kv, self.order)
                kalm_broadcast_rows(self.x0, self.q_off, self.x)
            self.launches += 2
        else:
            kalm_attention_schedule(self.q_off, self.pool_off, self.lq, self.n_q, self.n_kv, self.order)
            self._mark("schedule")
        kalm_chunk_pool(self.enc, self.tok_off, self.doc_len, self.pooled, self.pool_off, self.total_pooled,
                        self.chunk)
        self._mark("chunk_pool")

    def cross_kv(self) -> None:
        kalm_cross_kv_proj(self.pooled[: self.total_pooled], self.w.w_kv_cross, self.kv_cross[: self.total_pooled],
                           self.n_kv, self.D)
        self._mark("cross_kv_proj")

    def cross_views(self, l: int):
        w = self.n_kv * self.D
        kc = self.kv_cross[:, (2 * l) * w:(2 * l + 1) * w]
        vc = self.kv_cross[:, (2 * l + 1) * w:(2 * l + 2) * w]
        return kc, vc

    def qkv_views(self):
        D, nq, nkv = self.D, self.n_q, self.n_kv
        return (self.qkv[:, : nq * D], self.qkv[:, nq * D:(nq + nkv) * D], self.qkv[:, (nq + nkv) * D:])

    def qkv_proj(self, x: torch.Tensor, l: int, qkv: torch.Tensor, q_off: torch.Tensor) -> None:
        """Fused Q|K|V projection; with a rotary base the self Q and K heads are
        rotated in the projection's epilogue."""
        if self.rope_theta is None:
            kalm_linear(x, self.w.w_qkv[l], qkv)
        else:
            kalm_linear_rope(x, self.w.w_qkv[l], qkv, q_off, self.n_q + self.n_kv, self.rope_tab, self.D)
        self._mark("qkv_proj")

    def layer_qkv(self, l: int) -> None:
        self.qkv_proj(self.h if self.norms else self.x, l, self.qkv, self.q_off)

    def attend(self, l: int, q, ks, vs, in_off=None, last_tile_only: bool = False) -> None:
        """Merged attention of layer l into self.o, over this query's own documents or the cached ones."""
        if self.view is None:
            kc, vc = self.cross_views(l)
            kalm_merged_attention(q, ks, vs, kc, vc, self.q_off, self.pool_off, self.lq, self.n_q, self.n_kv, self.o,
                                  self.scale, in_off=in_off, last_tile_only=last_tile_only,
                                  order=None if last_tile_only else self.order)
        else:
            cache, w = self.view_cache, self.n_kv * self.D
            k, v = 2 * l * w, (2 * l + 1) * w
            g = cache.width // cache.scales.shape[1]
            kalm_merged_attention_cache(q, ks, vs, cache.codes[:, k:k + w], cache.scales[:, k // g:(k + w) // g],
                                        cache.codes[:, v:v + w], cache.scales[:, v // g:(v + w) // g],
                                        self.view.page_table, cache.page_rows, self.q_off, self.view.row_off, self.lq,
                                        self.n_q, self.n_kv, self.o, self.scale, in_off=in_off,
                                        last_tile_only=last_tile_only,
                                        order=None if last_tile_only else self.view_order, workspace=self.view_ws)
        self._mark("merged_attention")

    def layer_attention(self, l: int) -> None:
        q, ks, vs = self.qkv_views()
        self.attend(l, q, ks, vs)

    def _join_side(self) -> None:
        """The residual stream X is first read by an output projection: wait for the
        broadcast if it was issued on the second stream."""
        if self._side_pending:
            torch.cuda.current_stream().wait_stream(self.side)
            self._side_pending = False

    def layer_out(self, l: int) -> None:
        self._join_side()
        kalm_linear(self.o, self.w.w_o[l], self.x, residual=self.x)
        self._mark("o_proj")

    def block_out(self, l: int, last_rows_only: bool = False) -> None:
        """With norms: output projection of block l, its norm and gate, the residual sum and the norm
        before what comes next (block l + 1, or the readout), of every row or each document's last."""
        rows = slice(self.lq - 1, None, self.lq) if last_rows_only else slice(None)
        o, y, x, h = self.o[rows], self.y[rows], self.x[rows], self.h[rows]
        w = self.w
        self._join_side()
        kalm_linear(o, w.w_o[l], y)
        self._mark("o_proj")
        w_next = w.w_norm_pre[l + 1] if l + 1 < self.L else w.w_norm_final
        kalm_norm_residual(y, x, x, h=h if w_next is not None else None,
                           w_post=w.w_norm_post[l] if w.w_norm_post is not None else None, w_pre=w_next,
                           gate=w.gate[l] if w.gate is not None else None, residual_scale=w.residual_scale,
                           eps=w.norm_eps, weight_offset=w.norm_weight_offset)
        self._mark("norm_residual")

    def first_norm(self, x: torch.Tensor, h: torch.Tensor) -> torch.Tensor:
        """Block 0's input: the norm of x into h, or x itself without norms."""
        if not self.norms:
            return x
        kalm_rms_norm(x, self.w.w_norm_pre[0], h, eps=self.w.norm_eps, weight_offset=self.w.norm_weight_offset)
        self._mark("rms_norm")
        return h

    def attention_out(self, l: int, q, ks, vs, in_off=None) -> None:
        """Fused attention + output projection of layer l (X updated in place)."""
        kc, vc = self.cross_views(l)
        self._join_side()
        kalm_merged_attention_out_proj(q, ks, vs, kc, vc, self.q_off, self.pool_off, self.lq, self.n_q, self.n_kv,
                                       self.o, self.w.w_o[l], self.x, self.sync, self.scale, in_off=in_off,
                                       order=self.order)
        self._mark("attention_out_proj")

    def layer(self, l: int) -> None:
        if l == 0:
            self.first_norm(self.x, self.h if self.norms else self.x)
        self.layer_qkv(l)
        if self.fused_out and self.view is None:
            q, ks, vs = self.qkv_views()
            self.attention_out(l, q, ks, vs)
            return
        self.layer_attention(l)
        if self.norms:
            self.block_out(l)
        else:
            self.layer_out(l)

    def layer_pruned(self, l: int) -> None:
        """Layer l with the exact pruning described in the class docstring."""
        first, last = l == 0, l == self.L - 1
        Lq = self.lq
        if first:
            # every document's decoder input is the query's common input: one Q|K|V for all
            self.qkv_proj(self.first_norm(self.x0, self.h0 if self.norms else self.x0), l, self.qkv[:Lq],
                          self.one_doc_off)
            q, ks, vs = (t[:Lq] for t in self.qkv_views())
            in_off = self.zero_off
        else:
            if not (self.chain and self._qkv_ready == l):  # else the previous launch projected them
                self.layer_qkv(l)
            q, ks, vs = self.qkv_views()
            in_off = None
        if self.fused_out and not last and self.view is None:
            self.attention_out(l, q, ks, vs, in_off)
            return
        self.attend(l, q, ks, vs, in_off, last)
        if self.norms:
            self.block_out(l, last_rows_only=last)
        elif last:
            # only each document's final row reaches the readout
            x_last = self.x[Lq - 1::Lq]
            self._join_side()
            kalm_linear(self.o[Lq - 1::Lq], self.w.w_o[l], x_last, residual=x_last)
            self._mark("o_proj")
        elif self.chain:
            # X += O Wo, then the next layer's Q|K|V from the updated X, in one launch
            self._join_side()
            if self.rope_theta is None:
                kalm_linear_chain(self.o, self.w.w_o[l], self.x, self.w.w_qkv[l + 1], self.qkv, self.chain_sync)
            else:
                kalm_linear_chain_rope(self.o, self.w.w_o[l], self.x, self.w.w_qkv[l + 1], self.qkv, self.q_off,
                                       self.n_q + self.n_kv, self.rope_tab, self.chain_sync, self.D)
            self._mark("o_proj_qkv")
            self._qkv_ready = l + 1
        else:
            self.layer_out(l)

    def readout(self) -> None:
        hidden = self.h if self.w.w_norm_final is not None else self.x
        kalm_yes_no_score(hidden, self.q_off, self.w.w_yes, self.w.w_no, self.yes, self.no, self.score,
                          self.margin)
        self._mark("yes_no_score")

    def documents(self) -> None:
        """The document side: offsets, the pooled document cache and every layer's cross K/V."""
        self.pool()
        self.cross_kv()

    def decode(self, broadcast: bool = True) -> None:
        """The query side: the decoder stack over the cached cross K/V, then the readout."""
        self._qkv_ready = -1
        if broadcast and self.marks is None and self.prune:
            # layer 0's Q|K|V and attention read only the query input: the broadcast of X
            # runs beside them and the first output projection waits for it
            if self.side is None:
                self.side = torch.cuda.Stream()
            self.side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(self.side):
                kalm_broadcast_rows(self.x0, self.q_off, self.x)
            self.launches += 1
            self._side_pending = True
        elif broadcast:
            kalm_broadcast_rows(self.x0, self.q_off, self.x)
            self._mark("broadcast")
        for l in range(self.L):
            if self.prune:
                self.layer_pruned(l)
            else:
                self.layer(l)
        self.readout()

    def forward(self, cached: bool = False) -> None:
        """All steps on the current stream, from the inputs in self.enc / doc_len / x0.

        With ``cached`` only decode() runs: the documents' offsets, work order and
        cross K/V from the last full forward over the same documents are reused
        (the persistent-cache regime: one document set, many queries)."""
        if self._shape is None:
            raise RuntimeError("forward needs prepare() first")
        self.launches = 0
        if self.marks is not None:
            self._mark("start")
            self.launches = 0
        if cached:
            self.decode()
        elif self.marks is None:
            # the work order and the broadcast beside the pooling and cross projection
            if self.side is None:
                self.side = torch.cuda.Stream()
            self.pool(side=self.side)
            self.cross_kv()
            torch.cuda.current_stream().wait_stream(self.side)
            self.decode(broadcast=False)
        else:  # instrumented: one launch after another, so each gets its own interval
            self.documents()
            self.decode()

    def capture(self, instrument: bool = False) -> None:
        """Record forward() as a CUDA graph (buffers must stay allocated).

        With ``instrument`` a second graph is recorded with an external timing
        event after every launch (``graph_inst``), so each of its replays yields
        per-kernel durations (``kernel_times()``).  The events sit between the
        launches and keep them from overlapping, so the plain graph is the one to
        time a step with."""
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            self.forward()  # warm-up: one-time device set-up happens outside capture
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        self.marks = None
        slot = self.slot
        self.graphs = []
        for i in range(2):  # one graph per input slot
            self.use_slot(i)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                self.forward()
            self.graphs.append(g)
        self.graphs_decode = []
        for i in range(2):  # decode-only graphs (persistent-cache regime), one per input slot
            self.use_slot(i)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                self.forward(cached=True)
            self.graphs_decode.append(g)
        self.use_slot(slot)
        self.graph = self.graphs[slot]
        self.graph_inst = None
        if instrument:
            self.marks = []
            gi = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gi):
                self.forward()
            self.graph_inst = gi

    def kernel_times(self) -> dict:
        """{label: [ms per launch, ...]} of the last replay of the instrumented graph."""
        out: dict = {}
        if not self.marks:
            return out
        for (_, a), (label, b) in zip(self.marks[:-1], self.marks[1:]):
            out.setdefault(label, []).append(a.elapsed_time(b))
        return out

    def run(self) -> None:
        if self.graph is not None:
            self.graph.replay()
        else:
            self.forward()

    # ------------------------------------------------------------------ user API
    def load_inputs(self, enc_host: torch.Tensor, doc_len_host: torch.Tensor, x0_host: torch.Tensor) -> None:
        """Host -> device copies of one query's inputs (pinned host tensors copy asynchronously)."""
        self.enc[: enc_host.shape[0]].copy_(enc_host, non_blocking=True)
        self.doc_len.copy_(doc_len_host, non_blocking=True)
        self.x0.copy_(x0_host, non_blocking=True)

    def scores_to_host(self, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Device -> host copy of (yes, no, margin, score) as a [4][n_docs] fp32 tensor."""
        if out is None:
            return self.result.cpu()
        out.copy_(self.result, non_blocking=True)
        return out

    def score_stream(self, inputs, outs) -> None:
        """Score a stream of queries of this shape, overlapping transfers with compute.

        inputs[k] = (enc, doc_len, x0) pinned host tensors of query k; outs[k] a
        pinned [4][n_docs] fp32 host tensor that receives (yes, no, margin, score).
        Query k+1's inputs are copied on a side stream into the other input slot
        while query k runs (one captured graph per slot); every copy and every
        result read happen inside the call, which returns without synchronising.
        Device errors (an expired bounded wait, invalid device data) are only
        flagged on the device: call ``check_errors()`` before trusting ``outs``.
        Requires capture() first."""
        if self.graphs is None:
            raise RuntimeError("score_stream needs capture() first")
        comp = torch.cuda.current_stream()
        if getattr(self, "_copy_stream", None) is None:
            self._copy_stream = torch.cuda.Stream()
            self._ready = [torch.cuda.Event(), torch.cuda.Event()]
            self._free = [torch.cuda.Event(), torch.cuda.Event()]
        cs = self._copy_stream
        cs.wait_stream(comp)

        def h2d(k):
            i = k % 2
            slot = self.slots[i]
            with torch.cuda.stream(cs):
                if k >= 2:
                    cs.wait_event(self._free[i])  # the query that last used this slot is done with it
                enc, doc_len, x0 = inputs[k]
                slot["enc"][: enc.shape[0]].copy_(enc, non_blocking=True)
                slot["doc_len"].copy_(doc_len, non_blocking=True)
                slot["x0"].copy_(x0, non_blocking=True)
                self._ready[i].record(cs)

        if inputs:
            h2d(0)
        for k in range(len(inputs)):
            if k + 1 < len(inputs):
                h2d(k + 1)
            i = k % 2
            comp.wait_event(self._ready[i])
            self.graphs[i].replay()
            self._free[i].record(comp)
            outs[k].copy_(self.result, non_blocking=True)

    def cache_documents(self, enc_host: torch.Tensor, doc_len_host: torch.Tensor) -> None:
        """Build the document cache (pooled vectors and every layer's cross K/V) for a
        document set that many queries will be scored against; stream-ordered.  Both
        input slots share the cache, so score_cached_stream can use either."""
        for slot in self.slots:
            slot["enc"][: enc_host.shape[0]].copy_(enc_host, non_blocking=True)
            slot["doc_len"].copy_(doc_len_host, non_blocking=True)
        self.documents()

    def score_cached_stream(self, x0s, outs) -> None:
        """Score queries against the cached documents (decode-only graphs), overlapping
        each query's decoder-input copy with the previous query's compute.

        x0s[k]: pinned host bf16 [lq][H] decoder input of query k; outs[k]: pinned
        [4][n_docs] fp32 host tensor for (yes, no, margin, score).  Returns without
        synchronising; call ``check_errors()`` before trusting ``outs``.  Requires
        cache_documents() (or a full forward over the same documents) and capture()."""
        if not getattr(self, "graphs_decode", None):
            raise RuntimeError("score_cached_stream needs capture() first")
        comp = torch.cuda.current_stream()
        if getattr(self, "_copy_stream", None) is None:
            self._copy_stream = torch.cuda.Stream()
            self._ready = [torch.cuda.Event(), torch.cuda.Event()]
            self._free = [torch.cuda.Event(), torch.cuda.Event()]
        cs = self._copy_stream
        cs.wait_stream(comp)

        def h2d(k):
            i = k % 2
            with torch.cuda.stream(cs):
                if k >= 2:
                    cs.wait_event(self._free[i])
                self.slots[i]["x0"].copy_(x0s[k], non_blocking=True)
                self._ready[i].record(cs)

        if x0s:
            h2d(0)
        for k in range(len(x0s)):
            if k + 1 < len(x0s):
                h2d(k + 1)
            i = k % 2
            comp.wait_event(self._ready[i])
            self.graphs_decode[i].replay()
            self._free[i].record(comp)
            outs[k].copy_(self.result, non_blocking=True)

    def rerank(self, x0: np.ndarray, enc: np.ndarray, doc_len: np.ndarray, top_n: Optional[int] = None):
        """Score one query's documents and return [{index, relevance_score}] best first.

        x0: bf16 bits [lq][H] (decoder input of the query); enc: bf16 bits
        [sum(doc_len)][H] (packed encoder states); doc_len: int [n_docs]."""
        res = self.score_rows(x0, enc, doc_len)
        return rank(res[:, 2], res[:, 3], top_n)

    def rerank_sharded(self, x0: np.ndarray, enc: np.ndarray, doc_len: np.ndarray, top_n: Optional[int] = None,
                       group=None):
        """``rerank`` over the documents of one query split across the ranks of a
        process group (one process per GPU, each with its own scorer): every rank
        passes the whole query, scores its share of the documents (balanced by
        length) and receives the full ranking.  The only exchange is one gather of the
        per-document scores on the host."""
        from .sharding import sharded_rerank
        return sharded_rerank(self.score_rows, x0, enc, doc_len, top_n, group)

    def score_rows(self, x0: np.ndarray, enc: np.ndarray, doc_len: np.ndarray) -> np.ndarray:
        """Rows (yes, no, margin, score) of one query's documents, in input order
        (``[n_docs][4]`` float32 on the host); arguments as for ``rerank``."""
        doc_len = np.asarray(doc_len)
        if doc_len.ndim != 1:
            raise ValueError("rerank: doc_len must be one length per document")
        if doc_len.size and (doc_len.min() < 0 or doc_len.max() > MAX_DOC_TOKENS):
            raise ValueError(f"rerank: document lengths must lie in [0, {MAX_DOC_TOKENS}] "
                             f"(got {int(doc_len.min())}..{int(doc_len.max())})")
        lq = int(np.asarray(x0).shape[0])
        if not 1 <= lq <= MAX_QUERY_TOKENS:
            raise ValueError(f"rerank: the query input must have 1..{MAX_QUERY_TOKENS} rows (got {lq})")
        doc_len = doc_len.astype(np.int32)
        n = int(doc_len.shape[0])
        if n == 0:
            return np.zeros((0, 4), dtype=np.float32)
        total_tokens = int(doc_len.sum())
        if np.asarray(enc).shape[0] < total_tokens:
            raise ValueError(f"rerank: enc holds {np.asarray(enc).shape[0]} rows, doc_len sums to {total_tokens}")
        total_pooled = int(((doc_len.astype(np.int64) + self.chunk - 1) // self.chunk).sum())
        self.prepare(n, total_tokens, total_pooled, lq)
        self.load_inputs(torch.from_numpy(np.ascontiguousarray(enc).view(np.int16)).view(torch.bfloat16),
                         torch.from_numpy(doc_len), torch.from_numpy(np.ascontiguousarray(x0).view(np.int16))
                         .view(torch.bfloat16))
        self.run()
        res = self.scores_to_host().numpy()
        # a bounded wait that expired or invalid device data leaves only a flag on the
        # device: raise instead of returning scores computed past it
        self.check_errors()
        return np.ascontiguousarray(res.T)

    # ------------------------------------------------------------------ 8-bit document cache
    def new_cache(self, n_pages: int, page_rows: int = 64, device="cuda") -> DocumentCache:
        """A cache for this stack: a row holds the cross K/V of every layer of one pooled vector
        (kalm_cross_kv_proj's layout) in 8 bits, n_layers * 2 * n_kv * head_dim * 33 / 32 bytes."""
        return DocumentCache(n_pages, self.L * 2 * self.n_kv * self.D, page_rows, device, self._cache_layout())

    def _cache_layout(self) -> tuple:
        return ("cross K/V", self.L, self.n_kv, self.D)

    def cache_put(self, cache: DocumentCache, keys, enc: np.ndarray, doc_len: np.ndarray) -> None:
        """Pool documents, project their cross K/V and store them under ``keys``; arguments as for
        ``rerank`` (enc: bf16 bits of the documents' encoder states, packed).  Documents go through in groups
        whose cross K/V in bf16 take at most CACHE_PUT_BYTES; all of them are stored, or none."""
        self._check_cache(cache)
        doc_len = np.asarray(doc_len)
        if doc_len.ndim != 1 or len(keys) != doc_len.shape[0]:
            raise ValueError("cache_put: doc_len must be one length per document")
        if doc_len.size and (doc_len.min() < 0 or doc_len.max() > MAX_DOC_TOKENS):
            raise ValueError(f"cache_put: document lengths must lie in [0, {MAX_DOC_TOKENS}]")
        doc_len = doc_len.astype(np.int32)
        keys, enc, tokens = list(keys), np.asarray(enc), np.concatenate([[0], np.cumsum(doc_len, dtype=np.int64)])
        if enc.shape[0] < tokens[-1]:
            raise ValueError(f"cache_put: enc holds {enc.shape[0]} rows, doc_len sums to {tokens[-1]}")
        rows = ((doc_len.astype(np.int64) + self.chunk - 1) // self.chunk).tolist()
        cache.check_put(keys, rows)
        most, lo = CACHE_PUT_BYTES // (2 * cache.width), 0
        try:
            while lo < len(keys):
                hi, total = lo + 1, rows[lo]
                while hi < len(keys) and total + rows[hi] <= most:
                    total += rows[hi]
                    hi += 1
                cache.put(keys[lo:hi], rows[lo:hi], self._document_rows(cache, enc[tokens[lo]:tokens[hi]], doc_len[lo:hi], total))
                lo = hi
        except BaseException:
            cache.drop(keys[:lo])
            raise

    def _document_rows(self, cache: DocumentCache, enc: np.ndarray, doc_len: np.ndarray, total: int) -> torch.Tensor:
        """What cache_put stores of some documents, in bf16: their ``total`` pooled vectors' cross K/V."""
        dev = cache.device
        kv = torch.empty(total, cache.width, dtype=torch.bfloat16, device=dev)
        if total:
            lens = torch.from_numpy(doc_len).to(dev)
            tok_off, pool_off = (torch.empty(len(doc_len) + 1, dtype=torch.int64, device=dev) for _ in range(2))
            pooled = torch.empty(total, self.H, dtype=torch.bfloat16, device=dev)
            kalm_ragged_offsets(lens, tok_off, pool_off, self.chunk)
            kalm_chunk_pool(bf16_from_bits(enc, dev), tok_off, lens, pooled, pool_off, total, self.chunk)
            kalm_cross_kv_proj(pooled, self.w.w_kv_cross, kv, self.n_kv, self.D)
        return kv

    def score_rows_cached(self, x0: np.ndarray, cache: DocumentCache, keys) -> np.ndarray:
        """Rows (yes, no, margin, score) of cached documents for one query (``[len(keys)][4]`` float32 on
        the host), in the order of ``keys``; x0: bf16 bits [lq][H].  It has buffers of its own: what this scorer
        prepared, captured or cached for its own documents stays as it is."""
        self._check_cache(cache)
        lq = int(np.asarray(x0).shape[0])
        if not 1 <= lq <= MAX_QUERY_TOKENS:
            raise ValueError(f"rerank_cached: the query input must have 1..{MAX_QUERY_TOKENS} rows (got {lq})")
        if len(keys) == 0:
            return np.zeros((0, 4), dtype=np.float32)
        view = cache.view(keys)
        own = self._exchange(self._cached_set)
        try:
            self.prepare(len(keys), 0, 0, lq)
            self.x0.copy_(bf16_from_bits(np.asarray(x0), cache.device))
            items = kalm_attention_items(len(keys), lq, self.n_q, self.n_kv)
            self.view_order = torch.empty(items, dtype=torch.int32, device=cache.device)
            kalm_attention_schedule(self.q_off, view.row_off, lq, self.n_q, self.n_kv, self.view_order)
            # one layer's cross K/V of these documents, widened; every layer uses the same scratch
            self.view_ws = torch.empty(kalm_merged_attention_cache_rows(view.total_rows, len(keys)),
                                       2 * self.n_kv * self.D, dtype=torch.bfloat16, device=cache.device)
            self.view_cache, self.view = cache, view
            self.launches = 0
            self.decode()
            res = self.scores_to_host().numpy()
            self.check_errors()
        finally:
            self.view = self.view_cache = self.view_ws = self.view_order = None
            self._cached_set = self._exchange(own)
        return np.ascontiguousarray(res.T)

    def rerank_cached(self, x0: np.ndarray, cache: DocumentCache, keys, top_n: Optional[int] = None):
        """``rerank`` over documents of a cache: [{index, relevance_score}] best first, index into ``keys``."""
        res = self.score_rows_cached(x0, cache, keys)
        return rank(res[:, 2], res[:, 3], top_n)

    def _check_cache(self, cache: DocumentCache) -> None:
        if cache.layout != self._cache_layout():
            raise ValueError(f"the cache's rows are {cache.layout}, this stack's {self._cache_layout()}: use new_cache()")

    def check_errors(self) -> None:
        """Wait for this scorer's streams and raise ``KalmError`` if a kernel recorded a
        device error (a bounded wait that expired, or invalid device data) since the
        last check.  ``score_stream`` and ``score_cached_stream`` return without waiting;
        call this once their results are needed."""
        if self.side is not None:
            torch.cuda.current_stream().wait_stream(self.side)
        if getattr(self, "_copy_stream", None) is not None:
            torch.cuda.current_stream().wait_stream(self._copy_stream)
        kalm_check_device_errors()


def rank(margin: np.ndarray, score: np.ndarray, top_n: Optional[int] = None):
    """Best-first order: larger margin first, ties broken by the lower index."""
    order = sorted(range(len(margin)), key=lambda i: (-float(margin[i]), i))
    if top_n is not None:
        order = order[:top_n]
    return [{"index": i, "relevance_score": float(score[i])} for i in order]
