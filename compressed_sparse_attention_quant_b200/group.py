"""Host-side bookkeeping of a group of CSA2 layers: static modes, KV owners
and index aliases. Page "DeepSeek V4 1-Flash 架构拆解…" (blog.zulogic.cn),
section 3: a Full layer is the physical cache owner of the compressed global
KV, the indexer K / scale and the top-K metadata; Reindex and Reuse layers
consume them. Page "DeepSeek 首次公开 V4.1-Flash 技术报告…" (neodrop.ai),
architecture part 2: main KV and indexer keys are shared and top-K indices are
reused across layers.

No device work happens here beyond calling the library: a Reuse layer's index
tensor IS its source layer's tensor (same storage, no copy), and every layer
of an owner reads that owner's PagedCache.

With pool_size set (the hierarchical sparse indexer, neodrop.ai architecture
part 2), a Full layer keeps its top-pool_size positions as a candidate pool
and takes its own top-k inside it. A Reindex layer then scores only its KV
owner's pool instead of the whole context.

Three things a serving step needs beside the sparse attention are options of
step(): latents and indexer keys that come unrotated from their projection
(raw_append), attention queries that do (positions), and entries that many
requests share, a common prompt for instance, which every token of a group
attends to in full (shared). Indexer queries come rotated and quantised
(lib.rope_rows, lib.quant_indexer_fp8), their sigma multiplied into w.
"""
from __future__ import annotations

import math
from typing import Dict, List, Optional, Sequence

import torch

from . import lib

DEFAULT_SCALE = 1.0 / math.sqrt(lib.DIM)


class SharedContext:
    """Entries that groups of consecutive query tokens share: group g's are the first lens[g] of the pages
    page_table[g], and tokens[g] counts its query tokens (b * q_tokens + s, in order). Every token is in a group; one
    without shared entries is in a group of length 0. The tensors may be refreshed in place between replays, the
    counts are fixed. Groups without tokens only count towards the choice of the few-token form (csa2.h): leave them out."""

    def __init__(self, page_table: torch.Tensor, lens: torch.Tensor, tokens: Sequence[int]):
        if page_table.dim() != 2 or len(tokens) != page_table.shape[0] or tuple(lens.shape) != (len(tokens),):
            raise ValueError(f"shared context: {len(tokens)} token counts, lens {tuple(lens.shape)}, page_table "
                             f"{tuple(page_table.shape)}: expected one of each per group")
        if any(int(t) < 0 for t in tokens):
            raise ValueError("shared context: a token count is negative")
        self.page_table, self.lens = page_table, lens
        self.tokens = sum(int(t) for t in tokens)
        offsets = [0]
        for t in tokens:
            offsets.append(offsets[-1] + int(t))
        self.q_offsets = torch.tensor(offsets, dtype=torch.int32, device=page_table.device)


class LayerGroup:
    def __init__(self, modes: Sequence[str], batch: int, q_tokens: int, max_pages: int,
                 num_pages: int, top_k: int, device="cuda", softmax_scale: float = DEFAULT_SCALE,
                 pool_size: Optional[int] = None, rope: Optional[lib.Rope] = None,
                 idx_rope: Optional[lib.Rope] = None):
        """rope rotates the latents (raw_append) and the queries, idx_rope the raw indexer keys."""
        self.modes = tuple(modes)
        self.kv_owner, self.index_src = lib.plan(self.modes)
        self.B, self.Sq, self.k = batch, q_tokens, top_k
        self.max_pages, self.num_pages = max_pages, num_pages
        self.scale = softmax_scale
        self.device = device
        self.caches: Dict[int, lib.PagedCache] = {o: lib.PagedCache(num_pages, device)
                                                  for o in sorted(set(self.kv_owner))}
        self._index: Dict[int, torch.Tensor] = {
            i: torch.full((batch, q_tokens, top_k), -1, dtype=torch.int32, device=device)
            for i, m in enumerate(self.modes) if m in ("F", "R")}
        n = len(self.modes)
        self.out = [torch.empty(batch, q_tokens, lib.HEADS, lib.DIM, dtype=torch.float32, device=device)
                    for _ in range(n)]
        self.lse = [torch.empty(batch, q_tokens, lib.HEADS, dtype=torch.float32, device=device)
                    for _ in range(n)]
        self.pool_size = pool_size
        if pool_size is not None and pool_size < top_k:
            raise ValueError(f"pool_size {pool_size} must be at least top_k {top_k}")
        self._pool: Dict[int, torch.Tensor] = {} if pool_size is None else {
            i: torch.full((batch, q_tokens, pool_size), -1, dtype=torch.int32, device=device)
            for i, m in enumerate(self.modes) if m == "F"}
        self.ws_idx = lib.workspace(lib.indexer_topk_workspace_bytes(batch, q_tokens, max_pages, top_k), device)
        self.ws_att = lib.workspace(lib.sparse_attn_workspace_bytes(batch, q_tokens, top_k), device)
        self.rope, self.idx_rope = rope, idx_rope
        self._q_rot: Optional[torch.Tensor] = None         # rotated queries of the layer at hand
        self.joined: List[torch.Tensor] = []               # with a shared context: bf16 outputs and their lse
        self.joined_lse: List[torch.Tensor] = []
        self._ws_grp: Optional[torch.Tensor] = None        # one for any number of groups: their calls follow one another

    def index(self, layer: int) -> torch.Tensor:
        """The top-k index tensor layer `layer` attends with (an alias for Reuse)."""
        return self._index[self.index_src[layer]]

    def cache(self, layer: int) -> lib.PagedCache:
        return self.caches[self.kv_owner[layer]]

    def pool(self, layer: int) -> torch.Tensor:
        """The candidate pool a layer's selection reads (its KV owner's), when pool_size is set."""
        return self._pool[self.kv_owner[layer]]

    def step(self, page_table: torch.Tensor, seq_lens: torch.Tensor, q: List[torch.Tensor],
             swa: List[torch.Tensor], q_idx: Dict[int, torch.Tensor], w: Dict[int, torch.Tensor],
             append: Optional[Dict[int, tuple]] = None, out: Optional[List[torch.Tensor]] = None,
             lse: Optional[List[torch.Tensor]] = None, positions: Optional[torch.Tensor] = None,
             raw_append: Optional[Dict[int, tuple]] = None, shared: Optional[SharedContext] = None) -> None:
        """One decode step over every layer of the group, on the current stream.

        q[l], swa[l]: layer l's attention query and window rows.
        q_idx[l], w[l]: indexer query and head weights of Full / Reindex layers.
        append[l] = (x_new [n,576] bf16, slots [n] int32, kidx_new [n,64] u8,
                     ksig_new [n] f32): the new tokens a Full layer writes into
                     its cache before it indexes (None: cache already holds them).
        out[l], lse[l]: where layer l writes its output (default self.out, self.lse).
        positions [batch * q_tokens] int32: q holds unrotated rows of these positions.
        raw_append[l] = (x [n,576] bf16, positions [n] int32, slots [n] int32, kidx [n,64] bf16 or None): as append,
                     from unrotated latents and keys.
        shared: entries of the layer's cache that the tokens attend to in full, beside their own selection; the
                softmax over both is in self.joined[l] (bf16) and self.joined_lse[l], and out, lse hold the own part.
        """
        if (positions is not None or raw_append) and self.rope is None:
            raise ValueError("positions and raw_append: the group was built without a rope")
        if shared is not None:
            self._prepare_shared(shared)
        out = self.out if out is None else out
        lse = self.lse if lse is None else lse
        for li, mode in enumerate(self.modes):
            cache = self.cache(li)
            if mode == "F" and append is not None and li in append:
                x_new, slots, kidx_new, ksig_new = append[li]
                lib.quant_kv_fp4(x_new, slots, cache, kidx_new, ksig_new)
            if mode == "F" and raw_append is not None and li in raw_append:
                x_raw, x_pos, slots, kidx_raw = raw_append[li]
                lib.append_kv_rope(x_raw, x_pos, slots, cache, self.rope, kidx_raw,
                                   None if kidx_raw is None else self.idx_rope)
            if mode in ("F", "R") and self.pool_size is not None:
                if mode == "F":
                    lib.indexer_topk(q_idx[li], w[li], cache, page_table, seq_lens, self.pool_size,
                                     out=self._pool[li], ws=self.ws_idx)
                lib.indexer_pool_topk(q_idx[li], w[li], cache, page_table, seq_lens, self.pool(li), self.k,
                                      out=self._index[li])
            elif mode in ("F", "R"):
                lib.indexer_topk(q_idx[li], w[li], cache, page_table, seq_lens, self.k,
                                 out=self._index[li], ws=self.ws_idx)
            ql = q[li] if positions is None else self._rotated(q[li], positions)
            lib.sparse_attn_decode(ql, cache, page_table, seq_lens, self.index(li), swa[li], self.scale,
                                   out=out[li], lse=lse[li], ws=self.ws_att)
            if shared is not None:
                n = self.B * self.Sq
                lib.group_attn(ql.view(n, lib.HEADS, lib.DIM), cache, shared.page_table, shared.lens, shared.q_offsets,
                               self.scale, o_own=out[li].view(n, lib.HEADS, lib.DIM), lse_own=lse[li].view(n, lib.HEADS),
                               out=self.joined[li].view(n, lib.HEADS, lib.DIM),
                               lse=self.joined_lse[li].view(n, lib.HEADS), ws=self._ws_grp)

    def _rotated(self, q: torch.Tensor, positions: torch.Tensor) -> torch.Tensor:
        if self._q_rot is None:
            self._q_rot = torch.empty(self.B, self.Sq, lib.HEADS, lib.DIM, dtype=torch.bfloat16, device=self.device)
        n = self.B * self.Sq
        lib.rope_rows(q.reshape(n, lib.HEADS, lib.DIM), positions, self.rope, out=self._q_rot.view(n, lib.HEADS, lib.DIM))
        return self._q_rot

    def _prepare_shared(self, shared: SharedContext) -> None:
        n, groups = self.B * self.Sq, shared.lens.shape[0]
        if shared.tokens != n:
            raise ValueError(f"shared context: its groups count {shared.tokens} query tokens, the step has {n}")
        if not self.joined:
            for _ in self.modes:
                self.joined.append(torch.empty(self.B, self.Sq, lib.HEADS, lib.DIM, dtype=torch.bfloat16,
                                               device=self.device))
                self.joined_lse.append(torch.empty(self.B, self.Sq, lib.HEADS, dtype=torch.float32,
                                                   device=self.device))
        need = lib.group_attn_workspace_bytes(n, groups)   # the same for every number of groups
        if self._ws_grp is None or self._ws_grp.numel() < need:
            self._ws_grp = lib.workspace(need, self.device)


class StepGraph:
    """One decode step of a LayerGroup captured once as a CUDA graph and then
    replayed with a single launch: the same library kernels in the same order,
    the programmatic-dependent-launch overlap between consecutive kernels kept
    as graph edges, and no host work per kernel. The graph reads and writes the
    tensors given at capture time, so a caller refreshes those in place between
    replays (new query rows, new tokens to append, new page-table entries).

    The first eager step runs before the capture so that the library's one-time
    device set-up does not happen while the stream is being captured.
    """

    def __init__(self, group: LayerGroup, *step_args, **step_kwargs):
        group.step(*step_args, **step_kwargs)
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        n0 = lib.launch_count()
        # thread-local capture: other threads (a process group's watchdog) may
        # keep querying the device while this one captures
        with torch.cuda.graph(self.graph, capture_error_mode="thread_local"):
            group.step(*step_args, **step_kwargs)
        self.launches = lib.launch_count() - n0          # library kernels per replay

    def replay(self) -> None:
        """Enqueue the captured step on the current stream."""
        self.graph.replay()
