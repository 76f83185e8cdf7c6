"""A request's passes through the C ABI: buffers + the calls in order.

PromptPass owns the outputs and workspace of one batch of prompts (or of their
next chunks) and enqueues spec_kv_append (or spec_rope_append, from a
projection's output) -> spec_prompt_attention.

VerifyPass owns the device outputs and workspaces of one batch shape and
enqueues, on one stream and with no host synchronisation:
  spec_tree_mask_build -> [spec_kv_append or spec_rope_append] ->
  spec_tree_attention -> spec_tree_verify_{greedy, stochastic} ->
  [spec_path_logprobs] -> spec_kv_commit.
Allocation happens once, in the constructor; run() only launches.

CacheBudget holds the attention weight that cached slots gather over those
passes (spec_attention_weight) and cuts rows to a budget by it
(spec_kv_evict).
"""
from dataclasses import dataclass, replace

import torch

from . import _binding as S


@dataclass
class DeviceBatch:
    """Device-resident inputs of one pass (all CUDA tensors)."""
    B: int
    T: int
    n_max: int
    V: int
    Hq: int
    Hkv: int
    D: int
    block_size: int
    num_blocks: int
    max_prefix: int
    parent: torch.Tensor
    tree_off: torch.Tensor
    tokens: torch.Tensor
    prefix_len: torch.Tensor
    block_table: torch.Tensor
    q: torch.Tensor
    k_cache: torch.Tensor
    v_cache: torch.Tensor
    p_logits: torch.Tensor
    q_probs: torch.Tensor
    uniforms: torch.Tensor  # int32 [T, 2] raw words
    scale: float

    @property
    def max_blocks(self):
        return self.block_table.shape[1]

    @classmethod
    def from_workload(cls, w, device="cuda", max_prefix=None):
        def d(t):
            return None if t is None else t.to(device, non_blocking=False).contiguous()
        mp = int(w.prefix_len.max()) if max_prefix is None and w.B > 0 else (max_prefix or 0)
        return cls(B=w.B, T=w.T, n_max=w.n_max, V=w.V, Hq=w.Hq, Hkv=w.Hkv, D=w.D, block_size=w.block_size,
                   num_blocks=w.num_blocks, max_prefix=mp, parent=d(w.parent), tree_off=d(w.tree_off),
                   tokens=d(w.tokens), prefix_len=d(w.prefix_len), block_table=d(w.block_table), q=d(w.q),
                   k_cache=d(w.k_cache), v_cache=d(w.v_cache), p_logits=d(w.p_logits), q_probs=d(w.q_probs),
                   uniforms=d(w.uniforms), scale=w.scale)


@dataclass
class Rotary:
    """How a layer's query and key heads are normalised and rotated on their way
    from the projection (spec_rope_append)."""
    inv_freq: torch.Tensor = None  # float32 [rot_dim / 2], radians per position
    rot_dim: int = 0
    axis: torch.Tensor = None      # int32 [rot_dim / 2], for axes > 1
    axes: int = 1
    pairing: int = S.SPEC_ROPE_HALVES
    q_norm: torch.Tensor = None    # [D] of the caches' dtype, or None
    k_norm: torch.Tensor = None
    eps: float = 1e-6

    def append(self, qkv, q, k_cache, v_cache, block_table, prefix_len, tree_off, n_max, status, pos_base=None, pos=None, stream=None):
        num_blocks, Hkv, block_size, D = k_cache.shape
        T, Hq, _ = q.shape
        T = self._check(qkv, T, (Hq + 2 * Hkv) * D, D, tree_off.numel() - 1, pos_base, pos)
        S.spec_rope_append(qkv, self.q_norm, self.k_norm, self.eps, self.inv_freq, self.axis, self.rot_dim, self.pairing, pos_base, pos, self.axes, q, k_cache,
                           v_cache, block_table, block_table.shape[1], block_size, num_blocks, prefix_len, tree_off, tree_off.numel() - 1, T, n_max, Hq, Hkv, D,
                           status, stream)

    def _check(self, qkv, T, width, D, B, pos_base, pos):
        """Buffers that the call would read past the end of are refused: it knows
        their addresses alone.  Returns the rows that every buffer has: q may be
        longer than the batch, and a request behind them is flagged by the call."""
        def holds(t, n):
            return t is None or t.numel() >= n
        if qkv.dim() > 1 and qkv.shape[1:].numel() < width:
            raise ValueError("qkv has narrower rows than its heads")
        if self.axes == 1:
            T = min(T, qkv.shape[0], T if pos is None else pos.numel())
        elif qkv.shape[0] < T or not holds(pos, self.axes * T) or (pos is not None and pos.dim() > 1 and pos.shape[-1] != T):
            raise ValueError("several axes: qkv and each axis of pos must have q's rows, pos [axes][T]")
        if not holds(pos_base, B):
            raise ValueError("pos_base must hold an entry for each request")
        if not (holds(self.inv_freq, self.rot_dim // 2) and holds(self.axis, self.rot_dim // 2)):
            raise ValueError("inv_freq and axis must hold an entry for each pair")
        if not (holds(self.q_norm, D) and holds(self.k_norm, D)):
            raise ValueError("q_norm and k_norm must hold a weight for each element of a head")
        return T


def _clear(status, stream):
    with torch.cuda.stream(stream):  # None: the current one
        status.zero_()


def _one_source(kv, qkv, rotary):
    if qkv is not None and (kv is not None or rotary is None):
        raise ValueError("a projection's rows (qkv) come with their rotary, and not beside ready K/V rows")


class PromptPass:
    """Causal attention of packed prompts (or chunks) over the paged cache.

    seq_off int32 [B + 1] and prefix_len int32 [B] are device tensors; n_max
    and max_prefix bound the longest request and the longest prefix."""

    def __init__(self, q, k_cache, v_cache, block_table, seq_off, prefix_len, n_max, max_prefix, scale):
        self.q, self.k_cache, self.v_cache, self.block_table = q, k_cache, v_cache, block_table
        self.seq_off, self.prefix_len, self.scale = seq_off, prefix_len, scale
        self.num_blocks, Hkv, self.block_size, D = k_cache.shape
        T, Hq, _ = q.shape
        self.size = (seq_off.numel() - 1, T, n_max, max_prefix, Hq, Hkv, D)
        self.out = torch.empty_like(q)
        self.ws = torch.empty(S.spec_prompt_workspace_size(*self.size), dtype=torch.uint8, device=q.device)
        self.status = torch.zeros(max(self.size[0], 1), dtype=torch.int32, device=q.device)

    def run(self, prompt_kv=None, stream=None, prompt_qkv=None, rotary=None, pos_base=None, pos=None):
        """prompt_kv: (k_new, v_new) rows [T][Hkv][D] put behind the prefix
        first, or None when they are already in the cache.  prompt_qkv with
        rotary instead: a projection's rows, normalised and rotated into q and
        the cache (pos_base int32 [B], None: the prefix; pos int32 [axes][T],
        None: the row's index).  status is this run's: a request that an earlier
        one flagged is computed again."""
        B, T, n_max, max_prefix, Hq, Hkv, D = self.size
        _one_source(prompt_kv, prompt_qkv, rotary)
        _clear(self.status, stream)
        if prompt_qkv is not None:
            rotary.append(prompt_qkv, self.q, self.k_cache, self.v_cache, self.block_table, self.prefix_len, self.seq_off, n_max, self.status, pos_base, pos,
                          stream)
        if prompt_kv is not None:
            S.spec_kv_append(*prompt_kv, self.k_cache, self.v_cache, self.block_table, self.block_table.shape[1],
                             self.block_size, self.num_blocks, self.prefix_len, self.seq_off, B, n_max, Hkv, D,
                             self.status, stream)
        S.spec_prompt_attention(self.q, self.k_cache, self.v_cache, self.block_table, self.block_table.shape[1],
                                self.block_size, self.num_blocks, self.prefix_len, self.seq_off, *self.size,
                                self.scale, self.out, self.ws, self.status, stream)


class VerifyPass:
    # stochastic verification options used when verify() is not given them:
    # per-request inverse temperatures (float32 device tensor [B], or None for
    # 1) and the draft-row layout
    inv_temp = None
    q_layout = S.SPEC_Q_PER_PARENT

    def __init__(self, batch: DeviceBatch, logprob_top=None):
        """logprob_top: number of alternatives (0 to 32) that logprobs() gives
        for every emitted token; None: no buffers for them."""
        b = batch
        dev = b.q.device
        i32 = dict(dtype=torch.int32, device=dev)
        self.W = (b.n_max + 63) // 64
        self.mask = torch.zeros((max(b.T, 1), self.W), dtype=torch.int64, device=dev)
        self.depth = torch.zeros(max(b.T, 1), **i32)
        self.status = torch.zeros(max(b.B, 1), **i32)
        self.out = torch.empty_like(b.q)
        aws = S.spec_attention_workspace_size(b.B, b.T, b.n_max, b.max_prefix, b.Hq, b.Hkv, b.D)
        self.attn_ws = torch.empty(aws, dtype=torch.uint8, device=dev)
        vws = S.spec_verify_workspace_size(b.B, b.n_max, b.V)
        self.verify_ws = torch.empty(vws, dtype=torch.uint8, device=dev)
        self.path = torch.full((max(b.B, 1), b.n_max), -1, **i32)
        self.accept_len = torch.zeros(max(b.B, 1), **i32)
        self.emitted = torch.full((max(b.B, 1), b.n_max), -1, **i32)
        self.n_emitted = torch.zeros(max(b.B, 1), **i32)
        self.new_len = torch.zeros(max(b.B, 1), **i32)
        self.logprob_top = logprob_top
        if logprob_top is not None:
            shape, f32 = (max(b.B, 1), b.n_max), dict(dtype=torch.float32, device=dev)
            self.logprob, self.entropy = torch.empty(shape, **f32), torch.empty(shape, **f32)
            self.rank = torch.empty(shape, **i32)
            self.top_tokens = torch.empty(shape + (logprob_top,), **i32)
            self.top_logprobs = torch.empty(shape + (logprob_top,), **f32)
            # a word of its own: commit() leaves a request whose status is not 0 as it was
            self.logprob_status = torch.zeros(max(b.B, 1), **i32)
        self.batch = b

    def mask_build(self, stream=None):
        b = self.batch
        S.spec_tree_mask_build(b.parent, b.tree_off, b.B, b.n_max, self.mask, self.depth, self.status, stream)

    def append(self, k_new, v_new, stream=None):
        """Tree K/V rows [T][Hkv][D] into slots prefix_len + u (before attention)."""
        b = self.batch
        S.spec_kv_append(k_new, v_new, b.k_cache, b.v_cache, b.block_table, b.max_blocks, b.block_size,
                         b.num_blocks, b.prefix_len, b.tree_off, b.B, b.n_max, b.Hkv, b.D, self.status, stream)

    def project(self, qkv, rotary, pos_base=None, stream=None):
        """A projection's rows of the tree, normalised and rotated into the
        batch's q and slots prefix_len + u (before attention, after the mask
        build): node u's position is pos_base[b] (None: the prefix) plus its depth,
        on every axis that the rotary has (nodes are text)."""
        b = self.batch
        # one axis stands for all: depth holds no more
        rotary = replace(rotary, axis=None, axes=1)
        rotary.append(qkv, b.q, b.k_cache, b.v_cache, b.block_table, b.prefix_len, b.tree_off, b.n_max, self.status, pos_base, self.depth, stream)

    def attention(self, flags=S.SPEC_ATTN_AUTO, stream=None):
        b = self.batch
        S.spec_tree_attention(b.q, b.k_cache, b.v_cache, b.block_table, b.max_blocks, b.block_size, b.num_blocks,
                              b.prefix_len, b.tree_off, self.mask, b.B, b.T, b.n_max, b.max_prefix, b.Hq, b.Hkv, b.D,
                              b.scale, self.out, self.attn_ws, self.status, flags, stream)

    def verify(self, mode="stochastic", stream=None, inv_temp=None, q_layout=None):
        b = self.batch
        inv_temp = self.inv_temp if inv_temp is None else inv_temp
        q_layout = self.q_layout if q_layout is None else q_layout
        if mode == "greedy":
            S.spec_tree_verify_greedy(b.p_logits, b.tokens, b.parent, b.tree_off, b.B, b.n_max, b.V, self.path, self.accept_len, self.emitted, self.n_emitted,
                                      self.verify_ws, self.status, stream)
        else:
            S.spec_tree_verify_stochastic(b.p_logits, b.q_probs, b.tokens, b.parent, b.tree_off, b.uniforms, b.B,
                                          b.n_max, b.V, self.path, self.accept_len, self.emitted, self.n_emitted,
                                          self.verify_ws, self.status, stream, inv_temp=inv_temp, q_layout=q_layout)

    def logprobs(self, stream=None, inv_temp=None):
        """Log probability, entropy, rank and alternatives of every emitted
        token, [B][n_max] (after verify(); the target distribution is the
        stochastic verifier's, softmax(inv_temp * logits), after a greedy walk
        too).  Flags go to logprob_status, cleared first: what this call
        refuses (a temperature of 0, say, which a greedy walk ignores) does
        not stop the commit."""
        if self.logprob_top is None:
            raise ValueError("VerifyPass was made without logprob_top")
        b = self.batch
        _clear(self.logprob_status, stream)
        S.spec_path_logprobs(b.p_logits, b.tree_off, self.path, self.accept_len, self.emitted,
                             self.inv_temp if inv_temp is None else inv_temp, b.B, b.T, b.n_max, b.V,
                             self.logprob_top, self.logprob, self.entropy, self.rank, self.top_tokens,
                             self.top_logprobs, self.logprob_status, stream)

    def commit(self, stream=None):
        b = self.batch
        S.spec_kv_commit(b.k_cache, b.v_cache, b.block_table, b.max_blocks, b.block_size, b.num_blocks,
                         b.prefix_len, self.path, b.n_max, self.accept_len, b.B, b.Hkv, b.D, self.new_len,
                         self.status, stream)

    def run(self, mode="stochastic", attn_flags=S.SPEC_ATTN_AUTO, commit=True, stream=None, tree_kv=None, tree_qkv=None, rotary=None, pos_base=None):
        """tree_kv: (k_new, v_new) rows appended before attention, or None when
        the tree K/V are already in the cache; tree_qkv with rotary instead: a
        projection's rows (see project())."""
        _one_source(tree_kv, tree_qkv, rotary)
        self.mask_build(stream)
        if tree_qkv is not None:
            self.project(tree_qkv, rotary, pos_base, stream)
        if tree_kv is not None:
            self.append(*tree_kv, stream=stream)
        self.attention(attn_flags, stream)
        self.verify(mode, stream)
        if self.logprob_top is not None:
            self.logprobs(stream)
        if commit:
            self.commit(stream)


class CacheBudget:
    """What the attention of every layer gave each slot of a block table's rows,
    and eviction by it.  weight is float32 [layers][rows][Hkv][slots], by table
    row; a pass over part of the table says at which row its batch starts, and
    rows forked from others take their weights along by fork().  One workspace
    serves every call: observe on one stream at a time, and let another one wait
    for it first."""

    def __init__(self, layers, rows, Hkv, slots, decay=1.0, device="cuda"):
        self.weight = torch.zeros((layers, rows, Hkv, slots), dtype=torch.float32, device=device)
        self.layers, self.rows, self.Hkv, self.slots, self.decay = layers, rows, Hkv, slots, decay
        self._ws = torch.empty(0, dtype=torch.uint8, device=device)
        # calls in flight and captured graphs may still be using them; each is half of
        # the next at most, so together they are no larger than the last
        self._outgrown = []

    def reserve(self, B, T, n_max, max_prefix, Hq, D, stream=None):
        """Workspace for passes of up to these sizes, observed on `stream`
        (observing a larger one first makes it grow, which a captured graph must
        not)."""
        need = S.spec_weight_workspace_size(B, T, n_max, max_prefix, Hq, self.Hkv, D)
        if self._ws.numel() < need:
            self._outgrown.append(self._ws)
            with torch.cuda.stream(stream):  # another stream's free memory may still be in use there
                self._ws = torch.empty(max(need, 2 * self._ws.numel()), dtype=torch.uint8, device=self._ws.device)

    def _observe(self, layer, row, q, k_cache, block_table, prefix_len, off, path, accept_len, window, n_max, max_prefix, scale, status, stream):
        num_blocks, Hkv, block_size, D = k_cache.shape
        T, Hq, _ = q.shape
        B = off.numel() - 1
        if not (0 <= layer < self.layers and 0 <= row and row + B <= self.rows and Hkv == self.Hkv):
            raise ValueError("the pass's layer, rows or heads are not the budget's")
        self.reserve(B, T, n_max, max_prefix, Hq, D, stream)
        w = self.weight[layer, row:row + B]
        S.spec_attention_weight(q, k_cache, block_table, block_table.shape[1], block_size, num_blocks, prefix_len, off, path, accept_len, window, B, T, n_max,
                                max_prefix, Hq, Hkv, D, scale, self.decay, w, w, self.slots, self._ws, status, stream)

    def observe_prompt(self, layer, p, window=0, row=0, stream=None):
        """The rows of a PromptPass (their last `window`), after its run()."""
        _, _, n_max, max_prefix, *_ = p.size
        self._observe(layer, row, p.q, p.k_cache, p.block_table, p.prefix_len, p.seq_off, None, None, window, n_max, max_prefix, p.scale, p.status, stream)

    def observe_path(self, layer, v, window=0, row=0, stream=None):
        """The accepted path of a VerifyPass, after its commit()."""
        b = v.batch
        self._observe(layer, row, b.q, b.k_cache, b.block_table, b.prefix_len, b.tree_off, v.path, v.accept_len, window, b.n_max, b.max_prefix, b.scale, v.status,
                      stream)

    def fork(self, src, dst, status=None, stream=None):
        """Rows dst take the weights of rows src along (int32 [N], after
        spec_pages_fork of them, with its status: a flagged fork changes nothing).
        Empty rows (src -1) and rows out of range are left as they were."""
        if src.numel() == 0:
            return
        with torch.cuda.stream(stream):  # None: the current one
            done = (src >= 0) & (src < self.rows) & (dst >= 0) & (dst < self.rows)
            if status is not None:
                done &= status[:src.numel()] == 0
            # the others write what one that is done writes (or row 0 to itself), so that
            # nothing has to be counted on the host
            one = done.int().argmax().view(1)
            s, d = (torch.where(done, x, x.index_select(0, one)).long() for x in (src.masked_fill(~done, 0), dst.masked_fill(~done, 0)))
            for w in self.weight:
                w.index_copy_(0, d, w.index_select(0, s))

    def evict(self, k_ptrs, v_ptrs, block_table, block_size, num_blocks, src, dst, length, keep_max, first, last, D, dtype, keep=None, stream=None):
        """Rows src (int32 [N], of `length` slots) cut to rows dst, which have
        pages for them; block_table is the whole table, not a pass's rows of it.
        Returns (slots, new_len, status) of spec_kv_evict."""
        N, i32 = src.numel(), dict(dtype=torch.int32, device=src.device)
        if block_table.shape[0] < self.rows:
            raise ValueError("the block table has fewer rows than the budget")
        if dst.numel() < N or length.numel() < N or (keep is not None and keep.numel() < N):
            raise ValueError("dst, length and keep must hold an entry for each of src")
        with torch.cuda.stream(stream):  # None: the current one
            slots = torch.empty((self.layers, N, self.Hkv, keep_max), **i32)
            new_len, status = torch.empty(N, **i32), torch.empty(N, **i32)
        S.spec_kv_evict(k_ptrs, v_ptrs, self.layers, block_table, self.rows, block_table.shape[1], block_size, num_blocks, src, dst, length, keep, N, keep_max,
                        first, last, self.weight, self.slots, self.Hkv, D, dtype, slots, new_len, status, stream)
        return slots, new_len, status
