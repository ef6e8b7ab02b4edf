"""A layer's step over a paged latent cache on one GPU.

Every request brings a chunk of new tokens (one for a decoding request).  The
step norms the hidden states to E4M3, projects queries and latents with FP4
weights, plans pages and rows on the device, appends the latents (RoPE and
FP4, or E4M3) and attends causally over everything the requests hold.

This module only allocates device memory (torch) and issues C-ABI calls in
that order; all arithmetic runs in libcsa2.so.  A step issues the same calls
with the same pointers every time, so it can be captured in a CUDA graph: the
lengths stay on the device, and the host's bounds max_q and max_kv size the
launches.

Positions: FP4 latents are rotated by RoPE as they are appended (channel pairs
(2i, 2i+1) by pos * theta^(-2i/512)), unless the cache is made with rope_theta
None; E4M3 latents are stored as they are.  Over a cache that rotates, attend()
takes queries that are rotated by their positions (cache.pos): append_heads()
norms and rotates queries and latents alike and stores the latents, and a layer
that is made with norms of its heads, or with turn, steps that way; step() also
takes a function that rotates them.  The logits then depend on distances alone.
Without it they depend on where the keys lie.  Keys are also the values, so
outputs are sums of latents as they are stored.

Trees: a step whose new tokens are drafted, each behind a parent of its own,
plans pages, then tree(), appends, attends with attend_tree() and ends with
commit() in the place of advance(): what the model's choices accept stays, its
rows move together, and pages behind it go back.  TokenLogprobs gives choices
and log probabilities from logits.

A captured step keeps its workspace when a later one needs a larger;
the first step with larger bounds runs outside a capture.

Calls go to the given stream, or the current one; the device has to be the
current device.
"""
from __future__ import annotations

import ctypes
import math
import warnings

import torch

from . import abi

LATENT = abi.LATENT_DIM


def _stream(dev, stream):
    if dev.index != torch.cuda.current_device():
        raise ValueError(f"the current device is not {dev}")
    if isinstance(stream, int):  # a cudaStream_t, as the C calls take it
        return torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
    return torch.cuda.current_stream(dev) if stream is None else stream


def _made(dev):
    """What the current stream has filled is there for calls on any other one."""
    if dev.type == "cuda":
        torch.cuda.current_stream(dev).synchronize()


def _rows(name, x, n, shape, dev, dtype=torch.bfloat16):
    """x has at least n contiguous rows of this shape on the device."""
    if x.device != dev:
        raise ValueError(f"{name}: on {x.device}, not on {dev}")
    if x.dtype != dtype or tuple(x.shape[1:]) != tuple(shape) or x.shape[0] < n or not x.is_contiguous():
        raise ValueError(f"{name}: contiguous {dtype} rows of {tuple(shape)}, at least {n} of them, not {x.dtype} {tuple(x.shape)}")


def _at16(name, x):
    """x begins on a 16-byte boundary, which a view into other data may not."""
    if x.data_ptr() % 16:
        raise ValueError(f"{name}: not 16-byte aligned")


def fp4_weight(w):
    """FP4 form (codes [n][k/2], scales [n][k/16]) of bf16 weights w [n][k], k a multiple of 128, on the current stream."""
    n, k = w.shape
    if w.dtype != torch.bfloat16:
        raise ValueError("an FP4 weight is made of bf16 weights")
    if k % 128:
        raise ValueError("the channels of an FP4 weight come in multiples of 128")
    s = _stream(w.device, None)
    codes = torch.empty((n, k // 2), dtype=torch.uint8, device=w.device)
    scales = torch.empty((n, k // 16), dtype=torch.uint8, device=w.device)
    ws = torch.zeros(abi.STATUS_BYTES, dtype=torch.uint8, device=w.device)
    rows = n * k // 128
    abi.csa2_quantize_append(w.contiguous(), rows, 128, abi.FMT_FP4, abi.LAYOUT_ROWS, None, None, 0, None, rows, codes, scales,
                             ws, ws.numel(), s)
    return codes, scales


class PagedLatents:
    """Pages, block tables and latents of a batch of requests, and the calls over them.  rope_theta None: FP4 latents are
    stored without rotation, as E4M3 ones always are."""

    def __init__(self, n_req, max_tokens, n_pages, page_size, max_pages, heads=abi.ATTN_HEADS, fmt=abi.FMT_FP4, window=0,
                 sm_scale=1.0 / math.sqrt(float(LATENT)), rope_theta=10000.0, device="cuda"):
        d = torch.device(device)
        if d.type == "cuda" and d.index is None:
            d = torch.device("cuda", torch.cuda.current_device())
        if n_req < 1 or max_tokens < 1 or n_pages < 1 or max_pages < 1:
            raise ValueError("a cache has a request, a token of a step, a page and a place for it")
        if page_size < 8 or page_size > 65536 or page_size % 8 or not 1 <= heads <= 128:
            raise ValueError(f"pages of {page_size} entries or {heads} heads: multiples of 8 up to 65536, and up to 128 heads")
        if fmt not in (abi.FMT_FP4, abi.FMT_FP8) or window < 0 or \
                not 0.0 < ctypes.c_float(sm_scale).value < torch.finfo(torch.float32).max:
            raise ValueError(f"format {fmt}, window {window}, scale {sm_scale}")
        self.dev = d
        self.n_req, self.max_tokens, self.heads = n_req, max_tokens, heads
        self.n_pages, self.page_size, self.max_pages = n_pages, page_size, max_pages
        self.fmt, self.window, self.sm_scale = fmt, window, sm_scale
        self.n_rows = n_pages * page_size
        u8, i32, i64 = torch.uint8, torch.int32, torch.int64
        fp4 = fmt == abi.FMT_FP4
        self.codes = torch.zeros((self.n_rows, LATENT // 2 if fp4 else LATENT), dtype=u8, device=d)
        self.scales = torch.zeros((self.n_rows, LATENT // 16), dtype=u8, device=d) if fp4 else None
        self.table = torch.full((n_req, max_pages), -1, dtype=i32, device=d)
        self.free = torch.arange(n_pages - 1, -1, -1, dtype=i32, device=d)  # taken from the end: page 0 first
        self.n_free = torch.full((1,), n_pages, dtype=i32, device=d)
        self.cached = torch.zeros(n_req, dtype=i32, device=d)   # entries held before the step
        self.added = torch.zeros(n_req, dtype=i32, device=d)    # new tokens of the step
        self.kv_len = torch.zeros(n_req, dtype=i32, device=d)
        self.q_start = torch.zeros(n_req + 1, dtype=i32, device=d)
        self.slots = torch.zeros(max_tokens, dtype=i64, device=d)
        self.pos = torch.zeros(max_tokens, dtype=i64, device=d)
        self.max_pos = max_pages * page_size
        self.rope = None
        if fp4 and rope_theta is not None:
            self.rope = torch.empty(abi.csa2_rope_table_bytes(LATENT, self.max_pos), dtype=u8, device=d)
            abi.csa2_rope_table_init(rope_theta, LATENT, self.max_pos, self.rope, _stream(d, None))
        self.out = torch.zeros((max_tokens, heads, LATENT), dtype=torch.bfloat16, device=d)
        self.lse = torch.zeros((max_tokens, heads), dtype=torch.float32, device=d)
        self.ws_plan = torch.zeros(abi.STATUS_BYTES, dtype=u8, device=d)
        self.ws_app = torch.zeros(abi.STATUS_BYTES, dtype=u8, device=d)
        # trees: ancestor masks [n_tokens][words of the step], the accepted path
        self.mask = torch.zeros(max_tokens * ((min(max_tokens, abi.TREE_NODES) + 31) // 32), dtype=i32, device=d)
        self.path = torch.full((max_tokens,), -1, dtype=i32, device=d)
        self.accepted = torch.zeros(n_req, dtype=i32, device=d)
        self.next = torch.full((n_req,), -1, dtype=i64, device=d)
        self.ws_tree = torch.zeros(abi.STATUS_BYTES, dtype=u8, device=d)
        self._words = None  # of a mask's row, as tree() laid it out
        self.ws_attn = None
        self._captured, self._kept = False, []  # the workspace is in a graph; earlier ones that are
        _made(d)

    def _tokens(self, n):
        if not 0 <= n <= self.max_tokens:
            raise ValueError(f"{n} tokens: the cache's buffers are for up to {self.max_tokens}")

    def plan(self, stream=None):
        """Pages, rows and positions of the step's new tokens (self.cached, self.added)."""
        s = _stream(self.dev, stream)
        abi.csa2_page_plan(self.cached, self.added, self.n_req, self.page_size, self.table, self.max_pages, self.free,
                           self.n_pages, self.n_free, self.n_free, self.q_start, self.kv_len, self.slots, self.pos,
                           self.max_tokens, self.ws_plan, self.ws_plan.numel(), s)

    def append(self, latents, n_tokens, stream=None):
        """The new tokens' bf16 latents [n_tokens][512] into the planned rows.  Rows behind the planned tokens (a padded
        batch) are stored nowhere; the first of them is in the append's status."""
        self._tokens(n_tokens)
        _rows("latents", latents, n_tokens, (LATENT,), self.dev)
        s = _stream(self.dev, stream)
        if n_tokens == 0:
            return
        turn = self.rope is not None
        abi.csa2_quantize_append(latents, n_tokens, LATENT, self.fmt, abi.LAYOUT_ROWS, self.pos if turn else None, self.rope,
                                 self.max_pos if turn else 0, self.slots, self.n_rows, self.codes, self.scales, self.ws_app,
                                 self.ws_app.numel(), s)

    def append_heads(self, q, latents, n_tokens, q_norm=None, latent_norm=None, eps=1e-6, stream=None):
        """append() and the queries q [n_tokens][heads][512] in one pass: both normed over the 512 channels of a head by
        q_norm, latent_norm (bf16 [512]; None: not normed), both turned by self.pos where the cache rotates; q in place.
        Tokens behind the planned ones are left as they are."""
        self._tokens(n_tokens)
        _rows("q", q, n_tokens, (self.heads, LATENT), self.dev)
        _rows("latents", latents, n_tokens, (LATENT,), self.dev)
        for name, w in (("q_norm", q_norm), ("latent_norm", latent_norm)):
            if w is not None:
                _rows(name, w, LATENT, (), self.dev)
        if not 0.0 <= ctypes.c_float(eps).value < math.inf:
            raise ValueError(f"eps {eps}")
        s = _stream(self.dev, stream)
        if n_tokens == 0:
            return
        abi.csa2_head_norm_rope(q, self.heads * LATENT, self.heads, q_norm, q, latents, LATENT, latent_norm, n_tokens, eps, self.pos,
                                self.rope, self.max_pos if self.rope is not None else 0, self.fmt, self.slots, self.n_rows, self.codes,
                                self.scales, self.ws_app, self.ws_app.numel(), s)

    def workspace(self, n_tokens, max_q, max_kv, stream=None, tree=False):
        """The attention's workspace for these bounds (kept, and grown where a later step needs more; not while `stream`,
        or the current one, is being captured)."""
        size = abi.csa2_tree_attn_workspace_bytes if tree else abi.csa2_paged_attn_workspace_bytes
        need = size(n_tokens, self.heads, self.n_req, max_q, max_kv, self.window)
        if need == 0:
            raise ValueError("the attention does not run calls of these sizes")
        with torch.cuda.stream(_stream(self.dev, stream)):
            capturing = torch.cuda.is_current_stream_capturing()
        if self.ws_attn is None or self.ws_attn.numel() < need:
            if capturing:
                raise RuntimeError("a step with these bounds has to run once before it is captured: its workspace grows")
            torch.cuda.synchronize(self.dev)  # whatever stream still uses the old one
            old, self.ws_attn = self.ws_attn, torch.zeros(need, dtype=torch.uint8, device=self.dev)
            if self._captured:
                self._kept.append(old)
                self._captured = False
            elif old is not None:
                self.ws_attn[:16].copy_(old[:16])  # a problem on record stays on record
            torch.cuda.synchronize(self.dev)
        self._captured = self._captured or capturing
        return self.ws_attn

    def attend(self, q, n_tokens, max_q, max_kv, stream=None):
        """out, lse of the new tokens' queries q [n_tokens][heads][512] over all entries."""
        self._tokens(n_tokens)
        _rows("q", q, n_tokens, (self.heads, LATENT), self.dev)
        s = _stream(self.dev, stream)
        ws = self.workspace(n_tokens, max_q, max_kv, s)
        if n_tokens == 0:
            return self.out[:0], self.lse[:0]
        abi.csa2_paged_attn(q, n_tokens, self.heads, self.q_start, self.kv_len, self.n_req, max_q, max_kv, self.fmt, self.codes,
                            self.scales, self.n_rows, self.table, self.max_pages, self.page_size, self.window, self.sm_scale,
                            self.out, self.lse, ws, ws.numel(), s)
        return self.out[:n_tokens], self.lse[:n_tokens]

    def _nodes(self, max_q, **per_node):
        """What a tree's calls take is there: a bound that they run, and per token of the step a value."""
        if not 0 <= max_q <= min(abi.TREE_NODES, self.max_tokens):
            raise ValueError(f"{max_q} nodes of a request: up to {abi.TREE_NODES}, and to the {self.max_tokens} tokens of a step")
        for name, (x, n, dtype) in per_node.items():
            _rows(name, x, n, (), self.dev, dtype)
            _at16(name, x)

    def tree(self, parent, n_tokens, max_q, stream=None):
        """Behind plan(): the step's tokens are trees.  parent [n_tokens] int32: the place of a node's parent among its
        request's nodes, which comes before it; -1 continues the cached entries.  self.pos becomes the nodes' positions (by
        their depth), self.mask their ancestors."""
        self._tokens(n_tokens)
        self._nodes(max_q, parent=(parent, n_tokens, torch.int32))
        s = _stream(self.dev, stream)
        self._words = (max_q + 31) // 32
        if n_tokens == 0 or max_q == 0:
            return
        abi.csa2_tree_plan(parent, self.q_start, self.kv_len, self.n_req, n_tokens, max_q, self.window, self.pos, self.mask,
                           (max_q + 31) // 32, self.ws_tree, self.ws_tree.numel(), s)

    def attend_tree(self, q, n_tokens, max_q, max_kv, stream=None):
        """attend() for a step of trees (the same max_q as tree()'s): out, lse of nodes that see the entries before the step
        and their ancestors."""
        self._tokens(n_tokens)
        self._nodes(max_q)
        _rows("q", q, n_tokens, (self.heads, LATENT), self.dev)
        if self._words != (max_q + 31) // 32:
            raise ValueError(f"{max_q} nodes of a request: not the bound that tree() had")
        s = _stream(self.dev, stream)
        ws = self.workspace(n_tokens, max_q, max_kv, s, tree=True)
        if n_tokens == 0:
            return self.out[:0], self.lse[:0]
        abi.csa2_tree_attn(q, n_tokens, self.heads, self.q_start, self.kv_len, self.n_req, max_q, max_kv, self.pos, self.mask,
                           (max_q + 31) // 32, self.fmt, self.codes, self.scales, self.n_rows, self.table, self.max_pages,
                           self.page_size, self.window, self.sm_scale, self.out, self.lse, ws, ws.numel(), s)
        return self.out[:n_tokens], self.lse[:n_tokens]

    def commit(self, parent, token, choice, n_tokens, max_q, stream=None):
        """The end of a step of trees, in the place of advance(): from every request's first node the path goes to the child
        whose token [n_tokens] int64 is its parent's choice [n_tokens] int64, as long as there is one.  Returns (path, accepted,
        next): the path's nodes at each request's first tokens, their number, and the choice behind them.  self.cached, the
        path's rows and the pages follow.  Once a step; a refused step's requests keep their lengths."""
        self._tokens(n_tokens)
        self._nodes(max_q, parent=(parent, n_tokens, torch.int32), token=(token, n_tokens, torch.int64),
                    choice=(choice, n_tokens, torch.int64))
        s = _stream(self.dev, stream)
        abi.csa2_tree_commit(parent, token, choice, self.q_start, self.kv_len, self.n_req, n_tokens, max_q, self.fmt, self.codes,
                             self.scales, self.n_rows, self.table, self.max_pages, self.page_size, self.free, self.n_pages, self.n_free,
                             self.n_free, self.cached, self.path, self.accepted, self.next, self.ws_tree, self.ws_tree.numel(), s)
        return self.path[:n_tokens], self.accepted, self.next

    def advance(self, stream=None):
        """After a step, on its stream: what it added is cached.  A step whose plan was refused added nothing (its kv_len
        are all 0)."""
        with torch.cuda.stream(_stream(self.dev, stream)):
            self.cached.copy_(torch.where(self.kv_len.any(), self.kv_len, self.cached))

    def status(self, stream=None):
        """Status words of every workspace (first device-detected problem), behind what runs on the stream so far."""
        s = _stream(self.dev, stream)
        named = {"plan": abi.csa2_status_fetch(self.ws_plan, s), "append": abi.csa2_status_fetch(self.ws_app, s),
                 "tree": abi.csa2_status_fetch(self.ws_tree, s)}
        attn = [abi.csa2_status_fetch(ws, s) for ws in self._kept + [self.ws_attn] if ws is not None]
        if attn:
            named["attn"] = next((st for st in attn if st[0] != abi.OK), attn[-1])
        return named


class TokenLogprobs:
    """Log probabilities and alternatives of up to max_rows rows of logits: the `top` largest logits of a row and `given`
    tokens of the caller's.  The outputs are the object's own, so that calls can be captured."""

    def __init__(self, max_rows, given=0, top=1, device="cuda"):
        d = torch.device(device)
        if d.type == "cuda" and d.index is None:
            d = torch.device("cuda", torch.cuda.current_device())
        if max_rows < 1 or not 0 <= given <= abi.LOGPROBS_TOP or not 0 <= top <= abi.LOGPROBS_TOP:
            raise ValueError(f"{max_rows} rows, {given} given tokens, {top} alternatives: a row or more, up to {abi.LOGPROBS_TOP} of both")
        self.dev, self.max_rows, self.given, self.top = d, max_rows, given, top
        f32 = torch.float32
        self.logprobs = torch.zeros((max_rows, given), dtype=f32, device=d)
        self.lse, self.entropy = torch.zeros(max_rows, dtype=f32, device=d), torch.zeros(max_rows, dtype=f32, device=d)
        self.ids = torch.zeros((max_rows, top), dtype=torch.int32, device=d)
        self.best = torch.zeros((max_rows, top), dtype=f32, device=d)
        self.ws = torch.zeros(abi.STATUS_BYTES, dtype=torch.uint8, device=d)
        _made(d)

    def __call__(self, logits, tokens=None, scale=1.0, stream=None):
        """logits [n][vocab] bf16 or fp32 (rows may be strided), tokens [n][given] int64 (-1: none), scale one over the
        temperature.  Returns (logprobs [n][given], lse [n], entropy [n], ids [n][top], best [n][top])."""
        if logits.dtype not in (torch.bfloat16, torch.float32) or logits.dim() != 2 or logits.device != self.dev or \
                logits.shape[0] > self.max_rows or logits.shape[1] < 1 or (logits.shape[1] > 1 and logits.stride(1) != 1):
            raise ValueError(f"logits: up to {self.max_rows} rows of bf16 or fp32 on {self.dev}, not {logits.dtype} {tuple(logits.shape)} "
                             f"on {logits.device}")
        n, vocab = logits.shape
        stride = logits.stride(0) if n > 1 else vocab
        if stride < vocab:
            raise ValueError("logits: rows that overlap")
        if (tokens is None) != (self.given == 0):
            raise ValueError(f"{self.given} given tokens of a row")
        if tokens is not None:
            _rows("tokens", tokens, n, (self.given,), self.dev, torch.int64)
        s = _stream(self.dev, stream)
        if n > 0:
            abi.csa2_token_logprobs(logits, abi.OUT_BF16 if logits.dtype == torch.bfloat16 else abi.OUT_F32, stride, n, vocab, scale,
                                    tokens, self.given, self.logprobs if self.given else None, self.lse, self.entropy, self.top,
                                    self.ids if self.top else None, self.best if self.top else None, self.ws, self.ws.numel(), s)
        return self.logprobs[:n], self.lse[:n], self.entropy[:n], self.ids[:n], self.best[:n]

    def status(self, stream=None):
        return abi.csa2_status_fetch(self.ws, _stream(self.dev, stream))


class PagedLayer:
    """The front of an attention layer: norm, FP4 projections and the attention over a PagedLatents cache.  Without a
    rotary embedding where the cache does not rotate; where it does, see step()'s `rotate`.  With q_norm or latent_norm
    (bf16 [512], norms of every head's query and of the latents) or turn, queries and latents go through
    PagedLatents.append_heads: normed by the weights that are given, and both turned where the cache rotates.

    residual [max_tokens][hidden], the layer's residual stream, goes by the step's tokens: step() adds to its first n_tokens
    rows, so before every step they are set to what the tokens bring from the layer before (zeros at the first one).  A
    step that the plan refuses leaves out and lse as they were: status() tells."""

    def __init__(self, cache, hidden, norm_weight, wq, wlatent, eps=1e-6, q_norm=None, latent_norm=None, turn=False):
        """norm_weight bf16 [hidden]; wq, wlatent: bf16 weights [heads * 512][hidden], [512][hidden]."""
        d, T, H = cache.dev, cache.max_tokens, cache.heads
        sizes = [abi.csa2_fp4_matvec_workspace_bytes(T, hidden, n) for n in (H * LATENT, LATENT)]
        if 0 in sizes or hidden > 16384 or not 0.0 <= ctypes.c_float(eps).value < math.inf:
            raise ValueError(f"a layer of {hidden} channels for steps of {T} tokens, eps {eps}: multiples of 128 up to 16384, up to "
                             "65536 tokens")
        for name, w, shape in (("norm_weight", norm_weight, (hidden,)), ("wq", wq, (H * LATENT, hidden)),
                               ("wlatent", wlatent, (LATENT, hidden))):
            if w.dtype != torch.bfloat16 or tuple(w.shape) != shape or w.device != d:
                raise ValueError(f"{name}: bf16 {shape} on {d}, not {w.dtype} {tuple(w.shape)} on {w.device}")
        for name, w in (("q_norm", q_norm), ("latent_norm", latent_norm)):
            if w is not None:
                _rows(name, w, LATENT, (), d)
                _at16(name, w)  # (no step gets as far as its append otherwise)
        self.q_norm, self.latent_norm, self.heads_pass = q_norm, latent_norm, turn or q_norm is not None or latent_norm is not None
        self.cache, self.hidden, self.eps, self.norm_weight = cache, hidden, eps, norm_weight.contiguous()
        self.wq, self.wlatent = fp4_weight(wq), fp4_weight(wlatent)
        self.residual = torch.zeros((T, hidden), dtype=torch.bfloat16, device=d)
        self.x = torch.zeros((T, hidden), dtype=torch.uint8, device=d)  # E4M3
        self.x_scales = torch.zeros(T, dtype=torch.float32, device=d)
        self.q = torch.zeros((T, H, LATENT), dtype=torch.bfloat16, device=d)
        self.latents = torch.zeros((T, LATENT), dtype=torch.bfloat16, device=d)
        self.ws = torch.zeros(max(sizes), dtype=torch.uint8, device=d)
        self._told = False  # of queries that are not rotated
        _made(d)

    def _project(self, w, n, n_out, out, s):
        abi.csa2_fp4_matvec(self.x, abi.X_E4M3, self.x_scales, self.hidden, n, self.hidden, w[0], w[1], n_out, 1.0, out,
                            abi.OUT_BF16, self.ws, self.ws.numel(), s)

    def step(self, hidden, n_tokens, max_q, max_kv, stream=None, rotate=None, parent=None):
        """One step of n_tokens new tokens' bf16 hidden states (added to self.residual, the layer's residual stream):
        (out, lse) of the attention.  n_tokens above the planned ones (a padded batch) leaves the rows behind them of
        out and lse as they are; see PagedLatents.append.

        rotate(q, pos): called once the plan is made, with the step's stream current, to turn the queries
        q [n_tokens][heads][512] in place by their positions pos (-1 behind the planned tokens), as the cache turns the
        latents; it may run inside a capture.  A layer with norms of its heads, or turn, turns them itself.

        parent: the step's tokens are trees (PagedLatents.tree); PagedLatents.commit ends the step then, not advance."""
        c, n = self.cache, n_tokens
        c._tokens(n)
        _rows("hidden", hidden, n, (self.hidden,), c.dev)
        if parent is not None:
            c._nodes(max_q, parent=(parent, n, torch.int32))
        if rotate is not None and self.heads_pass:
            raise ValueError("the layer turns its queries itself")
        s = _stream(c.dev, stream)
        if rotate is None and c.rope is not None and not self.heads_pass and not self._told:
            warnings.warn("the cache rotates its latents and the step's queries are not rotated: logits depend on where the "
                          "keys lie (rotate=, or a cache with rope_theta=None)")
            self._told = True
        c.workspace(n, max_q, max_kv, s, tree=parent is not None)  # what refuses the step refuses it before the residual, pages and lengths change
        if n > 0:
            abi.csa2_rmsnorm_fp8(hidden, self.hidden, self.residual, self.residual, self.norm_weight, n, self.hidden, self.eps, 0,
                                 self.x, self.x_scales, None, s)
            self._project(self.wq, n, c.heads * LATENT, self.q, s)
            self._project(self.wlatent, n, LATENT, self.latents, s)
        c.plan(s)
        if parent is not None:
            c.tree(parent, n, max_q, s)
        if rotate is not None and n > 0:
            with torch.cuda.stream(s):
                rotate(self.q[:n], c.pos[:n])
        if self.heads_pass:
            c.append_heads(self.q, self.latents, n, self.q_norm, self.latent_norm, self.eps, s)
        else:
            c.append(self.latents, n, s)
        return (c.attend if parent is None else c.attend_tree)(self.q, n, max_q, max_kv, s)
