"""A paged MLA KV cache in torch device memory, driven through libleyline.so.

Plumbing for callers: it allocates the pool tensor (layout
``kv[layer][page][slot][latent + rope]``, bf16; with LEYLINE_POOL_SPLIT_ROPE the
latents ``[layer][page][slot][latent]`` followed by the rope bands
``[layer][page][slot][rope]``), the block table and the length arrays, takes pages
for new requests, and forwards splices and gathers to the C ABI.  It computes
nothing itself.
"""
from __future__ import annotations

import contextlib
import weakref
from typing import Sequence

import numpy as np

from . import leyline


class _DeviceArray:
    """int32 device memory owned by the pool, exposed through __cuda_array_interface__.  A tensor over it keeps it, and
    with it the cache whose end would free the memory."""

    def __init__(self, addr: int, n: int, device: int, owner):
        self.owner = owner
        self.__cuda_array_interface__ = {"shape": (n,), "typestr": "<i4", "data": (addr, False), "version": 3}
        self.device = device


class PagedCache:
    def __init__(self, num_layers: int, block_size: int, num_pages: int, max_reqs: int, max_blocks: int,
                 latent_dim: int = 512, rope_dim: int = 64, rope_theta: float = 10000.0,
                 pair_layout: int = leyline.LEYLINE_PAIRS_HALF_SPLIT,
                 rotate_precision: int = leyline.LEYLINE_ROTATE_FP32, flags: int = 0, rope_heads: int = 1,
                 device: str = "cuda"):
        import torch
        self.torch = torch
        self.num_layers = num_layers
        self.block_size = block_size
        self.num_pages = num_pages
        self.latent_dim = latent_dim
        self.rope_dim = rope_dim
        self.rope_heads = max(rope_heads, 1)
        self.row = latent_dim + self.rope_heads * rope_dim
        self.device = torch.device(device)
        self.kv = torch.empty(num_layers * num_pages * block_size * self.row, dtype=torch.bfloat16,
                              device=self.device)
        self.desc = leyline.pool_desc(num_layers, block_size, num_pages, latent_dim, rope_dim, rope_theta,
                                      pair_layout, rotate_precision, flags, rope_heads)
        self.pool = leyline.leyline_pool_create(self.desc, self.kv)
        self.table = torch.full((max_reqs, max_blocks), -1, dtype=torch.int32, device=self.device)
        self.seq_lens_dev = torch.zeros(max_reqs, dtype=torch.int32, device=self.device)
        self.tables = leyline.Tables(self.table, self.seq_lens_dev, np.zeros(max_reqs, dtype=np.int64))
        self._batches = weakref.WeakSet()

    # ------------------------------------------------------------------
    @property
    def seq_lens_host(self) -> np.ndarray:
        return self.tables.seq_lens_host

    @property
    def split(self) -> bool:
        return bool(self.desc.flags & leyline.LEYLINE_POOL_SPLIT_ROPE)

    def kv_view(self):
        """[layers][pages][block_size][row] view of a pool of whole rows."""
        if self.split:
            raise ValueError("a split-rope pool has no array of whole rows: use latent_view / rope_view")
        return self.kv.view(self.num_layers, self.num_pages, self.block_size, self.row)

    def latent_view(self):
        """[layers][pages][block_size][latent] view of the latents."""
        if not self.split:
            return self.kv_view()[..., :self.latent_dim]
        n = self.num_layers * self.num_pages * self.block_size * self.latent_dim
        return self.kv[:n].view(self.num_layers, self.num_pages, self.block_size, self.latent_dim)

    def rope_view(self):
        """[layers][pages][block_size][rope_heads * rope_dim] view of the rope bands."""
        if not self.split:
            return self.kv_view()[..., self.latent_dim:]
        n = self.num_layers * self.num_pages * self.block_size * self.latent_dim
        return self.kv[n:].view(self.num_layers, self.num_pages, self.block_size, self.row - self.latent_dim)

    def page_views(self):
        """The pool's arrays as [layers][pages][...] views, for comparing pages."""
        if not self.split:
            return [self.kv.view(self.num_layers, self.num_pages, -1)]
        return [self.latent_view().reshape(self.num_layers, self.num_pages, -1),
                self.rope_view().reshape(self.num_layers, self.num_pages, -1)]

    def read_rows(self, layers, pages, slots):
        """Stored whole rows [n][row] of (layer, page, slot) index tensors."""
        return self.torch.cat((self.latent_view()[layers, pages, slots], self.rope_view()[layers, pages, slots]), -1)

    def write_layer_rows(self, layer: int, flat_slots, rows) -> None:
        """Store whole rows [n][row] at flat slots (page * block_size + offset) of one layer."""
        if not self.split:
            flat = self.kv_view()[layer].reshape(self.num_pages * self.block_size, self.row)
            flat.index_copy_(0, flat_slots, rows)
            return
        lat = self.latent_view()[layer].reshape(self.num_pages * self.block_size, self.latent_dim)
        rope = self.rope_view()[layer].reshape(self.num_pages * self.block_size, self.row - self.latent_dim)
        lat.index_copy_(0, flat_slots, rows[:, :self.latent_dim].contiguous())
        rope.index_copy_(0, flat_slots, rows[:, self.latent_dim:].contiguous())

    def add_request(self, req: int, length: int) -> np.ndarray:
        """Take pages for a new request of `length` tokens and install its table row; returns the page ids."""
        n = -(-length // self.block_size)
        pages = leyline.leyline_alloc_pages(self.pool, n)
        row = np.full(self.table.shape[1], -1, dtype=np.int32)
        row[:n] = pages
        self.table[req].copy_(self.torch.from_numpy(row))
        self.seq_lens_dev[req] = length
        self.tables.seq_lens_host[req] = length
        return pages

    def slot_index(self, req: int, tokens) -> "np.ndarray":
        """Flat slot index page * block_size + offset of each token (host; reads the table)."""
        t = np.asarray(tokens, dtype=np.int64)
        row = self.table[req].cpu().numpy().astype(np.int64)
        return row[t // self.block_size] * self.block_size + t % self.block_size

    def splice(self, dirs, stream=None) -> None:
        """dirs: a list of leyline.directive() or one leyline.directive_batch() array."""
        leyline.leyline_splice(self.pool, self.tables, dirs, stream)

    def allocating(self, stream):
        """The context in which a call on `stream` makes its outputs: torch hands out a block for the stream that is
        current then, and may hand out one that another stream's kernels still use (None: the current stream)."""
        if stream is None:
            return contextlib.nullcontext()
        if not isinstance(stream, self.torch.cuda.Stream):  # an address, or another library's stream
            address = stream if isinstance(stream, int) else stream.cuda_stream
            stream = self.torch.cuda.ExternalStream(address, device=self.kv.device)
        return self.torch.cuda.stream(stream)

    def gather(self, req: int, layer: int, t0: int, t1: int, out=None, stream=None):
        """Rows [t0, t1) of a request in one layer.  An `out` made here belongs to `stream`, as if made with it
        current: a caller who uses it on another stream orders the two, as for any tensor."""
        if out is None:
            with self.allocating(stream):
                out = self.torch.empty((t1 - t0, self.row), dtype=self.torch.bfloat16, device=self.device)
        leyline.leyline_gather(self.pool, self.tables, req, layer, t0, t1, out, stream)
        return out

    def materialize(self, req: int, stream=None) -> None:
        leyline.leyline_materialize(self.pool, self.tables, req, stream)

    def materialize_requests(self, reqs, stream=None) -> None:
        """materialize several distinct requests in one launch per 64 of them."""
        leyline.leyline_materialize_requests(self.pool, self.tables, reqs, stream)

    def _on_device(self, t, what: str):
        if t.device != self.kv.device:
            raise ValueError(f"{what}: on {t.device}, the cache is on {self.kv.device}")
        return t

    def select_rows(self, weights, keeps, out=None, stream=None):
        """The rows that requests keep, by their weights [requests][rows] (Batch.attention_weights): of each entry
        (req, n_keep) or (req, n_keep, first, last) of `keeps` the rows at its ends and those of greatest weight, in
        ascending order in row k of `out` (default: a new int32 tensor, -1 behind each list)."""
        a = leyline.keep_batch(keeps)
        if out is None:
            with self.allocating(stream):
                longest = min(max(int(a["n_keep"].max()), 0), self.table.shape[1] * self.block_size) if a.size else 0
                out = self.torch.full((a.size, longest), -1, dtype=self.torch.int32, device=self.kv.device)
        leyline.leyline_select_rows(self.pool, self.tables, self._on_device(weights, "weights"), a,
                                    self._on_device(out, "out"), self._stream(stream))
        return out

    def evict(self, keeps, kept, weights=None, stream=None) -> None:
        """Drop the rows that the lists `kept` of select_rows(), or of another policy, do not name; weights move along
        (an array of weights for each layer: the others are the caller's to move, as all are after a splice)."""
        if weights is not None:
            self._on_device(weights, "weights")
        leyline.leyline_evict(self.pool, self.tables, keeps, self._on_device(kept, "kept"), weights, self._stream(stream))

    def _stream(self, stream):
        """The stream of a call: the one given, else the current one of the cache's device."""
        return leyline.current_stream_ptr(self.kv.device.index) if stream is None else stream

    def batch(self, max_chunks: int, max_tokens: int, q_heads: int) -> "Batch":
        """A batch for steps of at most max_tokens new tokens in max_chunks chunks (see Batch)."""
        b = Batch(self, max_chunks, max_tokens, q_heads)
        self._batches.add(b)
        return b

    def pending(self):
        """Pending counts [num_pages][block_size] of a lazy pool, as a torch view (None otherwise)."""
        addr = leyline.leyline_pending_ptr(self.pool)
        if not addr:
            return None
        n = self.num_pages * self.block_size
        holder = _DeviceArray(addr, n, self.device.index or 0, self)
        return self.torch.as_tensor(holder, device=self.device).view(self.num_pages, self.block_size)

    def free_pages(self) -> int:
        return leyline.leyline_free_page_count(self.pool)

    def last_stats(self) -> dict:
        return leyline.leyline_last_stats(self.pool).as_dict()

    def check_status(self) -> None:
        leyline.leyline_sync_status(self.pool)

    def close(self) -> None:
        if self.pool is not None:
            for b in list(self._batches):  # a pool outlives its batches
                b.close()
            leyline.leyline_pool_destroy(self.pool)
            self.pool = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Batch:
    """New tokens of a step: rows appended to the cache, queries turned, attention over the cache.

    plan() takes chunks of new tokens, once a step; append(), rotate(), attention() and
    attention_weights() then serve each layer, on tensors whose first axis is the plan's tokens, chunk after
    chunk.  The last four can be captured into a CUDA graph and replayed after each new plan,
    on tensors with room for max_tokens.  Outputs that a call makes belong to the stream it runs on.
    There is no backward pass: tensors that require a gradient are refused outside torch.no_grad().
    """

    def __init__(self, cache: PagedCache, max_chunks: int, max_tokens: int, q_heads: int):
        self.cache = cache
        self.max_chunks = max_chunks
        self.max_tokens = max_tokens
        self.q_heads = q_heads
        self.bands = cache.rope_heads
        self.value_dim = cache.latent_dim // self.bands
        self.tokens = 0
        self.device_index = cache.kv.device.index
        self.handle = None
        self.handle = leyline.leyline_batch_create(cache.pool, max_chunks, max_tokens, q_heads)

    def plan(self, chunks, stream=None) -> None:
        """chunks: (req, start, n) or (req, start, n, rope_start) of each: the n tokens at rows
        [start, start + n) of request req.  Rows past the request's length take pages."""
        a = leyline.chunk_batch(chunks)
        leyline.leyline_batch_plan(self.handle, self.cache.tables, a, self._stream(stream))
        self.tokens = int(a["n"].sum())

    def _stream(self, stream):
        """The stream of a call: the one given, else the current one of the cache's device."""
        return leyline.current_stream_ptr(self.device_index) if stream is None else stream

    def _device(self, t, what: str):
        if t.device != self.cache.kv.device:
            raise ValueError(f"{what}: on {t.device}, the cache is on {self.cache.kv.device}")
        return t

    def _weights(self, t, what: str, n: int):
        if t is not None and tuple(t.shape) != (n,):
            raise ValueError(f"{what}: shape {tuple(t.shape)}, expected ({n},)")
        return t if t is None else self._device(t, what)

    def _room(self, stream) -> int:
        """Tokens that the tensors of a call must have room for: the plan's, and under capture max_tokens, since the graph
        may be replayed with any plan."""
        if self.tokens == self.max_tokens:
            return self.tokens
        if stream is None:
            return self.max_tokens if leyline.current_stream_captures() else self.tokens
        with self.cache.allocating(stream):
            return self.max_tokens if leyline.current_stream_captures() else self.tokens

    def _heads(self, t, what: str, tokens: int, dim: int) -> leyline.Heads:
        return leyline.heads(self._device(t, what), what, tokens, self.q_heads, dim)

    def append(self, layer: int, rows, latent_norm=None, key_norm=None, eps: float = 1e-6, stream=None) -> None:
        """Write rows [tokens][row] of one layer, normed and turned by their positions."""
        tokens = self._room(stream)
        if rows.dim() != 2 or rows.shape[0] < tokens or rows.shape[1] != self.cache.row:
            raise ValueError(f"rows: shape {tuple(rows.shape)}, expected [>= {tokens}][{self.cache.row}]")
        leyline.leyline_append(self.handle, layer, rows,
                               self._weights(latent_norm, "latent_norm", self.cache.latent_dim),
                               self._weights(key_norm, "key_norm", self.cache.rope_dim), eps, self._stream(stream))

    def rotate(self, q, out=None, norm=None, eps: float = 1e-6, stream=None):
        """Norm and turn query bands [tokens][q_heads][rope_dim] into out (default: a new tensor; q itself is fine)."""
        if out is None:
            with self.cache.allocating(stream):
                out = self.cache.torch.empty_like(q)
        dim, tokens = self.cache.rope_dim, self._room(stream)
        leyline.leyline_rotate(self.handle, self._heads(q, "q", tokens, dim), self._heads(out, "out", tokens, dim),
                               self._weights(norm, "norm", dim), eps, self._stream(stream))
        return out

    def attention(self, layer: int, q_latent, q_rope, scale: float, out=None, lse=None, prefix: bool = False,
                  stream=None):
        """(out [tokens][q_heads][value], lse [tokens][q_heads]) of the turned queries over the rows up to
        their own (prefix: the rows before their chunk).  q_latent is None for rows of several bands."""
        torch = self.cache.torch
        if out is None:
            with self.cache.allocating(stream):
                out = torch.empty((q_rope.shape[0], self.q_heads, self.value_dim), dtype=torch.bfloat16,
                                  device=self.cache.kv.device)
        if lse is None:
            with self.cache.allocating(stream):
                lse = torch.empty((q_rope.shape[0], self.q_heads), dtype=torch.float32, device=self.cache.kv.device)
        tokens = self._room(stream)
        if (lse.dtype != torch.float32 or lse.dim() != 2 or lse.shape[0] < tokens
                or lse.shape[1] != self.q_heads or not lse.is_contiguous()):
            raise ValueError(f"lse: expected contiguous fp32 [>= {tokens}][{self.q_heads}]")
        if (q_latent is None) != (self.bands > 1):
            raise ValueError("q_latent goes with rows of one band (MLA), and only with those")
        leyline.leyline_attention(
            self.handle, layer,
            None if q_latent is None else self._heads(q_latent, "q_latent", tokens, self.cache.latent_dim),
            self._heads(q_rope, "q_rope", tokens, self.cache.rope_dim), self._heads(out, "out", tokens, self.value_dim),
            self._device(lse, "lse"), scale, leyline.LEYLINE_ATTENTION_PREFIX if prefix else 0, self._stream(stream))
        return out, lse

    def attention_weights(self, layer: int, q_latent, q_rope, lse, scale: float, weights, decay: float = 1.0,
                          prefix: bool = False, stream=None):
        """Add to weights [requests][rows] (fp32) what the queries gave to each row they attend to, w = decay * w + sum of
        exp(score - lse) over tokens and heads, with the lse that attention() returned for the same arguments.  decay is of a
        call: where one array serves all layers, give it in one layer of a step."""
        torch = self.cache.torch
        tokens = self._room(stream)
        if (lse.dtype != torch.float32 or lse.dim() != 2 or lse.shape[0] < tokens
                or lse.shape[1] != self.q_heads or not lse.is_contiguous()):
            raise ValueError(f"lse: expected contiguous fp32 [>= {tokens}][{self.q_heads}]")
        if (q_latent is None) != (self.bands > 1):
            raise ValueError("q_latent goes with rows of one band (MLA), and only with those")
        leyline.leyline_attention_weights(
            self.handle, layer,
            None if q_latent is None else self._heads(q_latent, "q_latent", tokens, self.cache.latent_dim),
            self._heads(q_rope, "q_rope", tokens, self.cache.rope_dim), self._device(lse, "lse"),
            self._device(weights, "weights"), scale, decay, leyline.LEYLINE_ATTENTION_PREFIX if prefix else 0,
            self._stream(stream))
        return weights

    def close(self) -> None:
        if self.handle is not None:
            leyline.leyline_batch_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
