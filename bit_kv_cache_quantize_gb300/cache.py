"""Device-side paged KVarN cache for a workload: torch owns the memory, every
computation goes through the C ABI (``kvarn``).

A ``PagedCache`` holds the packed block pool, the per-sequence block table,
the raw open-tile buffer, the decode workspace and the device error word, and
optionally the 16-bit paged pool of the comparison kernel.  With
``heads=(h0, h1)`` it holds only KV heads h0 .. h1-1 of the workload and
their query heads (one rank's shard, see ``shard``): every buffer, the
configuration and the generated inputs are those of that head range.
"""
from __future__ import annotations

import contextlib

import torch

from . import inputs as I
from . import kvarn as K

T = D = 128


class PagedCache:
    def __init__(self, w: I.Workload, device="cuda", fp16_pool: bool = False, extra_blocks: int = 0,
                 heads=None):
        self.w = w
        self.device = device
        self.h0, self.h1 = (0, w.num_kv_heads) if heads is None else heads
        self.H = self.h1 - self.h0                   # KV heads held here
        self.Hq = self.H * w.G                       # their query heads
        table, total = I.block_tables(w)
        self.table = table.to(device)
        self.max_blocks = table.shape[1]
        self.num_blocks = total + extra_blocks
        self.cfg = K.make_config(self.H, self.Hq, self.num_blocks, w.dtype, k_bits=w.k_bits, v_bits=w.v_bits)
        self.block_bytes = K.kvarn_block_bytes(self.cfg)
        self.pool = torch.zeros(self.num_blocks * self.block_bytes, dtype=torch.uint8, device=device)
        self.tail = torch.zeros(w.batch, self.H, 2, T, D, dtype=I.torch_dtype(w.dtype), device=device)
        self.ws_bytes = K.kvarn_decode_workspace_bytes(self.cfg, w.batch, self.max_blocks)
        self.ws = torch.empty(self.ws_bytes // 4 + 4, dtype=torch.float32, device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self.lens = torch.tensor(w.seq_lens, dtype=torch.int32, device=device)
        self._kept = {}  # buffers made on first use and kept: captured graphs hold their addresses
        self.pool16 = None
        if fp16_pool:
            self.pool16 = torch.zeros(self.num_blocks, self.H, 2, T, D, dtype=I.torch_dtype(w.dtype), device=device)

    # ------------------------------------------------------------ write path
    def quantize_sequence(self, b: int, k: torch.Tensor, v: torch.Tensor, stream=None):
        """k, v: [n_tok, H, D] of sequence b (device; the heads held here).
        Quantises the whole tiles into the sequence's blocks and copies the
        remainder into the open tile."""
        n = k.shape[0]
        n_full = n // T
        if n_full:
            first = torch.arange(n_full, dtype=torch.int64, device=self.device) * T
            dst = self.table[b, :n_full].contiguous()
            K.kvarn_quantize_tiles(self.cfg, k, v, self.H * D, n, first, dst, n_full, self.pool, self.err, stream)
        r = n - n_full * T
        if r:
            self.tail[b, :, 0, :r] = k[n_full * T:].permute(1, 0, 2)
            self.tail[b, :, 1, :r] = v[n_full * T:].permute(1, 0, 2)
        if self.pool16 is not None:
            nb = (n + T - 1) // T
            for i in range(nb):
                blk = int(self.table[b, i])
                m = min(T, n - i * T)
                self.pool16[blk, :, 0, :m] = k[i * T:i * T + m].permute(1, 0, 2)
                self.pool16[blk, :, 1, :m] = v[i * T:i * T + m].permute(1, 0, 2)

    def prefill(self, seqs=None, stream=None):
        """Generate each sequence's context on the device and write it."""
        heads = range(self.h0, self.h1)
        for b in (range(self.w.batch) if seqs is None else seqs):
            n = self.w.seq_lens[b]
            k = I.kv_sequence(self.w, "k", b, n, self.device, heads)
            v = I.kv_sequence(self.w, "v", b, n, self.device, heads)
            self.quantize_sequence(b, k, v, stream)

    def append(self, k_new, v_new, pos, stream=None):
        K.kvarn_append_tokens(self.cfg, k_new, v_new, pos, self.table, self.max_blocks, self.w.batch, self.tail,
                              self.pool, self.err, stream)

    # ------------------------------------------------------------ read path
    def decode(self, q, out, lens=None, stream=None):
        K.kvarn_decode_attention(self.cfg, q, self.table, self.max_blocks, self.lens if lens is None else lens,
                                 self.w.batch, self.pool, self.tail, self.w.scale, out, self.ws, self.ws_bytes,
                                 self.err, stream)

    def multiquery(self, q, n_queries, out, lens=None, stream=None):
        """q [B][n_queries][Hq][D]: the last n_queries tokens of each sequence
        attend causally to the cache (workspace grown on first use)."""
        need = K.kvarn_multiquery_workspace_bytes(self.cfg, self.w.batch, self.max_blocks, n_queries)
        if getattr(self, "mq_ws", None) is None or self.mq_ws.numel() * 4 < need:
            self.mq_ws = torch.empty(need // 4 + 4, dtype=torch.float32, device=self.device)
        K.kvarn_multiquery_attention(self.cfg, q, n_queries, self.table, self.max_blocks,
                                     self.lens if lens is None else lens, self.w.batch, self.pool, self.tail,
                                     self.w.scale, out, self.mq_ws, self.mq_ws.numel() * 4, self.err, stream)

    def decode_fp16(self, q, out, lens=None, stream=None):
        K.kvarn_fp16_decode_attention(self.cfg, q, self.table, self.max_blocks, self.lens if lens is None else lens,
                                      self.w.batch, self.pool16, self.w.scale, out, self.ws, self.ws_bytes,
                                      self.err, stream)

    @staticmethod
    def _on(stream):
        """The context in which torch's work (and the memory it hands out) is
        ordered with a call on `stream` (None: the current one, a torch stream
        or a raw handle)."""
        if stream is None:
            return contextlib.nullcontext()
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
        return torch.cuda.stream(stream)

    def _keep(self, key, make, stream=None):
        """A buffer made on first use, on the stream of the call that needs it
        first.  It is never replaced, so a captured graph may go on using it;
        making one inside a capture is refused (it would live in that graph's
        private memory)."""
        if key not in self._kept:
            with self._on(stream):
                if torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
                    raise RuntimeError("run the call once before capturing it: its workspace does not exist yet")
                self._kept[key] = make()
        return self._kept[key]

    def _workspace(self, op: str, need: int, stream=None):
        """The smallest workspace of `op` that holds `need` bytes; a new one
        has a power of two of them (64 KiB or more), so calls of every shape leave a few
        buffers behind, not one each."""
        size = 1 << max(need - 1, 0xFFFF).bit_length()
        held = [k[1] for k in self._kept if type(k) is tuple and k[0] == op and k[1] >= size]
        return self._keep((op, min(held, default=size)),
                          lambda: torch.empty(size, dtype=torch.uint8, device=self.device), stream)

    def _out_dtype(self, out) -> int:
        if out.dtype == torch.float32:
            return K.KVARN_OUT_F32
        if out.dtype == I.torch_dtype(self.w.dtype):
            return K.KVARN_OUT_16
        raise ValueError(f"out is float32 or {I.torch_dtype(self.w.dtype)}, got {out.dtype}")

    def _rows(self, q, name, n, heads):
        """q as [batch][n][heads][128] of the cache's 16-bit type."""
        want = (self.w.batch, n, heads, D)
        if q.numel() != self.w.batch * n * heads * D or q.shape[-2:] != want[-2:] or q.dtype != I.torch_dtype(self.w.dtype):
            raise ValueError(f"{name} is {want} {I.torch_dtype(self.w.dtype)}, got {tuple(q.shape)} {q.dtype}")
        return q

    def _each(self, x, name, width=1):
        """x as `width` entries per sequence: a shorter array would be read
        past its end on the device."""
        if x.numel() != self.w.batch * width:
            raise ValueError(f"{name} has {width} per sequence of {self.w.batch}, got {tuple(x.shape)}")
        return x

    def window(self, q, n_queries, out, window, n_sinks=0, lens=None, stream=None):
        """q [B][n_queries][Hq][D]: the last n_queries tokens of each sequence
        attend to the last `window` tokens up to their own and the first
        n_sinks; out of the same shape, float32 or the cache's 16-bit type
        (bfloat16 results of several queries take the products' operands at one
        rounding each: faster by a twelfth, see KVARN_OUT_16 in include/kvarn.h).
        Calls that overlap on the GPU need caches of their own."""
        self._rows(q, "q", n_queries, self.Hq)
        kind = self._out_dtype(out)
        if out.numel() != q.numel():
            raise ValueError(f"out has {out.numel()} elements, q {q.numel()}")
        lens = self._each(self.lens if lens is None else lens, "lens")
        need = K.kvarn_window_workspace_bytes(self.cfg, self.w.batch, self.max_blocks, n_queries, window, n_sinks)
        ws = self._workspace("window", need, stream)
        K.kvarn_window_attention(self.cfg, q, n_queries, self.table, self.max_blocks, lens, self.w.batch, window, n_sinks, self.pool,
                                 self.tail, self.w.scale, out, kind, ws, need, self.err, stream)

    def tree(self, q, k_draft, v_draft, mask, out, counts=None, lens=None, stream=None):
        """q [B][N][Hq][D], k_draft and v_draft [B][N][H][D], mask int64
        [B][N][ceil(N / 64)] (bit j of a row: the node sees node j), counts
        int32 [B] or None: the drafted nodes over the cache and each other.
        out as in `window` (bfloat16 results: one rounding per operand)."""
        n = q.shape[1]
        self._rows(q, "q", n, self.Hq)
        self._rows(k_draft, "k_draft", n, self.H)
        self._rows(v_draft, "v_draft", n, self.H)
        if mask.dtype != torch.int64 or tuple(mask.shape) != (self.w.batch, n, (n + 63) // 64):
            raise ValueError(f"mask is int64 {(self.w.batch, n, (n + 63) // 64)}, got {tuple(mask.shape)} {mask.dtype}")
        kind = self._out_dtype(out)
        if out.numel() != q.numel():
            raise ValueError(f"out has {out.numel()} elements, q {q.numel()}")
        lens = self._each(self.lens if lens is None else lens, "lens")
        if counts is not None:
            self._each(counts, "counts")
        need = K.kvarn_tree_workspace_bytes(self.cfg, self.w.batch, self.max_blocks, n)
        ws = self._workspace("tree", need, stream)
        K.kvarn_tree_attention(self.cfg, q, k_draft, v_draft, mask, n, counts, self.table, self.max_blocks,
                               lens, self.w.batch, self.pool, self.tail, self.w.scale,
                               out, kind, ws, need, self.err, stream)

    # ------------------------------------------------------------ drafts
    def commit(self, k_draft, v_draft, path, path_lens, pos, stream=None):
        """Append nodes path[b][0 .. path_lens[b]) (path None: the first ones)
        of the draft arrays at positions pos[b] ...; the caller's lengths grow
        by path_lens."""
        n = k_draft.shape[1]
        self._rows(k_draft, "k_draft", n, self.H)
        self._rows(v_draft, "v_draft", n, self.H)
        if path is not None:
            self._each(path, "path", path.shape[-1])
        self._each(path_lens, "path_lens")
        self._each(pos, "pos")
        K.kvarn_commit_tokens(self.cfg, k_draft, v_draft, n, path, min(n, T) if path is None else path.shape[1],
                              path_lens, pos, self.table, self.max_blocks, self.w.batch, self.tail, self.pool,
                              self.err, stream)

    # ------------------------------------------------------------ pages
    @property
    def refs(self):
        """Reference counts of the blocks, from the table on first use."""
        return self._refs()

    def _refs(self, stream=None):
        def make():
            ids = self.table[self.table >= 0].long()
            return torch.bincount(ids, minlength=self.num_blocks).to(torch.int32).contiguous()
        return self._keep("refs", make, stream)

    def alloc(self, tile_begin, tile_end, stream=None):
        """Give the open entries of tiles [tile_begin[b], tile_end[b]) free blocks."""
        self._each(tile_begin, "tile_begin")
        self._each(tile_end, "tile_end")
        need = K.kvarn_pages_workspace_bytes(self.cfg, self.w.batch)
        K.kvarn_alloc_blocks(self.cfg, self.table, self.max_blocks, self.w.batch, tile_begin, tile_end,
                             self._refs(stream), self._workspace("pages", need, stream), need, self.err, stream)

    def free(self, tile_begin, tile_end, stream=None):
        """Release the blocks of tiles [tile_begin[b], tile_end[b])."""
        self._each(tile_begin, "tile_begin")
        self._each(tile_end, "tile_end")
        K.kvarn_free_blocks(self.cfg, self.table, self.max_blocks, self.w.batch, tile_begin, tile_end,
                            self._refs(stream), self.err, stream)

    def free_behind_window(self, lens, window, n_sinks=0, stream=None):
        """Release the tiles that no query at position lens[b] - 1 or later sees."""
        self._each(lens, "lens")
        if window < 1 or n_sinks < 0:  # (as the window attention: such a range would reach tiles that are in use)
            raise ValueError(f"window >= 1 and n_sinks >= 0, got {window} and {n_sinks}")
        with self._on(stream):  # the ranges are written, and their memory reused, in the order of the call's stream
            begin = torch.full_like(lens, min(-(-n_sinks // T), self.max_blocks))
            end = ((lens - window).clamp_min(0) // T).to(torch.int32)
            self.free(begin, end, stream)
            del begin, end

    def fork(self, parent, group, lens=None, stream=None):
        """Slot b takes the sequence of slot parent[b] (within its group of
        `group` slots; -1 empties it): open tiles, table rows, counts, lens."""
        self._each(parent, "parent")
        lens = self._each(self.lens if lens is None else lens, "lens")
        refs = self._refs(stream)
        K.kvarn_fork_tails(self.cfg, parent, group, self.w.batch, lens, self.max_blocks, self.tail, self.err, stream)
        K.kvarn_fork_sequences(self.cfg, parent, group, self.w.batch, self.table, self.max_blocks, lens, refs,
                               self.err, stream)

    def compact(self, stream=None):
        """Move the live blocks to ids 0 .. L - 1; returns the device counts
        (L, moves)."""
        need = K.kvarn_pages_workspace_bytes(self.cfg, self.w.batch)
        ws = self._workspace("pages", need, stream)
        moves = self._keep("moves", lambda: torch.empty(2, self.num_blocks, dtype=torch.int32, device=self.device),
                           stream)
        counts = self._keep("counts", lambda: torch.zeros(2, dtype=torch.int32, device=self.device), stream)
        K.kvarn_compact_blocks(self.cfg, self.table, self.max_blocks, self.w.batch, self._refs(stream), moves[0],
                               moves[1], counts, ws, need, self.err, stream)
        K.kvarn_copy_blocks(self.cfg, self.pool, self.num_blocks, moves[0], self.pool, moves[1], self.num_blocks,
                            counts[1:], self.err, stream)
        return counts

    # ------------------------------------------------------------ access
    def record(self, blk: int, head: int, kv: int) -> torch.Tensor:
        kb, vb = self.cfg.k_bits, self.cfg.v_bits
        off = blk * self.block_bytes + head * K.head_rec(kb, vb) + kv * K.rec_bytes(kb)
        return self.pool[off:off + K.rec_bytes(vb if kv else kb)]

    def set_record(self, blk: int, head: int, kv: int, rec: torch.Tensor):
        self.record(blk, head, kv).copy_(rec)

    def check_error(self) -> int:
        return int(self.err.item())
