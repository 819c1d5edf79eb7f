"""One decode step of a paged-KV attention layer, chained through the C ABI:

  a1  host block manager: reserve each sequence's next slot (allocating a
      block or copying a shared one on write) and export tables + lengths;
  a2  paged_kv_copy_blocks for the copy-on-write pairs, if any;
  a3  paged_kv_append of the new token's K/V at its slot;
  a4-a8  paged_decode_attention (gather, scores, online softmax, p.V, merge).

With q_len > 1 every sequence appends q_len tokens per step (slots in order)
and attends them causally (the verify step of speculative decoding): q, out
are [B, q_len, Hq, D] and k_new, v_new [B, q_len, Hkv, D].  With a sliding
window W each row attends its W most recent positions, and a1 first releases
the blocks that no token of the step (or later) can see, so a sequence holds
at most ceil((W + q_len - 1) / 16) + 1 blocks.

Device state (caches, scales, workspace) stays resident.  Per step only q,
k_new, v_new and the host-produced slot mapping / copy pairs / tables /
lengths cross to the device, all from ONE pinned staging buffer with one copy
(two staging buffers alternate so the host can prepare step n+1 while step n's
copy is in flight).  Everything is asynchronous on `stream`.

TreeStep is the step of speculative decoding with a tree of drafted tokens per
sequence: the same chain with the tree's masks in the attention, then the
verification of the drafts, the move of the accepted path's rows in the cache
and, on the host, the release of the rejected positions.
"""
import numpy as np
import torch

from . import (BlockManager, lib, paged_decode_attention, paged_decode_workspace_bytes,
               paged_kv_append, paged_kv_copy_blocks, paged_tree_attention, paged_tree_commit,
               paged_tree_verify, paged_tree_workspace_bytes, pkv_copy)

_ALIGN = 256


def _buffer(t):
    """What a call marshalled for this tensor depends on: a tensor of another
    shape or type at the same address is another buffer."""
    return t.data_ptr(), t.dtype, t.shape, t.stride()


class _Staging:
    """One contiguous byte buffer with typed sections at 256-byte offsets."""

    def __init__(self, layout, total, device, pin):
        if device.type == "cuda":
            self.buf = torch.empty(total, dtype=torch.uint8, device=device)
        else:
            self.buf = torch.empty(total, dtype=torch.uint8, pin_memory=pin)
        self.views = {}
        for name, (off, shape, dtype) in layout.items():
            n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
            self.views[name] = self.buf[off:off + n].view(dtype).view(shape)
        self.done = None   # event recorded after the last copy out of this buffer
        self.replayed = None  # the event run() records after each graph replay

    def __getitem__(self, name):
        return self.views[name]


class DecodeStep:
    def __init__(self, k_cache, v_cache, Hq, q_dtype, max_blocks, k_scale=None, v_scale=None,
                 num_splits=0, stream=None, scale=None, q_len=1, window=0, calibrated=False):
        self.k_cache, self.v_cache = k_cache, v_cache
        self.k_scale, self.v_scale = k_scale, v_scale
        self.num_blocks, self.Hkv, _, self.D = k_cache.shape
        self.Hq, self.q_dtype, self.max_blocks = Hq, q_dtype, max_blocks
        self.new_dtype = q_dtype if k_cache.dtype == torch.float8_e4m3fn else k_cache.dtype
        self.num_splits = num_splits
        self.q_len = q_len
        self.window = window
        self.calibrated = calibrated
        self.scale = 1.0 / float(np.sqrt(self.D)) if scale is None else float(scale)
        self.device = k_cache.device
        self.stream = stream if stream is not None else torch.cuda.current_stream(self.device)
        self.bm = BlockManager(self.num_blocks)
        self.seqs = []
        self._ws = None
        self._B = None
        self._host = ()
        self._turn = 0
        self.ncow = 0
        self.graph = None
        self._calls = {}    # marshalled C calls (Prepared), keyed by their buffers
        self._graphs = {}   # run(): one captured step per (staging buffer, output)
        self._ran = False

    # -- buffers ---------------------------------------------------------------
    def _sections(self, B):
        """The staging buffer's sections, the step's inputs first."""
        L = self.q_len
        rows = (B, self.Hq, self.D) if L == 1 else (B, L, self.Hq, self.D)
        kv = (B, self.Hkv, self.D) if L == 1 else (B, L, self.Hkv, self.D)
        return [("q", rows, self.q_dtype),
                ("k_new", kv, self.new_dtype),
                ("v_new", kv, self.new_dtype),
                ("slots", (B * L,), torch.int64),
                ("pairs", (2 * B * L,), torch.int32),
                ("table", (B, self.max_blocks), torch.int32),
                ("lens", (B,), torch.int32)]

    def _layout(self, B):
        layout, off = {}, 0
        for name, shape, dtype in self._sections(B):
            layout[name] = (off, shape, dtype)
            n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
            off = (off + n + _ALIGN - 1) // _ALIGN * _ALIGN
        self._io_bytes = layout["slots"][0]           # q, k_new, v_new
        self._book_bytes = off - layout["slots"][0]   # slots .. lens
        return layout, off

    def _buffers(self, B):
        if self._B == B:
            return
        self._B = B
        self._calls.clear()     # their buffers are about to be replaced
        self._graphs.clear()
        for hs in self._host:   # a copy out of a buffer that is let go of here may be in flight
            if hs.done is not None:
                hs.done.synchronize()
        layout, total = self._layout(B)
        pin = torch.cuda.is_available()
        self._host = [_Staging(layout, total, torch.device("cpu"), pin) for _ in range(2)]
        # memory of the step's stream: what torch hands out here may still be in use on the
        # current one, and what is let go of is handed out again behind the step
        with torch.cuda.stream(self.stream):
            self._dev = _Staging(layout, total, self.device, False)
            self._ws = torch.empty(self._workspace_bytes(B), dtype=torch.uint8, device=self.device)
        self.h_seqs = np.empty(B, dtype=np.int64)
        self.h_tok_seqs = np.empty(B * self.q_len, dtype=np.int64)
        self.d_q, self.d_k_new, self.d_v_new = self._dev["q"], self._dev["k_new"], self._dev["v_new"]
        self.d_slots, self.d_pairs = self._dev["slots"], self._dev["pairs"]
        self.d_table, self.d_lens = self._dev["table"], self._dev["lens"]
        self._select(self._turn)

    def _workspace_bytes(self, B):
        return paged_decode_workspace_bytes(B, self.Hq, self.Hkv, self.D, self.k_cache.dtype,
                                            self.q_dtype, self.num_splits, q_len=self.q_len)

    def _select(self, turn):
        hs = self._host[turn]
        self.h_q, self.h_k_new, self.h_v_new = hs["q"], hs["k_new"], hs["v_new"]
        self.h_slots, self.h_pairs = hs["slots"], hs["pairs"]
        self.h_table, self.h_lens = hs["table"], hs["lens"]

    # -- a1 ----------------------------------------------------------------------
    def adopt(self, seq, blocks, num_tokens):
        self.bm.adopt(seq, blocks, num_tokens)
        self.seqs.append(seq)

    def prepare(self, seqs=None):
        """Host part of a step: switches to the other staging buffer (waiting
        for the copy that last read it), then writes the slots, copy pairs,
        tables and lengths of q_len new tokens per sequence into it.  Returns
        the number of copy-on-write pairs (raises on OOM)."""
        seqs = self.seqs if seqs is None else seqs
        self._switch(seqs)
        if self.q_len == 1:
            tok_seqs = self.h_seqs
        else:
            tok_seqs = self.h_tok_seqs
            tok_seqs.reshape(-1, self.q_len)[:] = self.h_seqs[:, None]
        self._reserve(tok_seqs, self.h_slots.numpy(), seqs)
        return self.ncow

    def _switch(self, seqs):
        """The other staging buffer, and the window's releases."""
        self._buffers(len(seqs))
        self._turn ^= 1
        if self._host[self._turn].done is not None:
            self._host[self._turn].done.synchronize()
        self._select(self._turn)
        self.h_seqs[:] = seqs
        if self.window:
            for seq in seqs:
                self.bm.release_outside_window(int(seq), self.window)

    def _reserve(self, tok_seqs, slots, seqs):
        """Reserves a slot per entry of tok_seqs and exports tables and lengths."""
        ncow = self.bm.append_slots_into(tok_seqs, slots, self.h_pairs.numpy())
        if ncow < 0:
            raise MemoryError("block manager out of blocks")
        self.ncow = ncow
        rc = lib().pkv_bm_export(self.bm._h, self.h_seqs.ctypes.data, len(seqs),
                                 self.h_table.data_ptr(), self.max_blocks, self.h_lens.data_ptr())
        if rc != 0:
            raise RuntimeError(f"export failed [{rc}]")

    def _copy_in(self, with_inputs):
        """One host->device copy of the current staging buffer (the step's
        bookkeeping, and q / k_new / v_new when with_inputs)."""
        hs = self._host[self._turn]
        lo = 0 if with_inputs else self._io_bytes
        hi = self._io_bytes + self._book_bytes
        pkv_copy(self._dev.buf[lo:hi], hs.buf[lo:hi], stream=self.stream)
        with torch.cuda.stream(self.stream):
            if not torch.cuda.is_current_stream_capturing():
                ev = torch.cuda.Event()
                ev.record(self.stream)
                hs.done = ev

    def upload(self):
        """Copies the bookkeeping written by prepare() to the device."""
        self._copy_in(with_inputs=False)

    def h2d_bytes(self, with_inputs=True):
        return (self._io_bytes if with_inputs else 0) + self._book_bytes

    # -- a2..a8 ------------------------------------------------------------------
    def launch(self, q, k_new, v_new, out):
        """Runs a2..a8 with device tensors q, k_new, v_new (bookkeeping from
        the last upload())."""
        s = self.stream
        if self.ncow:
            paged_kv_copy_blocks(self.k_cache, self.v_cache, self.d_pairs[:2 * self.ncow].view(-1, 2),
                                 self.k_scale, self.v_scale, stream=s)
        key = ("append", _buffer(k_new), _buffer(v_new), self.d_slots.data_ptr())
        call = self._calls.get(key)
        if call is None:
            if k_new.dim() == 4:
                k_new = k_new.view(-1, self.Hkv, self.D)
                v_new = v_new.view(-1, self.Hkv, self.D)
            call = self._remember(key, paged_kv_append(
                k_new, v_new, self.k_cache, self.v_cache, self.d_slots, self.k_scale, self.v_scale,
                stream=s, calibrated=self.calibrated, prepare=True))
        call()
        self.attend(q, out)

    def attend(self, q, out):
        """a4-a8 on the current bookkeeping.  The C call's arguments are
        marshalled once per (q, out) pair and reused."""
        key = ("attend", _buffer(q), _buffer(out), self.d_table.data_ptr())
        call = self._calls.get(key)
        if call is None:
            call = self._remember(key, paged_decode_attention(
                out, q, self.k_cache, self.v_cache, self.d_table, self.d_lens, self.scale,
                self.k_scale, self.v_scale, num_splits=self.num_splits, workspace=self._ws,
                stream=self.stream, window=self.window, prepare=True))
        call()

    def _remember(self, key, call):
        if len(self._calls) >= 8:
            self._calls.clear()
        self._calls[key] = call
        return call

    @property
    def workspace(self):
        return self._ws

    # -- a whole step from host memory as one CUDA graph ---------------------------
    def capture(self, h_out):
        """Captures one full step from the current staging buffer — one
        host->device copy of q, k_new, v_new (written into h_q / h_k_new /
        h_v_new) and the bookkeeping, the append, and the attention writing
        its output straight into the pinned tensor h_out over the host link
        (no separate device->host copy) — as a CUDA graph; replay() runs it.
        Re-capture after a prepare() that switches staging buffers or changes
        the copy pairs."""
        if not h_out.is_pinned():
            raise ValueError("h_out must be pinned host memory")
        self.g_out = h_out
        self._graph_body(h_out)          # eager once: kernels configured, tensor maps encoded
        self.stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=self.stream):
            self._graph_body(h_out)
        self.graph = graph
        return graph

    def _graph_body(self, h_out):
        self._copy_in(with_inputs=True)
        self.launch(self.d_q, self.d_k_new, self.d_v_new, h_out)

    # -- a serving loop from host memory ----------------------------------------
    def stage_inputs(self, q, k_new, v_new, both=False):
        """Writes a step's q, k_new, v_new (host tensors) into the current
        staging buffer (both=True: into both buffers)."""
        for t in ((0, 1) if both else (self._turn,)):
            hs = self._host[t]
            hs["q"].copy_(q)
            hs["k_new"].copy_(k_new)
            hs["v_new"].copy_(v_new)

    def run(self, h_out):
        """Issues one whole step from host memory, asynchronously: the copy of
        the current staging buffer (inputs and the bookkeeping of the last
        prepare()), the append and the attention writing into the pinned
        tensor h_out.  Each staging buffer has a CUDA graph of its own,
        captured on first use, so a loop can run step n from one buffer
        while prepare() writes step n + 1 into the other:

            step.prepare(); step.run(h_out)
            while serving:
                step.prepare()            # a1 of the next step, on the host
                stream.synchronize()      # this step's output is in h_out
                ...read h_out, stage the next inputs...
                step.run(h_out)

        The first step runs eagerly (it configures the kernels and encodes
        their tensor maps outside any capture), and so does a step with
        copy-on-write pairs (rare): the graphs hold no block copy.

        A loop may also keep one step queued ahead of the host (two pinned
        output tensors alternating): issue step n, wait for step n - 1 and
        read its output, then prepare() step n + 1 — prepare() waits for the
        step that last read the staging buffer it switches to."""
        if not h_out.is_pinned():
            raise ValueError("h_out must be pinned host memory")
        if self.stream.cuda_stream == 0:
            raise ValueError("run() captures CUDA graphs: give the DecodeStep a non-default stream")
        if self.ncow or not self._ran:
            self._graph_body(h_out)
            self._ran = True
            return
        key = (self._turn, _buffer(h_out))
        graph = self._graphs.get(key)
        if graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=self.stream):
                self._graph_body(h_out)
            self._graphs[key] = graph
        with torch.cuda.stream(self.stream):
            graph.replay()
        # the graph's copy out of this staging buffer is done once the step
        # is: prepare() waits for it before rewriting the buffer
        hs = self._host[self._turn]
        if hs.replayed is None:
            hs.replayed = torch.cuda.Event()
        hs.replayed.record(self.stream)
        hs.done = hs.replayed

    def replay(self):
        with torch.cuda.stream(self.stream):
            self.graph.replay()


class TreeStep(DecodeStep):
    """One step of speculative decoding with a tree of at most `nodes` drafted
    tokens per sequence, node 0 the last confirmed token:

        step.prepare(masks, lens)          # host: slots, tables, masks
        step.upload()                      # (or run(h_out), from host memory)
        step.launch(q, k_new, v_new, out)  # append the nodes, attend the tree
        ... the model's remaining work: the target's probabilities ...
        step.verify(draft_tokens, target_probs, draft_probs, uniforms)
        step.commit()                      # the accepted path's rows, together
        path_len, next_token = step.finish()

    finish() waits for the stream and shortens each sequence to its accepted
    tokens; the next step's node 0 is next_token.  A model of several layers
    attends and commits on each layer's cache (commit(k_cache, v_cache, ...))
    and finishes once.  The device tensors d_path, d_path_len, d_next_token and
    d_new_lens hold the last verify's and commit's results."""

    def __init__(self, k_cache, v_cache, Hq, q_dtype, max_blocks, nodes, k_scale=None, v_scale=None,
                 stream=None, scale=None, window=0, calibrated=False):
        super().__init__(k_cache, v_cache, Hq, q_dtype, max_blocks, k_scale, v_scale, stream=stream,
                         scale=scale, q_len=nodes, window=window, calibrated=calibrated)

    def _sections(self, B):
        L = self.q_len
        s = super()._sections(B)
        inputs = [("q", (B, L, self.Hq, self.D), self.q_dtype),     # (also for one node)
                  ("k_new", (B, L, self.Hkv, self.D), self.new_dtype),
                  ("v_new", (B, L, self.Hkv, self.D), self.new_dtype)]
        return inputs + s[3:] + [("mask", (B, L), torch.int64), ("tree_lens", (B,), torch.int32)]

    def _workspace_bytes(self, B):
        return paged_tree_workspace_bytes(B, self.q_len, self.Hq, self.Hkv, self.D, self.k_cache.dtype, self.q_dtype)

    def _buffers(self, B):
        if self._B == B:
            return
        super()._buffers(B)
        dev = self.device
        self.d_mask, self.d_tree_lens = self._dev["mask"], self._dev["tree_lens"]
        with torch.cuda.stream(self.stream):
            self.d_path = torch.empty((B, self.q_len), dtype=torch.int32, device=dev)
            self.d_path_len = torch.empty(B, dtype=torch.int32, device=dev)
            self.d_new_lens = torch.empty(B, dtype=torch.int32, device=dev)
            self.d_next_token = torch.empty(B, dtype=torch.int64, device=dev)
        pin = torch.cuda.is_available()
        self.h_path_len = torch.empty(B, dtype=torch.int32, pin_memory=pin)
        self.h_next_token = torch.empty(B, dtype=torch.int64, pin_memory=pin)

    def _select(self, turn):
        super()._select(turn)
        self.h_mask, self.h_tree_lens = self._host[turn]["mask"], self._host[turn]["tree_lens"]

    def prepare(self, masks, lens=None, seqs=None):
        """Host part of a step: reserves lens[b] slots for sequence b (None:
        `nodes` each) and writes masks ([B, nodes] or [nodes], bit j of node
        i's: i sees j), slots, copy pairs, tables and lengths into the other
        staging buffer.  seqs: distinct ids (None: self.seqs).  Returns the
        number of copy-on-write pairs (raises on OOM: nothing is reserved
        then)."""
        seqs = self.seqs if seqs is None else [int(s) for s in seqs]
        L, B = self.q_len, len(seqs)
        lens = np.full(B, L, dtype=np.int32) if lens is None else np.asarray(lens, dtype=np.int32)
        if len(set(seqs)) != B:   # (its nodes would be appended twice, behind each other)
            raise ValueError("a sequence may appear once in a step")
        if lens.shape != (B,) or (lens < 0).any() or (lens > L).any():
            raise ValueError(f"lens must be {B} numbers in [0, {L}]")
        masks = np.ascontiguousarray(np.asarray(masks)).astype(np.uint64, copy=False)
        if masks.shape not in ((L,), (B, L)):
            raise ValueError(f"masks must be [{B}, {L}] or [{L}], got {list(masks.shape)}")
        self._switch(seqs)
        self.h_mask.numpy()[:] = masks.view(np.int64)
        self.h_tree_lens.numpy()[:] = lens
        slots = np.empty(int(lens.sum()), dtype=np.int64)
        self._reserve(np.repeat(self.h_seqs, lens), slots, seqs)
        h = self.h_slots.numpy().reshape(B, L)
        h.fill(-1)                                   # rows past a tree's nodes: skipped by the append
        h[np.arange(L)[None, :] < lens[:, None]] = slots
        return self.ncow

    def attend(self, q, out):
        key = ("attend", _buffer(q), _buffer(out), self.d_table.data_ptr())
        call = self._calls.get(key)
        if call is None:
            call = self._remember(key, paged_tree_attention(
                out, q, self.k_cache, self.v_cache, self.d_table, self.d_lens, self.d_mask, self.scale,
                tree_lens=self.d_tree_lens, k_scale=self.k_scale, v_scale=self.v_scale, window=self.window,
                workspace=self._ws, stream=self.stream, prepare=True))
        call()

    def verify(self, draft_tokens, target_probs, draft_probs=None, uniforms=None):
        """paged_tree_verify of the step's trees; (path, path_len, next_token)."""
        paged_tree_verify(self.d_path, self.d_path_len, self.d_next_token, draft_tokens, self.d_mask,
                          target_probs, draft_probs, uniforms, self.d_tree_lens, stream=self.stream)
        return self.d_path, self.d_path_len, self.d_next_token

    def commit(self, k_cache=None, v_cache=None, k_scale=None, v_scale=None):
        """Moves the accepted path's rows of the step's cache, or of another
        layer's with the same tables."""
        if k_cache is None:
            k_cache, v_cache, k_scale, v_scale = self.k_cache, self.v_cache, self.k_scale, self.v_scale
        paged_tree_commit(k_cache, v_cache, self.d_path, self.d_path_len, self.d_table, self.d_lens,
                          k_scale, v_scale, self.d_tree_lens, self.d_new_lens, stream=self.stream,
                          calibrated=self.calibrated)

    def finish(self):
        """Waits for the step and releases the rejected positions on the host;
        (path_len, next_token) as numpy arrays."""
        with torch.cuda.stream(self.stream):
            self.h_path_len.copy_(self.d_path_len, non_blocking=True)
            self.h_next_token.copy_(self.d_next_token, non_blocking=True)
        self.stream.synchronize()
        path_len, next_token = self.h_path_len.numpy().copy(), self.h_next_token.numpy().copy()
        kept = self.h_lens.numpy() - self.h_tree_lens.numpy() + path_len
        for seq, n in zip(self.h_seqs, kept):
            self.bm.truncate(int(seq), int(n))
        return path_len, next_token
