"""A BitStack linear layer, a packed key/value cache and an attention block over
torch-allocated device memory.

Plumbing around the C ABI: torch allocates the device buffers (block records, 1/s,
workspace, outputs) and pinned host memory for the records, which stand in for the
storage device the blocks are loaded from and offloaded to (review page "BitStack:
Fine-Grained Size Control...", Fig. 2: blocks move between storage and memory as the
budget changes).  Every computation is a call into the CUDA library.
"""
from __future__ import annotations

import numpy as np
import torch

from . import binding as B


class BitStackLinear:
    """One weight's block stack on one GPU.

    Parameters
    ----------
    m, d : out_features, in_features (m % 128 == 0, d % 256 == 0 for BitStack blocks)
    capacity : the most blocks the device area holds
    inv_scale : length-d float32 1/s of the activation-aware scaling
    k : singular vectors per block (16 on the GPU path; k' for plain blocks)
    plain : the blocks are "w/o AVD" rank-k' factor pairs (vanilla SVD, no signs)
    """

    def __init__(self, m: int, d: int, capacity: int, inv_scale, k: int = 16, device: str | int = "cuda",
                 stream=None, plain: bool = False):
        self.m, self.d, self.k, self.capacity = int(m), int(d), int(k), int(capacity)
        self.plain = bool(plain)
        self.device = torch.device(device)
        nbytes = (B.bs_plain_stack_device_bytes if plain else B.bs_stack_device_bytes)(m, d, k, capacity)
        if nbytes == 0:
            raise B.BsError(B.BS_ERR_UNSUPPORTED_SHAPE, "BitStackLinear")
        self.dev_blocks = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self.inv_scale = torch.as_tensor(np.asarray(inv_scale, dtype=np.float32)).to(self.device).contiguous()
        self.block_bytes = (B.bs_plain_block_bytes if plain else B.bs_block_bytes)(m, d, k)
        create = B.bs_plain_stack_create if plain else B.bs_stack_create
        self.handle = create(m, d, k, capacity, self.dev_blocks, self.inv_scale, stream)
        self.host_records: list[torch.Tensor] = []   # the storage copy of every block, pinned
        self._inflight: list[torch.Tensor] = []
        self._ws: torch.Tensor | None = None
        self._outgrown: list[torch.Tensor] = []   # captured graphs may still use them

    # ----------------------------------------------------------- storage side ----
    def add_record(self, record) -> int:
        """Keeps a block record (uint8, bs_block_bytes long) in pinned host memory."""
        rec = torch.as_tensor(np.ascontiguousarray(record, dtype=np.uint8))
        if rec.numel() != self.block_bytes:
            raise ValueError("record has the wrong size")
        pinned = torch.empty(self.block_bytes, dtype=torch.uint8, pin_memory=True)
        pinned.copy_(rec)
        self.host_records.append(pinned)
        return len(self.host_records) - 1

    def add_pinned_record(self, pinned: torch.Tensor) -> int:
        """Keeps an already pinned record (uint8, bs_block_bytes long) without copying
        it; several stacks may share one storage copy."""
        if pinned.numel() != self.block_bytes or not pinned.is_pinned():
            raise ValueError("need a pinned record of the stack's block size")
        self.host_records.append(pinned)
        return len(self.host_records) - 1

    # ----------------------------------------------------------- memory side -----
    @property
    def n_blocks(self) -> int:
        return B.bs_stack_num_blocks(self.handle)

    def append(self, stream=None) -> None:
        """Loads the next stored block onto the GPU (one async copy)."""
        n = self.n_blocks
        if n >= len(self.host_records):
            raise IndexError("no stored block left to load")
        B.bs_append_block(self.handle, self.host_records[n], stream)

    def drop(self) -> None:
        """Offloads the last loaded block (no transfer)."""
        B.bs_drop_block(self.handle)

    def set_loaded(self, n: int, stream=None) -> None:
        """Appends or drops blocks until n are loaded."""
        while self.n_blocks < n:
            self.append(stream)
        while self.n_blocks > n:
            self.drop()

    def workspace(self, n_loaded: int, batch: int) -> torch.Tensor | None:
        need = (B.bs_plain_workspace_bytes if self.plain else B.bs_workspace_bytes)(self.m, self.d, self.k,
                                                                                     n_loaded, batch)
        if need == 0:
            return None
        if self._ws is None or self._ws.numel() < need:
            ws = torch.zeros(need, dtype=torch.uint8, device=self.device)
            if torch.cuda.is_initialized() and torch.cuda.is_current_stream_capturing():
                return ws   # the graph's own, which its replays zero: nothing has zeroed it for other calls
            if self._ws is not None:
                self._outgrown.append(self._ws)
            # zeroed once: completed calls leave it consistent (device_error re-zeroes it)
            self._ws = ws
        return self._ws

    def forward(self, x: torch.Tensor, n_loaded: int | None = None, out: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        n = self.n_blocks if n_loaded is None else int(n_loaded)
        x = x.contiguous()
        if out is None:
            out = torch.empty((x.shape[0], self.m), dtype=x.dtype, device=self.device)
        ws = workspace if workspace is not None else self.workspace(n, x.shape[0])
        B.bs_linear(self.handle, x, n, out, ws, stream)
        return out

    __call__ = forward

    def reconstruct(self, n: int | None = None, dtype=torch.float32, stream=None) -> torch.Tensor:
        n = self.n_blocks if n is None else int(n)
        W = torch.empty((self.m, self.d), dtype=dtype, device=self.device)
        B.bs_reconstruct(self.handle, n, W, stream)
        return W

    def unpack_signs(self, block: int, stream=None) -> torch.Tensor:
        out = torch.empty((self.m, self.d), dtype=torch.int8, device=self.device)
        B.bs_unpack_signs(self.handle, block, out, stream)
        return out

    def device_record(self, block: int) -> torch.Tensor:
        """A view of block `block`'s record bytes on the device."""
        off = block * self.block_bytes
        return self.dev_blocks[off:off + self.block_bytes]

    def device_error(self) -> int:
        """Reads and clears the stack's sticky device error word.  After an error the
        workspace's counters may be stale, so the layer's own workspaces are zeroed."""
        status = B.bs_get_device_error(self.handle)
        if status != B.BS_OK:
            for ws in self._outgrown + ([] if self._ws is None else [self._ws]):
                ws.zero_()
        return status

    def close(self) -> None:
        if self.handle:
            B.bs_stack_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def record_from_parts(sign_words: np.ndarray, U: np.ndarray, V: np.ndarray) -> np.ndarray:
    """A block record from sign words already in the device tile order (uint32) and
    fp16 factors U (m x k) and V (d x k): the three parts laid end to end."""
    return np.concatenate([np.ascontiguousarray(sign_words, dtype="<u4").view(np.uint8),
                           np.ascontiguousarray(U, dtype=np.float16).view(np.uint8).reshape(-1),
                           np.ascontiguousarray(V, dtype=np.float16).view(np.uint8).reshape(-1)])


class PageTable:
    """Which pages of a pool the sequences hold.  Host only; pages are handed out from
    the last one returned."""

    def __init__(self, n_pages: int, page_tokens: int):
        self.n_pages, self.page_tokens = int(n_pages), int(page_tokens)
        self.free = list(range(self.n_pages - 1, -1, -1))
        self.pages: dict[int, list[int]] = {}
        self.length: dict[int, int] = {}
        self._next = 0

    def open(self) -> int:
        """A new, empty sequence."""
        s, self._next = self._next, self._next + 1
        self.pages[s], self.length[s] = [], 0
        return s

    def close(self, seq: int) -> None:
        """Returns a sequence's pages."""
        self.free.extend(reversed(self.pages.pop(seq)))
        del self.length[seq]

    def advance(self, seqs, new, room: int = 0) -> tuple[list[int], list[list[int]]]:
        """Adds new[i] tokens to seqs[i], with pages for them and for `room` more: the
        lengths before, and the pages.  Raises with nothing changed if the pool has too
        few free pages."""
        seqs, new = [int(s) for s in seqs], [int(n) for n in new]
        if not seqs or len(set(seqs)) != len(seqs) or len(new) != len(seqs) or min(new) < 0 or room < 0:
            raise ValueError("need different sequences and one count >= 0 of new tokens for each")
        for s in seqs:
            if s not in self.length:
                raise KeyError(f"no sequence {s}")
        start = [self.length[s] for s in seqs]
        if max(a + n for a, n in zip(start, new)) + room > 2 ** 31 - 512:
            raise B.BsError(B.BS_ERR_RANGE, "PageTable.advance")
        need = [max(0, -(-(a + n + room) // self.page_tokens) - len(self.pages[s])) for s, a, n in zip(seqs, start, new)]
        if sum(need) > len(self.free):
            raise B.BsError(B.BS_ERR_CAPACITY, "PageTable.advance")
        for s, k, n in zip(seqs, need, new):
            self.pages[s].extend(self.free.pop() for _ in range(k))
            self.length[s] += n
        return start, [self.pages[s] for s in seqs]

    def undo(self, seqs, start, held) -> None:
        """Takes the last advance of seqs back: their lengths, and the counts of pages they held."""
        for s, a, n in reversed(list(zip(seqs, start, held))):
            self.length[s] = a
            self.free.extend(reversed(self.pages[s][n:]))
            del self.pages[s][n:]


class BitStackCache:
    """The packed key/value cache of a model: one pool of 4-bit pages a layer, and the
    sequences' page table, which all layers share.

    Parameters
    ----------
    heads, dim : key/value heads and their size (64, 128 or 256)
    n_pages, page_tokens : pages of a layer's pool and tokens of a page (16 to 256)
    layers : pools

    ``device_bytes`` is what it takes off the memory budget given to ``bs_plan_budget``.
    Calls run on the current stream.  ``attention`` uses the cache's own workspace, so
    calls that may overlap (other streams, other graphs) pass their own.
    """

    def __init__(self, heads: int, dim: int, n_pages: int, page_tokens: int = 64, layers: int = 1,
                 device: str | int = "cuda"):
        self.heads, self.dim, self.layers = int(heads), int(dim), int(layers)
        each = B.bs_cache_device_bytes(heads, dim, page_tokens, n_pages)
        if each == 0 or layers < 1:
            raise B.BsError(B.BS_ERR_UNSUPPORTED_SHAPE, "BitStackCache")
        self.device_bytes = each * self.layers
        self.table = PageTable(n_pages, page_tokens)
        device = torch.device(device)
        self.dev_pages = torch.empty((self.layers, each), dtype=torch.uint8, device=device)
        self.device = self.dev_pages.device
        self.handles: list = []
        with torch.cuda.device(self.device):
            for pool in self.dev_pages:
                self.handles.append(B.bs_cache_create(heads, dim, page_tokens, n_pages, pool))
        self._ws: torch.Tensor | None = None
        self._outgrown: list[torch.Tensor] = []   # captured graphs may still use them

    def open(self) -> int:
        """A new, empty sequence."""
        return self.table.open()

    def close_sequence(self, seq: int) -> None:
        """Returns a sequence's pages to the pool (steps that still run keep reading
        them: reuse is ordered by the stream)."""
        self.table.close(seq)

    def step(self, seqs, new, room: int = 0) -> "B.CacheStep":
        """The next new[i] tokens of seqs[i], as one step for every layer.  Takes the
        pages they need, and those of `room` more tokens a sequence, and moves the lengths
        on; rows of the dense tensors are the sequences' tokens end to end.  A captured
        step is taken further by copying a later step's ``start`` into its own, as far as
        its room goes.  Raises with nothing changed: for more than 4096 sequences, during a
        capture (the step's arrays are copied from the host), or as PageTable.advance."""
        seqs, new = [int(s) for s in seqs], [int(x) for x in new]
        if len(seqs) > B.CACHE_MAX_SEQS or sum(new) > 2 ** 31 - 1:
            raise B.BsError(B.BS_ERR_RANGE, "BitStackCache.step")
        if torch.cuda.is_initialized() and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("a step cannot be made during a capture: make it before, and copy later ones' start into it")
        held = [len(self.table.pages.get(s, ())) for s in seqs]
        start, pages = self.table.advance(seqs, new, room)
        try:
            width = max(1, max(map(len, pages)))
            n = len(start)
            host = np.zeros(2 * n + 1 + n * width, dtype=np.int32)
            host[:n] = start
            host[n + 1:2 * n + 1] = np.cumsum(np.asarray(new, dtype=np.int64))
            rows = host[2 * n + 1:].reshape(n, width)
            for r, p in zip(rows, pages):
                r[:len(p)] = p
            dev = torch.from_numpy(host).pin_memory().to(self.device, non_blocking=True)
            cu = None if all(x == 1 for x in new) else dev[n:2 * n + 1]
            return B.CacheStep(dev[:n], dev[2 * n + 1:].view(n, width), sum(new), max(new), cu)
        except Exception:                             # no memory for its arrays
            self.table.undo(seqs, start, held)
            raise

    def append(self, step, k: torch.Tensor, v: torch.Tensor, layer: int = 0) -> None:
        """Packs k and v [rows, heads, dim] into the step's positions."""
        B.bs_cache_append(self.handles[layer], step, k, v)

    def read(self, step, layer: int = 0, dtype=torch.float16) -> tuple[torch.Tensor, torch.Tensor]:
        """The numbers stored at the step's positions: k and v [rows, heads, dim]."""
        k, v = torch.zeros((2, step.n_tokens, self.heads, self.dim), dtype=dtype, device=self.device)
        B.bs_cache_read(self.handles[layer], step, k, v)
        return k, v

    def workspace(self, step, q_heads: int) -> torch.Tensor:
        need = B.bs_cache_attention_workspace_bytes(self.handles[0], step, q_heads)
        if self._ws is None or self._ws.numel() < need:
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("the cache's workspace is too small for this step: run it once before capturing it")
            if self._ws is not None:
                self._outgrown.append(self._ws)
            # zeroed once: completed calls leave it consistent (device_error re-zeroes it)
            self._ws = torch.zeros(max(need, 1), dtype=torch.uint8, device=self.device)
        return self._ws

    def attention(self, step, q: torch.Tensor, layer: int = 0, scale: float | None = None, window: int = 0,
                  out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None) -> torch.Tensor:
        """Attention of q [rows, q_heads, dim] over the positions that each row sees."""
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        ws = workspace if workspace is not None else self.workspace(step, q.shape[1])
        B.bs_cache_attention(self.handles[layer], step, q, out, ws, scale, window, lse)
        return out

    def device_error(self) -> int:
        """Reads and clears the layers' sticky device error words: the first that is set.
        After an error the cache's own workspaces are zeroed."""
        found = [e for e in map(B.bs_cache_get_device_error, self.handles) if e != B.BS_OK]
        if found:
            for ws in self._outgrown + ([] if self._ws is None else [self._ws]):
                ws.zero_()
        return found[0] if found else B.BS_OK

    def close(self) -> None:
        while self.handles:
            B.bs_cache_destroy(self.handles.pop())

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class BitStackAttention:
    """One attention block: the q, k and v linears (one grouped launch for up to 4 rows),
    the packed cache, and the output linear.

    q (m = q_heads x dim), k, v (m = heads x dim) and o (d = q_heads x dim) are
    BitStackLinear layers, each with its own number of loaded blocks; ``cache`` and
    ``layer`` name the pool.  Runs on the current stream; its workspaces are its own and
    the cache's, so calls of one cache's blocks must not overlap.
    """

    def __init__(self, q: BitStackLinear, k: BitStackLinear, v: BitStackLinear, o: BitStackLinear,
                 cache: BitStackCache, layer: int = 0, scale: float | None = None, window: int = 0):
        dim = cache.dim
        if (k.m != cache.heads * dim or v.m != k.m or q.m % (cache.heads * dim) or o.d != q.m or
                not q.d == k.d == v.d):
            raise B.BsError(B.BS_ERR_UNSUPPORTED_SHAPE, "BitStackAttention")
        if not 0 <= layer < cache.layers:
            raise IndexError("the cache has no such layer")
        self.q, self.k, self.v, self.o, self.cache, self.layer = q, k, v, o, cache, int(layer)
        self.q_heads, self.scale, self.window = q.m // dim, scale, int(window)
        self._ws: torch.Tensor | None = None
        self._outgrown: list[torch.Tensor] = []

    def _project(self, x: torch.Tensor) -> list[torch.Tensor]:
        lin = (self.q, self.k, self.v)
        if x.shape[0] > 4 or any(l.plain for l in lin):
            return [l.forward(x) for l in lin]
        handles, counts = [l.handle for l in lin], [l.n_blocks for l in lin]
        need = B.bs_group_workspace_bytes(handles, counts, x.shape[0])
        if self._ws is None or self._ws.numel() < need:
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("the workspace is too small for this step: run it once before capturing it")
            if self._ws is not None:
                self._outgrown.append(self._ws)
            self._ws = torch.zeros(need, dtype=torch.uint8, device=x.device)
        ys = [torch.empty((x.shape[0], l.m), dtype=x.dtype, device=x.device) for l in lin]
        B.bs_linear_group(handles, [x] * 3, counts, ys, self._ws)
        return ys

    def forward(self, x: torch.Tensor, step, between=None) -> torch.Tensor:
        """x [rows, d], the step's tokens, with every linear's loaded blocks -> [rows, o.m].
        between(q, k): called with q [rows, q_heads, dim] and k [rows, heads, dim] in front
        of the cache, for position encodings; returns the pair to use."""
        if x.dim() != 2 or x.shape[0] != step.n_tokens or x.shape[1] != self.q.d:
            raise ValueError(f"x: need [{step.n_tokens}, {self.q.d}], got {list(x.shape)}")
        if x.shape[0] == 0:
            return torch.empty((0, self.o.m), dtype=x.dtype, device=x.device)
        dim = self.cache.dim
        q, k, v = (y.view(x.shape[0], -1, dim) for y in self._project(x.contiguous()))
        if between is not None:
            q, k = between(q, k)
        self.cache.append(step, k, v, self.layer)
        y = self.cache.attention(step, q, self.layer, self.scale, self.window)
        return self.o.forward(y.view(x.shape[0], -1))

    __call__ = forward

    def device_error(self) -> int:
        """The first sticky error of the linears and the cache; clears them all."""
        found = [e for e in (l.device_error() for l in (self.q, self.k, self.v, self.o)) if e != B.BS_OK]
        if found:
            for ws in self._outgrown + ([] if self._ws is None else [self._ws]):
                ws.zero_()
        found.append(self.cache.device_error())
        return found[0]
