"""Device-side state for one decode step, built on the C ABI.

``DecodeStep`` owns the device buffers (PyTorch allocations) for one batch
shape and runs the hot path through libmla.so:
plan -> absorb (q_nope @ W_UK) -> split-KV latent attention (+ merge) ->
un-absorb (o_lat @ W_UV).  Nothing here computes: it allocates and marshals.
"""
from __future__ import annotations

import contextlib
import math

import numpy as np

from . import binding as L
from .workloads import Workload


def _u16_to_bf16(torch, a: np.ndarray, device):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).to(device).view(torch.bfloat16)


def pool_to_device(torch, w: Workload, device):
    """Materialise the [num_blocks, 64, 576] pool on the device (NaN outside the referenced blocks)."""
    pool = torch.full((w.num_blocks, 64, 576), float("nan"), dtype=torch.bfloat16, device=device)
    data = _u16_to_bf16(torch, w.pool_data, device)
    ids = torch.from_numpy(w.pool_ids).to(device)
    pool.index_copy_(0, ids, data)
    return pool


class DecodeStep:
    """cache_format "fp8": the bf16 pool is packed once into 656-byte FP8 rows
    (mla_fp8_pack_cache) and the decode reads those (mla_decode_fp8)."""

    def __init__(self, w: Workload, device="cuda", num_slots: int = 0, num_splits_override: int = 0,
                 checked: bool = False, with_absorb: bool = True, cache_format: str = "bf16"):
        import torch
        self.torch = torch
        self.w = w
        self.device = torch.device(device)
        self.geom = L.make_geom(w.H)
        self.batch = L.make_batch(w.B, w.T, w.causal, w.max_pages, num_slots, num_splits_override)
        self.checked = 1 if checked else 0
        dev = self.device
        self.pool = pool_to_device(torch, w, dev)
        self.cache = L.cache_from_pool(self.pool)
        self.cache_format = cache_format
        if cache_format == "fp8":
            self.pool_fp8 = torch.empty((w.num_blocks, 64, 656), dtype=torch.uint8, device=dev)
            L.check(L.mla_fp8_pack_cache(self.cache, self.pool_fp8), "mla_fp8_pack_cache")
        elif cache_format != "bf16":
            raise ValueError(f"cache_format {cache_format!r}")
        self.block_table = torch.from_numpy(w.block_table).to(dev)
        self.seq_lens = torch.from_numpy(w.seq_lens).to(dev)
        self.q_pe = _u16_to_bf16(torch, w.q_pe, dev)
        if with_absorb:
            self.q_nope = _u16_to_bf16(torch, w.q_nope, dev)
            self.w_uk = _u16_to_bf16(torch, w.w_uk, dev)
            self.w_uv = _u16_to_bf16(torch, w.w_uv, dev)
            self.q_lat = torch.empty((w.B, w.T, w.H, 512), dtype=torch.bfloat16, device=dev)
            self.o = torch.empty((w.B, w.T, w.H, 128), dtype=torch.bfloat16, device=dev)
        else:
            self.q_lat = _u16_to_bf16(torch, w.q_lat, dev)
        # The per-step inputs (query halves, lengths, block table) become views of one
        # device buffer, so that a step's host-to-device traffic can be one copy.
        parts = [n for n in ("q_nope", "q_pe", "seq_lens", "block_table") if hasattr(self, n)]
        offs, off = [], 0
        for n in parts:
            off = (off + 255) // 256 * 256
            offs.append(off)
            off += getattr(self, n).numel() * getattr(self, n).element_size()
        self.inputs = torch.empty(off, dtype=torch.uint8, device=dev)
        for n, o in zip(parts, offs):
            src = getattr(self, n)
            view = self.inputs[o: o + src.numel() * src.element_size()].view(src.dtype).view(src.shape)
            view.copy_(src)
            setattr(self, n, view)
        self._input_parts = list(zip(parts, offs))
        self.o_lat = torch.empty((w.B, w.T, w.H, 512), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((w.B, w.T, w.H), dtype=torch.float32, device=dev)
        self.ws_bytes = L.mla_workspace_size(self.geom, self.batch)
        if self.ws_bytes == 0:
            raise L.MlaError(L.MLA_ERR_ARG, "mla_workspace_size")
        self.workspace = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=dev)

    @property
    def BT(self) -> int:
        return self.w.B * self.w.T

    def io_set(self) -> dict:
        """The per-step input buffer (with its views) and output o of this step."""
        return {"inputs": self.inputs, "o": getattr(self, "o", None),
                **{n: getattr(self, n) for n, _ in self._input_parts}}

    def new_io_set(self) -> dict:
        """A second input buffer (same contents) and output, for double-buffered steps."""
        torch = self.torch
        inputs = self.inputs.clone()
        io = {"inputs": inputs, "o": torch.empty_like(self.o) if hasattr(self, "o") else None}
        for n, off in self._input_parts:
            src = getattr(self, n)
            io[n] = inputs[off: off + src.numel() * src.element_size()].view(src.dtype).view(src.shape)
        return io

    def bind(self, io: dict):
        """Point the step at an input/output set (the next calls use its buffers)."""
        self.inputs = io["inputs"]
        if io.get("o") is not None:
            self.o = io["o"]
        for n, _ in self._input_parts:
            setattr(self, n, io[n])

    def plan(self, stream=None):
        L.check(L.mla_plan(self.geom, self.batch, self.seq_lens, self.workspace, self.ws_bytes, stream), "mla_plan")

    def absorb(self, stream=None):
        L.check(L.mla_absorb_q(self.geom, self.q_nope, self.w_uk, self.q_lat, self.BT, stream), "mla_absorb_q")

    def decode(self, stream=None):
        if self.cache_format == "fp8":
            L.check(L.mla_decode_fp8(self.geom, self.batch, self.q_lat, self.q_pe, self.pool_fp8, self.w.num_blocks,
                                     self.block_table, self.block_table.shape[1], self.seq_lens, self.checked,
                                     self.o_lat, self.lse, self.workspace, self.ws_bytes, stream), "mla_decode_fp8")
            return
        L.check(L.mla_decode(self.geom, self.batch, self.q_lat, self.q_pe, self.cache, self.block_table,
                             self.block_table.shape[1], self.seq_lens, self.checked, self.o_lat, self.lse,
                             self.workspace, self.ws_bytes, stream), "mla_decode")

    def unabsorb(self, stream=None):
        L.check(L.mla_unabsorb_o(self.geom, self.o_lat, self.w_uv, self.o, self.BT, stream), "mla_unabsorb_o")

    def step(self, stream=None):
        """One pass of the whole hot path (plan, absorb, decode + merge, un-absorb)."""
        self.plan(stream)
        self.absorb(stream)
        self.decode(stream)
        self.unabsorb(stream)

    def plan_header(self):
        return read_plan_header(self.torch, self.workspace)

    def plan_tables(self):
        return read_plan_tables(self.torch, self.workspace)


def read_plan_header(torch, workspace):
    """The plan header words (include/mla.h) copied to the host."""
    return workspace[: L.HDR_WORDS * 4].view(torch.int32).cpu().numpy()


def read_plan_tables(torch, workspace):
    """(segments [n,8], range_ptr [n_ranges+1], merge [m,4]) copied from the workspace."""
    hdr = read_plan_header(torch, workspace)

    def words(off, n):
        return workspace[off: off + 4 * n].view(torch.int32).cpu().numpy()

    nseg = int(hdr[L.HDR["NUM_SEGMENTS"]])
    nr = int(hdr[L.HDR["NUM_RANGES"]])
    nm = int(hdr[L.HDR["NUM_MERGE"]])
    seg = words(int(hdr[L.HDR["OFF_SEGMENTS"]]), nseg * 8).reshape(nseg, 8)
    rp = words(int(hdr[L.HDR["OFF_RANGE_PTR"]]), nr + 1)
    mg = words(int(hdr[L.HDR["OFF_MERGE"]]), nm * 4).reshape(nm, 4)
    return seg, rp, mg


class SparseStep:
    """The index-driven decode (mla_decode_sparse) on one SparseWorkload: the
    absorbed query attends to the listed physical rows of the pool."""

    def __init__(self, sw, device="cuda", num_slots: int = 0, num_splits_override: int = 0, checked: bool = False):
        import torch
        self.torch = torch
        self.sw = sw
        w = sw.ctx
        dev = self.device = torch.device(device)
        self.geom = L.make_geom(w.H)
        self.batch = L.make_batch(w.B, w.T, False, 1, num_slots, num_splits_override)
        self.checked = 1 if checked else 0
        self.pool = pool_to_device(torch, w, dev)
        self.cache = L.cache_from_pool(self.pool)
        self.q_lat = _u16_to_bf16(torch, w.q_lat, dev)
        self.q_pe = _u16_to_bf16(torch, w.q_pe, dev)
        self.indices = torch.from_numpy(np.ascontiguousarray(sw.indices)).to(dev)
        self.topk_length = torch.from_numpy(np.ascontiguousarray(sw.topk_length)).to(dev)
        self.o_lat = torch.empty((w.B, w.T, w.H, 512), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((w.B, w.T, w.H), dtype=torch.float32, device=dev)
        self.ws_bytes = L.mla_sparse_workspace_size(self.geom, self.batch, sw.topk)
        if self.ws_bytes == 0:
            raise L.MlaError(L.MLA_ERR_ARG, "mla_sparse_workspace_size")
        self.workspace = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=dev)

    def decode(self, stream=None):
        L.check(L.mla_decode_sparse(self.geom, self.batch, self.q_lat, self.q_pe, self.cache, self.indices,
                                    self.sw.topk, self.topk_length, self.checked, self.o_lat, self.lse,
                                    self.workspace, self.ws_bytes, stream), "mla_decode_sparse")


def tree_words(parents: np.ndarray):
    """(mask int32 [B, T, ceil(T/32)], depth int32 [B, T]) of trees given by parents [B, T]
    (parents[b, t] < t for t > 0; node 0 is the root): node t sees itself and the nodes above
    it, and sits depth[b, t] positions past the root."""
    B, T = parents.shape
    W = (T + 31) // 32
    see = np.zeros((B, T, 32 * W), dtype=bool)
    depth = np.zeros((B, T), dtype=np.int32)
    rows = np.arange(B)
    for t in range(T):
        if t:
            up = parents[:, t]
            if not ((up >= 0) & (up < t)).all():
                raise ValueError(f"node {t}: a parent is not an earlier node")
            see[:, t] = see[rows, up]
            depth[:, t] = depth[rows, up] + 1
        see[:, t, t] = True
    words = (see.reshape(B, T, W, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1)
    return words.astype(np.uint32).view(np.int32), depth


class _PagedLayer:
    """What the steps of a layer over a paged cache that starts empty have in common: the pool, the pages' bookkeeping
    and the sequences' committed rows."""

    def __init__(self, B: int, H: int, T: int, max_pages: int, num_blocks: int, device, cache_format: str, interleaved: bool):
        import torch
        self.torch = torch
        dev = torch.device(device)
        self.B, self.H, self.T, self.max_pages, self.num_blocks = B, H, T, max_pages, num_blocks
        self.interleaved = interleaved
        self.geom = L.make_geom(H)
        if cache_format not in ("bf16", "fp8"):
            raise ValueError(f"cache_format {cache_format!r}")
        if not (0 <= B <= 8192 and 1 <= T <= 1024 and 1 <= num_blocks < 1 << 25 and 1 <= max_pages < 1 << 25
                and B * max_pages < 1 << 31 and B * T * (H + 1) < 1 << 31):
            raise ValueError(f"B {B}, T {T}, H {H}, max_pages {max_pages}, num_blocks {num_blocks}")
        self.cache_format = cache_format
        if cache_format == "fp8":
            self.pool = torch.zeros((num_blocks, 64, 656), dtype=torch.uint8, device=dev)
        else:
            self.pool = torch.zeros((num_blocks, 64, 576), dtype=torch.bfloat16, device=dev)
            self.cache = L.cache_from_pool(self.pool)
        self.refs = torch.zeros(num_blocks, dtype=torch.int32, device=dev)
        self.device = self.refs.device
        self.block_table = self._i32(B, max_pages, fill=-1)
        self.seq_lens, self.new_lens, self.held_lens, self.live = (self._i32(B) for _ in range(4))
        self.q_nope, self.q_pe = self._bf16(B, T, H, 128), self._bf16(B, T, H, 64)
        self.q_lat, self.o_lat, self.o = self._bf16(B, T, H, 512), self._bf16(B, T, H, 512), self._bf16(B, T, H, 128)
        self.lse = torch.empty((B, T, H), dtype=torch.float32, device=dev)

    def _i32(self, *shape, fill=0):
        return self.torch.full(shape, fill, dtype=self.torch.int32, device=self.refs.device)

    def _bf16(self, *shape):
        return self.torch.empty(shape, dtype=self.torch.bfloat16, device=self.refs.device)

    def _workspace(self, size: int):
        if size == 0:
            raise L.MlaError(L.MLA_ERR_ARG, "workspace size")
        self.ws_bytes = size
        self.workspace = self.torch.zeros(size, dtype=self.torch.uint8, device=self.device)

    def _new_rows(self, T, q, kv, cos_sin, w_uk, w_uv, q_weight, kv_weight, eps):
        """The arguments of a step's T tokens per sequence checked; the token strides of q and kv."""
        B, H = self.B, self.H
        bf16 = (self.torch.bfloat16,)
        q_step = self._fits("q", q, bf16, (B, T, H, 192), rows=True)
        kv_step = self._fits("kv", kv, bf16, (B, T, 576), rows=True)
        self._fits("cos_sin", cos_sin, (self.torch.float32,), (None, 64))
        if not eps >= 0 or cos_sin.shape[0] < 1:
            raise ValueError(f"eps {eps}, {cos_sin.shape[0]} positions")
        for name, t, shape in (("w_uk", w_uk, (H, 128, 512)), ("w_uv", w_uv, (H, 128, 512)), ("q_weight", q_weight, (192,)),
                               ("kv_weight", kv_weight, (512,))):
            if t is not None:
                self._fits(name, t, bf16, shape)
        return q_step, kv_step

    def _resize(self, cur, new, got, stream):
        L.check(L.mla_pages_resize(self.refs, self.num_blocks, self.block_table, self.max_pages, self.max_pages, cur, new,
                                   self.B, got, stream), "mla_pages_resize")

    def _append(self, N, positions, slots, q, q_step, kv, kv_step, cos_sin, w_uk, q_weight, kv_weight, eps, stream):
        """The N tokens' rows into the cache, and their absorbed queries."""
        H = self.H
        args = (self.geom, N, q, q_step, q.stride(2) if H > 1 else 192, kv, kv_step, q_weight, kv_weight, eps, cos_sin,
                cos_sin.shape[0], positions, self.interleaved)
        tail = (slots, self.q_nope, self.q_pe, stream)
        if self.cache_format == "fp8":
            L.check(L.mla_rope_append_fp8(*args, self.pool, self.num_blocks, *tail), "mla_rope_append_fp8")
        else:
            L.check(L.mla_rope_append(*args, self.cache, *tail), "mla_rope_append")
        L.check(L.mla_absorb_q(self.geom, self.q_nope, w_uk, self.q_lat, N, stream), "mla_absorb_q")

    def _fits(self, name, t, dtypes, shape, rows=False):
        """t has the shape, one of the types and the device, 16-byte aligned and contiguous; rows: of [B, T]
        rows that are contiguous, aligned and evenly spaced (the elements from one to the next are returned)."""
        if t.dtype not in dtypes or t.device != self.device or t.dim() != len(shape) or any(
                n is not None and n != m for n, m in zip(shape, t.shape)):
            raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype} on {t.device}")
        if t.data_ptr() % 16:
            raise ValueError(f"{name} is not 16-byte aligned")
        if not rows:
            if not t.is_contiguous():
                raise ValueError(f"{name} is not contiguous")
            return None
        B, T = t.shape[:2]
        step = t.stride(1) if T > 1 else t.stride(0)
        if (t.size(-1) > 1 and t.stride(-1) != 1) or (B > 1 and T > 1 and t.stride(0) != T * step) or any(
                m > 1 and s * t.element_size() % 16 for m, s in zip(t.shape[:-1], t.stride())):
            raise ValueError(f"{name}: strides {t.stride()}")
        return step if B * T > 1 else (math.prod(t.shape[2:]) + 7) // 8 * 8

    def _on(self, stream):
        """Torch's part of a call goes to the stream that the library's calls take (None: the current one of
        the step's device), and what it allocates belongs to that stream."""
        torch = self.torch
        if self.device.type != "cuda" or (stream is None and torch.cuda.current_device() == self.device.index):
            return contextlib.nullcontext()
        on = contextlib.ExitStack()
        on.enter_context(torch.cuda.device(self.device))
        if stream is not None:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
            on.enter_context(torch.cuda.stream(stream))
        return on

    def _released(self, src, dst):
        """Boolean [B]: the sequences that become another's fork, by the rules of mla_pages_fork."""
        torch, B = self.torch, self.B
        row = lambda v: torch.where((v >= 0) & (v < B), v, B).long()  # noqa: E731  (B: no sequence)
        s, d = row(src), row(dst)
        named = torch.zeros(B + 1, dtype=torch.int32, device=self.device).index_add_(0, d, torch.ones_like(dst))
        stands = (s < B) & (d < B) & (s != d) & (named[d] == 1) & (named[s] == 0)
        out = torch.zeros(B + 1, dtype=torch.bool, device=self.device)
        return out.index_fill_(0, torch.where(stands, d, B), True)[:B]

    def _lose_rows(self, which):
        """Sequences which (bool [B], on the device) are about to lose the rows that they have."""

    def fork(self, src, dst, stream=None):
        """Sequences dst become forks of src (int32 device arrays); what dst held is given back first.  src[f] =
        dst[f] gives the sequence a last page of its own.  A fork that mla_pages_fork refuses (a number
        outside [0, B), a dst named twice, a src that is another fork's dst) is reported and changes
        nothing; one for which no block is left is reported and leaves its dst empty."""
        n = src.numel()
        self._fits("src", src, (self.torch.int32,), (n,))
        self._fits("dst", dst, (self.torch.int32,), (n,))
        if n > 4096:
            raise ValueError(f"{n} forks")
        with self._on(stream):
            released = self._released(src, dst)
            self._lose_rows(released)
            keep = self.torch.where(released, 0, self.seq_lens)
            copies = self.torch.empty((3, n), dtype=self.torch.int32, device=self.device)
            self._resize(self.seq_lens, keep, self.seq_lens, stream)
            L.check(L.mla_pages_fork(self.refs, self.num_blocks, self.block_table, self.max_pages, self.max_pages,
                                     self.seq_lens, self.B, src, dst, n, copies, stream), "mla_pages_fork")
            if self.cache_format == "fp8":
                L.check(L.mla_cache_copy_fp8(self.pool, self.num_blocks, copies, n, stream), "mla_cache_copy_fp8")
            else:
                L.check(L.mla_cache_copy(self.cache, copies, n, stream), "mla_cache_copy")

    def check(self, stream=None):
        """Raise what the device reported since the last check (synchronises)."""
        with self._on(stream):
            status, info = L.mla_read_device_status(self.workspace, stream)
        if status != L.MLA_OK:
            raise L.MlaError(status, f"{self._name} ({info})")


class SpecStep(_PagedLayer):
    """Speculative decoding of one layer over a paged cache that starts empty.

    Each sequence has ``seq_lens`` committed rows.  A step drafts a tree of up to T nodes
    per sequence (node 0: the last token decided, whose row is not cached yet):
    ``set_tree`` -> ``attend`` (pages for the nodes' rows, norms + rotation + append,
    absorption, tree attention, un-absorption), then ``accept`` (verification against the
    target's probabilities) and ``commit`` (accepted rows moved together, the other pages
    given back), in this order; ``fork`` between steps.  attend, accept, commit and fork run on
    the device without a host synchronisation, so that they can be captured in a CUDA graph;
    set_tree copies from the host.  ``check`` raises what the device reported: the last step's
    attention, and everything else since the last check.  A sequence whose nodes get no pages
    (no free block, or past its table) is reported and sits the step out: outputs 0,
    accept_len 0, its rows as they were.  Arguments that do not fit raise ValueError before
    anything is launched.
    FP8 pages are converted ahead of the attention where T * H > 128, in a workspace of
    B * max_pages bf16 pages (72 KB each, however many are in use); convert_ahead=False does
    without it, at about half the speed.
    ``stream`` (a torch stream or its handle; None: torch's current one) is the same for every
    call of a step, and for the calls between steps.
    """

    _name = "speculative step"

    def __init__(self, B: int, H: int, T: int, max_pages: int, num_blocks: int, device="cuda",
                 cache_format: str = "bf16", interleaved: bool = True, num_slots: int = 0, convert_ahead: bool = True):
        super().__init__(B, H, T, max_pages, num_blocks, device, cache_format, interleaved)
        self.batch = L.make_batch(B, T, False, max_pages, num_slots)
        size = L.mla_tree_fp8_workspace_size if cache_format == "fp8" and convert_ahead else L.mla_workspace_size
        self._workspace(size(self.geom, self.batch))
        self.node_lens, self.tree_lens = self._i32(B), self._i32(B)
        self._stage, self._moved = "attend", False
        self.parents, self.depth, self.mask = self._i32(B, T), self._i32(B, T), self._i32(B, T, (T + 31) // 32)
        self.accept_len, self.accept_idx, self.out_tokens = self._i32(B), self._i32(B, T), self._i32(B, T)
        self.nodes = self.torch.arange(T, dtype=self.torch.int32, device=self.device)

    def _expect(self, stage):
        """The part that is next (it becomes another one when a part is through: what fails leaves the step where it was)."""
        if self._stage != stage:
            raise RuntimeError(f"{stage} where {self._stage} is next")

    def set_tree(self, parents: np.ndarray, node_lens: np.ndarray, stream=None):
        """The next step's trees (host arrays): parents [B, T], node_lens [B] (the first node_lens[b] nodes count,
        the other parents are not looked at).  Copied from the host: waits for the stream."""
        if self._stage != "attend":
            raise RuntimeError("set_tree within a step")
        parents, node_lens = np.asarray(parents), np.asarray(node_lens)
        if parents.shape != (self.B, self.T) or node_lens.shape != (self.B,):
            raise ValueError(f"parents {parents.shape}, node_lens {node_lens.shape}")
        if ((node_lens < 0) | (node_lens > self.T)).any():
            raise ValueError("a node count outside [0, T]")
        parents = np.where(np.arange(self.T) < node_lens[:, None], parents, 0)
        words, depth = tree_words(parents)
        with self._on(stream):
            for dst, src in ((self.parents, parents), (self.depth, depth), (self.mask, words), (self.node_lens, node_lens)):
                dst.copy_(self.torch.from_numpy(np.ascontiguousarray(src, dtype=np.int32)))

    def attend(self, q, kv, cos_sin, w_uk, w_uv, q_weight=None, kv_weight=None, eps: float = 1e-6, stream=None):
        """The nodes' rows into the cache and their attention: q [B, T, H, 192], kv [B, T, 576] -> o [B, T, H, 128].

        cos_sin [positions, 64] covers every position: a node past it is reported, its row is not written, and
        what the step gives for its sequence is not to be used."""
        torch, bt, N = self.torch, self.block_table, self.B * self.T
        q_step, kv_step = self._new_rows(self.T, q, kv, cos_sin, w_uk, w_uv, q_weight, kv_weight, eps)
        self._expect("attend")
        with self._on(stream):
            torch.add(self.seq_lens, self.node_lens, out=self.new_lens)
            self._resize(self.seq_lens, self.new_lens, self.held_lens, stream)
            try:
                granted = self.held_lens == self.new_lens
                torch.mul(self.node_lens, granted, out=self.live)
                torch.add(self.seq_lens, self.live, out=self.tree_lens)
                row = self.seq_lens[:, None] + self.nodes
                blk = bt.gather(1, (row // 64).clamp(max=self.max_pages - 1).long())
                counts = self.nodes < self.live[:, None]
                slots = torch.where(counts & (blk >= 0), blk * 64 + row % 64, -1).int()
                positions = torch.where(counts, self.seq_lens[:, None] + self.depth, 0).int()
                self._append(N, positions, slots, q, q_step, kv, kv_step, cos_sin, w_uk, q_weight, kv_weight, eps, stream)
                L.check(L.mla_plan_tree(self.geom, self.batch, self.tree_lens, self.live, self.workspace, self.ws_bytes,
                                        stream), "mla_plan_tree")
                tail = (bt, self.max_pages, self.tree_lens, self.live, self.mask, 0, self.o_lat, self.lse, self.workspace,
                        self.ws_bytes, stream)
                if self.cache_format == "fp8":
                    L.check(L.mla_decode_tree_fp8(self.geom, self.batch, self.q_lat, self.q_pe, self.pool, self.num_blocks,
                                                  *tail), "mla_decode_tree_fp8")
                else:
                    L.check(L.mla_decode_tree(self.geom, self.batch, self.q_lat, self.q_pe, self.cache, *tail),
                            "mla_decode_tree")
                L.check(L.mla_unabsorb_o(self.geom, self.o_lat, w_uv, self.o, N, stream), "mla_unabsorb_o")
            except BaseException:    # the pages are given back
                L.mla_pages_resize(self.refs, self.num_blocks, bt, self.max_pages, self.max_pages, self.held_lens,
                                   self.seq_lens, self.B, self.new_lens, stream)
                raise
        self._stage = "accept"
        return self.o

    def accept(self, target_probs, draft_probs, tokens, u_accept, u_sample, V: int, stream=None):
        """Verification: probabilities [B, T, >= V] fp32 or bf16 (draft_probs None: point masses), tokens int32 [B, T]."""
        torch, B, T = self.torch, self.B, self.T
        dtype = L.MLA_DTYPE_BF16 if target_probs.dtype == torch.bfloat16 else L.MLA_DTYPE_F32
        step = self._fits("target_probs", target_probs, (torch.float32, torch.bfloat16), (B, T, None), rows=True)
        if not 1 <= V <= min(target_probs.shape[2], 1 << 30) or step < V:
            raise ValueError(f"target_probs: {target_probs.shape[2]} entries {step} apart, of {V}")
        if draft_probs is not None and self._fits("draft_probs", draft_probs, (target_probs.dtype,),
                                                  target_probs.shape, rows=True) != step:
            raise ValueError(f"draft_probs: strides {draft_probs.stride()}, target_probs: {target_probs.stride()}")
        self._fits("tokens", tokens, (torch.int32,), (B, T))
        self._fits("u_accept", u_accept, (torch.float32,), (B, T))
        self._fits("u_sample", u_sample, (torch.float32,), (B,))
        self._expect("accept")
        with self._on(stream):
            L.check(L.mla_verify_tree(B, T, V, target_probs, draft_probs, dtype, step, tokens, self.parents, self.live,
                                      u_accept, u_sample, self.accept_len, self.accept_idx, self.out_tokens, stream),
                    "mla_verify_tree")
        self._stage = "commit"
        return self.accept_len, self.out_tokens

    def commit(self, stream=None):
        """The accepted nodes' rows become the sequences' own; the other pages are given back."""
        self._expect("commit")
        with self._on(stream):
            if not self._moved:       # (moving the rows twice would mix them)
                args = (self.block_table, self.max_pages, self.max_pages, self.tree_lens, self.live, self.accept_len,
                        self.accept_idx, self.B, self.T, self.new_lens, stream)
                if self.cache_format == "fp8":
                    L.check(L.mla_cache_compact_fp8(self.pool, self.num_blocks, *args), "mla_cache_compact_fp8")
                else:
                    L.check(L.mla_cache_compact(self.cache, *args), "mla_cache_compact")
                self._moved = True
            self._resize(self.held_lens, self.new_lens, self.seq_lens, stream)
            self._moved = False
        self._stage = "attend"

    def fork(self, src, dst, stream=None):
        """As in every paged layer, between steps."""
        if self._stage != "attend":
            raise RuntimeError("fork within a step")
        super().fork(src, dst, stream)


class ServeStep(_PagedLayer):
    """Ordinary decoding of one layer over a paged cache that starts empty: a batch whose sequences may share prefixes.

    Each sequence has ``seq_lens`` rows.  ``attend`` takes up to t new tokens of each (q [B, t, ...], any t up to T: a
    prompt's chunk, then one token at a time): pages, rows (norms, rotation, append), absorption, attention with the rows
    that a set of sequences shares attended once for all of them, un-absorption.  The rows are the sequence's own from then
    on.  ``sample`` draws the next tokens from the model's logits.  ``fork`` makes sequences of others (samples of one
    prompt, requests behind one system prompt): full pages are shared.  ``set_sharing`` tells which consecutive sequences
    share how many rows, in up to ``max_sets`` sets (none at first: shared pages are then attended for each sequence).  A set
    of which a sequence is released or becomes another's fork shares nothing until it is told anew.  A set may be told with
    empty sequences in it; once one of them has rows of its own it has to be told anew (a sequence that holds other rows than
    its set is reported, and does not see the set's).  ``release`` gives sequences' pages back.  All of these run on the device without a host synchronisation, so that they can be captured in a CUDA graph
    (but for set_sharing of host arrays).  ``check`` raises what the device reported: the last attention, and everything
    else since the last check.  A sequence whose tokens get no pages (no free block, or past its table) is reported and sits
    the step out: outputs 0, its rows as they were (``live``: the tokens of each sequence that took part).  Arguments that
    do not fit raise ValueError before anything is launched.  ``stream`` as for SpecStep.
    """

    _name = "serving step"

    def __init__(self, B: int, H: int, T: int, max_pages: int, num_blocks: int, device="cuda", cache_format: str = "bf16",
                 interleaved: bool = True, num_slots: int = 0, max_sets: int = 64):
        if not 0 <= max_sets <= 8192:
            raise ValueError(f"{max_sets} sets")
        super().__init__(B, H, T, max_pages, num_blocks, device, cache_format, interleaved)
        self.num_slots, self.max_sets = num_slots, max_sets
        # (t tokens a sequence may need more than T: multiples of 128 query rows share nothing)
        self._workspace(max(L.mla_shared_workspace_size(self.geom, L.make_batch(B, t, True, max_pages, num_slots))
                            for t in range(1, T + 1)))
        self.set_ptr, self.prefix_lens = self._i32(max_sets + 1), self._i32(max_sets)
        self.lens, self.tokens = self._i32(B), self._i32(B)
        self.positions, self.slots = self._i32(B * T), self._i32(B * T)

    def set_sharing(self, set_ptr, prefix_lens, stream=None):
        """Set p: sequences set_ptr[p] .. set_ptr[p + 1] - 1 hold the same blocks for their first prefix_lens[p] rows.
        Host sequences (copied: waits for the stream) or int32 device arrays."""
        n = len(prefix_lens)
        if len(set_ptr) != n + 1 or n > self.max_sets:
            raise ValueError(f"{len(set_ptr)} bounds and {n} prefixes, {self.max_sets} sets at most")
        torch = self.torch
        if torch.is_tensor(set_ptr) and torch.is_tensor(prefix_lens):
            self._fits("set_ptr", set_ptr, (torch.int32,), (n + 1,))
            self._fits("prefix_lens", prefix_lens, (torch.int32,), (n,))
        else:
            ptr, rows = np.asarray(set_ptr, dtype=np.int64), np.asarray(prefix_lens, dtype=np.int64)
            if (np.diff(ptr) < 0).any() or ptr.min() < 0 or ptr.max() > self.B or (rows < 0).any() or (rows >= 1 << 31).any():
                raise ValueError(f"sets {ptr.tolist()}, prefixes {rows.tolist()}")
            set_ptr, prefix_lens = torch.from_numpy(ptr.astype(np.int32)), torch.from_numpy(rows.astype(np.int32))
        with self._on(stream):
            # (the sets past these are empty)
            self.set_ptr[:n + 1].copy_(set_ptr)
            self.set_ptr[n + 1:] = self.set_ptr[n:n + 1]
            self.prefix_lens[:n].copy_(prefix_lens)
            self.prefix_lens[n:] = 0

    def _lose_rows(self, which):
        if self.max_sets == 0:
            return
        torch = self.torch
        upto = torch.zeros(self.B + 1, dtype=torch.int64, device=self.device)
        torch.cumsum(which, 0, out=upto[1:])
        upto = upto[self.set_ptr.clamp(0, self.B).long()]
        self.prefix_lens.masked_fill_(upto[1:] > upto[:-1], 0)

    def attend(self, q, kv, counts, cos_sin, w_uk, w_uv, q_weight=None, kv_weight=None, eps: float = 1e-6, stream=None):
        """counts int32 [B]: sequence b's tokens are q[b, :counts[b]], kv[b, :counts[b]] (q [B, t, H, 192], kv [B, t, 576],
        1 <= t <= T); -> o [B, t, H, 128], 0 for the others (it stands until the next attend).

        cos_sin [positions, 64] covers every position: a token past it is reported, its row is not written, and what
        the step gives for its sequence is not to be used."""
        if q.dim() != 4 or not 1 <= q.shape[1] <= self.T:
            raise ValueError(f"q: {tuple(q.shape)}, {self.T} tokens at most")
        bt, T = self.block_table, q.shape[1]
        N = self.B * T
        q_step, kv_step = self._new_rows(T, q, kv, cos_sin, w_uk, w_uv, q_weight, kv_weight, eps)
        self._fits("counts", counts, (self.torch.int32,), (self.B,))
        batch = L.make_batch(self.B, T, True, self.max_pages, self.num_slots)
        with self._on(stream):
            self.torch.add(self.seq_lens, counts.clamp(0, T), out=self.new_lens)
            self._resize(self.seq_lens, self.new_lens, self.held_lens, stream)
            try:
                L.check(L.mla_batch_map(self.B, T, N, self.seq_lens, counts, self.held_lens, bt, self.max_pages, self.max_pages,
                                        self.num_blocks, None, self.live, self.lens, None, None, self.positions, self.slots,
                                        stream), "mla_batch_map")
                self._append(N, self.positions, self.slots, q, q_step, kv, kv_step, cos_sin, w_uk, q_weight, kv_weight, eps, stream)
                L.check(L.mla_plan_shared(self.geom, batch, self.lens, self.live, self.max_sets, self.set_ptr,
                                          self.prefix_lens, self.workspace, self.ws_bytes, stream), "mla_plan_shared")
                tail = (bt, self.max_pages, self.lens, self.live, 0, self.o_lat, self.lse, self.workspace, self.ws_bytes, stream)
                if self.cache_format == "fp8":
                    L.check(L.mla_decode_shared_fp8(self.geom, batch, self.q_lat, self.q_pe, self.pool, self.num_blocks, *tail),
                            "mla_decode_shared_fp8")
                else:
                    L.check(L.mla_decode_shared(self.geom, batch, self.q_lat, self.q_pe, self.cache, *tail), "mla_decode_shared")
                L.check(L.mla_unabsorb_o(self.geom, self.o_lat, w_uv, self.o, N, stream), "mla_unabsorb_o")
            except BaseException:    # the pages are given back
                L.mla_pages_resize(self.refs, self.num_blocks, bt, self.max_pages, self.max_pages, self.held_lens,
                                   self.seq_lens, self.B, self.new_lens, stream)
                raise
            # (what a sequence got of pages without taking part goes back)
            self._resize(self.held_lens, self.lens, self.seq_lens, stream)
        return self.o.view(-1)[:N * self.H * 128].view(self.B, T, self.H, 128)

    def sample(self, logits, V: int, u=None, temperature=None, top_k=None, top_p=None, min_p=None, probs=None, stream=None):
        """The next token of each row of logits [N, >= V] (fp32 or bf16; mla_sample's rule) -> int32 [N] (u None: none), a
        new tensor each time (``tokens``: the last one); probs [N, >= V], fp32 or bf16: the probabilities that the filters leave."""
        torch = self.torch
        types = (torch.float32, torch.bfloat16)
        dtype = lambda t: L.MLA_DTYPE_BF16 if t.dtype == torch.bfloat16 else L.MLA_DTYPE_F32  # noqa: E731
        if logits.dim() != 2:
            raise ValueError(f"logits: {tuple(logits.shape)}")
        N = logits.shape[0]

        def rows(name, t):
            if t.dtype not in types or t.device != self.device or t.dim() != 2 or t.shape[0] != N or not 1 <= V <= t.shape[1]:
                raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype} on {t.device}, V {V}")
            step = t.stride(0) if N > 1 else (t.shape[1] + 7) // 8 * 8
            if t.data_ptr() % 16 or t.stride(1) != 1 and t.shape[1] > 1 or step < V or step * t.element_size() % 16:
                raise ValueError(f"{name}: strides {t.stride()} at {t.data_ptr() % 16}")
            return step

        if V >= 1 << 20 or (u is None and probs is None):
            raise ValueError(f"V {V}, u {u}, probs {probs}")
        step = rows("logits", logits)
        probs_step = 0 if probs is None else rows("probs", probs)
        for name, t, kind in (("u", u, torch.float32), ("temperature", temperature, torch.float32), ("top_k", top_k, torch.int32),
                              ("top_p", top_p, torch.float32), ("min_p", min_p, torch.float32)):
            if t is not None:
                self._fits(name, t, (kind,), (N,))
        with self._on(stream):
            tokens = None if u is None else torch.empty(N, dtype=torch.int32, device=self.device)
            L.check(L.mla_sample(N, V, logits, dtype(logits), step, temperature, top_k, top_p, min_p, u, tokens, probs,
                                 L.MLA_DTYPE_F32 if probs is None else dtype(probs), probs_step, stream), "mla_sample")
        if tokens is not None:
            self.tokens = tokens
        return tokens

    def release(self, which, stream=None):
        """The sequences with which[b] (bool [B], on the device) become empty, and their pages are given back."""
        self._fits("which", which, (self.torch.bool,), (self.B,))
        with self._on(stream):
            self._lose_rows(which)
            self._resize(self.seq_lens, self.torch.where(which, 0, self.seq_lens), self.seq_lens, stream)


class NormalStep:
    """The Normal (decompressed) arm on one workload: expand the latent cache into
    per-head keys and values (mla_normal_expand), then causal MHA over them
    (mla_normal_attention).  Inputs are q_nope / q_pe directly; no absorption."""

    def __init__(self, w: Workload, device="cuda", chunk_rows: int = 0):
        import torch
        self.torch = torch
        self.w = w
        self.device = torch.device(device)
        dev = self.device
        self.chunk_rows = int(chunk_rows)
        self.geom = L.make_geom(w.H)
        self.batch = L.make_batch(w.B, w.T, w.causal, w.max_pages)
        self.pool = pool_to_device(torch, w, dev)
        self.cache = L.cache_from_pool(self.pool)
        self.block_table = torch.from_numpy(w.block_table).to(dev)
        self.seq_lens = torch.from_numpy(w.seq_lens).to(dev)
        self.q_nope = _u16_to_bf16(torch, w.q_nope, dev)
        self.q_pe = _u16_to_bf16(torch, w.q_pe, dev)
        self.w_uk = _u16_to_bf16(torch, w.w_uk, dev)
        self.w_uv = _u16_to_bf16(torch, w.w_uv, dev)
        if self.chunk_rows > 0:
            # chunked prefix: one window of expanded rows plus the running fp32 state
            self.rows_per_seq = self.chunk_rows
            nbytes = L.mla_normal_chunk_bytes(self.geom, w.B, self.chunk_rows)
            sbytes = L.mla_normal_chunk_state_bytes(self.geom, self.batch)
            if nbytes == 0 or sbytes == 0:
                raise L.MlaError(L.MLA_ERR_ARG, "mla_normal_chunk_bytes")
            self.state = torch.empty(sbytes, dtype=torch.uint8, device=dev)
        else:
            self.rows_per_seq = L.mla_normal_rows_per_seq(w.max_pages)
            nbytes = L.mla_normal_expanded_bytes(self.geom, w.B, w.max_pages)
            if nbytes == 0 and w.B > 0:
                raise L.MlaError(L.MLA_ERR_ARG, "mla_normal_expanded_bytes")
        self.kv_exp = torch.empty(max(1, nbytes // 2), dtype=torch.bfloat16, device=dev)
        self.o = torch.empty((w.B, w.T, w.H, 128), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((w.B, w.T, w.H), dtype=torch.float32, device=dev)

    def expand(self, stream=None):
        L.check(L.mla_normal_expand(self.geom, self.cache, self.block_table, self.block_table.shape[1], self.seq_lens,
                                    self.w.B, self.w.max_pages, self.w_uk, self.w_uv, self.kv_exp, stream),
                "mla_normal_expand")

    def attention(self, stream=None):
        L.check(L.mla_normal_attention(self.geom, self.batch, self.q_nope, self.q_pe, self.cache, self.block_table,
                                       self.block_table.shape[1], self.seq_lens, self.kv_exp, self.o, self.lse,
                                       stream), "mla_normal_attention")

    def chunked(self, stream=None):
        L.check(L.mla_normal_chunked(self.geom, self.batch, self.q_nope, self.q_pe, self.cache, self.block_table,
                                     self.block_table.shape[1], self.seq_lens, self.w_uk, self.w_uv, self.chunk_rows,
                                     self.kv_exp, self.state, self.o, self.lse, stream), "mla_normal_chunked")

    def step(self, stream=None):
        if self.chunk_rows > 0:
            self.chunked(stream)
            return
        self.expand(stream)
        self.attention(stream)

    def expanded(self):
        """kv_exp viewed as [H, B * rows_per_seq, 256] (k_nope | v)."""
        return self.kv_exp[: self.w.H * self.w.B * self.rows_per_seq * 256].view(
            self.w.H, self.w.B * self.rows_per_seq, 256)
