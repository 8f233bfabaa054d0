"""Device-side state of one wavefront layer: paged K/V pools, page table and descriptor.

PyTorch provides the device memory and the stream; every step of the hot path runs through the
C ABI (:mod:`._abi`).  A pool may be shared by several layers (each with its own page-table row),
which is how the 30-layer round reuses one 4096-page pool.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence

import torch

from . import _abi


class PagedPool:
    """K and V pools, bf16 [num_pages, page_size, H, D] each, on one device."""

    def __init__(self, num_pages: int, page_size: int, heads: int, head_dim: int,
                 device="cuda", fill: Optional[float] = None):
        shape = (num_pages, page_size, heads, head_dim)
        self.k = torch.empty(shape, dtype=torch.bfloat16, device=device)
        self.v = torch.empty(shape, dtype=torch.bfloat16, device=device)
        if fill is not None:
            self.k.fill_(fill)
            self.v.fill_(fill)
        self.num_pages, self.page_size, self.heads, self.head_dim = shape


class PagedPoolFp8:
    """FP8 K/V pool with the geometry of a :class:`PagedPool`: e4m3 codes uint8
    [num_pages, page_size, H, D] and one fp32 scale per (token, head) row [num_pages, page_size, H]
    for K and for V.  Filled by wf_kv_append_fp8, read back by wf_kv_dequant."""

    def __init__(self, num_pages: int, page_size: int, heads: int, head_dim: int,
                 device="cuda"):
        shape = (num_pages, page_size, heads, head_dim)
        self.k_codes = torch.zeros(shape, dtype=torch.uint8, device=device)
        self.v_codes = torch.zeros(shape, dtype=torch.uint8, device=device)
        self.k_scale = torch.zeros(shape[:3], dtype=torch.float32, device=device)
        self.v_scale = torch.zeros(shape[:3], dtype=torch.float32, device=device)
        self.num_pages, self.page_size, self.heads, self.head_dim = shape

    @property
    def tensors(self):
        return self.k_codes, self.v_codes, self.k_scale, self.v_scale


class PagedPoolFp8Block:
    """FP8 cache that attention reads in place (wf_kv_pool_fp8_block_t): e4m3 codes uint8
    [num_pages, page_size, H, D] and e8m0 scales uint8 [num_pages, page_size / 16, H] (a byte b
    stands for 2^(b - 127)) for K and for V, zeroed.  Filled by wf_kv_append_fp8_block, read by
    wf_attn_forward_fp8_block."""

    def __init__(self, num_pages: int, page_size: int, heads: int, head_dim: int,
                 device="cuda"):
        if page_size < 16 or page_size % 16:
            raise ValueError(f"page_size: a positive multiple of 16, got {page_size}")
        shape = (num_pages, page_size, heads, head_dim)
        blocks = (num_pages, page_size // 16, heads)
        self.k_codes = torch.zeros(shape, dtype=torch.uint8, device=device)
        self.v_codes = torch.zeros(shape, dtype=torch.uint8, device=device)
        self.k_scale = torch.zeros(blocks, dtype=torch.uint8, device=device)
        self.v_scale = torch.zeros(blocks, dtype=torch.uint8, device=device)
        self.num_pages, self.page_size, self.heads, self.head_dim = shape

    @property
    def tensors(self):
        return self.k_codes, self.v_codes, self.k_scale, self.v_scale


def rotation_table(rows: int, axis_pairs: Sequence[int], base: float = 10000.0,
                   device="cuda") -> torch.Tensor:
    """The table of a :class:`NormRope`: fp32 [rows, pairs, 2], cos and sin of position times
    base^(-i / n) for pair i of an axis with n pairs, computed in 64 bits (far positions have
    angles that 32 bits cannot hold)."""
    freq = torch.cat([base ** (-torch.arange(n, dtype=torch.float64) / max(n, 1))
                      for n in axis_pairs])
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * freq
    return torch.stack((ang.cos(), ang.sin()), -1).float().to(device).contiguous()


def video_positions(first_token: int, tokens: int, rows: int, cols: int,
                    device="cuda") -> torch.Tensor:
    """int32 [tokens, 3]: frame, row and column of ``tokens`` tokens of a video whose frames are
    rows x cols patches, from ``first_token`` on."""
    t = torch.arange(first_token, first_token + tokens)
    pos = torch.stack((t // (rows * cols), t // cols % rows, t % cols), 1)
    return pos.to(torch.int32).to(device).contiguous()


class QkI8Buffers:
    """The device buffers of the INT8 attention tier for one wavefront shape (see
    ``wf_qk_quantize_i8``): int8 Q and K' codes, their per-128-row scales, the key mean and its
    fp64 scratch."""

    def __init__(self, desc, heads: int, head_dim: int, device="cuda"):
        from . import _abi
        sizes = _abi.qk_i8_sizes(desc, heads, head_dim)
        off = desc.chunk_offsets
        t_kv, t_q = off[-1], off[-1] - off[desc.num_ctx_chunks]
        self.q_codes = torch.empty(t_q, heads, head_dim, dtype=torch.int8, device=device)
        self.q_scale = torch.empty(sizes[1] // 4, dtype=torch.float32, device=device)
        self.k_codes = torch.empty(t_kv, heads, head_dim, dtype=torch.int8, device=device)
        self.k_scale = torch.empty(sizes[3] // 4, dtype=torch.float32, device=device)
        self.k_mean = torch.empty(heads, head_dim, dtype=torch.float32, device=device)
        self.k_sum = torch.empty(heads, head_dim, dtype=torch.float64, device=device)
        self.heads = heads


class QkE4m3Buffers:
    """The device buffers of the FP8 (e4m3) attention tier for one wavefront shape (see
    ``wf_qk_quantize_e4m3``): e4m3 Q and K codes (uint8) and their per-128-row scales."""

    def __init__(self, desc, heads: int, head_dim: int, device="cuda"):
        from . import _abi
        sizes = _abi.qk_e4m3_sizes(desc, heads, head_dim)
        off = desc.chunk_offsets
        t_kv, t_q = off[-1], off[-1] - off[desc.num_ctx_chunks]
        self.q_codes = torch.empty(t_q, heads, head_dim, dtype=torch.uint8, device=device)
        self.q_scale = torch.empty(sizes[1] // 4, dtype=torch.float32, device=device)
        self.k_codes = torch.empty(t_kv, heads, head_dim, dtype=torch.uint8, device=device)
        self.k_scale = torch.empty(sizes[3] // 4, dtype=torch.float32, device=device)
        self.heads = heads


class WavefrontLayer:
    """One layer of a wavefront: its descriptor and its page-table rows.

    ``page_tables`` is int32 [num_layers, max_pages_per_seq] on the device (row ``layer`` is this
    layer's); ``chunk_offsets`` / ``chunk_stage`` / ``num_ctx_chunks`` describe the chunks in
    logical order (context first, then active chunks cleanest to noisiest).
    """

    def __init__(self, pool: PagedPool, page_tables: torch.Tensor, layer: int,
                 chunk_offsets: Sequence[int], chunk_stage: Sequence[int], num_ctx_chunks: int):
        self.pool = pool
        self.page_tables = page_tables
        self.layer = int(layer)
        self.desc = _abi.WavefrontDesc(chunk_offsets, chunk_stage, num_ctx_chunks,
                                       page_tables.shape[1])
        self.chunk_offsets = list(chunk_offsets)
        self.num_ctx_chunks = int(num_ctx_chunks)
        self._workspace: Optional[torch.Tensor] = None   # split-KV partial results
        self._ws_bytes: dict = {}                          # workspace bytes per `splits`

    @property
    def t_q(self) -> int:
        return self.chunk_offsets[-1] - self.chunk_offsets[self.num_ctx_chunks]

    def append(self, chunk: int, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
        _abi.kv_append(self.pool.k, self.pool.v, self.layer, chunk, k, v, self.page_tables,
                       self.desc, stream)

    def append_range(self, k_all: torch.Tensor, v_all: torch.Tensor, chunks: Sequence[int],
                     stream=None) -> None:
        """Append the given chunks, slicing their rows out of logical-order K/V tensors."""
        for c in chunks:
            a, b = self.chunk_offsets[c], self.chunk_offsets[c + 1]
            self.append(c, k_all[a:b], v_all[a:b], stream)

    def append_rope(self, chunk_begin: int, chunk_end: int, k: torch.Tensor, v: torch.Tensor, rule,
                    positions=None, k_weight=None, stream=None) -> None:
        """Append chunks [chunk_begin, chunk_end), keys normed and rotated on the way (``rule``: a
        :class:`NormRope`); ``k``, ``v``: their rows, [L, H, D], slices of a projection's output
        as they are."""
        _abi.kv_append_rope(self.pool.k, self.pool.v, self.layer, chunk_begin, chunk_end, k, v,
                            self.page_tables, self.desc, rule, positions, k_weight, stream)

    def forward_i8(self, q: torch.Tensor, out: torch.Tensor, qk: "QkI8Buffers",
                   scale: Optional[float] = None, lse: Optional[torch.Tensor] = None,
                   stream=None) -> None:
        """The INT8 tier: quantize q and this layer's keys into ``qk``, then attend."""
        from . import _abi
        if scale is None:
            scale = 1.0 / math.sqrt(self.pool.head_dim)
        row = self.page_tables[self.layer]
        _abi.qk_quantize_i8(q, self.pool.k, self.pool.v, row, self.desc, qk, stream)
        _abi.attn_forward_i8(qk, self.pool.k, self.pool.v, row, self.desc, scale, out, lse,
                             stream)

    def forward_e4m3(self, q: torch.Tensor, out: torch.Tensor, qk: "QkE4m3Buffers",
                     scale: Optional[float] = None, lse: Optional[torch.Tensor] = None,
                     stream=None) -> None:
        """The FP8 tier: quantize q and this layer's keys into ``qk`` as e4m3, then attend."""
        from . import _abi
        if scale is None:
            scale = 1.0 / math.sqrt(self.pool.head_dim)
        row = self.page_tables[self.layer]
        _abi.qk_quantize_e4m3(q, self.pool.k, self.pool.v, row, self.desc, qk, stream)
        _abi.attn_forward_e4m3(qk, self.pool.k, self.pool.v, row, self.desc, scale, out, lse,
                               stream)

    def forward(self, q: torch.Tensor, out: torch.Tensor, scale: Optional[float] = None,
                lse: Optional[torch.Tensor] = None, stream=None,
                splits: Optional[int] = None) -> None:
        """Attention of ``q`` over this layer's pages.  ``splits`` None: wf_attn_forward; an int:
        wf_attn_forward_split with that many key splits (0: the library's choice), with a
        workspace this layer allocates once and reuses."""
        if scale is None:
            scale = 1.0 / math.sqrt(self.pool.head_dim)
        if splits is None:
            _abi.attn_forward(q, self.pool.k, self.pool.v, self.page_tables[self.layer],
                              self.desc, scale, out, lse, stream)
            return
        need = self._ws_bytes.get(splits)
        if need is None:
            need = _abi.attn_workspace_size(self.desc, self.pool.heads, self.pool.head_dim,
                                            splits)
            self._ws_bytes[splits] = need
        ws = None
        if need > 0:
            if self._workspace is None or self._workspace.numel() < need:
                self._workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
            ws = self._workspace
        _abi.attn_forward_split(q, self.pool.k, self.pool.v, self.page_tables[self.layer],
                                self.desc, scale, out, splits, ws, lse, stream)


def _scratch(kept: dict, need: int, device, stream) -> torch.Tensor:
    """Workspace of ``need`` bytes for a call on ``stream`` (None: the current one).

    ``kept`` holds one for each stream, whose calls follow one another; it grows, and a smaller one
    is given back to the allocator of its own stream.  A call that is being captured gets one of its
    own from the graph's memory, so that graphs share none with one another or with other calls.
    """
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(getattr(stream, "cuda_stream", stream), device)
        with torch.cuda.stream(stream):
            return _scratch(kept, need, device, None)
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(need, dtype=torch.uint8, device=device)
    key = torch.cuda.current_stream(device).cuda_stream, device
    ws = kept.get(key)
    if ws is None or ws.numel() < need:
        ws = kept[key] = torch.empty(need, dtype=torch.uint8, device=device)
    return ws


class Fp8BlockLayer:
    """One layer of a wavefront over an FP8 cache that attention reads in place.

    ``pool``: a :class:`PagedPoolFp8Block`, which several layers may share; the other arguments as
    for :class:`WavefrontLayer`.  Query heads may be a multiple of the pool's heads.
    """

    def __init__(self, pool: PagedPoolFp8Block, page_tables: torch.Tensor, layer: int,
                 chunk_offsets: Sequence[int], chunk_stage: Sequence[int], num_ctx_chunks: int):
        self.pool = pool
        self.page_tables = page_tables
        self.layer = int(layer)
        self.desc = _abi.WavefrontDesc(chunk_offsets, chunk_stage, num_ctx_chunks,
                                       page_tables.shape[1])
        off = self.chunk_offsets = list(chunk_offsets)
        first = off[num_ctx_chunks]
        self.segments = _abi.Segments([e - first for e in off[num_ctx_chunks + 1:]],
                                      off[num_ctx_chunks + 1:], off[-1], page_tables.shape[1])
        self._workspaces: dict = {}

    def append(self, chunk_begin: int, chunk_end: int, k: torch.Tensor, v: torch.Tensor, rule=None,
               positions=None, k_weight=None, stream=None) -> None:
        """Append chunks [chunk_begin, chunk_end) (``k``, ``v``: their rows, [L, H, D] bf16), keys
        normed and rotated on the way when ``rule`` is given."""
        _abi.kv_append_fp8_block(*self.pool.tensors, self.layer, chunk_begin, chunk_end, k, v,
                                 self.page_tables, self.desc, rule, positions, k_weight, stream)

    def workspace_size(self, q_heads: int, segments=None, splits: int = 0) -> int:
        return _abi.attn_fp8_block_workspace_size(segments or self.segments, q_heads,
                                                  self.pool.heads, self.pool.head_dim, splits)

    def forward(self, q: torch.Tensor, out: torch.Tensor, scale: Optional[float] = None,
                lse: Optional[torch.Tensor] = None, splits: int = 0,
                workspace: Optional[torch.Tensor] = None, segments=None, stream=None) -> None:
        """Attention of ``q`` over this layer's cache: the wavefront's query chunks, each up to its
        own end, or the rows of ``segments``.  Without ``workspace`` the layer keeps one for each
        stream, and a captured call has its own."""
        if scale is None:
            scale = 1.0 / math.sqrt(self.pool.head_dim)
        seg = segments or self.segments
        if workspace is None:
            need = self.workspace_size(q.shape[1], seg, splits)
            if need > 0:
                workspace = _scratch(self._workspaces, need, q.device, stream)
        _abi.attn_forward_fp8_block(q, *self.pool.tensors, self.page_tables[self.layer], seg, scale,
                                    out, lse, splits, workspace, stream)
