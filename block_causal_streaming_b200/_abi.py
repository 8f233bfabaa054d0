"""ctypes binding of ``libwf_b200.so`` (the C ABI in ``include/wf.h``).

Argument marshalling only: every step of append and attention runs in the library's kernels.
There is no CPU fallback; if the library is missing, importing the binding raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
# WF_B200_LIB points the binding at another build of the same library (e.g. a tuning variant).
LIB_PATH = os.environ.get("WF_B200_LIB") or os.path.join(HERE, "libwf_b200.so")

WF_OK = 0
WF_ERR_INVALID_ARG = 1
WF_ERR_SHAPE = 2
WF_ERR_STAGE_ORDER = 3
WF_ERR_CAPACITY = 4
WF_ERR_PAGE_OOB = 5
WF_ERR_TIMEOUT = 6
WF_ERR_CUDA = 7
WF_ERR_NO_DEVICE = 8
WF_ERR_POSITION = 9
WF_MAX_CHUNKS = 64

# Every symbol include/wf.h declares (checked by the CPU tests).
EXPORTED = ("wf_kv_append", "wf_attn_forward", "wf_check_status", "wf_strerror", "wf_version",
            "wf_selftest_timeout", "wf_attn_forward_split", "wf_attn_workspace_size",
            "wf_attn_forward_split_noalloc", "wf_kv_append_publish", "wf_attn_forward_published",
            "wf_ipc_export", "wf_ipc_import", "wf_ipc_close", "wf_kv_append_fp8",
            "wf_kv_dequant", "wf_kv_append_fp8_chunks", "wf_kv_dequant_chunks",
            "wf_attn_split_plan", "wf_qk_e4m3_sizes", "wf_qk_quantize_e4m3",
            "wf_attn_forward_e4m3", "wf_kv_append_publish_fp8", "wf_kv_dequant_published",
            "wf_qk_i8_sizes", "wf_qk_quantize_i8", "wf_attn_forward_i8",
            "wf_attn_forward_segments", "wf_attn_segments_workspace_size",
            "wf_window_slots", "wf_window_round", "wf_window_round_ring", "wf_qk_norm_rope",
            "wf_kv_append_rope", "wf_kv_append_fp8_block", "wf_attn_forward_fp8_block",
            "wf_attn_fp8_block_workspace_size")


class WfError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {strerror(code)}")


class PoolDst(ctypes.Structure):
    """wf_pool_dst_t: a destination pool (usually another GPU's, mapped by ipc_import)."""
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("flags", ctypes.c_void_p)]


class Fp8Dst(ctypes.Structure):
    """wf_fp8_dst_t: a destination FP8 pool (usually another GPU's, mapped by ipc_import)."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("flags", ctypes.c_void_p)]


class QkI8(ctypes.Structure):
    """wf_qk_i8_t: the quantized Q and K' of the INT8 tier (device pointers)."""
    _fields_ = [("q_codes", ctypes.c_void_p), ("q_scale", ctypes.c_void_p),
                ("k_codes", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("k_mean", ctypes.c_void_p), ("k_sum", ctypes.c_void_p)]


class QkE4m3(ctypes.Structure):
    """wf_qk_e4m3_t: the e4m3 Q and K of the FP8 tier (device pointers)."""
    _fields_ = [("q_codes", ctypes.c_void_p), ("q_scale", ctypes.c_void_p),
                ("k_codes", ctypes.c_void_p), ("k_scale", ctypes.c_void_p)]


class KvPool(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class KvPoolFp8(ctypes.Structure):
    """wf_kv_pool_fp8_t: e4m3 codes [pages, page_size, H, D] and fp32 scales [pages, page_size, H]."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class KvPoolFp8Block(ctypes.Structure):
    """wf_kv_pool_fp8_block_t: e4m3 codes [pages, page_size, H, D] and e8m0 scales
    [pages, page_size / 16, H]."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class NormRopeC(ctypes.Structure):
    """wf_norm_rope_t."""
    _fields_ = [("norm", ctypes.c_int32), ("eps", ctypes.c_float),
                ("weight_per_head", ctypes.c_int32), ("cos_sin", ctypes.c_void_p),
                ("table_rows", ctypes.c_int32), ("num_axes", ctypes.c_int32),
                ("axis_pairs", ctypes.c_int32 * 3), ("interleaved", ctypes.c_int32)]


class WindowC(ctypes.Structure):
    """wf_window_t."""
    _fields_ = [("chunk_len", ctypes.c_int32), ("num_stages", ctypes.c_int32),
                ("stages", ctypes.POINTER(ctypes.c_int32)), ("history", ctypes.c_int32)]


class RoundC(ctypes.Structure):
    """wf_round_t."""
    _fields_ = [("round", ctypes.c_int64), ("num_chunks", ctypes.c_int32),
                ("num_ctx_chunks", ctypes.c_int32), ("chunk_id", ctypes.c_int64 * 64),
                ("role", ctypes.c_int32 * 64), ("chunk_stage", ctypes.c_int32 * 64),
                ("chunk_offsets", ctypes.c_int32 * 65), ("store_to", ctypes.c_int32),
                ("evicted", ctypes.c_int64), ("store_kv_end", ctypes.c_int32)]


class SegmentsC(ctypes.Structure):
    """wf_segments_t."""
    _fields_ = [("num_segments", ctypes.c_int32),
                ("rows_end", ctypes.POINTER(ctypes.c_int32)),
                ("kv_end", ctypes.POINTER(ctypes.c_int32)),
                ("num_keys", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32)]


class Wavefront(ctypes.Structure):
    _fields_ = [("num_chunks", ctypes.c_int32), ("num_ctx_chunks", ctypes.c_int32),
                ("chunk_offsets", ctypes.POINTER(ctypes.c_int32)),
                ("chunk_stage", ctypes.POINTER(ctypes.c_int32)),
                ("max_pages_per_seq", ctypes.c_int32)]


def _load(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -m block_causal_streaming_b200.build` (nvcc, sm_100a)")
    lib = ctypes.CDLL(path)
    vp, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.wf_kv_append.argtypes = [ctypes.POINTER(KvPool), i32, i32, vp, vp,
                                 ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(Wavefront), vp]
    lib.wf_kv_append.restype = i32
    lib.wf_attn_forward.argtypes = [vp, ctypes.POINTER(KvPool), ctypes.POINTER(ctypes.c_int32),
                                    ctypes.POINTER(Wavefront), f32, vp,
                                    ctypes.POINTER(ctypes.c_float), vp]
    lib.wf_attn_forward.restype = i32
    lib.wf_check_status.argtypes = [vp]
    lib.wf_check_status.restype = i32
    lib.wf_strerror.argtypes = [i32]
    lib.wf_strerror.restype = ctypes.c_char_p
    lib.wf_version.argtypes = []
    lib.wf_version.restype = i32
    lib.wf_selftest_timeout.argtypes = [ctypes.c_uint, vp]
    lib.wf_selftest_timeout.restype = i32
    lib.wf_attn_forward_split.argtypes = [vp, ctypes.POINTER(KvPool),
                                          ctypes.POINTER(ctypes.c_int32),
                                          ctypes.POINTER(Wavefront), ctypes.c_float, vp,
                                          ctypes.POINTER(ctypes.c_float), i32, vp,
                                          ctypes.c_size_t, vp]
    lib.wf_attn_forward_split.restype = i32
    lib.wf_attn_forward_split_noalloc.argtypes = [vp, ctypes.POINTER(KvPool),
                                                  ctypes.POINTER(ctypes.c_int32),
                                                  ctypes.POINTER(Wavefront), ctypes.c_float, vp,
                                                  ctypes.POINTER(ctypes.c_float), i32, vp]
    lib.wf_attn_forward_split_noalloc.restype = i32
    lib.wf_kv_append_publish.argtypes = [ctypes.POINTER(KvPool), vp, ctypes.POINTER(PoolDst),
                                         i32, i32, i32, vp, vp, ctypes.POINTER(ctypes.c_int32),
                                         ctypes.POINTER(Wavefront), ctypes.c_uint32, vp]
    lib.wf_kv_append_publish.restype = i32
    lib.wf_attn_forward_published.argtypes = [vp, ctypes.POINTER(KvPool),
                                              ctypes.POINTER(ctypes.c_int32),
                                              ctypes.POINTER(Wavefront), ctypes.c_float, vp,
                                              ctypes.POINTER(ctypes.c_float), vp,
                                              ctypes.c_uint32, i32, vp, ctypes.c_size_t, vp]
    lib.wf_attn_forward_published.restype = i32
    lib.wf_ipc_export.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_size_t)]
    lib.wf_ipc_export.restype = i32
    lib.wf_ipc_import.argtypes = [vp, ctypes.c_size_t, ctypes.POINTER(ctypes.c_void_p)]
    lib.wf_ipc_import.restype = i32
    lib.wf_ipc_close.argtypes = [vp]
    lib.wf_ipc_close.restype = i32
    lib.wf_attn_workspace_size.argtypes = [ctypes.POINTER(Wavefront), i32, i32, i32]
    lib.wf_attn_workspace_size.restype = ctypes.c_size_t
    lib.wf_attn_split_plan.argtypes = [ctypes.POINTER(Wavefront), i32, i32, i32,
                                       ctypes.POINTER(ctypes.c_int32),
                                       ctypes.POINTER(ctypes.c_int32)]
    lib.wf_attn_split_plan.restype = i32
    lib.wf_kv_append_fp8.argtypes = [ctypes.POINTER(KvPoolFp8), i32, i32, vp, vp,
                                     ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(Wavefront), vp]
    lib.wf_kv_append_fp8.restype = i32
    lib.wf_kv_dequant.argtypes = [ctypes.POINTER(KvPoolFp8), ctypes.POINTER(KvPool), i32, i32,
                                  ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(Wavefront), vp]
    lib.wf_kv_dequant.restype = i32
    lib.wf_kv_append_fp8_chunks.argtypes = [ctypes.POINTER(KvPoolFp8), i32, i32, i32, vp, vp,
                                            ctypes.POINTER(ctypes.c_int32),
                                            ctypes.POINTER(Wavefront), vp]
    lib.wf_kv_append_fp8_chunks.restype = i32
    lib.wf_kv_dequant_chunks.argtypes = [ctypes.POINTER(KvPoolFp8), ctypes.POINTER(KvPool), i32,
                                         i32, i32, ctypes.POINTER(ctypes.c_int32),
                                         ctypes.POINTER(Wavefront), vp]
    lib.wf_kv_dequant_chunks.restype = i32
    lib.wf_kv_append_publish_fp8.argtypes = [ctypes.POINTER(KvPoolFp8), vp,
                                             ctypes.POINTER(Fp8Dst), i32, i32, i32, vp, vp,
                                             ctypes.POINTER(ctypes.c_int32),
                                             ctypes.POINTER(Wavefront), ctypes.c_uint32, vp]
    lib.wf_kv_append_publish_fp8.restype = i32
    lib.wf_kv_dequant_published.argtypes = [ctypes.POINTER(KvPoolFp8), ctypes.POINTER(KvPool),
                                            i32, i32, ctypes.POINTER(ctypes.c_int32),
                                            ctypes.POINTER(Wavefront), vp, ctypes.c_uint32, vp]
    lib.wf_kv_dequant_published.restype = i32
    lib.wf_qk_i8_sizes.argtypes = [ctypes.POINTER(Wavefront), i32, i32,
                                   ctypes.POINTER(ctypes.c_size_t)]
    lib.wf_qk_i8_sizes.restype = i32
    lib.wf_qk_quantize_i8.argtypes = [vp, ctypes.POINTER(KvPool), ctypes.POINTER(ctypes.c_int32),
                                      ctypes.POINTER(Wavefront), ctypes.POINTER(QkI8), vp]
    lib.wf_qk_quantize_i8.restype = i32
    lib.wf_attn_forward_i8.argtypes = [ctypes.POINTER(QkI8), ctypes.POINTER(KvPool),
                                       ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(Wavefront),
                                       f32, vp, ctypes.POINTER(ctypes.c_float), vp]
    lib.wf_attn_forward_i8.restype = i32
    lib.wf_qk_e4m3_sizes.argtypes = [ctypes.POINTER(Wavefront), i32, i32,
                                     ctypes.POINTER(ctypes.c_size_t)]
    lib.wf_qk_e4m3_sizes.restype = i32
    lib.wf_qk_quantize_e4m3.argtypes = [vp, ctypes.POINTER(KvPool),
                                        ctypes.POINTER(ctypes.c_int32),
                                        ctypes.POINTER(Wavefront), ctypes.POINTER(QkE4m3), vp]
    lib.wf_qk_quantize_e4m3.restype = i32
    lib.wf_attn_forward_e4m3.argtypes = [ctypes.POINTER(QkE4m3), ctypes.POINTER(KvPool),
                                         ctypes.POINTER(ctypes.c_int32),
                                         ctypes.POINTER(Wavefront), f32, vp,
                                         ctypes.POINTER(ctypes.c_float), vp]
    lib.wf_attn_forward_e4m3.restype = i32
    lib.wf_window_slots.argtypes = [ctypes.POINTER(WindowC), ctypes.POINTER(ctypes.c_int32),
                                    ctypes.POINTER(ctypes.c_int64)]
    lib.wf_window_slots.restype = i32
    lib.wf_window_round.argtypes = [ctypes.POINTER(WindowC), ctypes.c_int64,
                                    ctypes.POINTER(RoundC)]
    lib.wf_window_round.restype = i32
    lib.wf_window_round_ring.argtypes = [ctypes.POINTER(WindowC), ctypes.c_int64,
                                         ctypes.POINTER(RoundC)]
    lib.wf_window_round_ring.restype = i32
    lib.wf_attn_forward_segments.argtypes = [vp, ctypes.POINTER(KvPool),
                                             ctypes.POINTER(ctypes.c_int32),
                                             ctypes.POINTER(SegmentsC), f32, vp,
                                             ctypes.POINTER(ctypes.c_float), i32, vp,
                                             ctypes.c_size_t, vp]
    lib.wf_attn_forward_segments.restype = i32
    lib.wf_attn_segments_workspace_size.argtypes = [ctypes.POINTER(SegmentsC), i32, i32, i32]
    lib.wf_attn_segments_workspace_size.restype = ctypes.c_size_t
    i64 = ctypes.c_int64
    lib.wf_qk_norm_rope.argtypes = [vp, i64, vp, vp, i32, vp, i64, vp, vp, i32, i32, i32, vp,
                                    ctypes.POINTER(NormRopeC), vp]
    lib.wf_qk_norm_rope.restype = i32
    lib.wf_kv_append_rope.argtypes = [ctypes.POINTER(KvPool), i32, i32, i32, vp, i64, vp, i64, vp,
                                      vp, ctypes.POINTER(NormRopeC), vp,
                                      ctypes.POINTER(Wavefront), vp]
    lib.wf_kv_append_rope.restype = i32
    lib.wf_kv_append_fp8_block.argtypes = [ctypes.POINTER(KvPoolFp8Block), i32, i32, i32, vp, i64,
                                           vp, i64, vp, vp, ctypes.POINTER(NormRopeC), vp,
                                           ctypes.POINTER(Wavefront), vp]
    lib.wf_kv_append_fp8_block.restype = i32
    lib.wf_attn_forward_fp8_block.argtypes = [vp, i32, ctypes.POINTER(KvPoolFp8Block), vp,
                                              ctypes.POINTER(SegmentsC), f32, vp, vp, i32, vp,
                                              ctypes.c_size_t, vp]
    lib.wf_attn_forward_fp8_block.restype = i32
    lib.wf_attn_fp8_block_workspace_size.argtypes = [ctypes.POINTER(SegmentsC), i32, i32, i32, i32]
    lib.wf_attn_fp8_block_workspace_size.restype = ctypes.c_size_t
    return lib


lib = _load()


def strerror(code: int) -> str:
    return lib.wf_strerror(int(code)).decode()


class WavefrontDesc:
    """Host copy of a wavefront descriptor; keeps the arrays alive while C reads them."""

    def __init__(self, chunk_offsets: Sequence[int], chunk_stage: Sequence[int],
                 num_ctx_chunks: int, max_pages_per_seq: int):
        n = len(chunk_offsets) - 1
        self._off = (ctypes.c_int32 * (n + 1))(*[int(x) for x in chunk_offsets])
        self._stage = (ctypes.c_int32 * max(n, 1))(*[int(x) for x in chunk_stage])
        self.c = Wavefront(n, int(num_ctx_chunks),
                           ctypes.cast(self._off, ctypes.POINTER(ctypes.c_int32)),
                           ctypes.cast(self._stage, ctypes.POINTER(ctypes.c_int32)),
                           int(max_pages_per_seq))
        self.ref = ctypes.byref(self.c)
        self.chunk_offsets = [int(x) for x in chunk_offsets]
        self.num_ctx_chunks = int(num_ctx_chunks)


def _pool_struct(k_pool, v_pool) -> KvPool:
    num_pages, page_size, H, D = (int(x) for x in k_pool.shape)
    return KvPool(k_pool.data_ptr(), v_pool.data_ptr(), num_pages, page_size, H, D)


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


# ---- shapes.  The C ABI takes plain pointers and cannot see a buffer's size, so these checks
# are what keeps a wrongly shaped tensor from being read or written past its end on the device.
def _pool_shape(k_pool, v_pool, what: str = "pool"):
    if k_pool.dim() != 4 or tuple(v_pool.shape) != tuple(k_pool.shape):
        raise ValueError(f"{what}: K and V must both be [num_pages, page_size, H, D], got "
                         f"{tuple(k_pool.shape)} and {tuple(v_pool.shape)}")
    return tuple(int(x) for x in k_pool.shape)


def _check_chunk_rows(wf: "WavefrontDesc", chunk: int, k, v, H: int, D: int):
    off = wf.chunk_offsets
    if not 0 <= int(chunk) < len(off) - 1:
        return                                     # the library answers WF_ERR_INVALID_ARG
    want = (off[chunk + 1] - off[chunk], H, D)
    for t, n in ((k, "k"), (v, "v")):
        if tuple(t.shape) != want and not (want[0] == 0 and t.numel() == 0):
            raise ValueError(f"{n}: chunk {chunk} needs [{want[0]}, {H}, {D}], got {tuple(t.shape)}")


def _check_page_table(page_table, layer: int, wf: "WavefrontDesc"):
    if page_table.dim() != 2 or page_table.shape[1] != wf.c.max_pages_per_seq:
        raise ValueError(f"page_table: expected [num_layers, {wf.c.max_pages_per_seq}], got "
                         f"{tuple(page_table.shape)}")
    if not 0 <= int(layer) < page_table.shape[0]:
        raise ValueError(f"layer {layer} outside the page table's {page_table.shape[0]} rows")


def _check_page_table_row(row, wf: "WavefrontDesc"):
    if row.dim() != 1 or row.shape[0] < wf.c.max_pages_per_seq:
        raise ValueError(f"page_table_row: expected [{wf.c.max_pages_per_seq}], got "
                         f"{tuple(row.shape)}")


def _check_queries(q, out, lse, wf: "WavefrontDesc", H: int, D: int):
    off = wf.chunk_offsets
    t_q = off[-1] - off[wf.num_ctx_chunks] if 0 <= wf.num_ctx_chunks < len(off) else None
    if t_q is None:
        return                                     # the library answers WF_ERR_SHAPE
    if tuple(q.shape) != (t_q, H, D):
        raise ValueError(f"q: expected [{t_q}, {H}, {D}] (the query chunks' rows), got "
                         f"{tuple(q.shape)}")
    if tuple(out.shape) != tuple(q.shape):
        raise ValueError(f"out: expected {tuple(q.shape)}, got {tuple(out.shape)}")
    if lse is not None and tuple(lse.shape) != (H, t_q):
        raise ValueError(f"lse: expected [{H}, {t_q}], got {tuple(lse.shape)}")


def _check_tensor(t, name: str, dtype_name: str):
    import torch
    want = {"bf16": (torch.bfloat16,), "i32": (torch.int32,), "f32": (torch.float32,),
            "u8": (torch.uint8,), "i8": (torch.int8,), "f64": (torch.float64,),
            "u32": (torch.int32, torch.uint32)}[dtype_name]      # flag words: any 32-bit int
    if t.dtype not in want:
        raise TypeError(f"{name}: expected {want[0]}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")


def _check_qk_buffers(qk, fields, sizes):
    """Every buffer of an 8-bit tier's qk holds at least the bytes the library's sizes call
    gives for this wavefront (the quantize call writes them all, the attention call reads them)."""
    get = (lambda n: qk[n]) if isinstance(qk, dict) else (lambda n: getattr(qk, n))
    for n, sz in zip(fields, sizes):
        t = get(n)
        if t.numel() * t.element_size() < sz:
            raise ValueError(f"{n}: {t.numel() * t.element_size()} bytes, needs {sz}")


class Window:
    """Host copy of a wf_window_t; keeps the stage array alive while C reads it."""

    def __init__(self, chunk_len: int, stages: Sequence[int], history: int):
        self._stages = (ctypes.c_int32 * max(len(stages), 1))(*[int(s) for s in stages])
        self.c = WindowC(int(chunk_len), len(stages),
                         ctypes.cast(self._stages, ctypes.POINTER(ctypes.c_int32)), int(history))


def window_slots(window: Window):
    """wf_window_slots: (slots, tokens) of one layer of the window."""
    slots, tokens = ctypes.c_int32(), ctypes.c_int64()
    rc = lib.wf_window_slots(ctypes.byref(window.c), ctypes.byref(slots), ctypes.byref(tokens))
    if rc != WF_OK:
        raise WfError(rc, "wf_window_slots")
    return slots.value, tokens.value


def window_round(window: Window, round_index: int, ring: bool = False) -> RoundC:
    """wf_window_round (or, with ring, wf_window_round_ring): the plan of one round."""
    out = RoundC()
    fn = lib.wf_window_round_ring if ring else lib.wf_window_round
    rc = fn(ctypes.byref(window.c), int(round_index), ctypes.byref(out))
    if rc != WF_OK:
        raise WfError(rc, "wf_window_round_ring" if ring else "wf_window_round")
    return out


class Segments:
    """Host copy of a wf_segments_t; keeps the arrays alive while C reads them."""

    def __init__(self, rows_end: Sequence[int], kv_end: Sequence[int], num_keys: int,
                 max_pages_per_seq: int):
        n = len(rows_end)
        if n != len(kv_end):
            raise ValueError("rows_end and kv_end need one entry per segment")
        self._rows = (ctypes.c_int32 * max(n, 1))(*[int(x) for x in rows_end])
        self._kv = (ctypes.c_int32 * max(n, 1))(*[int(x) for x in kv_end])
        self.c = SegmentsC(n, ctypes.cast(self._rows, ctypes.POINTER(ctypes.c_int32)),
                           ctypes.cast(self._kv, ctypes.POINTER(ctypes.c_int32)),
                           int(num_keys), int(max_pages_per_seq))
        self.ref = ctypes.byref(self.c)
        self.rows_end = [int(x) for x in rows_end]
        self.kv_end = [int(x) for x in kv_end]
        self.num_keys = int(num_keys)

    @property
    def t_q(self) -> int:
        return self.rows_end[-1] if self.rows_end else 0


def attn_segments_workspace_size(seg: Segments, num_heads: int, head_dim: int,
                                 splits: int = 0) -> int:
    return int(lib.wf_attn_segments_workspace_size(ctypes.byref(seg.c), int(num_heads),
                                                   int(head_dim), int(splits)))


def attn_forward_segments(q, k_pool, v_pool, page_table_row, seg: Segments, scale: float, out,
                          lse=None, splits: int = 1, workspace=None, stream=None) -> None:
    """wf_attn_forward_segments: rows of segment i see logical keys [0, kv_end[i])."""
    _, page_size, H, D = _pool_shape(k_pool, v_pool)
    t_q = seg.t_q
    if tuple(q.shape) != (t_q, H, D) or tuple(out.shape) != (t_q, H, D):
        raise ValueError(f"q, out: expected [{t_q}, {H}, {D}], got {tuple(q.shape)}, "
                         f"{tuple(out.shape)}")
    if lse is not None and tuple(lse.shape) != (H, t_q):
        raise ValueError(f"lse: expected [{H}, {t_q}], got {tuple(lse.shape)}")
    if page_table_row.dim() != 1 or page_table_row.numel() < seg.c.max_pages_per_seq:
        raise ValueError(f"page_table_row: needs {seg.c.max_pages_per_seq} entries")
    for t, n, d in ((q, "q", "bf16"), (out, "out", "bf16"), (k_pool, "k_pool", "bf16"),
                    (v_pool, "v_pool", "bf16"), (page_table_row, "page_table_row", "i32")):
        _check_tensor(t, n, d)
    if lse is not None:
        _check_tensor(lse, "lse", "f32")
    need = attn_segments_workspace_size(seg, H, D, splits)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        raise ValueError(f"workspace: {need} bytes needed for {splits} key splits")
    pool = _pool_struct(k_pool, v_pool)
    rc = lib.wf_attn_forward_segments(
        q.data_ptr(), ctypes.byref(pool),
        ctypes.cast(ctypes.c_void_p(page_table_row.data_ptr()), ctypes.POINTER(ctypes.c_int32)),
        ctypes.byref(seg.c), float(scale), out.data_ptr(),
        ctypes.cast(ctypes.c_void_p(lse.data_ptr()), ctypes.POINTER(ctypes.c_float))
        if lse is not None else None,
        int(splits), workspace.data_ptr() if workspace is not None else None,
        workspace.numel() * workspace.element_size() if workspace is not None else 0,
        _stream_handle(stream))
    if rc != WF_OK:
        raise WfError(rc, "wf_attn_forward_segments")


def kv_append(k_pool, v_pool, layer: int, chunk: int, k, v, page_table, wf: WavefrontDesc,
              stream=None) -> None:
    """wf_kv_append: write chunk ``chunk``'s K/V ([L, H, D] bf16) into the pools' pages using row
    ``layer`` of ``page_table`` ([num_layers, max_pages_per_seq] int32, on the device)."""
    _, _, H, D = _pool_shape(k_pool, v_pool)
    _check_chunk_rows(wf, chunk, k, v, H, D)
    _check_page_table(page_table, layer, wf)
    for t, n, d in ((k_pool, "k_pool", "bf16"), (v_pool, "v_pool", "bf16"), (k, "k", "bf16"),
                    (v, "v", "bf16"), (page_table, "page_table", "i32")):
        _check_tensor(t, n, d)
    pool = _pool_struct(k_pool, v_pool)
    rc = lib.wf_kv_append(ctypes.byref(pool), int(layer), int(chunk), k.data_ptr(), v.data_ptr(),
                          ctypes.cast(ctypes.c_void_p(page_table.data_ptr()),
                                      ctypes.POINTER(ctypes.c_int32)),
                          ctypes.byref(wf.c), _stream_handle(stream))
    if rc != WF_OK:
        raise WfError(rc, "wf_kv_append")


def _fp8_pool_shape(k_codes, v_codes, k_scale, v_scale):
    num_pages, page_size, H, D = _pool_shape(k_codes, v_codes, "FP8 pool codes")
    if tuple(k_scale.shape) != (num_pages, page_size, H) or \
            tuple(v_scale.shape) != (num_pages, page_size, H):
        raise ValueError("FP8 pool: codes [pages, page_size, H, D] and scales [pages, page_size, H]")
    return num_pages, page_size, H, D


def _fp8_pool_struct(k_codes, v_codes, k_scale, v_scale) -> KvPoolFp8:
    num_pages, page_size, H, D = _fp8_pool_shape(k_codes, v_codes, k_scale, v_scale)
    for t, n, d in ((k_codes, "k_codes", "u8"), (v_codes, "v_codes", "u8"),
                    (k_scale, "k_scale", "f32"), (v_scale, "v_scale", "f32")):
        _check_tensor(t, n, d)
    return KvPoolFp8(k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(),
                     v_scale.data_ptr(), num_pages, page_size, H, D)


def kv_append_fp8(k_codes, v_codes, k_scale, v_scale, layer: int, chunk: int, k, v, page_table,
                  wf: WavefrontDesc, stream=None) -> None:
    """wf_kv_append_fp8: quantize chunk ``chunk``'s K/V ([L, H, D] bf16) to e4m3 codes with one
    fp32 scale per (token, head) row, into an FP8 pool through row ``layer`` of ``page_table``."""
    _, _, H, D = _fp8_pool_shape(k_codes, v_codes, k_scale, v_scale)
    _check_chunk_rows(wf, chunk, k, v, H, D)
    _check_page_table(page_table, layer, wf)
    for t, n, d in ((k, "k", "bf16"), (v, "v", "bf16"), (page_table, "page_table", "i32")):
        _check_tensor(t, n, d)
    pool = _fp8_pool_struct(k_codes, v_codes, k_scale, v_scale)
    rc = lib.wf_kv_append_fp8(ctypes.byref(pool), int(layer), int(chunk), k.data_ptr(),
                              v.data_ptr(), ctypes.cast(ctypes.c_void_p(page_table.data_ptr()),
                                                        ctypes.POINTER(ctypes.c_int32)),
                              ctypes.byref(wf.c), _stream_handle(stream))
    if rc != WF_OK:
        raise WfError(rc, "wf_kv_append_fp8")


def kv_dequant(k_codes, v_codes, k_scale, v_scale, k_pool, v_pool, layer: int, chunk: int,
               page_table, wf: WavefrontDesc, stream=None) -> None:
    """wf_kv_dequant: chunk ``chunk`` of an FP8 pool -> the same rows of a bf16 pool."""
    geo = _fp8_pool_shape(k_codes, v_codes, k_scale, v_scale)
    if _pool_shape(k_pool, v_pool) != geo:
        raise ValueError(f"bf16 pool {tuple(k_pool.shape)} differs from the FP8 pool {geo}")
    _check_page_table(page_table, layer, wf)
    for t, n, d in ((k_pool, "k_pool", "bf16"), (v_pool, "v_pool", "bf16"),
                    (page_table, "page_table", "i32")):
        _check_tensor(t, n, d)
    src = _fp8_pool_struct(k_codes, v_codes, k_scale, v_scale)
    dst = _pool_struct(k_pool, v_pool)
    rc = lib.wf_kv_dequant(ctypes.byref(src), ctypes.byref(dst), int(layer), int(chunk),
                           ctypes.cast(ctypes.c_void_p(page_table.data_ptr()),
                                       ctypes.POINTER(ctypes.c_int32)),
                           ctypes.byref(wf.c), _stream_handle(stream))
    if rc != WF_OK:
        raise WfError(rc, "wf_kv_dequant")


def kv_append_fp8_chunks(k_codes, v_codes, k_scale, v_scale, layer: int, chunk_begin: int,
                         chunk_end: int, k, v, page_table, wf: WavefrontDesc, stream=None) -> None:
    """wf_kv_append_fp8_chunks: kv_append_fp8 of chunks [chunk_begin, chunk_end) in one launch;
    ``k``, ``v``: those chunks' rows in order, [L, H, D] bf16."""
    _, _, H, D = _fp8_pool_shape(k_codes, v_codes, k_scale, v_scale)
    off = wf.chunk_offsets
    if 0 <= int(chunk_begin) < int(chunk_end) <= len(off) - 1:
        want = (off[chunk_end] - off[chunk_begin], H, D)
        for t, n in ((k, "k"), (v, "v")):
            if tuple(t.shape) != want and not (want[0] == 0 and t.numel() == 0):
                raise ValueError(f"{n}: chunks [{chunk_begin}, {chunk_end}) need "
                                 f"[{want[0]}, {H}, {D}], got {tuple(t.shape)}")
    _check_page_table(page_table, layer, wf)
    for t, n, d in ((k, "k", "bf16"), (v, "v", "bf16"), (page_table, "page_table", "i32")):
        _check_tensor(t, n, d)
    pool = _fp8_pool_struct(k_codes, v_codes, k_scale, v_scale)
    rc = lib.wf_kv_append_fp8_chunks(ctypes.byref(pool), int(layer), int(chunk_begin),
                                     int(chunk_end), k.data_ptr(), v.data_ptr(),
                                     ctypes.cast(ctypes.c_void_p(page_table.data_ptr()),
                                                 ctypes.POINTER(ctypes.c_int32)),
                                     ctypes.byref(wf.c), _stream_handle(stream))
    if rc != WF_OK:
        raise WfError(rc, "wf_kv_append_fp8_chunks")


def kv_dequant_chunks(k_codes, v_codes, k_scale, v_scale, k_pool, v_pool, layer: int,
                      chunk_begin: int, chunk_end: int, page_table, wf: WavefrontDesc,
                      stream=None) -> None:
    """wf_kv_dequant_chunks: kv_dequant of chunks [chunk_begin, chunk_end) in one launch."""
    geo = _fp8_pool_shape(k_codes, v_codes, k_scale, v_scale)
    if _pool_shape(k_pool, v_pool) != geo:
        raise ValueError(f"bf16 pool {tuple(k_pool.shape)} differs from the FP8 pool {geo}")
    _check_page_table(page_table, layer, wf)
    for t, n, d in ((k_pool, "k_pool", "bf16"), (v_pool, "v_pool", "bf16"),
                    (page_table, "page_table", "i32")):
        _check_tensor(t, n, d)
    src = _fp8_pool_struct(k_codes, v_codes, k_scale, v_scale)
    dst = _pool_struct(k_pool, v_pool)
    rc = lib.wf_kv_dequant_chunks(ctypes.byref(src), ctypes.byref(dst), int(layer),
                                  int(chunk_begin), int(chunk_end),
                                  ctypes.cast(ctypes.c_void_p(page_table.data_ptr()),
                                              ctypes.POINTER(ctypes.c_int32)),
                                  ctypes.byref(wf.c), _stream_handle(stream))
    if rc != WF_OK:
        raise WfError(rc, "wf_kv_dequant_chunks")


def kv_append_publish_fp8(k_codes, v_codes, k_scale, v_scale, flags, peers, layer: int,
                          chunk: int, k, v, page_table, wf: WavefrontDesc, generation: int,
                          stream=None) -> None:
    """wf_kv_append_publish_fp8: quantize one chunk into this FP8 pool and every peer FP8 pool,
    then raise the chunk's flag to ``generation`` here (``flags``: device uint32
    [layers, WF_MAX_CHUNKS] or None) and in every peer.  ``peers``: sequence of
    (k_codes_ptr, v_codes_ptr, k_scale_ptr, v_scale_ptr, flags_ptr)."""
    _, _, H, D = _fp8_pool_shape(k_codes, v_codes, k_scale, v_scale)
    _check_chunk_rows(wf, chunk, k, v, H, D)
    _check_page_table(page_table, layer, wf)
    if flags is not None and flags.numel() < (int(layer) + 1) * WF_MAX_CHUNKS:
        raise ValueError(f"flags: layer {layer} needs [>= {int(layer) + 1}, {WF_MAX_CHUNKS}] words, "
                         f"got {tuple(flags.shape)}")
    _check_tensor(page_table, "page_table", "i32")
    if k.numel() > 0:
        _check_tensor(k, "k", "bf16")
        _check_tensor(v, "v", "bf16")
    if flags is not None:
        _check_tensor(flags, "flags", "u32")
    arr = (Fp8Dst * max(1, len(peers)))(*[Fp8Dst(int(a), int(b), int(c), int(d),
                                                 int(f) if f else None)
                                          for a, b, c, d, f in peers])
    pool = _fp8_pool_struct(k_codes, v_codes, k_scale, v_scale)
    rc = lib.wf_kv_append_publish_fp8(
        ctypes.byref(pool), flags.data_ptr() if flags is not None else None, arr, len(peers),
        int(layer), int(chunk), k.data_ptr() if k.numel() else None,
        v.data_ptr() if v.numel() else None,
        ctypes.cast(ctypes.c_void_p(page_table.data_ptr()), ctypes.POINTER(ctypes.c_int32)),
        ctypes.byref(wf.c), int(generation) & 0xFFFFFFFF, _stream_handle(stream))
    if rc != WF_OK:
        raise WfError(rc, "wf_kv_append_publish_fp8")


def kv_dequant_published(k_codes, v_codes, k_scale, v_scale, k_pool, v_pool, layer: int,
                         chunk: int, page_table, wf: WavefrontDesc, flags_row, generation: int,
                         stream=None) -> None:
    """wf_kv_dequant_published: kv_dequant that first waits for ``flags_row[chunk]`` (device
    uint32 [WF_MAX_CHUNKS]) to reach ``generation``."""
    geo = _fp8_pool_shape(k_codes, v_codes, k_scale, v_scale)
    if _pool_shape(k_pool, v_pool) != geo:
        raise ValueError(f"bf16 pool {tuple(k_pool.shape)} differs from the FP8 pool {geo}")
    _check_page_table(page_table, layer, wf)
    if flags_row.numel() < len(wf.chunk_offsets) - 1:
        raise ValueError(f"flags_row: needs >= {len(wf.chunk_offsets) - 1} words")
    for t, n, d in ((k_pool, "k_pool", "bf16"), (v_pool, "v_pool", "bf16"),
                    (page_table, "page_table", "i32"), (flags_row, "flags_row", "u32")):
        _check_tensor(t, n, d)
    src = _fp8_pool_struct(k_codes, v_codes, k_scale, v_scale)
    dst = _pool_struct(k_pool, v_pool)
    rc = lib.wf_kv_dequant_published(ctypes.byref(src), ctypes.byref(dst), int(layer),
                                     int(chunk),
                                     ctypes.cast(ctypes.c_void_p(page_table.data_ptr()),
                                                 ctypes.POINTER(ctypes.c_int32)),
                                     ctypes.byref(wf.c), flags_row.data_ptr(),
                                     int(generation) & 0xFFFFFFFF, _stream_handle(stream))
    if rc != WF_OK:
        raise WfError(rc, "wf_kv_dequant_published")


QK_I8_FIELDS = ("q_codes", "q_scale", "k_codes", "k_scale", "k_mean", "k_sum")


def qk_i8_sizes(wf: WavefrontDesc, num_heads: int, head_dim: int):
    """wf_qk_i8_sizes: byte sizes of the six buffers of the INT8 tier, in QK_I8_FIELDS order."""
    sizes = (ctypes.c_size_t * 6)()
    rc = lib.wf_qk_i8_sizes(ctypes.byref(wf.c), int(num_heads), int(head_dim), sizes)
    if rc != WF_OK:
        raise WfError(rc, "wf_qk_i8_sizes")
    return [int(x) for x in sizes]


def _qk_struct(qk) -> QkI8:
    """qk: a mapping / object with the six QK_I8_FIELDS device tensors."""
    get = (lambda n: qk[n]) if isinstance(qk, dict) else (lambda n: getattr(qk, n))
    for n, d in zip(QK_I8_FIELDS, ("i8", "f32", "i8", "f32", "f32", "f64")):
        _check_tensor(get(n), n, d)
    return QkI8(*[get(n).data_ptr() for n in QK_I8_FIELDS])


def qk_quantize_i8(q, k_pool, v_pool, page_table_row, wf: WavefrontDesc, qk,
                   stream=None) -> None:
    """wf_qk_quantize_i8: int8 Q (from q) and K' (from the K pool) with their scales into qk."""
    _, _, H, D = _pool_shape(k_pool, v_pool)
    _check_queries(q, q, None, wf, H, D)
    _check_page_table_row(page_table_row, wf)
    _check_qk_buffers(qk, QK_I8_FIELDS, qk_i8_sizes(wf, H, D))
    for t, n, d in ((q, "q", "bf16"), (k_pool, "k_pool", "bf16"),
                    (page_table_row, "page_table_row", "i32")):
        _check_tensor(t, n, d)
    pool = _pool_struct(k_pool, v_pool)
    s = _qk_struct(qk)
    rc = lib.wf_qk_quantize_i8(q.data_ptr(), ctypes.byref(pool),
                               ctypes.cast(ctypes.c_void_p(page_table_row.data_ptr()),
                                           ctypes.POINTER(ctypes.c_int32)),
                               ctypes.byref(wf.c), ctypes.byref(s), _stream_handle(stream))
    if rc != WF_OK:
        raise WfError(rc, "wf_qk_quantize_i8")


def attn_forward_i8(qk, k_pool, v_pool, page_table_row, wf: WavefrontDesc, scale: float, out,
                    lse=None, stream=None) -> None:
    """wf_attn_forward_i8: block-causal attention on the quantized Q / K' of qk, V from v_pool."""
    _, _, H, D = _pool_shape(k_pool, v_pool)
    _check_queries(out, out, lse, wf, H, D)
    _check_page_table_row(page_table_row, wf)
    _check_qk_buffers(qk, QK_I8_FIELDS, qk_i8_sizes(wf, H, D))
    for t, n, d in ((out, "out", "bf16"), (v_pool, "v_pool", "bf16"),
                    (page_table_row, "page_table_row", "i32")):
        _check_tensor(t, n, d)
    if lse is not None:
        _check_tensor(lse, "lse", "f32")
    pool = _pool_struct(k_pool, v_pool)
    s = _qk_struct(qk)
    rc = lib.wf_attn_forward_i8(ctypes.byref(s), ctypes.byref(pool),
                                ctypes.cast(ctypes.c_void_p(page_table_row.data_ptr()),
                                            ctypes.POINTER(ctypes.c_int32)),
                                ctypes.byref(wf.c), float(scale), out.data_ptr(),
                                ctypes.cast(ctypes.c_void_p(lse.data_ptr()),
                                            ctypes.POINTER(ctypes.c_float))
                                if lse is not None else None,
                                _stream_handle(stream))
    if rc != WF_OK:
        raise WfError(rc, "wf_attn_forward_i8")


QK_E4M3_FIELDS = ("q_codes", "q_scale", "k_codes", "k_scale")


def qk_e4m3_sizes(wf: WavefrontDesc, num_heads: int, head_dim: int):
    """wf_qk_e4m3_sizes: byte sizes of the four buffers of the FP8 tier, in QK_E4M3_FIELDS
    order."""
    sizes = (ctypes.c_size_t * 4)()
    rc = lib.wf_qk_e4m3_sizes(ctypes.byref(wf.c), int(num_heads), int(head_dim), sizes)
    if rc != WF_OK:
        raise WfError(rc, "wf_qk_e4m3_sizes")
    return [int(x) for x in sizes]


def _qk_e4m3_struct(qk) -> QkE4m3:
    """qk: a mapping / object with the four QK_E4M3_FIELDS device tensors (codes uint8)."""
    get = (lambda n: qk[n]) if isinstance(qk, dict) else (lambda n: getattr(qk, n))
    for n, d in zip(QK_E4M3_FIELDS, ("u8", "f32", "u8", "f32")):
        _check_tensor(get(n), n, d)
    return QkE4m3(*[get(n).data_ptr() for n in QK_E4M3_FIELDS])


def qk_quantize_e4m3(q, k_pool, v_pool, page_table_row, wf: WavefrontDesc, qk,
                     stream=None) -> None:
    """wf_qk_quantize_e4m3: e4m3 Q (from q) and K (from the K pool) with their scales into qk."""
    _, _, H, D = _pool_shape(k_pool, v_pool)
    _check_queries(q, q, None, wf, H, D)
    _check_page_table_row(page_table_row, wf)
    _check_qk_buffers(qk, QK_E4M3_FIELDS, qk_e4m3_sizes(wf, H, D))
    for t, n, d in ((q, "q", "bf16"), (k_pool, "k_pool", "bf16"),
                    (page_table_row, "page_table_row", "i32")):
        _check_tensor(t, n, d)
    pool = _pool_struct(k_pool, v_pool)
    s = _qk_e4m3_struct(qk)
    rc = lib.wf_qk_quantize_e4m3(q.data_ptr(), ctypes.byref(pool),
                                 ctypes.cast(ctypes.c_void_p(page_table_row.data_ptr()),
                                             ctypes.POINTER(ctypes.c_int32)),
                                 ctypes.byref(wf.c), ctypes.byref(s), _stream_handle(stream))
    if rc != WF_OK:
        raise WfError(rc, "wf_qk_quantize_e4m3")


def attn_forward_e4m3(qk, k_pool, v_pool, page_table_row, wf: WavefrontDesc, scale: float, out,
                      lse=None, stream=None) -> None:
    """wf_attn_forward_e4m3: block-causal attention on the e4m3 Q / K of qk, V from v_pool."""
    _, _, H, D = _pool_shape(k_pool, v_pool)
    _check_queries(out, out, lse, wf, H, D)
    _check_page_table_row(page_table_row, wf)
    _check_qk_buffers(qk, QK_E4M3_FIELDS, qk_e4m3_sizes(wf, H, D))
    for t, n, d in ((out, "out", "bf16"), (v_pool, "v_pool", "bf16"),
                    (page_table_row, "page_table_row", "i32")):
        _check_tensor(t, n, d)
    if lse is not None:
        _check_tensor(lse, "lse", "f32")
    pool = _pool_struct(k_pool, v_pool)
    s = _qk_e4m3_struct(qk)
    rc = lib.wf_attn_forward_e4m3(ctypes.byref(s), ctypes.byref(pool),
                                  ctypes.cast(ctypes.c_void_p(page_table_row.data_ptr()),
                                              ctypes.POINTER(ctypes.c_int32)),
                                  ctypes.byref(wf.c), float(scale), out.data_ptr(),
                                  ctypes.cast(ctypes.c_void_p(lse.data_ptr()),
                                              ctypes.POINTER(ctypes.c_float))
                                  if lse is not None else None,
                                  _stream_handle(stream))
    if rc != WF_OK:
        raise WfError(rc, "wf_attn_forward_e4m3")


def attn_forward(q, k_pool, v_pool, page_table_row, wf: WavefrontDesc, scale: float, out,
                 lse=None, stream=None) -> None:
    """wf_attn_forward: block-causal chunk attention of q ([T_q, H, D] bf16) over the paged K/V
    of one layer (``page_table_row``: [max_pages_per_seq] int32 on the device) into ``out``."""
    _, _, H, D = _pool_shape(k_pool, v_pool)
    _check_queries(q, out, lse, wf, H, D)
    _check_page_table_row(page_table_row, wf)
    for t, n, d in ((q, "q", "bf16"), (k_pool, "k_pool", "bf16"), (v_pool, "v_pool", "bf16"),
                    (page_table_row, "page_table_row", "i32"), (out, "out", "bf16")):
        _check_tensor(t, n, d)
    if lse is not None:
        _check_tensor(lse, "lse", "f32")
    pool = _pool_struct(k_pool, v_pool)
    rc = lib.wf_attn_forward(
        q.data_ptr(), ctypes.byref(pool),
        ctypes.cast(ctypes.c_void_p(page_table_row.data_ptr()), ctypes.POINTER(ctypes.c_int32)),
        ctypes.byref(wf.c), float(scale), out.data_ptr(),
        ctypes.cast(ctypes.c_void_p(lse.data_ptr()), ctypes.POINTER(ctypes.c_float))
        if lse is not None else None,
        _stream_handle(stream))
    if rc != WF_OK:
        raise WfError(rc, "wf_attn_forward")


def attn_workspace_size(wf: WavefrontDesc, num_heads: int, head_dim: int, splits: int = 0) -> int:
    """wf_attn_workspace_size: bytes of workspace attn_forward_split needs (0: none)."""
    return int(lib.wf_attn_workspace_size(ctypes.byref(wf.c), int(num_heads), int(head_dim),
                                          int(splits)))


def attn_split_plan(wf: WavefrontDesc, num_heads: int, splits: int = 0, num_sms: int = 0):
    """wf_attn_split_plan: (parts, tail_units) -- every unit in ``parts`` parts, the last
    ``tail_units`` units of the dispatch order in parts + 1.  ``num_sms`` 0: the current device."""
    parts, tail = ctypes.c_int32(0), ctypes.c_int32(0)
    rc = lib.wf_attn_split_plan(ctypes.byref(wf.c), int(num_heads), int(splits), int(num_sms),
                                ctypes.byref(parts), ctypes.byref(tail))
    if rc != WF_OK:
        raise WfError(rc, "wf_attn_split_plan")
    return parts.value, tail.value


def attn_forward_split(q, k_pool, v_pool, page_table_row, wf: WavefrontDesc, scale: float, out,
                       splits: int = 0, workspace=None, lse=None, stream=None) -> None:
    """wf_attn_forward_split: attn_forward with every unit's keys split over ``splits`` CTAs
    (0: the library chooses) and merged; ``workspace`` is a device uint8 tensor of at least
    attn_workspace_size(...) bytes (None when that is 0)."""
    _, _, H, D = _pool_shape(k_pool, v_pool)
    _check_queries(q, out, lse, wf, H, D)
    _check_page_table_row(page_table_row, wf)
    for t, n, d in ((q, "q", "bf16"), (k_pool, "k_pool", "bf16"), (v_pool, "v_pool", "bf16"),
                    (page_table_row, "page_table_row", "i32"), (out, "out", "bf16")):
        _check_tensor(t, n, d)
    if lse is not None:
        _check_tensor(lse, "lse", "f32")
    pool = _pool_struct(k_pool, v_pool)
    rc = lib.wf_attn_forward_split(
        q.data_ptr(), ctypes.byref(pool),
        ctypes.cast(ctypes.c_void_p(page_table_row.data_ptr()), ctypes.POINTER(ctypes.c_int32)),
        ctypes.byref(wf.c), float(scale), out.data_ptr(),
        ctypes.cast(ctypes.c_void_p(lse.data_ptr()), ctypes.POINTER(ctypes.c_float))
        if lse is not None else None,
        int(splits), workspace.data_ptr() if workspace is not None else None,
        workspace.numel() * workspace.element_size() if workspace is not None else 0,
        _stream_handle(stream))
    if rc != WF_OK:
        raise WfError(rc, "wf_attn_forward_split")


def attn_forward_split_noalloc(q, k_pool, v_pool, page_table_row, wf: WavefrontDesc,
                               scale: float, out, splits: int = 0, lse=None, stream=None) -> None:
    """wf_attn_forward_split_noalloc: attn_forward_split with the library's static scratch
    instead of a workspace (calls on one device must be ordered on one stream)."""
    _, _, H, D = _pool_shape(k_pool, v_pool)
    _check_queries(q, out, lse, wf, H, D)
    _check_page_table_row(page_table_row, wf)
    for t, n, d in ((q, "q", "bf16"), (k_pool, "k_pool", "bf16"), (v_pool, "v_pool", "bf16"),
                    (page_table_row, "page_table_row", "i32"), (out, "out", "bf16")):
        _check_tensor(t, n, d)
    if lse is not None:
        _check_tensor(lse, "lse", "f32")
    pool = _pool_struct(k_pool, v_pool)
    rc = lib.wf_attn_forward_split_noalloc(
        q.data_ptr(), ctypes.byref(pool),
        ctypes.cast(ctypes.c_void_p(page_table_row.data_ptr()), ctypes.POINTER(ctypes.c_int32)),
        ctypes.byref(wf.c), float(scale), out.data_ptr(),
        ctypes.cast(ctypes.c_void_p(lse.data_ptr()), ctypes.POINTER(ctypes.c_float))
        if lse is not None else None,
        int(splits), _stream_handle(stream))
    if rc != WF_OK:
        raise WfError(rc, "wf_attn_forward_split_noalloc")


def kv_append_publish(k_pool, v_pool, flags, peers, layer: int, chunk: int, k, v, page_table,
                      wf: WavefrontDesc, generation: int, stream=None) -> None:
    """wf_kv_append_publish: append one chunk into this pool and every peer pool, then raise the
    chunk's flag to ``generation`` here (``flags``: device uint32 [layers, WF_MAX_CHUNKS] or
    None) and in every peer.  ``peers``: sequence of (k_pool_ptr, v_pool_ptr, flags_ptr)."""
    _, _, H, D = _pool_shape(k_pool, v_pool)
    _check_chunk_rows(wf, chunk, k, v, H, D)
    _check_page_table(page_table, layer, wf)
    if flags is not None and flags.numel() < (int(layer) + 1) * WF_MAX_CHUNKS:
        raise ValueError(f"flags: layer {layer} needs [>= {int(layer) + 1}, {WF_MAX_CHUNKS}] words, "
                         f"got {tuple(flags.shape)}")
    for t, n, d in ((k_pool, "k_pool", "bf16"), (v_pool, "v_pool", "bf16"),
                    (page_table, "page_table", "i32")):
        _check_tensor(t, n, d)
    if k.numel() > 0:
        _check_tensor(k, "k", "bf16")
        _check_tensor(v, "v", "bf16")
    if flags is not None:
        _check_tensor(flags, "flags", "u32")
    arr = (PoolDst * max(1, len(peers)))(*[PoolDst(int(a), int(b), int(c) if c else None)
                                          for a, b, c in peers])
    pool = _pool_struct(k_pool, v_pool)
    rc = lib.wf_kv_append_publish(
        ctypes.byref(pool), flags.data_ptr() if flags is not None else None, arr, len(peers),
        int(layer), int(chunk), k.data_ptr() if k.numel() else None,
        v.data_ptr() if v.numel() else None,
        ctypes.cast(ctypes.c_void_p(page_table.data_ptr()), ctypes.POINTER(ctypes.c_int32)),
        ctypes.byref(wf.c), int(generation) & 0xFFFFFFFF, _stream_handle(stream))
    if rc != WF_OK:
        raise WfError(rc, "wf_kv_append_publish")


def attn_forward_published(q, k_pool, v_pool, page_table_row, wf: WavefrontDesc, scale: float,
                           out, flags_row, generation: int, splits: int = 0, workspace=None,
                           lse=None, stream=None) -> None:
    """wf_attn_forward_published: attn_forward_split that waits, chunk by chunk, for the
    publication flags in ``flags_row`` (device uint32 [WF_MAX_CHUNKS]) to reach ``generation``."""
    _, _, H, D = _pool_shape(k_pool, v_pool)
    _check_queries(q, out, lse, wf, H, D)
    _check_page_table_row(page_table_row, wf)
    if flags_row.numel() < len(wf.chunk_offsets) - 1:
        raise ValueError(f"flags_row: one word per chunk needed, got {tuple(flags_row.shape)}")
    for t, n, d in ((q, "q", "bf16"), (k_pool, "k_pool", "bf16"), (v_pool, "v_pool", "bf16"),
                    (page_table_row, "page_table_row", "i32"), (out, "out", "bf16"),
                    (flags_row, "flags_row", "u32")):
        _check_tensor(t, n, d)
    if lse is not None:
        _check_tensor(lse, "lse", "f32")
    pool = _pool_struct(k_pool, v_pool)
    rc = lib.wf_attn_forward_published(
        q.data_ptr(), ctypes.byref(pool),
        ctypes.cast(ctypes.c_void_p(page_table_row.data_ptr()), ctypes.POINTER(ctypes.c_int32)),
        ctypes.byref(wf.c), float(scale), out.data_ptr(),
        ctypes.cast(ctypes.c_void_p(lse.data_ptr()), ctypes.POINTER(ctypes.c_float))
        if lse is not None else None,
        flags_row.data_ptr(), int(generation) & 0xFFFFFFFF, int(splits),
        workspace.data_ptr() if workspace is not None else None,
        workspace.numel() * workspace.element_size() if workspace is not None else 0,
        _stream_handle(stream))
    if rc != WF_OK:
        raise WfError(rc, "wf_attn_forward_published")


# ---- norm and rotation of queries and keys, and the appends that carry them
class NormRope:
    """A wf_norm_rope_t: RMS norm of every (token, head) row and the rotation by position.

    ``table``: fp32 [rows, pairs, 2] on the device (cos, sin of every position and pair, see
    :func:`layer.rotation_table`), or None for no rotation; kept alive here.  ``axis_pairs``: pairs
    that turn with each axis of the position (default: all with one axis)."""

    def __init__(self, table=None, axis_pairs: Optional[Sequence[int]] = None,
                 interleaved: bool = False, norm: bool = True, eps: float = 1e-6,
                 weight_per_head: bool = False):
        self.table, self.norm, self.weight_per_head = table, bool(norm), bool(weight_per_head)
        self.num_axes = self.pairs = 0
        rows = 0
        if table is not None:
            if table.dim() != 3 or table.shape[2] != 2:
                raise ValueError(f"table: expected [rows, pairs, 2], got {tuple(table.shape)}")
            _check_tensor(table, "table", "f32")
            rows, self.pairs = int(table.shape[0]), int(table.shape[1])
            axis_pairs = [self.pairs] if axis_pairs is None else [int(x) for x in axis_pairs]
            if not 1 <= len(axis_pairs) <= 3 or sum(axis_pairs) != self.pairs or \
                    min(axis_pairs) < 0:
                raise ValueError(f"axis_pairs: 1 to 3 counts that sum to the table's {self.pairs} "
                                 f"pairs, got {axis_pairs}")
            self.num_axes = len(axis_pairs)
        ap = (ctypes.c_int32 * 3)(*(list(axis_pairs) + [0, 0])[:3]) if table is not None else \
            (ctypes.c_int32 * 3)()
        self.c = NormRopeC(int(self.norm), float(eps), int(self.weight_per_head),
                           table.data_ptr() if table is not None else None, rows, self.num_axes,
                           ap, int(bool(interleaved)))
        self.ref = ctypes.byref(self.c)


# A call for one token is a few microseconds on the device, so these checks read every attribute of
# a tensor once and build nothing they do not pass on.
_torch = None


def _lib_torch():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _current_device() -> int:
    return _lib_torch()._C._cuda_getDevice()


def _raw_stream(stream, device: int):
    """Handle of ``stream``, or of the current stream of the current device."""
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(device)
    return getattr(stream, "cuda_stream", stream)


def _ptr(t, name: str, dtype, device: int) -> int:
    """Address of a contiguous tensor of ``dtype`` on the device the launch goes to."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name}: expected a tensor on the current CUDA device ({device}), got one "
                         f"on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


def _rows_arg(t, name: str, L: int, H: int, D: int, device: int):
    """(address, token stride) of a bf16 [L, H, D] tensor whose heads lie together."""
    if t.shape != (L, H, D):
        raise ValueError(f"{name}: expected [{L}, {H}, {D}], got {tuple(t.shape)}")
    if t.dtype is not _torch.bfloat16:
        raise TypeError(f"{name}: expected torch.bfloat16, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name}: expected a tensor on the current CUDA device ({device}), got one "
                         f"on {t.device}")
    if L == 0 or H == 0:
        return None, H * D
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != D and H > 1):
        raise ValueError(f"{name}: every token's [{H}, {D}] must be contiguous, strides "
                         f"{t.stride()}")
    if L == 1:
        return t.data_ptr(), H * D
    if s0 < H * D or s0 % 8:
        raise ValueError(f"{name}: the stride from token to token must be a multiple of 8 and at "
                         f"least {H * D}, got {s0}")
    return t.data_ptr(), s0


def _weight_arg(w, name: str, rule: Optional[NormRope], H: int, D: int, device: int):
    if w is None:
        return None
    if rule is None or not rule.norm:
        raise ValueError(f"{name}: a weight without a norm")
    if w.shape != ((H, D) if rule.weight_per_head else (D,)):
        raise ValueError(f"{name}: expected {[H, D] if rule.weight_per_head else [D]}, got "
                         f"{tuple(w.shape)}")
    return _ptr(w, name, _torch.bfloat16, device)


def _positions_arg(positions, rule: Optional[NormRope], L: int, D: int, device: int):
    if rule is None or rule.table is None:
        if positions is not None:
            raise ValueError("positions: the rule has no rotation")
        return None
    if rule.pairs * 2 > D:
        raise ValueError(f"table: {rule.pairs} pairs in rows of {D} values")
    if rule.table.get_device() != device:
        raise ValueError(f"table: on {rule.table.device}, the current CUDA device is {device}")
    if positions is None or positions.shape != (L, rule.num_axes):
        raise ValueError(f"positions: expected [{L}, {rule.num_axes}], got "
                         f"{None if positions is None else tuple(positions.shape)}")
    return _ptr(positions, "positions", _torch.int32, device)


def qk_norm_rope(q, q_out, k, k_out, rule: NormRope, positions=None, q_weight=None,
                 k_weight=None, stream=None) -> None:
    """wf_qk_norm_rope: norm and rotation of ``q`` ([T, Hq, D] bf16, tokens may be strided) into
    ``q_out`` and, in the same launch, of ``k`` into ``k_out`` (both None: queries only).
    ``positions``: int32 [T, axes].  The outputs are contiguous; an output may be its own input."""
    device = _current_device()
    if len(q.shape) != 3:
        raise ValueError(f"q: expected [T, H, D], got {tuple(q.shape)}")
    L, Hq, D = q.shape
    qp, qs = _rows_arg(q, "q", L, Hq, D, device)
    if q_out.shape != q.shape:
        raise ValueError(f"q_out: expected [{L}, {Hq}, {D}], got {tuple(q_out.shape)}")
    qo = _ptr(q_out, "q_out", _torch.bfloat16, device)
    Hk, kp, ks, ko = 0, None, 0, None
    if k is not None:
        if k_out is None or len(k.shape) != 3 or k_out.shape != k.shape:
            raise ValueError(f"k, k_out: expected the same [{L}, H, {D}], got {tuple(k.shape)} and "
                             f"{None if k_out is None else tuple(k_out.shape)}")
        Hk = k.shape[1]
        kp, ks = _rows_arg(k, "k", L, Hk, D, device)
        ko = _ptr(k_out, "k_out", _torch.bfloat16, device)
    elif k_out is not None:
        raise ValueError("k_out without k")
    if L > 0 and Hq > 0:
        # [begin, end) of every tensor's memory: an output may meet nothing but its own input, and
        # that only where it is the same contiguous rows
        qe, qoe = qp + 2 * ((L - 1) * qs + Hq * D), qo + 2 * L * Hq * D
        if qo < qe and qp < qoe and not (qo == qp and qs == Hq * D):
            raise ValueError("q_out overlaps q")
        if Hk > 0:
            ke, koe = kp + 2 * ((L - 1) * ks + Hk * D), ko + 2 * L * Hk * D
            if ko < ke and kp < koe and not (ko == kp and ks == Hk * D):
                raise ValueError("k_out overlaps k")
            if (qo < ke and kp < qoe) or (ko < qe and qp < koe) or (qo < koe and ko < qoe):
                raise ValueError("q_out or k_out overlaps the other's rows")
    qw = _weight_arg(q_weight, "q_weight", rule, Hq, D, device)
    kw = _weight_arg(k_weight, "k_weight", rule, Hk, D, device)
    pp = _positions_arg(positions, rule, L, D, device)
    rc = lib.wf_qk_norm_rope(qp, qs, qo, qw, Hq, kp, ks, ko, kw, Hk, L, D, pp, rule.ref,
                             _raw_stream(stream, device))
    if rc != WF_OK:
        raise WfError(rc, "wf_qk_norm_rope")


def _append_len(chunk_begin: int, chunk_end: int, wf: WavefrontDesc) -> int:
    off = wf.chunk_offsets
    if not 0 <= chunk_begin < chunk_end < len(off):
        raise ValueError(f"chunks [{chunk_begin}, {chunk_end}) outside the wavefront's "
                         f"{len(off) - 1}")
    return off[chunk_end] - off[chunk_begin]


def _page_table_arg(page_table, layer: int, wf: WavefrontDesc, device: int):
    if len(page_table.shape) != 2 or page_table.shape[1] != wf.c.max_pages_per_seq:
        raise ValueError(f"page_table: expected [num_layers, {wf.c.max_pages_per_seq}], got "
                         f"{tuple(page_table.shape)}")
    if not 0 <= layer < page_table.shape[0]:
        raise ValueError(f"layer {layer} outside the page table's {page_table.shape[0]} rows")
    return _ptr(page_table, "page_table", _torch.int32, device)


def kv_append_rope(k_pool, v_pool, layer: int, chunk_begin: int, chunk_end: int, k, v, page_table,
                   wf: WavefrontDesc, rule: NormRope, positions=None, k_weight=None,
                   stream=None) -> None:
    """wf_kv_append_rope: chunks [chunk_begin, chunk_end) into the bf16 pools, keys normed and
    rotated on the way.  ``k``, ``v``: those chunks' rows, [L, H, D] bf16, tokens may be strided."""
    device = _current_device()
    if len(k_pool.shape) != 4 or v_pool.shape != k_pool.shape:
        raise ValueError("pool: K and V must both be [num_pages, page_size, H, D], got "
                         f"{tuple(k_pool.shape)} and {tuple(v_pool.shape)}")
    num_pages, page_size, H, D = k_pool.shape
    L = _append_len(chunk_begin, chunk_end, wf)
    kp, ks = _rows_arg(k, "k", L, H, D, device)
    vp, vs = _rows_arg(v, "v", L, H, D, device)
    pool = KvPool(_ptr(k_pool, "k_pool", _torch.bfloat16, device),
                  _ptr(v_pool, "v_pool", _torch.bfloat16, device), num_pages, page_size, H, D)
    pt = _page_table_arg(page_table, layer, wf, device)
    kw = _weight_arg(k_weight, "k_weight", rule, H, D, device)
    pp = _positions_arg(positions, rule, L, D, device)
    rc = lib.wf_kv_append_rope(ctypes.byref(pool), layer, chunk_begin, chunk_end, kp, ks, vp, vs,
                               kw, pp, rule.ref, pt, wf.ref, _raw_stream(stream, device))
    if rc != WF_OK:
        raise WfError(rc, "wf_kv_append_rope")


def _fp8_block_pool(k_codes, v_codes, k_scale, v_scale, device: int) -> KvPoolFp8Block:
    if len(k_codes.shape) != 4 or v_codes.shape != k_codes.shape:
        raise ValueError("FP8 cache: K and V codes must both be [num_pages, page_size, H, D], got "
                         f"{tuple(k_codes.shape)} and {tuple(v_codes.shape)}")
    num_pages, page_size, H, D = k_codes.shape
    want = (num_pages, page_size // 16, H)
    if k_scale.shape != want or v_scale.shape != want:
        raise ValueError(f"FP8 cache: scales must be {list(want)} (pages, page_size / 16, H), got "
                         f"{tuple(k_scale.shape)} and {tuple(v_scale.shape)}")
    u8 = _torch.uint8
    return KvPoolFp8Block(_ptr(k_codes, "k_codes", u8, device), _ptr(v_codes, "v_codes", u8, device),
                          _ptr(k_scale, "k_scale", u8, device), _ptr(v_scale, "v_scale", u8, device),
                          num_pages, page_size, H, D)


def kv_append_fp8_block(k_codes, v_codes, k_scale, v_scale, layer: int, chunk_begin: int,
                        chunk_end: int, k, v, page_table, wf: WavefrontDesc,
                        rule: Optional[NormRope] = None, positions=None, k_weight=None,
                        stream=None) -> None:
    """wf_kv_append_fp8_block: chunks [chunk_begin, chunk_end) into an FP8 cache (uint8 e4m3 codes
    [pages, page_size, H, D], uint8 e8m0 scales [pages, page_size / 16, H]; zeroed at first), keys
    normed and rotated on the way when ``rule`` is given."""
    device = _current_device()
    pool = _fp8_block_pool(k_codes, v_codes, k_scale, v_scale, device)
    H, D = pool.num_heads, pool.head_dim
    L = _append_len(chunk_begin, chunk_end, wf)
    kp, ks = _rows_arg(k, "k", L, H, D, device)
    vp, vs = _rows_arg(v, "v", L, H, D, device)
    pt = _page_table_arg(page_table, layer, wf, device)
    kw = _weight_arg(k_weight, "k_weight", rule, H, D, device)
    pp = _positions_arg(positions, rule, L, D, device)
    rc = lib.wf_kv_append_fp8_block(ctypes.byref(pool), layer, chunk_begin, chunk_end, kp, ks, vp,
                                    vs, kw, pp, rule.ref if rule is not None else None, pt,
                                    wf.ref, _raw_stream(stream, device))
    if rc != WF_OK:
        raise WfError(rc, "wf_kv_append_fp8_block")


def attn_fp8_block_workspace_size(seg: Segments, num_q_heads: int, num_kv_heads: int,
                                  head_dim: int, splits: int = 0) -> int:
    """wf_attn_fp8_block_workspace_size: bytes of workspace attn_forward_fp8_block needs (0: none)."""
    return int(lib.wf_attn_fp8_block_workspace_size(ctypes.byref(seg.c), int(num_q_heads),
                                                    int(num_kv_heads), int(head_dim),
                                                    int(splits)))


def attn_forward_fp8_block(q, k_codes, v_codes, k_scale, v_scale, page_table_row, seg: Segments,
                           scale: float, out, lse=None, splits: int = 0, workspace=None,
                           stream=None) -> None:
    """wf_attn_forward_fp8_block: rows of segment i of ``q`` ([T, Hq, D] bf16) see logical keys
    [0, kv_end[i]) of an FP8 cache (see :func:`kv_append_fp8_block`) whose H heads each serve
    Hq / H query heads; ``lse``: fp32 [Hq, T]."""
    device = _current_device()
    pool = _fp8_block_pool(k_codes, v_codes, k_scale, v_scale, device)
    t_q = seg.t_q
    if len(q.shape) != 3 or q.shape[0] != t_q or q.shape[2] != pool.head_dim or \
            q.shape[1] % max(pool.num_heads, 1) or q.shape[1] == 0:
        raise ValueError(f"q: expected [{t_q}, a multiple of {pool.num_heads}, {pool.head_dim}], "
                         f"got {tuple(q.shape)}")
    if out.shape != q.shape:
        raise ValueError(f"out: expected {tuple(q.shape)}, got {tuple(out.shape)}")
    Hq = q.shape[1]
    if len(page_table_row.shape) != 1 or page_table_row.shape[0] < seg.c.max_pages_per_seq:
        raise ValueError(f"page_table_row: needs {seg.c.max_pages_per_seq} entries")
    if lse is not None and lse.shape != (Hq, t_q):
        raise ValueError(f"lse: expected [{Hq}, {t_q}], got {tuple(lse.shape)}")
    bf16 = _torch.bfloat16
    rc = lib.wf_attn_forward_fp8_block(
        _ptr(q, "q", bf16, device), Hq, ctypes.byref(pool),
        _ptr(page_table_row, "page_table_row", _torch.int32, device), seg.ref, scale,
        _ptr(out, "out", bf16, device),
        None if lse is None else _ptr(lse, "lse", _torch.float32, device), splits,
        None if workspace is None else _ptr(workspace, "workspace", _torch.uint8, device),
        0 if workspace is None else workspace.numel(), _raw_stream(stream, device))
    if rc != WF_OK:
        raise WfError(rc, "wf_attn_forward_fp8_block")


def ipc_export(device_ptr: int):
    """wf_ipc_export: (64-byte IPC handle of the allocation holding ``device_ptr``, offset)."""
    buf = ctypes.create_string_buffer(64)
    off = ctypes.c_size_t()
    rc = lib.wf_ipc_export(ctypes.c_void_p(int(device_ptr)), buf, ctypes.byref(off))
    if rc != WF_OK:
        raise WfError(rc, "wf_ipc_export")
    return buf.raw, int(off.value)


def ipc_import(exported) -> int:
    """wf_ipc_import: map another process's (handle, offset); returns the device pointer here."""
    handle, offset = exported
    if len(handle) != 64:
        raise ValueError("an IPC handle has 64 bytes")
    out = ctypes.c_void_p()
    rc = lib.wf_ipc_import(ctypes.create_string_buffer(handle, 64), int(offset),
                           ctypes.byref(out))
    if rc != WF_OK:
        raise WfError(rc, "wf_ipc_import")
    return int(out.value)


def ipc_close(device_ptr: int) -> None:
    rc = lib.wf_ipc_close(ctypes.c_void_p(int(device_ptr)))
    if rc != WF_OK:
        raise WfError(rc, "wf_ipc_close")


def selftest_timeout(timeout_us: int, stream=None) -> None:
    """wf_selftest_timeout: make one bounded in-kernel wait run out (read it with check_status)."""
    rc = lib.wf_selftest_timeout(int(timeout_us), _stream_handle(stream))
    if rc != WF_OK:
        raise WfError(rc, "wf_selftest_timeout")


def check_status(stream=None) -> int:
    """wf_check_status: synchronise the stream and return (and clear) the first device error."""
    return int(lib.wf_check_status(_stream_handle(stream)))
