"""Attention over the FP8 cache with the output in the queries' own memory."""
import pytest
import torch

from block_causal_streaming_b200 import (WF_OK, Segments, attn_forward_fp8_block,
                                         attn_fp8_block_workspace_size, check_status)
from cache_util import bf16_rows
from test_gpu_fp8_attention import make_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ends, kv, Hq, H, D, N", [
    ([1], [900], 8, 2, 128, 900), ([7, 20], [0, 500], 2, 2, 64, 500), ([150], [700], 4, 4, 128, 700),
    ([300, 1500], [1100, 400], 12, 6, 64, 1100)])
def test_out_may_be_q(ends, kv, Hq, H, D, N):
    cache, pt, _ = make_cache(N, H, D, 16, 5)
    q = bf16_rows(ends[-1], Hq, D, 6).cuda()
    seg = Segments(ends, kv, N, pt.numel())
    for splits in (0, 1):
        need = attn_fp8_block_workspace_size(seg, Hq, H, D, splits)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
        want, x = torch.empty_like(q), q.clone()
        attn_forward_fp8_block(q, *cache, pt, seg, 0.1, want, None, splits, ws)
        attn_forward_fp8_block(x, *cache, pt, seg, 0.1, x, None, splits, ws)
        assert torch.equal(x, want) and check_status() == WF_OK
