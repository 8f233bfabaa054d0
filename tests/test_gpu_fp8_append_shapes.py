"""The FP8 append's two launch shapes, a block's heads in one CTA or spread over several: one call for many
blocks equals calls for a few blocks each."""
import pytest
import torch

from block_causal_streaming_b200 import WF_OK, NormRope, WavefrontDesc, check_status, kv_append_fp8_block
from block_causal_streaming_b200.layer import PagedPoolFp8Block, rotation_table
from cache_util import bf16_rows, bf16_weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L, H, D, first", [(4680, 12, 128, 0), (4680, 3, 64, 4680), (1490, 5, 128, 8),
                                            (1470, 4, 128, 0), (2975, 2, 64, 16), (2950, 6, 64, 7)])
def test_one_call_equals_a_few_blocks_at_a_time(L, H, D, first):
    """Around the border of the rule (93 blocks of head_dim 128, 185 of 64 on 148 SMs) and at a chunk."""
    ps, end = 64, first + L
    pages = -(-end // ps)
    cuts = [0, first] + list(range(first // 16 * 16 + 272, end, 272)) + [end]   # 17 blocks a call
    stage = [0] * (len(cuts) - 1)
    wf = WavefrontDesc(cuts, stage, 1, pages)
    pt = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).int().view(1, -1).cuda()
    rule = NormRope(rotation_table(end, (D // 2,)))
    pos = torch.arange(first, end, dtype=torch.int32, device="cuda").view(-1, 1)
    old, x = bf16_rows(first, 2 * H, D, 2).cuda(), bf16_rows(L, 2 * H, D, 3).cuda()
    w = bf16_weight((D,), 4).cuda()
    pools = [PagedPoolFp8Block(pages, ps, H, D) for _ in range(2)]
    for i, p in enumerate(pools):
        if first:
            kv_append_fp8_block(*p.tensors, 0, 0, 1, old[:, :H], old[:, H:], pt, wf)
        runs = [(1, len(cuts) - 1)] if i == 0 else [(c, c + 1) for c in range(1, len(cuts) - 1)]
        for a, b in runs:
            r = slice(cuts[a] - first, cuts[b] - first)
            kv_append_fp8_block(*p.tensors, 0, a, b, x[r, :H], x[r, H:], pt, wf, rule, pos[r], w)
    assert check_status() == WF_OK
    for name, a, b in zip(("k codes", "v codes", "k scales", "v scales"), *(p.tensors for p in pools)):
        assert torch.equal(a, b), name
