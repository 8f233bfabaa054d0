"""A query row with an infinite value, in attention over the FP8 cache: softmax over logits that are all
-inf is NaN, so the row is NaN whatever the signs of the keys in that channel, on every path.

The other rows are held to the attention's own bound and not to their bits in a call without such a row:
in a tile of few rows one vote moves all rows' references to their maxima, and a weight's rounding to
f16 depends on its row's reference."""
import pytest
import torch

from block_causal_streaming_b200 import (WF_OK, Segments, attn_forward_fp8_block,
                                         attn_fp8_block_workspace_size, check_status)
from cache_util import bf16_rows
from oracle import cache as oc
from test_gpu_fp8_attention import check, make_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("N", [1, 2, 40, 600], ids=lambda n: f"{n}_keys")
@pytest.mark.parametrize("rows, group", [(1, 1), (1, 6), (10, 1), (12, 2), (130, 1), (140, 3)])
def test_row_is_nan_when_every_key_has_the_other_sign(rows, group, N, sign):
    H, D, ps, ch = 2, 64, 16, 7
    cache, pt, vals = make_cache(N, H, D, ps, 90)
    live = cache[0] != 0x7F
    codes = cache[0].clone()
    codes[..., ch] = 0x38                                   # 1.0 in that channel, every key
    cache[0].copy_(torch.where(live, codes, cache[0]))
    vals[0] = oc.decode_rows(cache[0].cpu().numpy(), cache[2].cpu().numpy(), pt.cpu().numpy(), N)
    q = bf16_rows(rows, H * group, D, 91).cuda()
    seg = Segments([rows], [N], N, pt.numel())

    def run(splits):
        out, lse = torch.zeros_like(q), torch.zeros(H * group, rows, device="cuda")
        need = attn_fp8_block_workspace_size(seg, H * group, H, D, splits)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
        attn_forward_fp8_block(q, *cache, pt, seg, 0.1, out, lse, splits, ws)
        assert check_status() == WF_OK
        return out, lse
    bad = torch.zeros(rows, H * group, dtype=torch.bool, device="cuda")
    bad[0, 0] = bad[-1, -1] = bad[rows // 2, H * group // 2] = True
    for splits in (0, 1):
        base, base_lse = run(splits)
        clean = q.clone()
        q[bad, ch] = sign * float("inf")
        out, lse = run(splits)
        q.copy_(clean)
        assert out[bad].isnan().all() and lse.t()[bad].isnan().all()
        out[bad], lse.t()[bad] = base[bad], base_lse.t()[bad]
        check(out, lse, q, vals, [rows], [N], 0.1)
