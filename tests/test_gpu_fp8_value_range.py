"""Attention over the FP8 cache where small values stand beside large ones: the bound that include/wf.h
states, |out - exact| <= 2^-8 |exact| + (2^-10 + 2^-18 L) sum p |v| + n 2^-36 V with V the largest visible
value of the K/V head, whether or not that value has any weight.

The last term: a weight is held as p 2^13 (against a reference no larger than the maximum, so the sum is
at least 1), times 2^(e - E) where the block's value exponent e lies under the largest, E.  In f16 its
rounding is at most 2^-25 once it falls under the normal range: 2^-38 2^E in units of codes of up to 448,
and V is over 224 2^E: 2^-37 V for each key.  Values held as f16 of code 2^(e - E + 7) are off by at most
2^-25 2^(E - 7), under 2^-39 V.  Together less than 2^-36 V for each of n keys."""
import numpy as np
import pytest
import torch

from block_causal_streaming_b200 import (WF_OK, Segments, WavefrontDesc, attn_forward_fp8_block,
                                         attn_fp8_block_workspace_size, check_status,
                                         kv_append_fp8_block)
from oracle import cache as oc
from cache_util import BF16_HALF, bf16_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("splits", [0, 1])
@pytest.mark.parametrize("rows, group", [(1, 1), (3, 4), (20, 1), (140, 1)])
@pytest.mark.parametrize("spread", [0, 12, 20, 30, 40, 60])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_small_values_beside_a_large_one_without_weight(where, spread, rows, group, splits):
    """One block of 16 keys holds values 2^spread times as large and has next to no weight."""
    H, D, ps, N = 2, 128, 32, 400
    pages = -(-N // ps)
    pt = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).int()
    k, v = bf16_rows(N, H, D, 2, 0.1), bf16_rows(N, H, D, 3)
    b = {"first": 0, "middle": 12, "last": 24}[where]
    big = slice(16 * b, 16 * b + 16)
    v[big] *= 2.0 ** spread
    k[:, :, 0] = 0.0
    k[big, :, 0] = -100.0                                   # logits about -200: weights of exp(-200)
    codes = [torch.zeros(pages, ps, H, D, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scale = [torch.zeros(pages, ps // 16, H, dtype=torch.uint8, device="cuda") for _ in "kv"]
    kv_append_fp8_block(*codes, *scale, 0, 0, 1, k.cuda(), v.cuda(), pt.view(1, -1).cuda(),
                        WavefrontDesc([0, N], [0], 0, pages))
    kd, vd = (oc.decode_rows(codes[i].cpu().numpy(), scale[i].cpu().numpy(), pt.numpy(), N)
              for i in range(2))
    q = bf16_rows(rows, H * group, D, 4)
    q[:, :, 0] = 20.0
    q = q.cuda()
    out = torch.full_like(q, float("nan"))
    seg = Segments([rows], [N], N, pages)
    need = attn_fp8_block_workspace_size(seg, H * group, H, D, splits)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    attn_forward_fp8_block(q, *codes, *scale, pt.cuda(), seg, 0.1, out, None, splits, ws)
    assert check_status() == WF_OK
    qd = q.double().cpu().numpy()
    want, _ = oc.attention(qd, kd, vd, [rows], [N], 0.1)
    A, _ = oc.attention(qd, kd, np.abs(vd), [rows], [N], 0.1)
    L = 0.1 * max((np.abs(qd[:, h]) @ np.abs(kd[:, h // group]).T).max() for h in range(H * group))
    V = np.abs(vd).max(axis=(0, 2)).repeat(group)[None, :, None]
    err = np.abs(out.double().cpu().numpy() - want)
    tol = BF16_HALF * np.abs(want) + (2.0 ** -10 + 2.0 ** -18 * L) * A + N * 2.0 ** -36 * V
    worst = (err / tol).max()
    assert worst <= 1, f"{worst:.3f} of the bound"
