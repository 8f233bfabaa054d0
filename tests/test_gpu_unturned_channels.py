"""Channels past the rotated ones are not turned: what stands there, infinities and NaN among them, stays
in its channel, and without a norm every bit of it does."""
import numpy as np
import pytest
import torch

from block_causal_streaming_b200 import (WF_OK, NormRope, WavefrontDesc, check_status,
                                         kv_append_fp8_block, kv_append_rope, qk_norm_rope)
from oracle import cache as oc
from cache_util import BF16_HALF, FP32_REL, bf16_rows, pair_size, positions_of, table_of

pytestmark = pytest.mark.gpu

CASES = [(64, (12,), True), (128, (20,), True), (128, (8, 4, 16), True), (64, (16,), False),
         (128, (20,), False), (128, (60,), False)]


def _rows(D, pairs, L=21, H=3):
    """Rows with an infinity, a NaN, zeros of both signs and large values past channel 2 pairs."""
    x = bf16_rows(L, H, D, 1)
    c = 2 * sum(pairs)
    x[0, 0, c], x[1, 1, c + 1], x[2, 2, D - 1] = float("inf"), float("nan"), -float("inf")
    x[3, 0, c:] = 3e38
    x[4, 1, c::2], x[5, 1, c + 1::2] = -0.0, -0.0
    x[6, 0, c + 2], x[6, 0, c + 5] = float("inf"), float("inf")
    return x


@pytest.mark.parametrize("norm", [False, True], ids=["plain", "normed"])
@pytest.mark.parametrize("D, pairs, interleaved", CASES)
def test_queries_and_appended_keys(D, pairs, interleaved, norm):
    x = _rows(D, pairs)
    L, H, _ = x.shape
    table, pos = table_of(97, sum(pairs)), positions_of(L, len(pairs), 97, 2)
    rule = NormRope(torch.from_numpy(table).cuda(), axis_pairs=pairs, interleaved=interleaved, norm=norm,
                    eps=1e-5)
    dpos = torch.from_numpy(pos).cuda()
    out = torch.zeros_like(x, device="cuda")
    qk_norm_rope(x.cuda(), out, None, None, rule, dpos)
    pools = [torch.zeros(2, 16, H, D, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    kv_append_rope(*pools, 0, 0, 1, x.cuda(), x.cuda(), torch.tensor([[1, 0]]).int().cuda(),
                   WavefrontDesc([0, L], [0], 0, 2), rule, dpos)
    assert check_status() == WF_OK
    appended = torch.cat((pools[0][1], pools[0][0]))[:L]
    assert torch.equal(appended.view(torch.int16)[~appended.isnan()],
                       out.view(torch.int16)[~out.isnan()])
    assert torch.equal(appended.isnan(), out.isnan())
    c = 2 * sum(pairs)
    if not norm:
        stays, was = out[..., c:].cpu(), x[..., c:]
        nan = was.isnan()
        assert torch.equal(stays.isnan(), nan)
        assert torch.equal(stays.view(torch.int16)[~nan], was.view(torch.int16)[~nan])
    with np.errstate(invalid="ignore", over="ignore"):
        xd = x.double().numpy()
        # rows of 3e38 are left to the plain case: their squares pass what fp32 holds
        rows = [t for t in range(L) if not (norm and t == 3)]
        want = oc.norm_rope(xd[rows], None, norm, 1e-5, table, pos[rows], pairs, interleaved)
        got = out.double().cpu().numpy()[rows]
        assert np.array_equal(np.isnan(got), np.isnan(want))
        ok = np.isfinite(want)
        assert np.array_equal(got[~ok & ~np.isnan(want)], want[~ok & ~np.isnan(want)])
        size = pair_size(np.where(ok, want, 0.0), c // 2, interleaved)
        tol = BF16_HALF * np.abs(want) + FP32_REL * size + 1e-38
        assert (np.abs(got - want)[ok] <= tol[ok]).all()


@pytest.mark.parametrize("D, pairs, interleaved", CASES)
def test_appended_to_the_fp8_cache(D, pairs, interleaved):
    """Only the channel itself is coded as NaN, and it has no say in the block's scale."""
    x = _rows(D, pairs)
    x[3] = 1.0
    L, H, _ = x.shape
    table, pos = table_of(97, sum(pairs)), positions_of(L, len(pairs), 97, 2)
    rule = NormRope(torch.from_numpy(table).cuda(), axis_pairs=pairs, interleaved=interleaved, norm=False)
    codes = [torch.zeros(2, 16, H, D, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scale = [torch.zeros(2, 1, H, dtype=torch.uint8, device="cuda") for _ in "kv"]

    def append(rows):
        kv_append_fp8_block(*codes, *scale, 0, 0, 1, rows.cuda(), rows.cuda(),
                            torch.tensor([[1, 0]]).int().cuda(), WavefrontDesc([0, L], [0], 0, 2), rule,
                            torch.from_numpy(pos).cuda())
        assert check_status() == WF_OK
        return torch.cat((codes[0][1], codes[0][0]))[:L].clone(), scale[0].clone()
    got, got_scale = append(x)
    bad = ~x.isfinite()
    clean, clean_scale = append(torch.where(bad, 0.0, x))
    bad = bad.cuda()
    assert torch.equal(got_scale, clean_scale)
    assert ((got[bad] & 0x7F) == 0x7F).all()
    assert torch.equal(got[~bad], clean[~bad])
