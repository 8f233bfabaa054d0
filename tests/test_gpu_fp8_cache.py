"""wf_kv_append_fp8_block on the GPU against the oracle's cache (oracle/cache.py)."""
import numpy as np
import pytest
import torch

from block_causal_streaming_b200 import (WF_ERR_PAGE_OOB, WF_ERR_POSITION, WF_OK, NormRope,
                                         WavefrontDesc, check_status, kv_append_fp8_block)
from oracle import cache as oc
from cache_util import FP32_REL, bf16_rows, bf16_weight, pair_size, positions_of, table_of

pytestmark = pytest.mark.gpu


class Pools:
    def __init__(self, pages, ps, H, D, fill=0):
        self.codes = [torch.full((pages, ps, H, D), fill, dtype=torch.uint8, device="cuda")
                      for _ in range(2)]
        self.scale = [torch.full((pages, ps // 16, H), fill, dtype=torch.uint8, device="cuda")
                      for _ in range(2)]
        self.oracle = [oc.Fp8Cache(pages, ps, H, D) for _ in range(2)]

    @property
    def tensors(self):
        return (*self.codes, *self.scale)

    def equal_to_oracle(self):
        return all(np.array_equal(self.codes[i].cpu().numpy(), self.oracle[i].codes) and
                   np.array_equal(self.scale[i].cpu().numpy(), self.oracle[i].scale)
                   for i in range(2))


def _desc(off, ps, extra=1):
    return WavefrontDesc(off, list(range(len(off) - 1)), 0, -(-off[-1] // ps) + extra)


@pytest.mark.parametrize("D, ps, H", [(128, 64, 3), (64, 16, 5), (128, 48, 1), (64, 128, 2)])
def test_plain_rows_are_coded_exactly_chunk_by_chunk(D, ps, H):
    """No norm, no rotation: codes and scales equal the oracle's, whatever the chunks' edges."""
    off = [0, 5, 6, 6, 40, 173, 200]
    pages = -(-200 // ps) + 1
    wf = _desc(off, ps)
    pt = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).int().view(1, -1)
    p = Pools(pages, ps, H, D)
    k, v = bf16_rows(200, H, D, 2, 0.7), bf16_rows(200, H, D, 3, 40.0)
    for a, b in ((0, 1), (1, 2), (2, 3), (3, 5), (5, 6), (3, 4), (1, 2)):   # two of them again
        lo, hi = off[a], off[b]
        if a in (1, 3) and b != 5:
            k[lo:hi] *= 3                                 # overwritten with other values
        kv_append_fp8_block(*p.tensors, 0, a, b, k[lo:hi].cuda(), v[lo:hi].cuda(), pt.cuda(), wf)
        if hi > lo:
            p.oracle[0].append(k[lo:hi].double().numpy(), lo, 200, pt[0])
            p.oracle[1].append(v[lo:hi].double().numpy(), lo, 200, pt[0])
        assert check_status() == WF_OK
        assert p.equal_to_oracle()


def test_single_tokens_growing_a_sequence():
    H, D, ps = 2, 128, 32
    pt = torch.tensor([[2, 0, 1]]).int()
    p = Pools(3, ps, H, D)
    k, v = bf16_rows(70, H, D, 4, 2.0), bf16_rows(70, H, D, 5)
    wf = WavefrontDesc([0, 19], [0], 0, 3)
    kv_append_fp8_block(*p.tensors, 0, 0, 1, k[:19].cuda(), v[:19].cuda(), pt.cuda(), wf)
    for i, x in enumerate((k, v)):
        p.oracle[i].append(x[:19].double().numpy(), 0, 19, pt[0])
    for t in range(19, 70):
        wf = WavefrontDesc([0, t, t + 1], [0, 0], 1, 3)
        kv_append_fp8_block(*p.tensors, 0, 1, 2, k[t:t + 1].cuda(), v[t:t + 1].cuda(), pt.cuda(),
                            wf)
        for i, x in enumerate((k, v)):
            p.oracle[i].append(x[t:t + 1].double().numpy(), t, t + 1, pt[0])
    assert check_status() == WF_OK and p.equal_to_oracle()


def test_dead_rows_and_their_scales_have_no_say():
    """A page that another sequence left behind: NaN codes, the largest scales."""
    H, D, ps = 2, 64, 16
    p = Pools(3, ps, H, D, fill=0xFF)
    for o in p.oracle:
        o.codes[:], o.scale[:] = 0xFF, 0xFF
    k = bf16_rows(21, H, D, 6)
    wf = _desc([0, 21], ps)
    pt = torch.tensor([[1, 2, 0]]).int()
    kv_append_fp8_block(*p.tensors, 0, 0, 1, k.cuda(), k.cuda(), pt.cuda(), wf)
    for o in p.oracle:
        o.append(k.double().numpy(), 0, 21, pt[0])
    assert check_status() == WF_OK and p.equal_to_oracle()
    assert (p.codes[0][2, 5:] == 0xFF).all() and (p.codes[0][0] == 0xFF).all()


def test_extreme_values():
    H, D, ps = 1, 128, 16
    x = torch.zeros(64, H, D)
    x[0, 0, 0], x[1, 0, 1], x[2, 0, 2] = float("nan"), float("inf"), -float("inf")
    x[3] = 0.001
    x[16:32] = 3.3e38                                     # saturates: the scale stops at 2^119
    x[20, 0, 7] = -3.3e38
    x[32:48] = 1e-38                                      # vanishes: the scale stops at 2^-100
    x[40] = 4e-30
    x = x.to(torch.bfloat16)                              # rows 48..63: zeros
    p = Pools(4, ps, H, D)
    wf = _desc([0, 64], ps, 0)
    pt = torch.arange(4).int().view(1, -1)
    kv_append_fp8_block(*p.tensors, 0, 0, 1, x.cuda(), x.cuda(), pt.cuda(), wf)
    ref = x.double().numpy()
    ref = np.where(np.isfinite(ref), ref, np.nan)
    for o in p.oracle:
        o.append(ref, 0, 64, pt[0])
    assert check_status() == WF_OK
    for i in range(2):
        got, want = p.codes[i].cpu().numpy(), p.oracle[i].codes
        nan = (want & 0x7F) == 0x7F
        assert np.array_equal((got & 0x7F) == 0x7F, nan) and np.array_equal(got[~nan], want[~nan])
        assert np.array_equal(p.scale[i].cpu().numpy(), p.oracle[i].scale)


@pytest.mark.parametrize("case", [
    (128, (22, 21, 21), True, 64, 3, 1), (64, (16,), False, 16, 2, 37), (128, (64,), False, 32, 4, 15),
    (64, (32,), False, 16, 1, 16), (128, None, False, 16, 2, 3)], ids=str)
@pytest.mark.parametrize("packed", [False, True])
def test_normed_and_turned_keys(case, packed):
    """Keys within half a step of the float64 row, in the block's own scale; values exact."""
    D, pairs, inter, ps, H, start = case
    L = 150
    table = None if pairs is None else table_of(211, sum(pairs))
    rule = NormRope(None if table is None else torch.from_numpy(table).cuda(), axis_pairs=pairs,
                    interleaved=inter, eps=1e-5)
    pos = None if pairs is None else positions_of(L, len(pairs), 211, 7)
    pages = -(-(start + L) // ps)
    wf = WavefrontDesc([0, start, start + L], [0, 1], 1, pages)
    pt = torch.randperm(pages, generator=torch.Generator().manual_seed(8)).int().view(1, -1)
    w = bf16_weight((D,), 9)
    p = Pools(pages, ps, H, D)
    old = bf16_rows(start, H, D, 10)
    kv_append_fp8_block(*p.tensors, 0, 0, 1, old.cuda(), old.cuda(), pt.cuda(), wf)
    x = bf16_rows(L, 3 * H, D, 11).cuda()
    k, v = x[:, H:2 * H], x[:, 2 * H:]
    if not packed:
        k, v = k.contiguous(), v.contiguous()
    kv_append_fp8_block(*p.tensors, 0, 1, 2, k, v, pt.cuda(), wf, rule,
                        None if pos is None else torch.from_numpy(pos).cuda(), w.cuda())
    assert check_status() == WF_OK
    want = oc.norm_rope(k.double().cpu().numpy(), w.double().numpy(), True, 1e-5, table, pos,
                        pairs or (), inter)
    for o, rows in zip(p.oracle, (want, v.double().cpu().numpy())):
        o.append(old.double().numpy(), 0, start + L, pt[0])
        o.append(rows, start, start + L, pt[0])
    assert np.array_equal(p.codes[1].cpu().numpy(), p.oracle[1].codes)
    assert np.array_equal(p.scale[1].cpu().numpy(), p.oracle[1].scale)
    # no block's largest key lies within the fp32 error of a change of scale (checked here, so that
    # the scales must agree)
    assert np.array_equal(p.scale[0].cpu().numpy(), p.oracle[0].scale)
    got = oc.decode_rows(p.codes[0].cpu().numpy(), p.scale[0].cpu().numpy(), pt[0], start + L)
    ref = p.oracle[0].values(pt[0], start + L)
    assert np.array_equal(got[:start], ref[:start])       # the rows that stayed
    exp = np.stack([p.oracle[0].scale[pt[0][t // ps], t % ps // 16].astype(float) - 127
                    for t in range(start, start + L)])
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.abs(want) + 1e-300)), exp[..., None] - 6) - 3)
    tol = step / 2 + FP32_REL * pair_size(want, sum(pairs or ()), inter)
    assert (np.abs(got[start:] - want) <= tol).all()
    assert (got[start:] != ref[start:]).mean() < 1e-3     # and nearly always the same code


def test_bad_pages_and_positions_leave_their_blocks_alone():
    H, D, ps = 2, 64, 32
    table = torch.from_numpy(table_of(9, 32)).cuda()
    wf = WavefrontDesc([0, 90], [0], 0, 3)
    x = bf16_rows(90, H, D, 12).cuda()
    pos = torch.zeros(90, 1, dtype=torch.int32, device="cuda")
    p = Pools(3, ps, H, D)
    kv_append_fp8_block(*p.tensors, 0, 0, 1, x, x, torch.tensor([[2, -1, 0]]).int().cuda(), wf,
                        NormRope(table), pos)
    assert check_status() == WF_ERR_PAGE_OOB
    assert (p.codes[0][1] == 0).all() and (p.scale[1][1] == 0).all()
    assert (p.scale[1][0, :2] > 0).all() and (p.scale[0][2] > 0).all()
    pos[17] = 9
    p = Pools(3, ps, H, D)
    kv_append_fp8_block(*p.tensors, 0, 0, 1, x, x, torch.tensor([[2, 1, 0]]).int().cuda(), wf,
                        NormRope(table), pos)
    assert check_status() == WF_ERR_POSITION
    for i in range(2):
        assert (p.codes[i][2, 16:] == 0).all() and (p.scale[i][2, 1] == 0).all()
        assert (p.scale[i][2, 0] > 0).all() and (p.scale[i][1] > 0).all()


def test_captured_append_replays():
    H, D, ps = 2, 128, 16
    wf = WavefrontDesc([0, 37], [0], 0, 3)
    pt = torch.tensor([[0, 2, 1]]).int().cuda()
    k, v = bf16_rows(37, H, D, 13).cuda(), bf16_rows(37, H, D, 14).cuda()
    p, r = Pools(3, ps, H, D), Pools(3, ps, H, D)
    kv_append_fp8_block(*r.tensors, 0, 0, 1, k, v, pt, wf)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv_append_fp8_block(*p.tensors, 0, 0, 1, k, v, pt, wf)
    assert (p.codes[0] == 0).all()
    g.replay()
    g.replay()
    assert check_status() == WF_OK
    assert all(torch.equal(a, b) for a, b in zip(p.tensors, r.tensors))
