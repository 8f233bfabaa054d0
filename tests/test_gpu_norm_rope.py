"""wf_qk_norm_rope and wf_kv_append_rope on the GPU against float64 (oracle/cache.py)."""
import numpy as np
import pytest
import torch

from block_causal_streaming_b200 import (WF_ERR_PAGE_OOB, WF_ERR_POSITION, WF_OK, NormRope,
                                         WavefrontDesc, attn_forward, check_status,
                                         kv_append_rope, qk_norm_rope)
from oracle import cache as oc
from cache_util import assert_bf16_rows, bf16_rows, bf16_weight, positions_of, table_of

pytestmark = pytest.mark.gpu

# tokens, q heads, k heads, D, axis pairs (None: no rotation), interleaved, norm, weight per head
CASES = [
    (1, 32, 8, 128, (64,), False, True, False),
    (1, 1, 1, 64, (32,), True, True, False),
    (7, 5, 1, 128, (22, 21, 21), True, True, True),
    (130, 12, 12, 128, (22, 21, 21), False, True, False),
    (33, 3, 2, 64, (16,), False, True, False),        # half of the channels turned, split
    (33, 3, 2, 128, (20,), False, True, True),        # partial, groups that straddle the halves
    (21, 2, 3, 128, (60,), False, False, False),      # nearly all of the channels
    (19, 4, 4, 64, (4,), False, True, False),
    (19, 4, 4, 64, (28,), False, True, False),
    (65, 7, 3, 64, (12,), True, False, False),
    (40, 4, 0, 128, (64,), True, True, False),        # queries only
    (40, 6, 2, 128, None, False, True, True),         # norm alone
    (5000, 3, 3, 64, (10, 11, 11), True, True, False),  # more tokens than warps
]


def _rule(pairs, interleaved, norm, per_head, rows=97):
    if pairs is None:
        return NormRope(None, norm=norm, weight_per_head=per_head), None
    table = table_of(rows, sum(pairs))
    return NormRope(torch.from_numpy(table).cuda(), axis_pairs=pairs, interleaved=interleaved,
                    norm=norm, eps=1e-5, weight_per_head=per_head), table


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_qk_against_float64(case, packed):
    L, Hq, Hk, D, pairs, inter, norm, per_head = case
    rule, table = _rule(pairs, inter, norm, per_head)
    pos = None if pairs is None else positions_of(L, len(pairs), 97, 1)
    x = bf16_rows(L, Hq + Hk + 1, D, 2, 3.0).cuda()
    q, k = x[:, :Hq], x[:, Hq:Hq + Hk]
    if not packed:
        q, k = q.contiguous(), k.contiguous()
    qw = bf16_weight((Hq, D) if per_head else (D,), 3) if norm else None
    kw = bf16_weight((Hk, D) if per_head else (D,), 4) if norm and Hk else None
    q_out = torch.full((L, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((L, Hk, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    qk_norm_rope(q, q_out, k if Hk else None, k_out if Hk else None, rule,
                 None if pos is None else torch.from_numpy(pos).cuda(),
                 qw.cuda() if qw is not None else None, kw.cuda() if kw is not None else None)
    assert check_status() == WF_OK
    for name, t, w, got in (("q", q, qw, q_out), ("k", k, kw, k_out)):
        if t.shape[1] == 0:
            continue
        want = oc.norm_rope(t.double().cpu().numpy(), None if w is None else w.double().numpy(),
                            norm, 1e-5 if pairs is not None else 1e-6, table, pos, pairs or (), inter)
        assert_bf16_rows(got, want, sum(pairs or ()), inter, name)


def test_qk_in_place_repeats_and_replays():
    rule, _ = _rule((64,), False, True, False)
    pos = torch.from_numpy(positions_of(50, 1, 97, 5)).cuda()
    q, k = bf16_rows(50, 4, 128, 6).cuda(), bf16_rows(50, 2, 128, 7).cuda()
    a, b = torch.empty_like(q), torch.empty_like(k)
    qk_norm_rope(q, a, k, b, rule, pos)
    c, d = q.clone(), k.clone()
    qk_norm_rope(c, c, d, d, rule, pos)
    assert torch.equal(a, c) and torch.equal(b, d)
    g = torch.cuda.CUDAGraph()
    e, f = torch.empty_like(q), torch.empty_like(k)
    with torch.cuda.graph(g):
        qk_norm_rope(q, e, k, f, rule, pos)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, e) and torch.equal(b, f)
    q.mul_(2)
    pos.add_(-pos)                                       # new values, the same memory
    g.replay()
    qk_norm_rope(q, a, k, b, rule, pos)
    assert torch.equal(a, e) and torch.equal(b, f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    e.zero_()
    torch.cuda.current_stream().synchronize()
    qk_norm_rope(q, e, k, f, rule, pos, stream=s)
    s.synchronize()
    assert torch.equal(a, e) and check_status() == WF_OK


def test_extreme_rows():
    """Rows of zeros, of the largest and of tiny values; a NaN stays in its own row."""
    rule, table = _rule((64,), False, True, False)
    x = torch.zeros(4, 1, 128)
    x[1] = 1e18
    x[2] = 1e-30
    x[3] = 1.0
    x[3, 0, 5] = float("nan")
    x = x.to(torch.bfloat16)
    pos = np.array([[3], [4], [5], [6]], np.int32)
    out = torch.empty_like(x, device="cuda")
    qk_norm_rope(x.cuda(), out, None, None, rule, torch.from_numpy(pos).cuda())
    want = oc.norm_rope(x[:3].double().numpy(), None, True, 1e-5, table, pos[:3], (64,), False)
    assert_bf16_rows(out[:3], want, 64, False)
    assert out[3].isnan().all()


def test_a_position_off_the_table_leaves_its_token_alone():
    rule, _ = _rule((30, 2, 32), True, True, False)
    x = bf16_rows(40, 3, 128, 8).cuda()
    pos = positions_of(40, 3, 97, 9)
    good = torch.empty_like(x)
    qk_norm_rope(x, good, None, None, rule, torch.from_numpy(pos).cuda())
    pos[5, 0], pos[9, 2], pos[39, 1] = 97, -1, 2 ** 31 - 1
    out = torch.full_like(x, 7.0)
    qk_norm_rope(x, out, None, None, rule, torch.from_numpy(pos).cuda())
    assert check_status() == WF_ERR_POSITION and check_status() == WF_OK
    for t in range(40):
        assert torch.equal(out[t], torch.full_like(out[t], 7.0) if t in (5, 9, 39) else good[t])


@pytest.mark.parametrize("case", [
    (1, 8, 128, 64, (64,), False, 100),
    (300, 12, 128, 16, (22, 21, 21), True, 77),
    (45, 3, 64, 48, (16,), False, 5),
    (45, 3, 64, 16, None, False, 0),
], ids=str)
@pytest.mark.parametrize("packed", [False, True])
def test_append_rope_against_float64(case, packed):
    L, H, D, ps, pairs, inter, start = case
    rule, table = _rule(pairs, inter, True, False)
    end = start + L + 3                                  # a later chunk of 3 tokens
    pages = -(-end // ps) + 1
    off = [0, start, start + L // 2, start + L, end]
    wf = WavefrontDesc(off, [0, 1, 2, 3], 1, pages)
    pt = torch.stack([torch.arange(pages), torch.randperm(pages)]).int().cuda()
    x = bf16_rows(L, 3 * H, D, 10).cuda()
    k, v = x[:, H:2 * H], x[:, 2 * H:]
    if not packed:
        k, v = k.contiguous(), v.contiguous()
    v[0, 0, 0] = float("inf")
    pos = None if pairs is None else positions_of(L, len(pairs), 97, 11)
    w = bf16_weight((D,), 12)
    pools = [torch.full((pages, ps, H, D), -3.0, dtype=torch.bfloat16, device="cuda")
             for _ in range(2)]
    kv_append_rope(*pools, 1, 1, 3, k, v, pt, wf, rule,
                   None if pos is None else torch.from_numpy(pos).cuda(), w.cuda())
    assert check_status() == WF_OK
    tok = torch.arange(start, start + L)
    rows = (pt[1].cpu().long()[tok // ps] * ps + tok % ps).cuda()
    want = oc.norm_rope(k.double().cpu().numpy(), w.double().numpy(), True,
                        1e-6 if pairs is None else 1e-5, table, pos, pairs or (), inter)
    assert_bf16_rows(pools[0].flatten(0, 1)[rows], want, sum(pairs or ()), inter)
    assert torch.equal(pools[1].flatten(0, 1)[rows], v.contiguous())
    for p in pools:                                      # nothing else was written
        rest = torch.ones(pages * ps, dtype=torch.bool)
        rest[rows.cpu()] = False
        assert (p.flatten(0, 1)[rest.cuda()] == -3.0).all()


def test_append_rope_skips_bad_pages_and_positions():
    H, D, ps = 2, 64, 16
    rule, _ = _rule((32,), False, True, False)
    wf = WavefrontDesc([0, 48], [0], 0, 3)
    x = bf16_rows(48, H, D, 13).cuda()
    pos = torch.zeros(48, 1, dtype=torch.int32, device="cuda")
    pools = [torch.zeros(3, ps, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kv_append_rope(*pools, 0, 0, 1, x, x, torch.tensor([[1, 3, 0]]).int().cuda(), wf, rule, pos)
    assert check_status() == WF_ERR_PAGE_OOB
    assert (pools[1][2] == 0).all() and torch.equal(pools[1][1], x[:16])
    pos[0] = -5
    for p in pools:
        p.zero_()
    kv_append_rope(*pools, 0, 0, 1, x, x, torch.tensor([[1, 2, 0]]).int().cuda(), wf, rule, pos)
    assert check_status() == WF_ERR_POSITION
    assert (pools[0][1, 0] == 0).all() and (pools[1][1, 0] == 0).all()
    assert torch.equal(pools[1][1, 1:], x[1:16]) and torch.equal(pools[1][0], x[32:])


def test_a_layer_from_projection_to_attention():
    """Queries and keys normed and turned, keys appended on the way, attention over the pages."""
    H, D, ps, L = 2, 128, 16, 70
    rule, table = _rule((22, 21, 21), True, True, False)
    wf = WavefrontDesc([0, 20, L], [0, 1], 1, 5)
    x = bf16_rows(L, 3 * H, D, 14).cuda()
    pos = positions_of(L, 3, 97, 15)
    dpos = torch.from_numpy(pos).cuda()
    pools = [torch.full((5, ps, H, D), float("nan"), dtype=torch.bfloat16, device="cuda")
             for _ in range(2)]
    pt = torch.tensor([[4, 0, 3, 1, 2]]).int().cuda()
    qw, kw = bf16_weight((D,), 16), bf16_weight((D,), 17)
    q = torch.empty(50, H, D, dtype=torch.bfloat16, device="cuda")
    qk_norm_rope(x[20:, :H], q, None, None, rule, dpos[20:], qw.cuda())
    kv_append_rope(*pools, 0, 0, 2, x[:, H:2 * H], x[:, 2 * H:], pt, wf, rule, dpos, kw.cuda())
    out = torch.empty_like(q)
    attn_forward(q, *pools, pt[0], wf, D ** -0.5, out)
    assert check_status() == WF_OK
    xd = x.double().cpu().numpy()
    qe = oc.norm_rope(xd[20:, :H], qw.double().numpy(), True, 1e-5, table, pos[20:], (22, 21, 21), True)
    ke = oc.norm_rope(xd[:, H:2 * H], kw.double().numpy(), True, 1e-5, table, pos, (22, 21, 21), True)
    want, _ = oc.attention(qe, ke, xd[:, 2 * H:], [50], [L], D ** -0.5)
    err = np.abs(out.double().cpu().numpy() - want)
    # q and k rounded to bf16: a logit is off by 2 x 2^-8 of its terms' sum of magnitudes at most,
    # and far less on average; the values are O(1), the library's stated bar is 1e-2
    assert err.max() <= 2e-2 and err.mean() <= 2e-3
