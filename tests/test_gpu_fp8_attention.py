"""wf_attn_forward_fp8_block on the GPU against float64 attention on the values the cache stands for.

Tolerance.  Weights are rounded to 11 bits before P.V and the sum is not: 2^-11 of A = sum p |v| / l,
and as much again for the fp32 steps around them.  A logit's fp32 sums are off by at most 2^-19 of
L = scale sum |q| |k| (128 terms, and the scaling steps), which moves every weight by that much,
twice (numerator and sum).  The output is rounded to bf16 once: 2^-8 of it.

Under f16's normal range the rounding is absolute.  A weight is held as p 2^13 against a reference no
larger than the maximum (so the sum is at least 1): half a step of 2^-24 is 2^-38 of it, a key's share
of the output is off by at most 2^-38 |v|.  Where weights carry the value scale, p 2^13 2^(e - E), the
half step is 2^-38 2^E in units of codes up to 448, and the largest value is at least 224 2^E: 2^-37 of
the largest value.  Values held as f16 of code 2^(e - E + 7) are off by at most 2^-25 2^(E - 7), under
2^-39 of the largest.  Together at most 2^-36 of the largest value for every key a row sees: FLOOR.
"""
import numpy as np
import pytest
import torch

from block_causal_streaming_b200 import (WF_ERR_PAGE_OOB, WF_OK, Segments, WavefrontDesc,
                                         attn_forward_fp8_block, attn_fp8_block_workspace_size,
                                         check_status, kv_append_fp8_block)
from oracle import cache as oc
from cache_util import BF16_HALF, bf16_rows

pytestmark = pytest.mark.gpu

FLOOR = 2.0 ** -36


def make_cache(N, Hk, D, ps, seed, extra_pages=1, k_scale=1.0, v_scale=1.0):
    """A cache filled through the library; dead rows and scales hold NaN."""
    pages = -(-N // ps) + extra_pages
    g = torch.Generator().manual_seed(seed)
    pt = torch.randperm(pages, generator=g).int()
    codes = [torch.full((pages, ps, Hk, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scale = [torch.full((pages, ps // 16, Hk), 0xFF, dtype=torch.uint8, device="cuda") for _ in "kv"]
    k, v = bf16_rows(N, Hk, D, seed + 1, k_scale), bf16_rows(N, Hk, D, seed + 2, v_scale)
    if N:
        kv_append_fp8_block(*codes, *scale, 0, 0, 1, k.cuda(), v.cuda(), pt.view(1, -1).cuda(),
                            WavefrontDesc([0, N], [0], 0, pages))
    vals = [oc.decode_rows(codes[i].cpu().numpy(), scale[i].cpu().numpy(), pt.numpy(), N)
            for i in range(2)]
    return codes + scale, pt.cuda(), vals


def run(q, cache, pt, seg, scale, splits=0, lse=True, stream=None):
    out = torch.full_like(q, float("nan"))
    ls = torch.full((q.shape[1], q.shape[0]), 7.0, device="cuda") if lse else None
    need = attn_fp8_block_workspace_size(seg, q.shape[1], cache[0].shape[2], q.shape[2], splits)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if need else None
    attn_forward_fp8_block(q, *cache, pt, seg, scale, out, ls, splits, ws, stream)
    return out, ls


def check(out, lse, q, vals, rows_end, kv_end, scale):
    qd = q.double().cpu().numpy()
    want, wl = oc.attention(qd, *vals, rows_end, kv_end, scale)
    A, _ = oc.attention(qd, vals[0], np.abs(vals[1]), rows_end, kv_end, scale)
    k, group = vals[0], q.shape[1] // vals[0].shape[1]
    L = max((np.abs(qd[:, h]) @ np.abs(k[:, h // group]).T).max() * scale
            for h in range(q.shape[1])) if k.shape[0] and q.shape[0] else 0.0
    seen = np.repeat(kv_end, np.diff([0] + list(rows_end)))[:, None, None]
    top = np.abs(vals[1]).max(axis=(0, 2), initial=0.0).repeat(group)[None, :, None]
    tol = BF16_HALF * np.abs(want) + A * (2.0 ** -10 + 2.0 ** -18 * L) + FLOOR * seen * top + 1e-38
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    worst = (np.abs(got - want) / tol).max()
    assert worst <= 1, f"{worst:.3f} of the tolerance"
    if lse is not None:
        gl = lse.double().cpu().numpy()
        live = np.isfinite(wl)
        assert np.array_equal(np.isneginf(gl), ~live)
        lt = 2.0 ** -18 * L + 2.0 ** -20 * (1 + np.abs(wl[live]))
        assert (np.abs(gl[live] - wl[live]) <= lt).all()


# rows_end, kv_end, q heads, k heads, D, page
CASES = [
    ([1], [1], 1, 1, 128, 16),
    ([1], [17], 8, 2, 64, 16),
    ([1], [5000], 32, 8, 128, 64),
    ([1], [777], 5, 1, 128, 48),
    ([3], [1000], 6, 3, 64, 32),
    ([16], [300], 2, 2, 128, 16),
    ([17], [300], 4, 2, 128, 16),
    ([40], [129], 3, 1, 64, 128),
    ([2, 2, 5, 30], [0, 3, 700, 513], 4, 2, 128, 16),       # empty rows, limits out of order
    ([3], [0], 4, 2, 64, 16),
    ([130], [130], 2, 1, 128, 16),
    ([127, 255, 300, 557], [100, 1500, 257, 2049], 3, 3, 128, 64),
    ([600], [1111], 4, 2, 64, 16),
    ([256], [128], 8, 1, 128, 128),
    # more row blocks than SMs: whole ones, shares that cut units, blocks without keys, odd halves
    ([130, 700, 1500], [0, 300, 129], 40, 40, 64, 16),
    ([1100, 4000], [1000, 700], 12, 12, 128, 64),
    ([40, 700, 1300], [3000, 1, 515], 28, 7, 64, 32),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_float64(case):
    rows_end, kv_end, Hq, Hk, D, ps = case
    N = max(kv_end)
    cache, pt, vals = make_cache(N, Hk, D, ps, 20)
    q = bf16_rows(rows_end[-1], Hq, D, 23).cuda()
    seg = Segments(rows_end, kv_end, N, pt.numel())
    for splits in (0, 1, 3):
        out, lse = run(q, cache, pt, seg, D ** -0.5, splits)
        assert check_status() == WF_OK
        check(out, lse, q, vals, rows_end, kv_end, D ** -0.5)


@pytest.mark.parametrize("rows", [1, 20, 150])
def test_large_logits_and_uneven_blocks(rows):
    """Keys of very different sizes, values over 2^20 of range between blocks, peaked softmax."""
    N, H, D, ps = 900, 2, 128, 16
    cache, pt, vals = make_cache(N, H, D, ps, 30, k_scale=4.0)
    for i in (2, 3):                                        # scales shifted block by block
        shift = (torch.arange(cache[i].shape[0]) % 21 - 10).to(torch.int16).cuda()
        s = cache[i].to(torch.int16)
        cache[i].copy_(torch.where(s == 255, s, s + shift[:, None, None] * (i - 2)).to(torch.uint8))
    vals = [oc.decode_rows(cache[i].cpu().numpy(), cache[2 + i].cpu().numpy(), pt.cpu().numpy(), N)
            for i in range(2)]
    q = bf16_rows(rows, 2 * H, D, 31, 5.0).cuda()
    seg = Segments([rows], [N], N, pt.numel())
    out, lse = run(q, cache, pt, seg, 0.2)
    assert check_status() == WF_OK
    check(out, lse, q, vals, [rows], [N], 0.2)


@pytest.mark.parametrize("splits", [0, 1])
@pytest.mark.parametrize("rows", [1, 20, 150])
@pytest.mark.parametrize("byte", [246, 27, 0], ids=["largest", "smallest", "mixed"])
def test_values_at_the_ends_of_the_scales_range(rows, byte, splits):
    """Values up to 448 2^119, just inside fp32, and down to 2^-109: sums over many keys stay in range."""
    N, H, D, ps = 3000, 2, 128, 16
    cache, pt, vals = make_cache(N, H, D, ps, 60)
    live = cache[3] != 255
    b = torch.full_like(cache[3], byte)
    if byte == 0:                                           # blocks of both ends side by side
        b[:, :, 0], b[:, :, 1] = 246, 27
        b[::2] = 127
    cache[3].copy_(torch.where(live, b, cache[3]))
    vals[1] = oc.decode_rows(cache[1].cpu().numpy(), cache[3].cpu().numpy(), pt.cpu().numpy(), N)
    q = bf16_rows(rows, 2 * H, D, 61).cuda()
    out, lse = run(q, cache, pt, Segments([rows], [N], N, pt.numel()), D ** -0.5, splits)
    assert check_status() == WF_OK
    check(out, lse, q, vals, [rows], [N], D ** -0.5)


@pytest.mark.parametrize("rows", [4, 140])
def test_what_rows_do_not_see_cannot_reach_them(rows):
    """A NaN value and a NaN key in tokens past a segment's limit leave its rows as they were; rows
    that see the NaN value are NaN in its channel, rows that see the NaN key altogether."""
    N, H, D, ps = 400, 2, 128, 32
    cache, pt, vals = make_cache(N, H, D, ps, 40)
    q = bf16_rows(3 * rows, H, D, 41).cuda()
    ends, kv = [rows, 2 * rows, 3 * rows], [205, 395, 400]
    seg = Segments(ends, kv, N, pt.numel())
    base, base_lse = run(q, cache, pt, seg, 0.1)
    at = lambda t: (int(pt[t // ps]), t % ps)               # noqa: E731
    cache[1][at(205)][1, 7] = 0x7F                          # value of token 205, head 1, channel 7
    cache[0][at(397)][0, 0] = 0xFF                          # key of token 397, head 0
    out, lse = run(q, cache, pt, seg, 0.1)
    assert check_status() == WF_OK
    assert torch.equal(out[:rows], base[:rows]) and torch.equal(lse[:, :rows], base_lse[:, :rows])
    ref = base.clone()
    ref[rows:, 1, 7] = float("nan")
    ref[2 * rows:, 0] = float("nan")
    assert torch.equal(out.isnan(), ref.isnan())
    assert torch.equal(out.nan_to_num(0), ref.nan_to_num(0))


def test_decoding_token_by_token():
    """Append one token, attend with one token, over a page's and a block's end."""
    Hq, Hk, D, ps = 6, 2, 64, 16
    pages = 4
    codes = [torch.zeros(pages, ps, Hk, D, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scale = [torch.zeros(pages, 1, Hk, dtype=torch.uint8, device="cuda") for _ in "kv"]
    pt = torch.tensor([[3, 1, 0, 2]]).int().cuda()
    k, v, q = (bf16_rows(50, h, D, s).cuda() for h, s in ((Hk, 50), (Hk, 51), (Hq, 52)))
    for t in range(50):
        kv_append_fp8_block(*codes, *scale, 0, 1, 2, k[t:t + 1], v[t:t + 1], pt,
                            WavefrontDesc([0, t, t + 1], [0, 0], 1, pages))
        out, lse = run(q[t:t + 1], codes + scale, pt[0], Segments([1], [t + 1], t + 1, pages), 0.2)
        assert check_status() == WF_OK
        if t % 7 == 0 or t in (15, 16, 17, 49):
            vals = [oc.decode_rows(codes[i].cpu().numpy(), scale[i].cpu().numpy(),
                                   pt[0].cpu().numpy(), t + 1) for i in range(2)]
            check(out, lse, q[t:t + 1], vals, [1], [t + 1], 0.2)


@pytest.mark.parametrize("rows", [2, 300])
def test_repeats_bitwise_replays_and_other_streams(rows):
    N, H, D, ps = 3000, 2, 128, 64
    cache, pt, _ = make_cache(N, H, D, ps, 60)
    q = bf16_rows(rows, H, D, 61).cuda()
    seg = Segments([rows], [N], N, pt.numel())
    a, la = run(q, cache, pt, seg, 0.1)
    b, lb = run(q, cache, pt, seg, 0.1)
    assert torch.equal(a, b) and torch.equal(la, lb)
    out, lse = torch.zeros_like(q), torch.zeros(H, rows, device="cuda")
    need = attn_fp8_block_workspace_size(seg, H, H, D)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attn_forward_fp8_block(q, *cache, pt, seg, 0.1, out, lse, 0, ws)
    for _ in range(3):
        ws.fill_(0xFF)
        out.zero_()
        g.replay()
        assert torch.equal(a, out) and torch.equal(la, lse)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        c, lc = run(q, cache, pt, seg, 0.1)
    s.synchronize()
    assert torch.equal(a, c) and torch.equal(la, lc) and check_status() == WF_OK


@pytest.mark.parametrize("rows", [1, 200])
def test_bad_pages_are_recorded(rows):
    cache, pt, _ = make_cache(100, 2, 64, 16, 70, extra_pages=0)
    pt[3] = 1000
    q = bf16_rows(rows, 2, 64, 71).cuda()
    run(q, cache, pt, Segments([rows], [48], 100, pt.numel()), 0.1)
    assert check_status() == WF_OK                          # the bad page is past the limit
    run(q, cache, pt, Segments([rows], [49], 100, pt.numel()), 0.1)
    assert check_status() == WF_ERR_PAGE_OOB and check_status() == WF_OK


@pytest.mark.parametrize("rows", [3, 130])
def test_a_query_that_is_not_finite_stays_in_its_row(rows):
    N, H, D, ps = 300, 2, 64, 16
    cache, pt, _ = make_cache(N, H, D, ps, 80)
    q = bf16_rows(rows, H, D, 81).cuda()
    seg = Segments([rows], [N], N, pt.numel())
    base, base_lse = run(q, cache, pt, seg, 0.1)
    q[1, 0, 3], q[2, 1, 5] = float("nan"), float("inf")
    out, lse = run(q, cache, pt, seg, 0.1)
    assert check_status() == WF_OK
    bad = torch.zeros(rows, H, dtype=torch.bool, device="cuda")
    bad[1, 0] = bad[2, 1] = True
    assert out[bad].isnan().all() and torch.equal(out[~bad], base[~bad])
    assert torch.equal(lse[~bad.t()], base_lse[~bad.t()]) and not lse[bad.t()].isfinite().any()


def test_a_cache_past_2_gib():
    """Pages whose codes (and bf16 pool values) lie past 2^31 bytes and values."""
    from block_causal_streaming_b200 import NormRope, kv_append_rope
    H, D, ps, N = 8, 128, 64, 300
    pages = 2 ** 31 // (ps * H * D) + 40
    row = torch.arange(pages - 5, pages).int().view(1, -1).cuda()
    codes = [torch.zeros(pages, ps, H, D, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scale = [torch.zeros(pages, ps // 16, H, dtype=torch.uint8, device="cuda") for _ in "kv"]
    k, v = bf16_rows(N, H, D, 90).cuda(), bf16_rows(N, H, D, 91).cuda()
    wf = WavefrontDesc([0, N], [0], 0, 5)
    kv_append_fp8_block(*codes, *scale, 0, 0, 1, k, v, row, wf)
    tail = [c[-5:].clone() for c in codes] + [s[-5:].clone() for s in scale]
    small = [torch.zeros(5, ps, H, D, dtype=torch.uint8, device="cuda") for _ in "kv"] + \
        [torch.zeros(5, ps // 16, H, dtype=torch.uint8, device="cuda") for _ in "kv"]
    at = torch.arange(5).int().cuda()
    kv_append_fp8_block(*small, 0, 0, 1, k, v, at.view(1, -1), wf)
    assert all(torch.equal(a, b) for a, b in zip(tail, small))
    assert all(int(c[:-5].sum(dtype=torch.int64)) == 0 for c in codes)
    for rows in (1, 150):
        q = bf16_rows(rows, H, D, 92).cuda()
        seg = Segments([rows], [N], N, 5)
        a, la = run(q, codes + scale, row[0], seg, 0.1)
        b, lb = run(q, small, at, seg, 0.1)
        assert torch.equal(a, b) and torch.equal(la, lb)
    del codes, scale
    pools = [torch.zeros(pages, ps, H, D, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    kv_append_rope(*pools, 0, 0, 1, k, v, row, wf, NormRope(None, norm=False))
    assert torch.equal(pools[0][-5:].flatten(0, 1)[:N], k)
    assert torch.equal(pools[1][-5:].flatten(0, 1)[:N], v)
    assert not pools[0][:-5].any() and check_status() == WF_OK
