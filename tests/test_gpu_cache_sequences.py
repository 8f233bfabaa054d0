"""The cache operators one after another without a pause: each call begins while the one before it still
runs, and must give what it gives when that one has long ended."""
import pytest
import torch

from block_causal_streaming_b200 import (WF_OK, NormRope, Segments, check_status, kv_append_rope,
                                         qk_norm_rope)
from block_causal_streaming_b200.layer import Fp8BlockLayer, PagedPoolFp8Block, rotation_table
from cache_util import bf16_rows, bf16_weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows, N, Hq, H, D", [(1, 700, 8, 4, 128), (3, 333, 12, 12, 64),
                                               (150, 900, 4, 2, 128), (600, 1100, 6, 3, 64)])
def test_back_to_back_equals_one_at_a_time(rows, N, Hq, H, D):
    """Weights, table, positions, page table, projection, cache and queries all written by the launches
    just before the calls that read them, over and over in the same memory."""
    ps, steps = 16, 25
    pages = -(-N // ps)
    pool = PagedPoolFp8Block(pages, ps, H, D)
    start = N - rows - 5                                      # the appends begin inside a block
    lay = Fp8BlockLayer(pool, torch.zeros(1, pages, dtype=torch.int32, device="cuda"), 0,
                        [0, start, N], [0, 0], 1)
    rule = NormRope(torch.zeros(N, D // 2, 2, device="cuda"))
    table = rotation_table(2 * N, (D // 2,))
    tables = [table[:N].contiguous(), table[N:].contiguous()]
    rowsets = [torch.randperm(pages, generator=torch.Generator().manual_seed(i)).int().cuda()
               for i in range(2)]
    proj = [bf16_rows(N, Hq + 2 * H, D, 10 + i).cuda() for i in range(3)]
    weights = [bf16_weight((D,), 20 + i).cuda() for i in range(3)]
    pos0 = torch.arange(N, dtype=torch.int32, device="cuda").view(-1, 1)
    x, w = torch.zeros_like(proj[0]), torch.zeros_like(weights[0])
    pos = torch.zeros_like(pos0)
    q = torch.zeros(N, Hq, D, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(rows, Hq, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(Hq, rows, device="cuda")
    seg = Segments([rows], [N], N, pages)
    ws = torch.zeros(max(lay.workspace_size(Hq, seg), 16), dtype=torch.uint8, device="cuda")
    bf = [torch.zeros(pages, ps, H, D, dtype=torch.bfloat16, device="cuda") for _ in "kv"]

    def step(i, pause):
        for call in (
                lambda: rule.table.copy_(tables[i % 2]),
                lambda: lay.page_tables[0].copy_(rowsets[i // 2 % 2]),
                lambda: x.copy_(proj[i % 3]),
                lambda: torch.remainder(pos0 + i, N, out=pos),
                lambda: w.copy_(weights[i % 3]),
                lambda: qk_norm_rope(x[:, :Hq], q, None, None, rule, pos, w),
                lambda: lay.append(0, 1, x[:start, Hq:Hq + H], x[:start, Hq + H:], rule, pos[:start], w),
                lambda: lay.append(1, 2, x[start:, Hq:Hq + H], x[start:, Hq + H:], rule, pos[start:], w),
                lambda: lay.forward(q[N - rows:], out, lse=lse, segments=seg, workspace=ws),
                lambda: qk_norm_rope(q, q, None, None, rule, pos),      # over the queries just read
                lambda: kv_append_rope(*bf, 0, 0, 2, x[:, Hq:Hq + H], x[:, Hq + H:], lay.page_tables,
                                       lay.desc, rule, pos, w)):
            call()
            pause()
        return [t.clone() for t in (q, out, lse, *pool.tensors, *bf)]

    def run(pause):
        for t in (*pool.tensors, *bf):
            t.zero_()
        torch.cuda.synchronize()
        return [step(i, pause) for i in range(steps)]
    slow = run(torch.cuda.synchronize)
    fast = run(lambda: None)
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(slow, fast)):
        for name, s, t in zip(("q", "out", "lse", "k codes", "v codes", "k scales", "v scales", "k pages",
                               "v pages"), a, b):
            assert torch.equal(s, t), f"step {i}: {name}"
    assert check_status() == WF_OK
