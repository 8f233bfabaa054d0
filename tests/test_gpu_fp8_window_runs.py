"""Rolling windows in the FP8 cache whose runs of consecutive slots are one append each."""
import math

import numpy as np
import pytest
import torch

from block_causal_streaming_b200 import WF_OK, NormRope, check_status
from block_causal_streaming_b200.layer import rotation_table
from block_causal_streaming_b200.window import ACTIVE, RollingCache, RollingWindow
from oracle import cache as oc
from cache_util import BF16_HALF, bf16_rows, bf16_weight

pytestmark = pytest.mark.gpu


def _runs(slots):
    """[first index, count] of the consecutive runs of a list of slots."""
    out = []
    for i, s in enumerate(slots):
        if out and s == slots[i - 1] + 1:
            out[-1][1] += 1
        else:
            out.append([i, 1])
    return out


@pytest.mark.parametrize("copy_free", [False, True], ids=["hand_over", "copy_free_ring"])
@pytest.mark.parametrize("chunk_len, stages, history, ps, D", [
    (200, (1000, 600, 200), 2, 64, 128), (73, (1000, 500), 3, 16, 64), (15, (1000, 700, 500), 2, 16, 64)])
def test_equals_a_replay_of_the_runs(chunk_len, stages, history, ps, D, copy_free):
    """Codes and scales bit for bit, attention against float64 on the values they stand for."""
    H, G, L, scale = 2, 2, chunk_len, 1.0 / math.sqrt(D)
    win = RollingWindow(chunk_len, stages, history, ps, copy_free=copy_free)
    cache = RollingCache(win, H, D, 1, "cuda", fp8_block=True, append_runs=True)
    row = cache.page_tables[0].cpu().numpy()
    replay = [oc.Fp8Cache(win.pages, ps, H, D) for _ in range(2)]
    for t in range(len(stages) + history + 4):
        view = win.view(t)
        slots, live = view.query_rows_slots, view.chunk_offsets[-1]
        n = L * len(slots)
        k, v = bf16_rows(n, H, D, 10 * t), bf16_rows(n, H, D, 10 * t + 1)
        q = bf16_rows(n, G * H, D, 10 * t + 2).cuda()
        out, lse = torch.empty_like(q), torch.empty(G * H, n, device="cuda")
        cache.run_layer(view, 0, q, k.cuda(), v.cuda(), out, scale, lse)
        assert check_status() == WF_OK
        for i, m in _runs(slots):
            for c, x in zip(replay, (k, v)):
                c.append(x[i * L:(i + m) * L].double().numpy(), view.chunk_offsets[slots[i]], live, row)
        vals = [c.values(row, live) for c in replay]
        ends, kv = view.segments() if copy_free else \
            ([(i + 1) * L for i in range(len(slots))], [view.chunk_offsets[s + 1] for s in slots])
        want, wl = oc.attention(q.double().cpu().numpy(), *vals, ends, kv, scale)
        A, _ = oc.attention(q.double().cpu().numpy(), vals[0], np.abs(vals[1]), ends, kv, scale)
        # the bounds of the attention's own tests: the output's rounding, weights to 11 bits and fp32
        # logits below 2^6, small weights and values
        tol = BF16_HALF * np.abs(want) + A * 2.0 ** -9 + 2.0 ** -36 * live * np.abs(vals[1]).max()
        assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
        assert np.abs(lse.double().cpu().numpy() - wl).max() <= 2.0 ** -11
        if view.store_to is not None:
            for c, x in zip(replay, (k, v)):
                c.append(x[:L].double().numpy(), view.chunk_offsets[view.store_to], live, row)
    for codes, sc, c in ((cache.pool.k_codes, cache.pool.k_scale, replay[0]),
                         (cache.pool.v_codes, cache.pool.v_scale, replay[1])):
        assert np.array_equal(codes.cpu().numpy(), c.codes) and np.array_equal(sc.cpu().numpy(), c.scale)


@pytest.mark.parametrize("with_rule", [False, True])
@pytest.mark.parametrize("copy_free", [False, True], ids=["hand_over", "copy_free_ring"])
def test_a_round_does_not_depend_on_what_its_slots_held(copy_free, with_rule):
    """The chunks in flight are 512 times as large in all rounds before the last: the last round's keys
    and values in its own slots, and what its rows see of them, are the same.  (73 tokens a chunk: every
    border between chunks lies inside a block.)"""
    L, ps, D, H, last = 73, 16, 64, 2, 7
    win = RollingWindow(L, (1000, 500), 3, ps, copy_free=copy_free)
    rule = NormRope(rotation_table(L, (D // 2,)), norm=False) if with_rule else None

    def held(loud):
        cache = RollingCache(win, H, D, 1, "cuda", fp8_block=True, append_runs=True)
        for t in range(last + 1):
            view = win.view(t)
            slots = view.query_rows_slots
            n = L * len(slots)
            x = bf16_rows(n, 2 * H, D, t)
            for i, s in enumerate(slots):
                if loud and t < last and view.roles[s] == ACTIVE:
                    x[i * L:(i + 1) * L] *= 512
            x = x.cuda()
            pos = torch.arange(L, dtype=torch.int32, device="cuda").repeat(len(slots)).view(-1, 1)
            out = torch.empty(n, H, D, dtype=torch.bfloat16, device="cuda")
            cache.run_layer(view, 0, torch.zeros_like(out), x[:, :H], x[:, H:], out, rule=rule,
                            positions=pos if with_rule else None)
        assert check_status() == WF_OK
        row = cache.page_tables[0].cpu().numpy()
        rows = np.concatenate([np.arange(view.chunk_offsets[s], view.chunk_offsets[s + 1])
                               for s in slots if view.roles[s] == ACTIVE])
        return [oc.decode_rows(c.cpu().numpy(), s.cpu().numpy(), row, view.chunk_offsets[-1])[rows]
                for c, s in ((cache.pool.k_codes, cache.pool.k_scale),
                             (cache.pool.v_codes, cache.pool.v_scale))]
    for a, b in zip(held(False), held(True)):
        assert np.array_equal(a, b)


def test_one_layer_of_a_full_ring_with_normed_keys():
    """Five chunks in flight and a store pass as one append: attention as with one append a chunk, within
    what coding a shared block twice may change (half a step of e4m3's smallest, 2^-10 of a scale)."""
    L, ps, D, H = 45, 16, 128, 2
    win = RollingWindow(L, (1000, 800, 600, 400, 200), 2, ps)
    rule = NormRope(rotation_table(4 * L, (D // 2,)))
    w = bf16_weight((D,), 1).cuda()
    caches = [RollingCache(win, H, D, 1, "cuda", fp8_block=True, append_runs=r) for r in (False, True)]
    for t in range(10):
        view = win.view(t)
        n = view.t_q
        x, q = bf16_rows(n, 2 * H, D, t).cuda(), bf16_rows(n, H, D, 50 + t).cuda()
        pos = torch.arange(n, dtype=torch.int32, device="cuda").remainder_(4 * L).view(-1, 1)
        outs = []
        for c in caches:
            outs.append(torch.empty_like(q))
            c.run_layer(view, 0, q, x[:, :H], x[:, H:], outs[-1], rule=rule, positions=pos, k_weight=w)
        assert check_status() == WF_OK
        a, b = (o.double() for o in outs)
        assert ((a - b).norm() / a.norm()).item() <= 2.0 ** -8
