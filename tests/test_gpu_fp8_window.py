"""The cache operators as a stream uses them: a rolling window whose K/V stay in the FP8 cache, and
one whose keys are normed and rotated on the way into either cache, round after round."""
import math

import numpy as np
import pytest
import torch

from block_causal_streaming_b200 import WF_OK, NormRope, check_status, qk_norm_rope
from block_causal_streaming_b200.layer import (Fp8BlockLayer, PagedPoolFp8Block, rotation_table,
                                               video_positions)
from block_causal_streaming_b200.window import RollingCache, RollingWindow
from oracle import cache as oc
from cache_util import BF16_HALF, bf16_rows, bf16_weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("copy_free", [False, True], ids=["hand_over", "copy_free_ring"])
@pytest.mark.parametrize("chunk_len, stages, history, ps, D", [
    (200, (1000, 600, 200), 2, 64, 128), (73, (1000, 500), 3, 16, 64)])
def test_fp8_window_equals_a_replay(chunk_len, stages, history, ps, D, copy_free):
    """Chunks that are no multiple of 16 tokens share blocks with neighbours that stay: the pools equal
    a replay of the same appends through the oracle's cache, bit for bit, and attention equals float64
    on the replayed values."""
    H, G, layers = 2, 2, 2
    win = RollingWindow(chunk_len, stages, history, ps, copy_free=copy_free)
    pt = torch.from_numpy(np.random.default_rng(3).permutation(win.pages * layers).astype(np.int32))
    pt = pt.view(layers, win.pages)
    cache = RollingCache(win, H, D, layers, "cuda", page_tables=pt, fp8_block=True)
    replay = [oc.Fp8Cache(win.pages * layers, ps, H, D) for _ in range(2)]
    L, scale = chunk_len, 1.0 / math.sqrt(D)
    for t in range(len(stages) + history + 4):
        view = win.view(t)
        for layer in range(layers):
            n = view.t_q if not copy_free else L * len(view.query_rows_slots)
            seed = 100 * t + 10 * layer
            k, v = bf16_rows(n, H, D, seed), bf16_rows(n, H, D, seed + 1)
            q = bf16_rows(n, G * H, D, seed + 2).cuda()
            out = torch.empty_like(q)
            lse = torch.empty(G * H, n, device="cuda")
            cache.run_layer(view, layer, q, k.cuda(), v.cuda(), out, scale, lse)
            assert check_status() == WF_OK
            row, live = pt[layer].numpy(), view.chunk_offsets[-1]

            def put(slot, i):
                for c, x in zip(replay, (k, v)):
                    c.append(x[i * L:(i + 1) * L].double().numpy(), view.chunk_offsets[slot], live,
                             row)
            slots = view.query_rows_slots if copy_free else view.query_slots
            for i, s in enumerate(slots):
                put(s, i)
            vals = [c.values(row, live) for c in replay]
            ends, kv = view.segments() if copy_free else \
                ([(i + 1) * L for i in range(len(slots))], [view.chunk_offsets[s + 1] for s in slots])
            want, wl = oc.attention(q.double().cpu().numpy(), *vals, ends, kv, scale)
            A, _ = oc.attention(q.double().cpu().numpy(), vals[0], np.abs(vals[1]), ends, kv, scale)
            # as in the attention's own tests; logits here are below 2^6
            tol = BF16_HALF * np.abs(want) + A * 2.0 ** -9 + 2.0 ** -36 * live * np.abs(vals[1]).max()
            assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
            assert np.abs(lse.double().cpu().numpy() - wl).max() <= 2.0 ** -11
            if view.store_to is not None:
                put(view.store_to, 0)
    for i, (codes, sc) in enumerate(((cache.pool.k_codes, cache.pool.k_scale),
                                     (cache.pool.v_codes, cache.pool.v_scale))):
        assert np.array_equal(codes.cpu().numpy(), replay[i].codes)
        assert np.array_equal(sc.cpu().numpy(), replay[i].scale)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_projection_to_attention_round_after_round(fp8):
    """A fused projection's rows, normed and rotated: queries in one call, keys on their way into the
    cache; the bf16 and the FP8 cache against float64 with unquantized keys and values."""
    H, D, L, ps = 2, 128, 45, 16
    axis_pairs = (22, 21, 21)
    win = RollingWindow(L, (1000, 500), 2, ps)
    cache = RollingCache(win, H, D, 1, "cuda", fp8_block=fp8)
    rule = NormRope(rotation_table(64, axis_pairs), axis_pairs=axis_pairs, interleaved=True, eps=1e-6)
    table = rule.table.double().cpu().numpy()
    qw, kw = bf16_weight((D,), 5).cuda(), bf16_weight((D,), 6).cuda()
    stored = {}
    for t in range(7):
        view = win.view(t)
        n = view.t_q
        pos = torch.cat([video_positions(view.chunk_ids[s] * L, L, 3, 5) for s in view.query_slots])
        proj = bf16_rows(n, 3 * H, D, 70 + t).cuda()
        qi, ki, vi = proj[:, :H], proj[:, H:2 * H], proj[:, 2 * H:]
        q = torch.empty(n, H, D, dtype=torch.bfloat16, device="cuda")
        qk_norm_rope(qi, q, None, None, rule, pos, qw)
        out = torch.empty_like(q)
        cache.run_layer(view, 0, q, ki, vi, out, rule=rule, positions=pos, k_weight=kw)
        assert check_status() == WF_OK
        p = pos.cpu().numpy()
        qe = oc.norm_rope(qi.double().cpu().numpy(), qw.double().cpu().numpy(), True, 1e-6, table, p,
                          axis_pairs, True)
        ke = oc.norm_rope(ki.double().cpu().numpy(), kw.double().cpu().numpy(), True, 1e-6, table, p,
                          axis_pairs, True)
        ve = vi.double().cpu().numpy()
        for i, s in enumerate(view.query_slots):
            stored[view.chunk_ids[s]] = (ke[i * L:(i + 1) * L], ve[i * L:(i + 1) * L])
        ka, va = (np.concatenate([stored[c][j] for c in view.chunk_ids]) for j in (0, 1))
        ends = [(i + 1) * L for i in range(len(view.query_slots))]
        want, _ = oc.attention(qe, ka, va, ends, [view.chunk_offsets[s + 1]
                                                  for s in view.query_slots], D ** -0.5)
        err = np.abs(out.double().cpu().numpy() - want)
        rel = np.linalg.norm(err) / np.linalg.norm(want)
        # bf16: q, k and the output rounded, 2^-8 each at most; FP8: keys and values within 2^-4 of
        # their size (half a step of e4m3), 2^-5 on average, which unit-size rows carry into logits
        # of unit size and the output alike
        assert rel <= (2.0 ** -6 if not fp8 else 2.0 ** -4)


def test_layers_share_a_pool_and_calls_may_share_a_stream():
    """Two layers in one pool, two calls at once on two streams with a workspace each, a graph and an
    eager call between: every one gives what it gives alone."""
    H, D, ps, N = 2, 64, 32, 500
    pages = -(-N // ps)
    pool = PagedPoolFp8Block(2 * pages, ps, H, D)
    pt = torch.randperm(2 * pages).int().view(2, pages).cuda()
    off = [0, 333, N]
    layers = [Fp8BlockLayer(pool, pt, i, off, [0, 1], 1) for i in range(2)]
    for i, lay in enumerate(layers):
        lay.append(0, 2, bf16_rows(N, H, D, i).cuda(), bf16_rows(N, H, D, 10 + i).cuda())
    q = [bf16_rows(N - 333, 3 * H, D, 20 + i).cuda() for i in range(2)]
    alone = []
    for lay, x in zip(layers, q):
        alone.append(torch.empty_like(x))
        lay.forward(x, alone[-1])
    need = layers[0].workspace_size(3 * H)
    ws = [torch.empty(max(need, 16), dtype=torch.uint8, device="cuda") for _ in range(3)]
    out = [torch.empty_like(x) for x in q]
    g, gout = torch.cuda.CUDAGraph(), torch.empty_like(q[0])
    with torch.cuda.graph(g):
        layers[0].forward(q[0], gout, workspace=ws[2])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for o in out:
            o.zero_()
        gout.zero_()
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                layers[i].forward(q[i], out[i], workspace=ws[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], alone[0]) and torch.equal(out[1], alone[1])
        assert torch.equal(gout, alone[0])
    assert check_status() == WF_OK



def test_a_decode_step_in_a_graph_between_other_work():
    """Memory copies, fills, other kernels and another stream's work before, between and after the calls of
    a captured step: every call sees what was written before it, replay after replay."""
    Hq, H, D, ps, N = 8, 2, 128, 16, 200
    pages = -(-N // ps)
    rule = NormRope(rotation_table(N, (64,)))
    pool = PagedPoolFp8Block(pages, ps, H, D)
    pt = torch.randperm(pages).int().view(1, -1).cuda()
    proj = torch.zeros(1, Hq + 2 * H, D, dtype=torch.bfloat16, device="cuda")
    host = torch.zeros(proj.shape, dtype=torch.bfloat16).pin_memory()
    q = torch.zeros(1, Hq, D, dtype=torch.bfloat16, device="cuda")
    out, copy = torch.zeros_like(q), torch.zeros_like(q)
    before = Fp8BlockLayer(pool, pt, 0, [0, N - 1], [0], 0)
    before.append(0, 1, bf16_rows(N - 1, H, D, 1).cuda(), bf16_rows(N - 1, H, D, 2).cuda())
    lay = Fp8BlockLayer(pool, pt, 0, [0, N - 1, N], [0, 0], 1)
    pos = torch.full((1, 1), N - 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(lay.workspace_size(Hq), 16), dtype=torch.uint8, device="cuda")

    def step():
        proj.copy_(host, non_blocking=True)                       # a copy, then our kernel
        qk_norm_rope(proj[:, :Hq], q, None, None, rule, pos)
        out.zero_()                                               # a fill, then our kernels
        lay.append(1, 2, proj[:, Hq:Hq + H], proj[:, Hq + H:], rule, pos)
        lay.forward(q, out, workspace=ws)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            copy.copy_(out)                                       # another stream reads the result
            qk_norm_rope(copy, copy, None, None, rule, pos)
        torch.cuda.current_stream().wait_stream(side)
        copy.mul_(2)
    side = torch.cuda.Stream()
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(6):
        host.copy_(bf16_rows(1, Hq + 2 * H, D, 10 + i))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = (q.clone(), out.clone(), copy.clone())
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (q, out, copy)))
        vals = [oc.decode_rows(c.cpu().numpy(), s.cpu().numpy(), pt[0].cpu().numpy(), N)
                for c, s in ((pool.k_codes, pool.k_scale), (pool.v_codes, pool.v_scale))]
        want, _ = oc.attention(q.double().cpu().numpy(), *vals, [1], [N], D ** -0.5)
        assert np.abs(out.double().cpu().numpy() - want).max() <= 2.0 ** -7
    assert check_status() == WF_OK


def test_one_layer_in_two_graphs_and_on_two_streams_without_a_workspace_given():
    """Calls that leave the workspace to the layer: two captured graphs replayed at the same time, calls
    on two other streams beside them, and a larger call afterwards, which must not take the graphs'
    memory."""
    Hq, H, D, ps, N = 16, 4, 128, 16, 4096
    pages = N // ps
    pool = PagedPoolFp8Block(pages, ps, H, D)
    pt = torch.randperm(pages).int().view(1, -1).cuda()
    lay = Fp8BlockLayer(pool, pt, 0, [0, N - 4, N], [0, 0], 1)
    lay.append(0, 2, bf16_rows(N, H, D, 1).cuda(), bf16_rows(N, H, D, 2).cuda())
    q = [bf16_rows(4, Hq, D, 3 + i).cuda() for i in range(4)]
    assert lay.workspace_size(Hq) > 0                             # keys are cut
    want = []
    for x in q:
        want.append(torch.empty_like(x))
        lay.forward(x, want[-1], workspace=torch.empty(lay.workspace_size(Hq), dtype=torch.uint8,
                                                       device="cuda"))
    out = [torch.empty_like(x) for x in q]
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            lay.forward(q[i], out[i])
    streams = [torch.cuda.Stream() for _ in range(4)]
    big = bf16_rows(300, Hq, D, 9).cuda()
    big_out = torch.empty_like(big)
    from block_causal_streaming_b200 import Segments
    seg = Segments([300], [N], N, pages)
    for rnd in range(6):
        for o in out:
            o.zero_()
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        with torch.cuda.stream(streams[2]):
            lay.forward(q[2], out[2])
        lay.forward(q[3], out[3], stream=streams[3])
        if rnd == 2:                                              # a larger workspace from now on
            lay.forward(big, big_out, segments=seg)
            torch.empty(1 << 24, dtype=torch.uint8, device="cuda").fill_(255)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert check_status() == WF_OK
