"""The cache operators on the host: argument checks of the C ABI (which answer before anything touches a
GPU) and of the binding, which keeps tensors of the wrong shape, layout or place from being read."""
import ctypes

import pytest
import torch

from block_causal_streaming_b200 import build as wf_build

wf_build.build()
from block_causal_streaming_b200 import _abi  # noqa: E402
from block_causal_streaming_b200.layer import (Fp8BlockLayer, PagedPoolFp8Block,  # noqa: E402
                                               rotation_table, video_positions)
from block_causal_streaming_b200.window import RollingCache, RollingWindow  # noqa: E402

FAKE = 0x10000      # an aligned address that is never read: the checks must answer first
ARG, SHAPE, CAP = _abi.WF_ERR_INVALID_ARG, _abi.WF_ERR_SHAPE, _abi.WF_ERR_CAPACITY


def _rule(**kw):
    d = dict(norm=1, eps=1e-6, weight_per_head=0, cos_sin=FAKE, table_rows=10, num_axes=1,
             axis_pairs=(ctypes.c_int32 * 3)(64, 0, 0), interleaved=0)
    d.update(kw)
    return _abi.NormRopeC(*[d[n] for n, _ in _abi.NormRopeC._fields_])


def _pairs(*n):
    return (ctypes.c_int32 * 3)(*(list(n) + [0, 0])[:3])


def _qk(rule=None, q=FAKE, qs=1024, qo=FAKE, qw=FAKE, hq=8, k=FAKE, ks=1024, ko=FAKE, kw=FAKE, hk=2,
        tokens=5, D=128, pos=FAKE):
    r = _rule() if rule is None else rule
    return _abi.lib.wf_qk_norm_rope(q, qs, qo, qw, hq, k, ks, ko, kw, hk, tokens, D, pos,
                                    ctypes.byref(r) if r != 0 else None, None)


@pytest.mark.parametrize("want, kw", [
    (ARG, dict(rule=0)), (ARG, dict(q=None)), (ARG, dict(q=FAKE + 8)), (ARG, dict(qo=None)),
    (ARG, dict(qo=FAKE + 2)), (ARG, dict(qs=1023)), (ARG, dict(qs=1020)), (ARG, dict(qs=1016)),
    (ARG, dict(qw=FAKE + 8)), (ARG, dict(k=None)), (ARG, dict(ko=FAKE + 8)), (ARG, dict(ks=0)),
    (ARG, dict(kw=FAKE + 2)), (ARG, dict(pos=None)), (ARG, dict(pos=FAKE + 2)),
    (SHAPE, dict(D=96)), (SHAPE, dict(hq=0)), (SHAPE, dict(hk=-1)), (SHAPE, dict(tokens=-1)),
    (ARG, dict(rule=_rule(norm=2))), (ARG, dict(rule=_rule(eps=-1.0))),
    (ARG, dict(rule=_rule(eps=float("nan")))), (ARG, dict(rule=_rule(eps=float("inf")))),
    (ARG, dict(rule=_rule(weight_per_head=2))), (ARG, dict(rule=_rule(interleaved=2))),
    (ARG, dict(rule=_rule(cos_sin=FAKE + 8))), (SHAPE, dict(rule=_rule(table_rows=0))),
    (SHAPE, dict(rule=_rule(num_axes=0))), (SHAPE, dict(rule=_rule(num_axes=4))),
    (SHAPE, dict(rule=_rule(axis_pairs=_pairs(65)))), (SHAPE, dict(rule=_rule(axis_pairs=_pairs(30)))),
    (SHAPE, dict(rule=_rule(axis_pairs=_pairs(0)))),
    (SHAPE, dict(rule=_rule(num_axes=2, axis_pairs=_pairs(68, -4)))),
    (SHAPE, dict(rule=_rule(num_axes=3, axis_pairs=_pairs(2 ** 31 - 1, 2 ** 31 - 1, 6)))),
])
def test_qk_refusals(want, kw):
    assert _qk(**kw) == want


def test_qk_without_tokens_is_a_no_op():
    assert _qk(tokens=0, q=None, qo=None, k=None, ko=None, pos=None) == _abi.WF_OK


def _pool(cls, **kw):
    d = dict(k_pool=FAKE, v_pool=FAKE, k_codes=FAKE, v_codes=FAKE, k_scale=FAKE, v_scale=FAKE,
             num_pages=8, page_size=64, num_heads=2, head_dim=128)
    d.update(kw)
    return cls(*[d[n] for n, _ in cls._fields_])


def _append(fp8, pool=None, begin=1, end=2, k=FAKE, ks=256, v=FAKE, vs=256, w=FAKE, pos=FAKE, rule=None,
            pt=FAKE, off=(0, 64, 200), pages=8, layer=0, stage=None):
    cls = _abi.KvPoolFp8Block if fp8 else _abi.KvPool
    fn = _abi.lib.wf_kv_append_fp8_block if fp8 else _abi.lib.wf_kv_append_rope
    wf = _abi.WavefrontDesc(off, stage or [0] * (len(off) - 1), 1, pages)
    r = _rule() if rule is None else rule
    p = _pool(cls) if pool is None else pool
    return fn(ctypes.byref(p) if p != 0 else None, layer, begin, end, k, ks, v, vs, w, pos,
              ctypes.byref(r) if r != 0 else None, pt, wf.ref, None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("want, kw", [
    (ARG, dict(pool=0)), (ARG, dict(begin=-1)), (ARG, dict(begin=1, end=1)), (ARG, dict(begin=2, end=1)),
    (ARG, dict(end=3)), (ARG, dict(layer=-1)), (ARG, dict(pt=None)), (ARG, dict(pt=FAKE + 2)),
    (ARG, dict(k=None)), (ARG, dict(v=None)), (ARG, dict(k=FAKE + 4)), (ARG, dict(v=FAKE + 8)),
    (ARG, dict(ks=255)), (ARG, dict(vs=248)), (ARG, dict(w=FAKE + 8)), (ARG, dict(pos=None)),
    (CAP, dict(off=(0, 64, 520))), (SHAPE, dict(off=(0, 64, 60))), (SHAPE, dict(off=(1, 64, 100))),
    (_abi.WF_ERR_STAGE_ORDER, dict(stage=[5, 1])),
    (SHAPE, dict(rule=_rule(axis_pairs=_pairs(68)))),
])
def test_append_refusals(fp8, want, kw):
    assert _append(fp8, **kw) == want


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("want, kw", [
    (SHAPE, dict(num_pages=0)), (SHAPE, dict(page_size=24)), (SHAPE, dict(page_size=0)),
    (SHAPE, dict(num_heads=0)), (SHAPE, dict(head_dim=96)),
    (SHAPE, dict(num_pages=2 ** 26, page_size=64)),
])
def test_append_pool_refusals(fp8, want, kw):
    assert _append(fp8, pool=_pool(_abi.KvPoolFp8Block if fp8 else _abi.KvPool, **kw)) == want


def test_append_special_cases():
    for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
        assert _append(True, pool=_pool(_abi.KvPoolFp8Block, **{name: None})) == ARG
    assert _append(True, pool=_pool(_abi.KvPoolFp8Block, v_codes=FAKE + 8)) == ARG
    assert _append(False, rule=0) == ARG
    for fp8 in (False, True):
        assert _append(fp8, off=(0, 64, 64), k=None, v=None, pos=None) == _abi.WF_OK


def _attn(q=FAKE, hq=4, pool=None, pt=FAKE, ends=(3, 7), kv=(10, 100), keys=100, pages=8, scale=0.1,
          out=FAKE, lse=None, splits=0, ws=None, ws_bytes=0):
    seg = _abi.Segments(list(ends), list(kv), keys, pages)
    p = _pool(_abi.KvPoolFp8Block) if pool is None else pool
    return _abi.lib.wf_attn_forward_fp8_block(q, hq, ctypes.byref(p) if p != 0 else None, pt, seg.ref,
                                              scale, out, lse, splits, ws, ws_bytes, None)


@pytest.mark.parametrize("want, kw", [
    (ARG, dict(pool=0)), (ARG, dict(pool=_pool(_abi.KvPoolFp8Block, v_scale=None))),
    (SHAPE, dict(pool=_pool(_abi.KvPoolFp8Block, page_size=8))),
    (SHAPE, dict(hq=3)), (SHAPE, dict(hq=0)), (SHAPE, dict(hq=-2)),
    (SHAPE, dict(ends=(), kv=())), (SHAPE, dict(ends=(3, 2))), (SHAPE, dict(ends=(-1, 2))),
    (SHAPE, dict(kv=(-1, 5))), (SHAPE, dict(kv=(10, 101))), (SHAPE, dict(keys=-1, kv=(0, 0))),
    (SHAPE, dict(ends=range(1, 66), kv=[1] * 65)),
    (CAP, dict(keys=513, kv=(1, 513))), (CAP, dict(pages=1)), (CAP, dict(pages=-1)),
    (ARG, dict(scale=0.0)), (ARG, dict(scale=-1.0)), (ARG, dict(scale=float("nan"))),
    (ARG, dict(scale=float("inf"))), (ARG, dict(splits=-1)),
    (ARG, dict(q=None)), (ARG, dict(q=FAKE + 8)), (ARG, dict(out=None)), (ARG, dict(out=FAKE + 4)),
    (ARG, dict(pt=None)), (ARG, dict(pt=FAKE + 1)), (ARG, dict(lse=FAKE + 2)),
])
def test_attention_refusals(want, kw):
    assert _attn(**kw) == want


def test_attention_without_rows_is_a_no_op():
    assert _attn(ends=(0, 0), kv=(5, 5), q=None, out=None, pt=None) == _abi.WF_OK


def test_workspace_of_uncut_or_wrong_calls_is_empty():
    seg = _abi.Segments([100], [1000], 1000, 70)
    assert _abi.attn_fp8_block_workspace_size(seg, 8, 8, 128, 1) == 0
    for args in ((3, 2, 128, 0), (0, 1, 128, 0), (8, 8, 96, 0), (8, 8, 128, -1)):
        assert _abi.attn_fp8_block_workspace_size(seg, *args) == 0


# ------------------------------------------------------------------------------ the binding
class _FakeLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    lib = _FakeLib()
    _abi._lib_torch()
    monkeypatch.setattr(_abi, "lib", lib)
    monkeypatch.setattr(_abi, "_current_device", lambda: -1)        # where CPU tensors are
    monkeypatch.setattr(_abi, "_raw_stream", lambda s, d: None)
    monkeypatch.setattr(_abi, "_check_tensor", lambda *a: None)
    return lib


H, D, PS = 2, 64, 16
OFF = [0, 40, 90, 130]


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _setup():
    rule = _abi.NormRope(rotation_table(50, (32,), device="cpu"))
    wf = _abi.WavefrontDesc(OFF, [0, 1, 2], 1, 9)
    pt = torch.arange(18, dtype=torch.int32).view(2, 9)
    pool = PagedPoolFp8Block(18, PS, H, D, "cpu")
    return rule, wf, pt, pool


def test_valid_calls_pass(fake):
    rule, wf, pt, pool = _setup()
    pos = torch.zeros(90, 1, dtype=torch.int32)
    proj = _bf(90, 4 + 2 * H, D)
    q, k, v = proj.split([4, H, H], 1)
    _abi.qk_norm_rope(q, _bf(90, 4, D), k, _bf(90, H, D), rule, pos, _bf(D), _bf(D))
    _abi.qk_norm_rope(q, _bf(90, 4, D), None, None, rule, pos)
    x = _bf(90, 4, D)
    _abi.qk_norm_rope(x, x, None, None, rule, pos)                   # in place
    _abi.qk_norm_rope(_bf(0, 4, D), _bf(0, 4, D), None, None, rule, pos[:0])
    _abi.qk_norm_rope(q, _bf(90, 4, D), None, None, _abi.NormRope(None, weight_per_head=True), None,
                      _bf(4, D))
    kp = _bf(18, PS, H, D)
    _abi.kv_append_rope(kp, kp.clone(), 1, 1, 3, k, v, pt, wf, rule, pos)
    _abi.kv_append_fp8_block(*pool.tensors, 1, 1, 3, k, v, pt, wf, rule, pos, _bf(D))
    _abi.kv_append_fp8_block(*pool.tensors, 0, 1, 3, k, v, pt, wf)
    lay = Fp8BlockLayer(pool, pt, 1, OFF, [0, 1, 2], 1)
    lay.append(0, 1, _bf(40, H, D), _bf(40, H, D))
    lay.forward(_bf(90, 4, D), _bf(90, 4, D), lse=torch.zeros(4, 90))
    for copy_free in (False, True):
        for fp8 in (False, True):
            win = RollingWindow(24, [1000, 500], 2, 16, copy_free=copy_free)
            cache = RollingCache(win, H, D, 2, "cpu", fp8_block=fp8)
            for t in range(7):
                view = win.view(t)
                n = 24 * len(view.query_rows_slots)
                kw = dict(rule=rule, positions=torch.zeros(n, 1, dtype=torch.int32))
                if not fp8:
                    continue
                cache.run_layer(view, 1, _bf(n, H, D), _bf(n, H, D), _bf(n, H, D), _bf(n, H, D), **kw)
    assert {"wf_qk_norm_rope", "wf_kv_append_rope", "wf_kv_append_fp8_block",
            "wf_attn_forward_fp8_block"} <= set(fake.calls)


def test_malformed_calls_raise_before_any_launch(fake):
    rule, wf, pt, pool = _setup()
    c = pool.tensors
    pos, q, k = torch.zeros(90, 1, dtype=torch.int32), _bf(90, 4, D), _bf(90, H, D)
    kp = _bf(18, PS, H, D)
    seg = _abi.Segments([90], [130], 130, 9)
    per_head = _abi.NormRope(rule.table, weight_per_head=True)
    big = _bf(200, 4, D)

    def qk(q=q, qo=None, k=k, ko=None, rule=rule, pos=pos, **kw):
        _abi.qk_norm_rope(q, _bf(*q.shape) if qo is None else qo, k,
                          _bf(*k.shape) if ko is None and k is not None else ko, rule, pos, **kw)

    def app(begin=1, end=3, k=k, v=k, pt=pt, layer=0, pos=pos, rule=rule, pools=(kp, kp), **kw):
        _abi.kv_append_rope(*pools, layer, begin, end, k, v, pt, wf, rule, pos, **kw)

    def app8(begin=1, end=3, k=k, v=k, pt=pt, layer=0, pos=pos, rule=rule, pools=c, **kw):
        _abi.kv_append_fp8_block(*pools, layer, begin, end, k, v, pt, wf, rule, pos, **kw)

    def attn(q=q, pools=c, row=pt[0], seg=seg, out=None, lse=None, ws=None):
        _abi.attn_forward_fp8_block(q, *pools, row, seg, 0.1, _bf(*q.shape) if out is None else out, lse,
                                    0, ws)

    bad = [
        lambda: qk(q=_bf(90, D)), lambda: qk(qo=_bf(89, 4, D)), lambda: qk(qo=_bf(4, 90, D).transpose(0, 1)),
        lambda: qk(q=_bf(4, 90, D).transpose(0, 1)), lambda: qk(q=_bf(90, 4, 2 * D)[..., ::2]),
        lambda: qk(q=_bf(1, 4, D).expand(90, 4, D)), lambda: qk(q=_bf(90 * (4 * D + 4)).as_strided(
            (90, 4, D), (4 * D + 4, D, 1))),
        lambda: qk(k=None, ko=_bf(90, H, D)), lambda: qk(k=_bf(89, H, D), ko=_bf(89, H, D)),
        lambda: qk(pos=None), lambda: qk(pos=pos[:89]), lambda: qk(pos=torch.zeros(90, 3).int()),
        lambda: qk(q_weight=_bf(D + 1)), lambda: qk(q_weight=_bf(4, D)),
        lambda: qk(rule=per_head, q_weight=_bf(D)),
        lambda: qk(rule=_abi.NormRope(rule.table, norm=False), q_weight=_bf(D)),
        lambda: qk(rule=_abi.NormRope(None)), lambda: qk(q=_bf(90, 4, 32), k=_bf(90, H, 32)),
        # outputs over inputs, in part or the wrong one's
        lambda: qk(q=big[:90], qo=big[1:91]), lambda: qk(q=big[:, :2][:90], qo=big.view(-1)[:90 * 2 * D]
                                                        .view(90, 2, D)),
        lambda: qk(q=big[:90], qo=big[:90], k=big[100:190], ko=big[50:140]),
        lambda: qk(qo=big[:90], ko=big.view(-1)[:90 * H * D].view(90, H, D)),
        lambda: app(begin=0), lambda: app(end=4), lambda: app(begin=-1, end=1), lambda: app(begin=2, end=2),
        lambda: app(k=_bf(91, H, D)), lambda: app(v=_bf(90, H + 1, D)), lambda: app(layer=2),
        lambda: app(pt=pt[:, :8]), lambda: app(pt=pt[0]), lambda: app(pools=(kp, kp[:9])),
        lambda: app(pools=(kp[0], kp[0])), lambda: app(pos=pos[:5]), lambda: app(k_weight=_bf(3)),
        lambda: app(pools=(kp.transpose(0, 1), kp.transpose(0, 1))),
        lambda: app8(begin=0), lambda: app8(k=_bf(91, H, D)), lambda: app8(layer=-1),
        lambda: app8(pools=(c[0], c[1][:9], c[2], c[3])), lambda: app8(pools=(c[0], c[1], c[2][:9], c[3])),
        lambda: app8(pools=(c[0], c[1], c[2], c[3].view(18, H, 1))), lambda: app8(rule=None),
        lambda: app8(rule=None, pos=None, k_weight=_bf(D)),
        lambda: attn(q=_bf(89, 4, D)), lambda: attn(q=_bf(90, 3, D)), lambda: attn(q=_bf(90, 4, 2 * D)),
        lambda: attn(out=_bf(90, 2, D)), lambda: attn(lse=torch.zeros(90, 4)), lambda: attn(row=pt[0][:8]),
        lambda: attn(row=pt), lambda: attn(q=_bf(4, 90, D).transpose(0, 1)),
        lambda: attn(pools=(c[0], c[1], c[2], c[3][:, :0])),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} passed")
    wrong_type = [
        lambda: qk(q=torch.zeros(90, 4, D)), lambda: qk(qo=torch.zeros(90, 4, D)),
        lambda: qk(pos=pos.long()), lambda: qk(q_weight=torch.zeros(D)), lambda: app(v=torch.zeros(90, H, D)),
        lambda: app(pt=pt.long()), lambda: app8(pools=(c[0].to(torch.int8),) + c[1:]),
        lambda: attn(q=torch.zeros(90, 4, D)), lambda: attn(lse=_bf(4, 90)), lambda: attn(row=pt[0].long()),
        lambda: attn(ws=torch.zeros(100)),
    ]
    for f in wrong_type:
        with pytest.raises(TypeError):
            f()
    assert fake.calls == []


def test_tensors_of_another_device_are_refused(fake, monkeypatch):
    """The launch goes to the current device: nothing else's memory is handed to it."""
    rule, wf, pt, pool = _setup()
    monkeypatch.setattr(_abi, "_current_device", lambda: 0)
    pos, q, k = torch.zeros(90, 1, dtype=torch.int32), _bf(90, 4, D), _bf(90, H, D)
    for f in (lambda: _abi.qk_norm_rope(q, _bf(90, 4, D), None, None, rule, pos),
              lambda: _abi.kv_append_rope(_bf(18, PS, H, D), _bf(18, PS, H, D), 0, 1, 3, k, k, pt, wf, rule,
                                          pos),
              lambda: _abi.kv_append_fp8_block(*pool.tensors, 0, 1, 3, k, k, pt, wf),
              lambda: _abi.attn_forward_fp8_block(q, *pool.tensors, pt[0],
                                                  _abi.Segments([90], [130], 130, 9), 0.1, q.clone())):
        with pytest.raises(ValueError, match="current CUDA device"):
            f()
    assert fake.calls == []


def test_norm_rope_and_helpers():
    table = rotation_table(7, (22, 21, 21), device="cpu")
    assert table.shape == (7, 64, 2) and table.dtype == torch.float32
    assert torch.equal(table[0, :, 0], torch.ones(64)) and torch.equal(table[0, :, 1], torch.zeros(64))
    assert torch.allclose(table[3, 22], torch.tensor([-0.9899925, 0.1411200]))   # cos 3, sin 3
    pos = video_positions(1560, 3, 30, 52, device="cpu")
    assert pos.tolist() == [[1, 0, 0], [1, 0, 1], [1, 0, 2]]
    assert video_positions(51, 2, 30, 52, device="cpu").tolist() == [[0, 0, 51], [0, 1, 0]]
    with pytest.raises(ValueError):
        _abi.NormRope(torch.zeros(3, 4))
    with pytest.raises(ValueError):
        PagedPoolFp8Block(2, 24, 1, 64, "cpu")
    with pytest.raises(ValueError):
        RollingCache(RollingWindow(24, [1000], 1, 16), 1, 64, device="cpu", fill=1.0, fp8_block=True)


def test_norm_rope_axis_pairs(fake):
    table = rotation_table(7, (22, 21, 21), device="cpu")
    for pairs in ((60,), (22, 21), (1, 2, 3, 58), (65, -1), ()):
        with pytest.raises(ValueError):
            _abi.NormRope(table, axis_pairs=pairs)
    r = _abi.NormRope(table, axis_pairs=(22, 21, 21), interleaved=True, norm=False, eps=0.5)
    assert (r.c.norm, r.c.num_axes, list(r.c.axis_pairs), r.c.interleaved, r.c.table_rows) == \
        (0, 3, [22, 21, 21], 1, 7)
