"""Rolling windows in the FP8 cache, on the host: which appends a round makes, and what it refuses."""
import pytest
import torch

from block_causal_streaming_b200 import build as wf_build

wf_build.build()
from block_causal_streaming_b200 import _abi  # noqa: E402
from block_causal_streaming_b200.window import RollingCache, RollingWindow  # noqa: E402

H, D, L = 2, 64, 24


class _FakeLib:
    def __init__(self, real):
        self.appends, self._real = [], real

    def __getattr__(self, name):
        if name.startswith("wf_window"):                    # the planner runs on the host
            return getattr(self._real, name)

        def call(*args):
            if name in ("wf_kv_append_fp8_block", "wf_kv_append_rope"):
                self.appends.append((args[2], args[3]))
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    lib = _FakeLib(_abi.lib)
    _abi._lib_torch()
    monkeypatch.setattr(_abi, "lib", lib)
    monkeypatch.setattr(_abi, "_current_device", lambda: -1)
    monkeypatch.setattr(_abi, "_raw_stream", lambda s, d: None)
    monkeypatch.setattr(_abi, "_check_tensor", lambda *a: None)
    return lib


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("copy_free", [False, True])
@pytest.mark.parametrize("runs", [False, True])
def test_appends_of_a_round(fake, copy_free, runs):
    """Every query chunk is appended once, in order; with append_runs consecutive slots in one call."""
    win = RollingWindow(L, [1000, 500, 250], 2, 16, copy_free=copy_free)
    cache = RollingCache(win, H, D, 1, "cpu", fp8_block=True, append_runs=runs)
    for view in [win.view(t) for t in range(9)]:
        fake.appends.clear()
        slots = view.query_rows_slots
        x = _bf(L * len(slots), H, D)
        cache.run_layer(view, 0, x, x.clone(), x.clone(), x.clone())
        done = list(fake.appends)
        if view.store_to is not None:
            assert done.pop() == (view.store_to, view.store_to + 1)
        assert [s for a, b in done for s in range(a, b)] == slots
        if not runs:
            assert all(b == a + 1 for a, b in done)
        else:
            assert all(done[i][1] != done[i + 1][0] for i in range(len(done) - 1))
            assert len(done) <= (2 if copy_free else 1)


def test_append_runs_is_for_the_fp8_cache():
    win = RollingWindow(L, [1000], 1, 16)
    with pytest.raises(ValueError, match="append_runs"):
        RollingCache(win, H, D, 1, "cpu", append_runs=True)
    RollingCache(win, H, D, 1, "cpu", fp8_block=True, append_runs=True)


@pytest.mark.parametrize("copy_free", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_positions_and_weights_without_a_rule_are_refused(fake, fp8, copy_free):
    """They would be left out: the keys would go into the cache neither normed nor turned."""
    win = RollingWindow(L, [1000, 500], 2, 16, copy_free=copy_free)
    cache = RollingCache(win, H, D, 1, "cpu", fp8_block=fp8)
    view = win.view(6)
    n = L * len(view.query_rows_slots)
    x = _bf(n, H, D)
    for kw in (dict(positions=torch.zeros(n, 1, dtype=torch.int32)), dict(k_weight=_bf(D)),
               dict(positions=torch.zeros(n, 1, dtype=torch.int32), k_weight=_bf(D))):
        with pytest.raises(ValueError, match="rule"):
            cache.run_layer(view, 0, x, x.clone(), x.clone(), x.clone(), **kw)
    assert fake.appends == []
