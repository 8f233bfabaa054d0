"""The largest sequences of the FP8 cache attention, on the host: token counts past what the kernels' 32-bit
indices hold are refused before anything is launched."""
import ctypes

import pytest

from block_causal_streaming_b200 import build as wf_build

wf_build.build()
from block_causal_streaming_b200 import _abi  # noqa: E402

FAKE = 0x10000      # an aligned address that is never read: the checks must answer first


def _call(keys, kv, page=4096):
    pages = -(-keys // page)
    pool = _abi.KvPoolFp8Block(FAKE, FAKE, FAKE, FAKE, 8, page, 2, 128)
    seg = _abi.Segments([5], [kv], keys, pages)
    # without a query pointer a call that passes the checks of its segments is refused for that
    return _abi.lib.wf_attn_forward_fp8_block(None, 2, ctypes.byref(pool), FAKE, seg.ref, 0.1, None, None,
                                              1, None, 0, None)


@pytest.mark.parametrize("keys, want", [
    (2 ** 31 - 1, _abi.WF_ERR_SHAPE), (2 ** 31 - 16, _abi.WF_ERR_SHAPE), (2 ** 31 - 4096, _abi.WF_ERR_SHAPE),
    (2 ** 31 - 4097, _abi.WF_ERR_INVALID_ARG), (2 ** 30, _abi.WF_ERR_INVALID_ARG)])
def test_keys_past_32_bit_indices_are_refused(keys, want):
    assert _call(keys, keys) == want
    assert _call(keys, 7) == want
