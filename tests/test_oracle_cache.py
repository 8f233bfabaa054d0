"""Pins of the oracle for the operators around the K/V cache (oracle/cache.py): closed forms,
PyTorch's own e4m3 cast, invariants and a plain softmax."""
import numpy as np
import pytest
import torch

from oracle import cache as oc


def _table(rows, pairs):
    ang = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(pairs) / pairs)
    return np.stack([np.cos(ang), np.sin(ang)], -1)


def test_norm_rows_have_unit_mean_square():
    x = np.random.default_rng(0).normal(size=(3, 2, 64)) * 7
    y = oc.norm_rope(x, eps=0.0)
    assert np.allclose((y ** 2).mean(-1), 1, rtol=1e-13)
    w = np.random.default_rng(1).normal(size=(2, 64))
    assert np.allclose(oc.norm_rope(x, weight=w, eps=0.0), y * w, rtol=1e-14)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product_and_depends_on_distance_alone(interleaved):
    rng = np.random.default_rng(2)
    D, pairs, table = 64, 32, _table(100, 32)
    a, b = rng.normal(size=(1, 1, D)), rng.normal(size=(1, 1, D))

    def at(x, p):
        return oc.norm_rope(x, norm=False, table=table, positions=[[p]], axis_pairs=(pairs,),
                            interleaved=interleaved)[0, 0]
    z = a[0, 0].reshape(pairs, 2) if interleaved else a[0, 0].reshape(2, pairs).T
    want = (z[:, 0] + 1j * z[:, 1]) * np.exp(1j * 5 * 10000.0 ** (-np.arange(pairs) / pairs))
    got = at(a, 5)
    got = got.reshape(pairs, 2) if interleaved else got.reshape(2, pairs).T
    assert np.allclose(got[:, 0] + 1j * got[:, 1], want, rtol=1e-12)
    assert np.isclose(at(a, 30) @ at(b, 23), at(a, 67) @ at(b, 60), rtol=1e-10)


def test_axes_turn_their_own_pairs():
    x = np.random.default_rng(3).normal(size=(1, 1, 64))
    table = _table(50, 32)
    y = oc.norm_rope(x, norm=False, table=table, positions=[[0, 7, 0]], axis_pairs=(12, 10, 10),
                     interleaved=True)
    same = np.isclose(y, x, rtol=0, atol=0).reshape(32, 2).all(1)
    assert same[:12].all() and same[22:].all() and not same[12:22].any()


def test_encoder_equals_the_library_cast():
    y = np.random.default_rng(4).normal(size=20000) * np.exp(np.random.default_rng(5).normal(
        size=20000) * 3)
    y = np.clip(y.astype(np.float32), -448, 448)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oc.encode(y), want)
    assert oc.encode([np.nan])[0] == 0x7F and oc.encode([1e9])[0] == 0x7E


@pytest.mark.parametrize("top, e", [(448.0, 0), (448.0 * (1 + 2.0 ** -23), 1), (224.0, -1),
                                    (1.75, -8), (1.0, -8), (2.0 ** -0.0, -8), (0.0, -100),
                                    (1e-36, -100), (3.0e38, 119)])
def test_scale_is_the_least_power_of_two(top, e):
    assert oc.scale_exponent(top) == e
    if -100 < e < 119:
        assert top <= 448 * 2.0 ** e and top > 448 * 2.0 ** (e - 1)


def test_single_token_appends_give_what_one_append_gives():
    """Values in e4m3's normal range of every scale they pass: nothing is rounded twice."""
    rng = np.random.default_rng(6)
    x = np.sign(rng.normal(size=(40, 2, 64))) * rng.uniform(1, 3, size=(40, 2, 64))
    pages = [2, 0, 1]
    bulk, single = oc.Fp8Cache(3, 16, 2, 64), oc.Fp8Cache(3, 16, 2, 64)
    bulk.append(x, 0, 40, pages)
    for t in range(40):
        single.append(x[t:t + 1], t, t + 1, pages)
    assert np.array_equal(bulk.codes, single.codes) and np.array_equal(bulk.scale, single.scale)
    err = np.abs(bulk.values(pages, 40) - x)
    assert (err <= 2.0 ** -4 * np.abs(x)).all()


def test_append_keeps_live_rows_and_leaves_dead_ones():
    rng = np.random.default_rng(7)
    c = oc.Fp8Cache(1, 32, 1, 64)
    c.codes[:] = 0x7F                                     # dead rows hold anything
    x = rng.uniform(1, 2, size=(20, 1, 64))
    c.append(x, 0, 20, [0])
    assert (c.codes[0, 20:] == 0x7F).all()
    big = np.full((3, 1, 64), 100.0)
    before = c.values([0], 20)
    c.append(big, 5, 20, [0])
    after = c.values([0], 20)
    assert np.array_equal(after[5:8], oc.e4m3_decode(oc.encode(big / 0.25)) * 0.25)
    keep = [t for t in range(20) if not 5 <= t < 8]
    # re-coded under the larger scale 2^-2: exact down to its smallest normal, 2^-8
    assert np.array_equal(after[keep], before[keep])


def test_attention_matches_a_plain_softmax_and_empty_rows_are_zero():
    rng = np.random.default_rng(8)
    q, k, v = rng.normal(size=(5, 4, 64)), rng.normal(size=(9, 2, 64)), rng.normal(size=(9, 2, 64))
    out, lse = oc.attention(q, k, v, [1, 3, 5], [0, 4, 9], 0.2)
    assert (out[0] == 0).all() and (lse[:, 0] == -np.inf).all()
    t = torch.from_numpy(k[:4, 1]) @ torch.from_numpy(q[2, 3]) * 0.2
    assert np.allclose(out[2, 3], (torch.softmax(t, 0) @ torch.from_numpy(v[:4, 1])).numpy())
    assert np.isclose(lse[3, 2], torch.logsumexp(t, 0).item())
    assert np.allclose(oc.attention(q, k, np.ones_like(v), [5], [9], 0.2)[0], 1)
