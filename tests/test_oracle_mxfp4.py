"""Pins of the MXFP4 oracle: hand cases, brute force against another rounding, bounds and relations."""
import numpy as np
import pytest

from oracle import mxfp4 as o4


def group(*v):
    g = np.zeros(32)
    g[:len(v)] = v
    return g


def test_hand_groups():
    # amax 6: scale 1; ties: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    q, b = o4.quantize_groups(group(6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5, -0.2))
    assert b == 127 and q[:10].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 14, 8]
    # amax just under 8 keeps scale 1 and saturates; 8 is 4 x 2
    assert [int(o4.quantize_groups(group(v))[1]) for v in (7.99, 8.0, 4.0, 3.99)] == [127, 128, 127, 126]
    assert o4.quantize_groups(group(7.99))[0][0] == 7 and o4.quantize_groups(group(8.0))[0][0] == 6
    q, b = o4.quantize_groups(group(0.0, -0.0))
    assert b == 0 and q[0] == 0 and q[1] == 8
    # the clamp: 2^-125 has e = -127, 2^-126 is 2 of it, 2^-130 rounds to nothing
    assert [int(o4.quantize_groups(group(2.0 ** -k))[1]) for k in (124, 125, 126, 130)] == [1, 0, 0, 0]
    assert o4.quantize_groups(group(2.0 ** -126))[0][0] == 4 and o4.quantize_groups(group(2.0 ** -130))[0][0] == 0
    assert o4.quantize_groups(group(2.0 ** 127 * 1.99))[1] == 252
    for bad in (np.nan, np.inf, -np.inf):
        assert o4.quantize_groups(group(1.0, bad))[1] == 255


def test_every_step_against_rounding_by_steps():
    v = np.concatenate([np.arange(0, 8, 1 / 256), -np.arange(0, 8, 1 / 256)])
    m = np.abs(v)
    step = np.where(m < 2, 0.5, np.where(m < 4, 1.0, 2.0))
    want = np.minimum(np.round(m / step) * step, 6.0)
    c = o4.to_e2m1(v)
    assert np.array_equal(np.abs(o4.e2m1_to_f64(c)), want)
    assert np.array_equal(c >= 8, np.signbit(v))


@pytest.mark.parametrize("rows,K,e4m3", [(1, 1, False), (3, 127, False), (5, 128, True), (4, 300, False), (2, 129, True)])
def test_operand_reads_back_within_a_step(rows, K, e4m3):
    rng = np.random.default_rng(rows * 1000 + K)
    v = rng.standard_normal((rows, K)) * 2.0 ** rng.integers(-20, 20, (rows, 1))
    q, s = o4.operand(v, e4m3)
    P = -(-K // 128)
    assert q.shape == ((2 if e4m3 else 1) * P, rows, 64) and s.shape == (P, rows, 4)
    r = o4.values(q, s)
    assert np.array_equal(r[:, K:], np.zeros((rows, 128 * P - K)))
    for g in range(-(-K // 32)):
        a, b = v[:, 32 * g:min(K, 32 * g + 32)], r[:, 32 * g:min(K, 32 * g + 32)]
        amax = np.abs(a).max(1, keepdims=True)
        # amax is in [4, 8) ([256, 512)) of the scale: half the widest step, or the saturation's 2 (64)
        assert (np.abs(a - b) <= amax * (2.0 / 8 if not e4m3 else 64.0 / 512)).all()
    # scaling by a power of two scales the values, the sign flips with the sign
    assert np.array_equal(o4.values(*o4.operand(v * 8, e4m3)), 8 * r)
    assert np.array_equal(o4.values(*o4.operand(-v, e4m3)), -r)


def test_nibbles_and_planes():
    v = np.zeros((2, 200))
    v[1, 0], v[1, 1], v[1, 130] = 6.0, -4.0, 3.0
    q, s = o4.operand(v)
    assert q[0, 1, 0] == 0xE7 and q[0, 0].sum() == 0     # k = 0 low, k = 1 high
    assert q[1, 1, 1] == 0x07 and s[1, 1, 0] == 126      # amax 3: e = -1, 3 / 0.5 = 6
    assert s[0, 1].tolist() == [127, 0, 0, 0]


@pytest.mark.parametrize("wrong", ["half_up", "nibbles", "no_saturation"])
def test_planted_mistakes_fail(wrong, monkeypatch):
    if wrong == "half_up":
        monkeypatch.setattr(o4, "to_e2m1", lambda v: (np.searchsorted([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.abs(v), side="right")
                                                      + np.where(np.signbit(v), 8, 0)).astype(np.uint8))
        with pytest.raises(AssertionError):
            test_every_step_against_rounding_by_steps()
    elif wrong == "nibbles":
        real = o4.operand
        monkeypatch.setattr(o4, "operand", lambda v, e=False: (lambda q, s: ((q >> 4) | (q << 4), s))(*real(v, e)))
        with pytest.raises(AssertionError):
            test_nibbles_and_planes()
    else:
        real = o4.scale_byte
        monkeypatch.setattr(o4, "scale_byte", lambda a, emax: real(a, emax) - 1)
        with pytest.raises(AssertionError):
            test_hand_groups()
