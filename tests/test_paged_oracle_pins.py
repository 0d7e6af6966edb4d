"""Pins of oracle/paged.py: the norm and rotation against complex numbers, rotation
matrices and their invariants, 4-bit rows against their error bound, paged rows against
plain indexing, attention over pages against the padded oracle."""
import numpy as np
import pytest

from oracle import attention, paged


def freqs(R):
    return 10000.0 ** (-2 * np.arange(R // 2) / R)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("R,D", [(64, 64), (16, 64), (128, 256)])
def test_rotation_is_a_complex_product(R, D, inter):
    rng = np.random.default_rng(1)
    x, f = rng.standard_normal(D), freqs(R)
    out, _ = paged.turn(x, None, 0.0, 77, f, inter)
    a, b = (np.arange(0, R, 2), np.arange(1, R, 2)) if inter else (np.arange(R // 2), np.arange(R // 2, R))
    z = (x[a] + 1j * x[b]) * np.exp(1j * 77 * f)
    assert np.allclose(out[a], z.real, atol=1e-12) and np.allclose(out[b], z.imag, atol=1e-12)
    assert np.array_equal(out[R:], x[R:])
    assert np.isclose(np.linalg.norm(out), np.linalg.norm(x))


def test_scores_depend_on_distance_only():
    rng = np.random.default_rng(2)
    q, k, f = rng.standard_normal(64), rng.standard_normal(64), freqs(64)

    def score(i, j):
        return paged.turn(q, None, 0, i, f, False)[0] @ paged.turn(k, None, 0, j, f, False)[0]

    assert np.isclose(score(5, 2), score(1005, 1002)) and not np.isclose(score(5, 2), score(5, 3))
    assert np.isclose(score(9, 9), q @ k)


def test_norm():
    rng = np.random.default_rng(3)
    x, w = rng.standard_normal(128) * 7, rng.standard_normal(128)
    out, _ = paged.turn(x, w, 0.0, 0, None, False)
    assert np.isclose(np.sqrt(((out / w) ** 2).mean()), 1.0)
    assert np.allclose(paged.turn(3 * x, w, 0.0, 0, None, False)[0], out)
    assert np.array_equal(paged.turn(x, None, 1e-6, 3, None, False)[0], x)
    assert np.array_equal(paged.turn(np.zeros(128), w, 1e-6, 0, None, False)[0], np.zeros(128))
    t, _ = paged.turn(x, w, 0.0, 5, freqs(32), True)     # the norm comes first
    assert np.allclose(t, paged.turn(out, None, 0.0, 5, freqs(32), True)[0])


@pytest.mark.parametrize("scale,shift", [(1.0, 0.0), (1e-3, 5.0), (300.0, -4000.0)])
def test_four_bits(scale, shift):
    rng = np.random.default_rng(4)
    x = rng.standard_normal(256) * scale + shift
    codes, scales = paged.store4(x)
    y = paged.load4(codes, scales)
    for g in range(4):
        s, m = (float(v) for v in scales[g])
        part = x[64 * g:64 * g + 64]
        # half a step, and at the ends the roundings of least value and step (2^-11 each)
        slack = s / 2 + abs(part.min()) * 2.0 ** -11 + 15 * s * 2.0 ** -11
        assert np.abs(y[64 * g:64 * g + 64] - part).max() <= slack
    assert codes.dtype == np.uint8 and codes.shape == (128,)
    low, _, _ = paged.quantise(x[:64])
    assert np.array_equal(codes[:32] & 15, low[0::2]) and np.array_equal(codes[:32] >> 4, low[1::2])


def test_four_bits_of_exact_and_constant_values():
    x = np.arange(64) % 16 * 0.25 - 1.0
    assert np.array_equal(paged.load4(*paged.store4(x)), x)
    assert np.array_equal(paged.load4(*paged.store4(np.full(64, 2.5))), np.full(64, 2.5))
    c, s, m = paged.quantise(np.array([0.5, 1.5] + [0.0] * 61 + [15.0]))   # ties go to even codes
    assert (s, m) == (1.0, 0.0) and list(c[:2]) == [0, 2]
    c, s, m = paged.quantise(np.linspace(-1e6, 1e6, 64))                   # held in half precision's range
    assert (s, m) == (65504.0, -65504.0)


def test_rows_in_pages():
    rng = np.random.default_rng(5)
    pages = rng.standard_normal((7, 2, 16, 64))
    table = [5, -1, 0, 7, 3]
    rows, there = paged.rows_of(pages, table, 10, 80)
    assert np.array_equal(rows[0], pages[5, :, 10]) and np.array_equal(rows[22], pages[0, :, 0])
    assert np.array_equal(rows[54], pages[3, :, 0])
    want = [t in (5, 0, 3) for t in np.repeat(table, 16)] + [False] * 10
    assert np.array_equal(there, want[10:90]) and not rows[~there].any()


def test_attention_over_pages():
    rng = np.random.default_rng(6)
    k, v = rng.standard_normal((40, 2, 64)), rng.standard_normal((40, 2, 64))
    kp, vp = np.zeros((4, 2, 16, 64)), np.zeros((4, 2, 16, 64))
    table = [2, 0, 3]
    for r in range(40):
        kp[table[r // 16], :, r % 16], vp[table[r // 16], :, r % 16] = k[r], v[r]
    q = rng.standard_normal((6, 64))
    o, _, _ = paged.decode(q, kp, vp, table, 36, 0.125)
    assert np.allclose(o, attention.attn(q[None], k[:37], v[:37], 0.125)[0][0])
    gone, _, _ = paged.decode(q, kp, vp, [2, 9, 3], 36, 0.125)
    keep = np.r_[0:16, 32:37]
    assert np.allclose(gone, attention.attn(q[None], k[keep], v[keep], 0.125)[0][0])
    assert not paged.decode(q, kp, vp, table, 48, 0.125)[0].any() and not paged.decode(q, kp, vp, table, -1, 1.0)[0].any()
    assert not paged.decode(q, kp, vp, [-1, -1, 4], 36, 0.125)[0].any()
