"""Pins of the fp64 attention oracles against mathematics (CPU)."""
import numpy as np
import pytest

from oracle import attention as att


def draw(seed, L, Hk=2, Hv=4, dk=5, dv=3):
    r = np.random.default_rng(seed)
    return (r.standard_normal((L, Hk, dk)), r.standard_normal((L, Hk, dk)),
            r.standard_normal((L, Hv, dv)), -r.uniform(0, 1.5, Hv), r.standard_normal((Hv, dk, dv)))


@pytest.mark.parametrize("L", [1, 2, 17])
def test_linattn_is_the_masked_quadratic_form(L):
    q, k, v, g, S0 = draw(L, L)
    o, S, _, _ = att.linattn(q, k, v, g, S0, scale=0.7)
    t = np.arange(L)
    for j in range(4):
        i = j // 2
        D = np.where(t[:, None] >= t, np.exp(g[j] * (t[:, None] - t)), 0)
        want = (q[:, i] @ k[:, i].T * D) @ v[:, j] + np.exp(g[j] * (t + 1))[:, None] * (q[:, i] @ S0[j])
        np.testing.assert_allclose(o[:, j], 0.7 * want, rtol=1e-11, atol=1e-12)
        end = np.exp(g[j] * L) * S0[j] + (k[:, i] * np.exp(g[j] * (L - 1 - t))[:, None]).T @ v[:, j]
        np.testing.assert_allclose(S[j], end, rtol=1e-11, atol=1e-12)


def test_linattn_without_decay_is_a_prefix_sum_and_without_memory_the_last_token():
    q, k, v, _, _ = draw(3, 9)
    _, S, _, _ = att.linattn(q, k, v, np.zeros(4))
    np.testing.assert_allclose(S[3], k[:, 1].T @ v[:, 3], rtol=1e-12)
    o, S, _, _ = att.linattn(q, k, v, np.full(4, -np.inf))
    np.testing.assert_allclose(S[0], np.outer(k[-1, 0], v[-1, 0]), rtol=1e-12)
    np.testing.assert_allclose(o[4, 2], (q[4, 1] @ k[4, 1]) * v[4, 2], rtol=1e-12)


@pytest.mark.parametrize("cut", [0, 1, 5, 11])
def test_linattn_split_continues(cut):
    q, k, v, g, S0 = draw(8, 11)
    o, S, ao, A = att.linattn(q, k, v, g, S0)
    o1, S1, _, _ = att.linattn(q[:cut], k[:cut], v[:cut], g, S0)
    o2, S2, _, _ = att.linattn(q[cut:], k[cut:], v[cut:], g, S1)
    np.testing.assert_allclose(np.concatenate([o1, o2]), o, rtol=1e-12)
    np.testing.assert_allclose(S2, S, rtol=1e-12)
    assert np.all(ao >= np.abs(o) - 1e-12) and np.all(A >= np.abs(S) - 1e-12)


def test_attn_one_key_is_its_value_and_equal_scores_the_mean():
    r = np.random.default_rng(1)
    q, k, v = r.standard_normal((1, 4, 6)), r.standard_normal((1, 2, 6)), r.standard_normal((1, 2, 6))
    o, _, _ = att.attn(q, k, v, 0.4)
    np.testing.assert_allclose(o[0], np.repeat(v[0], 2, axis=0), rtol=1e-13)
    q, v = r.standard_normal((5, 2, 6)), r.standard_normal((5, 1, 6))
    k = np.repeat(r.standard_normal((1, 1, 6)), 5, axis=0)
    o, _, _ = att.attn(q, k, v, 3.0)
    for t in range(5):
        np.testing.assert_allclose(o[t, 1], v[:t + 1, 0].mean(axis=0), rtol=1e-12)


def test_attn_later_queries_of_a_prefix_and_unseen_rows():
    r = np.random.default_rng(2)
    q, k, v = (r.standard_normal((9, h, 4)) for h in (2, 1, 1))
    whole, ao, _ = att.attn(q, k, v, 0.5)
    part, _, _ = att.attn(q[6:], k, v, 0.5)
    np.testing.assert_allclose(part, whole[6:], rtol=1e-12)
    few, _, _ = att.attn(q, k[:3], v[:3], 0.5)
    assert not few[:6].any() and few[6:].any()
    assert np.all(ao >= np.abs(whole) - 1e-12)
    # a very large score takes everything
    k2 = k.copy()
    k2[2, 0] = 1e3 * q[8, 0]
    o, _, _ = att.attn(q, k2, v, 1.0)
    np.testing.assert_allclose(o[8, 0], v[2, 0], rtol=1e-9)
