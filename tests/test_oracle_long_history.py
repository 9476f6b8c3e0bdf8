"""Pins of the long-history oracle (CPU): masks worked by hand, agreement with the causal and the
candidate-only oracles where the operators coincide, gradients against central differences."""

import numpy as np
import pytest
import torch

import oracle
import oracle.long_history as lh
import oracle.variants as ov


def _rand(rng, *shape):
    return rng.standard_normal(shape)


def test_window_mask_by_hand():
    got = lh.window_mask(6, window=2, n_sinks=1).astype(int)
    assert got.tolist() == [[1, 0, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0], [1, 1, 1, 0, 0, 0],
                            [1, 0, 1, 1, 0, 0], [1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]]
    padded = lh.window_mask(3, window=9, n_sinks=0, valid=[1, 0, 1]).astype(int)
    assert padded.tolist() == [[1, 0, 0], [0, 0, 0], [1, 0, 1]]


def test_tree_mask_by_hand():
    got = lh.tree_mask([-1, 0, 0, 2], n_hist=1).astype(int)
    assert got.tolist() == [[1, 1, 0, 0, 0], [1, 1, 1, 0, 0], [1, 1, 0, 1, 0], [1, 1, 0, 1, 1]]


def test_whole_window_is_causal():
    rng = np.random.default_rng(0)
    q, k, v = (_rand(rng, 13, 2, 8) for _ in range(3))
    out, lse, _, _ = lh.masked(q, k, v, lh.window_mask(13, 13, 0), 0.3)
    np.testing.assert_allclose(out, ov.jagged_causal_attn(q, k, v, [0, 13], 0.3), atol=1e-12)
    s = 0.3 * q[4, 1] @ k[:5, 1].T
    assert abs(lse[4, 1] - np.log(np.exp(s).sum())) < 1e-12


def test_star_tree_is_candidate_only():
    rng = np.random.default_rng(1)
    q, k, v = (torch.tensor(_rand(rng, 5, 2, 8)) for _ in range(3))
    hk, hv = (torch.tensor(_rand(rng, 7, 2, 8)) for _ in range(2))
    out, _, _, _ = lh.masked(q, torch.cat([hk, k]), torch.cat([hv, v]), lh.tree_mask([-1] * 5, 7),
                             0.4)
    ref = oracle.cand_only_attn(q, k, v, np.array([0, 5]), hk, hv, np.array([0, 7]), None, 0.4)
    np.testing.assert_allclose(out, ref, atol=1e-6)


@pytest.mark.parametrize("which", range(3))
def test_gradients_against_differences(which):
    rng = np.random.default_rng(2)
    L, H, Hkv, d = 7, 4, 2, 3
    x = [_rand(rng, L, H, d), _rand(rng, L, Hkv, d), _rand(rng, L, Hkv, d)]
    do = _rand(rng, L, H, d)
    mask = lh.window_mask(L, 3, 1, valid=[1, 1, 0, 1, 1, 1, 1])
    grads, _ = lh.gradients(*x, do, mask, 0.5)

    def f(y):
        z = list(x)
        z[which] = y
        return float((lh.masked(*z, mask, 0.5)[0] * np.where(mask.any(1)[:, None, None], do, 0)).sum())

    num = np.zeros_like(x[which])
    for i in np.ndindex(*num.shape):
        e = np.zeros_like(num)
        e[i] = 1e-6
        num[i] = (f(x[which] + e) - f(x[which] - e)) / 2e-6
    np.testing.assert_allclose(grads[which], num, atol=1e-8)


def test_one_axis_is_the_plain_rotation():
    rng = np.random.default_rng(3)
    x, pos = _rand(rng, 9, 2, 16), rng.integers(-50, 5000, 9)
    for per_axis in (False, True):
        got = lh.rope_axes(x, pos[:, None], [8], per_axis=per_axis)
        np.testing.assert_allclose(got, oracle.apply_rope(x, pos), atol=1e-9)


def test_axes_turn_their_own_pairs():
    rng = np.random.default_rng(4)
    x, pos = _rand(rng, 5, 1, 16), rng.integers(0, 99, (5, 3))
    base = lh.rope_axes(x, pos, [3, 2, 2])
    moved = pos.copy()
    moved[:, 1] += 7
    diff = np.abs(lh.rope_axes(x, moved, [3, 2, 2]) - base).max((0, 1)) > 0
    assert np.flatnonzero(diff).tolist() == [3, 4, 11, 12]
    np.testing.assert_array_equal(base[..., [7, 15]], x[..., [7, 15]])
    np.testing.assert_allclose(lh.rope_axes(base, pos, [3, 2, 2], sign=-1.0), x, atol=1e-12)
