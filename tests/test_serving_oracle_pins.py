"""Pins of the float64 definitions of the operators around attention (CPU)."""

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S


def _tables(positions, rot):
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(positions)[:, None] * f
    return np.cos(a), np.sin(a)


def test_page_plan_worked_example():
    # Request 0: 63 + 2 tokens, one new page; request 1: 0 + 64, one; request 2: idle; request 3: 10 + 1, none.
    table = np.full((4, 3), -1)
    table[0, 0], table[2, 0], table[3, 0] = 5, 6, 7
    p = S.page_plan([63, 0, 64, 10], [2, 64, 0, 1], table, [8, 9, 4], 70, 10)
    assert p["seq_lens"].tolist() == [65, 64, 64, 11] and p["cu_seqlens"].tolist() == [0, 2, 66, 66, 67]
    assert p["table"].tolist() == [[5, 8, -1], [9, -1, -1], [6, -1, -1], [7, -1, -1]]
    assert p["slots"].tolist() == [5 * 64 + 63, 8 * 64] + [9 * 64 + i for i in range(64)] + [7 * 64 + 10] + [-1] * 3
    assert p["positions"].tolist() == [63, 64] + list(range(64)) + [10] + [-1] * 3
    assert p["used"] == 2 and p["error"] == 0


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [128, 32])
def test_rotation_keeps_lengths_and_depends_on_distance_alone(rot, interleaved):
    rng = np.random.default_rng(0)
    cos, sin = _tables(64, rot)
    R = S.rotation(cos, sin, np.arange(64), 128, interleaved)
    assert np.allclose(np.einsum("nij,nkj->nik", R, R), np.eye(128), atol=1e-12)
    q, k = rng.standard_normal(128), rng.standard_normal(128)
    assert np.isclose((R[7] @ q) @ (R[3] @ k), (R[47] @ q) @ (R[43] @ k))
    assert not np.isclose((R[7] @ q) @ (R[3] @ k), (R[8] @ q) @ (R[3] @ k))


@pytest.mark.parametrize("norm", [True, False])
def test_norm_rope_gradients_are_the_forwards_differences(norm):
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((3, 2, 64)), rng.standard_normal((3, 2, 64))
    w = 1 + 0.1 * rng.standard_normal(64) if norm else None
    R = S.rotation(*_tables(8, 32), np.array([0, 5, 7]), 64, False)
    dx, dw = S.norm_rope_grad(x, dy, w, R, 1e-3, norm)
    loss = lambda x, w: (dy * S.norm_rope(x, w, R, 1e-3, norm)).sum()
    h = 1e-6
    for at in [(0, 0, 0), (1, 1, 17), (2, 0, 63), (1, 0, 40)]:
        e = np.zeros_like(x)
        e[at] = h
        assert np.isclose((loss(x + e, w) - loss(x - e, w)) / (2 * h), dx[at], rtol=1e-6, atol=1e-8)
    if norm:
        for c in (0, 31, 63):
            e = np.zeros(64)
            e[c] = h
            assert np.isclose((loss(x, w + e) - loss(x, w - e)) / (2 * h), dw[c], rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("d", [64, 128])
def test_blocks_hold_what_was_quantised(d):
    rng = np.random.default_rng(2)
    k, v = (torch.tensor(rng.standard_normal((2, 64, d))).bfloat16().float().numpy() for _ in range(2))
    block = S.q4_blocks(k, v)
    assert block.shape == (2, 72 * d)
    for x, got in zip((k, v), S.q4_unblock(block, d)):
        assert np.array_equal(got, S.q4_values(*S.q4_quantise(x)))
        # half a step, and the scale's rounding (2^-8 of 15 steps) at the far end
        step = np.repeat(S.q4_quantise(x)[1], 64, -1)
        assert (np.abs(got - x) <= step * (0.5 + 15 * 2.0 ** -8)).all()
        assert np.array_equal(got.reshape(2, 64, -1, 64).min(-1), x.reshape(2, 64, -1, 64).min(-1))


def test_places_are_a_permutation():
    for d in (64, 128):
        (kb, ks), (vb, vs) = S._places(d)
        at = np.concatenate([(2 * kb + ks // 4).ravel(), (2 * vb + vs // 4).ravel()])
        assert sorted(at.tolist()) == list(range(128 * d))


def test_quantise_edges():
    x = np.zeros((5, 64), np.float32)
    x[1] = 3.5                       # constant: exact
    x[2, 5] = np.inf
    x[3, 0], x[3, 1] = 3e38, -3e38   # range past fp32
    x[4, 9] = np.nan
    got = S.q4_values(*S.q4_quantise(x))
    assert (got[0] == 0).all() and (got[1] == 3.5).all() and np.isnan(got[2:]).all()
