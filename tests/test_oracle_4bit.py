"""The float64 oracle of the 4-bit weights and segment buffer, pinned."""

import numpy as np
import pytest

import oracle


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("kind", ["key", "value"])
def test_layout_is_a_permutation_of_nibbles(d, kind):
    bit = oracle.key_bit if kind == "key" else oracle.value_bit
    bits = sorted(bit(ch, d) for ch in range(d))
    assert bits == list(range(0, 4 * d, 4))
    rng = np.random.default_rng(d)
    q = rng.integers(0, 16, (5, 3 * d)).astype(np.uint8)
    p = oracle.packed_of(q, bit, d)
    assert p.shape == (5, 3 * d // 2)
    assert np.array_equal(oracle.codes_of(p, 3 * d, bit, d), q)
    # the words, read as the definition says
    word = 32 if kind == "key" else 16
    w = p.view(np.uint32 if kind == "key" else np.uint16)
    per = d // 32
    for ch in (0, 1, 5, d - 1, d // 2 + 3):
        if kind == "key":
            j, c, o = ch // 32, ch % 32 // 8, ch % 8
            at, shift = c * per + j, (2 * o if o % 2 == 0 else 2 * o + 14)
        else:
            j, i, t = ch // 32, ch % 32 // 4, ch % 4
            at, shift = i * per + j, 4 * t
        assert shift < word
        assert np.array_equal((w[:, at].astype(np.int64) >> shift) & 15, q[:, ch])


def test_bf16_rounds_to_nearest_even():
    x = np.array([1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 1 + 2.0 ** -8 + 2.0 ** -20, -3.1415927], np.float32)
    assert np.array_equal(oracle.bf16(x), [1.0, 1.0, 1 + 2.0 ** -6, 1 + 2.0 ** -7, -3.140625])


def test_w4_weight_single_elements():
    rng = np.random.default_rng(1)
    N, K, G = 3, 200, 64
    q = rng.integers(0, 16, (N, K)).astype(np.uint8)
    scales = oracle.bf16(rng.uniform(0.01, 1, (N, 4)))
    zeros = rng.integers(0, 16, (N, 4)).astype(np.uint8)
    w = oracle.w4_weight(oracle.packed_of(q, oracle.key_bit, 128), scales, zeros, K, G)
    sym = oracle.w4_weight(oracle.packed_of(q, oracle.key_bit, 128), scales, None, K, G)
    for n in range(N):
        for k in range(K):
            assert w[n, k] == scales[n, k // G] * (int(q[n, k]) - int(zeros[n, k // G]))
            assert sym[n, k] == scales[n, k // G] * (int(q[n, k]) - 8)


def test_cache_rounding_is_within_half_a_step():
    rng = np.random.default_rng(2)
    x = rng.normal(size=(40, 64)).astype(np.float32) * np.exp(rng.normal(size=(40, 1))).astype(np.float32)
    x[3] = 0.0
    x[4] = -2.5
    q, s, m = oracle.cache_codes(x)
    v = oracle.cache_values(q, s, m)
    # half a step, the scale's and the minimum's own rounding at the ends
    step = np.repeat(s, 32, axis=-1)
    slack = 15 * step * 2.0 ** -8 + np.repeat(np.abs(m), 32, axis=-1) * 2.0 ** -8
    assert np.all(np.abs(v - x) <= step / 2 + slack)
    assert np.all(v[3] == 0.0) and np.all(v[4] == -2.5)  # one value in a group: exact
    assert q.max() <= 15


@pytest.mark.parametrize("rule", ["linear", "delta"])
def test_decode_step_is_the_layer_forward(rule):
    """With the buffer's values as keys and values, the step gives the layer's
    own output of that token."""
    rng = np.random.default_rng(3)
    B, H_q, H_kv, d, S = 2, 4, 2, 32, 8
    L = S + 5
    q, k, v = (rng.normal(size=(B, h, L, d)) for h in (H_q, H_kv, H_kv))
    beta = rng.normal(size=H_q)
    M0, z0 = np.zeros((B, H_kv, d, d)), np.zeros((B, H_kv, d))
    ref, _, _ = oracle.infini_attention_forward(q, k, v, beta, M0, z0, S, rule)
    _, M1, z1 = oracle.infini_attention_forward(q[:, :, :S], k[:, :, :S], v[:, :, :S], beta, M0, z0, S, rule)
    buf = np.zeros((B, H_kv, S, d)), np.zeros((B, H_kv, S, d))
    for t in range(L):
        row = t % S
        buf[0][:, :, row], buf[1][:, :, row] = k[:, :, t], v[:, :, t]
        M, z = (M0, z0) if t < S else (M1, z1)
        got = oracle.decode_step_q4(q[:, :, t], *buf, [row, row], beta, M, z)
        assert np.max(np.abs(got - ref[:, :, t])) < 1e-12
    idle = oracle.decode_step_q4(q[:, :, 0], *buf, [-1, 0], beta, M0, z0)
    assert np.isnan(idle[0]).all() and np.isfinite(idle[1]).all()
