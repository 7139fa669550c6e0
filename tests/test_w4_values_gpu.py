"""GPU: 4-bit projections at the ends of fp32's range, against exact products."""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("M,N", [(3, 40), (40, 40), (20, 9600)])  # blocks shared out, and 64 rows a block
def test_fp32_tokens_of_every_size(cuda_lib, M, N):
    """One channel of each token is not zero, from fp32's smallest to its largest value
    (beyond bf16's largest, which would round to infinity), times an integer -1, 0 or 1 and a
    scale 2^-10 or 2^10: exact but for three additions and one product of 2^-23, and for what
    lies below the types' least values.  Those are 2^-149 for the result, and 2^-133 for a
    token's bf16 parts (8 exponent bits like fp32's, 7 bits of mantissa: 2^-126 2^-7): rounding the
    parts leaves less than that of the token, which counts times |q - z| = 1 and the scale."""
    K, group = 136, 32
    r = np.random.default_rng(1)
    code = r.integers(7, 10, (N, K)).astype(np.uint8)
    big = np.finfo(np.float32).max
    values = np.float32([big, -big, 3.3961775e38, 3.3895314e38, 1.0000001, 1e-38, -3e-42, 1.4e-45, 2.0 ** 127, -1 / 3])
    x = np.zeros((M, K), np.float32)
    for t in range(M):
        x[t, r.integers(0, K)] = values[t % len(values)]
    y = {}
    for power in (-10, 10):
        layer = cuda_lib.LinearW4(torch.from_numpy(oracle.packed_of(code, oracle.key_bit, 128)).cuda(),
                                  torch.full((N, 256 // group), 2.0 ** power).bfloat16().cuda(), None, K)
        y[power] = f64(layer(torch.from_numpy(x).cuda()))
        want = x.astype(np.float64) @ (code - 8.0).T * 2.0 ** power
        with np.errstate(over="ignore"):
            inf = np.abs(want) > big
        assert np.array_equal(np.sign(y[power][inf]) * np.inf, y[power][inf])
        assert np.array_equal(np.sign(want[inf]), np.sign(y[power][inf]))
        err = np.abs(y[power] - want)[~inf] - 4 * 2.0 ** -23 * np.abs(want[~inf]) - 2.0 ** -148 - 2.0 ** (power - 133)
        assert np.all(err <= 0), float(err.max())
