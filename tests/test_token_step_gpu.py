"""A layer's token step as a user runs it: norm, 4-bit Q/K/V projection with
rotary embedding, decode step over the 4-bit buffer, 4-bit output projection,
gated residual sum and next norm, token after token across segment ends.

Each stage is compared with the float64 oracle on that stage's own inputs (the
GPU's output of the stage before), in fp32, so that a rounding of one stage is
not counted in the next.  Tolerances: a norm or projection of K terms 2^-23 K
of the sum of magnitudes (K = 96 and 128 here: below 2^-16 of it, taken
against the output's scale of a few units: 1e-4); the decode step 1e-4: scores'
magnitudes stay below 2^4, so 2^-19 of them on either side of a probability and
values below 4 make 2 x 2^-15 x 4 = 2^-12 at the very most, and the mean over a
few rows whose signs differ keeps less than a quarter of it."""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

EPS = 1e-6


def f64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("rule", ["linear", "delta"])
def test_token_steps(cuda_lib, rule):
    api = cuda_lib
    B, H_q, H_kv, d, S, D, tokens = 3, 4, 2, 32, 5, 96, 12
    g = torch.Generator().manual_seed(7)

    def randn(*shape, std=1.0):
        return (std * torch.randn(*shape, generator=g)).cuda()

    n_qkv = (H_q + 2 * H_kv) * d
    qkv = api.LinearW4.from_weight(randn(n_qkv, D, std=D ** -0.5), group=32, bias=randn(n_qkv, std=0.1))
    proj = api.LinearW4.from_weight(randn(D, H_q * d, std=(H_q * d) ** -0.5), group=64, zeros=False)
    w_qkv, w_proj = f64(qkv.dequantize()), f64(proj.dequantize())
    w_in, w_post, w_next = (1 + randn(D, std=0.1) for _ in range(3))
    scale, gate_w = 0.5 + 0.1 * randn(D), api.LinearW4.from_weight(randn(D, D, std=D ** -0.5))
    beta = randn(H_q)
    cos, sin = api.rope_tables(tokens, d)
    c64, s64 = oracle.rope_tables(tokens, d)
    stream = api.DecodeStreamQ4(B, H_q, H_kv, d, S, rule, dtype=torch.float32)
    for t in range(tokens):
        r = randn(B, D)
        _, h, _, _ = api.block_norm(r, w_in, EPS)
        assert np.allclose(f64(h), oracle.block_norm(f64(r), f64(w_in), EPS)[1], rtol=0, atol=1e-4)
        at = torch.full((B, 1), t, dtype=torch.int32, device="cuda")
        q, k, v = qkv.qkv(h[:, None], H_q, H_kv, d, cos, sin, at)
        y = (f64(h) @ w_qkv.T + f64(qkv.bias)).reshape(B, H_q + 2 * H_kv, 1, d)
        y[:, :H_q + H_kv] = oracle.apply_rope(y[:, :H_q + H_kv], c64[t:t + 1], s64[t:t + 1])
        for got, sl in ((q, slice(0, H_q)), (k, slice(H_q, H_q + H_kv)), (v, slice(H_q + H_kv, None))):
            assert np.allclose(f64(got), y[:, sl], rtol=0, atol=1e-4)
        M, z = f64(stream.M), f64(stream.z)
        o = stream.step(q[:, :, 0], k[:, :, 0], v[:, :, 0], beta)
        kq, ksm, vq, vsm = stream.cache.tensors
        K, V = (oracle.cache_values(oracle.codes_of(c.cpu().numpy(), d, bit, d).astype(np.float64),
                                    f64(s)[..., 0], f64(s)[..., 1])
                for c, s, bit in ((kq, ksm, oracle.key_bit), (vq, vsm, oracle.value_bit)))
        ref = oracle.decode_step_q4(f64(q[:, :, 0]), K, V, [t % S] * B, f64(beta), M, z)
        assert np.allclose(f64(o), ref, rtol=0, atol=1e-4)
        x = proj(o.reshape(B, H_q * d))
        assert np.allclose(f64(x), f64(o).reshape(B, -1) @ w_proj.T, rtol=0, atol=1e-4)
        gate = gate_w(h)
        want = oracle.block_norm(f64(r), f64(w_next), EPS, o=f64(x), gate=f64(gate), scale=f64(scale),
                                 w_post=f64(w_post))
        r2, h2, _, _ = api.block_norm(r, w_next, EPS, o=x, gate=gate, scale=scale, w_post=w_post, r_out=r)
        assert np.allclose(f64(r2), want[0], rtol=0, atol=1e-4)
        assert np.allclose(f64(h2), want[1], rtol=0, atol=1e-4)
    api.sync_status()
    assert torch.count_nonzero(stream.M) > 0  # the segment ends were reached
