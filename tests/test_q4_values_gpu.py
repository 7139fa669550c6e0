"""GPU: what the decode step over the 4-bit segment buffer keeps of its weights,
against the float64 oracle, group by group.

A tile's weights (probability times scale) meet the codes in fp16 parts.  With p the
oracle's probabilities (sum 1), s and m the stored scales and minima of a group,
W = sum of p 15 s (the span that the codes can add), Y = sum of p |m| and T = 2 W + Y
(fp32 heads take codes less 8, with 8 s in the minimum):
  weights    two parts: 2^-21 of a weight (bf16 heads), 2^-22 (fp32); what the parts
             drop below fp16's 2^-24 is 2^-31 of the largest weight a row: n 2^-31 15 max(p s);
  codes      bf16 heads hold them as fp16 subnormals: of a product of 16 terms and the sum
             so far what lies 2^-13 of a code below its largest weight is dropped, so for each
             of its 17 terms at most 2^-13 of that weight: together 17 / 15 2^-13 W;
  sums       n / 64 + 64 additions in a row of 2^-23 of T, and 2^-21 T for 2^x;
  scores     in powers of two off by at most 2^-19 A (A: the magnitudes that a score is made
             of), for bf16 heads and each group of keys by 34 2^-13 of a code times the largest
             element of the query besides (two products of 16 channels): E of a row together;
             then its probability is within a factor of 1 +- E (E << 1), and the weighted mean
             of values v, of magnitude t = 2 15 s + |m| at most, within sum of p E (t + T);
and half a step of the output's own rounding.  The memory is switched off (beta = -100).
"""

import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(*shape, seed, dtype="f32"):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DT[dtype])


def rounded(x, bit):
    """Rows [..., d] as the buffer holds them: (bytes, scale and minimum, float64 values)."""
    q, s, m = oracle.cache_codes(x.float().numpy())
    return (torch.from_numpy(oracle.packed_of(q, bit, x.shape[-1])), torch.from_numpy(np.stack((s, m), -1)).bfloat16(),
            oracle.cache_values(q.astype(np.float64), s, m))


def step(api, keys, vals, q, dtype):
    """The step of the last row's token, given keys and values [B, H, n, d] in fp32
    (the last ones representable in dtype): output [B, H_q, d], the stored keys'
    and values' (scale and minimum, values)."""
    B, H, n, d = keys.shape
    kc, ks, K = rounded(keys, oracle.key_bit)
    vc, vs, V = rounded(vals, oracle.value_bit)
    cache = api.CacheQ4(*(t.cuda() for t in (kc, ks, vc, vs)))
    for t in cache.tensors:  # the step writes the last row itself
        t[:, :, n - 1] = 0
    last = [x[:, :, n - 1].contiguous().to(DT[dtype]) for x in (keys, vals)]
    assert all(torch.equal(t.float(), x[:, :, n - 1]) for t, x in zip(last, (keys, vals)))
    pos = torch.full((B,), n - 1, dtype=torch.int32)
    out = api.decode_step_q4(q.cuda(), last[0].cuda(), last[1].cuda(), torch.full((q.shape[1],), -100.0).cuda(), cache,
                             pos.cuda(), torch.zeros(B, H, d, d).cuda(), torch.ones(B, H, d).cuda())
    api.sync_status()
    assert torch.equal(cache.tensors[2].cpu(), vc)
    return f64(out), (f64(ks), K), (f64(vs), V)


def check(out, keys, vals, q, dtype):
    (ks, K), (vs, V) = keys, vals
    B, H_q, d = q.shape
    g, n = H_q // K.shape[1], K.shape[2]
    x = f64(q)
    for b in range(B):
        for h in range(H_q):
            kv = h // g
            s = K[b, kv] @ x[b, h] / math.sqrt(d)
            p = np.exp(s - s.max())
            p /= p.sum()
            unit = math.log2(math.e) / math.sqrt(d)
            ax = np.abs(x[b, h]).reshape(-1, 32)
            E = 2.0 ** -19 * unit * ((15 * ks[b, kv, :, :, 0] + np.abs(ks[b, kv, :, :, 1])) @ ax.sum(-1))
            if dtype == "bf16":
                E = E + 34 * 2.0 ** -13 * unit * (ks[b, kv, :, :, 0] @ ax.max(-1))
            assert np.all(E < 0.1)
            W, Y = 15 * (p @ vs[b, kv, :, :, 0]), p @ np.abs(vs[b, kv, :, :, 1])
            T = 2 * W + Y
            slack = 2.0 ** (-21 if dtype == "bf16" else -22) * W
            slack += n * 2.0 ** -31 * 15 * np.max(p[:, None] * vs[b, kv, :, :, 0], 0)
            slack += 17 / 15 * 2.0 ** -13 * W if dtype == "bf16" else 0
            slack += ((n / 64 + 64) * 2.0 ** -23 + 2.0 ** -21) * T
            slack += (p * E) @ (30 * vs[b, kv, :, :, 0] + np.abs(vs[b, kv, :, :, 1]) + T)
            ref = p @ V[b, kv]
            err = np.abs(out[b, h] - ref) - HALF[dtype] * np.abs(ref) - np.repeat(slack, 32)
            assert np.all(err <= 0), (b, h, float(err.max()), slack)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("g", [4, 6])  # the weights' second parts in free columns, or in products of their own
@pytest.mark.parametrize("k", [8, 12, 20])
def test_groups_of_unequal_size(cuda_lib, k, g, dtype):
    """Groups of channels 2^k and 2^-k as large as the others; scores all equal
    (no error of theirs), and scores that differ."""
    d, n = 128, 700
    keys = randn(2, 1, n, d, seed=1, dtype="bf16").float()
    vals = randn(2, 1, n, d, seed=2, dtype="bf16").float()
    vals[..., 32:64] *= 2.0 ** k
    vals[1, :, :, 96:] *= 2.0 ** -k
    q = randn(2, g, d, seed=3, dtype=dtype)
    q[0] = 0.0
    check(*step(cuda_lib, keys, vals, q, dtype), q, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("g", [4, 6])
@pytest.mark.parametrize("k", [8, 12, 20])
def test_rows_of_unequal_size(cuda_lib, k, g, dtype):
    """A row 2^k as large as the others, early, late and as the token's own, that some
    heads attend to and others next to not at all."""
    d, n = 64, 700
    keys, vals = (randn(3, 1, n, d, seed=i, dtype="bf16").float() for i in (1, 2))
    # Queries of one channel: the row's score is 12 for head 0, 5 for head 1 and -16 for
    # the others; the other rows' lie near 0.
    q = torch.zeros(3, g, d, dtype=DT[dtype])
    q[:, 0, 3], q[:, 1, 3], q[:, 2:, 3] = 0.75, 0.3125, -1.0
    for b, row in enumerate((5, 500, n - 1)):
        vals[b, 0, row] *= 2.0 ** k
        keys[b, 0, row] = 0.0
        keys[b, 0, row, 3] = 128.0
    check(*step(cuda_lib, keys, vals, q, dtype), q, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("g", [1, 4, 8])
def test_weights_keep_their_bits(cuda_lib, g, dtype):
    """Four rows: two of one key and two of another, each pair with values v and -v.  The
    output is 0, and what is left is the rounding of the weights: with s = 1 and
    weights w and 1 or 2^2 apart at most, no term of a product is dropped (the first
    parts have 11 bits, and 13 are kept), so at most 15 times 2^-21 (2^-22), and 16 additions
    of 2^-23 of the minima's 7.5 and the codes' 15.  (One fp16 part a weight would leave up to
    2.5 times 2^-12.)"""
    B, H, d = 40, 2, 64
    r = np.random.default_rng(5)
    code = r.integers(0, 16, (B, H, 2, d // 32, 32))
    code[..., 3], code[..., 17] = 0, 15
    v = torch.from_numpy((code - 7.5).reshape(B, H, 2, d)).float()
    vals = torch.stack((v[:, :, 0], -v[:, :, 0], v[:, :, 1], -v[:, :, 1]), 2)
    k = randn(B, H, 2, d, seed=6, dtype="bf16").float()
    keys = k[:, :, [0, 0, 1, 1]].contiguous()
    K = rounded(keys, oracle.key_bit)[2]
    x = randn(B, H, g, d, seed=7)
    gap = np.einsum("bhgd,bhd->bhg", f64(x), K[:, :, 0] - K[:, :, 3]) / math.sqrt(d) * math.log2(math.e)
    want = r.uniform(0.1, 1.9, gap.shape) * r.choice([-1, 1], gap.shape)
    q = (x * torch.from_numpy(want / gap)[..., None]).reshape(B, H * g, d).to(DT[dtype])
    out, _, (vs, V) = step(cuda_lib, keys, vals, q, dtype)
    assert np.all(vs == np.array([1.0, -7.5])) and np.all(V[:, :, 0] == -V[:, :, 1])
    bound = 15 * 2.0 ** (-21 if dtype == "bf16" else -22) + 16 * 2.0 ** -23 * 22.5
    assert np.abs(out).max() <= bound, float(np.abs(out).max())
