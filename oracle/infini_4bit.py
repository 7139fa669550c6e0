"""Float64 restatement of the 4-bit weights and of the decode step over a
4-bit segment buffer.

TEST INFRASTRUCTURE ONLY (see the package docstring): never imported by the
product path.

Everything here goes channel by channel from the layouts' definitions:
  weight or key rows: for each block of D channels (128 for weights, the head
    width d for keys), 32-bit word (D / 32) c + j holds channels
    32 j + 8 c + o, o = 0..7; even o in bits 2 o.., odd o in bits 2 o + 14..;
  value rows: 16-bit word (d / 32) i + j holds channels 32 j + 4 i + t,
    t = 0..3, in bits 4 t...

Pinned in ``tests/test_oracle_4bit.py``.
"""

import numpy as np

from .infini_oracle import elu_plus_one, gate_sigmoid


def key_bit(ch, D):
    """First bit of channel ch in its block of D channels."""
    j, c, o = ch // 32, (ch % 32) // 8, ch % 8
    return 32 * (c * (D // 32) + j) + (2 * o if o % 2 == 0 else 2 * o + 14)


def value_bit(ch, D):
    j, i, t = ch // 32, (ch % 32) // 4, ch % 4
    return 16 * (i * (D // 32) + j) + 4 * t


def codes_of(packed, n, bit, D):
    """uint8 [..., bytes] to codes [..., n] by ``bit`` (key_bit or value_bit)."""
    out = np.empty(packed.shape[:-1] + (n,), np.uint8)
    for ch in range(n):
        b = (ch // D) * D * 4 + bit(ch % D, D)
        out[..., ch] = (packed[..., b // 8] >> (b % 8)) & 15
    return out


def packed_of(codes, bit, D):
    """codes [..., n] to uint8 [..., ceil(n / D) * D / 2] (missing ones 0)."""
    n = codes.shape[-1]
    out = np.zeros(codes.shape[:-1] + (-(-n // D) * D // 2,), np.uint8)
    for ch in range(n):
        b = (ch // D) * D * 4 + bit(ch % D, D)
        out[..., b // 8] |= (codes[..., ch] << (b % 8)).astype(np.uint8)
    return out


def bf16(x):
    """float array rounded to bf16 (to nearest, ties to even), as float64."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16) << 16
    return r.astype(np.uint32).view(np.float32).astype(np.float64)


def w4_weight(packed, scales, zeros, K, group):
    """[N, K] float64: scales (codes - zeros)."""
    q = codes_of(packed, K, key_bit, 128).astype(np.float64)
    g = np.arange(K) // group
    z = zeros[:, g].astype(np.float64) if zeros is not None else 8.0
    return np.asarray(scales, np.float64)[:, g] * (q - z)


def cache_codes(x):
    """Rows [..., d] as the 4-bit segment buffer stores them: (codes, scale,
    minimum), in groups of 32 channels, with fp32 arithmetic and bf16 scale and
    minimum."""
    x = np.asarray(x, np.float32)
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // 32, 32))
    m = bf16(g.min(-1)).astype(np.float32)
    s = bf16(np.maximum(g.max(-1) - m, np.float32(0)) * np.float32(1 / 15)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint((g - m[..., None]) / s[..., None])
    q = np.where(s[..., None] > 0, np.clip(q, 0, 15), 0)
    return q.astype(np.uint8).reshape(x.shape), s.astype(np.float64), m.astype(np.float64)


def cache_values(codes, s, m):
    """scale code + minimum, float64."""
    return codes * np.repeat(s, 32, axis=-1) + np.repeat(m, 32, axis=-1)


def decode_step_q4(q_t, K, V, pos, beta, M, z):
    """One token per stream: q_t [B, H_q, d], K and V [B, H_kv, S, d] the
    buffer's values with the token's own row in place, pos [B] (a negative
    one: idle, output NaN).  Returns [B, H_q, d]."""
    B, H_q, d = q_t.shape
    H_kv = K.shape[1]
    out = np.full((B, H_q, d), np.nan)
    for b in range(B):
        n = int(pos[b]) + 1
        if n <= 0:
            continue
        for h in range(H_q):
            kv = h // (H_q // H_kv)
            s = K[b, kv, :n] @ q_t[b, h] / np.sqrt(d)
            p = np.exp(s - s.max())
            a_dot = (p / p.sum()) @ V[b, kv, :n]
            sq = elu_plus_one(q_t[b, h])
            den = sq @ z[b, kv]
            a_mem = sq @ M[b, kv] / den if den != 0 else np.zeros(d)
            g = gate_sigmoid(beta[h])
            out[b, h] = g * a_mem + (1 - g) * a_dot
    return out
