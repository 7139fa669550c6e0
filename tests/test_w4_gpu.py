"""GPU parity of the 4-bit weights and their projections (infini_attn_w4_*,
infini_attn_linear_w4, infini_attn_qkv_project_w4) against the float64 oracle.

Tolerance: codes, zeros and scales are exact in the kernel, bf16 tokens too,
and fp32 tokens enter as three bf16 parts that hold them up to 2^-24.  What is
rounded: the fp32 accumulators, at most K / 16 additions in a row inside a
group sum and one per group and warp after it, each off by at most 2^-23 of a
partial sum, which the sum of magnitudes A = |W| |x| bounds; the group's scaling
and the bias (2^-24 each); and the result's own rounding (half a step).  With
the three parts of fp32 tokens that is (3 K / 16 + 16) 2^-23 A at most.  The
rotation adds two products of such values with tables of fp32.
"""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def weights(N, K, group, zeros, seed=0):
    """Random codes, scales and zeros; the padding holds what must be ignored."""
    g = torch.Generator().manual_seed(seed)
    padded = -(-K // 128) * 128
    codes = torch.randint(0, 16, (N, K), generator=g, dtype=torch.int32).to(torch.uint8)
    scales = (0.01 + torch.rand(N, padded // group, generator=g)).bfloat16()
    scales[:, -(-K // group):] = float("nan")
    z = torch.randint(0, 16, (N, padded // group), generator=g, dtype=torch.int32).to(torch.uint8) \
        if zeros else None
    full = torch.cat((codes, torch.randint(0, 16, (N, padded - K), generator=g, dtype=torch.int32)
                      .to(torch.uint8)), 1)
    packed = torch.from_numpy(oracle.packed_of(full.numpy(), oracle.key_bit, 128))
    return packed, scales, z


def layer_of(api, N, K, group, zeros, bias, seed=0):
    packed, scales, z = weights(N, K, group, zeros, seed)
    b = torch.randn(N, generator=torch.Generator().manual_seed(seed + 1)) if bias else None
    w = oracle.w4_weight(packed.numpy(), f64(scales), z.numpy() if zeros else None, K, group)
    layer = api.LinearW4(packed.cuda(), scales.cuda(), z.cuda() if zeros else None, K,
                         bias=b.cuda() if bias else None)
    return layer, w, (f64(b) if bias else np.zeros(N))


def slack_of(x, w, bias):
    K = w.shape[1]
    return (3 * K / 16 + 16) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T + np.abs(bias))


def tokens(M, K, dtype, seed=5):
    return torch.randn(M, K, generator=torch.Generator().manual_seed(seed)).to(DT[dtype])


CASES = [(1, 16, 128, 128, False, False), (1, 100, 4096, 128, True, True), (2, 17, 8, 32, True, False),
         (7, 33, 120, 32, False, True), (8, 64, 136, 64, True, False), (9, 777, 1000, 32, True, True),
         (16, 48, 2048, 64, False, False), (17, 31, 1032, 128, True, True), (33, 1, 640, 64, True, False),
         (64, 130, 256, 32, True, True), (65, 16, 384, 128, False, False), (130, 19, 72, 64, True, True),
         (5, 1030, 8192, 128, False, True),
         # enough rows for 64 of them a CTA: every count of token tiles, blocks fewer
         # than are loaded ahead and more, a last CTA with 1 to 3 tiles past the end
         (9, 9473, 8, 32, True, True), (16, 9500, 1032, 64, False, True), (17, 9481, 136, 128, True, False),
         (32, 9600, 640, 32, True, True), (33, 9489, 392, 64, True, True), (64, 9537, 520, 128, False, False),
         (70, 9473, 256, 32, True, True)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K,group,zeros,bias", CASES)
def test_linear(cuda_lib, M, N, K, group, zeros, bias, dtype):
    layer, w, b = layer_of(cuda_lib, N, K, group, zeros, bias, seed=M)
    x = tokens(M, K, dtype)
    out = torch.full((M * N + 8,), 7.0, dtype=DT[dtype], device="cuda")
    y = layer(x.cuda(), out=out[:M * N].view(M, N))
    cuda_lib.sync_status()
    ref = f64(x) @ w.T + b
    err = np.abs(f64(y) - ref) - HALF[dtype] * np.abs(ref) - slack_of(f64(x), w, b)
    assert np.all(err <= 0), float(err.max())
    assert torch.all(out[M * N:] == 7.0)  # nothing behind the last row


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,L,H_q,H_kv,d,K,group,rope,positions",
                         [(1, 1, 2, 1, 128, 256, 128, True, True), (3, 1, 4, 2, 64, 200, 32, True, True),
                          (2, 5, 3, 1, 32, 128, 64, True, False), (2, 33, 2, 2, 64, 136, 64, False, False),
                          (1, 9, 6, 2, 128, 1024, 128, True, True),
                          (3, 7, 60, 8, 128, 200, 32, True, True)])  # 64 rows a CTA
def test_qkv(cuda_lib, B, L, H_q, H_kv, d, K, group, rope, positions, dtype):
    N = (H_q + 2 * H_kv) * d
    layer, w, b = layer_of(cuda_lib, N, K, group, True, True, seed=d)
    x = tokens(B * L, K, dtype).view(B, L, K)
    cos = sin = pos = None
    if rope:
        cos, sin = cuda_lib.rope_tables(50, d)
        if positions:
            pos = torch.randint(0, 50, (B, L), generator=torch.Generator().manual_seed(3)).int()
    got = layer.qkv(x.cuda(), H_q, H_kv, d, cos, sin, pos.cuda() if pos is not None else None)
    cuda_lib.sync_status()
    xf = f64(x).reshape(B * L, K)
    y = (xf @ w.T + b).reshape(B, L, H_q + 2 * H_kv, d).transpose(0, 2, 1, 3)
    mag = slack_of(xf, w, b).reshape(B, L, H_q + 2 * H_kv, d).transpose(0, 2, 1, 3)
    rot = slice(0, H_q + H_kv)
    if rope:
        at = pos.numpy() if positions else np.tile(np.arange(L), (B, 1))
        c64, s64 = oracle.rope_tables(50, d)
        for bi in range(B):
            y[bi, rot] = oracle.apply_rope(y[bi, rot], c64[at[bi]], s64[at[bi]])
        top = mag[..., :d // 2] + mag[..., d // 2:]
        top = np.concatenate((top, top), -1)
        size = np.sqrt(y[..., :d // 2] ** 2 + y[..., d // 2:] ** 2)
        mag = np.where(np.arange(H_q + 2 * H_kv)[:, None, None] < H_q + H_kv,
                       top + 2.0 ** -22 * np.concatenate((size, size), -1), mag)
    for t, sl in zip(got, (slice(0, H_q), slice(H_q, H_q + H_kv), slice(H_q + H_kv, None))):
        err = np.abs(f64(t) - y[:, sl]) - HALF[dtype] * np.abs(y[:, sl]) - mag[:, sl]
        assert np.all(err <= 0), float(err.max())


def test_position_out_of_range_is_reported(cuda_lib):
    layer, w, b = layer_of(cuda_lib, 4 * 32, 128, 32, False, False)
    cos, sin = cuda_lib.rope_tables(4, 32)
    x = tokens(3, 128, "f32").view(3, 1, 128).cuda()
    pos = torch.tensor([[1], [4], [-1]], dtype=torch.int32, device="cuda")
    q, k, v = layer.qkv(x, 2, 1, 32, cos, sin, pos)
    with pytest.raises(cuda_lib.InfiniError) as e:
        cuda_lib.sync_status()
    assert e.value.status == cuda_lib.ERR_RANGE
    cuda_lib.sync_status()  # reported once
    idle = layer.qkv(x, 2, 1, 32, cos, sin, pos.clamp_max(3) * 0 - 1)  # no report
    cuda_lib.sync_status()
    assert all(torch.equal(a, b) for a, b in zip(idle, layer.qkv(x, 2, 1, 32)))
    plain = layer.qkv(x, 2, 1, 32)
    assert torch.equal(q[1:], plain[0][1:]) and torch.equal(k[1:], plain[1][1:])
    assert not torch.equal(q[0], plain[0][0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K,group,zeros", [(5, 8, 32, True), (33, 200, 64, False), (64, 1000, 32, True),
                                             (7, 4096, 128, True), (1, 128, 128, False)])
def test_quantise_pack_dequantise(cuda_lib, N, K, group, zeros, dtype):
    w = torch.randn(N, K, generator=torch.Generator().manual_seed(K)) + 0.3
    if K >= 128:
        w[0, :32] = 0.0   # a group without range
    w = w.to(DT[dtype])
    packed, scales, z = cuda_lib.w4_quantize(w.cuda(), group, zeros)
    layer = cuda_lib.LinearW4(packed, scales, z, K)
    back = layer.dequantize()
    ref = oracle.w4_weight(packed.cpu().numpy(), f64(scales), z.cpu().numpy() if zeros else None, K, group)
    assert np.array_equal(f64(back), ref)  # 8 bits times 4 bits: exact in fp32
    # Half a step of the group, and what the scale's and zero's roundings
    # cost at the ends: the scale is within 2^-8 of range / 15 (or max / 7), so
    # the outermost code, up to 15 steps from zero, misses by up to
    # 15 2^-8 steps, and a rounded zero point by another half.
    step = np.repeat(f64(scales), group, axis=1)[:, :K]
    assert np.all(np.abs(f64(w) - ref) <= step * (0.5 + 0.5 * zeros + 15 * 2.0 ** -8) + 1e-30)
    codes = oracle.codes_of(packed.cpu().numpy(), K, oracle.key_bit, 128)
    again = cuda_lib.w4_pack(torch.from_numpy(codes).cuda())
    assert torch.equal(again, packed) or K % 128  # same codes, the padding aside
    assert np.array_equal(oracle.codes_of(again.cpu().numpy(), K, oracle.key_bit, 128), codes)
    assert torch.equal(layer.dequantize(torch.bfloat16), back.bfloat16())


def test_tokens_are_independent_and_repeats_equal(cuda_lib):
    layer, _, _ = layer_of(cuda_lib, 200, 520, 64, True, True)
    x = tokens(20, 520, "bf16").cuda()
    y = layer(x)
    assert torch.equal(layer(x), y)
    x2 = x.clone()
    x2[3] = float("nan")
    y2 = layer(x2)
    keep = [i for i in range(20) if i != 3]
    assert torch.equal(y2[keep], y[keep]) and torch.isnan(y2[3]).all()


@pytest.mark.parametrize("M", [1, 12])
def test_weights_beyond_32_bits(cuda_lib, M):
    """2^20 + 3 rows of 4096 codes: packed offsets pass 2^31 bytes."""
    N, K = (1 << 20) + 3, 4096
    g = torch.Generator(device="cuda").manual_seed(M)
    packed = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (0.01 + torch.rand(N, K // 128, generator=g, device="cuda")).bfloat16()
    x = tokens(M, K, "bf16")
    y = cuda_lib.LinearW4(packed, scales, None, K)(x.cuda())
    cuda_lib.sync_status()
    for rows in (slice(0, 5), slice(N - 40, N)):
        w = oracle.w4_weight(packed[rows].cpu().numpy(), f64(scales[rows]), None, K, 128)
        ref = f64(x) @ w.T
        err = np.abs(f64(y[:, rows]) - ref) - HALF["bf16"] * np.abs(ref) - slack_of(f64(x), w, np.zeros(len(w)))
        assert np.all(err <= 0), float(err.max())


def test_other_stream_captured_graph_and_other_shapes(cuda_lib):
    layer, _, _ = layer_of(cuda_lib, 256, 1024, 128, True, True)
    x = tokens(12, 1024, "bf16").cuda()
    ref = layer(x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = layer(x.view(3, 4, 1024), stream=s)
    s.synchronize()
    assert y.shape == (3, 4, 256) and torch.equal(y.view(12, 256), ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x)
    x.neg_()
    graph.replay()
    assert torch.equal(out, layer(x))


def test_binding_refuses(cuda_lib):
    layer, _, _ = layer_of(cuda_lib, 32, 256, 64, True, False)
    x = tokens(2, 256, "bf16").cuda()
    with pytest.raises(ValueError):
        layer(x[:, :128])
    with pytest.raises(ValueError):
        layer(x.half())
    with pytest.raises(ValueError):
        layer(x.cpu())
    with pytest.raises(ValueError):
        layer(x.t().contiguous().t())
    with pytest.raises(ValueError):
        cuda_lib.LinearW4(layer.packed, layer.scales[:, :3].contiguous(), None, 256)
    with pytest.raises(ValueError):
        cuda_lib.LinearW4(layer.packed, layer.scales.float(), None, 256)
    with pytest.raises(ValueError):
        cuda_lib.LinearW4(layer.packed, layer.scales, None, 1024)
    with pytest.raises(ValueError):
        layer.qkv(x.view(2, 1, 256), 4, 1, 32)
    with pytest.raises(cuda_lib.InfiniError):
        cuda_lib.LinearW4(layer.packed, layer.scales, None, 250)(x[:, :250].contiguous())
