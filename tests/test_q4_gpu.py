"""GPU parity of the 4-bit segment buffer (append, read back, decode step, state
update) against the float64 oracle.

Codes, scales and minima are compared exactly: both sides round the same fp32
operations once each.  The decode step's tolerance, with every quantity taken
from the oracle's operands (A: the largest sum of magnitudes a score is made of,
in powers of two; R: a group's largest scale times 15, the range its codes span;
V: the largest |value|):
  scores    16 additions of at most 2^-23 of A: every probability within a
            factor of 1 +- 2^-19 A, a weighted mean of values within twice
            that of V;
  bf16      each probability times scale rounded to bf16, half a step 2^-8 of a
            term: together at most 2^-8 of R;
  fp32      the parts that hold a probability keep it to 2^-22 of the largest (R
            is at most twice V: 2^-21 V); the sums over n rows in fp32: 2^-23 V for
            each of the n / 16 / warps + 64 additions in a row, bounded by
            (n / 128 + 64) 2^-23 V;
  retrieval d additions of 2^-24 of the sums of magnitudes;
and half a step of the output's own rounding.
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


def randn(*shape, seed=0, dtype="f32", std=1.0):
    return (std * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(DT[dtype])


def packed(x):
    """The buffer's four arrays for rows x, y [B, H, S, d] = (keys, values)."""
    out = []
    for rows, bit in zip(x, (oracle.key_bit, oracle.value_bit)):
        q, s, m = oracle.cache_codes(rows.float().numpy())
        out.append(torch.from_numpy(oracle.packed_of(q, bit, rows.shape[-1])))
        out.append(torch.from_numpy(np.stack((s, m), -1)).bfloat16())
    return out


def values_of(api_cache):
    """Float64 keys and values of a buffer, by the oracle's reading of its bytes."""
    kc, ks, vc, vs = (t.cpu() for t in api_cache.tensors)
    d = 2 * kc.shape[-1]
    out = []
    for codes, sm, bit in ((kc, ks, oracle.key_bit), (vc, vs, oracle.value_bit)):
        sm = f64(sm)
        out.append(oracle.cache_values(oracle.codes_of(codes.numpy(), d, bit, d).astype(np.float64), sm[..., 0],
                                       sm[..., 1]))
    return out


def bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t


def step_case(api, B, H_q, H_kv, d, S, pos, dtype, seed=0, check=None, workspace=True, beta=None):
    """One decode step; checks the output of streams ``check`` (default all),
    the stored rows, and that nothing else changed."""
    keys = randn(B, H_kv, S, d, seed=seed) * torch.exp(0.4 * randn(H_kv, 1, d, seed=seed + 1))
    cache = [t.cuda() for t in packed((keys, randn(B, H_kv, S, d, seed=seed + 2)))]
    pos_t = torch.tensor(pos, dtype=torch.int32)
    for b in range(B):  # rows behind the token: what must not be read
        n = max(0, pos[b])
        for t in cache:
            t[b, :, n:] = 255 if t.dtype == torch.uint8 else float("nan")
    before = [t.clone() for t in cache]
    q_t, k_t, v_t = randn(B, H_q, d, seed=seed + 3, dtype=dtype), randn(B, H_kv, d, seed=seed + 4, dtype=dtype), \
        randn(B, H_kv, d, seed=seed + 5, dtype=dtype)
    beta = randn(H_q, seed=seed + 6) if beta is None else beta
    z = (1 + S * torch.rand(B, H_kv, d, generator=torch.Generator().manual_seed(seed + 7)))
    M = randn(B, H_kv, d, d, seed=seed + 8, std=math.sqrt(S))
    out = torch.full((B, H_q, d), 3.0, dtype=DT[dtype], device="cuda")
    c = api.CacheQ4(*cache)
    ws = torch.zeros(api.decode_q4_workspace_bytes(B, H_q, H_kv, S, d), dtype=torch.uint8, device="cuda") \
        if workspace else None
    args = (q_t.cuda(), k_t.cuda(), v_t.cuda(), beta.cuda(), c, pos_t.cuda(), M.cuda(), z.cuda())
    api.decode_step_q4(*args, out=out, workspace=ws)
    api.sync_status()
    # the stored rows, and nothing else
    want = packed((k_t[:, :, None], v_t[:, :, None]))
    for t, old, new in zip(cache, before, want):
        for b in range(B):
            if pos[b] >= 0:
                old[b, :, pos[b]] = new[b, :, 0].cuda()
        assert torch.equal(bits(t), bits(old))
    K, V = values_of(c)
    ref = oracle.decode_step_q4(f64(q_t), K, V, pos, f64(beta), f64(M), f64(z))
    got = f64(out)
    q64 = f64(q_t)
    for b in range(B) if check is None else check:
        n = pos[b] + 1
        if n <= 0:
            assert np.all(got[b] == 3.0)
            continue
        for h in range(H_q):
            kv = h // (H_q // H_kv)
            ks, vs = f64(cache[1][b, kv, :n]), f64(cache[3][b, kv, :n])
            ax = np.abs(q64[b, h]).reshape(d // 32, 32).sum(-1)
            A = np.max((15 * ks[..., 0] + np.abs(ks[..., 1])) @ ax) / math.sqrt(d) * math.log2(math.e)
            top = np.max(np.abs(V[b, kv, :n]))
            span = 15 * np.max(vs[..., 0])
            slack = 2 * 2.0 ** -19 * A * top
            slack += 2.0 ** -8 * span if dtype == "bf16" else (n / 128 + 64) * 2.0 ** -23 * top
            sq = oracle.elu_plus_one(q64[b, h])
            slack = slack + (d + 8) * 2.0 ** -24 * 2 * (sq @ np.abs(f64(M)[b, kv])) / (sq @ f64(z)[b, kv])
            err = np.abs(got[b, h] - ref[b, h]) - HALF[dtype] * np.abs(ref[b, h]) - slack
            assert np.all(err <= 0), (b, h, float(err.max()))
    return args, out, ws


STEPS = [
    (1, 1, 1, 32, 1, [0]),
    (4, 4, 2, 32, 16, [-1, 0, 1, 15]),
    (5, 3, 1, 64, 200, [15, 16, -1, 127, 128]),       # unit and tile borders
    (3, 16, 2, 128, 300, [299, 17, 0]),               # 8 heads per KV head
    (2, 24, 2, 64, 140, [129, 31]),                   # 12: a full and a part chunk of heads
    (2, 9, 9, 128, 64, [40, 63]),                     # one head per KV head
    (1, 4, 1, 128, 2048, [2047]),
    (1, 2, 1, 32, 5000, [4999]),
    (4, 4, 2, 32, 16, [-1, -1, -1, -1]),              # nothing to do
    (70, 2, 1, 32, 300, [(37 * b) % 301 - 1 for b in range(70)]),     # more streams than a warp has lanes
    (33, 1, 1, 64, 2000, [-1] * 32 + [1999]),         # the last one alone
    (1100, 1, 1, 32, 40, [b % 41 - 1 for b in range(1100)]),          # more segments than CTAs
    (600, 3, 3, 32, 140, [139 - b % 7 for b in range(600)]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H_q,H_kv,d,S,pos", STEPS)
def test_step(cuda_lib, B, H_q, H_kv, d, S, pos, dtype):
    step_case(cuda_lib, B, H_q, H_kv, d, S, pos, dtype, seed=d + S)


def test_step_without_workspace_and_extreme_gates(cuda_lib):
    beta = torch.tensor([float("inf"), -float("inf"), 0.0, 100.0])
    step_case(cuda_lib, 2, 4, 2, 64, 50, [49, 3], "f32", seed=1, workspace=False, beta=beta)


def test_step_with_many_rows_per_block(cuda_lib):
    """Enough streams that a block takes several units of rows."""
    g = np.random.default_rng(0)
    pos = [int(x) for x in g.integers(0, 1024, 80)]
    pos[3], pos[7], pos[11] = -1, 1023, 0
    step_case(cuda_lib, 80, 8, 8, 32, 1024, pos, "bf16", seed=2, check=[0, 3, 7, 11, 40, 79])


def test_position_out_of_range_is_reported_and_left_alone(cuda_lib):
    api = cuda_lib
    cache = api.CacheQ4.empty(3, 1, 8, 32)
    before = [t.clone() for t in cache.tensors]
    pos = torch.tensor([8, -2, -1], dtype=torch.int32, device="cuda")
    tok = torch.ones(3, 1, 32, device="cuda")
    M, z = torch.zeros(3, 1, 32, 32, device="cuda"), torch.ones(3, 1, 32, device="cuda")
    out = torch.full((3, 2, 32), 5.0, device="cuda")
    api.decode_step_q4(torch.ones(3, 2, 32, device="cuda"), tok, tok, torch.zeros(2, device="cuda"), cache, pos,
                       M, z, out=out)
    with pytest.raises(api.InfiniError) as e:
        api.sync_status()
    assert e.value.status == api.ERR_RANGE
    api.sync_status()
    assert torch.all(out == 5.0)
    cache.append(tok[:, :, None].expand(3, 1, 3, 32).contiguous(), tok[:, :, None].expand(3, 1, 3, 32).contiguous(),
                 torch.tensor([6, -5, -1], dtype=torch.int32, device="cuda"))
    with pytest.raises(api.InfiniError) as e:
        api.sync_status()
    assert e.value.status == api.ERR_RANGE
    for a, b in zip(cache.tensors, before):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_lost_group_takes_nothing_else_with_it(cuda_lib, dtype):
    """A group of values with a NaN or an infinity in an attended row: its 32
    channels are NaN, the others what they are without it, whatever the scales'
    size (first and last rows, so that some are seen before and some after)."""
    api = cuda_lib
    H, d, S = 2, 128, 400
    for size in (1.0, 2.0 ** 60, 2.0 ** 118):
        keys, vals = randn(1, H, S, d, seed=1), randn(1, H, S, d, seed=2) * size
        vals[0, 0, 3, 40], vals[0, 0, 390, 50], vals[0, 1, 200, 96:] = math.nan, -math.inf, math.inf
        cache = api.CacheQ4(*(t.cuda() for t in packed((keys, vals))))
        rows = [randn(1, n, d, seed=3 + n, dtype=dtype) for n in (H, H)]
        q = randn(1, 2 * H, d, seed=9, dtype=dtype)
        M, z = torch.zeros(1, H, d, d), torch.ones(1, H, d)
        beta, pos = torch.full((2 * H,), -100.0), torch.tensor([S - 1], dtype=torch.int32)
        out = f64(api.decode_step_q4(q.cuda(), rows[0].cuda(), rows[1].cuda(), beta.cuda(), cache, pos.cuda(),
                                     M.cuda(), z.cuda()))
        api.sync_status()
        K, V = values_of(cache)
        lost = np.isnan(V).any(2)  # [1, H, d]
        assert lost.sum() == 64
        ref = oracle.decode_step_q4(f64(q), K, np.nan_to_num(V, nan=0.0), [S - 1], f64(beta), f64(M), f64(z))
        for h in range(2 * H):
            gone = lost[0, h // 2]
            assert np.isnan(out[0, h, gone]).all()
            top = np.max(np.abs(V[0, h // 2][:, ~gone]))
            # The docstring's bounds with R <= 2 V, A <= 32, n = 400: bf16 (2^-7 + 2^-13
            # + 2^-8) V < 2^-6 V, fp32 (2^-13 + 2^-16 + 2^-24) V < 2^-12 V.
            err = np.abs(out[0, h] - ref[0, h])[~gone]
            assert np.all(err <= (2.0 ** -6 if dtype == "bf16" else 2.0 ** -12) * top)


def test_offsets_beyond_32_bits(cuda_lib):
    """Rows whose offset passes 2^32 bytes and 2^31 elements: of the last of many
    streams, and of one long stream all of whose rows count."""
    api, d = cuda_lib, 128
    # 40 x 8 x 2^18 rows of 64 bytes; the last stream alone is attended
    B, H, S = 40, 8, 1 << 18
    cache = api.CacheQ4.empty(B, H, S, d)
    n = 70
    k, v = randn(1, H, n, d, seed=1), randn(1, H, n, d, seed=2)
    at = torch.full((B,), -1, dtype=torch.int32)
    at[-1] = S - n
    ks, vs = torch.zeros(B, H, n, d), torch.zeros(B, H, n, d)
    ks[-1], vs[-1] = k[0], v[0]
    cache.append(ks.cuda(), vs.cuda(), at.cuda())
    api.sync_status()
    for got, want in zip(cache.tensors, packed((k, v))):
        assert torch.equal(bits(got[-1, :, S - n:].cpu()), bits(want[0]))
        assert not got[-1, :, S - n - 100:S - n].any() and not got[:4].any()
    del cache
    # one stream of 2^26 + 77 rows, zeros but for the first and the last 64
    S = (1 << 26) + 77
    cache = api.CacheQ4.empty(1, 1, S, d)
    ends = packed((randn(1, 1, 128, d, seed=4), randn(1, 1, 128, d, seed=5)))
    for t, e in zip(cache.tensors, ends):
        t[0, 0, :64], t[0, 0, S - 65:S - 1] = e[0, 0, :64].cuda(), e[0, 0, 64:].cuda()
    q = randn(1, 2, d, seed=6)
    kt, vt = randn(1, 1, d, seed=7), randn(1, 1, d, seed=8)
    q *= 7.0  # largest scores of 17 and 18: they and the zeros count alike
    pos, beta = torch.tensor([S - 1], dtype=torch.int32), torch.full((2,), -100.0)
    out = f64(api.decode_step_q4(q.cuda(), kt.cuda(), vt.cuda(), beta.cuda(), cache, pos.cuda(),
                                 torch.zeros(1, 1, d, d, device="cuda"), torch.ones(1, 1, d, device="cuda")))
    api.sync_status()
    tail = [torch.cat((t[0, 0, :64], t[0, 0, S - 65:])).cpu() for t in cache.tensors]
    K, V = (oracle.cache_values(oracle.codes_of(c.numpy(), d, bit, d).astype(np.float64), f64(s)[..., 0],
                                f64(s)[..., 1])
            for c, s, bit in ((tail[0], tail[1], oracle.key_bit), (tail[2], tail[3], oracle.value_bit)))
    for h in range(2):
        s = K @ f64(q)[0, h] / math.sqrt(d)
        m = max(s.max(), 0.0)
        p = np.exp(s - m)
        ref = p @ V / (p.sum() + (S - len(s)) * math.exp(-m))
        A = (np.abs(K) @ np.abs(f64(q)[0, h])).max() / math.sqrt(d) * math.log2(math.e)
        # the zeros' sum: a lane adds 2 of every 16 rows that its warp has, of 296 CTAs' 4 or
        # more: below 2^12 additions in a row
        slack = (2 * 2.0 ** -19 * A + 2.0 ** 12 * 2.0 ** -23) * np.abs(V).max()
        assert 15.0 < m < 20.0 and np.all(np.abs(out[0, h] - ref) <= slack), float(np.abs(out[0, h] - ref).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_append_and_read(cuda_lib, d, dtype):
    api = cuda_lib
    B, H, S, n = 3, 2, 40, 7
    cache = api.CacheQ4.empty(B, H, S, d)
    k, v = randn(B, H, n, d, seed=d, dtype=dtype), randn(B, H, n, d, seed=d + 1, dtype=dtype)
    k[0, 0, 0], k[0, 0, 1], v[1, 1, 2] = 0.0, -2.5, 1e-30   # groups without a range
    k[2, 1, 6, 3] = float("nan")
    pos = [33, 0, -1]
    cache.append(k.cuda(), v.cuda(), torch.tensor(pos, dtype=torch.int32, device="cuda"))
    rk, rv = cache.read(S, DT[dtype])
    api.sync_status()
    for x, r, bit, at in ((k, rk, oracle.key_bit, 0), (v, rv, oracle.value_bit, 2)):
        q, s, m = oracle.cache_codes(x.float().numpy())
        want = np.zeros((B, H, S, d))
        codes = np.zeros((B, H, S, d // 2), np.uint8)
        for b in range(B):
            if pos[b] >= 0:
                want[b, :, pos[b]:pos[b] + n] = oracle.cache_values(q.astype(np.float64), s, m)[b]
                codes[b, :, pos[b]:pos[b] + n] = oracle.packed_of(q, bit, d)[b]
        assert np.array_equal(cache.tensors[at].cpu().numpy(), codes)
        got = f64(r)
        if dtype == "bf16":
            want = oracle.bf16(want.astype(np.float32))  # fp32 sum, rounded to bf16
        assert np.all(np.abs(got - want) <= 2.0 ** -24 * np.abs(want)) if dtype == "f32" else np.array_equal(got, want)
    # a NaN takes its group with it and nothing else
    cache.append(k.cuda(), v.cuda(), torch.tensor([-1, -1, 10], dtype=torch.int32, device="cuda"))
    rk, _ = cache.read(S)
    assert torch.isnan(rk[2, 1, 16, :32]).all()
    assert torch.isnan(rk).sum() == 32


def test_codes_at_ties_and_extreme_scales(cuda_lib):
    """Codes, scales and minima stay the definition's where a quotient is a half
    or next to one in fp32, and for scales from bf16's smallest to its largest."""
    api, g = cuda_lib, np.random.default_rng(3)
    n, d = 600, 64
    x = np.zeros((1, 2, n, d // 32, 32), np.float32)  # heads as two more sets of groups
    shape = x.shape[:-1]
    power = g.integers(-133, 122, shape)
    mant = g.integers(128, 256, shape)
    s = oracle.bf16(np.ldexp(mant.astype(np.float64), power - 7).astype(np.float32)).astype(np.float32)
    half = g.integers(0, 15, shape + (30,)).astype(np.float32) + np.float32(0.5)
    at = (half * s[..., None]).astype(np.float32)
    side = g.integers(0, 3, at.shape)
    at = np.where(side == 0, np.nextafter(at, np.float32(0)), np.where(side == 1, at, np.nextafter(at, np.float32(np.inf))))
    x[..., 0], x[..., 1], x[..., 2:] = 0.0, 15 * s, at
    x = x.reshape(1, 2, n, d)
    cache = api.CacheQ4.empty(1, 2, n, d)
    k, v = torch.from_numpy(x), torch.from_numpy(x[:, ::-1].copy())
    cache.append(k.cuda(), v.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"))
    api.sync_status()
    for got, want in zip(cache.tensors, packed((k, v))):
        assert torch.equal(bits(got.cpu()), bits(want))


@pytest.mark.parametrize("rule", ["linear", "delta"])
@pytest.mark.parametrize("dtype,d", [("f32", 32), ("bf16", 64), ("bf16", 128)])
def test_state_update(cuda_lib, dtype, d, rule):
    api = cuda_lib
    B, H, S = 2, 2, 70
    cache = api.CacheQ4(*(t.cuda() for t in packed((randn(B, H, S, d, seed=1), randn(B, H, S, d, seed=2)))))
    M0 = randn(B, H, d, d, seed=3).cuda()
    z0 = (5 + torch.rand(B, H, d, generator=torch.Generator().manual_seed(4))).cuda()
    for n in (1, 37, S):
        M, z = cache.state_update(n, M0, z0, rule, DT[dtype])
        k, v = cache.read(n, DT[dtype])
        M2, z2 = api.state_update(k, v, M0, z0, n, rule)
        assert torch.equal(M, M2) and torch.equal(z, z2)
        ws = torch.full((api.state_update_q4_workspace_bytes(B, H, n, d, rule, DT[dtype]),), 255,
                        dtype=torch.uint8, device="cuda")
        Mi, zi = M0.clone(), z0.clone()
        cache.state_update(n, Mi, zi, rule, DT[dtype], Mi, zi, workspace=ws)
        assert torch.equal(Mi, M) and torch.equal(zi, z)
        one = cache.row(1).state_update(n, M0[1:].clone(), z0[1:].clone(), rule, DT[dtype])
        assert torch.equal(one[0], M[1:]) and torch.equal(one[1], z[1:])
    api.sync_status()


@pytest.mark.parametrize("dtype,d,rule", [("f32", 32, "delta"), ("bf16", 64, "linear"), ("bf16", 128, "delta")])
def test_stream(cuda_lib, dtype, d, rule):
    """Token by token over several segments, the memory update included: each
    step against the oracle on the buffer's values and the stream's memory."""
    api = cuda_lib
    B, H_q, H_kv, S, L = 2, 4, 2, 9, 23
    q, k, v = (randn(B, L, h, d, seed=i, dtype=dtype) for i, h in ((1, H_q), (2, H_kv), (3, H_kv)))
    beta = randn(H_q, seed=4)
    st = api.DecodeStreamQ4(B, H_q, H_kv, d, S, rule, dtype=DT[dtype])
    for t in range(L):
        M, z = f64(st.M), f64(st.z)
        out = st.step(q[:, t].contiguous().cuda(), k[:, t].contiguous().cuda(), v[:, t].contiguous().cuda(),
                      beta.cuda())
        K, V = values_of(st.cache)
        ref = oracle.decode_step_q4(f64(q[:, t]), K, V, [t % S] * B, f64(beta), M, z)
        # n <= 9 rows of N(0, 1): spans below 10, scores' A below 2^8, values
        # below 6, retrieval a weighted mean of them
        slack = 2 * 2.0 ** -11 * 6 + 2.0 ** -8 * 10 if dtype == "bf16" else 2 * 2.0 ** -11 * 6
        assert np.all(np.abs(f64(out) - ref) <= HALF[dtype] * np.abs(ref) + slack)
        assert st.pos == (t + 1) % S
    M, z = st.final_state()
    k2, v2 = st.cache.read(L % S, DT[dtype])
    M2, z2 = api.state_update(k2, v2, st.M, st.z, L % S, rule)
    assert torch.equal(M, M2) and torch.equal(z, z2)
    api.sync_status()


def test_repeats_streams_and_graphs(cuda_lib):
    """Bitwise repeats; another stream; one captured step that serves other
    positions; two graphs at once with a workspace each."""
    api = cuda_lib
    args, out, ws = step_case(api, 3, 8, 2, 128, 600, [599, 130, -1], "bf16", seed=5)
    first = out.clone()
    for _ in range(3):
        api.decode_step_q4(*args, out=out, workspace=ws)
    assert torch.equal(out, first)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = torch.full_like(out, 3.0)
    torch.cuda.synchronize()
    api.decode_step_q4(*args, out=got, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(got, first)
    graphs, outs = [], []
    for _ in range(2):
        w, o = torch.zeros_like(ws), torch.full_like(out, 3.0)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.decode_step_q4(*args, out=o, workspace=w)
        graphs.append((g, w))
        outs.append(o)
    for p in ([599, 130, -1], [10, -1, 300], [0, 0, 0]):
        args[5].copy_(torch.tensor(p, dtype=torch.int32))
        want = outs[0].clone()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
        graphs[0][0].replay()
        torch.cuda.synchronize()
        api.decode_step_q4(*args, out=want, workspace=ws)
        # by their bits: stream 2's buffer holds NaN rows (see step_case), and
        # at position 300 its output is the formula's NaN
        assert torch.equal(bits(outs[0]), bits(want)) and torch.equal(bits(outs[1]), bits(want))


def test_binding_refuses(cuda_lib):
    api = cuda_lib
    cache = api.CacheQ4.empty(2, 2, 8, 64)
    q, k = torch.zeros(2, 4, 64, device="cuda"), torch.zeros(2, 2, 64, device="cuda")
    beta, pos = torch.zeros(4, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    M, z = torch.zeros(2, 2, 64, 64, device="cuda"), torch.zeros(2, 2, 64, device="cuda")

    def step(q=q, k=k, v=k, beta=beta, pos=pos, M=M, z=z, **kw):
        return api.decode_step_q4(q, k, v, beta, cache, pos, M, z, **kw)

    step()
    for bad in (dict(q=q.half()), dict(k=k.bfloat16()), dict(v=k[:, :1]), dict(beta=beta[:2]), dict(pos=pos.long()),
                dict(M=M.double()), dict(z=z.cpu()), dict(q=q[:1]), dict(out=q.bfloat16()),
                dict(workspace=torch.zeros(8, device="cuda"))):
        with pytest.raises(ValueError):
            step(**bad)
    with pytest.raises(api.InfiniError):
        step(q=torch.zeros(2, 3, 64, device="cuda"), beta=beta[:3].contiguous())   # 3 heads over 2
    with pytest.raises(api.InfiniError):
        step(out=q)                                                               # the output over the queries
    with pytest.raises(api.InfiniError):
        step(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(api.InfiniError):
        cache.read(9)
    with pytest.raises(ValueError):
        cache.append(torch.zeros(2, 2, 3, 32, device="cuda"), torch.zeros(2, 2, 3, 32, device="cuda"), pos)
    t = cache.tensors
    with pytest.raises(ValueError):
        api.CacheQ4(t[0], t[1].float(), t[2], t[3])
    with pytest.raises(ValueError):
        api.CacheQ4(t[0][..., :8].contiguous(), t[1], t[2], t[3])
