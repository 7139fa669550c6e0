"""Cases for measuring the serving and training operators around the layer.

Three operators, each next to an entry point of the library:

  block_norm   the normalisations before and after the layer, fused with the
               block's gate, its residual scale and the residual sum, forward
               and backward;
  w4           projections of a few tokens with weights in 4 bits and a scale
               for each group of input channels (a plain linear layer, and the
               query/key/value projection with its rotary embedding);
  q4           the decode step over a segment buffer held in 4 bits, and the
               filling and reading back of that buffer.

``run`` computes a pass in plain torch operations in 32 bits, or, where
``own`` is true, by the calls a user makes of the library.  ``exact`` computes
the definitions in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # The residual stream of one new token (the 8B shape's width): the
        # smallest call of a decode loop, latency alone.
        dict(name="norm_token", op="norm", rows=1, width=4096, dtype="bf16", block=True, post=True,
             gate=True, scale=True, next=True, backward=False),
        # The 8B shape's whole prompt batch, 2 x 32768 tokens.
        dict(name="norm_prompt", op="norm", rows=65536, width=4096, dtype="bf16", block=True, post=True,
             gate=True, scale=True, next=True, backward=False),
        # A plain norm before the block, in fp32, ragged on both axes.
        dict(name="norm_odd_f32", op="norm", rows=1003, width=1019, dtype="f32", block=False, post=False,
             gate=False, scale=False, next=True, backward=False),
        # A training step of the 200M shape (8 x 1024 tokens, 12 heads of 64).
        dict(name="norm_bwd_200m", op="norm", rows=8192, width=768, dtype="bf16", block=True, post=True,
             gate=True, scale=True, next=True, backward=True),
        # A training micro-batch at the 8B shape's width.
        dict(name="norm_bwd_8b", op="norm", rows=16384, width=4096, dtype="bf16", block=True, post=True,
             gate=True, scale=True, next=True, backward=True),
        # One token through the 8B shape's query/key/value projection.
        dict(name="w4_qkv_token", op="w4", kind="qkv", tokens=1, K=4096, H_q=32, H_kv=8, d=128, group=128,
             zeros=False, bias=False, dtype="bf16"),
        # Sixteen streams at once through a wide layer, zero points and all.
        dict(name="w4_wide_16", op="w4", kind="linear", tokens=16, K=4096, N=16384, group=64, zeros=True,
             bias=True, dtype="bf16"),
        # fp32 tokens, sizes that fill no tile, small groups.
        dict(name="w4_odd_f32", op="w4", kind="linear", tokens=3, K=1000, N=777, group=32, zeros=True,
             bias=False, dtype="f32"),
        # The 8B shape's decode step at the end of a 2048-token segment.
        dict(name="q4_step_8b", op="q4", kind="step", B=2, H_q=32, H_kv=8, d=128, S=2048, ragged=False,
             dtype="bf16"),
        # A serving batch of 64 streams with long segments, all at their own
        # positions.
        dict(name="q4_step_64x8192", op="q4", kind="step", B=64, H_q=32, H_kv=8, d=128, S=8192, ragged=True,
             dtype="bf16"),
        # fp32 streams of the 300M shape's heads, one of them idle.
        dict(name="q4_step_f32", op="q4", kind="step", B=3, H_q=16, H_kv=16, d=64, S=2048, ragged=True,
             dtype="f32"),
        # Eight prompts of ragged starts written into the cache and read back
        # for the memory update.
        dict(name="q4_fill", op="q4", kind="fill", B=8, H_kv=8, d=128, S=2048, n=1500, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "w4", "w4", "q4", "q4"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        width = _log(rng, 32, 8192)
        if rng.random() < 0.6:
            width = max(8, width // 8 * 8)
        rows = _log(rng, 1, 65536)
        backward = rng.random() < 0.5
        cost = 2 if dtype == "f32" else 1
        rows = max(1, min(rows, (65536 * 4096) // (width * cost * (2 if backward else 1))))
        block, post = rng.random() < 0.75, rng.random() < 0.7
        return dict(op=op, rows=rows, width=width, dtype=dtype, block=block, post=block and post,
                    gate=block and rng.random() < 0.6, scale=block and (not post or rng.random() < 0.6),
                    next=not block or rng.random() < 0.7, backward=backward)
    if op == "w4":
        tokens, group = _log(rng, 1, 64), rng.choice([32, 64, 128])
        K = max(8, _log(rng, 64, 8192) // 8 * 8)
        more = dict(group=group, zeros=rng.random() < 0.5, bias=rng.random() < 0.5, dtype=dtype)
        if rng.random() < 0.4:
            d, H_kv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
            return dict(op=op, kind="qkv", tokens=tokens, K=K, H_q=H_kv * rng.choice([1, 2, 3, 4]),
                        H_kv=H_kv, d=d, **more)
        return dict(op=op, kind="linear", tokens=tokens, K=K, N=_log(rng, 16, 16384), **more)
    d, H_kv, B = rng.choice([32, 64, 128]), rng.choice([1, 2, 4, 8]), _log(rng, 1, 64)
    S = _log(rng, 16, 32768)
    S = max(1, min(S, (64 * 8 * 8192 * 128) // (B * H_kv * d)))
    if rng.random() < 0.3:
        S = min(S, (64 * 8 * 2048 * 128) // (B * H_kv * d) // 4 + 1)
        return dict(op=op, kind="fill", B=B, H_kv=H_kv, d=d, S=S, n=max(1, int(S * rng.uniform(0.1, 0.9))),
                    dtype=dtype)
    return dict(op=op, kind="step", B=B, H_q=H_kv * rng.choice([1, 2, 4, 8]), H_kv=H_kv, d=d, S=S,
                ragged=rng.random() < 0.7, dtype=dtype)


# ------------------------------------------------------------- 4-bit layouts
#
# Key rows and weight rows: for each block of D channels (D = d for a key row,
# 128 for a weight row), 4 chunks of D / 32 little-endian 32-bit words; word j
# of chunk c holds channels 32 j + 8 c .. + 7, the even ones in its low half
# and the odd ones in its high half, lowest first.  Value rows: 8 chunks of
# D / 32 16-bit words; word j of chunk i holds channels 32 j + 4 i .. + 3,
# lowest first.


def _nibbles(b):
    return torch.stack((b & 15, b >> 4), -1)


def _unpack_k(codes, D=None):
    """uint8 [..., n / 2] -> uint8 codes [..., n] in channel order."""
    lead, half = codes.shape[:-1], codes.shape[-1]
    D = D or 2 * half
    x = _nibbles(codes).view(*lead, 2 * half // D, 4, D // 32, 2, 2, 2)  # blk c j bh bl n
    k = len(lead)
    x = x.permute(*range(k), k, k + 2, k + 1, k + 4, k + 5, k + 3)       # blk j c bl n bh
    return x.reshape(*lead, 2 * half)


def _pack_k(q, D=None):
    lead, n = q.shape[:-1], q.shape[-1]
    D = D or n
    k = len(lead)
    x = q.view(*lead, n // D, D // 32, 4, 2, 2, 2)                       # blk j c bl n bh
    x = x.permute(*range(k), k, k + 2, k + 1, k + 5, k + 3, k + 4)       # blk c j bh bl n
    return (x[..., 0] | (x[..., 1] << 4)).reshape(*lead, n // 2)


def _unpack_v(codes):
    lead, half = codes.shape[:-1], codes.shape[-1]
    k = len(lead)
    x = _nibbles(codes).view(*lead, 8, half // 16, 2, 2)                 # i j byte n
    return x.permute(*range(k), k + 1, k, k + 2, k + 3).reshape(*lead, 2 * half)


def _pack_v(q):
    lead, n = q.shape[:-1], q.shape[-1]
    k = len(lead)
    x = q.view(*lead, n // 32, 8, 2, 2).permute(*range(k), k + 1, k, k + 2, k + 3)
    return (x[..., 0] | (x[..., 1] << 4)).reshape(*lead, n // 2)


def _quantise(x):
    """fp32 [..., d] -> (codes uint8 [..., d], bf16 [..., d / 32, 2] of scale
    and minimum): 32-channel groups, value = scale code + minimum."""
    g = x.view(*x.shape[:-1], x.shape[-1] // 32, 32)
    lo, hi = g.amin(-1), g.amax(-1)
    m = lo.bfloat16()
    s = ((hi - m.float()).clamp_min(0) * (1 / 15)).bfloat16()
    step = s.float()[..., None]
    q = torch.where(step > 0, ((g - m.float()[..., None]) / step).round().clamp(0, 15), torch.zeros_like(g))
    return q.to(torch.uint8).view(x.shape), torch.stack((s, m), -1)


def _values(q, sm, dtype=torch.float32):
    g = q.view(*q.shape[:-1], q.shape[-1] // 32, 32).to(dtype)
    return (g * sm[..., 0:1].to(dtype) + sm[..., 1:2].to(dtype)).view(q.shape)


# ------------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    def rand(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    s = dict(case=dict(case))
    if case["op"] == "norm":
        R, D = case["rows"], case["width"]
        # A residual stream: a few channels much larger than the others.
        chan = torch.exp(randn(D, std=0.5))
        s["r"] = (randn(R, D) * chan).to(dt)
        s["o"] = randn(R, D, std=0.7).to(dt) if case["block"] else None
        s["gate"] = randn(R, D, std=1.5).to(dt) if case["gate"] else None
        s["scale"] = 0.1 + 0.5 * rand(D) if case["scale"] else None
        s["w_post"] = 1 + randn(D, std=0.1) if case["post"] else None
        s["w_next"] = 1 + randn(D, std=0.1) if case["next"] else None
        if case["backward"]:
            # What the forward left: the stream after the block and the
            # reciprocal norms.
            r_out, _, rp, rn = _norm_forward(s)
            s["r_out"] = r_out if case["block"] else s["r"]
            s["rstd_post"], s["rstd_next"] = rp, rn
            s["dr_out"] = randn(R, D, std=1e-2).to(dt)
            s["dh"] = randn(R, D, std=1e-2).to(dt) if case["next"] else None
        return s
    if case["op"] == "w4":
        K, G, M = case["K"], case["group"], case["tokens"]
        N = case["N"] if case["kind"] == "linear" else (case["H_q"] + 2 * case["H_kv"]) * case["d"]
        Kp = -(-K // 128) * 128
        q = (7.5 + randn(N, Kp, std=2.7)).round().clamp(0, 15).to(torch.uint8)
        s["packed"] = _pack_k(q, 128)
        s["scales"] = ((0.6 + 0.8 * rand(N, Kp // G)) / (2.7 * math.sqrt(K))).bfloat16()
        s["scales"][:, -(-K // G):] = 0
        s["zeros"] = torch.randint(6, 10, (N, Kp // G), generator=g, device="cuda").to(torch.uint8) \
            if case["zeros"] else None
        s["bias"] = randn(N, std=0.1) if case["bias"] else None
        if case["kind"] == "linear":
            s["x"] = randn(M, K).to(dt)
        else:
            s["x"] = randn(M, 1, K).to(dt)
            n_pos, d = 4096, case["d"]
            ang = torch.arange(n_pos, device="cuda", dtype=torch.float64)[:, None] * \
                10000.0 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
            s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
            s["positions"] = torch.randint(0, n_pos, (M, 1), generator=g, device="cuda").int()
        return s
    B, H, d, S = case["B"], case["H_kv"], case["d"], case["S"]
    chan = torch.exp(randn(H, 1, d, std=0.4))  # keys have large channels

    def rows(*shape, scale=None):
        x = randn(*shape)
        return (x * scale if scale is not None else x).to(dt)

    if case["kind"] == "fill":
        s["k"], s["v"] = rows(B, H, case["n"], d, scale=chan), rows(B, H, case["n"], d)
        s["pos"] = torch.randint(0, S - case["n"] + 1, (B,), generator=g, device="cuda").int()
        s["cache"] = (torch.zeros(B, H, S, d // 2, dtype=torch.uint8, device="cuda"),
                      torch.zeros(B, H, S, d // 32, 2, dtype=torch.bfloat16, device="cuda"),
                      torch.zeros(B, H, S, d // 2, dtype=torch.uint8, device="cuda"),
                      torch.zeros(B, H, S, d // 32, 2, dtype=torch.bfloat16, device="cuda"))
        return s
    kc = torch.empty(B, H, S, d // 2, dtype=torch.uint8, device="cuda")
    ks = torch.empty(B, H, S, d // 32, 2, dtype=torch.bfloat16, device="cuda")
    vc, vs = torch.empty_like(kc), torch.empty_like(ks)
    step = max(1, (1 << 27) // (H * S * d))
    for b in range(0, B, step):
        n = min(step, B - b)
        q, ks[b:b + n] = _quantise(rows(n, H, S, d, scale=chan).float())
        kc[b:b + n] = _pack_k(q)
        q, vs[b:b + n] = _quantise(rows(n, H, S, d).float())
        vc[b:b + n] = _pack_v(q)
    s["cache"] = (kc, ks, vc, vs)
    s["q_t"] = rows(B, case["H_q"], d)
    s["k_t"], s["v_t"] = rows(B, H, d, scale=chan[:, 0]), rows(B, H, d)
    s["beta"] = 8 * rand(case["H_q"]) - 4
    s["z"] = S * (0.9 + 0.4 * rand(B, H, d))
    s["M"] = randn(B, H, d, d) * (1.3 * math.sqrt(S))
    if case["ragged"]:
        pos = torch.randint(0, S, (B,), generator=g, device="cuda").int()
        if B > 2:
            pos[1] = -1  # an idle stream
        s["pos"] = pos
    else:
        s["pos"] = torch.full((B,), S - 1, dtype=torch.int32, device="cuda")
    s["out"] = torch.zeros(B, case["H_q"], d, dtype=dt, device="cuda")
    return s


# -------------------------------------------------------------- plain forms


def _norm_forward(s):
    r, o = s["r"].float(), s["o"]
    dt, rp, rn, h, r_out = s["r"].dtype, None, None, None, None
    if o is not None:
        u = o.float()
        if s["w_post"] is not None:
            rp = torch.rsqrt((u * u).mean(-1) + EPS)
            u = u * rp[:, None] * s["w_post"]
        if s["gate"] is not None:
            u = u / (1 + torch.exp(-s["gate"].float()))
        if s["scale"] is not None:
            u = u * s["scale"]
        r = r + u
        r_out = r.to(dt)
    if s["w_next"] is not None:
        rn = torch.rsqrt((r * r).mean(-1) + EPS)
        h = (r * rn[:, None] * s["w_next"]).to(dt)
    return r_out, h, rp, rn


def _norm_backward(s):
    dt, G = s["r"].dtype, s["dr_out"].float()
    got = dict(do=None, dgate=None, dscale=None, dw_post=None, dw_next=None)
    if s["w_next"] is not None:
        n, dh = s["r_out"].float() * s["rstd_next"][:, None], s["dh"].float()
        got["dw_next"] = (dh * n).sum(0)
        e = dh * s["w_next"]
        G = G + (e - n * (e * n).mean(-1, keepdim=True)) * s["rstd_next"][:, None]
    got["dr"] = G.to(dt)
    if s["o"] is None:
        return got
    n, w = s["o"].float(), 1.0
    if s["w_post"] is not None:
        n, w = n * s["rstd_post"][:, None], s["w_post"]
    c, u = s["scale"] if s["scale"] is not None else 1.0, 1.0
    if s["gate"] is not None:
        u = 1 / (1 + torch.exp(-s["gate"].float()))
        got["dgate"] = (G * c * (n * w) * u * (1 - u)).to(dt)
    if s["scale"] is not None:
        got["dscale"] = (G * u * (n * w)).sum(0)
    e = G * c * u
    if s["w_post"] is not None:
        got["dw_post"] = (e * n).sum(0)
        e = e * w
        e = (e - n * (e * n).mean(-1, keepdim=True)) * s["rstd_post"][:, None]
    got["do"] = e.to(dt)
    return got


def _rope(y, cos, sin):
    h = y.shape[-1] // 2
    return torch.cat((y[..., :h] * cos - y[..., h:] * sin, y[..., h:] * cos + y[..., :h] * sin), -1)


def _w4(s, case):
    K, G = case["K"], case["group"]
    q = _unpack_k(s["packed"], 128)
    q = q.view(q.shape[0], -1, G).float()
    z = s["zeros"].float()[..., None] if s["zeros"] is not None else 8.0
    w = ((q - z) * s["scales"].float()[..., None]).view(q.shape[0], -1)[:, :K]
    y = s["x"].float().view(-1, K) @ w.t()
    if s["bias"] is not None:
        y = y + s["bias"]
    dt = s["x"].dtype
    if case["kind"] == "linear":
        return dict(y=y.to(dt))
    H_q, H_kv, d, M = case["H_q"], case["H_kv"], case["d"], case["tokens"]
    y = y.view(M, H_q + 2 * H_kv, 1, d)
    at = s["positions"].long().view(M)
    cos, sin = s["cos"][at][:, None, None], s["sin"][at][:, None, None]
    return dict(q=_rope(y[:, :H_q], cos, sin).to(dt), k=_rope(y[:, H_q:H_q + H_kv], cos, sin).to(dt),
                v=y[:, H_q + H_kv:].to(dt))


def _elu1(x):
    return torch.where(x > 0, x + 1, torch.exp(x))


def _q4_fill(s, case):
    kc, ks, vc, vs = s["cache"]
    b = torch.arange(case["B"], device="cuda")[:, None]
    at = s["pos"].long()[:, None] + torch.arange(case["n"], device="cuda")
    k, k_new = _quantise(s["k"].float())
    v, v_new = _quantise(s["v"].float())
    kc[b, :, at] = _pack_k(k).transpose(1, 2)
    vc[b, :, at] = _pack_v(v).transpose(1, 2)
    ks[b, :, at] = k_new.transpose(1, 2)
    vs[b, :, at] = v_new.transpose(1, 2)
    dt = s["k"].dtype
    return dict(k=_values(_unpack_k(kc), ks).to(dt), v=_values(_unpack_v(vc), vs).to(dt))


def _q4_step(s, case):
    B, H, d, S = case["B"], case["H_kv"], case["d"], case["S"]
    kc, ks, vc, vs = s["cache"]
    pos = s["pos"].long()
    live = pos >= 0
    b, at = torch.arange(B, device="cuda"), pos.clamp_min(0)
    k, k_new = _quantise(s["k_t"].float())
    v, v_new = _quantise(s["v_t"].float())
    kc[b, :, at] = torch.where(live[:, None, None], _pack_k(k), kc[b, :, at])
    vc[b, :, at] = torch.where(live[:, None, None], _pack_v(v), vc[b, :, at])
    ks[b, :, at] = torch.where(live[:, None, None, None], k_new, ks[b, :, at])
    vs[b, :, at] = torch.where(live[:, None, None, None], v_new, vs[b, :, at])
    q = s["q_t"].float().view(B, H, -1, d)
    K = _values(_unpack_k(kc), ks)
    score = (q @ K.transpose(2, 3)) / math.sqrt(d)
    del K
    seen = torch.arange(S, device="cuda") <= at[:, None]
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    a_dot = p @ _values(_unpack_v(vc), vs)
    sq = _elu1(q)
    a_mem = (sq @ s["M"]) / (sq @ s["z"][..., None])
    gate = (1 / (1 + torch.exp(-s["beta"]))).view(1, H, -1, 1)
    o = (gate * a_mem + (1 - gate) * a_dot).view(s["out"].shape).to(s["out"].dtype)
    s["out"].copy_(torch.where(live[:, None, None], o, s["out"]))
    return dict(out=s["out"], cache=list(s["cache"]))


# ---------------------------------------------------------------------- run


def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "norm":
        if case["backward"]:
            return _norm_backward(s)
        r_out, h, rp, rn = _norm_forward(s)
        return dict(r_out=r_out, h=h, rstd_post=rp, rstd_next=rn)
    if case["op"] == "w4":
        return _w4(s, case)
    return _q4_fill(s, case) if case["kind"] == "fill" else _q4_step(s, case)


def _run_own(s, case):
    """The calls of a user's program: it keeps its weights' handle, its cache
    and its workspaces from one call to the next."""
    from compressive_memory_transformer_segment_b200 import api

    if case["op"] == "norm":
        if not case["backward"]:
            r_out, h, rp, rn = api.block_norm(s["r"], s["w_next"], EPS, o=s["o"], gate=s["gate"],
                                              scale=s["scale"], w_post=s["w_post"])
            return dict(r_out=r_out, h=h, rstd_post=rp, rstd_next=rn)
        if "workspace" not in s:
            n = api.block_norm_backward_workspace_bytes(case["rows"], case["width"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        g = api.block_norm_backward(s["dr_out"], s["dh"], s["r_out"], s["rstd_next"], s["w_next"], o=s["o"],
                                    gate=s["gate"], scale=s["scale"], w_post=s["w_post"],
                                    rstd_post=s["rstd_post"], workspace=s["workspace"])
        return dict(dr=g.dr, do=g.do, dgate=g.dgate, dscale=g.dscale, dw_post=g.dw_post, dw_next=g.dw_next)
    if case["op"] == "w4":
        if "layer" not in s:
            s["layer"] = api.LinearW4(s["packed"], s["scales"], s["zeros"], case["K"], bias=s["bias"])
        if case["kind"] == "linear":
            return dict(y=s["layer"](s["x"]))
        q, k, v = s["layer"].qkv(s["x"], case["H_q"], case["H_kv"], case["d"], s["cos"], s["sin"],
                                 s["positions"])
        return dict(q=q, k=k, v=v)
    if "q4" not in s:
        s["q4"] = api.CacheQ4(*s["cache"])
    if case["kind"] == "fill":
        s["q4"].append(s["k"], s["v"], s["pos"])
        k, v = s["q4"].read(case["S"], s["k"].dtype)
        return dict(k=k, v=v)
    if "workspace" not in s:
        s["workspace"] = torch.zeros(api.decode_q4_workspace_bytes(case["B"], case["H_q"], case["H_kv"],
                                                                   case["S"], case["d"]),
                                     dtype=torch.uint8, device="cuda")
    api.decode_step_q4(s["q_t"], s["k_t"], s["v_t"], s["beta"], s["q4"], s["pos"], s["M"], s["z"],
                       out=s["out"], workspace=s["workspace"])
    return dict(out=s["out"], cache=list(s["cache"]))


# --------------------------------------------------------------------- work


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        R, D = case["rows"], case["width"]
        reads = 1 + case["block"] + case["gate"]
        writes = case["block"] + case["next"]
        vec = case["scale"] + case["post"] + case["next"]
        stats = 4 * R * (case["post"] + case["next"])
        flops = 10 * R * D
        if case["backward"]:
            # without a next norm neither r_out and dh nor another dr are needed
            reads = 1 + 2 * case["next"] + case["block"] + case["gate"]
            writes = case["next"] + case["block"] + case["gate"]
            vec, flops = 2 * vec, 25 * R * D
        return dict(bytes=e * R * D * (reads + writes) + 4 * vec * D + stats, flops=flops)
    if case["op"] == "w4":
        K, G, M = case["K"], case["group"], case["tokens"]
        N = case["N"] if case["kind"] == "linear" else (case["H_q"] + 2 * case["H_kv"]) * case["d"]
        weights = N * K // 2 + N * -(-K // G) * (2 + case["zeros"])
        rot = M * case["d"] * 4 + 4 * M if case["kind"] == "qkv" else 0
        return dict(bytes=weights + e * M * (K + N) + 4 * N * case["bias"] + rot, flops=2 * M * N * K)
    B, H, d, S = case["B"], case["H_kv"], case["d"], case["S"]
    row = 2 * (d // 2 + 4 * (d // 32))  # key and value codes, scales and minima
    if case["kind"] == "fill":
        n = case["n"]
        return dict(bytes=B * H * (2 * n * d * e + n * row + (S - n) * row + 2 * S * d * e), flops=4 * B * H * S * d)
    # A ragged batch is half full on average.
    seen = S if not case["ragged"] else S / 2
    H_q = case["H_q"]
    mem = 4 * B * H * (d * d + d)
    io = e * B * d * (2 * H_q + 2 * H)
    return dict(bytes=B * H * seen * row + mem + io, flops=4 * B * H_q * d * (seen + d / 2))


# -------------------------------------------------------------------- exact


def exact(case, seed):
    s = prepare(case, seed)
    f = {k: (v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v) for k, v in s.items()}
    if case["op"] == "norm":
        return _exact_backward(f, case) if case["backward"] else _exact_forward(f, case)
    if case["op"] == "w4":
        return _exact_w4(f, case)
    if case["kind"] == "fill":
        return _exact_fill(s, case)
    return dict(out=_exact_step(s, case), cache=[None] * 4)


def _sigmoid64(a):
    return torch.where(a >= 0, 1 / (1 + torch.exp(-a.abs())), torch.exp(-a.abs()) / (1 + torch.exp(-a.abs())))


def _exact_forward(f, case):
    D = case["width"]
    blocks = []
    for i in range(0, case["rows"], 4096):
        cut = slice(i, i + 4096)
        x, rp, rn, h = f["r"][cut], None, None, None
        if case["block"]:
            t = f["o"][cut]
            if case["post"]:
                rp = 1 / torch.sqrt(torch.linalg.vector_norm(t, dim=1) ** 2 / D + EPS)
                t = torch.einsum("rd,r,d->rd", t, rp, f["w_post"])
            if case["gate"]:
                t = t * _sigmoid64(f["gate"][cut])
            if case["scale"]:
                t = torch.einsum("rd,d->rd", t, f["scale"])
            x = x + t
        if case["next"]:
            rn = 1 / torch.sqrt(torch.linalg.vector_norm(x, dim=1) ** 2 / D + EPS)
            h = torch.einsum("rd,r,d->rd", x, rn, f["w_next"])
        blocks.append((x if case["block"] else None, h, rp, rn))
    join = [None if part[0] is None else torch.cat(part) for part in zip(*blocks)]
    return dict(r_out=join[0], h=join[1], rstd_post=join[2], rstd_next=join[3])


def _normed_vjp(x, rstd, w, dy):
    """Gradient of y = x rstd w (rstd the reciprocal root mean square of x)
    with respect to x, by the quotient rule, and its rows' share of dw."""
    D = x.shape[1]
    t = dy * w
    dot = torch.einsum("rd,rd->r", t, x)
    return t * rstd[:, None] - x * (rstd ** 3 * dot / D)[:, None], torch.einsum("rd,rd,r->d", dy, x, rstd)


def _exact_backward(f, case):
    parts, sums = {}, {}
    for i in range(0, case["rows"], 4096):
        cut = slice(i, i + 4096)
        got, add = {}, {}
        G = f["dr_out"][cut]
        if case["next"]:
            dx, add["dw_next"] = _normed_vjp(f["r_out"][cut], f["rstd_next"][cut], f["w_next"], f["dh"][cut])
            G = G + dx
        got["dr"] = G
        if case["block"]:
            o = f["o"][cut]
            y = o * f["rstd_post"][cut][:, None] * f["w_post"] if case["post"] else o
            u = _sigmoid64(f["gate"][cut]) if case["gate"] else torch.ones_like(o)
            c = f["scale"] if case["scale"] else torch.ones_like(o[0])
            if case["scale"]:
                add["dscale"] = torch.einsum("rd,rd,rd->d", G, u, y)
            if case["gate"]:
                got["dgate"] = torch.einsum("rd,rd,d,rd->rd", G, y, c, u - u * u)
            dy = torch.einsum("rd,rd,d->rd", G, u, c)
            if case["post"]:
                got["do"], add["dw_post"] = _normed_vjp(o, f["rstd_post"][cut], f["w_post"], dy)
            else:
                got["do"] = dy
        for k, v in got.items():
            parts.setdefault(k, []).append(v)
        for k, v in add.items():
            sums[k] = sums[k] + v if k in sums else v
    done = {k: torch.cat(v) for k, v in parts.items()} | sums
    return {k: done.get(k) for k in ("dr", "do", "dgate", "dscale", "dw_post", "dw_next")}


def _exact_w4(f, case):
    K, G = case["K"], case["group"]
    packed, N = f["packed"], f["packed"].shape[0]
    x = f["x"].view(-1, K)
    # Channel k's code, straight from the layout's definition.
    k = torch.arange(K, device="cuda")
    blk, j, c, i = k // 128, (k % 128) // 32, (k % 32) // 8, k % 8
    bit = 4 * (i // 2) + 16 * (i % 2)
    at, shift = blk * 64 + c * 16 + j * 4 + bit // 8, bit % 8
    ys = []
    for n in range(0, N, 2048):
        cut = slice(n, n + 2048)
        code = ((packed[cut][:, at].int() >> shift) & 15).double()
        zero = f["zeros"][cut][:, k // G].double() if case["zeros"] else 8
        ys.append(x @ ((code - zero) * f["scales"][cut][:, k // G]).T)
    y = torch.cat(ys, 1)
    if case["bias"]:
        y = y + f["bias"]
    if case["kind"] == "linear":
        return dict(y=y)
    H_q, H_kv, d, M = case["H_q"], case["H_kv"], case["d"], case["tokens"]
    y = y.view(M, H_q + 2 * H_kv, d)
    at = f["positions"].view(M).long()
    turn = torch.complex(f["cos"][at], f["sin"][at])[:, None]
    z = torch.complex(y[..., :d // 2], y[..., d // 2:])[:, :H_q + H_kv] * turn
    rot = torch.cat((z.real, z.imag), -1)[:, :, None]
    return dict(q=rot[:, :H_q], k=rot[:, H_q:], v=y[:, H_q + H_kv:, None])


def _stored64(x):
    """The values that rows [..., d] take in the cache."""
    w = x.float().unflatten(-1, (-1, 32))
    m = w.min(-1, keepdim=True).values.bfloat16().float()
    step = ((w.max(-1, keepdim=True).values - m).clamp_min(0) * (1 / 15)).bfloat16().float()
    code = torch.where(step > 0, torch.round((w - m) / step).clamp(0, 15), torch.zeros_like(w))
    return (code.double() * step.double() + m.double()).flatten(-2)


def _exact_fill(s, case):
    full = [torch.zeros(case["B"], case["H_kv"], case["S"], case["d"], dtype=torch.float64, device="cuda")
            for _ in range(2)]
    for b, p in enumerate(s["pos"].tolist()):
        full[0][b, :, p:p + case["n"]] = _stored64(s["k"][b])
        full[1][b, :, p:p + case["n"]] = _stored64(s["v"][b])
    return dict(k=full[0], v=full[1])


def _exact_step(s, case):
    B, H, d = case["B"], case["H_kv"], case["d"]
    kc, ks, vc, vs = s["cache"]
    out = s["out"].double()
    ch = torch.arange(d, device="cuda")
    j, o = ch // 32, ch % 32
    kbit = 32 * ((o // 8) * (d // 32) + j) + 4 * (o % 8 // 2) + 16 * (o % 2)
    vbit = 16 * ((o // 4) * (d // 32) + j) + 4 * (o % 4)

    def values(codes, sm, bit):
        code = ((codes[..., bit // 8].int() >> (bit % 8)) & 15).double()
        return code * sm[..., j, 0].double() + sm[..., j, 1].double()

    for b, p in enumerate(s["pos"].tolist()):
        if p < 0:
            continue
        K = torch.cat((values(kc[b, :, :p], ks[b, :, :p], kbit), _stored64(s["k_t"][b])[:, None]), 1)
        V = torch.cat((values(vc[b, :, :p], vs[b, :, :p], vbit), _stored64(s["v_t"][b])[:, None]), 1)
        q = s["q_t"][b].double().view(H, -1, d)
        a = torch.softmax(torch.einsum("hgd,hsd->hgs", q, K) / math.sqrt(d), -1)
        a_dot = torch.einsum("hgs,hsd->hgd", a, V)
        sq = torch.where(q > 0, q + 1, torch.exp(q.clamp_max(0)))
        a_mem = torch.einsum("hgi,hij->hgj", sq, s["M"][b].double()) / \
            torch.einsum("hgi,hi->hg", sq, s["z"][b].double())[..., None]
        g = _sigmoid64(s["beta"].double()).view(H, -1, 1)
        out[b] = (g * a_mem + (1 - g) * a_dot).reshape(-1, d)
    return out
