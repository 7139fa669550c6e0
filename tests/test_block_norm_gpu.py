"""GPU parity of the norms around the layer (infini_attn_block_norm and its
backward) against the float64 oracle.

Tolerances.  Each result is rounded once to its type (half a step, eps / 2 of
the value).  Before that the kernels work in fp32: fewer than 32 roundings of
2^-24 per element, 2^x and reciprocal approximations good to 2^-21, row means
of D terms added pairwise over lanes (error below 2^-20 of the sum of
magnitudes): together below 2^-18 of the largest term an element's value is
made of.  That term is bounded by the row's largest |r| + |block's share|
(forward) or by the row's largest partial gradient (backward), for which the
oracle's row maxima stand, with 2^-16 to cover sums of two or three of them.
A parameter gradient adds R terms in fp32 in chains of at most R: error below
(R + 64) 2^-24 of the sum of magnitudes, plus 2^-18 of it for the terms' own.
"""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
EPS = 1e-6
ALL = dict(block=True, post=True, gate=True, scale=True, next=True)


def make(rows, width, dtype, f, seed=0):
    g = torch.Generator().manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g)

    dt = DT[dtype]
    x = dict(r=(randn(rows, width) * torch.exp(0.5 * randn(width))).to(dt),
             o=(0.7 * randn(rows, width)).to(dt) if f["block"] else None,
             gate=(1.5 * randn(rows, width)).to(dt) if f["gate"] else None,
             scale=0.1 + torch.rand(width, generator=g) if f["scale"] else None,
             w_post=1 + 0.1 * randn(width) if f["post"] else None,
             w_next=1 + 0.1 * randn(width) if f["next"] else None)
    d = dict(dr_out=randn(rows, width).to(dt), dh=randn(rows, width).to(dt))
    return x, d


def dev(x):
    return {k: v.cuda() if v is not None else None for k, v in x.items()}


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def forward(api, x, **kw):
    return api.block_norm(x["r"], x["w_next"], EPS, o=x["o"], gate=x["gate"], scale=x["scale"],
                          w_post=x["w_post"], **kw)


def backward(api, x, d, r_out, rp, rn, **kw):
    return api.block_norm_backward(d["dr_out"], d["dh"], r_out, rn, x["w_next"], o=x["o"],
                                   gate=x["gate"], scale=x["scale"], w_post=x["w_post"], rstd_post=rp, **kw)


def reference(x):
    return oracle.block_norm(f64(x["r"]), f64(x["w_next"]), EPS, o=f64(x["o"]), gate=f64(x["gate"]),
                             scale=f64(x["scale"]), w_post=f64(x["w_post"]))


def within(got, ref, half, slack):
    got = f64(got)
    assert got.shape == ref.shape
    assert np.all(np.abs(got - ref) <= half * np.abs(ref) + slack), \
        float(np.max(np.abs(got - ref) - half * np.abs(ref) - slack))


def row_max(a):
    return np.max(np.abs(a), axis=-1, keepdims=True)


def check_forward(api, x, dtype):
    r_out, h, rp, rn = forward(api, dev(x))
    ro, rh, rrp, rrn = reference(x)
    if ro is not None:
        top = row_max(f64(x["r"])) + row_max(ro - f64(x["r"]))
        within(r_out, ro, HALF[dtype], 2.0 ** -16 * top)
    else:
        assert r_out is None
        top = row_max(f64(x["r"]))
    if rh is not None:
        within(h, rh, HALF[dtype], 2.0 ** -16 * top * rrn[:, None] * np.max(np.abs(f64(x["w_next"]))))
        within(rn, rrn, 2.0 ** -18, 0.0)
    else:
        assert h is None and rn is None
    if rrp is not None:
        within(rp, rrp, 2.0 ** -18, 0.0)
    else:
        assert rp is None


def check_backward(api, x, d, dtype, ref_dr_out=True):
    xd, dd = dev(x), dev(d)
    if not ref_dr_out:
        dd["dr_out"] = None
    r_out, _, rp, rn = forward(api, xd)
    stream = r_out if x["o"] is not None else xd["r"]
    got = backward(api, xd, dd, stream, rp, rn)
    ref = oracle.block_norm_vjp(f64(d["dr_out"]) if ref_dr_out else None, f64(d["dh"]), f64(stream),
                                f64(rn), f64(x["w_next"]), o=f64(x["o"]), gate=f64(x["gate"]),
                                scale=f64(x["scale"]), w_post=f64(x["w_post"]), rstd_post=f64(rp))
    half, R = HALF[dtype], x["r"].shape[0]
    G = ref["dr"]
    within(got.dr, G, half if x["w_next"] is not None else 0.0, 2.0 ** -16 * row_max(G) + 2.0 ** -16 * 8)
    w_top = max([1.0] + [float(np.max(np.abs(f64(x[k])))) for k in ("scale", "w_post") if x[k] is not None])
    if x["o"] is not None:
        n = f64(x["o"]) * (f64(rp)[:, None] if rp is not None else 1.0)
        # do: a share f of G (at most w_top^2 |G|) minus n times the row's mean
        # of f n (at most max |f| max |n|), times rstd_post.
        f_top = w_top ** 2 * row_max(G)
        scale = f64(rp)[:, None] if rp is not None else 1.0
        within(got.do, ref["do"], half, 2.0 ** -16 * scale * f_top * (1 + row_max(n) ** 2))
        if x["gate"] is not None:
            within(got.dgate, ref["dgate"], half, 2.0 ** -16 * f_top * row_max(n))
        mags = np.sum(np.abs(G) * np.abs(n), axis=0) * w_top ** 2
        for name in ("dscale", "dw_post"):
            if name in ref:
                within(getattr(got, name), ref[name], 0.0, ((R + 64) * 2.0 ** -24 + 2.0 ** -16) * mags)
    if x["w_next"] is not None:
        mags = np.sum(np.abs(f64(d["dh"])) * np.abs(f64(stream)) * f64(rn)[:, None], axis=0)
        within(got.dw_next, ref["dw_next"], 0.0, ((R + 64) * 2.0 ** -24 + 2.0 ** -18) * mags)
    for name in ("do", "dgate", "dscale", "dw_post", "dw_next"):
        assert (getattr(got, name) is None) == (name not in ref)


# One row to many; one channel, odd widths (element-wise path), widths of one
# to several vectors per thread, the widest.
SIZES = [(1, 1), (1, 8), (3, 33), (5, 64), (70, 768), (17, 1019), (300, 1024), (9, 4096), (4, 4104),
         (6, 5001), (3, 8192), (2, 16384), (2, 16383)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,width", SIZES)
def test_sizes(cuda_lib, rows, width, dtype):
    x, d = make(rows, width, dtype, ALL, seed=rows * 20000 + width)
    check_forward(cuda_lib, x, dtype)
    check_backward(cuda_lib, x, d, dtype)


FLAGS = [dict(block=b, post=p, gate=g, scale=s, next=n)
         for b in (False, True) for p in (False, True) for g in (False, True) for s in (False, True)
         for n in (False, True) if (b or not (p or g or s)) and (b or n)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("f", FLAGS, ids=lambda f: "-".join(k for k, v in f.items() if v))
def test_parts(cuda_lib, f, dtype):
    """Every combination of the optional parts."""
    for width in (96, 101):
        x, d = make(11, width, dtype, f, seed=3)
        check_forward(cuda_lib, x, dtype)
        check_backward(cuda_lib, x, d, dtype)
        if f["next"]:
            check_backward(cuda_lib, x, d, dtype, ref_dr_out=False)


def test_many_rows_per_block(cuda_lib):
    """More rows than resident blocks, so that blocks walk over rows and add
    their shares of the parameter gradients."""
    x, d = make(5003, 264, "bf16", ALL, seed=9)
    check_backward(cuda_lib, x, d, "bf16")
    x, d = make(1501, 1001, "f32", ALL, seed=10)
    check_backward(cuda_lib, x, d, "f32")


def test_rows_are_independent_and_extremes(cuda_lib):
    """A NaN row leaves the others as they were; gate logits of +-infinity are
    gates of 1 and 0; an all-zero row is finite."""
    x, _ = make(6, 256, "f32", ALL, seed=4)
    clean = forward(cuda_lib, dev(x))
    x["o"][2] = float("nan")
    x["r"][4] = 0.0
    x["o"][4] = 0.0
    x["gate"][1, :128], x["gate"][1, 128:] = float("inf"), -float("inf")
    got = forward(cuda_lib, dev(x))
    for a, b in zip(clean, got):
        for row in (0, 3, 5):
            assert torch.equal(a[row], b[row])
    assert torch.isnan(got[1][2]).all()
    assert torch.count_nonzero(got[0][4]) == 0 and torch.count_nonzero(got[1][4]) == 0
    y = (x["o"][1] * got[2][1].cpu() * x["w_post"] * x["scale"])[:128]
    assert torch.allclose(got[0][1, :128].cpu(), x["r"][1, :128] + y, rtol=1e-5, atol=1e-5)
    assert torch.equal(got[0][1, 128:].cpu(), x["r"][1, 128:])
    d = dict(dr_out=torch.ones(6, 256), dh=torch.ones(6, 256))
    g = backward(cuda_lib, dev(x), dev(d), got[0], got[2], got[3])
    assert torch.count_nonzero(g.dgate[1]) == 0 and torch.isfinite(g.do[1]).all()


def test_in_place_stream_and_gradient(cuda_lib):
    x, d = make(7, 512, "bf16", ALL, seed=5)
    xd, dd = dev(x), dev(d)
    r_out, h, rp, rn = forward(cuda_lib, xd)
    own = dict(xd, r=xd["r"].clone())
    r2, h2, _, _ = forward(cuda_lib, own, r_out=own["r"])
    assert r2 is own["r"] and torch.equal(r2, r_out) and torch.equal(h2, h)


def test_repeats_are_bitwise_equal_and_workspace_contents_do_not_matter(cuda_lib):
    x, d = make(900, 768, "bf16", ALL, seed=6)
    xd, dd = dev(x), dev(d)
    r_out, _, rp, rn = forward(cuda_lib, xd)
    a = backward(cuda_lib, xd, dd, r_out, rp, rn)
    n = cuda_lib.block_norm_backward_workspace_bytes(900, 768)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    b = backward(cuda_lib, xd, dd, r_out, rp, rn, workspace=ws)
    c = backward(cuda_lib, xd, dd, r_out, rp, rn, workspace=ws)
    for u, v, w in zip(a, b, c):
        assert torch.equal(u, v) and torch.equal(v, w)


def test_other_stream_and_captured_graph(cuda_lib):
    x, d = make(40, 1024, "bf16", ALL, seed=7)
    xd, dd = dev(x), dev(d)
    ref = forward(cuda_lib, xd)
    ref_g = backward(cuda_lib, xd, dd, ref[0], ref[2], ref[3])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = forward(cuda_lib, xd, stream=s)
    got_g = backward(cuda_lib, xd, dd, got[0], got[2], got[3], stream=s)
    s.synchronize()
    for a, b in zip(tuple(ref) + tuple(ref_g), tuple(got) + tuple(got_g)):
        assert torch.equal(a, b)
    ws = torch.empty(cuda_lib.block_norm_backward_workspace_bytes(40, 1024), dtype=torch.uint8,
                     device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = forward(cuda_lib, xd)
        out_g = backward(cuda_lib, xd, dd, out[0], out[2], out[3], workspace=ws)
    xd["o"].mul_(2)
    graph.replay()
    want = forward(cuda_lib, xd)
    want_g = backward(cuda_lib, xd, dd, want[0], want[2], want[3])
    torch.cuda.synchronize()
    for a, b in zip(tuple(out) + tuple(out_g), tuple(want) + tuple(want_g)):
        assert torch.equal(a, b)


def test_binding_refuses(cuda_lib):
    x, _ = make(4, 64, "f32", ALL)
    xd = dev(x)
    with pytest.raises(ValueError):
        forward(cuda_lib, dict(xd, o=xd["o"].bfloat16()))
    with pytest.raises(ValueError):
        forward(cuda_lib, dict(xd, w_next=xd["w_next"][:32]))
    with pytest.raises(ValueError):
        forward(cuda_lib, dict(xd, r=xd["r"].t().contiguous().t()))
    with pytest.raises(ValueError):
        forward(cuda_lib, dict(xd, gate=xd["gate"].cpu()))
    with pytest.raises(cuda_lib.InfiniError):
        forward(cuda_lib, dict(xd, o=None))
    with pytest.raises(cuda_lib.InfiniError):
        cuda_lib.block_norm(xd["r"], xd["w_next"], 0.0)


def test_offsets_beyond_32_bits(cuda_lib):
    """131075 rows of 16384: elements past 2^31.  The last rows' results, forward
    and backward, are those of the rows alone (rows do not affect one another)."""
    api, rows, width, n = cuda_lib, (1 << 17) + 3, 16384, 5
    x, d = make(n, width, "bf16", dict(ALL, gate=False))
    big = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")

    def placed(t):
        out = torch.zeros_like(big)
        out[-n:] = t.cuda()
        return out

    small = dev(x)
    r_out, h, rp, rn = forward(api, small)
    large = dict(small, r=placed(x["r"]), o=placed(x["o"]))
    got = forward(api, large)
    api.sync_status()
    for a, b in zip(got, (r_out, h, rp, rn)):
        assert torch.equal(a[-n:], b)
    assert not got[0][:-n].any() and not got[1][:-n].any()
    grads = backward(api, small, dev(d), r_out, rp, rn)
    all_grads = backward(api, large, dict(dr_out=placed(d["dr_out"]), dh=placed(d["dh"])), got[0], got[2], got[3])
    api.sync_status()
    for a, b in ((all_grads.dr, grads.dr), (all_grads.do, grads.do)):
        assert torch.equal(a[-n:], b) and not a[:-n].any()
    # Sums of 5 rows among zeros, in another order: 8 roundings of 2^-24 of the largest terms.
    for a, b in ((all_grads.dscale, grads.dscale), (all_grads.dw_post, grads.dw_post),
                 (all_grads.dw_next, grads.dw_next)):
        assert float((a - b).abs().max()) <= 8 * 2.0 ** -24 * 5 * float(b.abs().max())
