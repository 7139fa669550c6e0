"""GPU: the block's norms called from two host threads, at extreme gates and with
infinite outputs of the block."""

import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def randn(*shape, seed=0, dtype="f32"):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DT[dtype]).cuda()


def test_host_threads_with_different_widths(cuda_lib):
    """Two widths of one kernel instance ask for different shared memory; neither
    thread's calls may be refused for the other's.  (The library's own entry point, so
    that the threads spend their time in it and not under the interpreter's lock.)"""
    lib = cuda_lib.load_library()
    keep, work = [], []
    for width in (4096, 2048, 4096, 2048):
        vec = [randn(width, seed=i, dtype="bf16") for i in range(5)]
        w, h = randn(width, seed=9), torch.empty(width, dtype=torch.bfloat16, device="cuda")
        stream = torch.cuda.Stream()
        keep.append((vec, w, h, stream))
        r, o, gate, r_out, _ = (t.data_ptr() for t in vec)
        # r, o, gate, scale, w_post, w_next, eps, rows, width, bf16, r_out, h, rstd_post, rstd_next, stream
        work.append((r, o, gate, w.data_ptr(), w.data_ptr(), w.data_ptr(), 1e-6, 1, width, cuda_lib.DTYPES[torch.bfloat16],
                     r_out, h.data_ptr(), None, None, stream.cuda_stream))
    torch.cuda.synchronize()
    refused = []

    def calls(args):
        fn = lib.infini_attn_block_norm
        refused.append(sum(fn(*args) != 0 for _ in range(50000)))

    threads = [threading.Thread(target=calls, args=(a,)) for a in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert refused == [0] * len(work)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("next_norm", [False, True])
def test_gradient_of_an_infinite_output_without_its_norm(cuda_lib, next_norm, dtype):
    """Without w_post, do = G scale sg(gate) does not depend on o: it is finite where o
    is infinite or NaN.  Against the call with a finite o: the same bits."""
    rows, width = 5, 264
    o = randn(rows, width, seed=1, dtype=dtype)
    lost = o.clone()
    lost[0, 3], lost[1, 200], lost[4, 263] = float("inf"), float("nan"), -float("inf")
    args = (randn(rows, width, seed=2, dtype=dtype), randn(rows, width, seed=3, dtype=dtype) if next_norm else None,
            randn(rows, width, seed=4, dtype=dtype) if next_norm else None,
            randn(rows, seed=5).abs() + 1 if next_norm else None, randn(width, seed=6) if next_norm else None)
    more = dict(gate=randn(rows, width, seed=7, dtype=dtype), scale=randn(width, seed=8))
    want = cuda_lib.block_norm_backward(*args, o=o, **more)
    got = cuda_lib.block_norm_backward(*args, o=lost, **more)
    assert torch.isfinite(want.do).all() and torch.equal(got.do, want.do) and torch.equal(got.dr, want.dr)
    here = ~torch.isfinite(lost)
    assert not torch.isfinite(got.dgate[here]).any() and torch.equal(got.dgate[~here], want.dgate[~here])
    plain = (~here).all(0)
    assert not torch.isfinite(got.dscale[~plain]).any() and torch.equal(got.dscale[plain], want.dscale[plain])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gates_of_every_size(cuda_lib, dtype):
    """Logits over -87 .. 87, where neither the logistic u nor u (1 - u) is subnormal.
    2^x is right to 2^-22, its argument's remainder adds two roundings, 2^-23, so t =
    e^-a to 1.5 2^-22; 1 + t and 1 / x: u to 2.25 2^-22; 1 - u = t u to 4 2^-22; three
    products: u (1 - u) to 7 2^-22.  bf16 rows leave the remainder out: |a| 2^-24 more of t, 2^-17.5 at
    87, once in u and twice in 1 - u; and half a step of the type."""
    left = 0.0 if dtype == "f32" else 2.0 ** -17.5
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for width in (4096, 1019):  # pieces of 16 bytes, and single elements
        a = torch.linspace(-87, 87, 3 * width, dtype=torch.float64).to(DT[dtype]).view(3, width).cuda()
        one, zero = torch.ones_like(a), torch.zeros_like(a)
        e = torch.exp(-a.double().abs())
        u, du = torch.where(a > 0, 1 / (1 + e), e / (1 + e)), e / (1 + e) ** 2
        r_out = cuda_lib.block_norm(zero, None, 1e-6, o=one, gate=a)[0]
        g = cuda_lib.block_norm_backward(one, None, None, None, None, o=one, gate=a)
        for got, want, bound in ((r_out, u, 2.25 * 2.0 ** -22 + left), (g.do, u, 2.25 * 2.0 ** -22 + left),
                                 (g.dgate, du, 7 * 2.0 ** -22 + 3 * left)):
            off = ((got.double() - want).abs() / want).max()
            assert off <= (bound + half) * (1 + 2.0 ** -7), (float(off), bound)
    # the limits
    a = torch.tensor([[float("inf"), -float("inf"), float("nan"), 300.0, -300.0, 3e38, -3e38, 0.0]], dtype=DT[dtype]).cuda()
    one, zero = torch.ones_like(a), torch.zeros_like(a)
    r_out = cuda_lib.block_norm(zero, None, 1e-6, o=one, gate=a)[0]
    g = cuda_lib.block_norm_backward(one, None, None, None, None, o=one, gate=a)
    nan = float("nan")
    for got, want in ((r_out, [1, 0, nan, 1, 0, 1, 0, 0.5]), (g.do, [1, 0, nan, 1, 0, 1, 0, 0.5]),
                      (g.dgate, [0, 0, nan, 0, 0, 0, 0, 0.25])):
        want = torch.tensor([want], dtype=DT[dtype]).cuda()
        assert torch.allclose(got, want, rtol=2.0 ** -7, atol=0, equal_nan=True), (got, want)
