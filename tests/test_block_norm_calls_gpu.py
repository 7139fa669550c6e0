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
