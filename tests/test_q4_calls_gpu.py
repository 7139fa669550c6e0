"""GPU: calls on the 4-bit segment buffer that share a workspace, or take a part of
a batch's arrays."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda()


def step_args(api, B, H_q, H_kv, d, S, pos, seed=0):
    cache = api.CacheQ4.empty(B, H_kv, S, d)
    cache.append(randn(B, H_kv, S, d, seed=seed), randn(B, H_kv, S, d, seed=seed + 1),
                 torch.zeros(B, dtype=torch.int32, device="cuda"))
    return (randn(B, H_q, d, seed=seed + 2), randn(B, H_kv, d, seed=seed + 3), randn(B, H_kv, d, seed=seed + 4),
            randn(H_q, seed=seed + 5), cache, torch.tensor(pos, dtype=torch.int32, device="cuda"),
            randn(B, H_kv, d, d, seed=seed + 6), 5 + randn(B, H_kv, d, seed=seed + 7).abs())


def test_one_workspace_for_batches_of_every_size(cuda_lib):
    """A workspace that was zeroed once serves other shapes in turn: what one leaves
    in it is no ticket of another.  (Segments whole in one block, and cut by several.)"""
    api, d, S = cuda_lib, 64, 2000
    shapes = [(1, 4, 2, d, S, [50]), (70, 4, 2, d, S, [(271 * b) % S for b in range(70)]),
              (2, 4, 2, d, S, [1999, 60]), (3, 16, 1, d, 40, [0, 39, -1]), (70, 4, 2, d, S, [S - 1 - b for b in range(70)])]
    ws = torch.zeros(max(api.decode_q4_workspace_bytes(B, H_q, H_kv, S, d) for B, H_q, H_kv, d, S, _ in shapes),
                     dtype=torch.uint8, device="cuda")
    for B, H_q, H_kv, d, S, pos in shapes:
        args = step_args(api, B, H_q, H_kv, d, S, pos, seed=B)
        want, got = (torch.full((B, H_q, d), 7.0, device="cuda") for _ in range(2))
        api.decode_step_q4(*args, out=want)
        for _ in range(2):
            api.decode_step_q4(*args, out=got.fill_(7.0), workspace=ws)
            assert torch.equal(got, want)
    api.sync_status()
