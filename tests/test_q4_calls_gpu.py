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


@pytest.mark.parametrize("d,S,H", [(32, 17, 1), (32, 9, 2), (64, 7, 3), (128, 5, 1)])
def test_a_batch_row_of_any_size_alone(cuda_lib, d, S, H):
    """Every stream's part of the arrays appends, reads and updates its memory, wherever
    the rows' scales begin (multiples of d / 8 bytes), with its element of pos."""
    api, B = cuda_lib, 5
    whole, parts = api.CacheQ4.empty(B, H, S, d), api.CacheQ4.empty(B, H, S, d)
    k, v = randn(B, H, S - 2, d, seed=1), randn(B, H, S - 2, d, seed=2)
    pos = torch.tensor([0, 2, -1, 1, 0], dtype=torch.int32, device="cuda")
    whole.append(k, v, pos)
    for b in range(B):
        parts.row(b).append(k[b:b + 1], v[b:b + 1], pos[b:b + 1])
    for a, b in zip(whole.tensors, parts.tensors):
        assert torch.equal(a, b)
    rk, rv = whole.read(S)
    M, z = randn(B, H, d, d, seed=3), 5 + randn(B, H, d, seed=4).abs()
    M2, z2 = whole.state_update(S, M, z, "delta", torch.float32)
    for b in range(B):
        k1, v1 = whole.row(b).read(S)
        assert torch.equal(k1, rk[b:b + 1]) and torch.equal(v1, rv[b:b + 1])
        M1, z1 = whole.row(b).state_update(S, M[b:b + 1].clone(), z[b:b + 1].clone(), "delta", torch.float32)
        assert torch.equal(M1, M2[b:b + 1]) and torch.equal(z1, z2[b:b + 1])
    api.sync_status()
