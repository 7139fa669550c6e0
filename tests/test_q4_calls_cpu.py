"""Argument checks of the calls that take one batch row's part of a 4-bit segment
buffer: addresses that a row's part may have pass, others are refused.  No CUDA call is
reached: the calls that pass the check of alignment are refused for a later one."""

import ctypes

import pytest

from compressive_memory_transformer_segment_b200 import api

MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    return api.load_library()


@pytest.mark.parametrize("d", [32, 64, 128])
def test_alignment_of_a_rows_part(lib, d):
    dims = api.make_dims(1, 2, 2, 3, d, d, 1)
    row = d // 8

    def cache(at, name="k_scale"):
        c = dict(k_codes=1 * MB, k_scale=2 * MB, v_codes=3 * MB, v_scale=4 * MB)
        c[name] += at
        return ctypes.byref(api._CacheQ4Ptrs(*c.values()))

    def append(c, pos=7 * MB, k=5 * MB):
        return lib.infini_attn_cache_q4_append(k, 6 * MB, pos, ctypes.byref(dims), 100, c, None)

    over = 1 * MB  # keys given where the buffer's lie: refused after the alignment
    for name in ("k_scale", "v_scale"):
        assert append(cache(row, name), k=over) == api.ERR_ALIAS
        assert append(cache(row // 2, name), k=over) == api.ERR_ALIGN
        assert lib.infini_attn_cache_q4_read(cache(row, name), ctypes.byref(dims), 100, over, 6 * MB, None) == api.ERR_ALIAS
        assert lib.infini_attn_cache_q4_read(cache(2, name), ctypes.byref(dims), 100, over, 6 * MB, None) == api.ERR_ALIGN
        assert lib.infini_attn_state_update_q4(cache(row, name), over, 6 * MB, 0, ctypes.byref(dims), 100, over + 16,
                                               8 * MB, None, 0, None) == api.ERR_ALIAS
        assert lib.infini_attn_state_update_q4(cache(2, name), over, 6 * MB, 0, ctypes.byref(dims), 100, over + 16,
                                               8 * MB, None, 0, None) == api.ERR_ALIGN
    assert append(cache(8, "k_codes"), k=over) == api.ERR_ALIGN
    assert append(cache(0), pos=7 * MB + 4, k=over) == api.ERR_ALIAS
    assert append(cache(0), pos=7 * MB + 2, k=over) == api.ERR_ALIGN


def test_more_units_of_work_than_32_bits_count_are_refused(lib):
    """A decode step whose 128-row units, one set for every 8 query heads of a KV head,
    pass 2^31 has no workspace and is refused."""
    def need(B, H_q, H_kv, seg):
        return lib.infini_attn_decode_q4_workspace_bytes(ctypes.byref(api.make_dims(B, H_q, H_kv, 1, 32, 32, 1)), seg)

    assert need(1, 65528, 1, 1 << 26) == 0      # 8191 (2^19 + 9) units
    assert need(1, 65528, 1, 1 << 24) > 0
    assert need(1, 65528, 65528, 1 << 20) > 0   # 65528 (2^13 + 9)
    assert need(7, 9362, 9362, 1 << 30) == 0
    assert need(1, 8, 1, 1 << 30) > 0
    d = ctypes.byref(api.make_dims(1, 65528, 1, 1, 32, 32, 1))
    MB = 1 << 20
    cache = ctypes.byref(api._CacheQ4Ptrs(1 << 40, 2 << 40, 3 << 40, 4 << 40))
    assert lib.infini_attn_decode_step_q4(5 * MB, 15 * MB, 16 * MB, 17 * MB, cache, 18 * MB, 19 * MB, 20 * MB, 1 << 26, d,
                                          30 * MB, None, 0, None) == api.ERR_UNSUPPORTED
