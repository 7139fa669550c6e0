"""The C-ABI library on a machine without a GPU: it loads, exports every
symbol include/infini_attn.h declares, and rejects bad arguments on the host
before any CUDA call (no compute is launched here)."""

import ctypes
import os
import re

import pytest

from compressive_memory_transformer_segment_b200 import api, configs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def header_symbols():
    names = set()
    for fn in os.listdir(os.path.join(ROOT, "include")):
        if fn.endswith(".h"):
            text = open(os.path.join(ROOT, "include", fn)).read()
            names |= set(re.findall(r"INFINI_API\s+[\w\s\*]*?\b(infini_attn_\w+)\s*\(", text))
    return names


@pytest.fixture(scope="module")
def lib():
    return api.load_library()


def test_library_exports_every_declared_symbol(lib):
    declared = header_symbols()
    assert {"infini_attn_init_state", "infini_attn_forward"} <= declared
    for name in declared:
        assert hasattr(lib, name), name
    assert declared == set(api.exported_symbols())
    assert lib.infini_attn_version() >> 16 == 1


def test_status_strings(lib):
    for code in (0, -1, -2, -3, -4, -5, -6, -7, 12345):
        assert api.status_string(code)


def dims_of(w):
    return api.make_dims(w.B, w.H_q, w.H_kv, w.L, w.d_k, w.d_v, 0 if w.dtype == "bf16" else 1)


@pytest.mark.parametrize("name", sorted(configs.WORKLOADS))
def test_plan_and_workspace_for_every_workload(name):
    w = configs.WORKLOADS[name]
    d = dims_of(w)
    p = api.plan(d, w.seg_len, w.rule)
    assert p["num_segments"] == w.T
    assert p["workspace_bytes"] == api.workspace_bytes(d, w.seg_len, w.rule) > 0
    # The workspace holds at least the z read by every segment.
    assert p["workspace_bytes"] >= w.T * w.B * w.H_kv * w.d_k * 4
    assert api.host_arena_bytes(d, w.seg_len, w.rule) > p["workspace_bytes"]


@pytest.mark.parametrize("bad", [
    dict(B=0), dict(H_q=3, H_kv=2), dict(L=0), dict(d_k=48), dict(d_v=256), dict(dtype=7),
])
def test_plan_rejects_bad_sizes(bad):
    base = dict(B=1, H_q=4, H_kv=2, L=128, d_k=64, d_v=64, dtype=0)
    base.update(bad)
    d = api.Dims(**base)
    with pytest.raises(api.InfiniError) as e:
        api.plan(d, 64, "linear")
    assert e.value.status in (api.ERR_ARG, api.ERR_UNSUPPORTED)
    assert api.workspace_bytes(d, 64, "linear") == 0


def test_plan_rejects_bad_rule_and_segment():
    d = api.Dims(1, 2, 2, 64, 32, 32, 1)
    for seg, rule in ((0, 0), (-3, 1), (16, 2)):
        with pytest.raises(api.InfiniError):
            api.plan(d, seg, rule)


def _fwd(lib, ptrs, dims, seg=64, rule=0, ws=0, ws_n=0):
    P = ctypes.c_void_p
    q, k, v, beta, M, z, out, Mo, zo = (P(x) for x in ptrs)
    return lib.infini_attn_forward(q, k, v, beta, M, z, seg, rule, ctypes.byref(dims), out, Mo, zo,
                                   P(ws), ws_n, P(0))


def test_forward_validates_on_host_before_any_cuda_call(lib):
    """Fake, never-dereferenced addresses: every case below must be rejected
    by the host checks, so no CUDA call happens (this machine has no GPU)."""
    d = api.Dims(1, 2, 2, 128, 32, 32, 1)  # f32: q = k = v = out = 32 KiB
    MB = 1 << 20
    good = [1 * MB, 2 * MB, 3 * MB, 4 * MB, 5 * MB, 6 * MB, 7 * MB, 8 * MB, 9 * MB]
    bad = list(good)
    bad[0] = 0
    assert _fwd(lib, bad, d) == api.ERR_ARG
    bad = list(good)
    bad[2] += 4
    assert _fwd(lib, bad, d) == api.ERR_ALIGN
    bad = list(good)
    bad[6] = good[0] + 1024  # out inside q
    assert _fwd(lib, bad, d) == api.ERR_ALIAS
    bad = list(good)
    bad[7] = good[6]  # M_out == out
    assert _fwd(lib, bad, d) == api.ERR_ALIAS
    bad = list(good)
    bad[8] = good[4] + 16  # z_out overlaps M_in (not the permitted in-place pair)
    assert _fwd(lib, bad, d) == api.ERR_ALIAS
    assert _fwd(lib, good, d, ws=10 * MB, ws_n=16) == api.ERR_WORKSPACE
    assert _fwd(lib, good, d, ws=10 * MB + 16, ws_n=1 << 30) == api.ERR_WORKSPACE
    assert _fwd(lib, good, d, ws=0, ws_n=64) == api.ERR_ARG
    assert _fwd(lib, good, d, ws=good[0], ws_n=1 << 20) == api.ERR_ALIAS
    d_bad = api.Dims(1, 2, 2, 128, 40, 32, 1)
    assert _fwd(lib, good, d_bad) == api.ERR_UNSUPPORTED


def test_state_update_validates_on_host_before_any_cuda_call(lib):
    P = ctypes.c_void_p
    d = api.Dims(1, 2, 2, 128, 32, 32, 1)
    MB = 1 << 20
    k, v, M, z, Mo, zo = 1 * MB, 2 * MB, 3 * MB, 4 * MB, 5 * MB, 6 * MB

    def call(k=k, v=v, M=M, z=z, Mo=Mo, zo=zo, seg=64, rule=0, ws=0, ws_n=0, dims=d):
        return lib.infini_attn_state_update(P(k), P(v), P(M), P(z), seg, rule, ctypes.byref(dims),
                                            P(Mo), P(zo), P(ws), ws_n, P(0))

    assert call(k=0) == api.ERR_ARG
    assert call(v=v + 8) == api.ERR_ALIGN
    assert call(Mo=k + 1024) == api.ERR_ALIAS      # M_out inside k
    assert call(zo=M + 16) == api.ERR_ALIAS        # z_out overlaps M_in
    assert call(rule=7) == api.ERR_ARG
    assert call(seg=0) == api.ERR_ARG
    assert call(ws=10 * MB, ws_n=16) == api.ERR_WORKSPACE
    assert call(dims=api.Dims(1, 2, 2, 128, 40, 32, 1)) == api.ERR_UNSUPPORTED


def test_decode_step_validates_on_host_before_any_cuda_call(lib):
    P = ctypes.c_void_p
    d = api.Dims(1, 4, 2, 1, 32, 32, 1)
    MB = 1 << 20
    good = dict(q=1 * MB, k=2 * MB, v=3 * MB, beta=4 * MB, kb=5 * MB, vb=6 * MB, M=7 * MB, z=8 * MB,
                out=9 * MB)

    def call(pos=0, seg=16, rule=0, ws=0, ws_n=0, dims=d, **over):
        a = dict(good, **over)
        return lib.infini_attn_decode_step(P(a["q"]), P(a["k"]), P(a["v"]), P(a["beta"]), P(a["kb"]),
                                           P(a["vb"]), pos, P(a["M"]), P(a["z"]), seg, rule,
                                           ctypes.byref(dims), P(a["out"]), P(ws), ws_n, P(0))

    assert lib.infini_attn_decode_workspace_bytes(ctypes.byref(d), 16, 0) > 0
    assert lib.infini_attn_decode_workspace_bytes(ctypes.byref(api.Dims(1, 4, 2, 1, 32, 64, 1)),
                                                  16, 0) == 0
    assert call(pos=16) == api.ERR_ARG            # pos must be < seg_len
    assert call(pos=-1) == api.ERR_ARG
    assert call(q=0) == api.ERR_ARG
    assert call(k=good["k"] + 4) == api.ERR_ALIGN
    assert call(out=good["q"]) == api.ERR_ALIAS    # out over q_t
    assert call(kb=good["vb"] + 64) == api.ERR_ALIAS
    assert call(M=good["kb"] + 256) == api.ERR_ALIAS
    assert call(ws=10 * MB, ws_n=16) == api.ERR_WORKSPACE
    assert call(ws=good["M"], ws_n=1 << 22) == api.ERR_ALIAS
    assert call(dims=api.Dims(1, 4, 2, 1, 32, 64, 1)) == api.ERR_UNSUPPORTED


def test_binding_fails_loudly_without_library(monkeypatch, tmp_path):
    monkeypatch.setattr(api, "_lib", None)
    with pytest.raises(FileNotFoundError):
        api.load_library(str(tmp_path / "missing.so"))


def test_state_sum_rejects_bad_arguments_on_the_host(lib):
    """Argument checks of infini_attn_state_sum return before any CUDA call."""
    P = ctypes.c_void_p
    MB = 1 << 20
    n_M, n_z = 2 * 3 * 8 * 8 * 4, 2 * 3 * 8 * 4
    base = (P(MB), P(2 * MB))
    assert lib.infini_attn_state_sum(P(0), P(2 * MB), P(0), 0, 2, 3, 8, 8, P(3 * MB), P(4 * MB),
                                     P(0)) == api.ERR_ARG
    assert lib.infini_attn_state_sum(*base, P(0), 2, 2, 3, 8, 8, P(3 * MB), P(4 * MB),
                                     P(0)) == api.ERR_ARG  # parts NULL with n_parts > 0
    assert lib.infini_attn_state_sum(*base, P(0), -1, 2, 3, 8, 8, P(3 * MB), P(4 * MB),
                                     P(0)) == api.ERR_ARG
    assert lib.infini_attn_state_sum(*base, P(0), 0, 0, 3, 8, 8, P(3 * MB), P(4 * MB),
                                     P(0)) == api.ERR_ARG
    assert lib.infini_attn_state_sum(*base, P(0), 0, 2, 3, 8, 8, P(3 * MB + 4), P(4 * MB),
                                     P(0)) == api.ERR_ALIGN
    # M_out overlapping z_out, or the parts, or another state's base
    assert lib.infini_attn_state_sum(*base, P(0), 0, 2, 3, 8, 8, P(3 * MB), P(3 * MB + n_M - 16),
                                     P(0)) == api.ERR_ALIAS
    assert lib.infini_attn_state_sum(*base, P(5 * MB), 1, 2, 3, 8, 8, P(5 * MB + 64), P(4 * MB),
                                     P(0)) == api.ERR_ALIAS
    assert lib.infini_attn_state_sum(*base, P(0), 0, 2, 3, 8, 8, P(MB + 16), P(4 * MB),
                                     P(0)) == api.ERR_ALIAS
    assert n_z < n_M


def test_backward_workspace_and_host_checks(lib):
    """The backward's sizing and argument checks run on the host: supported
    shapes (seg_len <= 64, d_k = d_v in {32, 64}) get a workspace that holds
    at least the fp32 states of every segment; others get 0, and the call
    returns INFINI_ERR_UNSUPPORTED (or INFINI_ERR_ARG for NULL pointers)
    before touching a GPU."""
    w = configs.WORKLOADS["200m-delta"]
    d = dims_of(w)
    nbytes = api.backward_workspace_bytes(d, w.seg_len, w.rule)
    assert nbytes >= w.T * w.B * w.H_kv * w.d_k * w.d_k * 4
    for over in (dict(d_k=128, d_v=128), dict(d_k=64, d_v=32)):
        dd = dims_of(w.with_(**over))
        assert api.backward_workspace_bytes(dd, w.seg_len, w.rule) == 0
    assert api.backward_workspace_bytes(d, 65, w.rule) == 0
    null = ctypes.c_void_p(0)
    args = [null] * 6 + [w.seg_len, 1, ctypes.byref(d)] + [null] * 9 + [null, 0, null]
    assert lib.infini_attn_backward(*args) == -1  # INFINI_ERR_ARG
    args[6] = 128
    assert lib.infini_attn_backward(*args) == -2  # INFINI_ERR_UNSUPPORTED


def test_qkv_project_and_rope_tables_check_arguments_on_the_host(lib):
    """The projection prologue's and the rotary tables' argument checks
    return before any CUDA call."""
    P = ctypes.c_void_p
    MB = 1 << 20
    d = api.make_dims(2, 4, 2, 256, 64, 64, 0)
    x, w, bias, cs, sn = P(1 * MB), P(8 * MB), P(12 * MB), P(13 * MB), P(14 * MB)
    q, k, v = P(20 * MB), P(24 * MB), P(28 * MB)

    def call(*a, dims=d, dm=256):
        a = list(a) if a else [x, w, bias, cs, sn]
        return lib.infini_attn_qkv_project(*a, ctypes.byref(dims), dm, q, k, v, P(0))

    assert call(P(0), w, bias, cs, sn) == api.ERR_ARG
    assert call(x, w, bias, cs, P(0)) == api.ERR_ARG         # one table without the other
    assert call(dm=0) == api.ERR_ARG
    assert call(dims=api.make_dims(2, 4, 2, 256, 128, 64, 0)) == api.ERR_UNSUPPORTED
    assert call(dims=api.make_dims(2, 4, 2, 256, 32, 32, 0)) == api.ERR_UNSUPPORTED
    assert call(dims=api.make_dims(2, 4, 2, 256, 64, 64, 1)) == api.ERR_UNSUPPORTED  # f32
    assert call(dm=60) == api.ERR_UNSUPPORTED
    assert call(dm=260) == api.ERR_UNSUPPORTED
    assert call(P(1 * MB + 8), w, bias, cs, sn) == api.ERR_ALIGN
    # q [2, 4, 256, 64] bf16 = 256 KB from 20 MB: an input there overlaps it.
    assert call(x, w, bias, P(20 * MB + 4096), sn) == api.ERR_ALIAS
    assert lib.infini_attn_qkv_project(x, w, bias, cs, sn, ctypes.byref(d), 256, q, P(20 * MB + 64),
                                       v, P(0)) == api.ERR_ALIAS
    assert lib.infini_attn_rope_tables(P(0), P(MB), 16, 64, 10000.0, P(0)) == api.ERR_ARG
    assert lib.infini_attn_rope_tables(P(MB), P(2 * MB), 0, 64, 10000.0, P(0)) == api.ERR_ARG
    assert lib.infini_attn_rope_tables(P(MB), P(2 * MB), 16, 63, 10000.0, P(0)) == api.ERR_ARG
    assert lib.infini_attn_rope_tables(P(MB), P(2 * MB), 16, 64, 0.0, P(0)) == api.ERR_ARG
    assert lib.infini_attn_rope_tables(P(MB), P(MB + 256), 16, 64, 1e4, P(0)) == api.ERR_ALIAS


def test_block_norm_checks_arguments_on_the_host(lib):
    """Argument checks of the norms around the layer return before any CUDA
    call (addresses are never dereferenced)."""
    MB = 1 << 20
    good = dict(r=1 * MB, o=2 * MB, gate=3 * MB, scale=4 * MB, w_post=5 * MB, w_next=6 * MB, eps=1e-6,
                rows=64, width=256, dtype=0, r_out=7 * MB, h=8 * MB, rp=9 * MB, rn=10 * MB)

    def call(**over):
        return lib.infini_attn_block_norm(*dict(good, **over).values(), None)

    assert call(r=None) == api.ERR_ARG
    assert call(rows=0) == api.ERR_ARG
    assert call(width=0) == api.ERR_ARG
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert call(eps=eps) == api.ERR_ARG
    assert call(dtype=2) == api.ERR_ARG
    assert call(o=None) == api.ERR_ARG                       # gate, scale, w_post belong to o
    assert call(r_out=None) == api.ERR_ARG
    assert call(w_next=None) == api.ERR_ARG                  # h without its weight
    assert call(w_next=None, h=None) == api.ERR_ARG          # rstd_next without its weight
    assert call(w_post=None) == api.ERR_ARG                  # rstd_post without its weight
    assert call(o=None, gate=None, scale=None, w_post=None, r_out=None, rp=None, w_next=None, h=None,
                rn=None) == api.ERR_ARG                      # nothing to do
    assert call(width=16385) == api.ERR_UNSUPPORTED
    assert call(rows=1 << 59) == api.ERR_ARG
    assert call(h=8 * MB + 8) == api.ERR_ALIGN
    assert call(h=good["o"] + 1024) == api.ERR_ALIAS
    assert call(r_out=good["r"] + 512) == api.ERR_ALIAS      # in place means the same pointer
    assert call(rn=good["rp"] + 16) == api.ERR_ALIAS

    assert lib.infini_attn_block_norm_backward_workspace_bytes(0, 256) == 0
    assert lib.infini_attn_block_norm_backward_workspace_bytes(64, 16385) == 0
    n = lib.infini_attn_block_norm_backward_workspace_bytes(64, 256)
    assert n >= 64 * 2 * 256 * 4
    # never more than the resident blocks' shares
    assert lib.infini_attn_block_norm_backward_workspace_bytes(1 << 30, 4096) <= 1 << 28
    bwd = dict(dr_out=1 * MB, dh=2 * MB, r_out=3 * MB, o=4 * MB, gate=5 * MB, scale=6 * MB, w_post=7 * MB,
               w_next=8 * MB, rp=9 * MB, rn=10 * MB, rows=64, width=256, dtype=0, dr=11 * MB, d_o=12 * MB,
               dgate=13 * MB, dscale=14 * MB, dw_post=15 * MB, dw_next=16 * MB, ws=32 * MB, ws_n=n)

    def back(**over):
        return lib.infini_attn_block_norm_backward(*dict(bwd, **over).values(), None)

    for name in ("dh", "r_out", "rn", "dr", "dw_next", "rp", "d_o", "dgate", "dscale", "dw_post"):
        assert back(**{name: None}) == api.ERR_ARG, name
    assert back(o=None) == api.ERR_ARG
    assert back(dr_out=None, w_next=None, dh=None, r_out=None, rn=None, dr=None, dw_next=None) == api.ERR_ARG
    assert back(width=16385) == api.ERR_UNSUPPORTED
    assert back(dgate=13 * MB + 4) == api.ERR_ALIGN
    assert back(ws_n=n - 1) == api.ERR_WORKSPACE
    assert back(ws=32 * MB + 16) == api.ERR_WORKSPACE
    assert back(ws=None) == api.ERR_ARG
    assert back(d_o=bwd["dgate"] + 64) == api.ERR_ALIAS
    assert back(dr=bwd["dr_out"] + 64) == api.ERR_ALIAS
    assert back(ws=bwd["dr"]) == api.ERR_ALIAS


def test_w4_checks_arguments_on_the_host(lib):
    """Argument checks of the 4-bit projections return before any CUDA call."""
    MB = 1 << 20
    good = dict(x=1 * MB, packed=2 * MB, scales=4 * MB, zeros=5 * MB, bias=6 * MB, M=4, N=256, K=512,
                group=64, dtype=0, y=8 * MB)

    def call(**over):
        return lib.infini_attn_linear_w4(*dict(good, **over).values(), None)

    for name in ("x", "packed", "scales", "y"):
        assert call(**{name: None}) == api.ERR_ARG
    for name in ("M", "N", "K", "group"):
        assert call(**{name: 0}) == api.ERR_ARG
    assert call(dtype=3) == api.ERR_ARG
    assert call(K=516) == api.ERR_UNSUPPORTED
    assert call(group=16) == api.ERR_UNSUPPORTED
    assert call(M=65535 * 64 + 1) == api.ERR_UNSUPPORTED
    assert call(N=0x7fffffff) == api.ERR_UNSUPPORTED
    assert call(zeros=5 * MB + 2) == api.ERR_ALIGN
    assert call(y=good["x"]) == api.ERR_ALIAS
    assert call(y=good["packed"] + 64) == api.ERR_ALIAS

    dims = api.make_dims(2, 4, 2, 3, 64, 64, 0)
    proj = dict(x=1 * MB, packed=2 * MB, scales=4 * MB, zeros=None, bias=None, cos=6 * MB, sin=7 * MB,
                n_pos=16, positions=9 * MB, dims=ctypes.byref(dims), d_model=256, group=128, q=10 * MB,
                k=11 * MB, v=12 * MB)

    def qkv(**over):
        return lib.infini_attn_qkv_project_w4(*dict(proj, **over).values(), None)

    for name in ("x", "packed", "scales", "q", "k", "v", "sin"):
        assert qkv(**{name: None}) == api.ERR_ARG
    assert qkv(n_pos=0) == api.ERR_ARG
    assert qkv(positions=None, n_pos=2) == api.ERR_ARG       # fewer table rows than tokens
    assert qkv(cos=None, sin=None) == api.ERR_ARG            # positions without tables
    assert qkv(dims=ctypes.byref(api.make_dims(2, 4, 2, 3, 64, 32, 0))) == api.ERR_UNSUPPORTED
    assert qkv(dims=ctypes.byref(api.make_dims(2, 4, 2, 3, 48, 48, 0))) == api.ERR_UNSUPPORTED
    assert qkv(dims=ctypes.byref(api.make_dims(1 << 12, 4, 2, 1 << 12, 64, 64, 0))) == api.ERR_UNSUPPORTED
    assert qkv(dims=ctypes.byref(api.make_dims(1, 1 << 25, 1, 1, 64, 64, 0))) == api.ERR_UNSUPPORTED
    assert qkv(d_model=12) == api.ERR_UNSUPPORTED
    assert qkv(q=10 * MB + 4) == api.ERR_ALIGN
    assert qkv(k=proj["v"] + 16) == api.ERR_ALIAS
    assert qkv(q=proj["positions"]) == api.ERR_ALIAS

    assert lib.infini_attn_w4_quantize(None, 4, 64, 32, 0, MB, 2 * MB, None, None) == api.ERR_ARG
    assert lib.infini_attn_w4_quantize(MB, 4, 60, 32, 0, 2 * MB, 3 * MB, None, None) == api.ERR_UNSUPPORTED
    assert lib.infini_attn_w4_quantize(MB, 4, 64, 48, 0, 2 * MB, 3 * MB, None, None) == api.ERR_UNSUPPORTED
    assert lib.infini_attn_w4_quantize(MB, 4, 64, 32, 0, MB + 64, 3 * MB, None, None) == api.ERR_ALIAS
    assert lib.infini_attn_w4_pack(MB, 4, 64, None, None) == api.ERR_ARG
    assert lib.infini_attn_w4_pack(MB, 0, 64, 2 * MB, None) == api.ERR_ARG
    assert lib.infini_attn_w4_dequantize(MB, 2 * MB, None, 4, 64, 32, 1, MB, None) == api.ERR_ALIAS
    assert lib.infini_attn_w4_dequantize(MB, 2 * MB, None, 4, 64, 32, 7, 3 * MB, None) == api.ERR_ARG
    assert api.status_string(api.ERR_RANGE) != api.status_string(12345)


def test_q4_checks_arguments_on_the_host(lib):
    """Argument checks of the 4-bit segment buffer's calls return before any
    CUDA call."""
    MB = 1 << 20
    d = api.make_dims(2, 4, 2, 3, 64, 64, 1)

    def cache(**over):
        c = dict(dict(k_codes=1 * MB, k_scale=2 * MB, v_codes=3 * MB, v_scale=4 * MB), **over)
        return ctypes.byref(api._CacheQ4Ptrs(*c.values()))

    n = lib.infini_attn_decode_q4_workspace_bytes(ctypes.byref(d), 100)
    assert n >= 2 * 4 * (64 + 2) * 4
    for bad in (api.make_dims(2, 3, 2, 1, 64, 64, 1), api.make_dims(0, 4, 2, 1, 64, 64, 1),
                api.make_dims(2, 4, 2, 1, 64, 32, 1), api.make_dims(2, 4, 2, 1, 48, 48, 1),
                api.make_dims(1 << 14, 4, 4, 1, 64, 64, 1)):
        assert lib.infini_attn_decode_q4_workspace_bytes(ctypes.byref(bad), 100) == 0
    assert lib.infini_attn_decode_q4_workspace_bytes(ctypes.byref(d), 0) == 0
    assert lib.infini_attn_decode_q4_workspace_bytes(ctypes.byref(d), (1 << 30) + 1) == 0
    good = dict(q=5 * MB, k=6 * MB, v=7 * MB, beta=8 * MB, cache=cache(), pos=9 * MB, M=10 * MB, z=11 * MB,
                seg=100, dims=ctypes.byref(d), out=12 * MB, ws=16 * MB, ws_n=n)

    def step(**over):
        return lib.infini_attn_decode_step_q4(*dict(good, **over).values(), None)

    for name in ("q", "k", "v", "beta", "cache", "pos", "M", "z", "out", "dims"):
        assert step(**{name: None}) == api.ERR_ARG, name
    for name in ("k_codes", "k_scale", "v_codes", "v_scale"):
        assert step(cache=cache(**{name: None})) == api.ERR_ARG
        assert step(cache=cache(**{name: 32 * MB + 8})) == api.ERR_ALIGN
        assert step(cache=cache(**{name: 12 * MB + 64})) == api.ERR_ALIAS     # over the output
        assert step(cache=cache(**{name: good["M"] + 64})) == api.ERR_ALIAS   # over an input
    assert step(cache=cache(v_codes=1 * MB + 512)) == api.ERR_ALIAS           # over each other
    assert step(seg=0) == api.ERR_ARG
    assert step(out=good["q"]) == api.ERR_ALIAS
    assert step(pos=9 * MB + 4) == api.ERR_ALIGN
    assert step(ws_n=n - 1) == api.ERR_WORKSPACE
    assert step(ws=16 * MB + 64) == api.ERR_WORKSPACE
    assert step(ws=None) == api.ERR_ARG
    assert step(ws=good["z"]) == api.ERR_ALIAS
    assert step(dims=ctypes.byref(api.make_dims(2, 4, 2, 1, 64, 64, 5))) == api.ERR_ARG

    def append(k=5 * MB, v=6 * MB, pos=7 * MB, dims=d, seg=100, c=None):
        return lib.infini_attn_cache_q4_append(k, v, pos, ctypes.byref(dims), seg, c or cache(), None)

    assert append(k=None) == api.ERR_ARG
    assert append(pos=None) == api.ERR_ARG
    assert append(seg=2) == api.ERR_ARG                                       # 3 rows into 2
    assert append(dims=api.make_dims(2, 4, 2, 0, 64, 64, 1)) == api.ERR_ARG
    assert append(k=3 * MB) == api.ERR_ALIAS
    assert append(v=6 * MB + 4) == api.ERR_ALIGN

    def read(k=5 * MB, v=6 * MB, dims=d, seg=100):
        return lib.infini_attn_cache_q4_read(cache(), ctypes.byref(dims), seg, k, v, None)

    assert read(k=None) == api.ERR_ARG
    assert read(seg=2) == api.ERR_ARG
    assert read(k=6 * MB) == api.ERR_ALIAS
    assert read(v=4 * MB) == api.ERR_ALIAS

    need = lib.infini_attn_state_update_q4_workspace_bytes(ctypes.byref(d), 0)
    assert need > 2 * 2 * 2 * 3 * 64 * 4
    assert lib.infini_attn_state_update_q4_workspace_bytes(ctypes.byref(d), 9) == 0

    def update(M=5 * MB, z=6 * MB, rule=0, dims=d, seg=100, Mo=7 * MB, zo=8 * MB, ws=16 * MB, ws_n=need):
        return lib.infini_attn_state_update_q4(cache(), M, z, rule, ctypes.byref(dims), seg, Mo, zo, ws, ws_n,
                                               None)

    assert update(M=None) == api.ERR_ARG
    assert update(rule=5) == api.ERR_ARG
    assert update(seg=2) == api.ERR_ARG
    assert update(ws_n=need - 1) == api.ERR_WORKSPACE
    assert update(Mo=8 * MB - 64) == api.ERR_ALIAS
    assert update(zo=5 * MB) == api.ERR_ALIAS
    assert update(ws=1 * MB) == api.ERR_ALIAS


def test_plain_c_program_uses_the_boundary(tmp_path):
    """The header compiles as C99 and a C program linked against the library
    gets the documented answers from the host-side calls (no GPU needed)."""
    import shutil
    import subprocess

    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lib_dir = os.path.dirname(api.LIB_PATH)
    exe = tmp_path / "c_abi_check"
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "c_abi_check.c"), api.LIB_PATH,
                    f"-Wl,-rpath,{lib_dir}", "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stderr
    assert res.stdout.strip() == "c-abi ok"
