"""CPU checks of the C ABI: the library loads, exports every function fa.h
declares, and rejects bad arguments before touching the GPU."""

import ctypes

import pytest

from exact_softmax_attention_fa_gb300 import _lib
from exact_softmax_attention_fa_gb300.build import build, LIB_PATH


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
P = 0x10000  # a 16-byte aligned fake device address.
# Every call below has at least one invalid argument, so the library returns
# before any CUDA call and the fake address is never used, even on a GPU machine.


def test_exports_every_header_function(lib):
    names = _lib.header_functions()
    assert {"fa_fwd", "fa_bwd", "fa_bwd_workspace_size", "fa_status_string"} <= set(names)
    raw = ctypes.CDLL(LIB_PATH)
    for n in names:
        assert hasattr(raw, n), n
    assert set(_lib._SIGNATURES) == set(names)


def test_status_strings(lib):
    for code, name in _lib.STATUS_NAMES.items():
        assert lib.fa_status_string(code).decode().startswith(name)
    assert lib.fa_version() >= 100


def test_status_detail_rejects_a_null_word(lib):
    """The argument check comes before any device access (no GPU needed)."""
    assert lib.fa_get_device_status_detail(None, None) == INVALID


def fwd(lib, q=P, k=P, v=P, o=P, lse=P, B=1, H=1, N=128, d=64, causal=0, scale=0.125):
    return lib.fa_fwd(q, k, v, o, lse, B, H, N, d, causal, scale, None)


def bwd(lib, ptr=P, lse=P, ws=P, ws_bytes=1 << 30, B=1, H=1, N=128, d=64, causal=0, scale=0.125):
    return lib.fa_bwd(ptr, ptr, ptr, ptr, lse, ptr, ptr, ptr, ptr, B, H, N, d, causal, scale, ws, ws_bytes, None)


@pytest.mark.parametrize("d", [0, 32, 96, 160, 512])
def test_unsupported_head_dim(lib, d):
    assert fwd(lib, d=d) == UNSUPPORTED
    assert bwd(lib, d=d) == UNSUPPORTED
    assert lib.fa_bwd_workspace_size(1, 1, 128, d) == 0


@pytest.mark.parametrize("kw", [dict(B=-1), dict(H=-2), dict(N=-1), dict(causal=2), dict(causal=-1),
                                dict(scale=0.0), dict(scale=-0.1), dict(scale=float("nan")),
                                dict(scale=float("inf")), dict(q=0), dict(o=0), dict(lse=0)])
def test_invalid_arguments(lib, kw):
    assert fwd(lib, **kw) == INVALID


def test_empty_problem_is_a_no_op(lib):
    for kw in (dict(N=0), dict(B=0), dict(H=0)):
        assert fwd(lib, q=0, k=0, v=0, o=0, lse=0, **kw) == OK
        assert bwd(lib, ptr=0, lse=0, ws=0, ws_bytes=0, **kw) == OK
        assert lib.fa_bwd_workspace_size(kw.get("B", 1), kw.get("H", 1), kw.get("N", 128), 64) == 0


def fwd_gqa(lib, ptr=P, lse=P, B=1, Hq=4, Hkv=2, N=128, d=64, causal=0, scale=0.125):
    return lib.fa_fwd_gqa(ptr, ptr, ptr, ptr, lse, B, Hq, Hkv, N, d, causal, scale, None)


def bwd_gqa(lib, ptr=P, lse=P, ws=P, ws_bytes=1 << 30, B=1, Hq=4, Hkv=2, N=128, d=64, causal=0, scale=0.125):
    return lib.fa_bwd_gqa(ptr, ptr, ptr, ptr, lse, ptr, ptr, ptr, ptr, B, Hq, Hkv, N, d, causal, scale, ws, ws_bytes,
                          None)


@pytest.mark.parametrize("Hq,Hkv", [(4, 0), (4, -1), (4, 3), (2, 4), (4, 8)])
def test_grouped_heads_must_divide(lib, Hq, Hkv):
    assert fwd_gqa(lib, Hq=Hq, Hkv=Hkv) == INVALID
    assert bwd_gqa(lib, Hq=Hq, Hkv=Hkv) == INVALID


def test_grouped_workspace_size(lib):
    for B, Hq, Hkv, N, d in ((2, 8, 2, 1000, 64), (1, 16, 1, 300, 128), (1, 4, 4, 100, 128), (1, 4, 2, 100, 256)):
        base = lib.fa_bwd_workspace_size(B, Hq, N, d)
        g = Hq // Hkv
        extra = 0 if (g == 1 or d == 256) else g * B * Hkv * N * d * 8  # fp32 dK + dV partial per chunk
        assert lib.fa_bwd_gqa_workspace_size(B, Hq, Hkv, N, d) == base + extra
    assert lib.fa_bwd_gqa_workspace_size(1, 4, 3, 128, 64) == 0
    assert lib.fa_bwd_gqa_workspace_size(1, 4, 0, 128, 64) == 0


def test_deterministic_backward_checks(lib):
    def det(d=64, Hq=4, Hkv=2, ws=P, ws_bytes=1 << 30, ptr=P):
        return lib.fa_bwd_gqa_deterministic(ptr, ptr, ptr, ptr, P, ptr, ptr, ptr, ptr, 1, Hq, Hkv, 128, d, 0, 0.125,
                                            ws, ws_bytes, None)
    assert det(d=256, ws=0) == WORKSPACE  # d = 256 is supported; the missing workspace is caught
    assert det(d=96) == UNSUPPORTED
    assert det(Hkv=3) == INVALID
    assert det(ptr=0) == INVALID
    assert det(ws=0) == WORKSPACE
    assert lib.fa_bwd_deterministic(P, P, P, P, P, P, P, P, P, 1, 1, 128, 256, 0, 0.125, 0, 0, None) == WORKSPACE
    assert lib.fa_bwd_deterministic(P, P, P, P, P, P, P, P, P, 1, 1, 128, 96, 0, 0.125, P, 1 << 30, None) == UNSUPPORTED


def test_split_key_forward_checks(lib):
    def fwd_split(Nq=64, Nk=256, causal=0, splits=1, ws=P, ws_bytes=1 << 30, Hq=2, Hkv=2, d=64, ptr=P):
        return lib.fa_fwd_splitkv(ptr, ptr, ptr, ptr, P, 1, Hq, Hkv, Nq, Nk, d, causal, 0.125, splits, ws, ws_bytes,
                                  None)
    assert fwd_split(Nq=300, Nk=200, causal=1) == INVALID  # a causal block longer than the keys
    assert fwd_split(Nk=0) == INVALID
    assert fwd_split(Nk=-1) == INVALID
    assert fwd_split(splits=-1) == INVALID
    assert fwd_split(splits=257) == INVALID
    assert fwd_split(Hkv=3) == INVALID
    assert fwd_split(d=96) == UNSUPPORTED
    assert fwd_split(splits=2, ws=0) == WORKSPACE
    assert fwd_split(splits=2, ws_bytes=16) == WORKSPACE
    assert fwd_split(splits=2, ws=P + 16) == MISALIGNED
    assert fwd_split(ptr=P + 8) == MISALIGNED
    assert fwd_split(Nq=0, ptr=0) == OK
    need = lib.fa_fwd_splitkv_workspace_size(1, 2, 64, 64, 3)
    assert need == 3 * 2 * 64 * 64 * 4 + ((3 * 2 * 64 * 4 + 255) // 256) * 256
    assert lib.fa_fwd_splitkv_workspace_size(1, 2, 64, 64, 1) == 0
    assert lib.fa_fwd_splitkv_workspace_size(1, 2, 64, 64, 300) == 0


def test_deterministic_phase_checks(lib):
    assert lib.fa_bwd_dkdv(P, P, P, P, P, P, 1, 1, 128, 96, 0, 0.125, P, 1 << 30, None) == UNSUPPORTED
    assert lib.fa_bwd_dq(P, P, P, P, P, 1, 1, 128, 96, 0, 0.125, P, 1 << 30, None) == UNSUPPORTED
    assert lib.fa_bwd_dkdv(P, P, P, P, 0, P, 1, 1, 128, 256, 0, 0.125, P, 1 << 30, None) == INVALID
    assert lib.fa_bwd_dq(P, P, P, P, P, 1, 1, 128, 256, 0, 0.125, 0, 0, None) == WORKSPACE
    assert lib.fa_bwd_dkdv(P, P, P, P, 0, P, 1, 1, 128, 64, 0, 0.125, P, 1 << 30, None) == INVALID
    assert lib.fa_bwd_dq(P, P, P, P, P, 1, 1, 128, 64, 0, 0.125, 0, 0, None) == WORKSPACE
    assert lib.fa_bwd_dq(P, P, P, P, P, 1, 1, 128, 64, 2, 0.125, P, 1 << 30, None) == INVALID
    assert lib.fa_bwd_dkdv(0, 0, 0, 0, 0, 0, 1, 1, 0, 64, 0, 0.125, 0, 0, None) == OK


def test_grouped_heads_other_checks(lib):
    assert fwd_gqa(lib, d=96) == UNSUPPORTED
    assert bwd_gqa(lib, scale=0.0) == INVALID
    assert fwd_gqa(lib, ptr=0) == INVALID
    assert bwd_gqa(lib, ws=0) == WORKSPACE
    assert fwd_gqa(lib, ptr=P + 8) == MISALIGNED
    # empty problems do nothing, null pointers allowed
    assert fwd_gqa(lib, ptr=0, lse=0, Hq=0, Hkv=0) == OK
    assert bwd_gqa(lib, ptr=0, lse=0, ws=0, ws_bytes=0, N=0) == OK


@pytest.mark.parametrize("which", ["q", "k", "v", "o"])
def test_misaligned_bf16(lib, which):
    assert fwd(lib, **{which: P + 8}) == MISALIGNED


def test_misaligned_lse(lib):
    assert fwd(lib, lse=P + 2) == MISALIGNED


def test_backward_workspace_checks(lib):
    need = lib.fa_bwd_workspace_size(1, 1, 128, 64)
    assert need > 0
    assert bwd(lib, ws=0) == WORKSPACE
    assert bwd(lib, ws_bytes=need - 1) == WORKSPACE
    assert bwd(lib, ws=P + 16, ws_bytes=need) == MISALIGNED
    assert bwd(lib, ptr=P + 8) == MISALIGNED


def test_workspace_size_formula(lib):
    # D and base-2 L (fp32 per padded row) + fp32 dQ accumulator, heads padded
    # to 128 rows, + 256 bytes of work-item counter
    for B, H, N, d in ((2, 4, 1024, 64), (1, 16, 1000, 128), (1, 2, 1, 256)):
        rows = B * H * ((N + 127) // 128 * 128)
        expect = 0
        for nbytes in (rows * 4, rows * 4, rows * d * 4, 256):
            expect = (expect + 255) // 256 * 256 + nbytes
        assert lib.fa_bwd_workspace_size(B, H, N, d) == expect


def test_python_binding_rejects_cpu_tensors():
    torch = pytest.importorskip("torch")
    import exact_softmax_attention_fa_gb300 as fa
    q = torch.zeros(1, 1, 128, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.fa_fwd(q, q, q, q.clone(), torch.zeros(1, 1, 128), False, 0.125)
    with pytest.raises(TypeError):
        fa.fa_fwd(q.float(), q, q, q, torch.zeros(1, 1, 128), False, 0.125)


def test_noalloc_backward_validation(lib):
    """Argument errors and oversized problems are rejected before any CUDA call."""
    def call(B=1, H=1, N=128, d=64, causal=0, scale=0.125, ptr=P, lse=P):
        return lib.fa_bwd_noalloc(ptr, ptr, ptr, ptr, lse, ptr, ptr, ptr, ptr, B, H, N, d, causal, scale, None)
    assert call(d=96) == UNSUPPORTED
    assert call(scale=-1.0) == INVALID
    assert call(N=0, ptr=0, lse=0) == OK
    # 16 heads x 8192 rows at d=128 need ~68 MB of scratch, beyond the compiled 16 MiB
    assert lib.fa_bwd_workspace_size(1, 16, 8192, 128) > (16 << 20)
    assert call(B=1, H=16, N=8192, d=128) == WORKSPACE


def test_host_entry_checks(lib):
    """fa_fwd_bwd_host: size formula and argument errors (all before any CUDA call)."""
    def call(ptr=P, lse=P, buf=P, nbytes=1 << 34, B=1, H=2, N=128, d=64, causal=0, scale=0.125):
        return lib.fa_fwd_bwd_host(ptr, ptr, ptr, ptr, ptr, lse, ptr, ptr, ptr, B, H, N, d, causal, scale, buf,
                                   nbytes, None)
    a = lambda n: (n + 255) // 256 * 256

    def groups(BH):
        """Head counts of the plan the header states: an eighth of the heads,
        the rest (less another eighth) in two halves, then that eighth."""
        g0 = (BH + 7) // 8
        last = (BH + 7) // 8 if BH - g0 >= 2 else BH - g0
        mid = BH - g0 - last
        return [h for h in (g0, mid // 2, mid - mid // 2, last) if h > 0]

    assert groups(32) == [4, 12, 12, 4] and groups(3) == [1, 1, 1] and groups(2) == [1, 1] and groups(1) == [1]
    shapes = [(1, 2, 128, 64), (2, 3, 1000, 128), (1, 1, 1, 256), (2, 16, 8192, 128), (1, 5, 300, 64)]
    shapes += [(1, bh, 640, 128) for bh in range(1, 41)]  # every group split up to 40 heads
    for B, H, N, d in shapes:
        rows = B * H * N
        need = 8 * a(rows * d * 2) + a(rows * 4)
        need += sum(a(lib.fa_bwd_workspace_size(1, h, N, d)) for h in groups(B * H))
        assert lib.fa_fwd_bwd_host_device_bytes(B, H, N, d) == need
    need = lib.fa_fwd_bwd_host_device_bytes(1, 2, 128, 64)
    assert lib.fa_fwd_bwd_host_device_bytes(1, 2, 0, 64) == 0
    assert lib.fa_fwd_bwd_host_device_bytes(1, 2, 128, 96) == 0
    assert call(d=96) == UNSUPPORTED
    assert call(scale=0.0) == INVALID
    assert call(causal=3) == INVALID
    assert call(ptr=0) == INVALID
    assert call(lse=0) == INVALID
    assert call(buf=0) == WORKSPACE
    assert call(nbytes=need - 1) == WORKSPACE
    assert call(buf=P + 16, nbytes=need) == MISALIGNED
    assert call(N=0, ptr=0, lse=0, buf=0, nbytes=0) == OK


def test_forward_host_entry_checks(lib):
    """fa_fwd_host: size formula and argument errors (all before any CUDA call)."""
    def call(ptr=P, lse=P, buf=P, nbytes=1 << 34, B=1, H=2, N=128, d=64, causal=0, scale=0.125):
        return lib.fa_fwd_host(ptr, ptr, ptr, ptr, lse, B, H, N, d, causal, scale, buf, nbytes, None)
    a = lambda n: (n + 255) // 256 * 256
    for B, H, N, d in ((1, 2, 128, 64), (2, 3, 1000, 128), (1, 1, 1, 256)):
        rows = B * H * N
        assert lib.fa_fwd_host_device_bytes(B, H, N, d) == 4 * a(rows * d * 2) + a(rows * 4)
    need = lib.fa_fwd_host_device_bytes(1, 2, 128, 64)
    assert lib.fa_fwd_host_device_bytes(0, 2, 128, 64) == 0
    assert call(d=32) == UNSUPPORTED
    assert call(scale=float("nan")) == INVALID
    assert call(ptr=0) == INVALID
    assert call(lse=0) == INVALID
    assert call(buf=0) == WORKSPACE
    assert call(nbytes=need - 1) == WORKSPACE
    assert call(buf=P + 64, nbytes=need) == MISALIGNED
    assert call(H=0, ptr=0, lse=0, buf=0, nbytes=0) == OK


def test_preprocess_stats_checks(lib):
    """The stats-only preprocess validates like the full one (no GPU needed)."""
    assert lib.fa_bwd_preprocess_stats(P, P, P, 1, 1, 128, 96, P, 1 << 30, None) == UNSUPPORTED
    assert lib.fa_bwd_preprocess_stats(0, P, P, 1, 1, 128, 64, P, 1 << 30, None) == INVALID
    assert lib.fa_bwd_preprocess_stats(P, P, P, 1, 1, 128, 64, 0, 0, None) == WORKSPACE
    assert lib.fa_bwd_preprocess_stats(P + 8, P, P, 1, 1, 128, 64, P, 1 << 30, None) == MISALIGNED
    assert lib.fa_bwd_preprocess_stats(0, 0, 0, 1, 1, 0, 64, 0, 0, None) == OK


def test_debug_skip_hook_checks(lib):
    """Only the role codes of the status word are accepted; 0 turns the hook off."""
    for bad in (4, 10, 15, 99, 1 << 31):
        assert lib.fa_debug_skip_arrival(bad) == INVALID
    for good in (1, 2, 3, 11, 12, 13, 14):
        assert lib.fa_debug_skip_arrival(good) == OK
    assert lib.fa_debug_skip_arrival(0) == OK


# ---------------------------------------------------------------------------
# Per-head norm with position rotation: refusals before any CUDA call.
# ---------------------------------------------------------------------------
def strides9(*v):
    return (ctypes.c_longlong * 9)(*(v or (6 * 64 * 8, 64, 6 * 64) * 3))


def norm_rope(lib, ptr=P, v_in=P, v=P, st=None, wq=P, wk=P, w_bf16=0, cos=P, rows=100, pos=P, B=2, Hq=4, Hkv=1, N=8,
              d=64, rot=64, inter=0, eps=1e-6):
    return lib.fa_norm_rope_fwd(ptr, ptr, v_in, strides9() if st is None else st, wq, wk, w_bf16, cos, cos, rows, pos,
                                ptr, ptr, v, B, Hq, Hkv, N, d, rot, inter, eps, None)


def norm_rope_bwd(lib, ptr=P, x=P, st=None, out=None, w=P, dw=P, ws=P, ws_bytes=1 << 30, B=2, Hq=4, Hkv=1, N=8, d=64):
    return lib.fa_norm_rope_bwd(ptr, ptr, ptr, x, x, strides9() if st is None else st, w, w, 0, P, P, 100, None, ptr,
                                ptr, ptr, strides9() if out is None else out, dw, dw, B, Hq, Hkv, N, d, 64, 0, 1e-6, ws,
                                ws_bytes, None)


@pytest.mark.parametrize("kw", [dict(B=-1), dict(Hq=-1), dict(Hkv=-1), dict(N=-1), dict(rows=-1), dict(rot=-16),
                                dict(rot=8), dict(rot=80), dict(inter=2), dict(w_bf16=2), dict(wq=0), dict(wk=0),
                                dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(cos=0),
                                dict(rows=0), dict(pos=0, rows=7), dict(ptr=0), dict(v_in=0), dict(v=0),
                                dict(st=strides9(-8, 64, 512, 0, 0, 0, 0, 0, 0)), dict(B=1 << 20, N=1 << 10)])
def test_norm_rope_invalid_arguments(lib, kw):
    assert norm_rope(lib, **kw) == INVALID


def test_norm_rope_alignment_and_sizes(lib):
    for kw in (dict(ptr=P + 8), dict(v=P + 2), dict(cos=P + 4), dict(wq=P + 8), dict(pos=P + 2),
               dict(st=strides9(6 * 64 * 8, 64, 6 * 64 + 4, 0, 0, 0, 0, 0, 0))):
        assert norm_rope(lib, **kw) == MISALIGNED
    for d in (32, 96, 512):
        assert norm_rope(lib, d=d, rot=0) == UNSUPPORTED
    assert norm_rope(lib, N=0, ptr=0) == OK and norm_rope(lib, B=0, ptr=0, st=strides9()) == OK
    assert norm_rope(lib, Hq=0, Hkv=0) == OK


def test_norm_rope_backward_checks(lib):
    assert norm_rope_bwd(lib, ptr=0) == INVALID
    assert norm_rope_bwd(lib, x=0) == INVALID
    assert norm_rope_bwd(lib, dw=0) == INVALID
    assert norm_rope_bwd(lib, dw=P + 2) == MISALIGNED
    assert norm_rope_bwd(lib, ws=0) == WORKSPACE
    size = lib.fa_norm_rope_bwd_workspace_size(2, 4, 1, 8, 64)
    assert size > 0 and norm_rope_bwd(lib, ws_bytes=size - 1) == WORKSPACE
    assert norm_rope_bwd(lib, ws=P + 128) == MISALIGNED
    # rows that overlap: a broadcast head, heads closer than d, tokens inside a head's rows
    good = (6 * 64 * 8, 64, 6 * 64)
    for bad in ((6 * 64 * 8, 0, 6 * 64), (6 * 64 * 8, 32, 6 * 64), (6 * 64 * 8, 64, 3 * 64), (0, 64, 6 * 64)):
        assert norm_rope_bwd(lib, out=strides9(*bad, *good, *good)) == INVALID
    assert lib.fa_norm_rope_bwd_workspace_size(2, 4, 1, 8, 96) == 0
    assert lib.fa_norm_rope_bwd_workspace_size(0, 4, 1, 8, 64) == 0


# ---------------------------------------------------------------------------
# The paged 8-bit cache: refusals before any CUDA call.
# ---------------------------------------------------------------------------
def kv8_append(lib, kv=P, cache=P, scale=P, table=P, lens=P, counts=None, B=2, Hkv=2, n=4, d=64, page=16, pages=8, mp=4):
    return lib.fa_kv8_append(kv, kv, cache, cache, scale, scale, table, lens, counts, B, Hkv, n, d, page, pages, mp,
                             None)


def kv8_gather(lib, kv=P, cache=P, scale=P, table=P, lens=P, counts=None, B=2, Hkv=2, n=4, d=64, page=16, pages=8, mp=4):
    return lib.fa_kv8_gather(cache, cache, scale, scale, table, lens, kv, kv, B, Hkv, n, d, page, pages, mp, None)


@pytest.mark.parametrize("call", [kv8_append, kv8_gather])
def test_kv8_refusals(lib, call):
    for kw in (dict(B=-1), dict(Hkv=-1), dict(n=-1), dict(pages=-1), dict(mp=-1), dict(pages=0), dict(mp=0), dict(kv=0),
               dict(cache=0), dict(scale=0), dict(table=0), dict(lens=0), dict(Hkv=65536), dict(mp=1 << 27),
               dict(n=(1 << 31) - 1), dict(B=1 << 20, n=1 << 16)):
        assert call(lib, **kw) == INVALID, kw
    for kw in (dict(d=96), dict(d=512), dict(page=8), dict(page=48), dict(page=256), dict(page=0)):
        assert call(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(kv=P + 8), dict(cache=P + 8), dict(scale=P + 2), dict(table=P + 1), dict(lens=P + 2)):
        assert call(lib, **kw) == MISALIGNED, kw
    for kw in (dict(B=0), dict(Hkv=0), dict(n=0)):
        assert call(lib, kv=0, cache=0, scale=0, table=0, lens=0, pages=0, mp=0, **kw) == OK, kw


def test_kv8_append_checks_counts(lib):
    assert kv8_append(lib, counts=P + 2) == MISALIGNED


def fwd_kv8(lib, q=P, cache=P, scale_t=P, table=P, lens=P, counts=None, o=P, lse=P, B=2, Hq=4, Hkv=2, Nq=1, d=64, page=16,
            pages=8, mp=4, causal=1, scale=0.125, ws=P, ws_bytes=1 << 30):
    return lib.fa_fwd_kv8(q, cache, cache, scale_t, scale_t, table, lens, counts, o, lse, B, Hq, Hkv, Nq, d, page, pages,
                          mp, causal, scale, ws, ws_bytes, None)


def test_fwd_kv8_refusals(lib):
    for kw in (dict(B=-1), dict(Hq=-4), dict(Hkv=-1), dict(Hkv=0), dict(Hkv=3), dict(Nq=-1), dict(pages=0), dict(mp=0),
               dict(q=0), dict(cache=0), dict(scale_t=0), dict(table=0), dict(lens=0), dict(o=0), dict(lse=0),
               dict(causal=2), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(mp=1 << 27), dict(B=1 << 15, Hq=1 << 10, Nq=1 << 8), dict(pages=1 << 30)):
        assert fwd_kv8(lib, **kw) == INVALID, kw
    for kw in (dict(d=96), dict(page=8), dict(page=256)):
        assert fwd_kv8(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(q=P + 8), dict(cache=P + 8), dict(scale_t=P + 2), dict(table=P + 2), dict(counts=P + 1), dict(o=P + 2),
               dict(lse=P + 2), dict(ws=P + 128)):
        assert fwd_kv8(lib, **kw) == MISALIGNED, kw
    size = lib.fa_fwd_kv8_workspace_size(2, 4, 2, 1, 64)
    assert size > 0
    for kw in (dict(ws=0), dict(ws_bytes=size - 1)):
        assert fwd_kv8(lib, **kw) == WORKSPACE, kw
    for kw in (dict(B=0), dict(Hq=0), dict(Hq=0, Hkv=0), dict(Nq=0)):
        assert fwd_kv8(lib, q=0, cache=0, scale_t=0, table=0, lens=0, o=0, lse=0, ws=0, ws_bytes=0, **kw) == OK, kw


def test_fwd_kv8_workspace_size(lib):
    size = lib.fa_fwd_kv8_workspace_size
    assert size(2, 4, 3, 1, 64) == 0 and size(0, 4, 2, 1, 64) == 0 and size(2, 4, 2, 0, 64) == 0
    assert size(2, 4, 2, 1, 96) == 0
    # it does not grow with the batch: parts belong to warps
    assert size(1, 4, 2, 1, 128) == size(500, 4, 2, 1, 128) > 0


def test_a_refused_append_leaves_the_cache_lengths():
    import torch
    import exact_softmax_attention_fa_gb300 as fa
    cache = fa.KV8Cache(2, 1, 64, 32, page=16, device="cpu")
    k = torch.zeros(2, 1, 3, 64, dtype=torch.bfloat16)
    for bad, counts in ((k, None), (k.float(), None), (k[:, :, :, :32], None), (k, torch.ones(2, dtype=torch.int32))):
        with pytest.raises(Exception):  # not on a CUDA device, and of the wrong type or shape
            cache.append(bad, bad, counts)
        assert cache.lens.tolist() == [0, 0]


def test_the_cache_attention_has_roles_of_its_own_for_the_skip_hook(lib):
    for bad in (21, 31, 33, 40, 45):
        assert lib.fa_debug_skip_arrival(bad) == INVALID
    for good in (41, 42, 43, 44):
        assert lib.fa_debug_skip_arrival(good) == OK
    assert lib.fa_debug_skip_arrival(0) == OK


def kv8_advance(lib, lens=P, counts=None, taken=P, B=2, n=4, page=16, mp=4):
    return lib.fa_kv8_advance(lens, counts, taken, B, n, page, mp, None)


def test_kv8_advance_refusals(lib):
    for kw in (dict(B=-1), dict(n=-1), dict(mp=-1), dict(lens=0), dict(taken=0), dict(mp=1 << 27), dict(n=(1 << 31) - 1)):
        assert kv8_advance(lib, **kw) == INVALID, kw
    for page in (0, 8, 48, 256):
        assert kv8_advance(lib, page=page) == UNSUPPORTED
    for kw in (dict(lens=P + 2), dict(counts=P + 1), dict(taken=P + 2)):
        assert kv8_advance(lib, **kw) == MISALIGNED, kw
    assert kv8_advance(lib, B=0, lens=0, taken=0) == OK


def test_fwd_kv8_filled_has_the_checks_of_fwd_kv8(lib):
    def call(q=P, ws_bytes=1 << 30, causal=1, Hkv=2, d=64):
        return lib.fa_fwd_kv8_filled(q, P, P, P, P, P, P, None, P, P, 2, 4, Hkv, 1, d, 16, 8, 4, causal, 0.125, P, ws_bytes, None)

    assert call(q=0) == INVALID and call(causal=2) == INVALID and call(Hkv=3) == INVALID
    assert call(d=96) == UNSUPPORTED and call(q=P + 8) == MISALIGNED and call(ws_bytes=16) == WORKSPACE
