"""Refusals of the entry points for packed sequences and for the rotation by axes, before any CUDA call."""

import ctypes

import pytest

from exact_softmax_attention_fa_gb300 import _lib

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
P = 1 << 20  # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def strides(*s):
    return (ctypes.c_longlong * len(s))(*s)


def plan(lib, cu=P, B=2, rows=100, causal=1, plan=P, size=None):
    return lib.fa_packed_plan(cu, B, rows, causal, plan, 1 << 30 if size is None else size, None)


def test_plan_refusals(lib):
    for kw in (dict(B=-1), dict(rows=-1), dict(causal=2), dict(causal=-1), dict(cu=0)):
        assert plan(lib, **kw) == INVALID, kw
    for kw in (dict(cu=P + 2), dict(plan=P + 128)):
        assert plan(lib, **kw) == MISALIGNED, kw
    need = lib.fa_packed_plan_size(2, 100)
    for kw in (dict(plan=0), dict(size=need - 1), dict(size=0)):
        assert plan(lib, **kw) == WORKSPACE, kw


def test_plan_size(lib):
    size = lib.fa_packed_plan_size
    assert size(-1, 4) == 0 and size(4, -1) == 0
    assert 0 < size(0, 0) <= 256
    # every list of lengths fits: full tiles, and one begun tile (and pair) a sequence
    for B, rows in ((1, 1), (3, 1000), (500, 500), (100000, 7), (7, 1 << 20)):
        tiles, pairs = rows // 128 + min(B, rows), rows // 256 + min(B, rows)
        assert size(B, rows) == 256 + 16 * (tiles + pairs)


def fwd(lib, q=P, k=P, v=P, st=None, o=P, lse=P, plan=P, rows=100, Hq=4, Hkv=2, d=64, causal=1, scale=0.125, fill=0):
    st = strides(256, 64, 128, 64, 128, 64, 256, 64) if st is None else st
    return lib.fa_fwd_packed(q, k, v, st, o, lse, plan, rows, Hq, Hkv, d, causal, scale, fill, None)


GOOD = (256, 64, 128, 64, 128, 64, 256, 64)


def but(at, value, base=GOOD):
    return strides(*(value if i == at else s for i, s in enumerate(base)))


def test_forward_refusals(lib):
    for kw in (dict(rows=-1), dict(Hq=-4), dict(Hkv=-1), dict(Hkv=0), dict(Hkv=3), dict(causal=2), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(fill=2), dict(fill=-1),
               dict(q=0), dict(k=0), dict(v=0), dict(o=0), dict(lse=0), dict(plan=0), dict(rows=1 << 29),
               dict(rows=1, Hq=65536, Hkv=1)):
        assert fwd(lib, **kw) == INVALID, kw
    for d in (0, 32, 96, 512):
        assert fwd(lib, d=d) == UNSUPPORTED
    for kw in (dict(q=P + 8), dict(k=P + 2), dict(v=P + 8), dict(o=P + 8), dict(lse=P + 2), dict(plan=P + 64)):
        assert fwd(lib, **kw) == MISALIGNED, kw
    for at in range(8):
        for bad in (0, -64, 1 << 38):
            assert fwd(lib, st=but(at, bad)) == INVALID, (at, bad)
        assert fwd(lib, st=but(at, GOOD[at] + 4)) == MISALIGNED
    for at, bad in ((6, 192), (6, 64), (7, 56), (7, 32)):  # rows of the output that overlap
        assert fwd(lib, st=but(at, bad)) == INVALID, (at, bad)
    for kw in (dict(rows=0), dict(Hq=0), dict(Hq=0, Hkv=0)):
        assert fwd(lib, q=0, k=0, v=0, o=0, lse=0, plan=0, **kw) == OK, kw


def bwd(lib, ptr=None, lse=P, st=None, gst=None, plan=P, rows=100, Hq=4, Hkv=2, d=64, causal=1, scale=0.125, fill=0, ws=P,
        size=1 << 30):
    p = dict.fromkeys(("q", "k", "v", "o", "do", "dq", "dk", "dv"), P)
    p.update(ptr or {})
    st = strides(*GOOD, 256, 64) if st is None else st
    gst = strides(*GOOD[:6]) if gst is None else gst
    return lib.fa_bwd_packed(p["q"], p["k"], p["v"], p["o"], lse, p["do"], st, p["dq"], p["dk"], p["dv"], gst, plan, rows,
                             Hq, Hkv, d, causal, scale, fill, ws, size, None)


def test_backward_refusals(lib):
    for kw in (dict(rows=-1), dict(Hkv=3), dict(causal=3), dict(scale=0.0), dict(fill=2), dict(lse=0), dict(plan=0),
               dict(rows=1 << 29)):
        assert bwd(lib, **kw) == INVALID, kw
    assert bwd(lib, d=96) == UNSUPPORTED
    for name in ("q", "k", "v", "o", "do", "dq", "dk", "dv"):
        assert bwd(lib, ptr={name: 0}) == INVALID, name
        assert bwd(lib, ptr={name: P + 8}) == MISALIGNED, name
    for at in range(10):
        assert bwd(lib, st=but(at, 0, GOOD + (256, 64))) == INVALID
        assert bwd(lib, st=but(at, 260, GOOD + (256, 64))) == MISALIGNED
    for at, bad in ((0, 192), (1, 32), (2, 64), (3, 0), (4, 64), (5, 56)):
        assert bwd(lib, gst=but(at, bad, GOOD[:6])) == INVALID, (at, bad)
    least = 256 + 2 * 1792  # 4 * 100 * 4 = 1600 bytes, rounded up
    assert bwd(lib, ws=0) == WORKSPACE and bwd(lib, size=least - 1) == WORKSPACE
    assert bwd(lib, ws=P + 128) == MISALIGNED
    for kw in (dict(rows=0), dict(Hq=0, Hkv=0)):
        assert bwd(lib, ptr=dict.fromkeys(("q", "k", "v", "o", "do", "dq", "dk", "dv"), 0), lse=0, plan=0, ws=0, size=0,
                   **kw) == OK


def test_backward_workspace_size(lib):
    size = lib.fa_bwd_packed_workspace_size
    assert size(0, 4, 2, 64) == 0 and size(100, 4, 3, 64) == 0 and size(100, 4, 2, 96) == 0
    fixed = 256 + 2 * 1792
    assert size(100, 4, 4, 64) == fixed and size(100, 4, 2, 256) == fixed  # groups of one, and d = 256: no split
    assert size(100, 4, 2, 64) == fixed + 2 * 100 * 2 * 64 * 8
    # the partial sums of long batches stay bounded
    assert size(1 << 20, 64, 8, 128) <= 256 + 2 * 4 * (1 << 20) * 64 + (512 << 20)


def axes_fwd(lib, axes=bytes(32), n=1, positions=P, rot=64, rows=500, cos=P, B=2, N=8):
    s = strides(3584, 64, 448, 3584, 64, 448, 3584, 64, 448)
    return lib.fa_norm_rope_axes_fwd(P, P, P, s, None, None, 0, cos, cos, rows, positions, axes, n, P, P, P, B, 4, 1, N, 64,
                                     rot, 0, 1e-6, None)


def test_axes_refusals(lib):
    for kw in (dict(n=0), dict(n=5), dict(n=-1), dict(axes=None), dict(positions=0), dict(axes=bytes([1] * 32)),
               dict(axes=bytes([0] * 31 + [2]), n=2), dict(axes=bytes([255] * 32), n=4), dict(cos=0), dict(rows=0)):
        assert axes_fwd(lib, **kw) == INVALID, kw
    assert axes_fwd(lib, positions=P + 2) == MISALIGNED
    for kw in (dict(B=0), dict(N=0)):
        assert axes_fwd(lib, axes=None, n=0, positions=0, cos=0, rows=0, **kw) == OK


def test_axes_backward_has_the_checks_of_the_forward(lib):
    s = strides(3584, 64, 448, 3584, 64, 448, 3584, 64, 448)

    def call(axes=bytes(32), n=1, positions=P):
        return lib.fa_norm_rope_axes_bwd(P, P, P, P, P, s, None, None, 0, P, P, 500, positions, axes, n, P, P, P, s, None,
                                         None, 2, 4, 1, 8, 64, 64, 0, 1e-6, None, 0, None)

    for kw in (dict(n=0), dict(n=5), dict(axes=None), dict(positions=0), dict(axes=bytes([1] * 32))):
        assert call(**kw) == INVALID, kw
    assert call(positions=P + 1) == MISALIGNED


def test_plan_sizes_beyond_32_bits(lib):
    size, most = lib.fa_packed_plan_size, 2**31 - 1
    fits = 2**30 - 2**24  # 2 B + rows / 128 + rows / 256 just below 2^31 at B = rows
    for B, rows in ((most, most), (1 << 30, most), (most, 2**31 - 2**23)):
        assert size(B, rows) == 0, (B, rows)
        assert plan(lib, B=B, rows=rows, size=1 << 62) == INVALID, (B, rows)
    for B, rows in ((fits, fits), (1, most), (most, 1000)):
        assert size(B, rows) == 256 + 16 * (rows // 128 + rows // 256 + 2 * min(B, rows))
        assert plan(lib, B=B, rows=rows, size=size(B, rows) - 1) == WORKSPACE, (B, rows)
