"""CPU tests of the paged calls' host checks: bad arguments are refused with the
documented status before anything is launched, and the binding refuses tensors
of the wrong type."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
GOOD, ODD8, ODD4, ODD2 = P(4096), P(4096 + 8), P(4096 + 4), P(4096 + 2)
NULL, SHAPE, ALIGN, RANGE, WS = -1, -2, -3, -4, -5


@pytest.fixture(scope="module")
def B():
    from sparse_attention_fp4_kv_b200 import build
    build.build()
    from sparse_attention_fp4_kv_b200 import binding
    return binding


def call(B, name, good, /, **change):
    args = dict(good)
    args.update(change)
    return getattr(B.lib, name)(*args.values())


ROPE = dict(x=GOOD, out=P(1 << 20), dtype=0, pos=GOOD, freq=GOOD, T=4, H=2, D=64, start=0, rot=64, layout=0, inverse=0,
            gain=1.0, xt=128, xh=64, ot=128, oh=64, stream=None)


@pytest.mark.parametrize("status,change", [
    (NULL, dict(x=None)), (NULL, dict(out=None)), (NULL, dict(pos=None)), (NULL, dict(freq=None)),
    (RANGE, dict(dtype=2)), (RANGE, dict(layout=2)), (SHAPE, dict(T=-1)), (SHAPE, dict(H=0)), (SHAPE, dict(rot=63)),
    (SHAPE, dict(rot=0)), (SHAPE, dict(rot=66)), (SHAPE, dict(start=2)), (SHAPE, dict(start=-2, rot=2)),
    (SHAPE, dict(D=1 << 17)), (SHAPE, dict(xt=-1)), (SHAPE, dict(xh=63)), (SHAPE, dict(oh=0)), (SHAPE, dict(ot=63)),
    (SHAPE, dict(ot=0)), (SHAPE, dict(ot=70, oh=72)), (SHAPE, dict(out=GOOD, xt=256)), (ALIGN, dict(x=P(4097))),
    (ALIGN, dict(out=ODD2, dtype=1)), (0, dict(T=0)), (0, dict(T=0, out=GOOD)), (SHAPE, dict(D=2048, rot=1026, xt=4096, xh=2048, ot=4096, oh=2048))])
def test_rope_refusals(B, status, change):
    assert call(B, "csa2_rope", ROPE, **change) == status


def test_rope_freqs_refusals(B):
    f = B.lib.csa2_rope_freqs
    assert f(64, 1e4, 0, 1.0, 0, 32.0, 1.0, None, None) == NULL
    assert f(63, 1e4, 0, 1.0, 0, 32.0, 1.0, GOOD, None) == SHAPE
    assert f(64, 1.0, 0, 1.0, 0, 32.0, 1.0, GOOD, None) == RANGE
    assert f(64, 1e4, 3, 1.0, 0, 32.0, 1.0, GOOD, None) == RANGE
    assert f(64, 1e4, 1, 0.5, 0, 32.0, 1.0, GOOD, None) == RANGE
    assert f(64, float("nan"), 0, 1.0, 0, 32.0, 1.0, GOOD, None) == RANGE
    assert f(64, 1e4, 2, 4.0, 0, 32.0, 1.0, GOOD, None) == RANGE
    assert f(64, 1e4, 2, 4.0, 4096, 1.0, 32.0, GOOD, None) == RANGE
    assert f(64, 1e4, 2, 4.0, 4096, 1.0, 0.0, GOOD, None) == RANGE


APPEND = dict(kv=GOOD, B=2, n=3, C=512, start=GOOD, valid=None, table=GOOD, M=4, page=16, N=100, fp4=GOOD, sf=GOOD, stream=None)
GATHER = dict(fp4=GOOD, sf=GOOD, table=GOOD, M=4, page=16, N=100, start=GOOD, valid=None, B=2, n=3, C=512, out=GOOD, stream=None)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("status,change", [
    (NULL, dict(start=None)), (NULL, dict(table=None)), (NULL, dict(fp4=None)), (NULL, dict(sf=None)),
    (SHAPE, dict(B=-1)), (SHAPE, dict(n=-1)), (SHAPE, dict(C=40)), (SHAPE, dict(C=0)), (SHAPE, dict(C=8224)),
    (SHAPE, dict(M=0)), (SHAPE, dict(page=0)), (SHAPE, dict(N=0)), (SHAPE, dict(page=1 << 30, M=1 << 12)),
    (SHAPE, dict(M=(1 << 30) + 1, page=1)), (SHAPE, dict(N=(1 << 30) + 1, page=1)),
    (SHAPE, dict(page=1 << 30, N=1 << 12)), (ALIGN, dict(fp4=ODD4)), (0, dict(B=0)), (0, dict(n=0))])
def test_append_and_gather_refusals(B, mx, status, change):
    fmt = "mxfp4" if mx else "fp4"
    assert call(B, "csa2_paged_kv_append_" + fmt, APPEND, **change) == status
    assert call(B, "csa2_paged_kv_gather_" + fmt, GATHER, **change) == status
    assert call(B, "csa2_paged_kv_append_" + fmt, APPEND, kv=None) == NULL
    assert call(B, "csa2_paged_kv_append_" + fmt, APPEND, kv=ODD8) == ALIGN
    assert call(B, "csa2_paged_kv_gather_" + fmt, GATHER, out=ODD8) == ALIGN


def test_page_call_refusals(B):
    need = B.pages_workspace_size(100, 5)
    assert need >= 4 * (3 * 100 + 5) and B.pages_workspace_size(0, 1) == 0 and B.pages_workspace_size(4, -1) == 0
    ext = dict(table=GOOD, S=5, M=4, ref=GOOD, N=100, page=16, want=GOOD, failed=GOOD, ws=GOOD, wsb=need, stream=None)
    for k in ("table", "ref", "want", "failed"):
        assert call(B, "csa2_pages_extend", ext, **{k: None}) == NULL
    fork = dict(table=GOOD, S=9, M=4, ref=GOOD, N=100, page=16, len=GOOD, src=GOOD, dst=GOOD, F=5, pairs=GOOD, failed=GOOD,
                ws=GOOD, wsb=need, stream=None)
    for k in ("table", "ref", "len", "src", "dst", "pairs", "failed"):
        assert call(B, "csa2_pages_fork", fork, **{k: None}) == NULL
    assert call(B, "csa2_pages_fork", fork, F=-1) == SHAPE and call(B, "csa2_pages_fork", fork, F=65537) == SHAPE
    free = dict(table=GOOD, S=9, M=4, ref=GOOD, N=100, page=16, seq=GOOD, keep=None, F=5, stream=None)
    for k in ("table", "ref", "seq"):
        assert call(B, "csa2_pages_free", free, **{k: None}) == NULL
    assert call(B, "csa2_pages_free", free, F=-1) == SHAPE and call(B, "csa2_pages_free", free, F=0) == 0
    for name, good in (("csa2_pages_extend", ext), ("csa2_pages_fork", fork), ("csa2_pages_free", free)):
        for change in (dict(S=-1), dict(M=0), dict(N=0), dict(page=0), dict(page=1 << 30, N=1 << 12),
                       dict(M=(1 << 30) + 1, page=1), dict(N=(1 << 30) + 1, page=1)):
            assert call(B, name, good, **change) == SHAPE, (name, change)
    for name, good in (("csa2_pages_extend", ext), ("csa2_pages_fork", fork)):
        assert call(B, name, good, ws=None) == WS and call(B, name, good, wsb=need - 1) == WS
        assert call(B, name, good, ws=ODD8) == ALIGN


def test_copy_and_compact_refusals(B):
    bufs = (B.csa2_page_buf * 17)()
    for i in range(17):
        bufs[i] = B.csa2_page_buf(4096, 64)
    copy = dict(pairs=GOOD, F=3, bufs=bufs, n=2, N=10, stream=None)
    assert call(B, "csa2_pages_copy", copy, pairs=None) == NULL and call(B, "csa2_pages_copy", copy, bufs=None) == NULL
    for change in (dict(F=-1), dict(n=0), dict(n=17), dict(N=0)):
        assert call(B, "csa2_pages_copy", copy, **change) == SHAPE
    assert call(B, "csa2_pages_copy", copy, F=0) == 0
    need = B.pages_workspace_size(10)
    comp = dict(table=GOOD, S=3, M=4, ref=GOOD, N=10, bufs=bufs, n=2, tout=GOOD, rout=GOOD, live=GOOD, ws=GOOD, wsb=need, stream=None)
    for k in ("table", "ref", "bufs", "tout", "rout", "live"):
        assert call(B, "csa2_pages_compact", comp, **{k: None}) == NULL
    for change in (dict(S=-1), dict(M=0), dict(N=0), dict(n=-1), dict(n=17), dict(M=(1 << 30) + 1), dict(N=(1 << 30) + 1)):
        assert call(B, "csa2_pages_compact", comp, **change) == SHAPE
    assert call(B, "csa2_pages_compact", comp, ws=None) == WS and call(B, "csa2_pages_compact", comp, wsb=need - 4) == WS
    assert call(B, "csa2_pages_compact", comp, ws=ODD8) == ALIGN
    bufs[1] = B.csa2_page_buf(None, 64)
    assert call(B, "csa2_pages_copy", copy) == NULL and call(B, "csa2_pages_compact", comp) == NULL
    bufs[1] = B.csa2_page_buf(4096, 0)
    assert call(B, "csa2_pages_copy", copy) == SHAPE


@pytest.mark.parametrize("mx", [False, True])
def test_attention_refusals(B, mx):
    name = "csa2_paged_attn_decode" + ("_mxfp4" if mx else "")
    need = B.paged_attn_workspace_size(2, 64, 512)
    assert need > 0 and B.paged_attn_workspace_size(0, 64, 512) == 0
    good = dict(q=GOOD, fp4=GOOD, sf=GOOD, table=GOOD, M=4, page=16, N=100, len=GOOD, win=0, sink=0, B=2, H=64, C=512,
                scale=0.1, out=GOOD, lse=None, ws=GOOD, wsb=need, stream=None)
    for k in ("q", "fp4", "sf", "table", "len", "out"):
        assert call(B, name, good, **{k: None}) == NULL
    for change in (dict(B=-1), dict(H=0), dict(H=257), dict(C=0), dict(C=48), dict(C=544), dict(M=0), dict(page=0), dict(N=0),
                   dict(page=1 << 30, M=1 << 12), dict(page=1 << 16, M=1 << 15),
                   dict(page=1 << 16, M=1 << 14, B=32, H=256)):  # 2^31 tiles of 64 keys in all
        assert call(B, name, good, **change) == SHAPE, change
    assert call(B, name, good, win=-1) == RANGE and call(B, name, good, sink=-1) == RANGE
    assert call(B, name, good, q=ODD8) == ALIGN and call(B, name, good, fp4=ODD8) == ALIGN
    assert call(B, name, good, out=ODD4) == ALIGN
    assert call(B, name, good, ws=None) == WS and call(B, name, good, wsb=need - 1) == WS
    assert call(B, name, good, ws=ODD8) == ALIGN
    assert call(B, name, good, B=0) == 0
    if not mx:
        assert call(B, name, good, sf=ODD2) == ALIGN


def test_binding_refuses_wrong_tensors(B):
    x = torch.zeros((2, 1, 8), dtype=torch.float16)
    with pytest.raises(TypeError):
        B.csa2_rope(x, torch.zeros(2, dtype=torch.int64), torch.zeros(4, dtype=torch.float64), x)
    y = x.bfloat16()
    with pytest.raises(ValueError):  # on the CPU
        B.csa2_rope(y, torch.zeros(2, dtype=torch.int64), torch.zeros(4, dtype=torch.float64), y)
    with pytest.raises(TypeError):
        B.csa2_paged_kv_append_fp4(x, None, None, None, None)
    with pytest.raises(TypeError):
        B.csa2_pages_free(torch.zeros((2, 2), dtype=torch.int64), None, None, 4)
    with pytest.raises(TypeError):
        B.csa2_paged_attn_decode(x, None, None, None, None, None, 1.0)
