"""GPU tests of the paged FP4 cache: rotary positions, appending to pages and
reading back, page management, and attention of one new token over the pages,
each against a plain restatement (paged_cases.py) or the oracle."""
import math

import numpy as np
import pytest
import torch

import oracle
import paged_cases as ref
from gpu_cases import bf16_np

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def B():
    from sparse_attention_fp4_kv_b200 import binding
    return binding


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def i64(v):
    return torch.tensor(v, dtype=torch.int64, device=DEV)


# ----------------------------------------------------------------------------- rotary positions
def freqs(rot):
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)


def check_rope(out, want, bound):
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    bad = (out.double() - want).abs() > bound * (1 + half) + half * want.abs()
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}"


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,D,start,rot", [
    (1, 1, 2, 0, 2), (1, 64, 512, 448, 64), (7, 8, 128, 0, 128), (129, 3, 70, 3, 50), (33, 1, 512, 0, 64),
    (5, 2, 1100, 38, 1024), (2, 1, 4096, 96, 16), (300, 5, 192, 128, 64), (3, 300, 64, 0, 32), (40, 2, 72, 8, 16)])
def test_rope_against_64_bits(B, T, H, D, start, rot, dtype, interleaved):
    g = gen(T * 7 + D)
    x = torch.randn((T, H, D), generator=g, device=DEV).to(dtype)
    pos = torch.randint(-5, 1 << 20, (T,), generator=g, device=DEV)
    pos[0] = (1 << 33) + 12345
    f = freqs(rot)
    for inverse, gain in ((False, 1.0), (True, 1.25)):
        out = torch.full_like(x, float("nan"))
        B.csa2_rope(x, pos, f, out, rot_start=start, interleaved=interleaved, inverse=inverse, mscale=gain)
        want, bound = ref.rope(x, pos, f, start, interleaved, inverse, gain)
        check_rope(out, want, bound)
        rest = torch.ones(D, dtype=torch.bool, device=DEV)
        rest[start:start + rot] = False
        assert torch.equal(out[..., rest], x[..., rest])
        y = x.clone()
        B.csa2_rope(y, pos, f, y, rot_start=start, interleaved=interleaved, inverse=inverse, mscale=gain)
        assert torch.equal(y, out)


@pytest.mark.parametrize("offset,pad", [(0, 16), (8, 24), (1, 3)])
@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_on_strided_rows(B, offset, pad, interleaved):
    """Queries and a cache row inside one projection's output, rotated in place;
    heads outside tokens; a broadcast input."""
    T, H, D, rot = 19, 4, 64, 32
    g = gen(offset)
    buf = torch.randn((T, H * D + pad), generator=g, device=DEV).to(torch.bfloat16)
    before = buf.clone()
    x = buf[:, offset:offset + H * D].unflatten(1, (H, D))
    pos, f = torch.arange(T, device=DEV) * 999, freqs(rot)
    want, bound = ref.rope(x, pos, f, D - rot, interleaved, False, 1.0)
    B.csa2_rope(x, pos, f, x, rot_start=D - rot, interleaved=interleaved)
    check_rope(x, want, bound)
    assert torch.equal(buf[:, :offset], before[:, :offset])
    assert torch.equal(buf[:, offset + H * D:], before[:, offset + H * D:])
    # out with heads outermost
    src = before[:, offset:offset + H * D].unflatten(1, (H, D))
    out = torch.zeros((H, T, D), dtype=torch.bfloat16, device=DEV)
    B.csa2_rope(src, pos, f, out.transpose(0, 1), rot_start=D - rot, interleaved=interleaved)
    assert torch.equal(out.transpose(0, 1), x)
    # one row for every token (stride 0)
    one = src[:1].expand(T, H, D)
    out2 = torch.empty((T, H, D), dtype=torch.bfloat16, device=DEV)
    B.csa2_rope(one, pos, f, out2, rot_start=D - rot, interleaved=interleaved)
    want, bound = ref.rope(one, pos, f, D - rot, interleaved, False, 1.0)
    check_rope(out2, want, bound)


def test_rope_inverse_is_the_transposed_map_and_the_gradient(B):
    T, H, D, rot = 6, 3, 96, 64
    g = gen(3)
    x, y = (torch.randn((T, H, D), generator=g, device=DEV) for _ in range(2))
    pos, f = torch.randint(0, 1 << 20, (T,), generator=g, device=DEV), freqs(rot)

    def fwd(v, inverse=False):
        out = torch.empty_like(v)
        B.csa2_rope(v, pos, f, out, rot_start=8, interleaved=False, inverse=inverse, mscale=1.5)
        return out.double()

    # <R x, y> = <x, R^T y>; both sides are off by at most 2^-19 of the norms' product
    lhs, rhs = (fwd(x) * y.double()).sum(), (x.double() * fwd(y, True)).sum()
    assert abs(lhs - rhs) <= 2.0 ** -18 * 1.5 * x.double().norm() * y.double().norm()
    # the gradient of <R x, y> by differences (the map is linear: any step serves)
    e = torch.zeros_like(x)
    e[2, 1, 10] = 1.0
    diff = ((fwd(x + 4 * e) - fwd(x - 4 * e)) * y.double()).sum() / 8
    assert abs(diff - fwd(y, True)[2, 1, 10]) <= 2.0 ** -18 * 1.5 * (x.double().norm() + 8) * y[2, 1].double().norm()


def test_rope_back_and_forth(B):
    x = torch.randn((50, 2, 64), generator=gen(1), device=DEV)
    pos, f = torch.arange(50, device=DEV) * 20011, freqs(64)
    y, z = torch.empty_like(x), torch.empty_like(x)
    B.csa2_rope(x, pos, f, y)
    B.csa2_rope(y, pos, f, z, inverse=True)
    pair = x.double().unflatten(-1, (-1, 2)).abs().sum(-1, keepdim=True).expand(-1, -1, -1, 2).flatten(-2)
    assert ((z.double() - x.double()).abs() <= 4 * 2.0 ** -20 * pair).all()


@pytest.mark.parametrize("rot", [2, 64, 130])
def test_rope_frequency_tables(B, rot):
    i = np.arange(rot // 2)
    plain = 10000.0 ** (-2 * i / rot)

    def table(**kw):
        t = torch.empty(rot // 2, dtype=torch.float64, device=DEV)
        B.csa2_rope_freqs(t, **kw)
        return t.cpu().numpy()

    close = dict(rtol=1e-14, atol=0)  # pow is off by a few fp64 steps at most
    np.testing.assert_allclose(table(), plain, **close)
    np.testing.assert_allclose(table(scaling=B.ROPE_LINEAR, factor=8.0), plain / 8, **close)
    turns = lambda n: rot * math.log(65536 / (n * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
    lo, hi = max(0, math.floor(turns(32))), min(rot - 1, math.ceil(turns(1)))
    r = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
    np.testing.assert_allclose(table(scaling=B.ROPE_YARN, factor=16.0, orig_ctx=65536),
                               plain * (1 - r) + plain / 16 * r, rtol=1e-13, atol=0)


# ----------------------------------------------------------------------------- append and read back
def pool_of(n_seq, n_tok, page, seed, spare=3):
    """Page tables for n_seq sequences of n_tok positions on shuffled pages."""
    m = -(-n_tok // page)
    n_pages = n_seq * m + spare
    perm = torch.randperm(n_pages, generator=gen(seed), device=DEV)[:n_seq * m]
    return perm.to(torch.int32).view(n_seq, m).contiguous(), n_pages


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("Bn,n,C,page,ragged", [
    (1, 1, 32, 1, False), (3, 1, 512, 64, False), (4, 37, 128, 16, True), (2, 130, 96, 17, True),
    (1, 300, 512, 33, False), (5, 9, 8192, 4, True)])
def test_append_and_gather_match_the_oracle(B, Bn, n, C, page, ragged, mx):
    g = gen(n + C)
    x = torch.randn((Bn, n, C), generator=g, device=DEV)
    x[..., ::7] *= 30
    x[0, 0] = 0
    x = x.to(torch.bfloat16)
    start = torch.randint(0, 50, (Bn,), generator=g, device=DEV)
    table, n_pages = pool_of(Bn, 50 + n, page, C)
    group = 32 if mx else 16
    fp4 = torch.full((n_pages, page, C // 2), 0xAB, dtype=torch.uint8, device=DEV)
    sf = torch.full((n_pages, page, C // group), 0xCD, dtype=torch.uint8, device=DEV)
    valid = torch.randint(0, n + 1, (Bn,), generator=g, device=DEV, dtype=torch.int32) if ragged else None
    B.csa2_paged_kv_append_fp4(x, start, table, fp4, sf, n_valid=valid, mx=mx)
    out = torch.full((Bn, n, C), -7.0, dtype=torch.bfloat16, device=DEV)
    B.csa2_paged_kv_gather(fp4, sf, table, start, out, n_valid=valid, mx=mx)
    quant, deq = (oracle.mxfp4_quantize, oracle.mxfp4_dequantize) if mx else (oracle.fp4_quantize, oracle.fp4_dequantize)
    codes, scales = quant(bf16_np(x))
    want4 = np.full((n_pages * page, C // 2), 0xAB, np.uint8)
    want_sf = np.full((n_pages * page, C // group), 0xCD, np.uint8)
    want_out = np.full((Bn, n, C), -7.0)
    t, st = table.cpu().numpy(), start.cpu().numpy()
    for b in range(Bn):
        for i in range(n if valid is None else int(valid[b])):
            p = int(st[b]) + i
            row = t[b, p // page] * page + p % page
            want4[row], want_sf[row] = codes[b, i], scales[b, i]
            want_out[b, i] = deq(codes[b, i][None], scales[b, i][None])[0]
    assert np.array_equal(fp4.cpu().numpy().reshape(want4.shape), want4)
    assert np.array_equal(sf.cpu().numpy().reshape(want_sf.shape), want_sf)
    assert np.array_equal(out.float().cpu().numpy().astype(np.float64), want_out)


@pytest.mark.parametrize("mx", [False, True])
def test_append_equals_the_contiguous_append_on_any_bits(B, mx):
    """Every bf16 pattern, infinities and NaN among them: the same bytes as
    csa2_kv_append_fp4 writes."""
    bits = torch.arange(1 << 16, device=DEV, dtype=torch.int32)
    bits = bits[torch.randperm(1 << 16, generator=gen(9), device=DEV)]
    x = bits.to(torch.int16).view(torch.bfloat16).view(1, 128, 512).contiguous()
    zero = i64([0])
    group = 32 if mx else 16
    a4, asf = (torch.zeros((1, 128, k), dtype=torch.uint8, device=DEV) for k in (256, 512 // group))
    b4, bsf = (torch.zeros((8, 16, k), dtype=torch.uint8, device=DEV) for k in (256, 512 // group))
    B.csa2_kv_append_fp4(x, zero, a4, asf, mx=mx)
    B.csa2_paged_kv_append_fp4(x, zero, torch.arange(8, device=DEV, dtype=torch.int32)[None], b4, bsf, mx=mx)
    assert torch.equal(a4.view(-1), b4.view(-1)) and torch.equal(asf.view(-1), bsf.view(-1))


def test_append_codes_of_every_value_under_every_scale(B):
    """The FP4 append takes its codes from products, not quotients: every bf16 value of
    up to six times the scale, for each of the 126 scales, gives the oracle's codes (IEEE
    division)."""
    every = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    scales = ref.scale_table(False, "cpu")[1:127]
    groups = []
    for s in scales:
        x = every[every.double().abs() <= 6 * s]  # NaN is not
        x = torch.cat([x, x[:-x.numel() % 15]]).view(-1, 15)
        groups.append(torch.cat([torch.full((x.shape[0], 1), float(6 * s), dtype=torch.bfloat16), x], 1))
        assert float(groups[-1][0, 0]) == float(6 * s)
    x = torch.cat(groups)
    x = torch.cat([x, x[:-x.shape[0] % 32]]).view(1, -1, 512).contiguous().to(DEV)
    n = x.shape[1]
    a4, asf = (torch.zeros((1, n, k), dtype=torch.uint8, device=DEV) for k in (256, 32))
    b4, bsf = (torch.zeros((n, 1, k), dtype=torch.uint8, device=DEV) for k in (256, 32))
    B.csa2_kv_append_fp4(x, i64([0]), a4, asf)
    B.csa2_paged_kv_append_fp4(x, i64([0]), torch.arange(n, device=DEV, dtype=torch.int32)[None], b4, bsf)
    codes, sf = oracle.fp4_quantize(bf16_np(x))
    assert set(np.unique(sf)) == set(range(1, 127))
    for got4, got_sf in ((a4, asf), (b4, bsf)):
        assert np.array_equal(got4.cpu().numpy().reshape(codes.shape), codes)
        assert np.array_equal(got_sf.cpu().numpy().reshape(sf.shape), sf)


@pytest.mark.parametrize("mx", [False, True])
def test_large_padded_batches(B, mx):
    """Chunks that are mostly padding, large enough for a CTA to take several of its
    sequence's pieces: the same bytes as one unpadded call per sequence."""
    Bn, n, C, page = 3, 40000, 512, 33
    valid = [39993, 0, 257]
    x = torch.randn((Bn, n, C), generator=gen(n), device=DEV).to(torch.bfloat16)
    start = i64([5, 0, 70])
    table, n_pages = pool_of(Bn, n + 70, page, 3)
    group = 32 if mx else 16
    got, want = ([torch.full((n_pages, page, k), 0xAB, dtype=torch.uint8, device=DEV) for k in (C // 2, C // group)]
                 for _ in range(2))
    B.csa2_paged_kv_append_fp4(x, start, table, *got, n_valid=i32(valid), mx=mx)
    out = torch.full((Bn, n, C), -7.0, dtype=torch.bfloat16, device=DEV)
    B.csa2_paged_kv_gather(*got, table, start, out, n_valid=i32(valid), mx=mx)
    for b, v in enumerate(valid):
        row = x[b:b + 1, :v].contiguous()
        B.csa2_paged_kv_append_fp4(row, start[b:b + 1], table[b:b + 1], *want, mx=mx)
        B.csa2_paged_kv_gather(*want, table[b:b + 1], start[b:b + 1], row, mx=mx)
        assert torch.equal(out[b, :v], row[0]) and bool((out[b, v:] == -7.0).all())
    assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_rows_without_a_page_are_skipped(B):
    page, C = 8, 64
    table = i32([[2, -1, 99, 0]])  # no page, a page outside the pool
    x = torch.ones((1, 40, C), dtype=torch.bfloat16, device=DEV)
    fp4 = torch.zeros((4, page, C // 2), dtype=torch.uint8, device=DEV)
    sf = torch.zeros((4, page, C // 16), dtype=torch.uint8, device=DEV)
    B.csa2_paged_kv_append_fp4(x, i64([-3]), table, fp4, sf)  # positions -3 .. 36; the table ends at 32
    got = (sf != 0).any(-1)
    want = torch.zeros((4, page), dtype=torch.bool, device=DEV)
    want[2] = want[0] = True
    assert torch.equal(got, want)
    out = torch.full_like(x, 5.0)
    B.csa2_paged_kv_gather(fp4, sf, table, i64([-3]), out)
    pos = torch.arange(-3, 37, device=DEV)
    here = ((pos >= 0) & (pos < 8)) | ((pos >= 24) & (pos < 32))
    # a row of ones is held as 6 * E4M3(1 / 6) = 6 * 11 / 64
    assert torch.equal(out[0, :, 0].float(), torch.where(here, 1.03125, 5.0))
    # far beyond the table, 64-bit positions
    B.csa2_paged_kv_append_fp4(x, i64([1 << 40]), table, fp4, sf)
    B.csa2_paged_kv_gather(fp4, sf, table, i64([(1 << 62)]), out)
    assert torch.equal((sf != 0).any(-1), want)


# ----------------------------------------------------------------------------- page management
def live_pool(S, M, N, page, seed, shared=True):
    """Random consistent tables: some pages shared, some rows empty."""
    r = np.random.RandomState(seed)
    table = np.full((S, M), -1, np.int32)
    refc = np.zeros(N, np.int32)
    lens = np.zeros(S, np.int64)
    free = list(r.permutation(N))
    for s in range(S - S // 3):
        lens[s] = r.randint(0, M * page + 1)
        for e in range(-(-int(lens[s]) // page)):
            if shared and s and r.rand() < 0.3 and table[s - 1, e] >= 0:
                table[s, e] = table[s - 1, e]
            elif free:
                table[s, e] = free.pop()
            if table[s, e] >= 0:
                refc[table[s, e]] += 1
    return i32(table), i32(refc), i64(lens)


def same(pool, table, refc):
    assert table.cpu().tolist() == pool.table
    assert refc.cpu().tolist() == pool.ref


@pytest.mark.parametrize("S,M,N,page", [(1, 1, 1, 1), (5, 7, 40, 16), (40, 33, 4095, 8), (64, 100, 4097, 3),
                                        (70, 600, 20000, 64), (3, 2000, 12288, 1)])
def test_extend(B, S, M, N, page):
    table, refc, lens = live_pool(S, M, N, page, N)
    want = lens + torch.randint(-20, M * page, (S,), generator=gen(S), device=DEV)
    want[0] = M * page + 5
    pool = ref.Pool(table, refc, page)
    failed = torch.full((1,), 77, dtype=torch.int32, device=DEV)
    B.csa2_pages_extend(table, refc, want, page, failed)
    assert int(failed) == pool.extend(want.tolist())
    same(pool, table, refc)


@pytest.mark.parametrize("S,lacking", [(200, (1 << 23) + 1), (258, (1 << 23) + 1)])
def test_extend_of_very_many_entries(B, S, lacking):
    """Up to more than 2^31 entries without a page: the first take what there is,
    nothing else is written, and the count of the others stops at 2^31 - 1."""
    M, N, page = lacking + 3, 5, 7
    table = torch.full((S, M), -1, dtype=torch.int32, device=DEV)
    table[2, 1] = 4
    refc, want, failed = i32([0, 0, 0, 0, 1]), i64([lacking * page - 2] * S), i32([-9])
    want[0] = 2 * page
    B.csa2_pages_extend(table, refc, want, page, failed)
    # lacking: two in the first row, all but one in the third; four pages were free
    assert int(failed) == min(2 ** 31 - 1, 2 + (S - 1) * lacking - 1 - 4)
    assert refc.tolist() == [1] * N
    assert table[0, :3].tolist() == [0, 1, -1] and table[1, :3].tolist() == [2, 3, -1] and table[2, :3].tolist() == [-1, 4, -1]
    table[0, :2] = table[1, :2] = table[2, 1] = -1
    assert int(table.max()) == int(table.min()) == -1


@pytest.mark.parametrize("S,M,N,page,F", [(2, 1, 3, 1, 1), (9, 7, 60, 16, 3), (90, 33, 4096, 8, 30),
                                          (200, 40, 9000, 7, 66), (60, 2100, 16385, 64, 20)])
def test_fork_and_free(B, S, M, N, page, F):
    table, refc, lens = live_pool(S, M, N, page, N + F)
    r = np.random.RandomState(F)
    src = r.randint(0, max(1, S - S // 3), F)
    dst = r.permutation(np.arange(S - S // 3, S) if S >= 3 else [1])[:F]
    src = src[:len(dst)]
    pool = ref.Pool(table, refc, page, lens)
    pairs = torch.full((len(src), 2), 5, dtype=torch.int32, device=DEV)
    failed = i32([9])
    B.csa2_pages_fork(table, refc, lens, i32(src), i32(dst), page, pairs, failed)
    want_pairs, want_failed = pool.fork(src.tolist(), dst.tolist())
    assert pairs.tolist() == [list(p) for p in want_pairs] and int(failed) == want_failed
    assert lens.tolist() == pool.len
    same(pool, table, refc)
    # the sources leave, some listed twice, one cut short instead, one no sequence
    seq = np.concatenate([src, src[:1], [S, -1]]).astype(np.int32)
    B.csa2_pages_free(table, refc, i32(seq), page)
    pool.free(seq.tolist())
    same(pool, table, refc)
    keep = torch.randint(-3, M * page + 9, (len(dst),), generator=gen(F), device=DEV)
    B.csa2_pages_free(table, refc, i32(dst), page, keep_len=keep)
    pool.free(dst.tolist(), keep.tolist())
    same(pool, table, refc)


def test_fork_refusals_and_exhaustion(B):
    page, M, N = 4, 3, 8
    table = i32([[0, 1, 2], [3, 4, -1], [-1] * 3, [-1] * 3, [-1] * 3, [-1] * 3, [-1] * 3])
    refc = i32([1, 1, 1, 1, 1, 0, 0, 0])
    lens = i64([10, 6, 0, 0, 0, 0, 0])
    # to itself, onto a source (twice), out of range (twice), onto an earlier dst
    # (twice: that the earlier fork was refused does not matter), then three that
    # take the three free pages
    src = [0, 0, 0, 7, 0, 0, 0, 1, 1, 1]
    dst = [0, 1, 1, 2, -1, 2, 2, 3, 4, 5]
    pool = ref.Pool(table, refc, page, lens)
    pairs, failed = torch.zeros((10, 2), dtype=torch.int32, device=DEV), i32([0])
    B.csa2_pages_fork(table, refc, lens, i32(src), i32(dst), page, pairs, failed)
    want_pairs, want_failed = pool.fork(src, dst)
    assert want_failed == 7 and pairs.tolist() == [list(p) for p in want_pairs] and int(failed) == 7
    assert lens.tolist() == pool.len and (refc > 0).all()
    same(pool, table, refc)
    # no page left: the whole pages alone
    B.csa2_pages_fork(table, refc, lens, i32([1]), i32([6]), page, pairs[:1], failed)
    want_pairs, want_failed = pool.fork([1], [6])
    assert want_failed == int(failed) == 1 and pairs[0].tolist() == list(want_pairs[0]) == [-1, -1]
    assert lens.tolist() == pool.len and int(lens[6]) == 4 and table[6].tolist() == [3, -1, -1]
    same(pool, table, refc)
    # nothing to do
    B.csa2_pages_fork(table, refc, lens, i32([]), i32([]), page, torch.empty((0, 2), dtype=torch.int32, device=DEV), failed)
    assert int(failed) == 0
    same(pool, table, refc)


@pytest.mark.parametrize("shapes", [[(3, 5)], [(16,), (4, 4)], [(64, 288), (64,), (1,)], [(33, 257), (33, 3), (7,), (9000,)]])
def test_copy_any_page_size(B, shapes):
    N, g = 40, gen(len(shapes))
    dtypes = [torch.uint8, torch.float32, torch.int8, torch.int16]
    bufs = [torch.randint(0, 100, (N,) + s, generator=g, device=DEV).to(dtypes[i]) for i, s in enumerate(shapes)]
    want = [b.clone() for b in bufs]
    perm = torch.randperm(N, generator=g, device=DEV).tolist()
    pairs = [(perm[2 * i], perm[2 * i + 1]) for i in range(15)] + [(-1, -1), (-1, perm[39]), (N, perm[38]), (perm[37], N)]
    for a, b in pairs:
        if 0 <= a < N and 0 <= b < N:
            for w in want:
                w[b] = w[a]
    B.csa2_pages_copy(i32(pairs), bufs)
    for b, w in zip(bufs, want):
        assert torch.equal(b, w)


def test_copy_from_unaligned_bases(B):
    N, g = 12, gen(4)
    for off, width in ((1, 48), (4, 48), (16, 48), (2, 6)):
        flat = torch.randint(0, 256, (off + N * width + 64,), generator=g, device=DEV, dtype=torch.uint8)
        buf, before = flat[off:off + N * width].view(N, width), flat.clone()
        B.csa2_pages_copy(i32([[3, 5], [0, 11]]), [buf])
        want = before.clone()
        w = want[off:off + N * width].view(N, width)
        w[5], w[11] = w[3].clone(), w[0].clone()
        assert torch.equal(flat, want)


@pytest.mark.parametrize("N,live", [(1, 0), (1, 1), (50, 20), (50, 50), (4096, 1), (4097, 3000), (20000, 9000), (8192, 8191)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(B, N, live, in_place):
    r = np.random.RandomState(N + live)
    pages = r.permutation(N)[:live]
    refc = np.zeros(N, np.int32)
    refc[pages] = r.randint(1, 4, live)
    S, M = 7, max(2, -(-live // 6))
    flat = np.full(S * M, -1, np.int32)
    flat[:live] = pages
    flat[-1] = N + 3  # no page: stays as it is
    table, refc = i32(r.permutation(flat).reshape(S, M)), i32(refc)
    bufs = [torch.randint(0, 256, (N, 3, 48), generator=gen(N), device=DEV, dtype=torch.uint8),
            torch.rand((N, 5), generator=gen(N), device=DEV)]
    want = [b.clone() for b in bufs]
    pool = ref.Pool(table, refc, 1)
    L, moves = pool.compact()
    for a, b in moves.items():
        for w in want:
            w[b] = w[a]
    t_out, r_out = (table, refc) if in_place else (torch.full_like(table, 9), torch.full_like(refc, 9))
    n_live = i32([-1])
    B.csa2_pages_compact(table, refc, bufs, t_out, r_out, n_live)
    assert int(n_live) == L == live
    same(pool, t_out, r_out)
    for b, w in zip(bufs, want):
        assert torch.equal(b, w)
    # a second time there is nothing to move; without buffers the tables alone
    B.csa2_pages_compact(t_out, r_out, [], t_out, r_out, n_live)
    same(pool, t_out, r_out)


# ----------------------------------------------------------------------------- attention
def filled(n_pages, page, C, mx, seed):
    g = gen(seed)
    fp4 = torch.randint(0, 256, (n_pages, page, C // 2), generator=g, device=DEV, dtype=torch.uint8)
    lo, hi = (122, 130) if mx else (0x20, 0x40)
    sf = torch.randint(lo, hi, (n_pages, page, C // (32 if mx else 16)), generator=g, device=DEV, dtype=torch.uint8)
    return fp4, sf


def attend(B, q, fp4, sf, table, lens, scale=None, win=0, sink=0, mx=False, what="", **kw):
    scale = 1 / math.sqrt(q.shape[2]) if scale is None else scale
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device=DEV)
    B.csa2_paged_attn_decode(q, fp4, sf, table, lens, out, scale, n_win=win, n_sink=sink, lse=lse, mx=mx, **kw)
    want, want_lse, bound, lse_bound = ref.attend(q, fp4, sf, table, lens, scale, win, sink, mx)
    err = (out.double() - want).abs()
    assert (err <= bound).all(), f"{what}: worst {(err / bound).max():.2f} of the bound"
    none = want_lse == -math.inf
    assert torch.equal(lse == -math.inf, none), what
    assert ((lse.double() - want_lse)[~none].abs() <= lse_bound[~none]).all(), what
    assert B.device_status() == 0
    return out, lse


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("Hq,C,page", [(1, 32, 1), (8, 128, 64), (64, 512, 64), (23, 320, 17), (3, 96, 16), (65, 256, 128),
                                       (16, 64, 5), (40, 448, 33), (200, 192, 64), (128, 512, 256)])
def test_attention_lengths(B, Hq, C, page, mx):
    """Lengths around the tiles' and pages' ends, an empty sequence, a long one."""
    lens = [0, 1, 2, page, page + 1, 63, 64, 65, 127, 128, 129, 255, 257, 700, 3001]
    m = -(-max(lens) // page)
    table, n_pages = pool_of(len(lens), m * page, page, C)
    fp4, sf = filled(n_pages, page, C, mx, C + Hq)
    q = (2 * torch.randn((len(lens), Hq, C), generator=gen(Hq), device=DEV)).to(torch.bfloat16)
    attend(B, q, fp4, sf, table, i64(lens), mx=mx)


@pytest.mark.parametrize("Hq,C", [(64, 512), (8, 128), (17, 160)])
@pytest.mark.parametrize("win,sink", [(1, 0), (128, 4), (128, 0), (100, 300), (4096, 1), (5, 1 << 40), (1 << 40, 0), (300, 129)])
def test_attention_window_and_first_tokens(B, Hq, C, win, sink):
    lens = [0, 1, 5, 127, 128, 129, 132, 133, 400, 1000, 5000]
    page = 16
    table, n_pages = pool_of(len(lens), 5008, page, win & 0xFFFF)
    fp4, sf = filled(n_pages, page, C, False, C + sink % 1000)
    q = torch.randn((len(lens), Hq, C), generator=gen(win & 0xFFFF), device=DEV).to(torch.bfloat16)
    attend(B, q, fp4, sf, table, i64(lens), win=win, sink=sink)


@pytest.mark.parametrize("mx", [False, True])
def test_attention_skips_what_it_does_not_see(B, mx):
    """Positions without a page are no keys; the bytes of unseen slots (NaN scales
    among them) and of foreign pages do not reach the result."""
    C, page, Hq = 512, 16, 64
    lens = [300, 40, 16, 33]
    table, n_pages = pool_of(4, 304, page, 5)
    fp4, sf = filled(n_pages, page, C, mx, 5)
    table[0, 3] = -1
    table[0, 10:14] = n_pages
    table[1, :3] = -5          # no key left
    table[2, 1:] = 1 << 30     # behind its length
    q = torch.randn((4, Hq, C), generator=gen(2), device=DEV).to(torch.bfloat16)
    used = torch.zeros((n_pages, page), dtype=torch.bool, device=DEV)
    for b, n in enumerate(lens):
        for p in range(n):
            v = int(table[b, p // page])
            if 0 <= v < n_pages:
                used[v, p % page] = True
    clean = attend(B, q, fp4, sf, table, i64(lens), mx=mx)
    assert (clean[0][1] == 0).all() and (clean[1][1] == -math.inf).all()
    # lengths beyond the table, below zero (on bytes an append can write: the NaN
    # codes below are for slots that no query sees)
    attend(B, q, fp4, sf, table, i64([10 ** 12, -7, 16, 33]), mx=mx)
    sf[~used] = 0xFF
    fp4[~used] = 0xFF
    dirty = attend(B, q, fp4, sf, table, i64(lens), mx=mx)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("kind", ["rising", "falling", "spike", "equal", "cold", "zero", "huge"])
def test_attention_score_orders(B, kind, mx):
    """Running maxima that move at every tile, never, or once; scores far apart;
    equal scores; keys or queries of zero; queries of extreme size."""
    C, page, Hq, n = 128, 32, 24, 1500
    table, n_pages = pool_of(1, n, page, 8)
    fp4, sf = filled(n_pages, page, C, mx, 8)
    rows = table[0].long()[torch.arange(n, device=DEV) // page] * page + torch.arange(n, device=DEV) % page
    flat4, flats = fp4.flatten(0, 1), sf.flatten(0, 1)
    q = torch.randn((1, Hq, C), generator=gen(6), device=DEV)
    one = 127 if mx else 0x38
    if kind in ("rising", "falling"):
        # rows are all +0.5 x their scale, scales grow with the position
        flat4[rows] = 0x11
        steps = torch.linspace(0, 8 if mx else 40, n, device=DEV).to(torch.uint8)
        flats[rows] = ((118 if mx else 0x18) + (steps if kind == "rising" else steps.flip(0)))[:, None]
        q = q.abs()
    elif kind == "spike":
        flats[rows] = one - (3 if mx else 16)
        flat4[rows[777]] = 0x77
        flats[rows[777]] = one
        q = q.abs() * 3
    elif kind == "equal":
        flat4[rows], flats[rows] = flat4[rows[0]].clone(), flats[rows[0]].clone()
    elif kind == "cold":
        q = q * 1e-30
    elif kind == "zero":
        flat4[rows[::2]] = 0
        q[0, ::2] = 0
    else:
        q = q * torch.logspace(-38, 3, Hq, device=DEV)[None, :, None]
    attend(B, q.to(torch.bfloat16), fp4, sf, table, i64([n]), mx=mx, what=kind)


def test_attention_nan_query_stays_in_its_head(B):
    C, Hq, page = 512, 64, 64
    table, n_pages = pool_of(2, 640, page, 1)
    fp4, sf = filled(n_pages, page, C, False, 1)
    q = torch.randn((2, Hq, C), generator=gen(1), device=DEV).to(torch.bfloat16)
    lens = i64([600, 333])
    clean, clean_lse = attend(B, q, fp4, sf, table, lens)
    q[0, 5, 7] = float("nan")
    q[1, 60, 0] = float("inf")
    out, lse = torch.empty_like(q), torch.empty((2, Hq), device=DEV)
    B.csa2_paged_attn_decode(q, fp4, sf, table, lens, out, 1 / math.sqrt(C), lse=lse)
    keep = torch.ones((2, Hq), dtype=torch.bool, device=DEV)
    keep[0, 5] = keep[1, 60] = False
    assert torch.equal(out[keep], clean[keep]) and torch.equal(lse[keep], clean_lse[keep])
    assert out[0, 5].isnan().all() and out[1, 60].isnan().all()


def test_attention_scale_sign_and_zero(B):
    table, n_pages = pool_of(1, 500, 20, 3)
    fp4, sf = filled(n_pages, 20, 64, False, 3)
    q = torch.randn((1, 4, 64), generator=gen(3), device=DEV).to(torch.bfloat16)
    for scale in (0.0, -0.3, 2.0):
        attend(B, q, fp4, sf, table, i64([500]), scale=scale)


@pytest.mark.parametrize("Bn,Hq,C,page,ctx", [(1, 64, 512, 64, 70001), (3, 8, 128, 48, 30011), (150, 16, 64, 32, 300), (400, 64, 512, 16, 33),
                                               (1300, 80, 32, 16, 130)])
def test_attention_split_and_batched(B, Bn, Hq, C, page, ctx):
    """Long sequences cut over many CTAs; more sequences than CTAs."""
    r = np.random.RandomState(Bn)
    lens = [ctx] + [int(r.randint(0, ctx + 1)) for _ in range(Bn - 1)]
    table, n_pages = pool_of(Bn, ctx, page, Bn)
    fp4, sf = filled(n_pages, page, C, False, Bn)
    q = (1.5 * torch.randn((Bn, Hq, C), generator=gen(Bn), device=DEV)).to(torch.bfloat16)
    a = attend(B, q, fp4, sf, table, i64(lens))
    b = attend(B, q, fp4, sf, table, i64(lens))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def ctas():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("C,page", [(96, 33), (224, 64), (352, 17), (480, 5), (512, 64)])
@pytest.mark.parametrize("Hq", [11, 27, 50, 67])
def test_attention_of_many_tiles_a_cta(B, Hq, C, page, mx):
    """Every width of head groups and of rows in both formats, ten tiles and more to a
    CTA: long sequences whose shares go round the ring of tiles, and short ones, several
    to a CTA, between them."""
    r = np.random.RandomState(Hq + C)
    lens = [60001, 0, 1] + [int(v) for v in r.randint(0, 700, 60)] + [64, 65, 24000] + [int(v) for v in r.randint(0, 200, 30)]
    share = ref.shares([-(-n // 64) for n in lens for _ in range(-(-Hq // 64))], ctas())
    assert min(sum(b - a for _, a, b in own) for own in share) >= 10 and max(len(own) for own in share) >= 3
    need = [-(-n // page) for n in lens]
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=DEV)
    n_pages = sum(need) + 3
    perm = torch.randperm(n_pages, generator=gen(C), device=DEV).to(torch.int32)
    for b, k in enumerate(need):
        table[b, :k] = perm[sum(need[:b]):sum(need[:b]) + k]
    fp4, sf = filled(n_pages, page, C, mx, C + Hq)
    q = (1.5 * torch.randn((len(lens), Hq, C), generator=gen(Hq), device=DEV)).to(torch.bfloat16)
    a = attend(B, q, fp4, sf, table, i64(lens), mx=mx)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    B.csa2_paged_attn_decode(q, fp4, sf, table, i64(lens), out, 1 / math.sqrt(C), lse=lse, mx=mx)
    assert torch.equal(a[0], out) and torch.equal(a[1], lse)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("Hq,C", [(64, 512), (16, 512), (24, 128), (40, 320), (9, 224)])
@pytest.mark.parametrize("kind", ["rising", "falling", "saw", "spikes"])
def test_attention_references_move_within_a_share(B, kind, Hq, C, mx):
    """Scores that climb by more than 2^8 several times inside one CTA's share of a
    sequence, with one buffer of weights (64 heads of 512 channels) and with two. A
    rescale that is left out exceeds the bound on these scores (test_paged_cases.py)."""
    n, page, Bn = 704, 32, ctas() + 37
    q, codes, sf_rows, scale = ref.stepped(kind, n, Hq, C, mx, gen(Hq + C), DEV)
    x = (scale / math.log(2.0)) * (q[0].double() @ ref.dequant(codes, sf_rows, mx).T).cpu()
    moves = torch.zeros(Hq, dtype=torch.int64)
    for own in ref.shares([n // 64] * Bn, ctas()):
        for _, lo, hi in own:
            moves += ref.online(x[:, 64 * lo:64 * hi], torch.zeros((64 * (hi - lo), 1), dtype=torch.float64),
                                lambda o, l, f: (o, l))[2]
    assert int(moves.max()) == 0 if kind == "falling" else int(moves.min()) >= Bn
    table, n_pages = pool_of(Bn, n, page, C)
    fp4, sf = filled(n_pages, page, C, mx, C)
    i = torch.arange(n, device=DEV)
    rows = table.long()[:, i // page] * page + i % page
    fp4.flatten(0, 1)[rows], sf.flatten(0, 1)[rows] = codes, sf_rows
    attend(B, q.expand(Bn, Hq, C).contiguous(), fp4, sf, table, i64([n] * Bn), scale=scale, mx=mx, what=kind)


@pytest.mark.parametrize("Hq,C", [(64, 512), (8, 128), (17, 160), (23, 320)])
@pytest.mark.parametrize("win,sink", [(1, 0), (128, 4), (100, 300), (4096, 1), (5, 1 << 40), (300, 129)])
def test_attention_window_and_first_tokens_mx(B, Hq, C, win, sink):
    lens = [0, 1, 5, 127, 128, 129, 132, 133, 400, 1000, 5000]
    page = 16
    table, n_pages = pool_of(len(lens), 5008, page, win & 0xFFFF)
    fp4, sf = filled(n_pages, page, C, True, C + sink % 1000)
    q = torch.randn((len(lens), Hq, C), generator=gen(win & 0xFFFF), device=DEV).to(torch.bfloat16)
    attend(B, q, fp4, sf, table, i64(lens), win=win, sink=sink, mx=True)


@pytest.mark.parametrize("Hq,C", [(64, 512), (16, 256)])
def test_attention_nan_query_stays_in_its_head_mx(B, Hq, C):
    page = 64
    table, n_pages = pool_of(2, 640, page, 1)
    fp4, sf = filled(n_pages, page, C, True, 1)
    q = torch.randn((2, Hq, C), generator=gen(1), device=DEV).to(torch.bfloat16)
    lens = i64([600, 333])
    clean, clean_lse = attend(B, q, fp4, sf, table, lens, mx=True)
    q[0, 5, 7] = float("nan")
    q[1, Hq - 4, 0] = float("inf")
    out, lse = torch.empty_like(q), torch.empty((2, Hq), device=DEV)
    B.csa2_paged_attn_decode(q, fp4, sf, table, lens, out, 1 / math.sqrt(C), lse=lse, mx=True)
    keep = torch.ones((2, Hq), dtype=torch.bool, device=DEV)
    keep[0, 5] = keep[1, Hq - 4] = False
    assert torch.equal(out[keep], clean[keep]) and torch.equal(lse[keep], clean_lse[keep])
    assert out[0, 5].isnan().all() and out[1, Hq - 4].isnan().all()


@pytest.mark.parametrize("Bn,Hq,C,page,ctx", [(1, 64, 512, 64, 70001), (3, 8, 128, 48, 30011), (400, 64, 512, 16, 33),
                                               (1300, 80, 32, 16, 130)])
def test_attention_split_and_batched_mx(B, Bn, Hq, C, page, ctx):
    r = np.random.RandomState(Bn)
    lens = [ctx] + [int(r.randint(0, ctx + 1)) for _ in range(Bn - 1)]
    table, n_pages = pool_of(Bn, ctx, page, Bn)
    fp4, sf = filled(n_pages, page, C, True, Bn)
    q = (1.5 * torch.randn((Bn, Hq, C), generator=gen(Bn), device=DEV)).to(torch.bfloat16)
    a = attend(B, q, fp4, sf, table, i64(lens), mx=True)
    b = attend(B, q, fp4, sf, table, i64(lens), mx=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("mx", [False, True])
def test_two_calls_over_disjoint_keys_are_joined_by_their_lse(B, mx):
    """Each call sees every second page (a sequence among them whose second half is
    empty); out = sum_i exp(lse_i - lse) out_i with lse = ln sum_i exp(lse_i)."""
    C, Hq, page = 256, 24, 16
    lens, scale = [900, 33, 7, 2000], 0.05
    table, n_pages = pool_of(4, 2000, page, 9)
    fp4, sf = filled(n_pages, page, C, mx, 9)
    q = (2 * torch.randn((4, Hq, C), generator=gen(9), device=DEV)).to(torch.bfloat16)
    want, want_lse, _, _ = ref.attend(q, fp4, sf, table, lens, scale, mx=mx)
    parts = []
    for odd in (0, 1):
        half = table.clone()
        half[:, 1 - odd::2] = -1
        out, lse = attend(B, q, fp4, sf, half, i64(lens), scale=scale, mx=mx)
        exact, _, bound, lse_bound = ref.attend(q, fp4, sf, half, lens, scale, mx=mx)
        parts.append((out.double(), lse.double(), exact, bound, lse_bound))
    lse = torch.logsumexp(torch.stack([p[1] for p in parts]), 0)
    off = torch.stack([p[4] for p in parts]).amax(0)
    weight = [torch.exp(p[1] - lse)[..., None] for p in parts]
    joined = sum(w * p[0] for w, p in zip(weight, parts))
    # a part is off by its own bound, its weight by a factor of exp(+- 2 off); off is far below 1
    bound = sum(w * (p[3] + 3 * off[..., None] * (p[2].abs() + p[3])) for w, p in zip(weight, parts))
    assert float(off.max()) < 0.01
    assert ((joined - want).abs() <= bound * (1 + 4 * off[..., None]) + 1e-30).all()
    assert ((lse - want_lse).abs() <= off).all()


def test_offsets_past_32_bits(B):
    """A pool of over 4 GB of codes, a sequence on its last pages."""
    C, page = 512, 64
    n_pages = (1 << 32) // (page * C // 2) + 50
    fp4 = torch.zeros((n_pages, page, C // 2), dtype=torch.uint8, device=DEV)
    sf = torch.zeros((n_pages, page, C // 16), dtype=torch.uint8, device=DEV)
    table = torch.arange(n_pages - 40, n_pages, device=DEV, dtype=torch.int32).flip(0)[None].contiguous()
    x = torch.randn((1, 2500, C), generator=gen(4), device=DEV).to(torch.bfloat16)
    B.csa2_paged_kv_append_fp4(x, i64([60]), table, fp4, sf)
    out = torch.empty_like(x)
    B.csa2_paged_kv_gather(fp4, sf, table, i64([60]), out)
    codes, scales = oracle.fp4_quantize(bf16_np(x))
    assert np.array_equal(out[0].float().cpu().numpy().astype(np.float64), oracle.fp4_dequantize(codes[0], scales[0]))
    q = torch.randn((1, 64, C), generator=gen(5), device=DEV).to(torch.bfloat16)
    attend(B, q, fp4, sf, table, i64([2560]))
    pairs = i32([[n_pages - 1, 0]])
    B.csa2_pages_copy(pairs, [fp4, sf])
    assert torch.equal(fp4[0], fp4[n_pages - 1]) and torch.equal(sf[0], sf[n_pages - 1])


def test_calls_over_nothing(B):
    """Empty batches and lists are no-ops."""
    def empty(*shape, dtype=torch.int32):
        return torch.empty(shape, dtype=dtype, device=DEV)

    none = empty(0, dtype=torch.int64)
    bf = torch.bfloat16
    fp4, sf = filled(4, 8, 64, False, 1)
    table, refc, failed = i32([[1, 2]]), i32([0, 1, 1, 0]), i32([7])
    B.csa2_rope(empty(0, 2, 64, dtype=bf), none, freqs(64), empty(0, 2, 64, dtype=bf))
    B.csa2_paged_kv_append_fp4(empty(0, 3, 64, dtype=bf), none, empty(0, 2), fp4, sf)
    B.csa2_paged_kv_append_fp4(empty(1, 0, 64, dtype=bf), i64([3]), table, fp4, sf)
    B.csa2_paged_kv_gather(fp4, sf, empty(0, 2), none, empty(0, 3, 64, dtype=bf))
    B.csa2_pages_extend(empty(0, 2), refc, none, 8, failed)
    assert int(failed) == 0
    B.csa2_pages_free(table, refc, empty(0), 8)
    B.csa2_pages_copy(empty(0, 2), [fp4, sf])
    B.csa2_paged_attn_decode(empty(0, 4, 64, dtype=bf), fp4, sf, empty(0, 2), none, empty(0, 4, 64, dtype=bf), 1.0)
    assert table.tolist() == [[1, 2]] and refc.tolist() == [0, 1, 1, 0]


# ----------------------------------------------------------------------------- together
def test_a_serving_run(B):
    """Prompts are appended, forked into samples that continue on their own,
    some leave, the pool is compacted, and attention sees the same rows all
    along; queries and rows carry rotary positions, outputs are turned back."""
    C, Hq, page, S, M, N, rot = 512, 64, 16, 8, 12, 70, 64
    g = gen(12)
    table = torch.full((S, M), -1, dtype=torch.int32, device=DEV)
    refc = torch.zeros(N, dtype=torch.int32, device=DEV)
    fp4 = torch.zeros((N, page, C // 2), dtype=torch.uint8, device=DEV)
    sf = torch.zeros((N, page, C // 16), dtype=torch.uint8, device=DEV)
    keys = torch.zeros((N, page, 40), dtype=torch.int8, device=DEV)
    lens = i64([100, 37] + [0] * 6)
    failed, n_live, freq = i32([0]), i32([0]), torch.empty(rot // 2, dtype=torch.float64, device=DEV)
    B.csa2_rope_freqs(freq, scaling=B.ROPE_YARN, factor=4.0, orig_ctx=64)
    history = [torch.zeros((0, C), dtype=torch.bfloat16, device=DEV) for _ in range(S)]

    def append(n_new, valid, start):
        rows = torch.randn((S, n_new, C), generator=g, device=DEV).to(torch.bfloat16)
        pos = start[:, None] + torch.arange(n_new, device=DEV)
        turned = rows.clone()
        B.csa2_rope(turned.view(S * n_new, 1, C), pos.flatten(), freq, turned.view(S * n_new, 1, C), rot_start=C - rot)
        B.csa2_paged_kv_append_fp4(turned, start, table, fp4, sf, n_valid=valid)
        for s in range(S):
            history[s] = torch.cat([history[s], turned[s, :int(valid[s])]])

    def check():
        q = torch.randn((S, Hq, C), generator=g, device=DEV).to(torch.bfloat16)
        B.csa2_rope(q, lens - 1, freq, q, rot_start=C - rot)
        out, _ = attend(B, q, fp4, sf, table, lens)
        back = torch.empty((S, Hq, C), device=DEV)
        B.csa2_rope(out.float(), lens - 1, freq, back, rot_start=C - rot, inverse=True)
        for s in range(S):
            n = int(lens[s])
            assert history[s].shape[0] == n
            if n == 0:
                assert (back[s] == 0).all()
                continue
            codes, scales = oracle.fp4_quantize(bf16_np(history[s]))
            rows = torch.empty((1, n, C), dtype=torch.bfloat16, device=DEV)
            B.csa2_paged_kv_gather(fp4, sf, table[s:s + 1], i64([0]), rows)
            assert np.array_equal(rows[0].float().cpu().numpy().astype(np.float64), oracle.fp4_dequantize(codes, scales))

    B.csa2_pages_extend(table, refc, lens, page, failed)
    assert int(failed) == 0 and int((refc > 0).sum()) == 7 + 3
    append(100, lens.to(torch.int32), i64([0] * S))
    check()
    pairs = torch.empty((4, 2), dtype=torch.int32, device=DEV)
    B.csa2_pages_fork(table, refc, lens, i32([0, 1, 0, 1]), i32([2, 3, 4, 5]), page, pairs, failed)
    B.csa2_pages_copy(pairs, [fp4, sf, keys])
    assert int(failed) == 0 and lens.tolist() == [100, 37, 100, 37, 100, 37, 0, 0]
    for d, s in ((2, 0), (3, 1), (4, 0), (5, 1)):
        history[d] = history[s].clone()
    check()
    for _ in range(20):  # across a page's end
        valid = i32([1] * 6 + [0, 0])
        start = lens.clone()
        lens += valid
        B.csa2_pages_extend(table, refc, lens, page, failed)
        append(1, valid, start)
    assert int(failed) == 0
    check()
    B.csa2_pages_free(table, refc, i32([0, 3]), page)
    lens[0] = lens[3] = 0
    for s in (0, 3):
        history[s] = history[s][:0]
    before = int((refc > 0).sum())
    B.csa2_pages_compact(table, refc, [fp4, sf, keys], table, refc, n_live)
    assert int(n_live) == before and (refc[:before] > 0).all() and (refc[before:] == 0).all()
    check()


def test_graphs_and_streams(B):
    """Every call captured and replayed on another stream, twice over in two
    graphs with workspaces of their own; eager calls on a side stream."""
    C, Hq, page, S, M, N = 256, 16, 16, 6, 20, 90
    g = gen(20)
    x = torch.randn((S, 50, C), generator=g, device=DEV).to(torch.bfloat16)
    q = torch.randn((S, Hq, C), generator=g, device=DEV).to(torch.bfloat16)
    freq = freqs(64)

    def state():
        return dict(table=torch.full((S, M), -1, dtype=torch.int32, device=DEV),
                    ref=torch.zeros(N, dtype=torch.int32, device=DEV),
                    fp4=torch.zeros((N, page, C // 2), dtype=torch.uint8, device=DEV),
                    sf=torch.zeros((N, page, C // 16), dtype=torch.uint8, device=DEV),
                    len=i64([50, 33, 1, 0, 0, 0]), failed=i32([0]), live=i32([0]),
                    pairs=torch.empty((2, 2), dtype=torch.int32, device=DEV), src=i32([0, 1]), dst=i32([3, 4]),
                    all=i32(list(range(S))), zero=i64([0] * S), valid=i32([50, 33, 1, 0, 0, 0]), pos=i64([0] * S),
                    q=torch.empty_like(q), out=torch.empty_like(q), back=torch.empty_like(x),
                    ws=torch.empty(B.paged_attn_workspace_size(S, Hq, C), dtype=torch.uint8, device=DEV),
                    pws=torch.empty(B.pages_workspace_size(N, S), dtype=torch.uint8, device=DEV))

    def step(s, stream=None):
        B.csa2_pages_free(s["table"], s["ref"], s["all"], page, stream=stream)
        B.csa2_pages_extend(s["table"], s["ref"], s["len"], page, s["failed"], ws=s["pws"], stream=stream)
        B.csa2_paged_kv_append_fp4(x, s["zero"], s["table"], s["fp4"], s["sf"], n_valid=s["valid"], stream=stream)
        B.csa2_pages_free(s["table"], s["ref"], s["dst"], page, stream=stream)
        B.csa2_pages_fork(s["table"], s["ref"], s["len"], s["src"], s["dst"], page, s["pairs"], s["failed"], ws=s["pws"], stream=stream)
        B.csa2_pages_copy(s["pairs"], [s["fp4"], s["sf"]], stream=stream)
        B.csa2_pages_compact(s["table"], s["ref"], [s["fp4"], s["sf"]], s["table"], s["ref"], s["live"], ws=s["pws"], stream=stream)
        B.csa2_rope(q, s["pos"], freq, s["q"], stream=stream)
        B.csa2_paged_kv_gather(s["fp4"], s["sf"], s["table"], s["zero"], s["back"], n_valid=s["valid"], stream=stream)
        B.csa2_paged_attn_decode(s["q"], s["fp4"], s["sf"], s["table"], s["len"], s["out"], 0.07, ws=s["ws"], stream=stream)

    eager = state()
    step(eager)
    first = {k: v.clone() for k, v in eager.items()}
    step(eager)  # the lengths of the forks are now their sources'
    torch.cuda.synchronize()
    keys = ("table", "ref", "len", "out", "live", "pairs", "failed")
    graphs = []
    for _ in range(2):
        s = state()
        step(s)  # warm-up: attributes and occupancy are looked up once
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(s)
        graphs.append((gr, s, torch.cuda.Stream()))
    for _ in range(3):
        for gr, s, st in graphs:
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for gr, s, st in graphs:
        for k in keys:
            assert torch.equal(s[k], eager[k]), k
    side = torch.cuda.Stream()
    s = state()
    side.wait_stream(torch.cuda.current_stream())
    step(s, side)
    side.synchronize()
    for k in keys:
        assert torch.equal(s[k], first[k]), k
    assert torch.equal(s["back"][0], first["back"][0])
    assert B.workspace_status(s["ws"]) == 0
