"""Cases of the paged FP4 cache's operators: rotary positions, appending rows to
pages and reading them back, forking sequences, compacting the page pool, and
attention of one new token over the pages.

Every case is a dict of plain values. ``prepare`` draws its inputs on the GPU
from the seed, ``run`` makes one pass: the framework's calls where ``own`` is
true, elementary torch operations otherwise. ``exact`` restates an operator in
64 bits from its definition.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------------- cases
def listed():
    return [
        # The queries of four sequences' new tokens near 1M positions, the last
        # 64 channels of each head rotated: the smallest call of a decode step.
        {"name": "rope_decode_q", "op": "rope", "tokens": 4, "heads": 64, "dim": 512, "start": 448,
         "rot": 64, "interleaved": True, "fp32": False, "inverse": False, "factor": 1.0, "far": 1048576},
        # Main-KV rows of a whole 64K + 4096 prompt (one head), positions
        # stretched 16 times, half layout.
        {"name": "rope_prompt_kv_scaled", "op": "rope", "tokens": 69632, "heads": 1, "dim": 512,
         "start": 0, "rot": 64, "interleaved": False, "fp32": False, "inverse": False, "factor": 16.0,
         "far": 1048576},
        # Attention outputs of a 4096-token chunk turned back (K = V rows carry
        # the rotation, so the output does too), in fp32 as attention writes them.
        {"name": "rope_chunk_out_inverse", "op": "rope", "tokens": 4096, "heads": 64, "dim": 512,
         "start": 448, "rot": 64, "interleaved": True, "fp32": True, "inverse": True, "factor": 1.0,
         "far": 69632},
        # One new row for each of 32 sequences at up to 256K: a decode step.
        {"name": "append_decode", "op": "append", "seqs": 32, "new": 1, "channels": 512, "page": 64,
         "mx": False, "ragged": False, "far": 262144},
        # Prompt chunks of eight sequences with different numbers of rows, in
        # the variant with power-of-two scales, pages of an odd size.
        {"name": "append_chunks_mx", "op": "append", "seqs": 8, "new": 8192, "channels": 512,
         "page": 33, "mx": True, "ragged": True, "far": 65536},
        # Eight continuations of two prompts of about 4K, small cache rows.
        {"name": "fork_beams", "op": "fork", "parents": 2, "forks": 8, "ctx": 4096, "page": 16,
         "channels": 128, "index": 256},
        # 256 samples drawn from eight prompts of up to 32K: many table rows,
        # and a shared last page to copy for almost each.
        {"name": "fork_samples", "op": "fork", "parents": 8, "forks": 256, "ctx": 32768, "page": 64,
         "channels": 512, "index": 2048},
        # A pool of 8192 pages after many sequences have left: the pages behind
        # the live ones move into the holes.
        {"name": "compact_pool", "op": "compact", "pages": 8192, "live": 0.6, "seqs": 64, "page": 64,
         "channels": 512, "index": 2048},
        # One sequence of 4K, eight heads of 128 channels: latency.
        {"name": "attend_4k", "op": "attend", "seqs": 1, "ctx": 4096, "ragged": False, "heads": 8,
         "channels": 128, "page": 64, "mx": False, "win": 0, "sinks": 0},
        # Eight sequences of 128K, 64 heads of 512 channels.
        {"name": "attend_8x128k", "op": "attend", "seqs": 8, "ctx": 131072, "ragged": False, "heads": 64,
         "channels": 512, "page": 64, "mx": False, "win": 0, "sinks": 0},
        # Window layers of 32 sequences: the last 128 tokens and the first four.
        {"name": "attend_window", "op": "attend", "seqs": 32, "ctx": 16384, "ragged": True, "heads": 64,
         "channels": 512, "page": 64, "mx": False, "win": 128, "sinks": 4},
        # A mixed batch (an empty sequence and one of a single token among
        # them), power-of-two scales, odd head count and page size.
        {"name": "attend_mixed_mx", "op": "attend", "seqs": 13, "ctx": 20011, "ragged": True, "heads": 23,
         "channels": 320, "page": 17, "mx": True, "win": 0, "sinks": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "fork", "compact", "attend", "attend"])
    if op == "rope":
        dim = rng.choice([64, 128, 192, 320, 512])
        rot = rng.choice([r for r in (32, 48, 64, 96, 128, dim) if r <= dim])
        fp32 = rng.random() < 0.4
        heads = rng.choice([1, 2, 5, 8, 16, 64])
        most = (4096 * 64 * 512) // (heads * dim)
        return {"op": op, "tokens": _log(rng, 1, min(most, 300000)), "heads": heads, "dim": dim,
                "start": rng.choice([0, dim - rot]), "rot": rot, "interleaved": rng.random() < 0.5,
                "fp32": fp32, "inverse": rng.random() < 0.5, "factor": rng.choice([1.0, 1.0, 4.0, 16.0]),
                "far": _log(rng, 1000, 1048576)}
    if op == "append":
        new = _log(rng, 1, 8192)
        return {"op": op, "seqs": _log(rng, 1, max(1, 65536 // new) if new > 256 else 64), "new": new,
                "channels": rng.choice([32, 96, 128, 256, 320, 512]),
                "page": rng.choice([1, 16, 17, 33, 64, 128]), "mx": rng.random() < 0.5,
                "ragged": rng.random() < 0.6, "far": _log(rng, 1000, 65536)}
    if op == "fork":
        return {"op": op, "parents": _log(rng, 1, 8), "forks": _log(rng, 1, 256),
                "ctx": _log(rng, 50, 32768), "page": rng.choice([16, 17, 32, 64]),
                "channels": rng.choice([128, 256, 512]), "index": rng.choice([0, 256, 2048])}
    if op == "compact":
        page = rng.choice([16, 33, 64])
        return {"op": op, "pages": _log(rng, 64, 8192), "live": rng.uniform(0.05, 0.95),
                "seqs": _log(rng, 1, 64), "page": page, "channels": rng.choice([128, 256, 512]),
                "index": rng.choice([0, 256, 2048])}
    seqs = _log(rng, 1, 64)
    win = rng.choice([0, 0, _log(rng, 1, 4096)])
    return {"op": op, "seqs": seqs, "ctx": _log(rng, 1, 1000000 // seqs if seqs > 8 else 131072),
            "ragged": rng.random() < 0.6, "heads": rng.choice([1, 3, 8, 16, 23, 32, 40, 64]),
            "channels": rng.choice([32, 64, 96, 128, 192, 256, 320, 512]),
            "page": rng.choice([1, 16, 17, 64, 128, 256]), "mx": rng.random() < 0.4, "win": win,
            "sinks": rng.choice([0, 1, 4, 130]) if win else 0}


# ---------------------------------------------------------------------- inputs
def _lens(case):
    """Lengths of the sequences, by the case alone: a full one first, then, in a
    ragged batch, an empty one, one of one token and log-uniform ones."""
    n, top = case["seqs"], case["ctx"] if case["op"] == "attend" else case["new"]
    if not case["ragged"]:
        return [top] * n
    r = random.Random(n * 1000003 + top)
    return ([top, 0, 1] + [int(math.exp(r.uniform(0, math.log(top + 0.5)))) for _ in range(n)])[:n]


def _page_bytes(case):
    """Bytes of one page in each buffer of a cache: FP4 codes, scales and, where
    the layer has an indexer, its int8 keys and fp32 key scales."""
    p, c = case["page"], case["channels"]
    return [p * c // 2, p * c // 16] + ([p * case["index"], p * 4] if case["index"] else [])


def _buffers(case, pages, g):
    p, c = case["page"], case["channels"]
    bufs = [torch.randint(0, 256, (pages, p, c // 2), generator=g, device=DEV, dtype=torch.uint8),
            torch.randint(0, 120, (pages, p, c // 16), generator=g, device=DEV, dtype=torch.uint8)]
    if case["index"]:
        bufs += [torch.randint(-127, 128, (pages, p, case["index"]), generator=g, device=DEV, dtype=torch.int8),
                 torch.rand((pages, p), generator=g, device=DEV) + 0.5]
    return bufs


def _table(lens, page, g):
    """Page tables over randomly placed pages, -1 behind each sequence's last
    page, and the number of pages in the pool (some of them free)."""
    need = [-(-n // page) for n in lens]
    wide, total = max(1, max(need)), sum(need)
    pool = total + 7
    perm = torch.randperm(pool, generator=g, device=DEV)[:total].to(torch.int32)
    have = torch.arange(wide, device=DEV)[None] < torch.tensor(need, device=DEV)[:, None]
    table = torch.full((len(lens), wide), -1, dtype=torch.int32, device=DEV)
    table[have] = perm
    return table, pool


def _freqs(case):
    """Radians per position of each pair, base 10000; a factor above 1 stretches
    the slow pairs by it and leaves the fast ones (YaRN, original length 65536)."""
    r, factor = case["rot"], case["factor"]
    f = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device=DEV) / r)
    if factor == 1.0:
        return f, 1.0
    at = lambda turns: r * math.log(65536 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
    low, high = max(0, math.floor(at(32))), min(r - 1, math.ceil(at(1)))
    ramp = ((torch.arange(r // 2, dtype=torch.float64, device=DEV) - low) / max(high - low, 0.001)).clamp(0, 1)
    return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 11)
    op = case["op"]
    s = {"case": case}
    if op == "rope":
        shape = (case["tokens"], case["heads"], case["dim"])
        x = torch.randn(shape, generator=g, device=DEV)
        s["x"] = x if case["fp32"] else x.to(torch.bfloat16)
        first = torch.randint(0, max(1, case["far"] - case["tokens"]), (1,), generator=g, device=DEV)
        s["pos"] = first + torch.arange(case["tokens"], device=DEV)
        s["freq"], s["gain"] = _freqs(case)
        s["out"] = torch.empty_like(s["x"])
    elif op == "append":
        n, new, c, group = case["seqs"], case["new"], case["channels"], 32 if case["mx"] else 16
        rows = torch.randn((n, new, c), generator=g, device=DEV)
        rows[..., :: max(1, c // 5)] *= 16.0  # outlier channels
        s["rows"] = rows.to(torch.bfloat16)
        s["start"] = torch.randint(0, case["far"], (n,), generator=g, device=DEV)
        s["table"], pool = _table([case["far"] + new] * n, case["page"], g)
        s["valid"] = torch.tensor(_lens(case), dtype=torch.int32, device=DEV)
        s["fp4"] = torch.zeros((pool, case["page"], c // 2), dtype=torch.uint8, device=DEV)
        s["sf"] = torch.zeros((pool, case["page"], c // group), dtype=torch.uint8, device=DEV)
        s["out"] = torch.zeros((n, new, c), dtype=torch.bfloat16, device=DEV)
    elif op == "fork":
        p, f, page = case["parents"], case["forks"], case["page"]
        lens = torch.randint(max(1, case["ctx"] * 3 // 4), case["ctx"] + 1, (p,), generator=g, device=DEV)
        lens[0] = case["ctx"]
        wide = -(-case["ctx"] // page) + 1
        pool = p * wide + f + 5
        s["table"] = torch.full((p + f, wide), -1, dtype=torch.int32, device=DEV)
        have = torch.arange(wide, device=DEV)[None] < (-(-lens // page))[:, None]
        perm = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
        s["table"][:p] = torch.where(have, perm[: p * wide].view(p, wide), -1)
        s["ref"] = torch.zeros(pool + 1, dtype=torch.int32, device=DEV).index_fill_(
            0, torch.where(have, perm[: p * wide].view(p, wide), pool).flatten().long(), 1)[:pool].contiguous()
        s["len"] = torch.cat([lens, torch.zeros(f, dtype=torch.int64, device=DEV)])
        s["src"] = torch.randint(0, p, (f,), generator=g, device=DEV, dtype=torch.int32)
        s["dst"] = (p + torch.randperm(f, generator=g, device=DEV)).to(torch.int32)
        s["pairs"] = torch.empty((f, 2), dtype=torch.int32, device=DEV)
        s["failed"] = torch.empty(1, dtype=torch.int32, device=DEV)
        s["bufs"] = _buffers(case, pool, g)
    elif op == "compact":
        n, seqs = case["pages"], case["seqs"]
        live = max(1, int(round(n * case["live"])))
        wide = -(-live // seqs) + 2
        perm = torch.randperm(n, generator=g, device=DEV)[:live].to(torch.int32)
        s["ref"] = torch.zeros(n, dtype=torch.int32, device=DEV).index_fill_(0, perm.long(), 1)
        table = torch.full((seqs * wide,), -1, dtype=torch.int32, device=DEV)
        table[:live] = perm
        s["table"] = table.view(wide, seqs).t().contiguous()
        s["table_out"], s["ref_out"] = torch.empty_like(s["table"]), torch.empty_like(s["ref"])
        s["live"] = torch.empty(1, dtype=torch.int32, device=DEV)
        s["bufs"] = _buffers(case, n, g)
    else:
        lens, c, group = _lens(case), case["channels"], 32 if case["mx"] else 16
        s["table"], pool = _table(lens, case["page"], g)
        rows = torch.randn((pool, case["page"], c), generator=g, device=DEV)
        rows[..., :: max(1, c // 5)] *= 4.0  # outlier channels
        s["fp4"], s["sf"] = _quantize(rows, case["mx"])
        s["len"] = torch.tensor(lens, dtype=torch.int64, device=DEV)
        # some heads attend broadly, some sharply
        sharp = torch.linspace(0.5, 3.0, case["heads"], device=DEV)[None, :, None]
        q = torch.randn((case["seqs"], case["heads"], c), generator=g, device=DEV) * sharp
        s["q"] = q.to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((case["seqs"], case["heads"]), device=DEV)
        s["scale"] = 1.0 / math.sqrt(c)
        s["group"] = group
    return s


def _pow2(e):
    """2^e in fp64 for whole e, from its exponent field: exact, which a power or
    an exponential on the GPU need not be."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


# ----------------------------------------------------------------- plain forms
def _quantize(x, mx):
    """fp32 rows -> (packed E2M1 codes, scale bytes): E4M3(amax / 6) per 16
    channels, or with mx the power of two 2^(floor(log2 amax) - 2) per 32."""
    group = 32 if mx else 16
    # divided by a tensor: a division by a number may be done as a product, and
    # amax / 6 may lie on the midpoint of two scales
    v = x.float().unflatten(-1, (-1, group))
    amax = v.abs().amax(-1)
    if mx:
        e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, -127).clamp(-127, 127)
        scale, sf = _pow2(e).float(), (e + 127).to(torch.uint8)
    else:
        f8 = (amax / torch.full_like(amax, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
        scale, sf = f8.float(), f8.view(torch.uint8)
    y = torch.where(scale[..., None] > 0, v / scale[..., None].clamp(min=1e-45), 0.0)
    # the nearest of 0 .5 1 1.5 2 3 4 6, a tie to the even code
    a = y.abs()
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
            + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte())
    code = (code + 8 * (torch.signbit(y) & (scale[..., None] > 0)).byte()).flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous(), sf


def _values(codes, sf, mx):
    """Packed codes [.., C/2] and scale bytes -> fp32 values [.., C]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = lut[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    scale = _pow2(sf.int() - 127).float() if mx else sf.view(torch.float8_e4m3fn).float()
    return (v.unflatten(-1, (-1, 32 if mx else 16)) * scale[..., None]).flatten(-2)


def _rows(table, page, pos, ok, pool):
    """Row of the page pool for each position [B, n], and whether it has one."""
    e = pos // page
    ok = ok & (pos >= 0) & (e < table.shape[1])
    p = table.long().gather(1, e.clamp(0, table.shape[1] - 1))
    ok = ok & (p >= 0) & (p < pool)
    return torch.where(ok, p * page + pos % page, 0), ok


def _plain_rope(s):
    case = s["case"]
    a, b = case["start"], case["start"] + case["rot"]
    ang = s["pos"].double()[:, None] * s["freq"][None]
    c = (ang.cos() * s["gain"]).float()[:, None]
    d = (ang.sin() * s["gain"]).float()[:, None]
    d = -d if case["inverse"] else d
    y = s["x"].float().clone()
    r = y[..., a:b]
    if case["interleaved"]:
        u, v = r[..., 0::2].clone(), r[..., 1::2].clone()
        r[..., 0::2], r[..., 1::2] = u * c - v * d, v * c + u * d
    else:
        h = case["rot"] // 2
        u, v = r[..., :h].clone(), r[..., h:].clone()
        r[..., :h], r[..., h:] = u * c - v * d, v * c + u * d
    return y.to(s["x"].dtype)


def _plain_append(s):
    case = s["case"]
    codes, sf = _quantize(s["rows"], case["mx"])
    i = torch.arange(case["new"], device=DEV)[None]
    row, ok = _rows(s["table"], case["page"], s["start"][:, None] + i, i < s["valid"][:, None], s["fp4"].shape[0])
    s["fp4"].flatten(0, 1)[row[ok]] = codes[ok]
    s["sf"].flatten(0, 1)[row[ok]] = sf[ok]
    back = _values(s["fp4"].flatten(0, 1)[row], s["sf"].flatten(0, 1)[row], case["mx"])
    return torch.where(ok[..., None], back, 0.0).to(torch.bfloat16)


def _plain_fork(s):
    case = s["case"]
    page, table, ref = case["page"], s["table"], s["ref"]
    src, dst = s["src"].long(), s["dst"].long()
    old = table[dst]
    ref.scatter_add_(0, old.clamp(min=0).flatten().long(), -(old >= 0).int().flatten())
    table[dst] = -1
    n = s["len"][src]
    full, part = n // page, n % page > 0
    row = table[src]
    at = torch.arange(table.shape[1], device=DEV)[None]
    keep = (at < full[:, None]) & (row >= 0)
    last = row.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    want = part & (last >= 0)
    used = ref > 0
    order = torch.argsort(used.int(), stable=True)
    turn = torch.cumsum(want.int(), 0) - 1
    got = want & (turn < (~used).sum())
    new = torch.where(got, order[turn.clamp(0, ref.numel() - 1)], -1).int()
    fresh = torch.where(keep, row, -1)
    table[dst] = torch.where((at == full[:, None]) & got[:, None], new[:, None], fresh)
    ref.scatter_add_(0, row.clamp(min=0).flatten().long(), keep.int().flatten())
    ref.scatter_add_(0, new.clamp(min=0).long(), got.int())
    s["len"][dst] = torch.where(want & ~got, full * page, n)
    pairs = torch.stack([torch.where(got, last, -1), new], 1)
    a, b = pairs[got, 0].long(), pairs[got, 1].long()
    for buf in s["bufs"]:
        buf[b] = buf[a]
    return [table, ref, s["len"], pairs, (want & ~got).sum().int().view(1)] + s["bufs"]


def _plain_compact(s):
    ref, table = s["ref"], s["table"]
    used = ref > 0
    live = used.sum()
    at = torch.arange(ref.numel(), device=DEV)
    holes, movers = at[~used & (at < live)], at[used & (at >= live)]
    to = at.clone()
    to[movers] = holes
    s["table_out"].copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], -1))
    s["ref_out"].zero_()
    s["ref_out"][to[used]] = ref[used]
    for buf in s["bufs"]:
        buf[holes] = buf[movers]
    return [s["table_out"], s["ref_out"], live.int().view(1)] + s["bufs"]


def _visible(case, lens):
    """(positions of the visible keys [B, n], whether slot j holds one): the
    first ``sinks`` tokens and the last ``win``, or all without a window."""
    n = lens[:, None]
    win, sinks = case["win"], case["sinks"]
    most = case["ctx"] if not win else min(case["ctx"], win + sinks)
    j = torch.arange(most, device=lens.device)[None]
    if not win:
        return j.expand(lens.numel(), -1), j < n
    ns = n.clamp(max=sinks)
    w0 = torch.maximum(n - win, ns)
    return torch.where(j < ns, j, w0 + j - ns), j < ns + n - w0


def _plain_attend(s):
    case = s["case"]
    pos, ok = _visible(case, s["len"])
    row, ok = _rows(s["table"], case["page"], pos, ok, s["fp4"].shape[0])
    kv = _values(s["fp4"].flatten(0, 1)[row], s["sf"].flatten(0, 1)[row], case["mx"])
    kv = torch.where(ok[..., None], kv, 0.0)
    x = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * s["scale"]
    x = torch.where(ok[:, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, torch.matmul(p, kv) / total, 0.0)
    return out.to(torch.bfloat16), (m + torch.log(total))[..., 0]


def run(s):
    case, op = s["case"], s["case"]["op"]
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "fork": _plain_fork, "compact": _plain_compact,
                "attend": _plain_attend}[op](s)
    from sparse_attention_fp4_kv_b200 import binding as b
    if op == "rope":
        b.csa2_rope(s["x"], s["pos"], s["freq"], s["out"], rot_start=case["start"],
                    interleaved=case["interleaved"], inverse=case["inverse"], mscale=s["gain"])
        return s["out"]
    if op == "append":
        b.csa2_paged_kv_append_fp4(s["rows"], s["start"], s["table"], s["fp4"], s["sf"], n_valid=s["valid"],
                                   mx=case["mx"])
        b.csa2_paged_kv_gather(s["fp4"], s["sf"], s["table"], s["start"], s["out"], n_valid=s["valid"],
                               mx=case["mx"])
        return s["out"]
    if op == "fork":
        b.csa2_pages_free(s["table"], s["ref"], s["dst"], case["page"])
        b.csa2_pages_fork(s["table"], s["ref"], s["len"], s["src"], s["dst"], case["page"], s["pairs"], s["failed"])
        b.csa2_pages_copy(s["pairs"], s["bufs"])
        return [s["table"], s["ref"], s["len"], s["pairs"], s["failed"]] + s["bufs"]
    if op == "compact":
        b.csa2_pages_compact(s["table"], s["ref"], s["bufs"], s["table_out"], s["ref_out"], s["live"])
        return [s["table_out"], s["ref_out"], s["live"]] + s["bufs"]
    b.csa2_paged_attn_decode(s["q"], s["fp4"], s["sf"], s["table"], s["len"], s["out"], s["scale"],
                             n_win=case["win"], n_sink=case["sinks"], lse=s["lse"], mx=case["mx"])
    return s["out"], s["lse"]


# ------------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * case["dim"] * (4 if case["fp32"] else 2) + 8 * case["tokens"] + 4 * case["rot"],
                "flops": 3 * n * case["rot"]}
    if op == "append":
        c, rows = case["channels"], sum(_lens(case))
        return {"bytes": rows * (2 * c + c // 2 + c // (32 if case["mx"] else 16) + 2 * c) + 12 * case["seqs"],
                "flops": 4 * rows * c}
    if op == "fork":
        entries = case["forks"] * (case["ctx"] * 7 // 8 // case["page"])
        # table rows of parents read and forks written, counts updated, and the
        # part pages read and written
        return {"bytes": 4 * (case["parents"] + case["forks"]) * -(-case["ctx"] // case["page"]) + 4 * entries
                + 2 * case["forks"] * sum(_page_bytes(case)), "flops": 0}
    if op == "compact":
        n = case["pages"]
        live = max(1, int(round(n * case["live"])))
        # pages behind the live count, on average over random placements
        moves = live * (n - live) / n
        return {"bytes": 8 * n + 8 * case["seqs"] * (-(-live // case["seqs"]) + 2) + 2 * moves * sum(_page_bytes(case)),
                "flops": 0}
    c, group = case["channels"], 32 if case["mx"] else 16
    keys = sum(n if not case["win"] else min(n, case["win"] + case["sinks"]) for n in _lens(case))
    heads = case["seqs"] * case["heads"]
    return {"bytes": keys * (c // 2 + c // group) + 4 * -(-keys // case["page"]) + heads * (4 * c + 4),
            "flops": 4 * keys * case["heads"] * c}


# ------------------------------------------------------- definitions in 64 bits
def _decode64(codes, sf, group):
    """Values of cache rows from the formats' fields: E2M1 (sign, two exponent
    bits with bias 1, one mantissa bit), E4M3 (bias 7) or E8M0 (bias 127)."""
    out = torch.empty(codes.shape[:-1] + (codes.shape[-1] * 2,), dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        n = (codes >> (4 * half)) & 15
        e, m = ((n >> 1) & 3).double(), (n & 1).double()
        v = torch.where(e == 0, m * 0.5, _pow2(e - 1) * (1 + m * 0.5))
        out[..., half::2] = torch.where(n >= 8, -v, v)
    if group == 32:
        scale = _pow2(sf.int() - 127)
    else:
        e, m = ((sf >> 3) & 15).double(), (sf & 7).double()
        scale = torch.where(e == 0, m * 2.0 ** -9, _pow2(e - 7) * (1 + m / 8))
    return out * scale.repeat_interleave(group, -1)


def _nearest64(y):
    """The nearest E2M1 value, ties to the even code, from the midpoints."""
    grid = torch.tensor(E2M1, dtype=torch.float64, device=y.device)
    a = y.abs().clamp(max=6.0)
    hi = torch.bucketize(a, grid).clamp(1, 7)
    lo = hi - 1
    mid = (grid[lo] + grid[hi]) / 2
    up = (a > mid) | ((a == mid) & (hi % 2 == 0))
    return torch.copysign(torch.where(up, grid[hi], grid[lo]), y)


def exact(case, seed):
    op = case["op"]
    if op in ("fork", "compact"):
        return None  # whole numbers and copies
    s = prepare(case, seed)
    if op == "rope":
        x = s["x"].double()
        turn = torch.polar(torch.full((), float(s["gain"]), dtype=torch.float64, device=DEV).expand(len(s["pos"]), case["rot"] // 2).contiguous(),
                           torch.outer(s["pos"].double(), s["freq"]) * (-1.0 if case["inverse"] else 1.0))[:, None]
        part = x[..., case["start"]:case["start"] + case["rot"]]
        pairs = part.unflatten(-1, (-1, 2)) if case["interleaved"] else part.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.complex(pairs[..., 0], pairs[..., 1]) * turn)
        part.copy_(z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2))
        return x
    if op == "append":
        group = 32 if case["mx"] else 16
        x = s["rows"].double().unflatten(-1, (-1, group))
        top = x.abs().amax(-1, keepdim=True)
        if case["mx"]:
            scale = _pow2(torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(-127, 127))
        else:
            t = (top / 6).clamp(max=448.0)
            unit = _pow2((torch.frexp(t)[1] - 1).clamp(min=-6) - 3)
            scale = (t / unit).round() * unit
        y = torch.where(scale > 0, _nearest64(x / scale.clamp(min=1e-300)) * scale, 0.0).flatten(-2)
        i = torch.arange(case["new"], device=DEV)
        return torch.where((i[None] < s["valid"][:, None])[..., None], y, 0.0)
    outs, lses = [], []
    for b, n in enumerate(_lens(case)):
        see = [p for p in range(n)] if not case["win"] else [p for p in range(n) if p < case["sinks"] or p >= n - case["win"]]
        q = s["q"][b].double()
        if not see:
            outs.append(torch.zeros_like(q))
            lses.append(torch.full((case["heads"],), -math.inf, dtype=torch.float64, device=DEV))
            continue
        pos = torch.tensor(see, device=DEV)
        page = s["table"][b].long()[pos // case["page"]]
        kv = _decode64(s["fp4"][page, pos % case["page"]], s["sf"][page, pos % case["page"]], s["group"])
        x = (q @ kv.T) * s["scale"]
        lse = torch.logsumexp(x, -1)
        outs.append(torch.exp(x - lse[:, None]) @ kv)
        lses.append(lse)
    return torch.stack(outs), torch.stack(lses)
