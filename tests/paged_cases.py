"""Plain restatements of the paged FP4 cache's operators, in 64 bits or whole
numbers, that the tests compare against."""
import math

import torch


def e2m1_table(device):
    v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=device)
    return torch.cat([v, -v])


def scale_table(mx, device):
    """Values of all 256 scale bytes: E8M0, or E4M3 (NaN codes left at 480, never written)."""
    c = torch.arange(256, device=device)
    if mx:
        return torch.pow(torch.tensor(2.0, dtype=torch.float64), (c - 127).double().cpu()).to(device)
    e, m = ((c >> 3) & 15).double(), (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, torch.pow(torch.tensor(2.0, dtype=torch.float64), (e - 7).cpu()).to(device)
                    * (1 + m / 8))
    return torch.where(c >= 128, -v, v)


def dequant(codes, sf, mx):
    """Packed rows [.., C/2], scales -> fp64 [.., C]."""
    lut, st = e2m1_table(codes.device), scale_table(mx, codes.device)
    v = lut[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    return v * st[sf.int()].repeat_interleave(32 if mx else 16, -1)


def visible(n, win, sink):
    return [p for p in range(n) if win == 0 or p >= n - win or p < sink]


def attend(q, fp4, sf, table, lens, scale, win=0, sink=0, mx=False):
    """fp64 outputs, lse, and the per-element error bound of an fp32 kernel.

    Bound: a score is a sum of C products that are exact in fp32 (8 + 6 bits),
    so it is off by at most C 2^-23 |scale| sum|q k| (any summation order, and
    accumulators that truncate); the weights then by a factor of 1 +- 2 d with d
    that bound, by 2^-11 for weights rounded to 16-bit floats, and by 2^-18 for
    exp and the fp32 sums; the output once more by half a bf16 step, 2^-8. A
    16-bit float of step 2^-24 rounds a small weight by up to 2^-25; the largest
    weight is held at 2^7 or more, so that is 2^-32 of the weights' sum, for each
    key: 2^-32 sum_j |v_j|, felt where a channel is zero in all keys that count."""
    B, H, C = q.shape
    n_pages, page = fp4.shape[:2]
    outs, lses, bounds, lse_bounds = [], [], [], []
    for b in range(B):
        n = max(0, min(int(lens[b]), table.shape[1] * page))
        see = []
        row = table[b].tolist()
        for p in visible(n, win, sink):
            if 0 <= row[p // page] < n_pages:
                see.append(row[p // page] * page + p % page)
        x = q[b].double()
        if not see:
            outs.append(torch.zeros_like(x))
            lses.append(torch.full((H,), -math.inf, dtype=torch.float64, device=q.device))
            bounds.append(torch.zeros_like(x))
            lse_bounds.append(torch.zeros(H, dtype=torch.float64, device=q.device))
            continue
        at = torch.tensor(see, device=q.device)
        kv = dequant(fp4.flatten(0, 1)[at], sf.flatten(0, 1)[at], mx)
        s = scale * (x @ kv.T)
        d = C * 2.0 ** -23 * abs(scale) * (x.abs() @ kv.abs().T).amax(-1)
        lse = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[:, None])
        o = p @ kv
        eps = 2 * d + 2.0 ** -11 + 2.0 ** -18
        outs.append(o)
        lses.append(lse)
        bounds.append(2.0 ** -8 * o.abs() + (1 + 2.0 ** -8) * eps[:, None] * (p @ kv.abs()) + 2.0 ** -32 * kv.abs().sum(0) + 1e-30)
        lse_bounds.append(d + 2.0 ** -20 * (1 + lse.abs()))
    return torch.stack(outs), torch.stack(lses), torch.stack(bounds), torch.stack(lse_bounds)


def shares(tiles, ctas):
    """How the attention divides its list of tiles: [(sequence and head group, first
    tile, behind the last)] of each CTA, where `tiles` has the tiles of each pair in
    the list's order."""
    total = sum(tiles)
    ctas = min(ctas, total)
    got, pair, at = [], 0, 0
    for c in range(ctas):
        left, own = (c + 1) * total // ctas - c * total // ctas, []
        while left:
            if at == tiles[pair]:
                pair, at = pair + 1, 0
                continue
            n = min(left, tiles[pair] - at)
            own.append((pair, at, at + n))
            at, left = at + n, left - n
        got.append(own)
    return got


def online(x, rows, moved, tile=64, far=8.0):
    """The attention of one share as the kernel goes about it, in fp64: x [H][n] scores
    in units of log2, rows [n][C]. The reference is the first tile's maximum and moves
    when a score exceeds it by `far`; moved(o, l, factor) gives the sums after that.
    (out, lse, moves of each head)"""
    ref, count = None, torch.zeros(x.shape[0], dtype=torch.int64)
    for j in range(0, x.shape[1], tile):
        s, v = x[:, j:j + tile], rows[j:j + tile]
        m = s.amax(-1)
        if ref is None:
            ref, l, o = m, torch.zeros_like(m), torch.zeros((x.shape[0], rows.shape[1]), dtype=x.dtype)
        else:
            up = m > ref + far
            now = torch.where(up, m, ref)
            o, l = moved(o, l, torch.exp2(ref - now))
            ref, count = now, count + up
        w = torch.exp2(s - ref[:, None])
        o, l = o + w @ v, l + w.sum(-1)
    return o / l[:, None], (ref + l.log2()) * math.log(2.0), count


LEVELS = [m * 2.0 ** k for k in range(-1, 6) for m in (1.0, 1.5)] + [64.0]


def stepped(kind, n, H, C, mx, g, device):
    """(queries [1][H][C], codes [n][C/2], scales, softmax scale) whose scores go by
    steps: the first 32 channels of key j all hold one value, the rest is random and no
    query looks at it. Scores reach 64 to 120."""
    i = torch.arange(n, device=device)
    if kind == "rising":
        level = i * len(LEVELS) // n
    elif kind == "falling":
        level = (n - 1 - i) * len(LEVELS) // n
    elif kind == "saw":  # up and down from tile to tile, and up on the whole
        t = i // 64
        level = (t * 3 // 2 + 7 * (t % 2) - 4 * (t % 3 == 2).long()).clamp(0, len(LEVELS) - 1)
    else:  # a single high key in every second tile, each above the last
        level = torch.where(i % 128 == 73, 6 + 2 * (i // 128), 0).clamp(max=len(LEVELS) - 1)
    v = torch.tensor(LEVELS, dtype=torch.float64, device=device)[level]
    e = torch.floor(torch.log2(v)).long()
    group = 32 if mx else 16
    codes = torch.randint(0, 256, (n, C // 2), generator=g, device=device, dtype=torch.uint8)
    lo, hi = (122, 130) if mx else (0x20, 0x40)
    sf = torch.randint(lo, hi, (n, C // group), generator=g, device=device, dtype=torch.uint8)
    codes[:, :16] = torch.where(v > 1.25 * 2.0 ** e.double(), 0x33, 0x22).to(torch.uint8)[:, None]  # 1.5 or 1, twice a byte
    sf[:, :32 // group] = (e + 127 if mx else (e + 7) << 3).to(torch.uint8)[:, None]
    q = torch.zeros((1, H, C), device=device)
    q[..., :32] = torch.randn((1, H, 32), generator=g, device=device).abs()
    q *= (torch.linspace(0.8, 1.5, H, device=device)[:, None] * 25 / q.sum(-1, keepdim=True))
    return q.to(torch.bfloat16), codes, sf, 0.05


def rope(x, pos, freq, start, interleaved, inverse, gain):
    """fp64 rotation and its per-element error bound, without the rounding of the
    result: the reduced angle is off by at most pi 2^-25 (rounded to fp32), sin
    and cos by 2^-23, the gain and its product, the two products and the sum by
    2^-24 each, all relative to gain (|u| + |v|); together below 2^-20."""
    y = x.double().clone()
    rot = 2 * freq.numel()
    a = pos.double()[:, None] * freq[None]
    c, s = (a.cos() * gain)[:, None], (a.sin() * gain * (-1 if inverse else 1))[:, None]
    idx = torch.arange(rot // 2, device=x.device)
    u, v = (2 * idx, 2 * idx + 1) if interleaved else (idx, idx + rot // 2)
    u, v = u + start, v + start
    bound = torch.zeros_like(y)
    p, q = x.double()[..., u], x.double()[..., v]
    y[..., u], y[..., v] = p * c - q * s, q * c + p * s
    bound[..., u] = bound[..., v] = 2.0 ** -20 * gain * (p.abs() + q.abs())
    return y, bound


class Pool:
    """Page bookkeeping with lists: what the calls have to leave behind."""

    def __init__(self, table, ref, page, lens=None):
        self.table, self.ref, self.page = table.tolist(), ref.tolist(), page
        self.len = lens.tolist() if lens is not None else None
        self.M, self.N = table.shape[1], ref.numel()

    def has(self, v):
        return 0 <= v < self.N

    def free_pages(self):
        return [p for p in range(self.N) if self.ref[p] <= 0]

    def extend(self, want):
        left, failed = self.free_pages(), 0
        for s, n in enumerate(want):
            for e in range(min(self.M, max(0, -(-n // self.page)))):
                if not self.has(self.table[s][e]):
                    if left:
                        p = left.pop(0)
                        self.table[s][e], self.ref[p] = p, 1
                    else:
                        failed += 1
        return failed

    def fork(self, src, dst):
        left, failed, pairs = self.free_pages(), 0, []
        S = len(self.table)
        empty = [all(not self.has(v) for v in row) for row in self.table]
        for f, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < S and 0 <= d < S) or d in src or d in dst[:f] or not empty[d]:
                pairs.append((-1, -1))
                failed += 1
                continue
            n = self.len[s]
            m = max(0, min(n, self.M * self.page))
            full = m // self.page
            for e in range(full):
                v = self.table[s][e]
                self.table[d][e] = v if self.has(v) else -1
                if self.has(v):
                    self.ref[v] += 1
            self.len[d] = n
            pair = (-1, -1)
            if m % self.page and self.has(self.table[s][full]):
                if left:
                    p = left.pop(0)
                    pair = (self.table[s][full], p)
                    self.table[d][full], self.ref[p] = p, 1
                else:
                    failed += 1
                    self.len[d] = full * self.page
            pairs.append(pair)
        return pairs, failed

    def free(self, seq, keep=None):
        for f, s in enumerate(seq):
            if not 0 <= s < len(self.table):
                continue
            k = 0 if keep is None else max(0, -(-keep[f] // self.page))
            for e in range(k, self.M):
                v = self.table[s][e]
                self.table[s][e] = -1
                if self.has(v):
                    self.ref[v] -= 1

    def compact(self):
        live = [p for p in range(self.N) if self.ref[p] > 0]
        L = len(live)
        moves = dict(zip([p for p in live if p >= L], [p for p in range(L) if self.ref[p] <= 0]))
        self.table = [[moves.get(v, v) for v in row] for row in self.table]
        new = [0] * self.N
        for p in live:
            new[moves.get(p, p)] = self.ref[p]
        self.ref = new
        return L, moves
