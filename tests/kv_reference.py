"""Plain 64-bit forms of the paged 8-bit key/value cache and of the attention over it,
for the tests, and batches to run them on."""
import math

import torch

import block_reference as block
import w8a8_quantised_moe_gb300 as moe


def exponent(amax):
    """The least integer e >= -64 with amax <= 448 * 2^e."""
    e = -64
    while amax > 448 * 2.0**e:
        e += 1
    return e


def e4m3_round(v):
    """The E4M3 value nearest to each binary64 |v| <= 448 (1 + 2^-30), ties to the even mantissa."""
    table = block.e4m3_values()[:127].to(v.device)
    a = v.abs().contiguous()
    hi = torch.searchsorted(table, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = table[hi] - a, a - table[lo]
    got = table[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)]
    return torch.where(v < 0, -got, got)


def turned(x, rope, pos, interleaved):
    """(x [heads, dim] at one position in binary64, magnitude of the two products)."""
    x = x.double()
    if rope is None:
        return x, torch.zeros_like(x)
    R = rope.shape[1]
    cos, sin = rope[pos, : R // 2].double(), rope[pos, R // 2:].double()
    first = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
    second = first + (1 if interleaved else R // 2)
    y, mag = x.clone(), torch.zeros_like(x)
    a, b = x[:, first], x[:, second]
    y[:, first], y[:, second] = a * cos - b * sin, b * cos + a * sin
    mag[:, first], mag[:, second] = (a * cos).abs() + (b * sin).abs(), (b * cos).abs() + (a * sin).abs()
    return y, mag


class Batch:
    """Sequences [(new tokens, length)], their pages anywhere in a pool of more."""

    def __init__(self, seqs, page, n_pages=None, seed=0, extra_rows=0, extra_pages=2):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.page = seqs, page
        used = [-(-length // page) for _, length in seqs]
        self.n_pages = sum(used) + 5 if n_pages is None else n_pages
        order = torch.randperm(self.n_pages, generator=g).int()
        table = torch.full((len(seqs), max(used, default=0) + extra_pages), 1 << 30, dtype=torch.int32)  # not pages
        at = 0
        for b, u in enumerate(used):
            table[b, :u] = order[at:at + u]
            at += u
        starts = [0]
        for n, _ in seqs:
            starts.append(starts[-1] + n)
        self.T = starts[-1] + extra_rows
        self.starts = starts
        self.table = table
        self.spare = order[at:].tolist()
        self.args = (torch.tensor(starts, dtype=torch.int32).cuda(),
                     torch.tensor([length for _, length in seqs], dtype=torch.int32).cuda(), table.cuda())


def filled_cache(batch, heads, dim, seed=0, spread=1.0, scales=(-8, -4)):
    """A cache full of random codes (the rows behind a sequence hold NaN codes), scales 2^[scales)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (batch.n_pages, heads, batch.page, dim)
    parts = []
    for _ in range(2):
        x = spread * 60 * torch.randn(shape, generator=g, device="cuda")
        parts.append(x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    cache = moe.KVCache(*parts, *(torch.exp2(torch.randint(*scales, shape[:2], generator=g, device="cuda").float())
                                  for _ in range(2)))
    for b, (_, length) in enumerate(batch.seqs):
        if length % batch.page:
            last = int(batch.table[b, length // batch.page])
            cache.k[last, :, length % batch.page:] = 0x7F
            cache.v[last, :, length % batch.page:] = 0xFF
    for p in batch.spare:
        cache.k[p] = cache.v[p] = 0x7F
        cache.k_scale[p] = cache.v_scale[p] = float("nan")
    return cache


def attention(q, cache, batch, scale, window=0):
    """[(rows, out, lse, weighted mean of |v|, bound of |score error| / 2^-16, keys seen, largest |v|)] of the
    sequences' rows, binary64."""
    T, Hq, D = q.shape
    group = Hq // cache.heads
    val = block.e4m3_values().to(q.device)
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=q.device)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    mean, vmax = torch.zeros_like(out), torch.zeros_like(lse)
    terms, qterms, keys = torch.zeros_like(lse), torch.zeros_like(lse), torch.zeros_like(lse)
    for b, (n, length) in enumerate(batch.seqs):
        pages = batch.args[2][b, : -(-length // batch.page)].long()
        if n == 0 or length == 0:
            continue
        rows = slice(batch.starts[b], batch.starts[b] + n)
        pos = torch.arange(length - n, length, device=q.device)[:, None]
        j = torch.arange(length, device=q.device)
        seen = (j <= pos) & ((j > pos - window) if window else True)
        some = seen.any(1)
        for h in range(cache.heads):
            k = (val[cache.k[pages, h].long()] * cache.k_scale[pages, h].double()[:, None, None]).flatten(0, 1)[:length]
            v = (val[cache.v[pages, h].long()] * cache.v_scale[pages, h].double()[:, None, None]).flatten(0, 1)[:length]
            for i in range(h * group, (h + 1) * group):
                x = q[rows, i].double()
                s = (scale * (x @ k.T)).masked_fill(~seen, -math.inf)
                top = s.amax(1, keepdim=True)
                p = torch.where(seen, torch.exp(s - torch.where(some[:, None], top, 0.0)), 0.0)
                den = p.sum(1, keepdim=True)
                safe = torch.where(some[:, None], den, 1.0)
                out[rows, i] = p @ v / safe
                mean[rows, i] = p @ v.abs() / safe
                lse[rows, i] = torch.where(some, (torch.log(safe) + top)[:, 0], -math.inf)
                terms[rows, i] = (scale * (x.abs() @ k.abs().T)).masked_fill(~seen, 0).amax(1)
                qterms[rows, i] = scale * x.abs().amax(1) * torch.where(seen, k.abs().sum(1), 0.0).amax(1)
                keys[rows, i] = seen.sum(1).double()
                vmax[rows, i] = torch.where(seen[:, :, None], v.abs(), 0.0).amax((1, 2))
    return out, lse, mean, terms, qterms, keys, vmax


# Errors, u = 2^-24.  A score: its 128 products are exact and summed in binary32 with at
# most one rounding (or truncation, 2 u) each: 2^7 * 2^-23 of the sum of their magnitudes;
# a query channel is off by at most 2^-17 of the row's largest (two E4M3 parts; fp16 is
# nearer), so the score by that times sum |k|.  The factors, the exponent's argument (a few
# hundred at most, base 2) and ex2 (2^-22) add 2^-14 * 2^-4 at most for |argument| <= 2^9.
# A weight off by a relative e moves the result by at most 2 e of the weighted mean of |v|;
# its rounding to fp16 by 2^-11 of that, and 2^-25 where it is subnormal, the largest being
# at least 2^6: 2^-31 of the largest |v| for each key.  Sums of N terms in binary32, in runs
# of 16 keys or more: (N / 16 + 64) 2^-23, of the values and of the weights.
SCORE, QUERY, WEIGHT, BF16 = 2.0**-16, 2.0**-17, 2.0**-18, 2.0**-8


def check_attention(q, cache, batch, got, lse=None, scale=None, window=0, rows=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    want, want_lse, mean, terms, qterms, keys, vmax = attention(q, cache, batch, scale, window)
    n = slice(0, batch.starts[-1]) if rows is None else rows
    score = SCORE * terms + QUERY * qterms + WEIGHT
    sums = (keys / 16 + 64) * 2.0**-23
    bound = (mean * (2 * score + 2.0**-11 + 2 * sums)[:, :, None] + (keys * vmax * 2.0**-31)[:, :, None]) * (1 + BF16)
    bound = bound + BF16 * want.abs() + 2.0**-134
    err = (got.double() - want).abs()
    assert (err <= bound)[n].all(), (float((err / bound)[n].max()), int((err > bound)[n].sum()))
    if lse is not None:
        off = (lse.double() - want_lse).abs()
        ok = off <= score + sums + 2.0**-20 + 2.0**-22 * want_lse.abs()
        assert (ok | (lse.double() == want_lse))[n].all(), float(off[n].nan_to_num(0).max())


class Stored:
    """What a cache stands for: codes' values and scales, binary64, changed by append()."""

    def __init__(self, cache):
        val = block.e4m3_values()
        self.k, self.v = (val[c.cpu().long()] for c in (cache.k, cache.v))
        self.k_scale, self.v_scale = cache.k_scale.cpu().double(), cache.v_scale.cpu().double()

    def _store(self, codes, scales, p, h, held, x):
        """Vectors x [tokens, dim] behind the `held` ones of block (p, h)."""
        s = 2.0 ** exponent(float(x.abs().max())) if x.isfinite().all() else math.nan
        if held:
            old = float(scales[p, h])
            s = math.nan if math.isnan(s) or math.isnan(old) else max(s, old)
            if s > old:
                codes[p, h, :held] = e4m3_round(codes[p, h, :held] * (old / s))
        codes[p, h, held:held + len(x)] = 0.0 if math.isnan(s) else e4m3_round(x / s)
        scales[p, h] = s

    def append(self, k, v, batch, rope=None, interleaved=False):
        k, v = k.cpu(), v.cpu()
        rope = None if rope is None else rope.cpu()
        for b, (n, length) in enumerate(batch.seqs):
            lo = max(length - n, 0)
            end = length if rope is None else min(length, len(rope))
            row = batch.starts[b] - (length - n)
            while lo < end:
                hi = min(end, (lo // batch.page + 1) * batch.page)
                p = int(batch.table[b, lo // batch.page])
                if 0 <= p < self.k.shape[0]:
                    kk = torch.stack([turned(k[row + i], rope, i, interleaved)[0] for i in range(lo, hi)])
                    for h in range(k.shape[1]):
                        self._store(self.k, self.k_scale, p, h, lo % batch.page, kk[:, h])
                        self._store(self.v, self.v_scale, p, h, lo % batch.page, v[row + lo:row + hi, h].double())
                lo = hi

    def check(self, cache):
        """The cache holds exactly this."""
        val = block.e4m3_values()
        for name in ("k_scale", "v_scale", "k", "v"):
            got, want = getattr(cache, name).cpu(), getattr(self, name)
            got = got.double() if got.is_floating_point() else val[got.long()]
            same = (got == want) | (got.isnan() & want.isnan())
            assert same.all(), (name, int((~same).sum()), same.logical_not().nonzero()[:4].tolist())


def rope_table(positions, dim):
    turns = 1e4 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * turns
    return torch.cat([angle.cos(), angle.sin()], 1).float().cuda()


def check_queries(q, got, batch, rope, interleaved):
    """Turned queries: the second product and the sum each rounded once in binary32, then to bf16."""
    for b, (n, length) in enumerate(batch.seqs):
        for i in range(n):
            pos, r = length - n + i, batch.starts[b] + i
            if pos < 0 or (rope is not None and pos >= len(rope)):
                continue
            want, mag = turned(q[r].cpu(), None if rope is None else rope.cpu(), pos, interleaved)
            bound = BF16 * want.abs() + (1 + BF16) * 2.0**-23 * mag + 2.0**-134
            assert ((got[r].cpu().double() - want).abs() <= bound).all(), (b, i)
