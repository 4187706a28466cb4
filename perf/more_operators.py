"""Measured cases of the paged 8-bit key/value cache and of the attention over it.

Two operators, reached through ``w8a8_quantised_moe_gb300``:

* ``kv_append``: the keys and values of new tokens go into the cache's pages, the keys
  (and the queries) rotated by their positions on the way, as E4M3 codes with one scale
  for each page and head;
* ``kv_attention``: softmax attention of new tokens' queries over the cached keys and
  values of their sequence, causal, with or without a window.

A block of the cache is the tokens of one page and head.  Its scale is the smallest
power of two s (at least 2^-64) with max |value| <= 448 s, its codes the E4M3 values
nearest to value / s.  A page that already holds tokens keeps the larger of its scale
and the new tokens'; where that grows, the codes it holds are rounded again.

``run`` computes them either in plain 32-bit torch operations (``own`` false) or by the
framework's calls (``own`` true); ``exact`` computes them in 64 bits from the definition.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
LEAST = -64  # exponent of the smallest scale
ROPE_BASE = 10000.0

# A case's sizes: B sequences; `new` tokens each (the first has `chunk` where given); the
# longest context `ctx` (new tokens included), the others' spread over [ctx / 4, ctx] where
# `ragged`; Hq query and Hkv key/value heads of D channels; pages of `page` tokens.
ATTEND = {"op": "attend", "chunk": 0, "ragged": False, "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "window": 0}
APPEND = {"op": "append", "chunk": 0, "ragged": False, "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "rope": 128,
          "pairs": False}


def listed():
    return [
        # one token of one sequence: the latency of a decode step
        {"name": "append_one_token", **APPEND, "B": 1, "new": 1, "ctx": 4096},
        # a decode step of the framework's batch of 64 sequences, their lengths anywhere in a page
        {"name": "append_decode", **APPEND, "B": 64, "new": 1, "ctx": 4096, "ragged": True},
        # short prompts of odd lengths in small pages, half of the channels rotated, neighbours paired
        {"name": "append_ragged", **APPEND, "B": 7, "new": 137, "ctx": 1111, "ragged": True, "Hq": 15, "Hkv": 5,
         "D": 64, "page": 16, "rope": 32, "pairs": True},
        # the framework's prompt of 8192 tokens
        {"name": "append_prompt", **APPEND, "B": 1, "new": 8192, "ctx": 8192},
        # one token against a context of 4096: the latency of a decode step
        {"name": "attend_one_token", **ATTEND, "B": 1, "new": 1, "ctx": 4096},
        # a decode step of 64 sequences of very different lengths
        {"name": "attend_decode", **ATTEND, "B": 64, "new": 1, "ctx": 8192, "ragged": True},
        # two long conversations, heads of the framework's 7168-wide layer (7 to a key head)
        {"name": "attend_long", **ATTEND, "B": 2, "new": 1, "ctx": 131072, "Hq": 56},
        # small heads and pages, a window that ends inside a page, an odd number of heads in a group
        {"name": "attend_window", **ATTEND, "B": 13, "new": 1, "ctx": 1777, "ragged": True, "Hq": 15, "Hkv": 5,
         "D": 64, "page": 16, "window": 500},
        # four drafted tokens to check in each of 32 sequences
        {"name": "attend_draft", **ATTEND, "B": 32, "new": 4, "ctx": 4096, "ragged": True, "Hkv": 4},
        # a prompt's chunk of 512 tokens together with 8 sequences that decode
        {"name": "attend_mixed", **ATTEND, "B": 9, "new": 1, "chunk": 512, "ctx": 8192, "ragged": True},
        # five prompts of about a thousand tokens, some after a cached beginning
        {"name": "attend_prompts", **ATTEND, "B": 5, "new": 1003, "ctx": 2345, "ragged": True, "page": 32},
        # the framework's prompt of 8192 tokens
        {"name": "attend_prompt", **ATTEND, "B": 1, "new": 8192, "ctx": 8192},
    ]


def _size(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi], a power of two now and then."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, 1 << int(math.log2(v)) if rng.random() < 0.3 else int(v)))


def draw(rng):
    most = work(listed()[-1])["flops"]
    while True:
        attend = rng.random() < 0.65
        Hkv = _size(rng, 1, 8)
        c = {**(ATTEND if attend else APPEND), "B": _size(rng, 1, 64), "ragged": rng.random() < 0.7, "Hkv": Hkv,
             "Hq": Hkv * _size(rng, 1, 16), "D": rng.choice((64, 128)), "page": rng.choice((16, 32, 64, 128))}
        c["new"] = 1 if rng.random() < 0.5 else _size(rng, 2, 8192)
        c["ctx"] = max(c["new"], _size(rng, 16, 131072 if attend else 16384))
        if attend:
            c["window"] = _size(rng, 16, 4096) if rng.random() < 0.25 else 0
            c["chunk"] = _size(rng, 2, 1024) if c["new"] == 1 and rng.random() < 0.3 else 0
            c["ctx"] = max(c["ctx"], c["chunk"])
        else:
            c["pairs"] = rng.random() < 0.5
            c["rope"] = rng.choice((0, 16, c["D"] // 2, c["D"]))
        w, cached = work(c), c["B"] * c["ctx"] * c["Hkv"] * c["D"]
        tokens = c["B"] * c["new"] + c["chunk"]
        scores = tokens * c["Hq"] * c["ctx"] if attend else 0  # of the plain form
        if cached <= 1 << 29 and tokens <= 8192 and scores <= 32 << 26 and w["flops"] <= most:
            return c


def _sequences(c):
    """[(new tokens, context with them)], by the case alone."""
    got = []
    for b in range(c["B"]):
        n = c["chunk"] if b == 0 and c.get("chunk") else c["new"]
        length = c["ctx"]
        if c["ragged"] and b:
            length = int(c["ctx"] * (0.25 + 0.75 * (b * 0.6180339887 % 1)))
            if n > 1:  # prompts of different lengths, some of them whole
                n = max(1, int(n * (0.25 + 0.75 * (b * 0.7548776662 % 1))))
        got.append((n, max(n, length)))
    return got


# ---------------------------------------------------------------- inputs


def _exponent(amax):
    """Exponent of the scale of a block with this largest magnitude."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
    return (e - 9 + (m > 0.875)).clamp(min=LEAST)


def _power(e):
    """2^e, binary64, of whole numbers e."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _scale(amax):
    return _power(_exponent(amax)).float()


def _pages(g, n, c, spread):
    """Codes and scales of n pages of random vectors, some channels louder than the others."""
    H, P, D = c["Hkv"], c["page"], c["D"]
    loud = 1 + 7 * (torch.rand(H, 1, D, generator=g, device="cuda") < 0.02)
    codes = torch.empty(n, H, P, D, dtype=torch.uint8, device="cuda")
    scales = torch.empty(n, H, device="cuda")
    for at in range(0, n, 2048):
        x = spread * loud * torch.randn(min(2048, n - at), H, P, D, generator=g, device="cuda")
        s = _scale(x.abs().amax((2, 3)))
        codes[at:at + 2048] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[at:at + 2048] = s
    return codes, scales


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    seqs, P, D, Hq, Hkv = _sequences(c), c["page"], c["D"], c["Hq"], c["Hkv"]
    T = sum(n for n, _ in seqs)
    used = [-(-length // P) for _, length in seqs]
    n_pages = sum(used) + 3  # a pool with pages that no sequence uses, in no order
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    table = torch.zeros(c["B"], max(used), dtype=torch.int32, device="cuda")
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    starts = [0]
    for n, _ in seqs:
        starts.append(starts[-1] + n)
    k_codes, k_scale = _pages(g, n_pages, c, 1.0)
    v_codes, v_scale = _pages(g, n_pages, c, 0.5)
    st = {"case": c, "op": c["op"], "seqs": seqs, "k_codes": k_codes, "v_codes": v_codes, "k_scale": k_scale,
          "v_scale": v_scale, "table": table, "q_start": torch.tensor(starts, dtype=torch.int32, device="cuda"),
          "lengths": torch.tensor([length for _, length in seqs], dtype=torch.int32, device="cuda")}
    if c["op"] == "append":
        # rows of a fused projection: queries, keys and values next to each other
        rows = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device="cuda")
        rows *= 1 + 7 * (torch.rand(rows.shape[1], generator=g, device="cuda") < 0.02)
        rows = rows.bfloat16()
        st["q"] = rows[:, : Hq * D].unflatten(1, (Hq, D))
        st["k"] = rows[:, Hq * D: (Hq + Hkv) * D].unflatten(1, (Hkv, D))
        st["v"] = rows[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
        st["rope"] = None
        if c["rope"]:  # cosines, then sines, of every position's angles
            turns = ROPE_BASE ** (-torch.arange(0, c["rope"], 2, device="cuda", dtype=torch.float64) / c["rope"])
            angle = torch.arange(c["ctx"], device="cuda", dtype=torch.float64)[:, None] * turns
            st["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        # what a program that lacks the operator knows of its batch: each new token's sequence and position
        st["seq_of"] = torch.tensor([b for b, (n, _) in enumerate(seqs) for _ in range(n)], device="cuda")
        st["pos_of"] = torch.tensor([length - n + i for n, length in seqs for i in range(n)], device="cuda")
    else:
        st["q"] = (2 * torch.randn(T, Hq, D, generator=g, device="cuda")).bfloat16()
        # the same: sequences with equally many new tokens are computed together
        groups = {}
        for b, (n, length) in enumerate(seqs):
            groups.setdefault(n, []).append(b)
        st["groups"] = [(n, max(seqs[b][1] for b in bs), torch.tensor(bs, device="cuda"),
                         torch.tensor([starts[b] for b in bs], device="cuda")) for n, bs in groups.items()]
    if own:  # a serving loop keeps its cache's handle and its workspace from call to call
        import w8a8_quantised_moe_gb300 as moe

        st["lib"] = moe
        st["cache"] = moe.KVCache(k_codes, v_codes, k_scale, v_scale)
        if c["op"] == "attend":
            st["ws"] = moe.new_workspace(moe.kv_attention_workspace_size(c["B"], T, Hq, Hkv, D))
    return st


# ---------------------------------------------------------------- one pass


def _rotated(x, rope, pos, pairs):
    """x [T, heads, D] with its first channels turned by the angles of its positions, fp32."""
    x = x.float()
    if rope is None:
        return x
    half = rope.shape[1] // 2
    cos, sin = rope[pos, None, :half], rope[pos, None, half:]
    turned = x[..., : 2 * half]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if pairs else turned.chunk(2, dim=-1)
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((a, b), -1).flatten(-2) if pairs else torch.cat((a, b), -1)
    return torch.cat((turned, x[..., 2 * half:]), -1)


def _plain_store(codes, scales, x, st):
    """New tokens' vectors x [T, H, D] (fp32) into the pages, in place."""
    P, pos = codes.shape[2], st["pos_of"]
    page = st["table"][st["seq_of"], pos // P].long()
    first = pos - torch.arange(len(pos), device=pos.device) + st["q_start"][st["seq_of"]]  # a sequence's first new
    held = torch.where(first // P == pos // P, first % P, 0)  # tokens that the token's page holds before
    amax = torch.zeros_like(scales).index_reduce_(0, page, x.abs().amax(2), "amax", include_self=True)
    fresh = _scale(amax[page])
    old = scales[page]
    s = torch.where(held[:, None] > 0, torch.maximum(old, fresh), fresh)
    # what a page holds, rounded again to its scale (the same for every new token of the page)
    one, kept = page[held > 0], held[held > 0]
    again = codes[one].view(torch.float8_e4m3fn).float() * (old / s)[held > 0][:, :, None, None]
    stays = torch.arange(P, device=pos.device) < kept[:, None]
    codes[one] = torch.where(stays[:, None, :, None], again.to(torch.float8_e4m3fn).view(torch.uint8), codes[one])
    codes[page, :, pos % P] = (x / s[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    scales[page] = s


def _plain_append(st):
    pairs = st["case"]["pairs"]
    k = _rotated(st["k"], st["rope"], st["pos_of"], pairs)
    _plain_store(st["k_codes"], st["k_scale"], k, st)
    _plain_store(st["v_codes"], st["v_scale"], st["v"].float(), st)
    return _rotated(st["q"], st["rope"], st["pos_of"], pairs).bfloat16()


def _plain_attend(st):
    c, q = st["case"], st["q"]
    Hq, Hkv, D, P, window = (c[n] for n in ("Hq", "Hkv", "D", "page", "window"))
    out = torch.empty_like(q)

    def values(codes, scales, pages):  # [b, Hkv, tokens, D]
        x = codes[pages].view(torch.float8_e4m3fn).float() * scales[pages][:, :, :, None, None]
        return x.transpose(1, 2).flatten(2, 3)

    for n, longest, seqs, starts in st["groups"]:
        pages = st["table"][seqs, : -(-longest // P)].long()
        rows = starts[:, None] + torch.arange(n, device=q.device)
        qs = q[rows].float().view(len(seqs), n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).flatten(2, 3)
        s = (qs / math.sqrt(D)) @ values(st["k_codes"], st["k_scale"], pages).transpose(2, 3)
        j = torch.arange(pages.shape[1] * P, device=q.device)
        at = st["lengths"][seqs, None].long() - n + torch.arange(n, device=q.device)  # positions of the rows
        seen = j <= at[:, :, None]
        if window:
            seen &= j > at[:, :, None] - window
        s = s.view(*s.shape[:2], Hq // Hkv, n, -1)
        s.masked_fill_(~seen[:, None, None], -math.inf)
        s -= s.amax(-1, keepdim=True)
        p = s.exp_()
        p /= p.sum(-1, keepdim=True)
        o = p.flatten(2, 3) @ values(st["v_codes"], st["v_scale"], pages)
        o = o.view(len(seqs), Hkv, Hq // Hkv, n, D).permute(0, 3, 1, 2, 4).reshape(len(seqs), n, Hq, D)
        out[rows] = o.bfloat16()
    return out


def run(state):
    st = state
    if st["op"] == "append":
        if own:
            q = st["lib"].kv_append(st["cache"], st["k"], st["v"], st["q_start"], st["lengths"], st["table"],
                                    q=st["q"], rope=st["rope"], interleaved=st["case"]["pairs"])
        else:
            q = _plain_append(st)
        fp8 = torch.float8_e4m3fn
        return [q, st["k_codes"].view(fp8), st["v_codes"].view(fp8), st["k_scale"], st["v_scale"]]
    if own:
        return st["lib"].kv_attention(st["q"], st["cache"], st["q_start"], st["lengths"], st["table"],
                                      window=st["case"]["window"], workspace=st["ws"])
    return _plain_attend(st)


# ---------------------------------------------------------------- cost


def _seen(n, length, window):
    """Keys that the n rows of a sequence see together."""
    if not window:
        return n * length - n * (n - 1) // 2
    return sum(min(window, length - n + i + 1) for i in range(n))


def work(case):
    c = case
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    seqs = _sequences(c)
    T = sum(n for n, _ in seqs)
    if c["op"] == "append":
        return {"bytes": T * D * (4 * Hq + 6 * Hkv) + 4 * T * c["rope"], "flops": 6 * T * c["rope"] * (Hq + Hkv)}
    keys = sum(min(length, c["window"] + n - 1) if c["window"] else length for n, length in seqs)
    pairs = sum(_seen(n, length, c["window"]) for n, length in seqs)
    return {"bytes": 2 * keys * Hkv * D + 4 * T * Hq * D, "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------- 64 bits


def _e4m3_values():
    c = torch.arange(256)
    man, ex = (c & 7).double(), (c >> 3) & 15
    v = torch.where(ex > 0, (1 + man / 8) * 2.0 ** (ex - 7).double(), man / 8 * 2.0**-6)
    return torch.where(c >= 128, -v, v).cuda()


def _e4m3_round(v):
    """The E4M3 value nearest to each v (binary64), ties to the even mantissa."""
    m, e = torch.frexp(v.abs())
    step = _power((e - 1).clamp(min=-6) - 3)
    return torch.sign(v) * (torch.round(v.abs() / step) * step).clamp(max=E4M3_MAX)


def _exact_append(st):
    c = st["case"]
    P, rope, val = c["page"], c["rope"], _e4m3_values()
    k, v = val[st["k_codes"].long()], val[st["v_codes"].long()]
    ks, vs = st["k_scale"].double(), st["v_scale"].double()
    table = st["table"].tolist()
    turn = None
    if rope:
        half = rope // 2
        turn = torch.complex(*(st["rope"][:, i * half:(i + 1) * half].double() for i in (0, 1)))

    def rotated(x, pos):
        x = x.double()
        if turn is None:
            return x
        y, part = x.clone(), x[..., :rope]
        a, b = (part[..., ::2], part[..., 1::2]) if c["pairs"] else (part[..., : rope // 2], part[..., rope // 2:])
        z = torch.complex(a.contiguous(), b.contiguous()) * turn[pos][:, None]
        if c["pairs"]:
            y[..., 0:rope:2], y[..., 1:rope:2] = z.real, z.imag
        else:
            y[..., : rope // 2], y[..., rope // 2: rope] = z.real, z.imag
        return y

    qs, row = [], 0
    for b, (n, length) in enumerate(st["seqs"]):
        pos = torch.arange(length - n, length, device="cuda")
        qs.append(rotated(st["q"][row:row + n], pos))
        for codes, scales, x in ((k, ks, rotated(st["k"][row:row + n], pos)), (v, vs, st["v"][row:row + n].double())):
            for page in range((length - n) // P, (length - 1) // P + 1):
                lo, hi = max(page * P, length - n), min(page * P + P, length)
                part, p, held = x[lo - length + n:hi - length + n], table[b][page], lo - page * P
                s = _power(_exponent(part.abs().amax((0, 2))))
                if held:
                    s = torch.maximum(s, scales[p])
                    codes[p, :, :held] = _e4m3_round(codes[p, :, :held] * (scales[p] / s)[:, None, None])
                codes[p, :, held:hi - page * P] = _e4m3_round(part / s[:, None]).transpose(0, 1)
                scales[p] = s
        row += n
    return [torch.cat(qs), k, v, ks, vs]


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "append":
        return _exact_append(st)
    Hkv, P, val = c["Hkv"], c["page"], _e4m3_values()
    group = c["Hq"] // Hkv
    out, row = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda"), 0
    for b, (n, length) in enumerate(st["seqs"]):
        pages = st["table"][b, : -(-length // P)].long()
        past = (torch.arange(length, device="cuda")[None] - torch.arange(length - n, length, device="cuda")[:, None])
        hidden = past > 0
        if c["window"]:
            hidden |= past <= -c["window"]
        for h in range(Hkv):
            k = (val[st["k_codes"][pages, h].long()] * st["k_scale"][pages, h].double()[:, None, None]).flatten(0, 1)
            v = (val[st["v_codes"][pages, h].long()] * st["v_scale"][pages, h].double()[:, None, None]).flatten(0, 1)
            for j in range(h * group, (h + 1) * group):
                s = st["q"][row:row + n, j].double() @ k[:length].T / c["D"] ** 0.5
                out[row:row + n, j] = torch.softmax(s.masked_fill(hidden, -math.inf), 1) @ v[:length]
        row += n
    return out
