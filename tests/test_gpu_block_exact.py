"""The block-scaled layer on inputs whose every intermediate is exact up to the codes
of h, so that y shows each code: one nonzero product a sum in the second product, a
weight of one per token, and gates where silu is exact in binary32."""
import pytest
import torch

import block_reference as ref
import w8a8_quantised_moe_gb300 as moe

pytestmark = pytest.mark.gpu

H, I = 256, 256
ONE = 0x38  # E4M3 code of 1.0
UP = 2.0**60  # scale of the second product's unit weights: small h become normal numbers of y


class ExactLayer:
    """h[t][n] = silu(gate_t * |c|) * p_t * u for values[expert of t][n] = c * u, exactly.

    values: integers, products of a c of 1..15 (a weight of the gate row) and a u of
    -255..255 (16 hi + lo in two weights of the up row).  p_t: a power of two, at least 1
    with a gate of 32 p_t (1 + exp(-32) rounds to 1, so silu(g) = g), or below 2^-30
    with a gate of p_t (1 + exp(-g) rounds to 2, so silu(g) = g / 2)."""

    def __init__(self, values, p):
        E, T = len(values), len(p)
        v = torch.tensor(values)
        c = torch.ones_like(v)
        for d in range(2, 16):
            c = torch.where((v.abs() > 255 * c) & (v % d == 0), d, c)
        u = v // c
        assert v.shape == (E, I) and u.abs().max() <= 255
        codes = ref.e4m3_codes(torch.arange(16).float()).int()
        sign = 128 * (u < 0)
        w13 = torch.zeros(E, 2 * I, H, dtype=torch.uint8)
        w13[:, :I, 2] = codes[c].to(torch.uint8)
        w13[:, I:, 0] = (codes[u.abs() // 16] + sign * (u.abs() >= 16)).to(torch.uint8)
        w13[:, I:, 1] = (codes[u.abs() % 16] + sign * (u.abs() % 16 > 0)).to(torch.uint8)
        w2 = torch.zeros(E, H, I, dtype=torch.uint8)
        w2[:, torch.arange(H), torch.arange(H)] = ONE
        p = torch.tensor(p, dtype=torch.float64)
        assert ((p >= 1) | (p < 2.0**-30)).all()
        gate = torch.where(p >= 1, 32 * p, p)
        self.e = torch.arange(T) % E
        x = torch.zeros(T, H, dtype=torch.float64)
        x[:, 0], x[:, 1], x[:, 2], x[:, 3] = 16 * p, p, gate, 448 * p  # the scale of this block is p
        x[torch.arange(T), 128 + self.e] = p  # the router's choice
        router_w = torch.zeros(H, E)
        router_w[128 + torch.arange(E), torch.arange(E)] = 1
        self.h = (torch.where(p >= 1, gate, gate / 2) * p)[:, None] * v[self.e].double()
        assert torch.equal(self.h.float().double(), self.h)
        self.args = tuple(t.cuda() if t is not None else None for t in (
            x.bfloat16(), router_w, None, w13, torch.ones(E, 2 * I // 128, H // 128), w2,
            torch.full((E, H // 128, I // 128), UP))) + (1,)
        assert torch.equal(x.bfloat16().double(), x)

    def codes(self):
        """Codes [T, I] of h and the value that each stands for in y."""
        code, s = ref.quantize_rows(self.h.float())
        return code, ref.e4m3_values()[code.long()] * s.double().repeat_interleave(128, 1) * UP

    def check(self):
        y = moe.fp8_block_forward(*self.args).double().cpu()
        _, want = self.codes()
        # neighbouring codes are at least 2^-4 of each other apart; y is rounded to bf16's 2^-8
        bad = (y - want).abs() > 2.0**-7 * want.abs()
        bad |= ~y.isfinite()
        assert not bad.any(), (bad.sum().item(), y[bad][:4], want[bad][:4])


# tokens, experts: the form for a few tokens, few rows an expert, many rows
FORMS = [(7, 2), (40, 20), (300, 2)]


def random_values(E, seed):
    g = torch.Generator().manual_seed(seed)
    v = torch.randint(-255, 256, (E, I), generator=g)
    v[:, ::5] = 0  # channels that are exactly zero
    v[:, 128:] = v[:, 128:] // 16  # a block of smaller values
    return v.tolist()


@pytest.mark.parametrize("T,E", FORMS)
def test_codes_of_h_over_the_range_of_binary32(T, E):
    """Rows whose h reaches from binary32's smallest subnormal to 2^22."""
    powers = [2.0**e for e in (-74, -72, -70, -67, -66, -65, -64, -63, -62, -60, -58, -50, -32, 0, 4)]
    ExactLayer(random_values(E, T), [powers[(4 * t) % len(powers)] for t in range(T)]).check()


@pytest.mark.parametrize("T,E", FORMS)
def test_codes_of_h_next_to_midpoints(T, E):
    """Quotients so near the midpoint of two codes that a product with the rounded
    reciprocal of the scale lands on its other side: block maximum, and values under it."""
    near = [(868, [837]), (1148, [1107]), (1540, [1045, 1265, 1485]), (1736, [837, 1674]), (2296, [1107, 2214]),
            (2324, [2241]), (3080, [1045, 1265, 1485, 2090, 2530, 2970]), (3388, [2299]), (3472, [837, 1674])]
    blocks = [[top, *v, *(-i for i in v)] + [0] * (127 - 2 * len(v)) for top, v in near]
    layer = ExactLayer([blocks[2 * e % 9] + blocks[(2 * e + 1) % 9] for e in range(E)], [1.0] * T)
    h = layer.h.float().reshape(T, 2, 128)
    product = h * (1 / (h.abs().amax(2) * ref.RECIPROCAL))[:, :, None]
    assert (ref.e4m3_codes(product.reshape(T, I).clamp(-448, 448)) != layer.codes()[0]).sum() >= 2 * T
    layer.check()


# ---------------------------------------------------------------- rows between the product and the combine


def set_rows(layer, rows, scale):
    """Rows of the second product's weights {column: {channel: weight}}, each an E4M3 value."""
    w2 = torch.zeros(H, I, dtype=torch.uint8)
    for c, row in rows.items():
        for n, w in row.items():
            w2[c, n] = ref.e4m3_codes(torch.tensor(w))
    layer.args[5][:] = w2.cuda()
    layer.args[6][:] = scale


@pytest.mark.parametrize("T,E", FORMS)
def test_rows_are_rounded_once(T, E):
    """257 + 2^-6 lies above the midpoint of bf16's 256 and 258, 259 - 2^-6 below that of 258
    and 260; 11 bits in between would take each to the midpoint and then to the other neighbour."""
    layer = ExactLayer([[448, 256, 1, -1] + [0] * (I - 4)] * E, [1.0] * T)
    up, down = {1: 1.0, 2: 1.0, 3: -(2.0**-6)}, {1: 1.0, 2: 3.0, 3: 2.0**-6}
    set_rows(layer, {c: (up, down)[c % 2] for c in range(H)}, 1.0 / 32)  # h = 32 * values
    y = moe.fp8_block_forward(*layer.args).float().cpu()
    assert (y[:, ::2] == 258).all() and (y[:, 1::2] == 258).all()


@pytest.mark.parametrize("T,E", FORMS)
def test_an_infinite_sum_leaves_its_neighbours(T, E):
    """One column's sum passes binary32's range; the others of its 128 stay what they are."""
    layer = ExactLayer([[448, 1, 7] + [0] * (I - 3)] * E, [1.0] * T)
    rows = {c: {1: 1.0} if c % 3 else {2: 1.0} for c in range(H)}
    rows[5] = {0: 448.0, 1: 448.0, 2: 448.0}
    set_rows(layer, rows, 2.0**112 / 32)
    y = moe.fp8_block_forward(*layer.args).double().cpu()
    want = torch.where(torch.arange(H) % 3 == 0, 7.0, 1.0).double() * 2.0**112
    want[5] = float("inf")
    assert torch.equal(y, want.expand(T, H))


# ---------------------------------------------------------------- far negative gates


def gate_blocks(n_blocks, seed):
    """Blocks of (gate in quarters, up) for 128 channels, the first the largest h, whose quotients lie
    2^-19 to 2^-17.5 from a midpoint of two codes (relatively), far enough for the error below."""
    g = torch.Generator().manual_seed(seed)
    quarters, ups = torch.arange(200, 241).double(), torch.arange(1, 256).double()
    h = (quarters / -4 / (1 + torch.exp(quarters / 4)))[:, None] * ups
    v = ref.e4m3_values()[:127]
    mids = ((v[:-1] + v[1:]) / 2)[16:]
    blocks = []
    while len(blocks) < n_blocks:
        i, j = (torch.randint(0, n, (1,), generator=g).item() for n in h.shape)
        s = h[i, j].abs().float() * ref.RECIPROCAL
        q = h.abs() / s.double()
        at = torch.searchsorted(mids, q.contiguous()).clamp(1, len(mids) - 1)
        off = torch.minimum((q / mids[at] - 1).abs(), (q / mids[at - 1] - 1).abs())
        near = ((h.abs() < h[i, j].abs()) & (off > 2.0**-19) & (off < 2.0**-17.5)).nonzero()
        if len(near) >= 3:
            picked = [(i, j)] + [tuple(r) for r in near[:127].tolist()]
            blocks.append([(int(quarters[a]), int(ups[b])) for a, b in picked])
    return blocks


@pytest.mark.parametrize("T,E", FORMS)
def test_codes_of_h_for_far_negative_gates(T, E):
    """Gates of -50 to -60.  h is within 5 * 2^-23 of its value: expf within 2 units in the last
    place, the sum half a unit, the quotient 2 and the product half; its block's maximum
    likewise, the scale and the quotient by it half a unit each: under 2^-19 together."""
    layer = ExactLayer([[0] * I] * E, [1.0] * T)
    w13, x = layer.args[3], layer.args[0]
    codes = ref.e4m3_codes(torch.arange(16).float())
    blocks = gate_blocks(2 * E, T)
    gate, up = torch.zeros(E, I, dtype=torch.long), torch.zeros(E, I, dtype=torch.long)
    for i, block in enumerate(blocks):
        at = slice(i % 2 * 128, i % 2 * 128 + len(block))
        gate[i // 2, at], up[i // 2, at] = torch.tensor(block).T
    x[:, 2], x[:, 4] = -4, -0.25
    w13[:, :I, 2], w13[:, :I, 4] = codes[gate // 16].cuda(), codes[gate % 16].cuda()
    w13[:, I:, 0], w13[:, I:, 1] = codes[up // 16].cuda(), codes[up % 16].cuda()
    layer.args[6][:] = 2.0**100
    g = gate.double() / -4
    layer.h = (g / (1 + torch.exp(-g)) * up.double())[layer.e]
    code, _ = layer.codes()
    y = moe.fp8_block_forward(*layer.args).double().cpu()
    s = layer.h.float().reshape(T, 2, 128).abs().amax(2) * ref.RECIPROCAL
    want = ref.e4m3_values()[code.long()] * s.double().repeat_interleave(128, 1) * 2.0**100
    assert (up > 0).sum() >= 8 * E
    assert ((y - want).abs() <= 2.0**-7 * want.abs()).all()


@pytest.mark.parametrize("T,E", FORMS)
def test_codes_of_h_where_the_exponential_nears_its_range(T, E):
    """Gates of -86 to -95, where exp(-g) passes 2^126 and then binary32's range.  exp(g) is
    subnormal there: an error of half 2^-149 of it, |g| times in silu's product, besides the
    6 * 2^-23 of h and of its block's maximum, and half a unit each for scale and quotient.
    Within that of a midpoint either code will do."""
    layer = ExactLayer([[0] * I] * E, [1.0] * T)
    w13, x = layer.args[3], layer.args[0]
    codes = ref.e4m3_codes(torch.arange(16).float())
    gen = torch.Generator().manual_seed(T)
    gate = torch.randint(344, 381, (E, I), generator=gen)
    up = torch.randint(0, 256, (E, I), generator=gen)
    # gate / -4 in three weights
    x[:, 2], x[:, 4], x[:, 5] = -64, -4, -0.25
    w13[:, :I, 2] = codes[gate // 256].cuda()
    w13[:, :I, 4], w13[:, :I, 5] = codes[gate // 16 % 16].cuda(), codes[gate % 16].cuda()
    w13[:, I:, 0], w13[:, I:, 1] = codes[up // 16].cuda(), codes[up % 16].cuda()
    layer.args[6][:] = 2.0**100
    g, u = gate.double() / -4, up.double()
    h = g / (1 + torch.exp(-g)) * u
    layer.h = h[layer.e]
    code, _ = layer.codes()
    s = (layer.h.float().reshape(T, 2, 128).abs().amax(2) * ref.RECIPROCAL).double().repeat_interleave(128, 1)
    q = layer.h / s
    slack = q.abs() * 13 * 2.0**-23 + ((u * (g.abs() + 2))[layer.e] * 2.0**-149) / s
    low, high = (ref.e4m3_values()[ref.e4m3_codes((q + d).clamp(-448, 448).float()).long()] for d in (-slack, slack))
    y = moe.fp8_block_forward(*layer.args).double().cpu() / 2.0**100 / s
    assert y.isfinite().all() and (code % 128 > 0).float().mean() > 0.5
    assert ((y >= low - 2.0**-7 * low.abs()) & (y <= high + 2.0**-7 * high.abs())).all()
