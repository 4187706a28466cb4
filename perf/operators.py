"""Measured cases of the block-scaled FP8 operators and of the norms around a block.

Three operators, each reached through ``w8a8_quantised_moe_gb300``:

* ``fp8_block_linear``: y = x W^T with E4M3 operands, one scale for each token and 128
  input channels of x (found in the call) and one for each 128 x 128 block of W;
* ``fp8_block_forward``: the whole mixture-of-experts layer (router, top-k, both expert
  products with the SiLU gate, combine) with that quantisation;
* ``norm_residual``: x' = x + scale * gate * rms_norm(branch) * post_w and
  rms_norm(x') * pre_w, the norms after one block and before the next.

``run`` computes them either in plain 32-bit torch operations (``own`` false) or by the
framework's calls (``own`` true); ``exact`` computes them in 64 bits from the definition.
"""
import math

import torch

own = False

BLOCK = 128  # input channels, and output channels of a weight, that share a scale
E4M3_MAX = 448.0
EPS = 1e-6
OUTLIER_GAIN = 20.0  # 1 % of the hidden channels carry activations this much larger
GAP = 1e-3  # the logits that decide the choice of experts differ by more than this

GATES = ("none", "channel", "token", "element")


def listed():
    return [
        # one token through a square projection: a decode step of one sequence
        {"name": "linear_one_token", "op": "linear", "M": 1, "N": 4096, "K": 4096},
        # a decode step of a batch of 64 sequences
        {"name": "linear_decode", "op": "linear", "M": 64, "N": 4096, "K": 4096},
        # a prompt of odd length, and both dimensions ending inside a scale block
        {"name": "linear_ragged", "op": "linear", "M": 1003, "N": 2064, "K": 1488},
        # the framework's linear layer: a prompt chunk of 4096 tokens
        {"name": "linear_prompt", "op": "linear", "M": 4096, "N": 4096, "K": 4096},
        # one token through the layer of 64 experts: the latency of a decode step
        {"name": "moe_one_token", "op": "moe", "T": 1, "H": 4096, "I": 1536, "E": 64, "k": 2, "bias": "none"},
        # the framework's decode layer: 64 sequences
        {"name": "moe_decode", "op": "moe", "T": 64, "H": 4096, "I": 1536, "E": 64, "k": 2, "bias": "none"},
        # few experts, an odd number of tokens, widths that are odd multiples of 128
        {"name": "moe_ragged", "op": "moe", "T": 333, "H": 1408, "I": 640, "E": 7, "k": 3, "bias": "normal"},
        # the framework's prompt layer: 8192 tokens, a few experts take most of them
        {"name": "moe_prompt", "op": "moe", "T": 8192, "H": 4096, "I": 1536, "E": 64, "k": 2, "bias": "zipf"},
        # the framework's layer of 256 experts
        {"name": "moe_wide", "op": "moe", "T": 4096, "H": 7168, "I": 2048, "E": 256, "k": 8, "bias": "normal"},
        # the norms around the blocks of one decoded token
        {"name": "norm_one_token", "op": "norm", "T": 1, "H": 4096, "residual": "bf16", "branch": True,
         "post": True, "gate": "none"},
        # an odd length and width, the residual kept in 32 bits, one gate value a token
        {"name": "norm_ragged", "op": "norm", "T": 1003, "H": 2056, "residual": "fp32", "branch": True,
         "post": True, "gate": "token"},
        # a prompt of 8192 tokens with a gate for every channel
        {"name": "norm_prompt", "op": "norm", "T": 8192, "H": 4096, "residual": "bf16", "branch": True,
         "post": True, "gate": "channel"},
    ]


def _size(rng, lo, hi, step=1):
    """A power of two, or an odd multiple of step, spread over the logarithm of [lo, hi]."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    if rng.random() < 0.4:
        return max(1 << math.ceil(math.log2(lo)), 1 << int(math.log2(v)))
    return max(step, (int(v) // step - 1 | 1) * step)


def draw(rng):
    op = rng.choice(("linear", "moe", "norm"))
    if op == "linear":
        return {"op": op, "M": _size(rng, 1, 4096), "N": _size(rng, 112, 4096, 16), "K": _size(rng, 112, 4096, 16)}
    if op == "norm":
        branch = rng.random() < 0.8
        return {"op": op, "T": _size(rng, 1, 8192), "H": _size(rng, 64, 4096, 8),
                "residual": rng.choice(("bf16", "fp32")), "branch": branch, "post": branch and rng.random() < 0.7,
                "gate": rng.choice(GATES) if branch else "none"}
    E = _size(rng, 2, 256)
    return {"op": op, "T": _size(rng, 1, 4096), "H": _size(rng, 256, 7168, 128),
            "I": _size(rng, 128, 2048, 128), "E": E, "k": rng.randint(1, min(8, E)),
            "bias": rng.choice(("none", "normal", "zipf"))}


# ---------------------------------------------------------------- inputs


def _activations(g, T, H):
    x = torch.randn(T, H, generator=g, device="cuda")
    loud = torch.randperm(H, generator=g, device="cuda")[: max(1, H // 100)]
    x[:, loud] *= OUTLIER_GAIN
    return x.bfloat16(), loud


def _quantized_weight(w):
    """E4M3 codes (bytes) and one scale for each 128 x 128 block of w [N, K]."""
    N, K = w.shape
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    tiles = torch.nn.functional.pad(w, (0, kb * BLOCK - K, 0, nb * BLOCK - N)).view(nb, BLOCK, kb, BLOCK)
    s = tiles.abs().amax((1, 3)) / E4M3_MAX
    q = (tiles / s[:, None, :, None]).to(torch.float8_e4m3fn).view(nb * BLOCK, kb * BLOCK)[:N, :K]
    return q.contiguous().view(torch.uint8), s


def _zipf_bias(logits, k, E, g):
    share = torch.arange(1, E + 1, device="cuda", dtype=torch.float64) ** -1.2
    share = (share / share.sum())[torch.randperm(E, generator=g, device="cuda")]
    b = torch.zeros(E, device="cuda", dtype=torch.float64)
    for _ in range(60):
        top = (logits + b).topk(k, dim=1).indices
        got = torch.bincount(top.flatten(), minlength=E).clamp(min=0.5) / top.numel()
        b += 0.3 * (share.log() - got.log())
        b -= b.mean()
    return b.float()


def _prepare_moe(c, g):
    T, H, I, E, k = (c[n] for n in ("T", "H", "I", "E", "k"))
    x, loud = _activations(g, T, H)
    var = (H - len(loud)) + len(loud) * OUTLIER_GAIN**2
    router_w = torch.randn(H, E, generator=g, device="cuda") / math.sqrt(var)
    bias = None
    if c["bias"] == "normal":
        bias = 0.5 * torch.randn(E, generator=g, device="cuda")
    elif c["bias"] == "zipf":
        bias = _zipf_bias(x.double() @ router_w.double(), k, E, g)
    rows = torch.arange(T, device="cuda")  # tokens whose choice of experts could hang on rounding are drawn again
    while k < E and len(rows):
        logits = x[rows].double() @ router_w.double()
        top = (logits if bias is None else logits + bias.double()).topk(k + 1, dim=1).values
        rows = rows[top[:, k - 1] - top[:, k] <= GAP]
        again = torch.randn(len(rows), H, generator=g, device="cuda")
        again[:, loud] *= OUTLIER_GAIN
        x[rows] = again.bfloat16()
    w13 = torch.empty(E, 2 * I, H, dtype=torch.uint8, device="cuda")
    s13 = torch.empty(E, 2 * I // BLOCK, H // BLOCK, device="cuda")
    w2 = torch.empty(E, H, I, dtype=torch.uint8, device="cuda")
    s2 = torch.empty(E, H // BLOCK, I // BLOCK, device="cuda")
    for e in range(E):
        w13[e], s13[e] = _quantized_weight(0.02 * torch.randn(2 * I, H, generator=g, device="cuda"))
        w2[e], s2[e] = _quantized_weight(0.02 * torch.randn(H, I, generator=g, device="cuda"))
    return {"x": x, "router_w": router_w, "bias": bias, "w13": w13, "s13": s13, "w2": w2, "s2": s2, "k": k}


def _prepare_norm(c, g):
    T, H = c["T"], c["H"]
    x, _ = _activations(g, T, H)
    st = {"x": x.float() + 1e-3 * torch.randn(T, H, generator=g, device="cuda") if c["residual"] == "fp32" else x,
          "branch": None, "post_w": None, "gate": None, "scale": 0.5,
          "pre_w": (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).bfloat16()}
    if c["branch"]:
        st["branch"] = (3 * torch.randn(T, H, generator=g, device="cuda")).bfloat16()
    if c["post"]:
        st["post_w"] = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).bfloat16()
    shape = {"none": None, "channel": (H,), "token": (T, 1), "element": (T, H)}[c["gate"]]
    if shape is not None:
        st["gate"] = torch.rand(shape, generator=g, device="cuda").bfloat16()
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "linear":
        x, _ = _activations(g, case["M"], case["K"])
        w_q, w_s = _quantized_weight(0.02 * torch.randn(case["N"], case["K"], generator=g, device="cuda"))
        st = {"x": x, "w_q": w_q, "w_s": w_s}
    elif case["op"] == "moe":
        st = _prepare_moe(case, g)
    else:
        st = _prepare_norm(case, g)
    st["op"] = case["op"]
    if own:  # a serving loop keeps its workspace from call to call
        import w8a8_quantised_moe_gb300 as moe

        st["lib"] = moe
        if case["op"] == "linear":
            st["ws"] = moe.new_workspace(moe.fp8_block_linear_workspace_size(case["M"], case["N"], case["K"]))
        elif case["op"] == "moe":
            st["ws"] = moe.new_workspace(
                moe.fp8_block_workspace_size(case["T"], case["H"], case["I"], case["E"], case["k"]))
    return st


# ---------------------------------------------------------------- one pass


def _quantized_tokens(x):
    """x [T, K] rounded to E4M3 with one scale for each token and 128 channels, as fp32 values."""
    T, K = x.shape
    kb = -(-K // BLOCK)
    xb = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - K)).view(T, kb, BLOCK)
    s = xb.abs().amax(-1, keepdim=True) / E4M3_MAX
    q = torch.where(s == 0, 0.0, xb / s).to(torch.float8_e4m3fn).float()
    return (q * s).view(T, kb * BLOCK)[:, :K]


def _weight_values(w_q, w_s):
    N, K = w_q.shape
    s = w_s.repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    return w_q.view(torch.float8_e4m3fn).float() * s


def _plain_linear(st):
    return (_quantized_tokens(st["x"]) @ _weight_values(st["w_q"], st["w_s"]).T).bfloat16()


def _plain_moe(st):
    x, k = st["x"], st["k"]
    logits = x.float() @ st["router_w"]
    if st["bias"] is not None:
        logits = logits + st["bias"]
    top, ids = logits.sort(dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    w = torch.exp(top - top[:, :1])
    w = w / w.sum(1, keepdim=True)
    xq = _quantized_tokens(x)
    slots = ids.flatten().sort(stable=True).indices  # (token, choice) pairs, expert by expert
    o = torch.empty(x.shape[0] * k, x.shape[1], device=x.device)
    counts = torch.bincount(ids.flatten(), minlength=st["w13"].shape[0]).tolist()
    for e, rows in enumerate(slots.split(counts)):
        if len(rows):
            gate, up = (xq[rows // k] @ _weight_values(st["w13"][e], st["s13"][e]).T).chunk(2, dim=1)
            h = gate / (1 + torch.exp(-gate)) * up
            o[rows] = _quantized_tokens(h) @ _weight_values(st["w2"][e], st["s2"][e]).T
    return (o.view(-1, k, x.shape[1]) * w[:, :, None]).sum(1).bfloat16()


def _plain_norm(st):
    r = st["x"].float()
    if st["branch"] is not None:
        b = st["branch"].float()
        if st["post_w"] is not None:
            b = b * torch.rsqrt((b * b).mean(1, keepdim=True) + EPS) * st["post_w"].float()
        if st["gate"] is not None:
            b = b * st["gate"].float()
        r = r + st["scale"] * b
    n = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * st["pre_w"].float()
    return [r.to(st["x"].dtype), n.bfloat16()]


def run(state):
    st = state
    if not own:
        return {"linear": _plain_linear, "moe": _plain_moe, "norm": _plain_norm}[st["op"]](st)
    moe = st["lib"]
    if st["op"] == "linear":
        return moe.fp8_block_linear(st["x"], st["w_q"], st["w_s"], workspace=st["ws"])
    if st["op"] == "moe":
        return moe.fp8_block_forward(st["x"], st["router_w"], st["bias"], st["w13"], st["s13"], st["w2"], st["s2"],
                                     st["k"], workspace=st["ws"])
    return list(moe.norm_residual(st["x"], st["branch"], post_w=st["post_w"], gate=st["gate"], scale=st["scale"],
                                  pre_w=st["pre_w"], eps=EPS))


# ---------------------------------------------------------------- cost


def _touched(c):
    """Experts that receive a token, on average."""
    T, E, k = c["T"], c["E"], c["k"]
    share = [(i + 1) ** -1.2 for i in range(E)] if c["bias"] == "zipf" else [1.0] * E
    total = sum(share)
    return sum(1 - (1 - min(1.0, k * s / total)) ** T for s in share)


def work(case):
    c = case
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        scales = 4 * -(-N // BLOCK) * -(-K // BLOCK)
        return {"bytes": N * K + scales + 2 * M * K + 2 * M * N, "flops": 2 * M * N * K}
    if c["op"] == "moe":
        T, H, I, E, k = (c[n] for n in ("T", "H", "I", "E", "k"))
        expert = 3 * H * I + 4 * 3 * H * I // BLOCK**2
        return {"bytes": _touched(c) * expert + 4 * H * E + 4 * T * H, "flops": 2 * T * H * E + 6 * T * k * H * I}
    T, H = c["T"], c["H"]
    per = (4 if c["residual"] == "fp32" else 2) * (2 if c["branch"] else 1)
    per += 2 + (2 if c["branch"] else 0) + (2 if c["gate"] == "element" else 0)
    row = 2 * H * (1 + c["post"] + (c["gate"] == "channel")) + (2 * T if c["gate"] == "token" else 0)
    return {"bytes": T * H * per + row, "flops": 12 * T * H}


# ---------------------------------------------------------------- 64 bits


def _e4m3(v):
    """The E4M3 value nearest to each v (binary64), ties to the even mantissa, saturated."""
    m, e = torch.frexp(v.abs())  # |v| = m 2^e, m in [1/2, 1): the leading bit stands for 2^(e-1)
    step = torch.ldexp(torch.ones_like(m), (e - 1).clamp(min=-6) - 3)
    return torch.sign(v) * (torch.round(v.abs() / step) * step).clamp(max=E4M3_MAX)


def _exact_rows(x):
    """Rows of fp32 values to what their codes stand for; the scale and the quotient that is
    rounded are binary32 by the definition of the codes."""
    out = torch.zeros_like(x, dtype=torch.float64)
    for at in range(0, x.shape[1], BLOCK):
        part = x[:, at:at + BLOCK]
        s = part.abs().max(dim=1, keepdim=True).values / E4M3_MAX
        code = _e4m3(torch.where(s > 0, part / torch.where(s > 0, s, 1.0), 0.0).double())
        out[:, at:at + BLOCK] = code * s.double()
    return out


def _e4m3_table():
    c = torch.arange(256)
    man, ex = (c & 7).double(), (c >> 3) & 15
    v = torch.where(ex > 0, (1 + man / 8) * 2.0 ** (ex - 7).double(), man / 8 * 2.0**-6)
    return torch.where(c >= 128, -v, v)


def _exact_weight(codes, scales):
    v = _e4m3_table().to(codes.device)[codes.to(torch.int64)]
    for i in range(scales.shape[0]):
        row = torch.repeat_interleave(scales[i].double(), BLOCK)[: v.shape[1]]
        v[i * BLOCK:(i + 1) * BLOCK] *= row
    return v


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "linear":
        return _exact_rows(st["x"].float()) @ _exact_weight(st["w_q"], st["w_s"]).T
    if case["op"] == "norm":
        x = st["x"].double()
        if case["branch"]:
            b = st["branch"].double()
            if case["post"]:
                b = b / torch.sqrt(b.square().sum(1, keepdim=True) / b.shape[1] + EPS) * st["post_w"].double()
            g = 1.0 if st["gate"] is None else st["gate"].double()
            x = x + st["scale"] * g * b
        n = x / torch.sqrt(x.square().sum(1, keepdim=True) / x.shape[1] + EPS) * st["pre_w"].double()
        return [x, n]
    x, k, E = st["x"], case["k"], case["E"]
    logits = x.double() @ st["router_w"].double() + (0.0 if st["bias"] is None else st["bias"].double())
    top, ids = logits.topk(k, dim=1)
    weight = torch.softmax(top, dim=1)
    xq = _exact_rows(x.float())
    y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if len(t) == 0:
            continue
        a = xq[t] @ _exact_weight(st["w13"][e], st["s13"][e]).T
        g, u = a[:, : case["I"]], a[:, case["I"]:]
        h = (g / (1 + torch.exp(-g)) * u).float()  # h is quantised from its binary32 value
        y[t] += weight[t, j, None] * (_exact_rows(h) @ _exact_weight(st["w2"][e], st["s2"][e]).T)
    return y
