"""Plain 64-bit forms of the block-scaled FP8 operators and of the norms around a
block, for the tests.  A block's scale and the quotient that is rounded to a code
are binary32 by the operators' definition; everything else is binary64."""
import torch

BLOCK = 128
RECIPROCAL = torch.tensor(1.0) / torch.tensor(448.0)  # binary32


def blocks(n):
    return -(-n // BLOCK)


def e4m3_values():
    """The 256 E4M3 values by code (binary64)."""
    c = torch.arange(256)
    man, ex = (c % 8).double(), c // 8 % 16
    v = torch.where(ex == 0, man * 2.0**-9, (8 + man) * torch.exp2((ex - 10).double()))
    v[127] = v[255] = float("nan")
    return torch.where(c < 128, v, -v)


def e4m3_codes(q):
    """Codes of binary32 values |q| <= 448 (1 + 2^-22): nearest, ties to the even mantissa."""
    v = q.double().abs()
    table = e4m3_values()[:127].to(v.device)  # ascending; the largest is 448
    hi = torch.searchsorted(table, v.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = table[hi] - v, v - table[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code + 128 * torch.signbit(q)).to(torch.uint8)


def quantize_rows(x):
    """bf16 or fp32 x [M, K] -> (codes [M, K], scales fp32 [M, blocks])."""
    x = x.float()
    M, K = x.shape
    codes = torch.empty(M, K, dtype=torch.uint8, device=x.device)
    scales = torch.empty(M, blocks(K), device=x.device)
    for b in range(blocks(K)):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        s = part.abs().amax(1) * RECIPROCAL.to(x.device)
        q = part / torch.where(s == 0, 1.0, s)[:, None]
        codes[:, b * BLOCK:(b + 1) * BLOCK] = torch.where((s == 0)[:, None], 0, e4m3_codes(q).int()).to(torch.uint8)
        scales[:, b] = s
    return codes, scales


def quantize_weight(w):
    """fp32 w [N, K] -> (codes [N, K], scales fp32 [blocks(N), blocks(K)])."""
    N, K = w.shape
    codes = torch.empty(N, K, dtype=torch.uint8, device=w.device)
    scales = torch.empty(blocks(N), blocks(K), device=w.device)
    for i in range(blocks(N)):
        for j in range(blocks(K)):
            at = (slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK))
            s = w[at].abs().max() * RECIPROCAL.to(w.device)
            codes[at] = e4m3_codes(w[at] / s) if s != 0 else 0
            scales[i, j] = s
    return codes, scales


def row_values(codes, scales):
    v = e4m3_values().to(codes.device)[codes.long()]
    return v * scales.double().repeat_interleave(BLOCK, 1)[:, : v.shape[1]]


def weight_values(codes, scales):
    v = e4m3_values().to(codes.device)[codes.long()]
    s = scales.double().repeat_interleave(BLOCK, 0)[: v.shape[0]]
    return v * s.repeat_interleave(BLOCK, 1)[:, : v.shape[1]]


def linear(x, w_q, w_s):
    """(x W^T, sum of the magnitudes of its terms), both binary64."""
    a, w = row_values(*quantize_rows(x)), weight_values(w_q, w_s)
    return a @ w.T, a.abs() @ w.abs().T


def moe(x, router_w, bias, w13, s13, w2, s2, k):
    logits = x.double() @ router_w.double()
    if bias is not None:
        logits = logits + bias.double()
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    weight = torch.softmax(top, 1)
    I = w2.shape[2]
    xq = row_values(*quantize_rows(x))
    y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for e in range(w2.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if len(t):
            a = xq[t] @ weight_values(w13[e], s13[e]).T
            h = (a[:, :I] * torch.sigmoid(a[:, :I]) * a[:, I:]).float()
            y[t] += weight[t, j, None] * (row_values(*quantize_rows(h)) @ weight_values(w2[e], s2[e]).T)
    return y


def norm_residual(x, branch, post_w, gate, scale, pre_w, eps):
    """(r, n, magnitude of what is added to x), binary64."""
    r, added = x.double(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    if branch is not None:
        b = branch.double()
        if post_w is not None:
            b = b / torch.sqrt(b.pow(2).mean(1, keepdim=True) + eps) * post_w.double()
        added = scale * (1.0 if gate is None else gate.double()) * b
        r = r + added
    n = None if pre_w is None else r / torch.sqrt(r.pow(2).mean(1, keepdim=True) + eps) * pre_w.double()
    return r, n, added.abs()
