"""Block-scaled FP8 operators against their plain 64-bit forms."""
import pytest
import torch

import block_reference as ref
import w8a8_quantised_moe_gb300 as moe

pytestmark = pytest.mark.gpu

# Units: u = 2^-24 is binary32's roundoff and 2^-8 bf16's.
#   A product's block sum: the tensor cores' binary32 sum of exact products is
#   held to 2^-16 of the sum of magnitudes A, the bound of this layer's FP8
#   tests.  The scale product, and one multiply-add a block (up to 64 blocks
#   here): at most 66 u A < 2^-17 A.  The result is rounded to bf16 once.
SUM_REL = 2.0**-16 + 2.0**-17
BF16 = 2.0**-8
# The layer: the tolerance of its other forms (gpu_helpers), on the bf16 rounding of the 64-bit result.
Y_MAX_REL, Y_MEAN_REL = 1e-2, 2e-3


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def activations(g, M, K):
    x = torch.randn(M, K, generator=g, device="cuda")
    x[:, torch.randperm(K, generator=g, device="cuda")[: max(1, K // 100)]] *= 20
    return x.bfloat16()


def weight(g, *shape):
    return moe.fp8_block_quantize_weights(0.02 * torch.randn(*shape, generator=g, device="cuda"))


def check_linear(x, w_q, w_s, **kw):
    y = moe.fp8_block_linear(x, w_q, w_s, **kw)
    want, mag = ref.linear(x, w_q, w_s)
    err = (y.double() - want).abs()
    bound = SUM_REL * mag * (1 + BF16) + BF16 * want.abs() + 2.0**-134  # half of bf16's smallest value
    assert (err <= bound).all(), (err - bound).max().item()
    return y


@pytest.mark.parametrize("shape", [(16, 16), (128, 128), (144, 272), (2, 128, 256), (3, 256, 384), (1040, 1488)])
def test_weight_quantizer_is_exact(shape):
    g = gen(1)
    w = 0.02 * torch.randn(*shape, generator=g, device="cuda")
    w[..., :16, :16] *= 100
    if shape[-1] > 128:
        w[..., :128, 128:] = 0  # a block of zeros
    q, s = moe.fp8_block_quantize_weights(w)
    for i, wi in enumerate(w.reshape(-1, *shape[-2:])):
        rq, rs = ref.quantize_weight(wi)
        assert torch.equal(s.reshape(-1, *rs.shape)[i], rs)
        assert torch.equal(q.reshape(-1, *shape[-2:])[i], rq)


@pytest.mark.parametrize("M,K", [(1, 16), (5, 128), (9, 272), (130, 640), (300, 256)])
def test_activation_codes_are_exact(M, K):
    """Through unit weights the product returns each code times its scale."""
    g = gen(2)
    x = activations(g, M, K)
    x[:, K // 2] = 0
    if M > 4:
        x[3] = 0
        x[4] = (x[4].float() * 2.0**100).bfloat16()
        x[2] = (x[2].float() * 2.0**-100).bfloat16()
        # amax 7 * 2^j: the scale is a power of two to an ulp, so quotients fall on code midpoints
        x[1] = torch.randint(-112, 113, (K,), generator=g, device="cuda").bfloat16() / 16
        x[1, ::128] = 7.0
    w_q = torch.zeros(K, K, dtype=torch.uint8, device="cuda").fill_diagonal_(0x38)
    w_s = torch.ones(ref.blocks(K), ref.blocks(K), device="cuda")
    codes, scales = ref.quantize_rows(x)
    want = ref.row_values(codes, scales).float().bfloat16()
    assert torch.equal(moe.fp8_block_linear(x, w_q, w_s), want)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("N,K", [(16, 16), (144, 112), (384, 640), (272, 2064)])
def test_linear(M, N, K):
    g = gen(M * 7 + N)
    check_linear(activations(g, M, K), *weight(g, N, K))


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (3, 16, 8192), (8, 2064, 7184), (40, 1024, 4112), (1003, 528, 1488),
                                   (520, 4112, 144), (2100, 1040, 256),
                                   (16, 512, 16400), (100, 272, 8208), (128, 2064, 4096), (2, 128, 65536)])
def test_linear_long(M, N, K):
    g = gen(M + K)
    check_linear(activations(g, M, K), *weight(g, N, K))


@pytest.mark.parametrize("M", [1, 6, 200])
def test_linear_magnitudes(M):
    """Rows far apart in size, zero rows and weights with zero blocks."""
    g = gen(5)
    x = activations(g, M, 384)
    x *= torch.exp2(torch.randint(-60, 60, (M, 1), generator=g, device="cuda").float()).bfloat16()
    x[M // 2] = 0
    x[:, 128:256] = 0
    w = torch.randn(272, 384, generator=g, device="cuda")
    w[128:256] = 0
    w[:, :128] *= 1e-20
    y = check_linear(x, *moe.fp8_block_quantize_weights(w))
    assert not y[M // 2].any()


@pytest.mark.parametrize("M", [3, 150])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_non_finite_value_stays_in_its_row(M, bad):
    g = gen(6)
    x = activations(g, M, 512)
    w_q, w_s = weight(g, 256, 512)
    clean = moe.fp8_block_linear(x, w_q, w_s)
    x[1, 200] = bad
    y = moe.fp8_block_linear(x, w_q, w_s)
    assert y[1].isnan().all()
    keep = torch.arange(M) != 1
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("M,N,K", [(1, 4096, 1024), (20, 512, 2048), (700, 384, 640)])
def test_linear_repeats_bit_for_bit_and_ignores_old_workspace(M, N, K):
    g = gen(7)
    x, (w_q, w_s) = activations(g, M, K), weight(g, N, K)
    first = moe.fp8_block_linear(x, w_q, w_s)
    ws = moe.new_workspace(moe.fp8_block_linear_workspace_size(M, N, K))
    ws[256:] = 0xFF  # NaN codes and scales
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert moe.fp8_block_linear(x, w_q, w_s, workspace=ws, out=out) is out
    assert torch.equal(out, first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            y = moe.fp8_block_linear(x, w_q, w_s, workspace=ws)
    side.synchronize()
    assert torch.equal(y, first)
    assert moe.device_error(ws) == 0


def test_linear_in_a_graph():
    g = gen(8)
    x, (w_q, w_s) = activations(g, 5, 1024), weight(g, 1024, 1024)
    ws = moe.new_workspace(moe.fp8_block_linear_workspace_size(5, 1024, 1024))
    want = moe.fp8_block_linear(x, w_q, w_s, workspace=ws)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.fp8_block_linear(x, w_q, w_s, workspace=ws, out=out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_no_tokens():
    g = gen(9)
    w_q, w_s = weight(g, 128, 128)
    ws = moe.new_workspace(1024)
    y = moe.fp8_block_linear(torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"), w_q, w_s, workspace=ws)
    assert y.shape == (0, 128)


# ---------------------------------------------------------------- the layer


class Layer:
    def __init__(self, T, H, I, E, k, seed, bias=None, one_expert=False):
        g = gen(seed)
        self.k = k
        self.router_w = torch.randn(H, E, generator=g, device="cuda") / H**0.5
        self.bias = None
        if bias:
            self.bias = bias * torch.randn(E, generator=g, device="cuda")
        if one_expert:
            self.bias = torch.zeros(E, device="cuda")
            self.bias[E // 2] = 100
        self.x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
        rows = torch.arange(T, device="cuda")  # no choice of experts hangs on rounding
        while len(rows) and k < E:
            logits = self.x[rows].double() @ self.router_w.double()
            if self.bias is not None:
                logits += self.bias.double()
            top = logits.topk(k + 1, dim=1).values
            rows = rows[top[:, k - 1] - top[:, k] <= 1e-3]
            self.x[rows] = torch.randn(len(rows), H, generator=g, device="cuda").bfloat16()
        self.w13, self.s13 = weight(g, E, 2 * I, H)
        self.w2, self.s2 = weight(g, E, H, I)
        self.shape = (T, H, I, E, k)

    def args(self):
        return self.x, self.router_w, self.bias, self.w13, self.s13, self.w2, self.s2, self.k

    def check(self, y):
        want = ref.moe(*self.args())
        got, want = y.double(), want.bfloat16().double()
        assert (got - want).abs().max() <= Y_MAX_REL * want.abs().max()
        assert (got - want).abs().sum() <= Y_MEAN_REL * want.abs().sum()


LAYERS = [
    # T, H, I, E, k, bias
    (1, 128, 128, 1, 1, None), (1, 1408, 640, 9, 3, None), (2, 256, 128, 2, 2, None), (3, 512, 384, 256, 8, 0.5),
    (16, 256, 512, 8, 2, None), (33, 640, 256, 5, 1, None), (64, 1024, 512, 64, 2, None), (128, 384, 256, 4, 4, None),
    (129, 384, 256, 4, 4, None), (333, 1408, 640, 7, 3, 1.0), (700, 512, 1024, 3, 2, None),
    (1500, 256, 256, 40, 6, 0.7),
    # few tokens: up to 32 (token, choice) pairs, few and many tiles, shared experts
    (1, 4096, 256, 64, 8, None), (2, 512, 1408, 256, 8, None), (4, 1024, 384, 64, 8, 0.5), (8, 640, 256, 33, 4, None),
    (8, 2048, 1024, 6, 2, 1.0), (7, 16384, 128, 3, 3, None), (5, 128, 2048, 20, 1, None), (8, 256, 128, 64, 4, None),
    (9, 256, 128, 64, 3, None), (8, 256, 128, 40, 5, None),
]


@pytest.mark.parametrize("shape", LAYERS)
def test_layer(shape):
    layer = Layer(*shape[:5], seed=sum(shape[:5]), bias=shape[5])
    y = moe.fp8_block_forward(*layer.args())
    layer.check(y)
    ws = moe.new_workspace(moe.fp8_block_workspace_size(*layer.shape))
    for _ in range(2):  # the same bits from a workspace that has been used
        again = moe.fp8_block_forward(*layer.args(), workspace=ws)
        assert torch.equal(again, y)
        ws[256:] = 0xFF
    assert moe.device_error(ws) == 0


@pytest.mark.parametrize("T", [1, 40, 600])
def test_layer_with_every_token_at_one_expert(T):
    layer = Layer(T, 512, 256, 6, 1, seed=T, one_expert=True)
    layer.check(moe.fp8_block_forward(*layer.args()))


def test_layer_tokens_do_not_depend_on_their_neighbours():
    """A token's row is the same whatever else is in a batch of the same size."""
    layer = Layer(200, 512, 256, 8, 2, seed=4)
    y = moe.fp8_block_forward(*layer.args())
    layer.x[:100] = layer.x[100:]
    again = moe.fp8_block_forward(*layer.args())
    assert torch.equal(again[100:], y[100:]) and torch.equal(again[:100], y[100:])


@pytest.mark.parametrize("T", [4, 300])
def test_layer_reports_a_nan_token(T):
    layer = Layer(T, 256, 256, 8, 2, seed=3)
    ws = moe.new_workspace(moe.fp8_block_workspace_size(*layer.shape))
    y = moe.fp8_block_forward(*layer.args(), workspace=ws)
    layer.x[1, 5] = float("nan")
    bad = moe.fp8_block_forward(*layer.args(), workspace=ws)
    assert moe.device_error(ws) == -7
    keep = torch.arange(T) != 1
    assert torch.equal(bad[keep], y[keep])
    layer.x[1, 5] = 0.5
    moe.fp8_block_forward(*layer.args(), workspace=ws)
    assert moe.device_error(ws) == 0


def test_layer_on_a_side_stream_with_no_tokens_between():
    layer = Layer(48, 512, 256, 8, 2, seed=6)
    want = moe.fp8_block_forward(*layer.args())
    ws = moe.new_workspace(moe.fp8_block_workspace_size(*layer.shape))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    args = layer.args()
    moe.fp8_block_forward(args[0][:0], *args[1:], workspace=ws, stream=side)
    moe.fp8_block_forward(*args, workspace=ws, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("M", [4, 20, 400])
def test_a_wait_that_runs_out_is_reported(monkeypatch, M):
    """The test hook makes the tensor-core product's producer wait for nothing."""
    g = gen(11)
    x, (w_q, w_s) = activations(g, M, 512), weight(g, 512, 512)
    ws = moe.new_workspace(moe.fp8_block_linear_workspace_size(M, 512, 512))
    want = moe.fp8_block_linear(x, w_q, w_s, workspace=ws)
    prev = moe.set_wait_timeout_ns(2_000_000)
    try:
        monkeypatch.setenv("MOE_INJECT", "stall")
        moe.fp8_block_linear(x, w_q, w_s, workspace=ws)
        assert moe.device_error(ws) == -5
    finally:
        monkeypatch.delenv("MOE_INJECT")
        moe.set_wait_timeout_ns(prev)
    assert torch.equal(moe.fp8_block_linear(x, w_q, w_s, workspace=ws), want)
    assert moe.device_error(ws) == 0


# one launch's tiles split over clusters, whole tiles, grouped few rows, many rows
@pytest.mark.parametrize("shape", [(3, 512, 256, 8, 2), (8, 2048, 1024, 64, 4), (40, 512, 256, 64, 2),
                                   (300, 512, 256, 8, 2)])
def test_a_wait_of_the_layer_that_runs_out_is_reported(monkeypatch, shape):
    layer = Layer(*shape, seed=13)
    ws = moe.new_workspace(moe.fp8_block_workspace_size(*shape))
    want = moe.fp8_block_forward(*layer.args(), workspace=ws)
    prev = moe.set_wait_timeout_ns(2_000_000)
    try:
        monkeypatch.setenv("MOE_INJECT", "stall")
        moe.fp8_block_forward(*layer.args(), workspace=ws)
        assert moe.device_error(ws) == -5
    finally:
        monkeypatch.delenv("MOE_INJECT")
        moe.set_wait_timeout_ns(prev)
    assert torch.equal(moe.fp8_block_forward(*layer.args(), workspace=ws), want)
    assert moe.device_error(ws) == 0


def test_checked_build_gives_the_same_bits():
    from w8a8_quantised_moe_gb300 import _lib, build
    checked = _lib.open_library(build.build(checked=True))
    for shape in ((3, 512, 256, 8, 2), (300, 512, 256, 8, 2)):
        layer = Layer(*shape, seed=12)
        want = moe.fp8_block_forward(*layer.args())
        ws = moe.new_workspace(moe.fp8_block_workspace_size(*shape))
        y = torch.empty_like(want)
        p = [t.data_ptr() for t in (layer.x, layer.router_w)]
        q = [t.data_ptr() for t in (layer.w13, layer.s13, layer.w2, layer.s2)]
        assert checked.moe_w8a8_fp8_block_forward(*p, None, *q, *shape, y.data_ptr(), ws.data_ptr(), ws.numel(),
                                                  torch.cuda.current_stream().cuda_stream) == 0
        assert moe.device_error(ws) == 0
        assert torch.equal(y, want)
