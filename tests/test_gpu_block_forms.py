"""The launch forms of the block-scaled operators and norms that large calls take: several
tiles a CTA in every product, four vectors a lane in the quantisers, two vectors a lane and
several rows a CTA in the norms."""
import pytest
import torch

import test_gpu_block as block
import test_gpu_norm as norm
import w8a8_quantised_moe_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(4100, 2064, 1040), (9001, 784, 272), (2600, 4112, 2064)])
def test_linear_with_several_tiles_a_cta(M, N, K):
    g = block.gen(M)
    x, (w_q, w_s) = block.activations(g, M, K), block.weight(g, N, K)
    y = block.check_linear(x, w_q, w_s)
    for _ in range(2):
        assert torch.equal(moe.fp8_block_linear(x, w_q, w_s), y)


@pytest.mark.parametrize("shape", [(5001, 1408, 256, 8, 2, None), (3000, 1152, 640, 3, 3, 1.0),
                                   (2500, 2048, 1024, 24, 2, 0.7)])
def test_layer_with_several_tiles_a_cta(shape):
    layer = block.Layer(*shape[:5], seed=shape[0], bias=shape[5])
    y = moe.fp8_block_forward(*layer.args())
    layer.check(y)
    for _ in range(2):
        assert torch.equal(moe.fp8_block_forward(*layer.args()), y)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
@pytest.mark.parametrize("T,H", [(10001, 264), (10003, 512), (4001, 776), (5001, 1032), (2500, 1544), (2403, 2048),
                                 (700, 4096), (500, 6152), (400, 8200)])
def test_norms_of_many_rows(T, H, gate, fp32):
    a = norm.make(T, H, fp32, gate)
    norm.check(a, moe.norm_residual(**a))


@pytest.mark.parametrize("T,H", [(10001, 264), (2500, 1544), (500, 6152)])
def test_norms_of_many_rows_in_parts(T, H):
    for branch, post, pre in ((True, False, True), (True, True, False), (False, False, True)):
        a = norm.make(T, H, True, "none", branch, post, pre)
        norm.check(a, moe.norm_residual(**a))
