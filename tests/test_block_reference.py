"""The tests' plain forms of the block-scaled operators against hand-worked values
and against other ways to the same numbers (CPU)."""
import torch

import block_reference as ref


def test_e4m3_values_and_codes_agree_with_torch():
    v = ref.e4m3_values()
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    assert torch.equal(torch.nan_to_num(v, nan=-1.0), torch.nan_to_num(t, nan=-1.0))
    g = torch.Generator().manual_seed(0)
    q = torch.cat([torch.randn(20000, generator=g) * s for s in (1e-3, 0.1, 10, 150)]).clamp(-448, 448)
    mid = (v[:126] + v[1:127]) / 2  # every midpoint, both signs
    q = torch.cat([q, mid.float(), -mid.float(), v[:127].float()])
    assert torch.equal(ref.e4m3_codes(q), q.to(torch.float8_e4m3fn).view(torch.uint8))


def test_quantized_row_by_hand():
    # one block: largest magnitude 448 * 2^-3, so s = 2^-3 to an ulp and the quotients are 8 x
    x = torch.zeros(1, 130)
    x[0, :4] = torch.tensor([56.0, -28.0, 0.109375, 1.0])  # codes of 448, -224, 0.875, 8
    x[0, 129] = 7.0  # alone in the second block
    codes, scales = ref.quantize_rows(x)
    assert abs(scales[0, 0].item() - 0.125) <= 2**-26 and abs(scales[0, 1].item() - 7 / 448) <= 2**-29
    v = ref.e4m3_values()
    assert v[codes[0, :4].long()].tolist() == [448.0, -224.0, 0.875, 8.0]
    assert v[int(codes[0, 129])] == 448.0 and int(codes[0, 128]) == 0


def test_zero_block_has_zero_scale_and_codes():
    codes, scales = ref.quantize_rows(torch.zeros(2, 256))
    assert not codes.any() and not scales.any()


def test_linear_equals_a_sum_over_blocks():
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(3, 300, generator=g), torch.randn(200, 300, generator=g)
    w_q, w_s = ref.quantize_weight(w)
    y, mag = ref.linear(x, w_q, w_s)
    c, s = ref.quantize_rows(x)
    v = ref.e4m3_values()
    for n in (0, 127, 128, 199):
        want = sum(float(s[1, b]) * float(w_s[n // 128, b])
                   * float((v[c[1, b * 128:(b + 1) * 128].long()] * v[w_q[n, b * 128:(b + 1) * 128].long()]).sum())
                   for b in range(3))
        assert abs(y[1, n].item() - want) <= 1e-13 * mag[1, n].item()


def test_layer_with_one_expert_is_its_three_products():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(4, 128, generator=g).bfloat16()
    q13, s13 = ref.quantize_weight(0.1 * torch.randn(256, 128, generator=g))
    q2, s2 = ref.quantize_weight(0.1 * torch.randn(128, 128, generator=g))
    a, _ = ref.linear(x, q13, s13)
    h = torch.nn.functional.silu(a[:, :128]) * a[:, 128:]
    want, _ = ref.linear(h.float(), q2, s2)
    got = ref.moe(x, torch.randn(128, 1, generator=g), None, q13[None], s13[None], q2[None], s2[None], 1)
    assert torch.allclose(got, want, rtol=1e-12, atol=1e-14)


def test_norms_by_hand():
    x = torch.tensor([[1.0, 2.0]])
    branch = torch.tensor([[3.0, -4.0]])  # mean square 12.5
    r, n, _ = ref.norm_residual(x, branch, torch.tensor([1.0, 2.0]), torch.tensor([[0.5]]), 2.0,
                                torch.tensor([1.0, 1.0]), 0.0)
    want = torch.tensor([[1 + 3 / 12.5**0.5, 2 - 8 / 12.5**0.5]], dtype=torch.float64)
    assert torch.allclose(r, want, rtol=1e-12)
    assert torch.allclose(n, want / want.pow(2).mean().sqrt(), rtol=1e-12)
