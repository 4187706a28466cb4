"""The norms around a block against their plain 64-bit form."""
import pytest
import torch

import block_reference as ref
import w8a8_quantised_moe_gb300 as moe

pytestmark = pytest.mark.gpu

# u = 2^-24.  A row's sum of squares: at most 16 terms in a lane, 5 steps in a warp
# and 32 warps, all positive: 53 u of the sum, half of that after the square root; the
# reciprocal square root is within 2 ulp (4 u), and at most 6 products follow: 37 u < 2^-18.
BRANCH_REL = 2.0**-18
U, BF16 = 2.0**-24, 2.0**-8


def make(T, H, fp32, gate, branch=True, post=True, pre=True, seed=0, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 31 * T + H)

    def r(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    x = (size * r(T, H)) if fp32 else (size * r(T, H)).bfloat16()
    shape = {"none": None, "channel": (H,), "token": (T, 1), "element": (T, H)}[gate]
    return dict(x=x, branch=(3 * r(T, H)).bfloat16() if branch else None,
                post_w=(1 + 0.1 * r(H)).bfloat16() if post else None,
                gate=None if shape is None else r(*shape).bfloat16(), scale=-0.37,
                pre_w=(1 + 0.1 * r(H)).bfloat16() if pre else None, eps=1e-6)


def check(a, got):
    r, n = got
    want_r, want_n, added = ref.norm_residual(**a)
    err = BRANCH_REL * added + U * (want_r.abs() + added)  # of the unrounded r
    rounding = U if a["x"].dtype == torch.float32 else BF16
    if a["branch"] is not None:
        assert ((r.double() - want_r).abs() <= err + rounding * want_r.abs() + 2.0**-134).all()
    if a["pre_w"] is None:
        assert n is None
        return
    # n = r * f * w: the error of r, and that of f (through every r of the row: at most the largest
    # relative error of the sum of squares), then one rounding to bf16
    w = a["pre_w"].double()
    f = 1 / (want_r.pow(2).mean(1, keepdim=True) + a["eps"]).sqrt()
    f_err = BRANCH_REL + (err * want_r.abs()).mean(1, keepdim=True) * f * f
    bound = err * f * w.abs() + f_err * want_n.abs()
    assert ((n.double() - want_n).abs() <= bound * (1 + BF16) + BF16 * want_n.abs() + 2.0**-134).all()


@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("T,H", [(1, 8), (3, 264), (9, 512), (5, 520), (7, 1024), (4, 2056), (2, 4096), (3, 4104),
                                 (2, 8200), (2, 16384), (1003, 1024)])
def test_norm_residual(T, H, fp32, gate):
    a = make(T, H, fp32, gate)
    check(a, moe.norm_residual(**a))


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("branch,post,pre", [(True, False, True), (True, True, False), (True, False, False),
                                             (False, False, True)])
@pytest.mark.parametrize("T,H", [(1, 4096), (33, 1096)])
def test_parts_left_out(T, H, branch, post, pre, fp32):
    a = make(T, H, fp32, "none", branch, post, pre)
    got = moe.norm_residual(**a)
    if not branch:
        assert got[0] is a["x"]
    check(a, got)


@pytest.mark.parametrize("fp32", [False, True])
def test_rows_of_zeros_and_large_rows(fp32):
    a = make(6, 640, fp32, "token")
    a["x"][1] = 0
    a["branch"][1] = 0
    a["branch"][2] = 0
    a["x"][3] *= 2.0**40
    a["branch"][4] = (a["branch"][4].float() * 2.0**40).bfloat16()
    a["gate"][5] = 0
    r, n = moe.norm_residual(**a)
    check(a, (r, n))
    assert not r[1].any() and not n[1].any()
    assert torch.equal(r[2], a["x"][2]) and torch.equal(r[5], a["x"][5])


def test_a_nan_stays_in_its_row():
    a = make(20, 1032, False, "channel")
    r, n = moe.norm_residual(**a)
    a["branch"][7, 3] = float("nan")
    r2, n2 = moe.norm_residual(**a)
    keep = torch.arange(20) != 7
    assert r2[7].isnan().all() and n2[7].isnan().all()
    assert torch.equal(r2[keep], r[keep]) and torch.equal(n2[keep], n[keep])


@pytest.mark.parametrize("fp32", [False, True])
def test_in_place_on_another_stream(fp32):
    a = make(300, 2048, fp32, "element")
    r, n = moe.norm_residual(**a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x = a["x"].clone()
    n_out = torch.empty_like(n)
    side.wait_stream(torch.cuda.current_stream())
    got = moe.norm_residual(**{**a, "x": x}, x_out=x, n_out=n_out, stream=side)
    side.synchronize()
    assert got[0] is x and got[1] is n_out
    assert torch.equal(x, r) and torch.equal(n_out, n)


def test_no_rows():
    a = make(1, 64, False, "none")
    r, n = moe.norm_residual(a["x"][:0], a["branch"][:0], pre_w=a["pre_w"])
    assert r.shape == (0, 64) and n.shape == (0, 64)
