"""Refusals of the block-scaled FP8 operators and of the norms around a block, on
the host: nothing is launched, no pointer is read."""
import pytest
import torch

import w8a8_quantised_moe_gb300 as moe
from w8a8_quantised_moe_gb300 import _lib
from w8a8_quantised_moe_gb300 import build as lib_build

OK, INVALID, SHAPE, WS_SMALL, CUDA, NOT_IMPL = 0, -1, -2, -3, -4, -6
FAKE = 1 << 20  # an aligned, never dereferenced address


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return _lib.load()


def linear(lib, M=64, N=256, K=256, x=FAKE, w=FAKE, s=FAKE, y=FAKE, ws=FAKE, short=0):
    need = lib.moe_w8a8_fp8_block_linear_workspace_size(M, N, K) or 1 << 30
    return lib.moe_w8a8_fp8_block_linear(x, w, s, M, N, K, y, ws, need - short, None)


def test_linear_refusals(lib, monkeypatch):
    for bad in (dict(N=8), dict(N=250), dict(K=100), dict(K=0), dict(M=-1), dict(M=(1 << 20) + 1), dict(N=65552),
                dict(K=65552)):
        assert linear(lib, **bad) == SHAPE, bad
        shape = {**dict(M=64, N=256, K=256), **bad}
        assert lib.moe_w8a8_fp8_block_linear_workspace_size(shape["M"], shape["N"], shape["K"]) == 0
    for name in ("x", "w", "s", "y", "ws"):
        assert linear(lib, **{name: None}) == INVALID
        assert linear(lib, **{name: FAKE + 8}) == INVALID
    assert linear(lib, ws=FAKE + 16) == INVALID  # 256-byte aligned
    assert linear(lib, short=1) == WS_SMALL
    assert linear(lib, M=0, x=None) == OK
    monkeypatch.setenv("MOE_INJECT", "ws_short")
    assert linear(lib) == WS_SMALL
    monkeypatch.setenv("MOE_INJECT", "launch_fail")
    assert linear(lib) == CUDA
    monkeypatch.delenv("MOE_INJECT")
    lib.moe_w8a8_set_gemm_path(3)
    try:
        assert linear(lib) == NOT_IMPL
    finally:
        lib.moe_w8a8_set_gemm_path(-1)


def layer(lib, T=16, H=256, I=512, E=8, k=2, short=0, **ptrs):
    p = {**dict(x=FAKE, rw=FAKE, bias=None, w13=FAKE, s13=FAKE, w2=FAKE, s2=FAKE, y=FAKE, ws=FAKE), **ptrs}
    need = lib.moe_w8a8_fp8_block_workspace_size(T, H, I, E, k) or 1 << 30
    return lib.moe_w8a8_fp8_block_forward(p["x"], p["rw"], p["bias"], p["w13"], p["s13"], p["w2"], p["s2"], T, H, I, E,
                                          k, p["y"], p["ws"], need - short, None)


def test_layer_refusals(lib, monkeypatch):
    for bad in (dict(H=100), dict(I=500), dict(E=0), dict(E=257), dict(k=0), dict(k=9), dict(E=4, k=5), dict(T=-1),
                dict(H=32768)):
        assert layer(lib, **bad) == SHAPE, bad
    for name in ("x", "rw", "w13", "s13", "w2", "s2", "y", "ws"):
        assert layer(lib, **{name: None}) == INVALID
        assert layer(lib, **{name: FAKE + 4}) == INVALID
    assert layer(lib, bias=FAKE + 4) == INVALID
    assert layer(lib, ws=FAKE + 128) == INVALID
    assert layer(lib, short=1) == WS_SMALL
    assert layer(lib, T=0, x=None) == OK
    monkeypatch.setenv("MOE_INJECT", "bad_ptr")
    assert layer(lib) == INVALID
    monkeypatch.setenv("MOE_INJECT", "launch_fail")
    assert layer(lib) == CUDA


def test_quantizer_refusals(lib):
    def q(groups=2, rows=256, K=256, w=FAKE, w_q=FAKE, s=FAKE):
        return lib.moe_w8a8_fp8_block_quantize_weights(w, groups, rows, K, w_q, s, None)
    for bad in (dict(groups=-1), dict(rows=0), dict(rows=100), dict(K=8), dict(K=130)):
        assert q(**bad) == SHAPE, bad
    for name in ("w", "w_q", "s"):
        assert q(**{name: None}) == INVALID and q(**{name: FAKE + 4}) == INVALID
    assert q(groups=0, w=None) == OK


def test_norm_refusals(lib):
    def n(x=FAKE, branch=FAKE, post=FAKE, gate=FAKE, form=1, scale=1.0, pre=FAKE, eps=1e-6, T=4, H=64, xo=FAKE, no=FAKE):
        return lib.moe_w8a8_norm_residual(x, 0, branch, post, gate, form, scale, pre, eps, T, H, xo, no, None)
    for bad in (dict(T=-1), dict(H=0), dict(H=12), dict(H=16392), dict(T=(1 << 20) + 1)):
        assert n(**bad) == SHAPE, bad
    for bad in (dict(x=None), dict(xo=None), dict(no=None), dict(gate=None), dict(form=4), dict(form=-1),
                dict(branch=None), dict(branch=None, form=0), dict(branch=None, post=None, form=0, pre=None),
                dict(eps=-1.0), dict(eps=float("nan"))):
        assert n(**bad) == INVALID, bad
    for name in ("x", "branch", "post", "gate", "pre", "xo", "no"):
        assert n(**{name: FAKE + 8}) == INVALID, name
    assert n(T=0) == OK
    assert n(T=0, eps=-1.0) == INVALID


def test_python_refusals():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    w, s = torch.zeros(128, 128, dtype=torch.uint8), torch.zeros(1, 1)
    with pytest.raises(ValueError, match="x: expected contiguous cuda"):
        moe.fp8_block_linear(x, w, s)
    with pytest.raises(ValueError, match="x: expected"):
        moe.norm_residual(x, pre_w=x[0])
    with pytest.raises(ValueError, match="2 or 3 dimensions"):
        moe.fp8_block_quantize_weights(torch.zeros(4))
    with pytest.raises(moe.MoeError):
        moe.fp8_block_linear_workspace_size(4, 100, 128)
    with pytest.raises(moe.MoeError):
        moe.fp8_block_workspace_size(4, 100, 128, 8, 2)
