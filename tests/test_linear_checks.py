"""Dense products: refusals on the host (no GPU call is made)."""
import ctypes

import pytest
import torch

import sparse_mixture_experts_24_amd as moe


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(moe.LIB_PATH):
        from sparse_mixture_experts_24_amd import build
        build.build()
    return moe.lib()


def desc(**kw):
    base = dict(M=10, N=100, K=64, ldx=0, ldw=0, ldr=0, ldo=0, dtype=1, out_dtype=1, act=0)
    base.update(kw)
    return moe.LinearDesc(**base)


@pytest.mark.parametrize("kw,plain,fp8", [
    ({}, 0, 0),
    ({"M": 0}, 0, 0),
    ({"M": -1}, 2, 2),
    ({"N": 0}, 2, 2),
    ({"K": 0}, 2, 2),
    ({"K": 60}, 3, 3),
    ({"K": 72}, 0, 3),
    ({"K": 68}, 3, 3),
    ({"K": 68, "dtype": 0, "out_dtype": 0}, 0, 3),
    ({"dtype": 0}, 0, 3),
    ({"dtype": 2}, 3, 3),
    ({"out_dtype": -1}, 3, 3),
    ({"act": 5}, 3, 3),
    ({"act": -1}, 3, 3),
    ({"ldx": 63}, 2, 2),
    ({"ldx": 65}, 3, 3),
    ({"ldx": 72}, 0, 0),
    ({"ldw": 72}, 0, 3),
    ({"ldw": 80}, 0, 0),
    ({"ldr": 99}, 2, 2),
    ({"ldo": 99}, 2, 2),
    ({"ldr": 101, "ldo": 103}, 0, 0),
    ({"ldx": -8}, 2, 2),
    ({"ldo": (1 << 24) + 1}, 3, 3),
    ({"ldx": 1 << 24, "ldo": 1 << 24}, 0, 0),
    ({"M": (1 << 24) + 1}, 3, 3),
    ({"N": (1 << 20) + 1}, 3, 3),
    ({"K": 1 << 21}, 3, 3),
    ({"M": 1 << 24, "N": 1 << 20}, 3, 3),
    ({"M": (1 << 63) - 1, "N": (1 << 63) - 1, "K": (1 << 63) - 1}, 3, 3),
])
def test_descriptions(L, kw, plain, fp8):
    d = desc(**kw)
    assert L.moe_linear_validate(ctypes.byref(d), 0) == plain
    assert L.moe_linear_validate(ctypes.byref(d), 1) == fp8


def test_null_and_misaligned_arguments(L):
    f, odd, P = 0x100000, 0x100004, ctypes.byref(desc())
    assert L.moe_linear_validate(None, 0) == 1
    assert L.moe_linear(None, f, f, None, None, f, None) == 1
    assert L.moe_linear(P, None, f, None, None, f, None) == 1
    assert L.moe_linear(P, f, None, None, None, f, None) == 1
    assert L.moe_linear(P, f, f, None, None, None, None) == 1
    assert L.moe_linear_gated(P, f, f, None, None, None, None, f, None) == 1
    assert L.moe_linear_fp8(P, f, f, None, None, None, f, None) == 1
    assert L.moe_linear_gated_fp8(P, f, f, f, f, None, None, None, None, f, None) == 1
    assert L.moe_linear(P, odd, f, None, None, f, None) == 3
    assert L.moe_linear(P, f, odd, None, None, f, None) == 3
    assert L.moe_linear(P, f, f, odd + 1, None, f, None) == 3
    assert L.moe_linear(P, f, f, None, odd + 1, f, None) == 3
    assert L.moe_linear(P, f, f, None, None, odd + 1, None) == 3
    assert L.moe_linear_gated(P, f, f, odd, None, None, None, f, None) == 3
    assert L.moe_linear_fp8(P, f, f, odd + 2, None, None, f, None) == 3
    # no rows: nothing is enqueued, so no tensor but the weights is needed
    zero = ctypes.byref(desc(M=0))
    assert L.moe_linear(zero, None, f, None, None, None, None) == 0
    assert L.moe_linear(zero, None, None, None, None, None, None) == 1


def test_binding_refuses_what_it_cannot_pass_on():
    x, W = torch.zeros(4, 64), torch.zeros(8, 64)
    with pytest.raises(ValueError, match="act"):
        moe.linear_desc(x, W, act="tanh")
    with pytest.raises(ValueError, match="matrices"):
        moe.linear_desc(x[0], W)
    with pytest.raises(ValueError, match="shape"):
        moe.linear_desc(x, W[:, :32])
    with pytest.raises(TypeError, match="dtype"):
        moe.linear_desc(x, W.bfloat16())
    with pytest.raises(TypeError, match="unsupported"):
        moe.linear_desc(x.half(), W.half())
    with pytest.raises(ValueError, match="contiguous rows"):
        moe.linear_desc(torch.zeros(64, 4).t(), W)
    with pytest.raises(ValueError, match="overlapping"):
        moe.linear_desc(x, torch.zeros(64).expand(8, 64))
    with pytest.raises(TypeError, match="residual"):
        moe.linear_desc(x, W, residual=torch.zeros(4, 8).bfloat16())
    with pytest.raises(ValueError, match="out"):
        moe.linear_desc(x, W, out=torch.zeros(4, 9))
    d = moe.linear_desc(torch.zeros(4, 80)[:, :64], W, act="gelu", out=torch.zeros(4, 10)[:, :8])
    assert (d.M, d.N, d.K, d.ldx, d.ldw, d.ldr, d.ldo, d.act) == (4, 8, 64, 80, 64, 0, 10, 2)
