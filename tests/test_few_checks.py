"""The layer for a few tokens: refusals on the host (no GPU call is made)."""
import ctypes

import pytest

import sparse_mixture_experts_24_amd as moe


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(moe.LIB_PATH):
        from sparse_mixture_experts_24_amd import build
        build.build()
    return moe.lib()


def desc(**kw):
    base = dict(T=4, d_model=256, n_experts=8, d_ff=512, top_k=2, n_shared=0,
                capacity_factor=0.0, dtype=moe.MOE_DTYPE_BF16, out_dtype=moe.MOE_DTYPE_BF16)
    base.update(kw)
    return moe.MoeDesc(**base)


F = 0x100000      # never dereferenced: validation fails first


def few(L, d, x=F, wr=F, b=None, w=(F, F, F), s=None, r=None, out=F, f=None, p=None, ws=F,
        n=1 << 40):
    d = None if d is None else ctypes.byref(d)
    if s is None:
        return L.moe_forward_few(d, x, wr, b, *w, r, out, f, p, ws, n, None)
    return L.moe_forward_few_fp8(d, x, wr, b, *w, *s, r, out, f, p, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    ({"T": 17}, 3), ({"T": 4096}, 3), ({"T": -1}, 2), ({"top_k": 9}, 2), ({"n_experts": 0}, 2),
    ({"d_model": 100}, 3), ({"d_ff": 96}, 3), ({"n_experts": 513}, 3), ({"dtype": 2}, 3),
    ({"out_dtype": 9}, 3), ({"n_shared": 2}, 2), ({"capacity_factor": float("nan")}, 2),
])
def test_descriptions(L, kw, status):
    d = desc(**kw)
    assert L.moe_workspace_bytes_few(ctypes.byref(d)) == 0
    assert few(L, d) == status
    assert few(L, d, s=(F, F, F)) == status


def test_workspace(L):
    d = desc()
    need = L.moe_workspace_bytes_few(ctypes.byref(d))
    assert need > 0 and need % 256 == 0
    assert need <= L.moe_workspace_bytes_few(ctypes.byref(desc(T=16)))
    assert L.moe_workspace_bytes_few(ctypes.byref(desc(T=0))) > 0
    assert few(L, d, ws=None) == 4
    assert few(L, d, n=need - 1) == 4
    assert few(L, d, ws=F + 16) == 4


def test_null_and_misaligned_arguments(L):
    d = desc()
    assert few(L, None) == 1
    assert few(L, d, x=None) == 1 and few(L, d, wr=None) == 1 and few(L, d, out=None) == 1
    for i in range(3):
        assert few(L, d, w=[None if i == j else F for j in range(3)]) == 1
        assert few(L, d, s=[None if i == j else F for j in range(3)]) == 1
        assert few(L, d, w=[F + 8 if i == j else F for j in range(3)]) == 3
        assert few(L, d, s=[F + 2 if i == j else F for j in range(3)]) == 3
    assert few(L, desc(dtype=0), s=(F, F, F)) == 3      # 8-bit weights: bf16 layers only
    for name in ("x", "wr", "r", "out"):
        assert few(L, d, **{name: F + 8}) == 3
    for name in ("b", "f", "p"):
        assert few(L, d, **{name: F + 2}) == 3
