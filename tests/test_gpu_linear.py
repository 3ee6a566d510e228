"""Dense products with a fused epilogue against a plain 64-bit evaluation.

Tolerance.  z is a sum of K products in float32; the order is the kernel's own.  Each of the
K products and K additions rounds by at most half a step of the running value, so
|dz| <= 2 K u S with u = 2^-24 and S = sum |x w| + |b| in the worst case; the roundings are
independent, and 4 sqrt(K) u S + 8 u S holds with room (a random walk of K steps of u S / 2
at most has a standard deviation of sqrt(K) u S / 2).  8-bit weights multiply the sum by a
scale: one more u.  The activations have slopes of at most 1.13 and are evaluated to an
absolute 1e-6 (|z| + 1).  The output is then rounded once: half a step, eps / 2 relative.
"""
import math

import pytest
import torch

import sparse_mixture_experts_24_amd as moe

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z) if act == "silu" else z


def e4m3_rows(w):
    s = (w.abs().amax(1) / 448.0).clamp_min(1e-30)
    q = (w / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8), s, q.double() * s.double()[:, None]


def make(M, N, K, kind, gated, bias, residual, out_dtype, seed, ldx=0, ldw=0, ldr=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)   # noqa: E731
    xt = F32 if kind == "f32" else BF
    strided = lambda t, ld: (torch.full((t.shape[0], max(ld, t.shape[1])), float("nan"),   # noqa: E731
                                        device=DEV).to(t.dtype) if t.dtype != torch.uint8 else
                             torch.full((t.shape[0], max(ld, t.shape[1])), 0x7F,
                                        dtype=torch.uint8, device=DEV))

    def place(t, ld):   # a view of a wider buffer whose padding must never be used
        if not ld:
            return t
        b = strided(t, ld)
        b[:, :t.shape[1]] = t
        return b[:, :t.shape[1]]

    x = place(rnd(M, K).to(xt), ldx)
    ws, ss, wide = [], [], []
    for _ in range(2 if gated else 1):
        w = rnd(N, K) / math.sqrt(K)
        if kind == "fp8":
            q, s, wd = e4m3_rows(w)
        else:
            q, s = w.to(xt), None
            wd = q.double()
        ws.append(place(q, ldw))
        ss.append(s)
        wide.append(wd)
    bs = [rnd(N) if bias else None for _ in ws]
    r = place(rnd(M, N).to(out_dtype), ldr) if residual else None
    return x, ws, ss, wide, bs, r


def reference(x, wide, bs, r, act):
    """(value, bound on the 32-bit error before the final rounding)."""
    K = x.shape[1]
    z, dz = [], []
    for w, b in zip(wide, bs):
        v, S = x.double() @ w.t(), x.double().abs() @ w.abs().t()
        if b is not None:
            v, S = v + b.double(), S + b.double().abs()
        z.append(v)
        dz.append((4 * math.sqrt(K) + 8) * U * S)
    y = act64(z[0], act)
    dy = 1.13 * dz[0] + (0 if act == "none" else 1e-6 * (z[0].abs() + 1))
    if len(z) == 2:
        dy = dy * (z[1].abs() + dz[1]) + y.abs() * dz[1] + U * (y * z[1]).abs()
        y = y * z[1]
    if r is not None:
        y = y + r.double()
    return y, dy + 2 * U * y.abs()


def check(got, y, dy, what=""):
    half = torch.finfo(got.dtype).eps / 2
    err = (got.double() - y).abs()
    tol = dy + half * (y.abs() + dy) + 1e-30
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} elements off, worst "
                           f"{float((err / tol).nan_to_num(1e9).max()):.2f} of the tolerance")


def call(x, ws, ss, bs, r, act, **kw):
    if len(ws) == 2:
        if ss[0] is not None:
            return moe.linear_gated_fp8(x, *ws, *ss, *bs, act=act, residual=r, **kw)
        return moe.linear_gated(x, *ws, *bs, act=act, residual=r, **kw)
    if ss[0] is not None:
        return moe.linear_fp8(x, ws[0], ss[0], bs[0], act=act, residual=r, **kw)
    return moe.linear(x, ws[0], bs[0], act=act, residual=r, **kw)


# (M, N, K): single tokens, the borders of every tile, odd sizes, K shorter than a step
SIZES = [(1, 1, 16), (1, 257, 64), (2, 64, 4096), (7, 1000, 144), (15, 33, 2064), (16, 512, 1024),
         (17, 96, 528), (33, 130, 64), (63, 65, 80), (64, 256, 2048), (65, 127, 1008),
         (100, 1001, 336), (129, 128, 4112), (200, 300, 208), (255, 513, 640), (257, 255, 1040),
         (333, 1001, 1984), (512, 768, 512), (1025, 320, 192)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("gated", [False, True])
def test_sizes(M, N, K, kind, gated):
    print(f"\n[linear] {M}x{N}x{K} {kind} gated={gated}", flush=True)
    out = F32 if kind == "f32" or (M + N) % 2 else BF
    x, ws, ss, wide, bs, r = make(M, N, K, kind, gated, M % 2 == 0, N % 2 == 0, out, M + N + K)
    act = "silu" if gated else "none"
    got = call(x, ws, ss, bs, r, act, out_dtype=out)
    check(got, *reference(x, wide, bs, r, act))


@pytest.mark.parametrize("act", list(moe.ACTS))
@pytest.mark.parametrize("M,N,K,kind", [(3, 200, 256, "bf16"), (130, 200, 264, "bf16"),
                                        (600, 300, 128, "bf16"), (40, 72, 100, "f32"),
                                        (5, 90, 48, "fp8"), (300, 90, 48, "fp8")])
@pytest.mark.parametrize("gated", [False, True])
def test_activations(act, M, N, K, kind, gated):
    print(f"\n[linear] act {act} {M}x{N}x{K} {kind} gated={gated}", flush=True)
    x, ws, ss, wide, bs, r = make(M, N, K, kind, gated, True, False, F32, 5)
    x = x * 6          # far into both tails of the activation
    got = call(x, ws, ss, bs, r, act, out_dtype=F32)
    check(got, *reference(x, wide, bs, r, act))


@pytest.mark.parametrize("M,N,K,kind", [(1, 130, 128, "bf16"), (9, 130, 512, "fp8"),
                                        (80, 200, 136, "bf16"), (400, 260, 320, "bf16"),
                                        (400, 260, 320, "fp8"), (70, 66, 68, "f32")])
def test_strided_rows(M, N, K, kind):
    """Rows of every tensor inside wider buffers: the padding holds NaN and must neither be
    read into the result nor (out) be written."""
    print(f"\n[linear] strided {M}x{N}x{K} {kind}", flush=True)
    x, ws, ss, wide, bs, r = make(M, N, K, kind, False, True, True, BF, 9, ldx=K + 48, ldw=K + 16,
                                  ldr=N + 3)
    buf = torch.full((M, N + 7), -3.0, dtype=BF, device=DEV)
    got = call(x, ws, ss, bs, r, "relu", out=buf[:, :N], out_dtype=BF)
    assert got.data_ptr() == buf.data_ptr()
    check(got, *reference(x, wide, bs, r, "relu"))
    assert bool((buf[:, N:] == -3.0).all())


@pytest.mark.parametrize("M,N,K", [(17, 20, 8208), (33, 130, 2064), (83, 70, 5488),
                                   (320, 98, 5632), (40, 33, 16400)])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("gated", [False, True])
def test_few_columns_and_long_rows(M, N, K, kind, gated):
    """More than 16 rows, too few tiles for the GPU: rows go through in blocks of 16."""
    x, ws, ss, wide, bs, r = make(M, N, K, kind, gated, True, True, F32, 23, ldx=K + 64,
                                  ldw=K + 32, ldr=N + 4)
    y, dy = reference(x, wide, bs, r, "silu")
    got = call(x, ws, ss, bs, r, "silu", out_dtype=F32)
    check(got, y, dy, f"{M} {N} {K}")
    assert torch.equal(got, call(x, ws, ss, bs, r, "silu", out_dtype=F32))


@pytest.mark.parametrize("M,N,K", [(1, 2048, 2048), (16, 512, 4096), (300, 256, 512)])
def test_in_place_residual_and_determinism(M, N, K):
    print(f"\n[linear] in place {M}x{N}x{K}", flush=True)
    x, ws, ss, wide, bs, r = make(M, N, K, "bf16", False, True, True, BF, 2)
    a = call(x, ws, ss, bs, r, "none", out_dtype=BF)
    b = call(x, ws, ss, bs, r, "none", out_dtype=BF)
    assert torch.equal(a, b)
    hidden = r.clone()
    got = call(x, ws, ss, bs, hidden, "none", out=hidden, out_dtype=BF)
    assert got.data_ptr() == hidden.data_ptr() and torch.equal(got, a)


@pytest.mark.parametrize("M", [1, 24, 300])
def test_graph_replays_and_two_streams(M):
    """Captured calls replay bit for bit, and calls on two streams at once give the eager
    results."""
    print(f"\n[linear] graph and streams M={M}", flush=True)
    N, K = 512, 2048
    sets = [make(M, N, K, "bf16", False, True, True, BF, s) for s in (1, 2)]
    ref = [call(x, w, s, b, r, "gelu", out_dtype=BF) for x, w, s, _, b, r in sets]
    outs = [torch.empty_like(t) for t in ref]
    run = lambda i: call(*[sets[i][j] for j in (0, 1, 2, 4, 5)], "gelu", out=outs[i],   # noqa: E731
                         out_dtype=BF)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                run(i)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref[0]) and torch.equal(outs[1], ref[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(0)
        run(1)
    for _ in range(3):
        for o in outs:
            o.zero_()
        junk = torch.randn(1 << 18, device=DEV).sum()
        g.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(junk)
        assert torch.equal(outs[0], ref[0]) and torch.equal(outs[1], ref[1])


def test_most_rows():
    """2^24 rows: more blocks than a grid's second dimension holds."""
    M, K = 1 << 24, 16
    g = torch.Generator(device=DEV).manual_seed(31)
    x = torch.randn(M, K, generator=g, device=DEV).to(BF)
    W = torch.randn(3, K, generator=g, device=DEV).to(BF)
    got = moe.linear(x, W, out_dtype=F32)
    rows = torch.cat([torch.arange(64), torch.arange(M // 2, M // 2 + 64),
                      torch.arange(M - 64, M)]).to(DEV)
    y, dy = reference(x[rows], [W.double()], [None], None, "none")
    check(got[rows], y, dy)
    far = (got - x.float() @ W.float().t()).abs().max()
    assert float(far) < 1e-4


def test_no_rows():
    W = torch.randn(64, 64, device=DEV).to(BF)
    got = moe.linear(torch.empty(0, 64, dtype=BF, device=DEV), W)
    assert got.shape == (0, 64)


def test_offsets_past_32_bits():
    """x and out rows more than 2^32 bytes from their first element."""
    K, ld, M = 64, 1 << 24, 140          # 140 rows 2^24 elements apart: 4.7 GB
    buf = torch.zeros(M * ld, dtype=BF, device=DEV)
    x = buf.view(M, ld)[:, :K]
    g = torch.Generator(device=DEV).manual_seed(3)
    x.copy_(torch.randn(M, K, generator=g, device=DEV))
    W = torch.randn(48, K, generator=g, device=DEV).to(BF)
    out = torch.zeros(M * ld, dtype=BF, device=DEV).view(M, ld)[:, :48]
    for rows in (M, 3):
        got = moe.linear(x[-rows:], W, out=out[-rows:])
        check(got, *reference(x[-rows:], [W.double()], [None], None, "none"))


@pytest.mark.parametrize("M,N,K,kind", [(1, 70, 2056, "bf16"), (3, 70, 36, "f32"),
                                        (16, 200, 13320, "bf16"), (16, 70, 4108, "f32"),
                                        (40, 70, 520, "bf16"), (40, 70, 44, "f32"),
                                        (300, 260, 8200, "bf16"), (300, 260, 1100, "f32")])
@pytest.mark.parametrize("act", list(moe.ACTS))
def test_infinite_and_nan_values(M, N, K, kind, act):
    """Rows and columns that hold infinities or NaN give what the formula gives, also where K
    ends inside a step, and leave the others alone."""
    x, ws, ss, wide, bs, r = make(M, N, K, kind, False, True, True, F32, 17)
    x.abs_().add_(0.5)
    W = ws[0]
    W[1, K - 1] = math.inf      # z = +inf
    W[2, K // 2] = math.nan
    if act in ("none", "relu"):
        W[5, K - 1] = -math.inf
    if M > 2:
        x[1, K - 1] = math.nan
    got = moe.linear(x, W, bs[0], act=act, residual=r, out_dtype=F32)
    y, dy = reference(x.nan_to_num(0.0), [W.double().nan_to_num(0.0, 0.0, 0.0)], bs, r, act)
    y[:, 1] = math.inf          # every activation of +inf
    if act in ("none", "relu"):
        y[:, 5] = -math.inf if act == "none" else r[:, 5].double()
    y[:, 2] = math.nan
    if M > 2:
        y[1] = math.nan
    assert torch.equal(torch.isnan(got), torch.isnan(y))
    inf = torch.isinf(y)
    assert inf.any() and torch.equal(got[inf].double(), y[inf])
    ok = torch.isfinite(y)
    check(got[ok], y[ok], dy[ok])
