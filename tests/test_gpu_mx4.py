"""Microscaled 4-bit weights: conversion bit for bit, and the products against their formulas in 64 bits.

Bounds, fixed before any run: a product sums C terms in fp32 in any order (helpers.assert_elementwise: 2^-23 C sum|x w|,
then half an ulp of the output's type); the weight's values are exact in every type here unless a test says otherwise."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
from helpers import as_f64, assert_elementwise

pytestmark = pytest.mark.gpu

sp = pytest.importorskip("unstructured_sparse_linear_gb300")

DEV = torch.device("cuda:0")
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def rand(rng, fmt, rows, cols, std=1.0, pad=0, left=None):
    """A matrix; with pad, columns of a wider one that is NaN elsewhere."""
    x = torch.from_numpy(rng.standard_normal((rows, cols)) * std).to(DTYPES[fmt]).to(DEV)
    if not pad:
        return x
    left = pad if left is None else left
    wide = torch.full((rows, cols + 2 * pad), float("nan"), dtype=x.dtype, device=DEV)
    wide[:, left:left + cols] = x
    return wide[:, left:left + cols]


def bits(t):
    return t.contiguous().view({4: torch.int32, 2: torch.int16, 1: torch.uint8}[t.element_size()]).cpu()


def check_quantized(x):
    q = sp.mx4_quantize(x)
    codes, scales = ref.quantize(as_f64(x))
    assert q.shape == tuple(x.shape) and q.dtype == x.dtype
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    want = ref.values(codes, scales, x.shape[1])
    got = sp.mx4_dequantize(q)
    assert got.dtype == x.dtype and np.array_equal(as_f64(got), want, equal_nan=True)
    return q


@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 33), (5, 31), (2, 8), (64, 96), (9, 256), (130, 1025), (1, 5000),
                                       (700, 384), (33, 2047)])
def test_quantize(fmt, rows, cols):
    rng = np.random.default_rng([rows, cols])
    check_quantized(rand(rng, fmt, rows, cols, std=0.02))
    check_quantized(rand(rng, fmt, rows, cols, std=3.0, pad=8))
    check_quantized(rand(rng, fmt, rows, cols, pad=5, left=3))


@pytest.mark.parametrize("fmt", list(DTYPES))
def test_quantize_special_values(fmt):
    dt = DTYPES[fmt]
    info = torch.finfo(dt)
    tiny = info.smallest_normal
    least = tiny * info.eps
    x = torch.zeros(16, 64, dtype=torch.float64)
    x[0, :17] = torch.tensor([6, -6, .25, -.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 5.01, .26, -0.0, 0.24, 7, 7.9, -7.99])
    x[1, ::2] = info.max
    x[1, 1] = -info.max
    x[2, 5] = float("inf")
    x[2, 40] = 1.5
    x[3, 33] = float("nan")
    x[3, 2] = -1.0
    x[4, 7] = -float("inf")
    x[5, 0], x[5, 1] = least, -3 * least
    x[6, 0], x[6, 9] = tiny, 0.4 * tiny
    x[7, 0], x[7, 1], x[7, 32] = info.max, tiny, tiny
    x[8] = torch.arange(64) * least
    x[9, 3] = 1.0
    x[10] = -torch.arange(64).double()
    x[11, :] = float("nan")
    x[12, :9] = torch.tensor([4.0, .125, 0.1249, .3749, .375, .625, 1 / 3, 3.999, -3.5])
    check_quantized(x.to(dt).to(DEV))


@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("pad", [0, 5])
def test_dequantize_every_code_and_scale(fmt, pad):
    """All 16 codes with all 256 scales, rounded to the type (infinite beyond it, subnormal or zero below)."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)[:, :16 * 16].contiguous().to(DEV)
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16).contiguous().to(DEV)
    want = torch.from_numpy(ref.values(codes.cpu().numpy(), scales.cpu().numpy(), 512)).to(DTYPES[fmt])
    W = sp.Mx4(codes, scales, 512)
    out = torch.full((256, 512 + 2 * pad), 7.0, dtype=DTYPES[fmt], device=DEV)[:, pad:pad + 512]
    for got in (sp.mx4_dequantize(W, DTYPES[fmt]), sp.mx4_dequantize(W, out=out)):
        assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want))
        keep = ~torch.isnan(want)
        assert torch.equal(bits(got)[keep], bits(want)[keep])
    if pad:
        assert (out._base[:, :pad] == 7).all() and (out._base[:, pad + 512:] == 7).all()


def weight(rng, rows, cols):
    """Random codes and scales (zero codes behind the last column) and their values."""
    w = rng.standard_normal((rows, cols)) * 0.05 * np.exp(0.5 * rng.standard_normal((rows, 1)))
    codes, scales = ref.quantize(w)
    return sp.Mx4(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), cols), ref.values(codes, scales, cols)


def check_product(fmt, back, tokens, rows, cols, pad=0, left=None, seed=0):
    rng = np.random.default_rng([seed, tokens, rows, cols])
    W, w = weight(rng, rows, cols)
    m = w if back else w.T
    X = rand(rng, fmt, tokens, m.shape[0], pad=pad, left=left)
    call = sp.mx4_linear_grad if back else sp.mx4_linear
    x = as_f64(X)
    want, mass = x @ m, np.abs(x) @ np.abs(m)
    Y = call(X, W)
    assert_elementwise(Y, want, mass, m.shape[0], fmt, "Y")
    n = m.shape[1]
    # into columns of a wider matrix, with rows behind the last: everything else stays as it was
    side = max(pad, 3 if pad else 8)
    wide = torch.full((tokens + 3, n + 2 * side), 5.0, dtype=X.dtype, device=DEV)
    out = wide[:tokens, side:side + n]
    assert call(X, W, out=out) is out
    if pad == 0 or fmt == "f32":
        assert torch.equal(out, Y)
    else:
        assert_elementwise(out, want, mass, m.shape[0], fmt, "out")
    assert (wide[tokens:] == 5).all() and (wide[:, :side] == 5).all() and (wide[:, side + n:] == 5).all()
    return Y


SIZES = [(1, 1, 1), (1, 128, 64), (1, 1000, 4096), (2, 33, 31), (3, 64, 32), (5, 130, 97), (7, 16, 1024), (8, 256, 256),
         (9, 17, 640), (16, 384, 128), (17, 256, 96), (31, 136, 72), (33, 520, 264), (64, 256, 1024), (65, 1000, 200),
         (100, 72, 2048), (128, 256, 512), (129, 264, 520), (200, 1536, 384), (257, 128, 128), (300, 640, 1032), (513, 96, 40)]


@pytest.mark.parametrize("back", [False, True], ids=["linear", "grad"])
@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("tokens,rows,cols", SIZES)
def test_products(fmt, back, tokens, rows, cols):
    check_product(fmt, back, tokens, rows, cols)


@pytest.mark.parametrize("back", [False, True], ids=["linear", "grad"])
@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("pad,left", [(8, 8), (16, 8), (3, 3), (8, 1)])
@pytest.mark.parametrize("tokens,rows,cols", [(3, 64, 96), (40, 192, 320), (140, 333, 129), (300, 256, 264)])
def test_products_of_columns(fmt, back, tokens, rows, cols, pad, left):
    check_product(fmt, back, tokens, rows, cols, pad, left)


@pytest.mark.parametrize("back", [False, True], ids=["linear", "grad"])
@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("tokens", [1, 12, 70, 600])
def test_without_anything_to_sum(fmt, back, tokens):
    W = sp.Mx4(torch.empty((0, 32) if back else (40, 0), dtype=torch.uint8, device=DEV),
               torch.empty((0, 2) if back else (40, 0), dtype=torch.uint8, device=DEV), 64 if back else 0)
    X = torch.empty(tokens, 0, dtype=DTYPES[fmt], device=DEV)
    call = sp.mx4_linear_grad if back else sp.mx4_linear
    out = torch.full((tokens, 64 if back else 40), float("nan"), dtype=X.dtype, device=DEV)
    assert not call(X, W, out=out).any() and not call(X, W).any()
    none = call(torch.empty(0, 0, dtype=X.dtype, device=DEV), W)
    assert none.shape == (0, out.shape[1])


def test_no_tokens():
    W, _ = weight(np.random.default_rng(1), 64, 96)
    assert sp.mx4_linear(torch.empty(0, 96, device=DEV), W).shape == (0, 64)
    assert sp.mx4_linear_grad(torch.empty(0, 64, device=DEV), W).shape == (0, 96)
    assert sp.mx4_dequantize(sp.mx4_quantize(torch.empty(0, 33, device=DEV))).shape == (0, 33)
    assert sp.mx4_dequantize(sp.mx4_quantize(torch.empty(4, 0, device=DEV))).shape == (4, 0)


@pytest.mark.parametrize("back", [False, True], ids=["linear", "grad"])
@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("tokens", [1, 32, 64, 256])
def test_every_scale(fmt, back, tokens):
    """A one in each row of X picks single values of W, whose scales run through those that leave all codes finite and
    normal in the type: the products are the values, bit for bit."""
    rng = np.random.default_rng(tokens)
    lo, hi = {"f32": (2, 252), "bf16": (2, 252), "f16": (127 - 13, 127 + 13)}[fmt]
    C, F = 256, 512
    rows, cols = (C, F) if back else (F, C)
    codes = torch.from_numpy(rng.integers(0, 256, (rows, cols // 2), dtype=np.uint8))
    scales = torch.from_numpy(rng.integers(lo, hi + 1, (rows, cols // 32)).astype(np.uint8))
    w = ref.values(codes.numpy(), scales.numpy(), cols)
    m = w if back else w.T  # [C, F]
    pick = rng.permutation(C)[:tokens]
    X = torch.zeros(tokens, C, dtype=DTYPES[fmt])
    X[torch.arange(tokens), torch.from_numpy(pick)] = 1.0
    W = sp.Mx4(codes.to(DEV), scales.to(DEV), cols)
    Y = (sp.mx4_linear_grad if back else sp.mx4_linear)(X.to(DEV), W)
    assert np.array_equal(as_f64(Y), m[pick])


@pytest.mark.parametrize("back", [False, True], ids=["linear", "grad"])
@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("tokens", [4, 40, 150])
def test_infinities_and_nan_stay_where_they_are(fmt, back, tokens):
    rng = np.random.default_rng(3)
    W, w = weight(rng, 256, 320)
    m = w if back else w.T
    X = rand(rng, fmt, tokens, m.shape[0])
    call = sp.mx4_linear_grad if back else sp.mx4_linear
    clean = call(X, W)
    bad = X.clone()
    bad[1, 7], bad[2, 100] = float("nan"), float("inf")
    Y = call(bad, W)
    rest = torch.ones(tokens, dtype=torch.bool, device=DEV)
    rest[1:3] = False
    assert torch.equal(Y[rest], clean[rest]) and torch.isnan(Y[1]).all()
    want = np.where(m[100] == 0, np.nan, np.copysign(np.inf, m[100]))
    assert np.array_equal(as_f64(Y[2]), want, equal_nan=True)
    # a block of the weight that is NaN: the features that it is part of
    scales = W.scales.clone()
    scales[5, 3] = 255
    Y = call(X, sp.Mx4(W.codes, scales, 320))
    hit = torch.zeros(m.shape[1], dtype=torch.bool, device=DEV)
    hit[slice(96, 128) if back else slice(5, 6)] = True
    assert torch.isnan(Y[:, hit]).all() and torch.equal(Y[:, ~hit], clean[:, ~hit])


@pytest.mark.parametrize("fmt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("back", [False, True], ids=["linear", "grad"])
def test_values_beyond_the_type(fmt, back):
    """Large scales, where values leave fp16's (or bf16's) range: infinite, as the conversion rounds them."""
    rows, cols, tokens = 128, 64, 200
    codes = torch.full((rows, 32), 0x22, dtype=torch.uint8)  # ones
    codes[:, ::2] = 0x2A  # 1, -1
    scales = torch.full((rows, 2), 127 + 16, dtype=torch.uint8)
    scales[:, 1] = 127 + 15
    W = sp.Mx4(codes.to(DEV), scales.to(DEV), cols)
    w = sp.mx4_dequantize(W, DTYPES[fmt])
    assert torch.isinf(w[:, :32]).all() == (fmt == "f16") and torch.isfinite(w[:, 32:]).all()
    C = rows if back else cols
    X = torch.zeros(tokens, C, dtype=DTYPES[fmt], device=DEV)
    X[:, 40] = 1.0
    Y = (sp.mx4_linear_grad if back else sp.mx4_linear)(X, W)
    want = X.double() @ (w.double() if back else w.double().t())
    assert np.array_equal(as_f64(Y), as_f64(want), equal_nan=True)


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
def test_bench_shapes(fmt):
    """The shapes of the adapters' layers, a sample of tokens in 64 bits, and the same bits on every call."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    for tokens, rows, cols in ((1, 4096, 4096), (16, 11008, 4096), (64, 11008, 4096), (1037, 4096, 4096), (8192, 8192, 2048),
                               (2048, 4096, 4096)):
        W = sp.mx4_quantize(torch.randn(rows, cols, device=DEV, generator=g).mul_(0.02).to(DTYPES[fmt]))
        w = sp.mx4_dequantize(W).double()
        for back in (False, True):
            X = torch.randn(tokens, rows if back else cols, device=DEV, generator=g).to(DTYPES[fmt])
            call, m = (sp.mx4_linear_grad, w) if back else (sp.mx4_linear, w.t())
            Y = call(X, W)
            for _ in range(3):
                assert torch.equal(call(X, W), Y)
            at = torch.cat([torch.arange(min(tokens, 40)), torch.arange(max(0, tokens - 40), tokens)]).unique().to(DEV)
            x = X[at].double()
            assert_elementwise(Y[at], (x @ m).cpu().numpy(), (x.abs() @ m.abs()).cpu().numpy(), m.shape[0], fmt,
                               f"{tokens} {rows} {cols} {back}")


@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("tokens,rows,cols", [(1, 8200, 8192), (5, 8448, 4096), (1300, 4352, 96), (1300, 4352, 352), (2600, 2304, 352), (2600, 2304, 200),
                                              (9000, 520, 64), (700, 6400, 416)])
def test_many_tiles(fmt, tokens, rows, cols):
    """Tiles that follow each other on an SM, with boxes of codes that end within a stage, and a weight of more values than
    the kernel for a few tokens takes."""
    g = torch.Generator(device=DEV)
    g.manual_seed(tokens + cols)
    W = sp.mx4_quantize(torch.randn(rows, cols, device=DEV, generator=g))
    w = sp.mx4_dequantize(W).double()
    for back in (False, True):
        X = torch.randn(tokens, rows if back else cols, device=DEV, generator=g).to(DTYPES[fmt])
        call, m = (sp.mx4_linear_grad, w) if back else (sp.mx4_linear, w.t())
        Y, x = call(X, W), X.double()
        assert torch.equal(call(X, W), Y)
        assert_elementwise(Y, (x @ m).cpu().numpy(), (x.abs() @ m.abs()).cpu().numpy(), m.shape[0], fmt, f"{back}")


@pytest.mark.parametrize("tokens,rows,cols,pad", [(3776, 5304, 24, 3), (3776, 5304, 24, 0), (3000, 5000, 96, 8), (2900, 5304, 300, 1)])
def test_short_sums_of_many_tiles(tokens, rows, cols, pad):
    """A stage or two of the contraction in each of a pair's many tiles, whose codes may arrive in any order: the same right
    result every time."""
    g = torch.Generator(device=DEV)
    g.manual_seed(cols)
    W = sp.mx4_quantize(torch.randn(rows, cols, device=DEV, generator=g))
    w = sp.mx4_dequantize(W).double()
    X = torch.randn(tokens, cols + 2 * pad, device=DEV, generator=g).bfloat16()[:, pad:pad + cols]
    x = X.double()
    want, mass = x @ w.t(), x.abs() @ w.t().abs()
    first = sp.mx4_linear(X, W)
    assert_elementwise(first, want.cpu().numpy(), mass.cpu().numpy(), cols, "bf16", "Y")
    for _ in range(300):
        assert torch.equal(sp.mx4_linear(X, W), first)


def test_streams_and_graphs():
    """Two streams at once, and a captured run whose replays see new inputs."""
    rng = np.random.default_rng(9)
    W, _ = weight(rng, 768, 512)
    xs = [rand(rng, "bf16", t, 512) for t in (1, 24, 90, 400)]
    want = [sp.mx4_linear(x, W) for x in xs]
    back = [sp.mx4_linear_grad(y, W) for y in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got.append([(y := sp.mx4_linear(x, W), sp.mx4_linear_grad(y, W)) for x in xs])
        torch.cuda.synchronize()
        for g in got:
            for (y, d), a, b in zip(g, want, back):
                assert torch.equal(y, a) and torch.equal(d, b)
    static = [torch.zeros_like(x) for x in xs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = [(y := sp.mx4_linear(x, W), sp.mx4_linear_grad(y, W)) for x in static]
        q = sp.mx4_dequantize(sp.mx4_quantize(static[3]))
    for _ in range(2):
        for a, b in zip(static, xs):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for (y, d), a, b in zip(out, want, back):
            assert torch.equal(y, a) and torch.equal(d, b)
        assert torch.equal(q, sp.mx4_dequantize(sp.mx4_quantize(xs[3])))


def test_two_graphs():
    """Graphs whose products have workspaces, replayed in turn with other inputs."""
    rng = np.random.default_rng(11)
    W, _ = weight(rng, 264, 320)
    graphs = []
    for fmt, pad in (("f32", 0), ("bf16", 3)):
        x = rand(rng, fmt, 50, 320, pad=pad)
        want = [sp.mx4_linear(x * f, W) for f in (1, 2)]
        back = [sp.mx4_linear_grad(y, W) for y in want]
        static = x.clone() if pad == 0 else torch.zeros(50, 320 + 2 * pad, dtype=x.dtype, device=DEV)[:, pad:pad + 320]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = sp.mx4_linear(static, W)
            d = sp.mx4_linear_grad(y, W)
        graphs.append((g, static, x, y, d, want, back))
    for i in (0, 1, 0):
        for g, static, x, *_ in graphs:
            static.copy_(x * (i + 1))
        for g, *_ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, static, x, y, d, want, back in graphs:
            assert torch.equal(y, want[i]) and torch.equal(d, back[i])


@pytest.mark.parametrize("tokens", [1, 5, 40])
def test_scales_of_any_alignment(tokens):
    rng = np.random.default_rng(12)
    W, _ = weight(rng, 192, 256)
    for offset in (1, 2, 3):
        buf = torch.empty(W.scales.numel() + offset, dtype=torch.uint8, device=DEV)
        scales = buf[offset:].view(W.scales.shape)
        scales.copy_(W.scales)
        V = sp.Mx4(W.codes, scales, 256)
        for fmt in DTYPES:
            X, G = rand(rng, fmt, tokens, 256), rand(rng, fmt, tokens, 192)
            assert torch.equal(sp.mx4_linear(X, V), sp.mx4_linear(X, W))
            assert torch.equal(sp.mx4_linear_grad(G, V), sp.mx4_linear_grad(G, W))
        assert torch.equal(sp.mx4_dequantize(V), sp.mx4_dequantize(W))


@pytest.mark.parametrize("cols", [4096, 4100])
def test_conversion_of_more_than_a_pass(cols):
    """More values than the threads of one grid take at a time."""
    X = torch.randn(6000, cols, device=DEV, generator=torch.Generator(device=DEV).manual_seed(cols)).bfloat16()
    W = sp.mx4_quantize(X)
    back = sp.mx4_dequantize(W)
    for r in (0, 1, 2999, 4444, 5999):
        codes, scales = ref.quantize(as_f64(X[r:r + 1]))
        assert np.array_equal(W.codes[r:r + 1].cpu().numpy(), codes) and np.array_equal(W.scales[r:r + 1].cpu().numpy(), scales)
        assert np.array_equal(as_f64(back[r:r + 1]), ref.values(codes, scales, cols))
    for lo in range(0, 6000, 1000):  # and the rows between: the same as by themselves
        part = sp.mx4_quantize(X[lo:lo + 1000])
        assert torch.equal(part.codes, W.codes[lo:lo + 1000]) and torch.equal(part.scales, W.scales[lo:lo + 1000])
        assert torch.equal(sp.mx4_dequantize(part), back[lo:lo + 1000])


def test_refusals():
    rng = np.random.default_rng(2)
    W, _ = weight(rng, 64, 96)
    X = rand(rng, "bf16", 10, 96)
    for bad, match in ((X[:, :95], "must be 10 x 96"), (X.t(), "must be"), (X[0], "2-D"), (X.double(), "dtype"),
                       (X.cpu(), "expected"), (X[:, ::2], "must be"), (X.expand(3, 10, 96), "2-D"),
                       (torch.zeros(10, 192, device=DEV)[:, ::2], "contiguous rows")):
        with pytest.raises(ValueError, match=match):
            sp.mx4_linear(bad, W)
    for bad, match in ((torch.empty(10, 63, dtype=X.dtype, device=DEV), "out must be"),
                       (torch.empty(10, 64, device=DEV), "dtype"), (X[:, :64], "overlaps")):
        with pytest.raises(ValueError, match=match):
            sp.mx4_linear(X, W, out=bad)
    leaf = torch.zeros(10, 64, dtype=X.dtype, device=DEV, requires_grad=True)
    with pytest.raises(RuntimeError, match="out is part of an autograd graph"):
        sp.mx4_linear(X, W, out=leaf)
    with torch.no_grad():
        sp.mx4_linear(X, W, out=leaf)
    assert torch.equal(leaf, sp.mx4_linear(X, W))
    out = torch.ones(10, 64, dtype=X.dtype, device=DEV)
    loss = (out * torch.ones_like(out).requires_grad_()).sum()
    sp.mx4_linear(X, W, out=out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    for codes, scales, cols in ((W.codes[:, :32], W.scales, 96), (W.codes, W.scales[:, :2], 96), (W.codes, W.scales, 97),
                                (W.codes.int(), W.scales, 96), (W.codes.t(), W.scales, 96), (W.codes, W.scales.cpu(), 96)):
        with pytest.raises(ValueError):
            sp.Mx4(codes, scales, cols)
    with pytest.raises(ValueError, match="16-byte"):
        sp.mx4_linear(X, sp.Mx4(torch.zeros(64 * 48 + 1, dtype=torch.uint8, device=DEV)[1:].view(64, 48), W.scales, 96))
    with pytest.raises(ValueError, match="dtype"):
        sp.mx4_dequantize(W, torch.float64)
