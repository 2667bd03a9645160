"""Products with a 4-bit weight where X's values lie far apart, in every kernel (1 token, 2 to 8, the tiles), against 64 bits.

Bounds, fixed before any run: an output of one product (significands of 8 bits and 2, 11 and 2 in fp16, 22 and 2 in fp32, all
exact in fp32) is that product rounded once, bit for bit, whatever zeros meet; sums are bound as everywhere
(helpers.assert_elementwise), by the products that there are."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
from helpers import as_f64, assert_elementwise, ulp

pytestmark = pytest.mark.gpu

sp = pytest.importorskip("unstructured_sparse_linear_gb300")

DEV = torch.device("cuda:0")
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BACK = pytest.mark.parametrize("back", [False, True], ids=["linear", "grad"])
LOW = {"f32": -100, "f16": -24, "bf16": -100}  # the least exponent of X: the products stay normal in the 8-bit exponents' types


def stored(codes, scales, cols):
    """A weight of codes (one of 0 to 15 a value) and scales, and its values in 64 bits."""
    rows = codes.shape[0]
    c = np.zeros((rows, scales.shape[1] * 32), dtype=np.uint8)
    c[:, :cols] = codes
    packed = c[:, ::2] | c[:, 1::2] << 4
    W = sp.Mx4(torch.from_numpy(packed).to(DEV), torch.from_numpy(scales.astype(np.uint8)).to(DEV), cols)
    return W, ref.values(packed, scales.astype(np.uint8), cols)


def sparse_weight(rng, C, F, back, terms):
    """A weight with `terms` values that are not zero for each of F results."""
    picks = np.stack([rng.choice(C, terms, replace=False) for _ in range(F)])
    m = np.zeros((C, F), dtype=np.int64)
    m[picks.T, np.arange(F)] = rng.integers(1, 8, (terms, F)) + 8 * rng.integers(0, 2, (terms, F))
    codes = m if back else m.T
    rows, cols = codes.shape
    return stored(codes, rng.integers(124, 131, (rows, -(-cols // 32))), cols)


def spread(rng, fmt, tokens, C, low=-1000):
    mant = rng.integers(2 ** 21, 2 ** 22, (tokens, C)) * 2.0 ** -21  # (22 bits; fewer types have fewer)
    x = mant * np.ldexp(1.0, rng.integers(max(LOW[fmt], low), 1, (tokens, C))) * rng.choice([-1.0, 1.0], (tokens, C))
    return torch.from_numpy(x).to(DTYPES[fmt]).to(DEV)


def product(X, W, back):
    return (sp.mx4_linear_grad if back else sp.mx4_linear)(X, W)


@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("tokens", [1, 2, 5, 8, 9, 40])
@pytest.mark.parametrize("C,F", [(32, 40), (97, 64), (1000, 264), (17000, 96)])
@pytest.mark.parametrize("low", [-1000, -30, -24])
@BACK
def test_single_products(fmt, tokens, C, F, back, low):
    rng = np.random.default_rng([tokens, C])
    W, w = sparse_weight(rng, C, F, back, 1)
    X = spread(rng, fmt, tokens, C, low)
    want = torch.from_numpy(as_f64(X) @ (w if back else w.T)).to(X.dtype)
    assert torch.equal(product(X, W, back).cpu(), want)


@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("tokens", [1, 2, 5, 8, 9, 40])
@pytest.mark.parametrize("terms", [2, 300])
@BACK
def test_sums(fmt, tokens, terms, back):
    rng = np.random.default_rng([tokens, terms])
    C, F = 520, 200
    W, w = sparse_weight(rng, C, F, back, terms)
    X, m = spread(rng, fmt, tokens, C), w if back else w.T
    x = as_f64(X)
    assert_elementwise(product(X, W, back), x @ m, np.abs(x) @ np.abs(m), C, fmt, "Y")


@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("tokens", [2, 5, 8, 40])
def test_tokens_do_not_meet(fmt, tokens):
    """The bits of a token's result, whatever values its neighbours have."""
    rng = np.random.default_rng(tokens)
    W, _ = sparse_weight(rng, 640, 200, False, 400)
    X = torch.from_numpy(rng.standard_normal((tokens, 640))).to(DTYPES[fmt]).to(DEV)
    plain, other = sp.mx4_linear(X, W), X.clone()
    other[1] = spread(rng, fmt, 1, 640)[0]
    got = sp.mx4_linear(other, W)
    rest = torch.arange(tokens) != 1
    assert torch.equal(got[rest], plain[rest]) and not torch.equal(got[1], plain[1])


@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("tokens", [1, 2, 8, 40])
@BACK
def test_an_infinity_beside_them(fmt, tokens, back):
    rng = np.random.default_rng(tokens)
    W, w = sparse_weight(rng, 96, 64, back, 96)  # (no zeros)
    X = spread(rng, fmt, tokens, 96)
    X[:, 40] = float("inf")
    want = np.copysign(np.inf, (w if back else w.T)[40])
    assert np.array_equal(as_f64(product(X, W, back)), np.tile(want, (tokens, 1)))


@pytest.mark.parametrize("fmt", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 2, 5, 8, 9, 40])
@pytest.mark.parametrize("x_exp,w_byte", [(-70, 60), (-20, 10), (-115, 105), (-44, 36), (-47, 61), (-2, 0)])
@BACK
def test_small_values_on_both_sides(fmt, tokens, x_exp, w_byte, back):
    """Sums of 4096 products of about 2^-134 (2^-122 and more), in range although X's power of two times the scale is not. Products
    are multiples of 2^-149, as fp32's sums are, so the bound on sums holds for them; one more half step for those below a
    multiple in bf16's and fp32's subnormal numbers is in helpers.ulp."""
    rng = np.random.default_rng(tokens)
    C, F = 4096, 40
    rows, cols = (C, F) if back else (F, C)
    W, w = stored(rng.integers(4, 8, (rows, cols)), np.full((rows, -(-cols // 32)), w_byte), cols)
    m = w if back else w.T
    X = torch.from_numpy((1 + rng.integers(0, 64, (tokens, C)) / 64) * 2.0 ** x_exp).to(DTYPES[fmt]).to(DEV)
    x = as_f64(X)
    assert_elementwise(product(X, W, back), x @ m, np.abs(x) @ np.abs(m), C, fmt, "Y")


@pytest.mark.parametrize("tokens", [1, 2, 8])
def test_a_large_scale_and_large_values(tokens):
    """X's power of two times the scale beyond fp32's range, the products within it."""
    rng = np.random.default_rng(tokens)
    C, F = 96, 64
    x = np.ldexp(1.0, rng.integers(100, 128, (tokens, C))) * rng.choice([-1.0, 1.0], (tokens, C))
    x[:, ::32] = 2.0 ** 127
    pick = rng.choice(np.setdiff1d(np.arange(C), [0, 32, 64]), F)
    x[:, pick] = np.ldexp(1.0, rng.integers(96, 100, F))  # 2^99 at most; times 6 * 2^20 no more than 2^122
    codes = np.zeros((F, C), dtype=np.int64)
    codes[np.arange(F), pick] = rng.integers(1, 8, F)
    W, w = stored(codes, np.full((F, 3), 147), C)
    X = torch.from_numpy(x).to(torch.bfloat16).to(DEV)
    assert torch.equal(sp.mx4_linear(X, W).cpu(), torch.from_numpy(as_f64(X) @ w.T).bfloat16())


@pytest.mark.parametrize("tokens", [1, 8, 40, 300])
@BACK
def test_small_fp32_numbers(tokens, back):
    """All 24 bits from 2^-110 on; below, the third bf16 part is off by half of 2^-133. One product an output, of fp32's normal numbers,
    rounded once."""
    rng = np.random.default_rng(tokens)
    C, F = 320, 200
    codes = np.zeros((C, F) if back else (F, C), dtype=np.int64)
    pick = rng.integers(0, C, F)
    codes[(pick, np.arange(F)) if back else (np.arange(F), pick)] = rng.integers(1, 8, F)
    W, w = stored(codes, np.full((codes.shape[0], -(-codes.shape[1] // 32)), 127 + 60), codes.shape[1])
    m = w if back else w.T
    x = (rng.integers(2 ** 23, 2 ** 24, (tokens, C)) * 2.0 ** -23) * np.ldexp(1.0, rng.integers(-126, -104, (tokens, C)))
    X = torch.from_numpy(x).float().to(DEV)
    assert np.array_equal(as_f64(X), x)
    want = x @ m
    left = np.where(x[:, pick] < 2.0 ** -110, 2.0 ** -134, 0.0) * m[pick, np.arange(F)]
    assert np.all(np.abs(as_f64(product(X, W, back)) - want) <= left + 0.5 * ulp(want + left, "f32"))
