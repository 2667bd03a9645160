"""4-bit weights whose scales are uncommon, in every kernel of the products (1 token, 2 to 8, the tiles), against the stored
values in 64 bits.

Bounds, fixed before any run: where one product makes an output, the product of an 8-bit and a 2-bit significand (11 bits in fp16)
is exact in fp32 and the output is it, rounded once; sums are bound as everywhere (helpers.assert_elementwise)."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
from helpers import as_f64, assert_elementwise

pytestmark = pytest.mark.gpu

sp = pytest.importorskip("unstructured_sparse_linear_gb300")

DEV = torch.device("cuda:0")
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BACK = pytest.mark.parametrize("back", [False, True], ids=["linear", "grad"])


def stored(codes, scales, cols):
    """A weight of codes (one of 0 to 15 a value) and scales, and its values in 64 bits."""
    rows = codes.shape[0]
    c = np.zeros((rows, scales.shape[1] * 32), dtype=np.uint8)
    c[:, :cols] = codes
    packed = c[:, ::2] | c[:, 1::2] << 4
    W = sp.Mx4(torch.from_numpy(packed).to(DEV), torch.from_numpy(scales.astype(np.uint8)).to(DEV), cols)
    return W, ref.values(packed, scales.astype(np.uint8), cols)


def product(X, W, back):
    return (sp.mx4_linear_grad if back else sp.mx4_linear)(X, W)


@pytest.mark.parametrize("fmt", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 2, 5, 8, 9, 40])
@BACK
def test_largest_scales(fmt, tokens, back):
    """2^125 to 2^127 with codes that stay finite, and X so small that the sums are ordinary numbers."""
    rng = np.random.default_rng(tokens)
    rows, cols = 72, 160
    scales = rng.integers(252, 255, (rows, 5))
    most = np.repeat(np.array([8, 6, 4])[scales - 252], 32, axis=1)  # 252: up to 6, 253: 3, 254: 1.5
    codes = rng.integers(0, most) + 8 * rng.integers(0, 2, (rows, cols))
    W, w = stored(codes, scales, cols)
    assert np.isfinite(w.astype(np.float32)).all()
    m = w if back else w.T
    X = torch.from_numpy(rng.standard_normal((tokens, m.shape[0])) * 2.0 ** -60).to(DTYPES[fmt]).to(DEV)
    x = as_f64(X)
    Y = product(X, W, back)
    assert_elementwise(Y, x @ m, np.abs(x) @ np.abs(m), m.shape[0], fmt, "Y")
    # (what cancels, too)
    ones, _ = stored(np.tile([2, 10], (rows, cols // 2)), np.full((rows, 5), 253), cols)
    if not back:
        assert not product(torch.full((tokens, cols), 2.0 ** -60, dtype=X.dtype, device=DEV), ones, False).any()


@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("tokens", [1, 2, 5, 8, 9, 40, 256])
@BACK
def test_every_scale_with_a_finite_value(fmt, tokens, back):
    """A one in each row of X picks single values, of scales that follow each other at random: all bytes but 255 with codes that
    stay finite, in fp16 from one whose values are all zero on; rounded to the type."""
    rng = np.random.default_rng([tokens, 1])
    C, F = 320, 136
    rows, cols = (C, F) if back else (F, C)
    blocks = -(-cols // 32)
    scales = rng.integers(98, 142, (rows, blocks)) if fmt == "f16" else rng.integers(0, 255, (rows, blocks))
    at = np.repeat(scales, 32, axis=1)[:, :cols]
    most = np.where(at == 141, 6, 8) if fmt == "f16" else np.where(at == 253, 6, np.where(at == 254, 4, 8))
    codes = rng.integers(0, most, (rows, cols)) + 8 * rng.integers(0, 2, (rows, cols))
    W, w = stored(codes, scales, cols)
    w = torch.from_numpy(w).to(DTYPES[fmt]).double().numpy()
    assert np.isfinite(w).all()
    m = w if back else w.T
    pick = rng.permutation(C)[:tokens]
    X = torch.zeros(tokens, C, dtype=DTYPES[fmt])
    X[torch.arange(tokens), torch.from_numpy(pick)] = 1.0
    assert np.array_equal(as_f64(product(X.to(DEV), W, back)), m[pick])


@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("tokens", [1, 2, 8, 9, 40])
@BACK
def test_sums_of_uncommon_scales(fmt, tokens, back):
    """Dense products; blocks of common scales among others."""
    rng = np.random.default_rng([tokens, 2])
    C, F = 1056, 200
    rows, cols = (C, F) if back else (F, C)
    blocks = -(-cols // 32)
    uncommon = rng.integers(96, 140, (rows, blocks)) if fmt == "f16" else rng.integers(20, 240, (rows, blocks))
    scales = np.where(rng.random((rows, blocks)) < 0.5, rng.integers(120, 130, (rows, blocks)), uncommon)
    codes = rng.integers(0, 16, (rows, cols))
    W, w = stored(codes, scales, cols)
    w = torch.from_numpy(w).to(DTYPES[fmt]).double().numpy()
    m = w if back else w.T
    std = 2.0 ** -9 if fmt == "f16" else 1.0  # (6 * 2^12 * 33 of them: within fp16)
    X = torch.from_numpy(rng.standard_normal((tokens, C)) * std).to(DTYPES[fmt]).to(DEV)
    x = as_f64(X)
    assert_elementwise(product(X, W, back), x @ m, np.abs(x) @ np.abs(m), C, fmt, "Y")


@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("tokens", [1, 2, 8, 9, 40])
@BACK
def test_beyond_the_type_beside_others(fmt, tokens, back):
    """Every other block of features has values that the type does not hold: infinite there (of both signs: NaN where they
    meet), untouched elsewhere. fp32 may have NaN for an infinity, from the parts of X that are zero."""
    rng = np.random.default_rng([tokens, 3])
    C, F = 96, 192
    rows, cols = (C, F) if back else (F, C)
    blocks = cols // 32
    top = (141, 146) if fmt == "f16" else (252, 255)
    scales = rng.integers(120, 130, (rows, blocks))
    feature = np.arange(F) // 32 % 2 == 1
    high = rng.integers(*top, (rows, blocks))
    scales = np.where(feature[::32][None, :] if back else feature[:, None], high, scales)
    codes = rng.integers(0, 16, (rows, cols))
    W, w = stored(codes, scales, cols)
    w = torch.from_numpy(w).to(DTYPES[fmt]).double().numpy()
    m = w if back else w.T
    assert np.isinf(m[:, feature]).any() and np.isfinite(m[:, ~feature]).all()
    std = 1.0 if fmt == "f16" else 2.0 ** -8  # (sums of finite values of 2^126 and more)
    X = torch.from_numpy(rng.standard_normal((tokens, C)) * std).to(DTYPES[fmt]).to(DEV)
    x, Y = as_f64(X), as_f64(product(X, W, back))
    assert (x != 0).all()
    with np.errstate(invalid="ignore"):
        want = x @ m
    hit = ~np.isfinite(want)
    assert np.isfinite(want[:, ~feature]).all() and not np.isfinite(Y[hit]).any()
    if fmt != "f32":
        assert np.array_equal(Y[hit], want[hit], equal_nan=True)
    plain = ~feature
    assert_elementwise(torch.from_numpy(Y[:, plain]), want[:, plain], np.abs(x) @ np.abs(m[:, plain]), C, fmt, "Y")
