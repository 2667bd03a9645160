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
