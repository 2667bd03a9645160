"""Products of fp32 activations with a 4-bit weight: that all three parts of X take part, in every form of the kernels (stages of 64
and 128 of the contraction, splits, rings that are used again, several tiles a pair), and how exact the sums are.

Bounds, fixed before any run. One product an output, of 22 bits and 2: exact in fp32, so is the output. Sums of C products of normal numbers:
relative Frobenius errors within four times the documented 4e-8 (C up to 384) and 2e-7 (up to 4096); they do not grow with
the count of outputs, and leaving out the third part of X (2^-16 of each number) or one of the two accumulators (1.2e-6) is
outside, the first of which is computed here."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
from helpers import as_f64, rel_fro

pytestmark = pytest.mark.gpu

sp = pytest.importorskip("unstructured_sparse_linear_gb300")

DEV = torch.device("cuda:0")
BACK = pytest.mark.parametrize("back", [False, True], ids=["linear", "grad"])


def product(X, W, back):
    return (sp.mx4_linear_grad if back else sp.mx4_linear)(X, W)


@pytest.mark.parametrize("tokens,C,F", [(1, 4096, 256), (9, 64, 512), (20, 11008, 300), (33, 4096, 4096), (64, 1000, 264), (130, 11008, 512),
                                        (200, 72, 3000), (501, 384, 1536), (700, 2048, 6136), (2600, 352, 2304), (3000, 40, 5000)])
@BACK
def test_every_bit_of_x(tokens, C, F, back):
    g = torch.Generator(device=DEV).manual_seed(tokens + C)
    pick = torch.randint(0, C, (F,), device=DEV, generator=g)
    code = torch.randint(1, 8, (F,), device=DEV, generator=g)
    m = torch.zeros(C, F, dtype=torch.uint8, device=DEV)
    m[pick, torch.arange(F, device=DEV)] = code.to(torch.uint8)
    rows, cols = (C, F) if back else (F, C)
    codes = torch.nn.functional.pad(m if back else m.t(), (0, -cols % 32)).contiguous()
    scales = torch.full((rows, codes.shape[1] // 32), 127, dtype=torch.uint8, device=DEV)
    W = sp.Mx4(codes[:, ::2] | codes[:, 1::2] << 4, scales, cols)
    mant = torch.randint(2 ** 21, 2 ** 22, (tokens, C), device=DEV, generator=g).float()  # (22 bits)
    X = mant * 2.0 ** -21 * (torch.randint(0, 2, (tokens, C), device=DEV, generator=g) * 2 - 1)
    w = torch.tensor(ref.GRID, dtype=torch.float32, device=DEV)[code]
    assert torch.equal(product(X, W, back), X[:, pick] * w)


@pytest.mark.parametrize("tokens,C,F,limit", [(17, 384, 512, 1.6e-7), (501, 384, 1536, 1.6e-7), (3000, 256, 2304, 1.6e-7),
                                              (9, 4096, 1024, 8e-7), (64, 4096, 4096, 8e-7), (700, 4096, 2048, 8e-7)])
@BACK
def test_exactness_of_sums(tokens, C, F, limit, back):
    g = torch.Generator(device=DEV).manual_seed(tokens + C)
    rows, cols = (C, F) if back else (F, C)
    W = sp.mx4_quantize(torch.randn(rows, cols, device=DEV, generator=g))
    w = sp.mx4_dequantize(W).double()
    m = w if back else w.t()
    X = torch.randn(tokens, C, device=DEV, generator=g)
    want = as_f64(X.double() @ m)
    assert rel_fro(as_f64(product(X, W, back)), want) <= limit
    top = (X.view(torch.int32) & -65536).view(torch.float32)
    middle = ((X - top).view(torch.int32) & -65536).view(torch.float32)
    assert rel_fro(as_f64((top.double() + middle.double()) @ m), want) > limit
