"""Host-side checks of the 4-bit weights and of dropout that need no GPU: the reference they are tested against, and
arguments refused before the device is touched (the pointers below are never dereferenced)."""
import ctypes

import numpy as np
import pytest
import torch

import mx4_reference as ref

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from unstructured_sparse_linear_gb300 import _lib, build
    build.build()
    return _lib.load()


def test_reference_generator_known_answers():
    """Published vectors of Philox4x32 with 7 rounds (the generator's own test set)."""
    zero = ref.philox7(np.zeros(1, dtype=np.uint64), 0, 0)
    assert [int(w[0]) for w in zero] == [0x5f6fb709, 0x0d893f64, 0x4f121f81, 0x4f730a48]
    ones = ref.philox7(np.full(1, 2 ** 64 - 1, dtype=np.uint64), 2 ** 64 - 1, 2 ** 64 - 1)
    assert [int(w[0]) for w in ones] == [0x5207ddc2, 0x45165e59, 0x4d8ee751, 0x8c52f662]


def test_reference_quantization_by_hand():
    x = np.zeros((3, 33))
    x[0, :9] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.3]
    x[0, 32] = 7.9  # beyond 6: to 6
    x[1, 0] = np.inf
    x[1, 32] = -2.0 ** -130
    codes, scales = ref.quantize(x)
    assert scales.tolist() == [[127, 127], [255, 0], [0, 0]]
    got = ref.values(codes, scales, 33)
    assert got[0, :9].tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -0.5] and got[0, 32] == 6.0
    assert np.isnan(got[1, :32]).all() and got[1, 32] == 0 and not got[2].any()
    assert codes.shape == (3, 32) and not codes[:, 17:].any()


def product(lib, back=False, **kw):
    from unstructured_sparse_linear_gb300 import mx4
    a = dict(X=0x100000, ldx=64, codes=0x200000, scales=0x300000, Y=0x400000, ldy=64, ws=0, size=0, stream=0, dtype=2,
             tokens=8, rows=64, cols=64)
    a.update(kw)
    f = lib.spops_mx4_linear_grad if back else lib.spops_mx4_linear
    return f(mx4._ARGS(*a.values()))


@pytest.mark.parametrize("back", [False, True])
def test_product_refusals(lib, back):
    assert (lib.spops_mx4_linear_grad if back else lib.spops_mx4_linear)(None) == 1
    assert product(lib, back, tokens=0) == 0 and product(lib, back, **{"cols" if back else "rows": 0}) == 0
    for bad in (dict(dtype=3), dict(dtype=-1), dict(tokens=-1), dict(rows=-1), dict(cols=-1), dict(X=0), dict(Y=0),
                dict(codes=0), dict(scales=0), dict(X=0x100001), dict(Y=0x400001), dict(codes=0x200008), dict(ldx=63),
                dict(ldy=63), dict(Y=0x100000), dict(Y=0x100040), dict(Y=0x200000), dict(Y=0x300010)):
        assert product(lib, back, **bad) == 1, bad
        assert lib.spops_last_error()
    odd = dict(X=0x100002, tokens=20, ldx=72, ldy=72)  # rows that need a copy
    need = lib.spops_mx4_workspace_size(20, 64, 64, 2)
    assert lib.spops_mx4_workspace_size(20, 64, 64, 0) >= 20 * 64 * (3 * 2 + 4) and lib.spops_mx4_workspace_size(-1, 64, 64, 2) == 0
    assert product(lib, back, dtype=0) == 3
    assert need >= 2 * 20 * 64 * 2
    for bad in (dict(), dict(ws=0x500000, size=need - 1), dict(ws=0x500008, size=need)):
        assert product(lib, back, **odd, **bad) == 3, bad
    for bad in (0x400040, 0x100040, 0x200000, 0x300010):
        assert product(lib, back, **odd, ws=bad, size=need) == 1
    big = 0x7fff0001
    assert product(lib, back, tokens=big) == 2 and product(lib, back, rows=big) == 2 and product(lib, back, cols=big) == 2
    long = dict(rows=715827841) if back else dict(cols=715827841)  # three parts of fp32 beside each other pass 2^31
    assert product(lib, back, dtype=0, **long) == 2 and product(lib, back, dtype=1, tokens=0, **long) == 0


def test_conversion_refusals(lib):
    def q(X=0x100000, ldx=64, dtype=1, rows=4, cols=64, codes=0x200000, scales=0x300000):
        return lib.spops_mx4_quantize(P(X), ldx, dtype, rows, cols, P(codes), P(scales), None)

    def d(codes=0x200000, scales=0x300000, rows=4, cols=64, Y=0x100000, ldy=64, dtype=1):
        return lib.spops_mx4_dequantize(P(codes), P(scales), rows, cols, P(Y), ldy, dtype, None)

    for f in (q, d):
        assert f(rows=0) == 0 and f(cols=0) == 0
        for bad in (dict(dtype=5), dict(rows=-1), dict(cols=-2), dict(codes=0), dict(scales=0), dict(codes=0x200004),
                    dict(codes=0x100010), dict(scales=0x100010)):
            assert f(**bad) == 1, bad
        assert f(rows=0x7fff0001) == 2 and f(cols=0x7fff0001) == 2
    assert q(X=0) == 1 and q(X=0x100001) == 1 and q(ldx=63) == 1 and q(scales=0x200001) == 1
    assert d(Y=0) == 1 and d(Y=0x100001) == 1 and d(ldy=63) == 1


def drop(lib, **kw):
    from unstructured_sparse_linear_gb300.dropout import _ARGS
    a = dict(X=0x100000, ldx=64, base=0x200000, ldb=64, Y=0x300000, ldy=64, state=0, seed=1, call=2, stream=0, p=0.1,
             dtype=2, rows=8, cols=64)
    a.update(kw)
    return lib.spops_dropout(_ARGS(*a.values()))


def test_dropout_refusals(lib):
    assert lib.spops_dropout(None) == 1
    assert drop(lib, rows=0) == 0 and drop(lib, cols=0) == 0
    for bad in (dict(p=-0.1), dict(p=1.1), dict(p=float("nan")), dict(dtype=4), dict(rows=-1), dict(cols=-1), dict(X=0),
                dict(Y=0), dict(X=0x100001), dict(base=0x200001), dict(ldx=63), dict(ldb=63), dict(ldy=63),
                dict(state=0x400004), dict(Y=0x100040), dict(Y=0x100000, ldy=72), dict(Y=0x200010), dict(Y=0x200000, ldy=72),
                dict(state=0x300008)):
        assert drop(lib, **bad) == 1, bad
        assert lib.spops_last_error()


def test_weights_are_checked():
    import unstructured_sparse_linear_gb300 as sp
    codes, scales = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="codes must be a CUDA tensor"):
        sp.Mx4(codes, scales, 64)
    with pytest.raises(TypeError, match="codes must be a torch.Tensor"):
        sp.Mx4(None, scales, 64)
    for call in (lambda: sp.mx4_linear(torch.zeros(2, 64), codes), lambda: sp.mx4_linear_grad(torch.zeros(2, 4), codes),
                 lambda: sp.mx4_dequantize(codes)):
        with pytest.raises(TypeError, match="must be an Mx4"):
            call()
    with pytest.raises(ValueError, match="X must be a CUDA tensor"):
        sp.mx4_quantize(torch.zeros(2, 64))
    with pytest.raises(ValueError, match="X must be a CUDA tensor"):
        sp.dropout(torch.zeros(2, 64), 0.5, (0, 0))
