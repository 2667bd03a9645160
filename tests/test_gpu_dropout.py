"""Dropout without a stored mask, against the generator and the formula in numpy.

Bounds, fixed before any run: the mask is exact; base + x f with f rounded to fp32 and at most two fp32 roundings: off by
at most 2^-22 (|x f| + |base|), then half an ulp of the output's type."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
from helpers import as_f64, ulp

pytestmark = pytest.mark.gpu

sp = pytest.importorskip("unstructured_sparse_linear_gb300")

DEV = torch.device("cuda:0")
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SEED, CALL = 0x0123456789ABCDEF, 0xFEDCBA9876543210


def state(seed=SEED, call=CALL):
    return torch.from_numpy(np.array([seed, call], dtype=np.uint64).view(np.int64)).to(DEV)


def rand(fmt, rows, cols, seed, pad=0):
    x = torch.from_numpy(np.random.default_rng([seed, rows, cols]).standard_normal((rows, cols + pad)))
    return x.to(DTYPES[fmt]).to(DEV)[:, pad:]


def check(got, X, p, base, fmt, seed=SEED, call=CALL):
    x, b = as_f64(X), as_f64(base) if base is not None else np.zeros(X.shape)
    want = ref.dropout(x, p, seed, call, b)
    err = 2.0 ** -22 * (np.abs(want - b) + np.abs(b))
    assert np.all(np.abs(as_f64(got) - want) <= err + 0.5 * ulp(np.abs(want) + err, fmt))
    dropped = ref.numbers(*X.shape, seed, call) < ref.threshold(p)
    assert np.array_equal(as_f64(got)[dropped], b[dropped])


@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (3, 7), (5, 64), (2, 1000), (129, 33), (64, 4096), (300, 257)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout(fmt, rows, cols, p):
    X, base = rand(fmt, rows, cols, 1), rand(fmt, rows, cols, 2)
    Y = sp.dropout(X, p, state())
    check(Y, X, p, None, fmt)
    assert torch.equal(sp.dropout(X, p, (SEED, CALL)), Y)
    Z = sp.dropout(X, p, state(), base=base)
    check(Z, X, p, base, fmt)
    # columns of a wider matrix, aligned and not; in place
    for pad in (8, 3):
        wide = torch.full((rows + 1, cols + pad), 7.0, dtype=X.dtype, device=DEV)
        out = wide[:rows, pad:]
        xs, bs = rand(fmt, rows, cols, 3, pad), rand(fmt, rows, cols, 4, pad)
        assert sp.dropout(xs, p, state(), base=bs, out=out) is out
        check(out, xs, p, bs, fmt)
        assert (wide[:, :pad] == 7).all() and (wide[rows:] == 7).all()
        want = sp.dropout(xs, p, state(), base=bs)
        assert torch.equal(out, want)
        assert torch.equal(sp.dropout(xs.clone(), p, state(), base=bs, out=bs), want)
        want = sp.dropout(xs, p, state())
        assert torch.equal(sp.dropout(xs, p, state(), out=xs), want)


def test_what_is_dropped_is_zero_whatever_it_was():
    X = torch.full((64, 64), float("nan"), device=DEV)
    X[::2] = float("inf")
    keep = ref.numbers(64, 64, 1, 2) >= ref.threshold(0.3)
    Y = as_f64(sp.dropout(X, 0.3, (1, 2)))
    assert np.array_equal(Y == 0, ~keep) and np.isinf(Y[::2][keep[::2]]).all() and np.isnan(Y[1::2][keep[1::2]]).all()
    assert not sp.dropout(X, 1.0, (1, 2)).any()
    assert torch.equal(sp.dropout(X, 0.0, (1, 2)), X) or torch.isnan(X).any()


def test_share_and_independence():
    """Of 2^22 places a share p drops, within five standard deviations; another seed, call or row has another mask, whose
    agreement is that of chance."""
    n, p = 2 ** 22, 0.2
    X = torch.ones(1024, 4096, device=DEV)
    masks = [sp.dropout(X, p, s) == 0 for s in ((0, 0), (0, 1), (1, 0), (0, 2 ** 32), (2 ** 32, 0))]
    q = ref.threshold(p) / 65536
    sd = np.sqrt(q * (1 - q) / n)
    for m in masks:
        assert abs(float(m.double().mean()) - q) < 5 * sd
    both = q * q
    for i, a in enumerate(masks):
        for b in masks[i + 1:] + [a.roll(1, 0), a.roll(1, 1)]:
            assert abs(float((a & b).double().mean()) - both) < 5 * np.sqrt(both * (1 - both) / n)


def test_many_rows():
    """Rows and places beyond 2^31."""
    X = torch.ones(2 ** 28 + 3, 9, dtype=torch.bfloat16, device=DEV)
    Y = sp.dropout(X, 0.5, (5, 6))
    rows = 40
    for r0 in (0, 2 ** 27, 2 ** 28 + 3 - rows):
        index = np.arange(2 * r0, 2 * (r0 + rows), dtype=np.uint64)
        w = ref.philox7(index, 6, 5)
        u = np.stack([v for x in w for v in (x & np.uint64(0xFFFF), x >> np.uint64(16))], -1).reshape(rows, 16)[:, :9]
        assert np.array_equal(as_f64(Y[r0:r0 + rows]), np.where(u >= 32768, 2.0, 0.0))


def test_graph_replays_read_the_state():
    X = rand("bf16", 70, 384, 1)
    s = state(3, 0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y = sp.dropout(X, 0.25, s)
        s[1:].add_(1)
    for call in range(3):
        graph.replay()
        torch.cuda.synchronize()
        check(Y, X, 0.25, None, "bf16", 3, call)


def test_refusals():
    X = rand("bf16", 6, 16, 1)
    for kw, match in ((dict(p=1.5), "p must"), (dict(p=-0.1), "p must"), (dict(p=float("nan")), "p must"),
                      (dict(state=(-1, 0)), "seed and call"), (dict(state=(0, 2 ** 64)), "seed and call"),
                      (dict(state=torch.zeros(2, dtype=torch.int32, device=DEV)), "dtype"),
                      (dict(state=torch.zeros(2, dtype=torch.int64)), "CUDA"),
                      (dict(state=torch.zeros(3, dtype=torch.int64, device=DEV)), "seed and a call"),
                      (dict(base=X[:5]), "base must be"), (dict(out=X.float()), "dtype"), (dict(X=X.t()), "contiguous rows"),
                      (dict(X=X[0]), "2-D"), (dict(X=X.double()), "dtype")):
        args = dict(X=X, p=0.5, state=(0, 0))
        args.update(kw)
        with pytest.raises(ValueError, match=match):
            sp.dropout(**args)
    wide = torch.zeros(6, 40, dtype=X.dtype, device=DEV)
    with pytest.raises(ValueError, match="overlaps"):
        sp.dropout(wide[:, :16], 0.5, (0, 0), out=wide[:, 8:24])
    leaf = torch.zeros_like(X).requires_grad_()
    with pytest.raises(RuntimeError, match="out is part of an autograd graph"):
        sp.dropout(X, 0.5, (0, 0), out=leaf)
