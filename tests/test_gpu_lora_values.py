"""Infinities and values of very different magnitudes in the low-rank products, on both kernels."""
import numpy as np
import pytest
import torch

from helpers import ACC_UNIT, as_f64, ulp

pytestmark = pytest.mark.gpu

sp = pytest.importorskip("unstructured_sparse_linear_gb300")

DEV = torch.device("cuda:0")
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
K, N = 72, 136


def operands(fmt, tokens, rank, seed=0, k=K, n=N):
    rng = np.random.default_rng([seed, tokens, rank])

    def rand(*shape):
        return torch.from_numpy(rng.standard_normal(shape)).to(DTYPES[fmt]).to(DEV)

    return dict(X=rand(tokens, k), A=rand(1, rank, k).abs() * 0.125, B=rand(1, n, rank).abs() * 0.25, base=rand(tokens, n),
                dY=rand(tokens, n), dX_base=rand(tokens, k), plan=sp.lora_plan(None, 1, tokens=tokens, device=DEV))


# on both sides of the choice between the kernels
SIZES = [(5, 1), (11000, 1), (2600, 5), (40, 24), (700, 24), (700, 33), (300, 100)]


@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("tokens,rank", SIZES)
def test_an_infinity_in_a_row_gives_the_formulas_infinity(fmt, tokens, rank):
    """With A, B > 0 a row of X with an infinity has P = inf in every column, Y = inf; the gradients likewise."""
    d = operands(fmt, tokens, rank)
    args = d["A"], d["B"], d["plan"]
    clean = sp.lora_add(d["X"], *args, base=d["base"])
    clean_dX = sp.lora_grad(d["dY"], d["X"], *args, dX_base=d["dX_base"], need=(True, False, False))[0]
    hit = tokens // 2
    X, dY = d["X"].clone(), d["dY"].clone()
    X[hit, 3], dY[hit, 2] = float("inf"), float("inf")
    Y, h = sp.lora_add(X, *args, base=d["base"], return_h=True)
    dX, dA, _ = sp.lora_grad(dY, d["X"], *args, dX_base=d["dX_base"])
    torch.cuda.synchronize()
    keep = torch.arange(tokens, device=DEV) != hit
    assert torch.equal(Y[keep], clean[keep]) and torch.equal(dX[keep], clean_dX[keep])
    assert (Y[hit] == float("inf")).all() and (h[hit] == float("inf")).all() and (dX[hit] == float("inf")).all()
    want = torch.full((rank, K), float("inf"), device=DEV) * d["X"][hit].float()
    assert torch.equal(dA[0].float(), want)


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("rank", [16, 64])
def test_scattered_tokens_give_the_bits_of_tokens_in_runs(fmt, rank):
    """Rows that come by fours and leave by ordinary stores, through many reuses of every stage of the ring."""
    T, k, n, adapters = 1900, 1032, 2056, 5
    d = operands(fmt, T, rank, seed=2, k=k, n=n)
    A, B = (d[x] * torch.arange(1, adapters + 1, device=DEV, dtype=DTYPES[fmt])[:, None, None] for x in "AB")
    ids = torch.randint(-1, adapters, (T,), dtype=torch.int32, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    runs = torch.argsort(torch.where(ids < 0, adapters, ids), stable=True)
    plan, plan_runs = sp.lora_plan(ids, adapters), sp.lora_plan(ids[runs].contiguous(), adapters)
    Y = sp.lora_add(d["X"][runs], A, B, plan_runs, base=d["base"][runs])
    dX = sp.lora_grad(d["dY"][runs], d["X"][runs], A, B, plan_runs, dX_base=d["dX_base"][runs])
    for _ in range(3):
        got = sp.lora_add(d["X"], A, B, plan, base=d["base"])
        grads = sp.lora_grad(d["dY"], d["X"], A, B, plan, dX_base=d["dX_base"])
        assert torch.equal(got[runs], Y) and torch.equal(grads[0][runs], dX[0])
        assert torch.equal(grads[1], dX[1]) and torch.equal(grads[2], dX[2])


# What the two fp16 parts of P hold: 22 bits, or what is below 2^-50 of the largest value of its row (second
# product) or of its rank's column (weight gradients).
FP16_BITS, FP16_FLOOR = 2.0 ** -22, 2.0 ** -50


def spread(rng, exps, *shape):
    """fp16 values of four bits each, every rank j of about 2^exps[j]; shape[-2] or shape[-1] is the rank."""
    x = (1 + rng.integers(0, 8, shape) / 8) * rng.choice([-1.0, 1.0], shape)
    at = 1 if shape[1] == len(exps) else 2
    return x * (2.0 ** np.asarray(exps)).reshape([-1 if i == at else 1 for i in range(3)])


def assert_within(got, want, err, fmt, what):
    g = as_f64(got)
    bound = err + 0.5 * ulp(np.abs(want) + err, fmt)
    diff = np.abs(g - want)
    assert np.isfinite(g).all() and (diff <= bound).all(), (what, float((diff / bound)[np.isfinite(diff)].max()))


@pytest.mark.parametrize("tokens,rank", [(40, 16), (700, 16), (2500, 24), (700, 40), (400, 100)])
def test_fp16_ranks_of_very_different_magnitudes(tokens, rank):
    """A's rows fall from 2^14 to 2^-20 while B's columns rise by as much: every rank counts in Y and in dX."""
    rng = np.random.default_rng([11, tokens, rank])
    exps = np.round(np.linspace(14, -20, rank))
    d = operands("f16", tokens, rank, seed=11)
    A, B = (torch.from_numpy(spread(rng, e, *s)).half().to(DEV) for e, s in ((exps, (1, rank, K)), (-6 - exps, (1, N, rank))))
    a, b = as_f64(A)[0], as_f64(B)[0]
    assert (np.abs(a) > 0).all() and (np.abs(b) > 0).all()

    def want(U, W1, W2, base):
        P, terms = U @ W1, np.abs(U) @ np.abs(W1)
        e = ACC_UNIT * U.shape[1] * terms + np.maximum(FP16_BITS * np.abs(P), FP16_FLOOR * np.abs(P).max(1, keepdims=True))
        return base + P @ W2, e @ np.abs(W2) + ACC_UNIT * (rank + 4) * (np.abs(base) + np.abs(P) @ np.abs(W2))

    Y = sp.lora_add(d["X"], A, B, d["plan"], base=d["base"])
    assert_within(Y, *want(as_f64(d["X"]), a.T, b.T, as_f64(d["base"])), "f16", "Y")
    dY = d["dY"] * 0.0625
    dX = sp.lora_grad(dY, d["X"], A, B, d["plan"], dX_base=d["dX_base"], need=(True, False, False))[0]
    assert_within(dX, *want(as_f64(dY), b, a, as_f64(d["dX_base"])), "f16", "dX")


@pytest.mark.parametrize("tokens,rank", [(40, 16), (700, 16), (2500, 24), (700, 40), (400, 100)])
def test_fp16_weight_gradients_beside_large_ranks_and_tokens(tokens, rank):
    """Ranks 2^16 apart and one token 2^12 above the others that meets zeros: the small ones keep their bits."""
    rng = np.random.default_rng([12, tokens, rank])
    exps = np.round(np.linspace(8, -8, rank))
    d = operands("f16", tokens, rank, seed=12)
    X, dY, hit = d["X"].clone(), d["dY"] * 0.0625, tokens // 3

    def weight_gradient(U, W, V):
        """sum over t of (U W)[t, j] V[t, x] and its bound."""
        P, terms = U @ W, np.abs(U) @ np.abs(W)
        e = ACC_UNIT * U.shape[1] * terms + np.maximum(FP16_BITS * np.abs(P), FP16_FLOOR * np.abs(P).max(0, keepdims=True))
        return P.T @ V, (e + ACC_UNIT * (tokens + 4) * np.abs(P)).T @ np.abs(V)

    # dB: the outlier is a row of X
    A = torch.from_numpy(spread(rng, exps, 1, rank, K)).half().to(DEV)
    X1, dY1 = X.clone(), dY.clone()
    X1[hit] *= 4096
    dY1[hit] = 0
    dB = sp.lora_grad(dY1, X1, A, d["B"], d["plan"], need=(False, False, True))[2]
    G, e = weight_gradient(as_f64(X1), as_f64(A)[0].T, as_f64(dY1))
    assert_within(dB[0], G.T, e.T, "f16", "dB")
    # dA: of dY
    B = torch.from_numpy(spread(rng, exps, 1, N, rank)).half().to(DEV)
    X2, dY2 = X.clone(), dY.clone()
    dY2[hit] *= 4096
    X2[hit] = 0
    dA = sp.lora_grad(dY2, X2, d["A"], B, d["plan"], need=(False, True, False))[1]
    G, e = weight_gradient(as_f64(dY2), as_f64(B)[0], as_f64(X2))
    assert_within(dA[0], G, e, "f16", "dA")


@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("tokens,rank", [(5, 3), (700, 16), (2600, 24), (700, 33), (300, 100)])
def test_an_infinity_beside_p_gives_the_formulas_infinity(fmt, tokens, rank):
    """An infinity in the operand that meets P: the sign of the sum is P's, whatever parts P is multiplied in."""
    d = operands(fmt, tokens, rank, seed=4)
    hit = tokens // 2
    _, h = sp.lora_add(d["X"], d["A"], d["B"], d["plan"], return_h=True)
    dY, X, A, B = d["dY"].clone(), d["X"].clone(), d["A"].clone(), d["B"].clone()
    dY[hit, 2] = float("inf")
    dB = sp.lora_grad(dY, X, A, B, d["plan"], need=(False, False, True))[2][0]
    assert torch.equal(dB[2].float(), h[hit] * float("inf")) and dB[3:].isfinite().all()
    X[hit, 3] = float("inf")
    dA = sp.lora_grad(d["dY"], X, A, B, d["plan"], need=(False, True, False))[1][0]
    assert torch.equal(dA[:, 3].double(), (d["dY"][hit].double() @ B[0].double()) * float("inf"))
    assert dA[:, 4:].isfinite().all()
    B[0, 7, rank - 1] = float("inf")
    Y = sp.lora_add(d["X"], A, B, d["plan"], base=d["base"])
    assert torch.equal(Y[:, 7].float(), h[:, rank - 1] * float("inf")) and Y[:, 8:].isfinite().all()
    A[0, 0, 5] = float("inf")
    dX, _, _ = sp.lora_grad(d["dY"], d["X"], A, d["B"], d["plan"], dX_base=d["dX_base"], need=(True, False, False))
    assert torch.equal(dX[:, 5].double(), (d["dY"].double() @ d["B"][0, :, 0].double()) * float("inf"))
    assert dX[:, 6:].isfinite().all()


# What the parts of P hold of it where it meets the second operand (three of 8 bits, two of 11).
BITS = {"bf16": 2.0 ** -24, "f16": 2.0 ** -22}
LOW = {"bf16": 128, "f16": 64}  # integers from here to twice it: P is one of 23 bits (bf16), of 21 (fp16)


def integers(fmt, rng, rows, cols, pairs_along_rows=True):
    """Integers; row (or column) 2 i + 1 is row 2 i with one entry changed by one."""
    x = rng.integers(LOW[fmt], 2 * LOW[fmt], (rows, cols))
    if not pairs_along_rows:
        return integers(fmt, rng, cols, rows).T
    x[1::2] = x[0:rows // 2 * 2:2]
    at = rng.integers(0, cols, rows // 2)
    x[2 * np.arange(rows // 2) + 1, at] += np.where(x[2 * np.arange(rows // 2) + 1, at] > LOW[fmt], -1, 1)
    return x


def differences(rows, cols):
    """[rows, cols] with 1 and -1 at the pair 2 i, 2 i + 1 of columns of row r, i = r mod cols / 2."""
    d = np.zeros((rows, cols))
    i = np.arange(rows) % (cols // 2)
    d[np.arange(rows), 2 * i], d[np.arange(rows), 2 * i + 1] = 1, -1
    return d


@pytest.mark.parametrize("fmt", list(BITS))
@pytest.mark.parametrize("tokens,rank", [(6, 4), (700, 16), (700, 32), (700, 40), (400, 64), (400, 100), (300, 128)])
def test_small_differences_of_large_values_of_p(fmt, tokens, rank):
    """Every sum is of integers below 2^24, so P is exact, and the differences of neighbours that the second
    products take show each bit that P lost on its way there."""
    rng = np.random.default_rng([31, tokens, rank])
    k, n, scale = 128, 136, 2.0 ** -7
    plan = sp.lora_plan(None, 1, tokens=tokens, device=DEV)

    def dev(x):
        t = torch.from_numpy(np.ascontiguousarray(x)).to(DTYPES[fmt]).to(DEV)
        assert np.array_equal(as_f64(t), x)
        return t

    def near(got, want, P, what):
        err = 2 * BITS[fmt] * scale * np.abs(P).max()
        assert_within(got, scale * want, err, fmt, what)

    X, A, D = integers(fmt, rng, tokens, k), integers(fmt, rng, rank, k), differences(n, rank)
    Y = sp.lora_add(dev(X), dev(A)[None], dev(D)[None], plan, scale=scale)
    near(Y, (X @ A.T) @ D.T, X @ A.T, "Y")
    Z = differences(n, tokens).T  # [tokens, n]: pairs of tokens
    dB = sp.lora_grad(dev(Z), dev(X), dev(A)[None], dev(D)[None], plan, scale=scale, need=(False, False, True))[2]
    near(dB[0], Z.T @ (X @ A.T), X @ A.T, "dB")
    dY, B, D = integers(fmt, rng, tokens, n), integers(fmt, rng, n, rank, False), differences(k, rank).T
    dX = sp.lora_grad(dev(dY), dev(X), dev(D)[None], dev(B)[None], plan, scale=scale, need=(True, False, False))[0]
    near(dX, (dY @ B) @ D, dY @ B, "dX")
    Z = differences(k, tokens).T
    dA = sp.lora_grad(dev(dY), dev(Z), dev(D)[None], dev(B)[None], plan, scale=scale, need=(False, True, False))[1]
    near(dA[0], (dY @ B).T @ Z, dY @ B, "dA")
