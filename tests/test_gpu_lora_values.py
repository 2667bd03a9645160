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
