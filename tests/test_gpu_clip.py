"""Global gradient norm and clipping (GradSet, grad_norm, clip_grads) against 64-bit sums.

Bounds, fixed before any run: the squares of a group of at most 32 elements, at most 4 groups and
4 single elements, and 32 lanes, are added in fp32 (2^-24 relative per step, at most 45 steps, all
terms positive), the rest in fp64, then a square root (halves the relative error) and one rounding
to fp32: the norm is within 2^-19 of itself. A clipped element is the product of g with c, which
is within 2^-18 of the exact factor, rounded once to the element's type."""
import numpy as np
import pytest
import torch

from helpers import as_f64, ulp

pytestmark = pytest.mark.gpu

sp = pytest.importorskip("unstructured_sparse_linear_gb300")

DEV = torch.device("cuda:0")
FMT = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def grads_of(sizes, dtypes, std=1.0, seed=0):
    rng = np.random.default_rng([seed, len(sizes)])
    return [torch.from_numpy(rng.standard_normal(s) * std).to(dtypes[i % len(dtypes)]).to(DEV)
            for i, s in enumerate(sizes)]


def norm64(grads):
    return float(np.sqrt(sum((as_f64(g) ** 2).sum() for g in grads)))


def check_clipped(before, after, norm, max_norm):
    c = min(1.0, max_norm / (norm + 1e-6))
    for i, (b, a) in enumerate(zip(before, after)):
        want = as_f64(b) * c
        err = 2.0 ** -18 * np.abs(want)
        bound = err + 0.5 * ulp(np.abs(want) + err, FMT[a.dtype])
        assert (np.abs(as_f64(a) - want) <= bound).all(), i


SETS = {
    "one_element": ([1], [F32]),
    "odd": ([1, 2, 3, 7, 8, 9, 15, 17, 31, 33, 8191, 8192, 8193, 16385, 0, 5], [F32, F16, BF16]),
    "empty_ones": ([0, 0, 100, 0, 0, 9000, 0], [BF16]),
    "all_empty": ([0, 0], [F32]),
    "none": ([], [F32]),
    "many": ([(i * 37) % 211 for i in range(1500)], [BF16, F32]),
    "large": ([3_000_001, 77, 5_000_000], [BF16, F16, F32]),
    "factors": ([(16, 512), (300, 16), (2, 3, 5)], [F16]),
}


@pytest.mark.parametrize("name", list(SETS))
@pytest.mark.parametrize("max_norm", [0.5, 1e9, 0.0])
def test_norm_and_clip(name, max_norm):
    grads = grads_of(*SETS[name])
    before = [g.clone() for g in grads]
    want = norm64(grads)
    n1 = sp.grad_norm(grads)
    n2 = sp.clip_grads(grads, max_norm)
    assert n1.shape == () and n1.dtype == F32
    assert torch.equal(n1, n2) and abs(float(n1) - want) <= 2.0 ** -19 * want
    check_clipped(before, grads, want, max_norm)
    if max_norm == 1e9:  # nothing to do: the same bits
        assert all(torch.equal(a, b) for a, b in zip(before, grads))


@pytest.mark.parametrize("shift_in,shift_out", [(0, 0), (1, 1), (1, 0), (0, 3), (5, 5)])
def test_set_with_outputs_at_any_alignment(shift_in, shift_out):
    """Views of one flat buffer, the gradients' and the outputs' offsets alike or not."""
    sizes = [1000, 13, 8192, 20001, 1, 9999]
    for dt in (F32, BF16):
        flat = grads_of([sum(sizes) + 8], [dt])[0]
        out = torch.full_like(flat, 7.0)
        grads = list(flat[shift_in:shift_in + sum(sizes)].split(sizes))
        outs = list(out[shift_out:shift_out + sum(sizes)].split(sizes))
        before = flat.clone()
        s = sp.GradSet(grads, out=outs)
        want = norm64(grads)
        for _ in range(2):  # the set serves every step
            norm = sp.clip_grads(s, 1.0)
            assert abs(float(norm) - want) <= 2.0 ** -19 * want
            check_clipped(grads, outs, want, 1.0)
        assert torch.equal(flat, before)
        assert (out[:shift_out] == 7).all() and (out[shift_out + sum(sizes):] == 7).all()
        sp.clip_grads(s, 1e9)  # c = 1: the outputs still get the gradients
        assert torch.equal(out[shift_out:shift_out + sum(sizes)], flat[shift_in:shift_in + sum(sizes)])


@pytest.mark.parametrize("value,dtype", [(1e25, F32), (3e38, F32), (1e-25, F32), (1e-38, F32), (2e38, BF16),
                                         (1e-38, BF16), (6e4, F16), (6e-8, F16)])
def test_norm_of_the_largest_and_the_smallest_numbers(value, dtype):
    for n in (1, 64, 100_000):
        g = torch.full((n,), value, dtype=dtype, device=DEV)
        g[n // 2] = 0
        want = norm64([g])
        got = float(sp.grad_norm([g]))
        if want > float(np.finfo(np.float32).max):
            assert got == float("inf")
        else:
            assert abs(got - want) <= 2.0 ** -19 * want + 2.0 ** -149


def test_infinities_and_nan_follow_the_formula():
    g = [torch.ones(100, device=DEV), torch.ones(50, device=DEV)]
    g[1][7] = float("inf")
    assert float(sp.clip_grads(g, 1.0)) == float("inf")
    assert not g[0].any() and g[1][7].isnan() and not g[1][:7].any()
    g = [torch.ones(100, device=DEV, dtype=BF16), torch.ones(50, device=DEV)]
    g[0][3] = float("nan")
    assert sp.clip_grads(g, 1.0).isnan()
    assert g[0].isnan().all() and g[1].isnan().all()
    g = [torch.full((9,), 2.0, device=DEV)]
    assert float(sp.clip_grads(g, float("inf"))) == 6.0 and (g[0] == 2).all()


def test_same_bits_every_time_and_in_a_graph():
    grads = grads_of([100_000, 3333, 70_001], [BF16, F32])
    outs = [torch.empty_like(g) for g in grads]
    s = sp.GradSet(grads, out=outs)
    norm = sp.clip_grads(s, 1.0)
    first = [o.clone() for o in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        norm2 = sp.clip_grads(s, 1.0)
    for o in outs:
        o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, norm2) and all(torch.equal(a, b) for a, b in zip(first, outs))


def test_set_made_on_a_busy_stream_and_used_on_another():
    grads = grads_of([70_000, 33], [BF16])
    outs = [torch.empty_like(g) for g in grads]
    want = sp.grad_norm(grads)
    torch.cuda.synchronize()
    maker, user = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(maker):
        torch.cuda._sleep(20_000_000)  # the table is written some 10 ms from now
        s = sp.GradSet(grads, out=outs)
    with torch.cuda.stream(user):
        norm = sp.clip_grads(s, 1.0)
    user.synchronize()
    assert torch.equal(norm, want)
    check_clipped(grads, outs, float(want), 1.0)


def test_refusals():
    a, b = torch.ones(10, device=DEV), torch.ones(10, device=DEV, dtype=F16)
    with pytest.raises(ValueError, match="contiguous"):
        sp.GradSet([torch.ones(4, 6, device=DEV)[:, ::2]])
    with pytest.raises(ValueError, match="CUDA"):
        sp.GradSet([torch.ones(4)])
    with pytest.raises(ValueError, match="dtype"):
        sp.GradSet([torch.ones(4, device=DEV, dtype=torch.float64)])
    with pytest.raises(ValueError, match="dtype"):
        sp.GradSet([a], out=[b])
    with pytest.raises(ValueError, match="elements"):
        sp.GradSet([a], out=[torch.ones(9, device=DEV)])
    with pytest.raises(ValueError, match="outputs"):
        sp.GradSet([a, b], out=[a])
    with pytest.raises(ValueError, match="overlap"):
        sp.GradSet([a, a])
    with pytest.raises(ValueError, match="overlap"):
        sp.GradSet([a[:6], a[5:]])
    with pytest.raises(ValueError, match="overlap"):
        sp.GradSet([a[:5]], out=[a[2:7]])
    with pytest.raises(ValueError, match="max_norm"):
        sp.clip_grads([a], -1.0)
    with pytest.raises(ValueError, match="max_norm"):
        sp.clip_grads([a], float("nan"))
    assert torch.equal(a, torch.ones_like(a))
