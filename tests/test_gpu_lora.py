"""Low-rank adapters (lora_plan, lora_add, lora_grad) against their formulas in 64 bits.

Bounds, element by element, fixed before any run. With u = 2^-23 (one fp32 ulp per added term,
any order): P = U W1 over K terms is off by at most eP = u K |U||W1| plus 2^-17 |U||W1| for the
two 16-bit parts that the tensor cores multiply (8 + 8 bits of a bf16 pair at least, rounded).
O = base + s P W2 over r terms is then off by |s| eP |W2| + u (r + 4) (|base| + |s| |P| |W2|), and half
an ulp of the output's type. The weight gradients sum P[t, j] U[t, x] over the adapter's tokens."""
import numpy as np
import pytest
import torch

from helpers import ACC_UNIT, as_f64, ulp

pytestmark = pytest.mark.gpu

sp = pytest.importorskip("unstructured_sparse_linear_gb300")

DEV = torch.device("cuda:0")
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SPLIT = 2.0 ** -17


def make_ids(kind, T, n, rng):
    if kind == "one":
        return np.zeros(T, dtype=np.int32)
    if kind == "none":
        return np.full(T, -1, dtype=np.int32)
    if kind == "decode":
        return rng.integers(-1, n, T).astype(np.int32)
    ids = []
    while len(ids) < T:  # requests one behind the other
        ids += [int(rng.integers(-1, n))] * int(rng.integers(1, max(2, T // 3 + 1)))
    return np.asarray(ids[:T], dtype=np.int32)


def make(fmt, T, k, n_out, r, n, kind, seed=0, strided=False):
    rng = np.random.default_rng([seed, T, k, n_out, r, n])
    dt = DTYPES[fmt]

    def rand(*shape, std=1.0, pad=0):
        x = torch.from_numpy(rng.standard_normal(shape) * std).to(dt)
        if not pad:
            return x.to(DEV)
        wide = torch.full((shape[0], shape[1] + 2 * pad), float("nan"), dtype=dt, device=DEV)
        wide[:, pad:pad + shape[1]] = x.to(DEV)
        return wide[:, pad:pad + shape[1]]

    pad = 24 if strided else 0
    return dict(ids=make_ids(kind, T, n, rng), X=rand(T, k, pad=pad), A=rand(n, r, k, std=k ** -0.5),
                B=rand(n, n_out, r, std=0.3), base=rand(T, n_out, pad=pad), dY=rand(T, n_out, pad=pad),
                dX_base=rand(T, k, pad=pad), scale=torch.from_numpy(rng.uniform(0.5, 2, n)).float().to(DEV), n=n)


def plan_of(d):
    return sp.lora_plan(torch.from_numpy(d["ids"]).to(DEV), d["n"])


def want_rows(ids, U, W1, W2, s, base):
    """(O, bound, P, eP): the product of each token's adapter. W1 [n, K, r], W2 [n, r, N]."""
    T, K, r = U.shape[0], U.shape[1], W1.shape[2]
    O, eO = base.copy(), np.zeros_like(base)
    P, eP = np.zeros((T, r)), np.zeros((T, r))
    for a in np.unique(ids[(ids >= 0) & (ids < W1.shape[0])]):
        at = ids == a
        p, pa = U[at] @ W1[a], np.abs(U[at]) @ np.abs(W1[a])
        e = (ACC_UNIT * K + SPLIT) * pa
        P[at], eP[at] = p, e
        lr = s[a] * (p @ W2[a])
        O[at] += lr
        w2 = np.abs(W2[a])
        eO[at] = abs(s[a]) * (e @ w2) + ACC_UNIT * (r + 4) * (np.abs(base[at]) + abs(s[a]) * (np.abs(p) @ w2))
    return O, eO, P, eP


def want_wgrad(ids, n, U, P, eP, s):
    """(G, bound) [n, r, N] = s_a sum over the adapter's tokens of P[t]^T U[t]."""
    G, eG = np.zeros((n, P.shape[1], U.shape[1])), np.zeros((n, P.shape[1], U.shape[1]))
    for a in np.unique(ids[(ids >= 0) & (ids < n)]):
        at = ids == a
        G[a] = s[a] * (P[at].T @ U[at])
        eG[a] = abs(s[a]) * ((eP[at] + (ACC_UNIT * (at.sum() + 4) + SPLIT) * np.abs(P[at])).T @ np.abs(U[at]))
    return G, eG


def check(got, want, err, fmt, what):
    g = as_f64(got)
    assert g.shape == want.shape, (what, g.shape, want.shape)
    if fmt == "f16":  # values beyond the type round to the infinity of their sign
        over = np.abs(want) - err >= 65520.0
        assert np.array_equal(g[over], np.copysign(np.inf, want[over])), f"{what}: overflow"
        over |= (np.abs(want) + err >= 65520.0) & (g == np.copysign(np.inf, want))  # within err of the limit
        g, want, err = g[~over], want[~over], err[~over]
    assert np.all(np.isfinite(g)), f"{what}: non-finite output"
    bound = err + 0.5 * ulp(np.abs(want) + err, fmt)
    diff = np.abs(g - want)
    bad = diff > bound
    if bad.any():
        i = np.unravel_index(int(np.argmax(diff - bound)), diff.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {diff.size} outside the bound; worst at "
                             f"{tuple(int(x) for x in i)}: got {g[i]!r} want {want[i]!r} bound {bound[i]:.3e}")


def check_add(d, fmt, in_place=False, with_base=True):
    s = as_f64(d["scale"])
    base = as_f64(d["base"]) if with_base else np.zeros((len(d["ids"]), d["B"].shape[1]))
    O, eO, P, eP = want_rows(d["ids"], as_f64(d["X"]), as_f64(d["A"]).transpose(0, 2, 1),
                             as_f64(d["B"]).transpose(0, 2, 1), s, base)
    b = d["base"] if with_base else None
    Y, h = sp.lora_add(d["X"], d["A"], d["B"], plan_of(d), base=b, scale=d["scale"], out=b if in_place else None,
                       return_h=True)
    torch.cuda.synchronize()
    check(Y, O, eO, fmt, "Y")
    check(h, P, eP, "f32", "h")
    return h


def check_grad(d, fmt, h=None, in_place=False, need=(True, True, True)):
    s, ids = as_f64(d["scale"]), d["ids"]
    X, dY, A, B = (as_f64(d[x]) for x in ("X", "dY", "A", "B"))
    dX, eX, dP, eP = want_rows(ids, dY, B, A, s, as_f64(d["dX_base"]))
    _, _, H, eH = want_rows(ids, X, A.transpose(0, 2, 1), np.zeros((d["n"], A.shape[1], 1)), s, np.zeros((len(ids), 1)))
    dA, eA = want_wgrad(ids, d["n"], X, dP, eP, s)
    dBt, eBt = want_wgrad(ids, d["n"], dY, H, eH, s)
    got = sp.lora_grad(d["dY"], d["X"], d["A"], d["B"], plan_of(d), scale=d["scale"], h=h, dX_base=d["dX_base"],
                       dX_out=d["dX_base"] if in_place else None, need=need)
    torch.cuda.synchronize()
    assert [x is not None for x in got] == list(need)
    if need[0]:
        check(got[0], dX, eX, fmt, "dX")
    if need[1]:
        check(got[1], dA, eA, fmt, "dA")
    if need[2]:
        check(got[2], dBt.transpose(0, 2, 1), eBt.transpose(0, 2, 1), fmt, "dB")


# (tokens, in, out, rank, adapters, batch)
SHAPES = [
    (1, 256, 512, 16, 4, "decode"), (1, 8, 8, 1, 1, "one"), (2, 64, 200, 8, 1, "one"), (7, 384, 136, 4, 3, "decode"),
    (9, 72, 40, 5, 2, "prompts"), (64, 512, 1000, 16, 48, "decode"), (127, 64, 64, 32, 1, "one"),
    (128, 128, 192, 16, 1, "one"), (129, 200, 72, 64, 2, "prompts"), (300, 136, 328, 33, 5, "prompts"),
    (257, 512, 256, 128, 3, "decode"), (515, 384, 1536, 8, 300, "decode"), (1000, 264, 520, 24, 4, "prompts"),
    (200, 64, 64, 2, 2, "none"), (1500, 1024, 768, 16, 1, "one"), (700, 96, 96, 100, 2, "prompts"),
    (260, 37, 51, 6, 3, "prompts"), (33, 1, 3, 1, 2, "decode"), (400, 45, 64, 8, 2, "prompts"),
    (1, 256, 136, 64, 1, "one"), (3, 64, 72, 128, 2, "decode"), (17, 128, 64, 40, 1, "one"),
    (3000, 72, 136, 12, 2, "prompts"), (1200, 64, 200, 18, 3, "decode"), (900, 200, 64, 36, 2, "prompts"),
]


@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_add_and_grad(shape, fmt):
    d = make(fmt, *shape)
    h = check_add(d, fmt)
    check_grad(d, fmt, h=h)


# more tiles than the GPU holds at once: clusters of one CTA, of four and of eight, and the general kernel
@pytest.mark.parametrize("fmt,shape", [("bf16", (45000, 64, 72, 16, 3, "prompts")), ("f16", (45000, 72, 64, 4, 1, "one")),
                                       ("f16", (12500, 136, 64, 64, 2, "prompts")), ("bf16", (5200, 64, 136, 128, 2, "prompts")),
                                       ("f32", (12500, 24, 40, 4, 2, "prompts"))], ids=str)
def test_several_tiles_per_cluster(fmt, shape):
    d = make(fmt, *shape)
    h = check_add(d, fmt)
    check_grad(d, fmt, h=h)


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("shape", [(1500, 264, 328, 16, 1, "one"), (1300, 136, 264, 24, 3, "prompts"),
                                   (800, 264, 136, 64, 2, "prompts")], ids=lambda s: "-".join(map(str, s)))
def test_parts_alone_on_the_tensor_cores(shape, fmt):
    """P without O (h formed inside, the weights' gradients without dX), O without base, rows in place."""
    d = make(fmt, *shape, strided=True)
    check_add(d, fmt, with_base=False)
    check_grad(d, fmt, h=None)
    for need in ((True, False, False), (False, True, False), (False, False, True), (False, True, True)):
        check_grad(d, fmt, need=need)
    h = check_add(dict(d, base=d["base"].clone()), fmt)
    check_grad(d, fmt, h=h, in_place=True)


def test_one_row_with_any_stride():
    d = make("bf16", 1, 256, 136, 64, 1, "one")
    X, dY = (d[x].t().contiguous().t() for x in ("X", "dY"))
    X, dY = X.as_strided((1, 256), (3, 1)), dY.as_strided((1, 136), (0, 1))
    assert torch.equal(sp.lora_add(X, d["A"], d["B"], plan_of(d)), sp.lora_add(d["X"], d["A"], d["B"], plan_of(d)))
    got = sp.lora_grad(dY, X, d["A"], d["B"], plan_of(d))
    for x, y in zip(got, sp.lora_grad(d["dY"], d["X"], d["A"], d["B"], plan_of(d))):
        assert torch.equal(x, y)


@pytest.mark.parametrize("fmt", list(DTYPES))
@pytest.mark.parametrize("shape", [(5, 256, 136, 16, 2, "decode"), (333, 264, 400, 16, 3, "prompts"),
                                   (256, 128, 128, 8, 1, "one")], ids=lambda s: "-".join(map(str, s)))
def test_strided_rows_in_place_no_base_and_h_formed_inside(shape, fmt):
    d = make(fmt, *shape, strided=True)
    check_add(d, fmt, with_base=False)
    check_grad(d, fmt, h=None)
    for need in ((True, False, False), (False, True, False), (False, False, True)):
        check_grad(d, fmt, need=need)
    sides = {x: d[x]._base.clone() for x in ("base", "dX_base")}
    ref = dict(d, base=d["base"].clone(), dX_base=d["dX_base"].clone())
    Y, _ = sp.lora_add(ref["X"], d["A"], d["B"], plan_of(d), base=ref["base"], scale=d["scale"], return_h=True)
    sp.lora_add(d["X"], d["A"], d["B"], plan_of(d), base=d["base"], scale=d["scale"], out=d["base"])
    dX = sp.lora_grad(d["dY"], d["X"], d["A"], d["B"], plan_of(d), scale=d["scale"], dX_base=ref["dX_base"])[0]
    sp.lora_grad(d["dY"], d["X"], d["A"], d["B"], plan_of(d), scale=d["scale"], dX_base=d["dX_base"],
                 dX_out=d["dX_base"])
    torch.cuda.synchronize()
    assert torch.equal(d["base"], Y) and torch.equal(d["dX_base"], dX)
    for x, before in sides.items():  # the columns beside the slice are untouched
        after, w = d[x]._base, d[x].shape[1]
        assert torch.equal(after[:, :24].isnan(), before[:, :24].isnan())
        assert torch.equal(after[:, 24 + w:].isnan(), before[:, 24 + w:].isnan())


def test_odd_alignment():
    """Operands that start at an element that no 16-byte access may."""
    d = make("bf16", 300, 264, 136, 16, 2, "prompts")
    want = sp.lora_add(d["X"], d["A"], d["B"], plan_of(d), base=d["base"], scale=d["scale"])

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        flat[1:] = t.reshape(-1)
        return flat[1:].view(t.shape)

    s = dict(d, **{x: shifted(d[x]) for x in ("X", "A", "B", "base", "dY", "dX_base")})
    check_add(s, "bf16")
    check_grad(s, "bf16")
    got = sp.lora_add(s["X"], s["A"], s["B"], plan_of(d), base=s["base"], scale=d["scale"])
    torch.cuda.synchronize()
    assert (got.float() - want.float()).abs().max() <= 2 ** -6 * want.float().abs().max()


@pytest.mark.parametrize("T,n,kind", [(1, 1, "one"), (31, 3, "decode"), (1000, 7, "prompts"), (5000, 255, "decode"),
                                      (5000, 256, "decode"), (40000, 70000, "decode"), (1025, 2, "none")])
def test_plan_order_is_the_stable_sort(T, n, kind):
    rng = np.random.default_rng(T + n)
    ids = make_ids(kind, T, n, rng)
    ids[rng.integers(0, T, max(1, T // 50))] = n  # out of range: no adapter
    if kind == "one":
        ids[:] = 0
    plan = sp.lora_plan(torch.from_numpy(ids).to(DEV), n)
    key = np.where((ids >= 0) & (ids < n), ids, n)
    assert np.array_equal(plan.order().cpu().numpy(), np.argsort(key, kind="stable"))


@pytest.mark.parametrize("fmt", ["f32", "bf16"])
@pytest.mark.parametrize("T", [40, 700, 2500])
def test_one_tokens_infinities_and_one_adapters_nan_stay_there(T, fmt):
    d = make(fmt, T, 264, 520, 16, 3, "prompts", seed=3)
    d["ids"][:] = np.arange(T) % 3  # every tile of an adapter lies between the others' tokens
    d["ids"][-3:] = -1
    clean = sp.lora_add(d["X"], d["A"], d["B"], plan_of(d), base=d["base"], scale=d["scale"])
    clean_g = sp.lora_grad(d["dY"], d["X"], d["A"], d["B"], plan_of(d), scale=d["scale"], dX_base=d["dX_base"])
    hit = 4  # a token of adapter 1
    A, B, X, dY = d["A"].clone(), d["B"].clone(), d["X"].clone(), d["dY"].clone()
    A[2], B[2] = float("nan"), float("nan")
    X[hit], dY[hit] = float("inf"), float("inf")
    X[-3:], dY[-3:] = float("nan"), float("nan")  # tokens without an adapter: never read into a product
    Y = sp.lora_add(X, A, B, plan_of(d), base=d["base"], scale=d["scale"])
    dX, dA, dB = sp.lora_grad(dY, X, A, B, plan_of(d), scale=d["scale"], dX_base=d["dX_base"])
    torch.cuda.synchronize()
    ids = torch.from_numpy(d["ids"]).to(DEV)
    keep = ids != 2
    keep[hit] = False
    assert torch.equal(Y[keep], clean[keep]) and torch.equal(dX[keep], clean_g[0][keep])
    assert Y[ids == 2].isnan().all() and not Y[hit].isfinite().any()
    assert torch.equal(dA[0], clean_g[1][0]) and torch.equal(dB[0], clean_g[2][0])
    assert not dA[1].isfinite().any() and not dB[1].isfinite().any()


@pytest.mark.parametrize("scale", [1e-7, 1e-3, 1e4])
def test_fp16_keeps_small_and_large_intermediate_values(scale):
    """X A^T far below the smallest and above the largest fp16 number: it stays in fp32."""
    for T in (5, 300, 2500):
        d = make("f16", T, 256, 256, 16, 1, "one", seed=5)
        d["X"] = (d["X"].float() * (scale if scale < 1 else 300.0)).half()
        d["A"] = (d["A"].float() * (1 if scale < 1 else 3000.0)).half()
        d["B"] = (d["B"].float() * (1 if scale < 1 else 1e-4)).half()
        d["scale"][:] = 1.0 / scale if scale < 1 else 1.0
        d["dY"] = (d["dY"].float() * min(scale, 1.0)).half()
        h = check_add(d, "f16")
        check_grad(d, "f16", h=h)


@pytest.mark.parametrize("x,a,dy", [(1e-6, 1, 1e3), (1e4, 8, 1e-4)])
def test_fp16_columns_of_db_beside_an_infinite_one(x, a, dy):
    d = make("f16", 700, 136, 72, 16, 1, "one", seed=17)
    d["X"], d["A"], d["dY"] = d["X"] * x, d["A"] * a, d["dY"] * dy
    A = as_f64(d["A"]).copy()
    d["A"][0, 3, 5] = float("inf")
    _, _, P, eP = want_rows(d["ids"], as_f64(d["X"]), A.transpose(0, 2, 1), as_f64(d["B"]).transpose(0, 2, 1),
                            as_f64(d["scale"]), np.zeros((700, 72)))
    G, eG = want_wgrad(d["ids"], 1, as_f64(d["dY"]), P, eP, as_f64(d["scale"]))
    dB = sp.lora_grad(d["dY"], d["X"], d["A"], d["B"], plan_of(d), scale=d["scale"], need=(False, False, True))[2]
    rest = [j for j in range(16) if j != 3]
    check(dB[:, :, rest], G.transpose(0, 2, 1)[:, :, rest], eG.transpose(0, 2, 1)[:, :, rest], "f16", "dB")
    assert not np.any(np.isfinite(as_f64(dB[:, :, 3])))


@pytest.mark.parametrize("fmt", ["f32", "f16"])
def test_row_offsets_beyond_32_bits(fmt):
    """Rows so far apart that the last ones lie past 2^31 elements."""
    T, k, n_out = 150, 72, 64
    ld = 2 ** 31 // 140 // 8 * 8
    d = make(fmt, T, k, n_out, 8, 2, "prompts")
    wide = torch.empty(T * ld, dtype=DTYPES[fmt], device=DEV)
    for name, cols in (("X", k), ("base", n_out), ("dY", n_out), ("dX_base", k)):
        at = {"X": 0, "base": 1000, "dY": 2000, "dX_base": 3000}[name]
        v = wide[at:].as_strided((T, cols), (ld, 1))
        v.copy_(d[name])
        d[name] = v
    h = check_add(d, fmt)
    check_grad(d, fmt, h=h)


def test_empty_batch():
    A, B = torch.randn(2, 4, 16, device=DEV), torch.randn(2, 24, 4, device=DEV)
    plan = sp.lora_plan(torch.empty(0, dtype=torch.int32, device=DEV), 2)
    X, dY = torch.empty(0, 16, device=DEV), torch.empty(0, 24, device=DEV)
    assert sp.lora_add(X, A, B, plan).shape == (0, 24)
    dX, dA, dB = sp.lora_grad(dY, X, A, B, plan)
    assert dX.shape == (0, 16) and not dA.any() and not dB.any()


def test_scalar_scale_and_plan_without_ids():
    d = make("bf16", 300, 128, 256, 16, 1, "one")
    p1, p2 = plan_of(d), sp.lora_plan(None, 1, tokens=300, device=DEV)
    assert torch.equal(p1.order(), p2.order())
    d["scale"][:] = 0.75
    a = sp.lora_add(d["X"], d["A"], d["B"], p1, base=d["base"], scale=d["scale"])
    b = sp.lora_add(d["X"], d["A"], d["B"], p2, base=d["base"], scale=0.75)
    assert torch.equal(a, b)


@pytest.mark.parametrize("T", [3, 600, 2500])
def test_same_bits_every_time_on_a_side_stream_and_in_a_graph(T):
    d = make("bf16", T, 512, 768, 16, 4, "prompts", seed=9)
    plan = plan_of(d)

    def step():
        Y = sp.lora_add(d["X"], d["A"], d["B"], plan, base=d["base"], scale=d["scale"])
        return (Y, *sp.lora_grad(d["dY"], d["X"], d["A"], d["B"], plan, scale=d["scale"], dX_base=d["dX_base"]))

    first = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step()
    g.replay()
    torch.cuda.synchronize()
    for x, y, z in zip(first, again, captured):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_plan_made_on_a_busy_stream_and_used_on_another():
    d = make("bf16", 700, 128, 256, 16, 4, "prompts", seed=13)
    want = sp.lora_add(d["X"], d["A"], d["B"], plan_of(d), base=d["base"], scale=d["scale"])
    ids = torch.from_numpy(d["ids"]).to(DEV)
    torch.cuda.synchronize()
    maker, user = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(maker):
        torch.cuda._sleep(20_000_000)  # the plan is written some 10 ms from now
        plan = sp.lora_plan(ids, d["n"])
    with torch.cuda.stream(user):
        got = sp.lora_add(d["X"], d["A"], d["B"], plan, base=d["base"], scale=d["scale"])
    user.synchronize()
    assert torch.equal(got, want)


def test_one_plan_in_graphs_and_threads_at_the_same_time():
    """Calls that share a plan but not an order (graphs replayed on two streams, threads on one
    stream) do not share what lies between their two products."""
    import threading

    T = 700
    d = [make("bf16", T, 512, 1024, 16, 1, "one", seed=31 + i) for i in range(4)]
    p = plan_of(d[0])

    def call(x):
        return sp.lora_grad(x["dY"], x["X"], x["A"], x["B"], p, scale=x["scale"], dX_base=x["dX_base"])

    want = [call(x) for x in d]
    graphs, outs = [], []
    torch.cuda.synchronize()
    for x in d:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append([call(x) for _ in range(8)])
    streams = [torch.cuda.Stream() for _ in d]
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for ref, runs in zip(want, outs):
        for out in runs:
            assert all(torch.equal(a, b) for a, b in zip(out, ref))

    got = [[] for _ in d]

    def work(i):
        for _ in range(50):
            got[i].append(call(d[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(d))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for ref, runs in zip(want, got):
        assert len(runs) == 50
        for out in runs:
            assert all(torch.equal(a, b) for a, b in zip(out, ref))


@pytest.mark.parametrize("T", [5, 300, 1500])
def test_inputs_written_just_before_by_kernels_copies_and_other_streams(T):
    """Each launch may begin while the one before it ends: what that one writes is waited for,
    whether it is a kernel, a copy or a memset, here or on a stream that this one waits for."""
    d = make("bf16", T, 512, 384, 16, 3, "prompts", seed=23)
    p = plan_of(d)
    args = dict(scale=d["scale"])
    want = sp.lora_add(d["X"], d["A"], d["B"], p, base=d["base"], **args)
    want_g = sp.lora_grad(d["dY"], d["X"], d["A"], d["B"], p, dX_base=d["dX_base"], **args)
    zero = sp.lora_add(d["X"], d["A"], d["B"], p, **args)
    bufs = {k: torch.empty_like(d[k]) for k in ("X", "A", "B", "base", "dY", "dX_base")}
    big = torch.empty(1 << 27, device=DEV)
    other = torch.cuda.Stream()

    def step(wait):
        for b in bufs.values():
            b.fill_(float("nan"))
        if wait:
            fork = torch.cuda.current_stream().record_event()
            with torch.cuda.stream(other):
                other.wait_event(fork)
                big.fill_(1.0)
                for k in ("A", "dY"):
                    bufs[k].copy_(d[k])
                join = other.record_event()
        for k in bufs:
            if not (wait and k in ("A", "dY")):
                bufs[k].copy_(d[k])
        if wait:
            torch.add(bufs["X"], 0, out=bufs["X"])  # a kernel, still running at the wait
            torch.cuda.current_stream().wait_event(join)
        y = sp.lora_add(bufs["X"], bufs["A"], bufs["B"], p, base=bufs["base"], **args)
        bufs["base"].zero_()
        y2 = sp.lora_add(bufs["X"], bufs["A"], bufs["B"], p, base=bufs["base"], **args)
        g = sp.lora_grad(bufs["dY"], bufs["X"], bufs["A"], bufs["B"], p, dX_base=bufs["dX_base"], **args)
        bufs["dX_base"].copy_(d["dX_base"])
        return (y, y2) + g

    for wait in (False, True):
        outs = [step(wait) for _ in range(3)]
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            outs.append(step(wait))
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        for out in outs:
            for got, ref in zip(out, (want, zero) + want_g):
                assert torch.equal(got, ref)


def test_gradient_against_differences():
    """Y is linear in X, in A and in B apart, so a central difference of L = sum(Y * W) over a
    step of 1 along a direction equals the gradient's product with it, but for rounding: each Y is
    off by 2^-23 (K + r + 8) of its absolute sums at most (twice, halved), and the gradient likewise."""
    T, k, n_out, r, n = 50, 40, 56, 6, 3
    d = make("f32", T, k, n_out, r, n, "prompts", seed=21)
    plan = plan_of(d)
    W = d["dY"]

    def loss(X, A, B):
        return (as_f64(sp.lora_add(X, A, B, plan, scale=d["scale"])) * as_f64(W)).sum()

    grads = sp.lora_grad(W, d["X"], d["A"], d["B"], plan, scale=d["scale"])
    rng = np.random.default_rng(4)
    for i, name in enumerate(("X", "A", "B")):
        v = torch.from_numpy(rng.standard_normal(tuple(d[name].shape))).float().to(DEV)
        args = {x: d[x] for x in ("X", "A", "B")}
        hi = loss(**{**args, name: d[name] + v})
        lo = loss(**{**args, name: d[name] - v})
        want = (as_f64(grads[i]) * as_f64(v)).sum()
        big = {x: np.abs(as_f64(args[x])) for x in args}
        big[name] = big[name] + np.abs(as_f64(v))
        mass = 0.0
        for a in range(n):
            at = d["ids"] == a
            lr = big["X"][at] @ big["A"][a].T @ big["B"][a].T
            mass += as_f64(d["scale"])[a] * (np.abs(as_f64(W))[at] * lr).sum()
        assert abs((hi - lo) / 2 - want) <= 4 * ACC_UNIT * (k + r + T + n_out + 8) * mass, name


def test_refusals():
    d = make("bf16", 20, 64, 48, 8, 2, "decode")
    plan = plan_of(d)
    ok = (d["X"], d["A"], d["B"], plan)
    with pytest.raises(ValueError, match="rank"):
        sp.lora_add(d["X"], torch.zeros(2, 129, 64, dtype=torch.bfloat16, device=DEV),
                    torch.zeros(2, 48, 129, dtype=torch.bfloat16, device=DEV), plan)
    with pytest.raises(ValueError, match="dtype"):
        sp.lora_add(d["X"].float(), d["A"], d["B"], plan)
    with pytest.raises(ValueError, match="20 x 64"):
        sp.lora_add(d["X"][:10], d["A"], d["B"], plan)
    with pytest.raises(ValueError, match="contiguous rows"):
        sp.lora_add(d["X"].t().contiguous().t(), d["A"], d["B"], plan)
    with pytest.raises(ValueError, match="contiguous rows"):
        sp.lora_add(*ok, base=d["base"][:1].expand(20, 48), out=d["base"][:1].expand(20, 48))
    with pytest.raises(ValueError, match="adapters"):
        sp.lora_add(d["X"], d["A"][:1].contiguous(), d["B"][:1].contiguous(), plan)
    with pytest.raises(ValueError, match="scale"):
        sp.lora_add(*ok, scale=torch.ones(3, device=DEV))
    with pytest.raises(ValueError, match="finite"):
        sp.lora_add(*ok, scale=float("nan"))
    with pytest.raises(ValueError, match="overlap"):
        sp.lora_add(d["X"], d["A"], torch.zeros(2, 64, 8, dtype=torch.bfloat16, device=DEV), plan, out=d["X"])
    with pytest.raises(ValueError, match="overlap"):
        buf = torch.zeros(21, 48, dtype=torch.bfloat16, device=DEV)
        sp.lora_add(*ok, base=buf[:20], out=buf[1:])
    with pytest.raises(ValueError, match="CUDA"):
        sp.lora_add(d["X"].cpu(), d["A"], d["B"], plan)
    with pytest.raises(ValueError, match="h must be"):
        sp.lora_grad(d["dY"], *ok, h=torch.zeros(20, 9, device=DEV))
    with pytest.raises(ValueError, match="adapter_ids"):
        sp.lora_plan(torch.zeros(3, dtype=torch.int64, device=DEV), 2)
    with pytest.raises(ValueError, match="n_adapters"):
        sp.lora_plan(torch.zeros(3, dtype=torch.int32, device=DEV), 0)
    with pytest.raises(TypeError):
        sp.lora_add(d["X"], d["A"], d["B"], None)
    # columns of one wide buffer side by side are no overlap
    wide = torch.zeros(20, 64 + 48 + 48, dtype=torch.bfloat16, device=DEV)
    sp.lora_add(wide[:, :64], d["A"], d["B"], plan, base=wide[:, 64:112], out=wide[:, 112:])
