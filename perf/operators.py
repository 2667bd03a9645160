"""The measured cases of the low-rank adapter operators and of the global-norm clipping.

Three operators, the low-rank half of a RoSA adapter (a low-rank and a sparse update beside one
frozen projection) and the step that closes its training iteration:

  add   Y = base + s_i (X A_i^T) B_i^T, adapter i chosen per token (many requests at once)
  grad  dX = dX_base + s_i (dY B_i) A_i, dA_i = s_i (dY B_i)^T X, dB_i = s_i dY^T (X A_i^T)
  clip  the global 2-norm of many gradients, and every gradient times min(1, max_norm / (norm + 1e-6))

``own`` false: plain 32-bit torch operations. ``own`` true: this package's calls.
"""
import math
import random

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
CLIP_EPS = 1e-6


# ---------------------------------------------------------------- cases


def listed():
    return [
        # one generated token of one request: the smallest call of a serving loop (latency)
        dict(name="add_token_1", op="add", dtype="bf16", tokens=1, k=4096, n=4096, rank=16, adapters=8, batch="decode"),
        # a decode step of 64 requests, 48 adapters in hand, some requests without one, up-projection of an MLP
        dict(name="add_decode_64", op="add", dtype="bf16", tokens=64, k=4096, n=11008, rank=16, adapters=48,
             batch="decode"),
        # a scheduler's mixed batch: ragged prompts and single tokens of 24 adapters, output into a fused projection
        dict(name="add_mixed_1037", op="add", dtype="fp16", tokens=1037, k=4096, n=4096, rank=32, adapters=24,
             batch="prompts", fused=3),
        # long prompts, four adapters of a high rank, the butterfly layer's shape
        dict(name="add_prompt_8192", op="add", dtype="bf16", tokens=8192, k=2048, n=8192, rank=64, adapters=4,
             batch="prompts"),
        # full-precision check runs with an odd rank and an odd token count
        dict(name="add_fp32_501", op="add", dtype="fp32", tokens=501, k=384, n=1536, rank=5, adapters=3,
             batch="prompts"),
        # a short training sequence on the small MLP (launches count)
        dict(name="grad_small_512", op="grad", dtype="bf16", tokens=512, k=384, n=1536, rank=8, adapters=1, batch="one"),
        # the RoSA adapter's training step: one adapter, 4096 x 4096, 2048 tokens
        dict(name="grad_rosa_2048", op="grad", dtype="fp16", tokens=2048, k=4096, n=4096, rank=16, adapters=1,
             batch="one"),
        # several adapters trained at once on the LLaMA MLP shape, ragged sequences
        dict(name="grad_llama_4096", op="grad", dtype="bf16", tokens=4096, k=4096, n=11008, rank=16, adapters=6,
             batch="prompts"),
        # one layer's adapters: seven projections, two factors and the sparse values each
        dict(name="clip_layer_1", op="clip", dtype="bf16", layers=1, pack="flat"),
        # every adapter of a 32-layer model in one flat gradient buffer (672 gradients)
        dict(name="clip_layers_32", op="clip", dtype="bf16", layers=32, pack="flat"),
        # fp32 gradients kept as separate tensors
        dict(name="clip_fp32_2", op="clip", dtype="fp32", layers=2, pack="separate"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("add", "add", "grad", "clip"))
    if op == "clip":
        pack = rng.choice(("flat", "flat", "separate"))
        return dict(op="clip", dtype=rng.choice(("bf16", "fp16", "fp32") if pack == "separate" else ("bf16", "fp16")),
                    layers=rng.randint(1, 2) if pack == "separate" else _log_int(rng, 1, 31), pack=pack,
                    layout=rng.randint(1, 10 ** 6))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp16", "fp32"))
    kind = rng.choice(("decode", "prompts", "one")) if op == "add" else rng.choice(("prompts", "one"))
    tokens = _log_int(rng, 1, 128) if kind == "decode" else _log_int(rng, 130, 8000 if dtype != "fp32" else 1000)
    k, n = 8 * (_log_int(rng, 32, 511) | 1), 8 * (_log_int(rng, 32, 767) | 1)  # odd multiples of 16 bytes (16-bit types)
    if rng.random() < 0.12:  # rows that are no multiple of 16 bytes
        k, n, tokens = k - rng.randint(1, 7), n - rng.randint(1, 7), min(tokens, 600)
    # odd ranks as often as the usual ones
    rank = rng.choice((4, 8, 16, 32, 64, _log_int(rng, 1, 64), _log_int(rng, 1, 64)))
    return dict(op=op, dtype=dtype, tokens=tokens, k=k, n=n, rank=rank,
                adapters=1 if kind == "one" else rng.randint(2, 16), batch=kind)


# ---------------------------------------------------------------- inputs


def _ids(case, rng):
    """The adapter of every token (-1: none)."""
    t, n, kind = case["tokens"], case["adapters"], case["batch"]
    if kind == "one":
        return [0] * t
    if kind == "decode":  # one token per request, in the order the requests arrived
        return [rng.randrange(n) if t < 8 or rng.random() < 0.9 else -1 for _ in range(t)]
    ids = []
    while len(ids) < t:   # requests one behind the other: prompts of many lengths, and single tokens
        a = rng.randrange(n) if rng.random() < 0.95 else -1
        ids += [a] * (1 if rng.random() < 0.3 else max(1, int(rng.expovariate(1.0) * t / (2.0 * n))))
    return ids[:t]


def _clip_sizes(case):
    """Per layer: four 4096 x 4096 and three 11008 x 4096 projections, each with its two factors of rank
    16 and the values of its sparse mask (1 % and 0.5 %)."""
    attn, mlp = (4096 * 16, 4096 * 16, 167772), (4096 * 16, 11008 * 16, 225444)
    sizes = list(attn * 4 + mlp * 3) * case["layers"]
    if "layout" in case:  # drawn cases: other shapes, odd lengths
        rng = random.Random(case["layout"])
        sizes = [_log_int(rng, max(1, s // 64), s) for s in sizes]
    return sizes


def _inputs(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def randn(*shape, std=1.0):
        return torch.empty(shape, dtype=torch.float32, device=dev).normal_(0.0, std, generator=g)

    if case["op"] == "clip":
        sizes = _clip_sizes(case)
        total = sum(sizes)
        if case["pack"] == "flat":
            flat, flat_out = randn(total, std=3e-3).to(dt), torch.empty(total, dtype=dt, device=dev)
            grads, outs = list(flat.split(sizes)), list(flat_out.split(sizes))
        else:
            grads = [randn(s, std=3e-3).to(dt) for s in sizes]
            flat, flat_out, outs = None, None, [torch.empty_like(x) for x in grads]
        return dict(case=case, max_norm=1.0, grads=grads, outs=outs, flat=flat, flat_out=flat_out)

    t, k, n, r, na = (case[x] for x in ("tokens", "k", "n", "rank", "adapters"))
    ids = torch.tensor(_ids(case, random.Random(int(seed) * 7919 + 1)), dtype=torch.int32, device=dev)
    s = dict(case=case, ids=ids)
    s["X"] = randn(t, k).to(dt)
    s["A"] = randn(na, r, k, std=k ** -0.5).to(dt)
    s["B"] = randn(na, n, r, std=0.02).to(dt)
    s["scale"] = torch.rand(na, device=dev, generator=g) + 0.5
    if case["op"] == "add":
        fused = case.get("fused", 1)  # the projection's share of a fused output, one row stride for all
        s["base"] = randn(t, fused * n).to(dt)[:, (fused - 1) * n:]
        s["out"] = torch.empty((t, fused * n), dtype=dt, device=dev)[:, (fused - 1) * n:]
    else:
        s["dY"] = randn(t, n, std=1e-2).to(dt)
        s["dX_base"] = randn(t, k, std=1e-2).to(dt)
        # X A_i^T as the forward pass saved it
        s["h"] = _own_blocks(s["X"].float() @ _cat_a(s), s, scaled=False).sum(1)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # what the framework's user keeps: the handle of a set of gradients, the plan of a batch of tokens
        import unstructured_sparse_linear_gb300 as sp
        if case["op"] == "clip":
            s["set"] = sp.GradSet(s["grads"], out=s["outs"])
        else:
            s["plan"] = sp.lora_plan(s["ids"], case["adapters"])
    return s


# ---------------------------------------------------------------- plain forms


def _cat_a(s):
    """All adapters' A side by side: k x (adapters * rank)."""
    return s["A"].float().flatten(0, 1).t()


def _cat_b(s):
    """All adapters' B side by side, transposed: (adapters * rank) x n."""
    return s["B"].float().transpose(1, 2).flatten(0, 1)


def _own_blocks(p, s, scaled):
    """tokens x (adapters * rank) -> tokens x adapters x rank, zero outside each token's own adapter."""
    own_block = (s["ids"][:, None] == torch.arange(s["A"].shape[0], device=p.device)).float()
    if scaled:
        own_block = own_block * s["scale"]
    return p.view(p.shape[0], own_block.shape[1], -1) * own_block[:, :, None]


def _plain_add(s):
    p = _own_blocks(s["X"].float() @ _cat_a(s), s, scaled=True)
    return (s["base"].float() + p.flatten(1) @ _cat_b(s)).to(s["base"].dtype)


def _plain_grad(s):
    dt = s["X"].dtype
    dY, X = s["dY"].float(), s["X"].float()
    dp = _own_blocks(dY @ _cat_b(s).t(), s, scaled=True).flatten(1)
    dX = s["dX_base"].float() + dp @ _cat_a(s).t()
    dA = (dp.t() @ X).view(s["A"].shape)
    h = _own_blocks(s["h"].repeat(1, s["A"].shape[0]), s, scaled=True).flatten(1)
    dB = (dY.t() @ h).view(dY.shape[1], s["A"].shape[0], -1).transpose(0, 1)
    return {"dX": dX.to(dt), "dA": dA.to(dt), "dB": dB.to(dt).contiguous()}


def _plain_clip(s):
    parts = s["grads"] if s["flat"] is None else [s["flat"]]  # a flat buffer is one tensor to a plain program
    norm = torch.stack([g.float().square().sum() for g in parts]).sum().sqrt()
    c = torch.clamp(s["max_norm"] / (norm + CLIP_EPS), max=1.0)
    if s["flat"] is not None:
        return {"norm": norm, "grads": (s["flat"].float() * c).to(s["flat"].dtype)}
    return {"norm": norm, "grads": [(g.float() * c).to(g.dtype) for g in s["grads"]]}


# ---------------------------------------------------------------- one pass


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"add": _plain_add, "grad": _plain_grad, "clip": _plain_clip}[op](s)
    import unstructured_sparse_linear_gb300 as sp
    if op == "add":
        return sp.lora_add(s["X"], s["A"], s["B"], s["plan"], base=s["base"], scale=s["scale"], out=s["out"])
    if op == "grad":
        dX, dA, dB = sp.lora_grad(s["dY"], s["X"], s["A"], s["B"], s["plan"], scale=s["scale"], h=s["h"],
                                  dX_base=s["dX_base"])
        return {"dX": dX, "dA": dA, "dB": dB}
    norm = sp.clip_grads(s["set"], s["max_norm"])
    return {"norm": norm, "grads": s["flat_out"] if s["flat_out"] is not None else s["outs"]}


def work(case):
    b = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "clip":
        total = sum(_clip_sizes(case))
        # read for the norm and, with the factor known, read and written
        return {"bytes": 2 * total * b, "flops": 3 * total}
    t, k, n, r = (case[x] for x in ("tokens", "k", "n", "rank"))
    used = min(case["adapters"], t)
    weights = used * r * (k + n) * b
    if case["op"] == "add":
        return {"bytes": t * (k + 2 * n) * b + weights + 4 * t, "flops": 2 * t * r * (k + n)}
    return {"bytes": t * (n + 3 * k) * b + 2 * weights + 4 * t * (r + 1), "flops": 4 * t * r * (k + n)}


# ---------------------------------------------------------------- 64 bits


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "clip":
        grads = [x.double() for x in s["grads"]]
        norm = math.sqrt(math.fsum(float((x * x).sum()) for x in grads))
        c = min(1.0, s["max_norm"] / (norm + CLIP_EPS))
        scaled = [x * c for x in grads]
        norm = torch.tensor(norm, dtype=torch.float64)
        return {"norm": norm, "grads": torch.cat(scaled) if s["flat"] is not None else scaled}
    X, A, B, scale = s["X"].double(), s["A"].double(), s["B"].double(), s["scale"].double()
    ids = s["ids"].tolist()
    rows = {a: torch.tensor([i for i, x in enumerate(ids) if x == a], device=X.device) for a in set(ids) if a >= 0}
    if case["op"] == "add":
        Y = s["base"].double()
        for a, at in rows.items():
            Y[at] += scale[a] * ((X[at] @ A[a].t()) @ B[a].t())
        return Y
    dY, dX, dA, dB = s["dY"].double(), s["dX_base"].double(), torch.zeros_like(A), torch.zeros_like(B)
    h = s["h"].double()
    for a, at in rows.items():
        dp = scale[a] * (dY[at] @ B[a])
        dX[at] += dp @ A[a]
        dA[a] = dp.t() @ X[at]
        dB[a] = scale[a] * (dY[at].t() @ h[at])
    return {"dX": dX, "dA": dA, "dB": dB}
