"""The measured cases of the 4-bit frozen weight and of the dropout in front of a low-rank adapter.

Four operators, what a RoSA adapter needs to be trained and served beside a frozen projection that is kept in 4 bits:

  quant    blocks of 32 values of a row as microscaled 4-bit floating point (E2M1 codes, one E8M0 scale), and back
  linear   Y = X W^T for a 4-bit W [n, k]
  grad     dX = dY W for the same W
  dropout  Y = base + keep x / (1 - p), keep from a counter-based generator (Philox4x32-7, 16 bits a value)

``own`` false: plain 32-bit torch operations. ``own`` true: this package's calls.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
BLOCK = 32
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases


def listed():
    return [
        # full-precision values with an odd row length, the smallest weight to convert (launches count)
        dict(name="quant_fp32_384", op="quant", dtype="fp32", rows=384, cols=1537),
        # one MLP projection of a LLaMA-style model, converted when the model is loaded
        dict(name="quant_llama_11008", op="quant", dtype="bf16", rows=11008, cols=4096),
        # one generated token of one request (latency, then the weight's bytes)
        dict(name="linear_token_1", op="linear", dtype="bf16", tokens=1, k=4096, n=4096),
        # a decode step of 64 requests, up-projection of an MLP
        dict(name="linear_decode_64", op="linear", dtype="bf16", tokens=64, k=4096, n=11008),
        # a scheduler's mixed batch of prompts and single tokens, output into a fused projection
        dict(name="linear_mixed_1037", op="linear", dtype="fp16", tokens=1037, k=4096, n=4096, fused=3),
        # long prompts, the butterfly layer's shape
        dict(name="linear_prompt_8192", op="linear", dtype="bf16", tokens=8192, k=2048, n=8192),
        # a full-precision check run with an odd token count
        dict(name="linear_fp32_501", op="linear", dtype="fp32", tokens=501, k=384, n=1536),
        # a short training sequence on the small MLP (launches count)
        dict(name="grad_small_512", op="grad", dtype="bf16", tokens=512, k=384, n=1536),
        # the RoSA adapter's training step, 4096 x 4096, 2048 tokens
        dict(name="grad_rosa_2048", op="grad", dtype="fp16", tokens=2048, k=4096, n=4096),
        # a training batch on the LLaMA MLP shape
        dict(name="grad_llama_4096", op="grad", dtype="bf16", tokens=4096, k=4096, n=11008),
        # the adapter's input of a short training sequence
        dict(name="dropout_small_512", op="dropout", dtype="fp16", rows=512, cols=384, p=0.1, base=False),
        # a training batch: the adapter's part of the input gradient added to the projection's
        dict(name="dropout_llama_4096", op="dropout", dtype="bf16", rows=4096, cols=11008, p=0.05, base=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quant", "linear", "linear", "grad", "grad", "dropout"))
    if op == "quant":
        return dict(op="quant", dtype=rng.choice(("bf16", "fp16", "fp32")), rows=_log_int(rng, 1, 11008),
                    cols=_log_int(rng, 8, 4096))
    if op == "dropout":
        return dict(op="dropout", dtype=rng.choice(("bf16", "fp16", "fp32")), rows=_log_int(rng, 1, 4096),
                    cols=_log_int(rng, 8, 5504), p=rng.choice((0.05, 0.1, 0.25, round(rng.uniform(0.01, 0.9), 3))),
                    base=rng.random() < 0.5)
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp16", "fp32"))
    tokens = _log_int(rng, 1, 8000 if dtype != "fp32" else 700)
    if op == "linear" and rng.random() < 0.4:  # decode steps
        tokens = _log_int(rng, 1, 128)
    k, n = 8 * (_log_int(rng, 32, 511) | 1), 8 * (_log_int(rng, 32, 767) | 1)  # odd multiples of 16 bytes (16-bit types)
    if rng.random() < 0.12:  # rows that are no multiple of 16 bytes
        k, n, tokens = k - rng.randint(1, 7), n - rng.randint(1, 7), min(tokens, 600)
    return dict(op=op, dtype=dtype, tokens=tokens, k=k, n=n)


# ---------------------------------------------------------------- plain 4-bit values


def _blocks(x):
    """rows x cols -> rows x blocks x 32 in 32 bits, zeros behind the last column."""
    pad = -x.shape[1] % BLOCK
    return torch.nn.functional.pad(x.float(), (0, pad)).view(x.shape[0], -1, BLOCK)


def _quantize(x):
    """(codes with their sign [rows, blocks, 32], exponents [rows, blocks, 1]) of the rows of x."""
    b = _blocks(x)
    e = (torch.frexp(b.abs().amax(-1, keepdim=True))[1] - 3).clamp(-127, 127)
    y = torch.ldexp(b, -e)
    a = y.abs()
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return code + 8 * torch.signbit(y), e


def _values(code, e, cols):
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=code.device)
    return torch.ldexp(grid[code.long()], e).flatten(1)[:, :cols]


def _stored(w):
    """A weight as it is kept: two codes a byte (the first in the low bits) and a scale byte per block."""
    code, e = _quantize(w)
    pair = code.view(w.shape[0], -1, 2)
    return (pair[..., 0] + 16 * pair[..., 1]).to(torch.uint8), (e[..., 0] + 127).to(torch.uint8)


def _weight(s):
    """The stored weight in 32 bits, n x k."""
    code = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).view(s["codes"].shape[0], -1, BLOCK)
    return _values(code, s["scales"].int()[..., None] - 127, s["case"]["k"])


# ---------------------------------------------------------------- inputs


def _inputs(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def randn(*shape, std=1.0):
        return torch.empty(shape, dtype=torch.float32, device=dev).normal_(0.0, std, generator=g)

    s = dict(case=case)
    if case["op"] == "quant":
        # (rows of different size, as a trained weight has them)
        s["W"] = (randn(case["rows"], case["cols"], std=0.02) * torch.exp(randn(case["rows"], 1, std=0.5))).to(dt)
        return s
    if case["op"] == "dropout":
        s["X"] = randn(case["rows"], case["cols"]).to(dt)
        s["base"] = randn(case["rows"], case["cols"]).to(dt) if case["base"] else None
        rng = random.Random(int(seed) * 7919 + 1)
        s["seed"], s["call"] = rng.getrandbits(62), rng.getrandbits(40)
        return s
    t, k, n = case["tokens"], case["k"], case["n"]
    s["codes"], s["scales"] = _stored((randn(n, k, std=0.02) * torch.exp(randn(n, 1, std=0.5))).to(dt))
    if case["op"] == "linear":
        s["X"] = randn(t, k).to(dt)
        fused = case.get("fused", 1)  # the projection's share of a fused output, one row stride for all
        s["out"] = torch.empty((t, fused * n), dtype=dt, device=dev)[:, (fused - 1) * n:]
    else:
        s["dY"] = randn(t, n, std=1e-2).to(dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "dropout":  # the generator's state stays on the device, where captured graphs can move it on
        s["state"] = torch.tensor([s["seed"], s["call"]], dtype=torch.int64, device=s["X"].device)
    if own and case["op"] in ("linear", "grad"):  # the handle of the frozen weight
        import unstructured_sparse_linear_gb300 as sp
        s["W"] = sp.Mx4(s["codes"], s["scales"], case["k"], DTYPES[case["dtype"]])
    return s


# ---------------------------------------------------------------- plain forms


def _threshold(p):
    return int(math.floor(p * 65536.0 + 0.5))


def _plain_keep(s):
    """The mask of the values that stay: Philox4x32-7 in 64-bit integers, a block of eight numbers per step."""
    rows, cols = s["X"].shape
    low = 0xFFFFFFFF
    seed, call = s["state"][0], s["state"][1]
    groups = (cols + 7) // 8
    c0 = torch.arange(rows * groups, dtype=torch.int64, device=s["X"].device)
    c = [c0 & low, (c0 >> 32) & low, (call & low).expand_as(c0), ((call >> 32) & low).expand_as(c0)]
    key = [seed & low, (seed >> 32) & low]
    for _ in range(7):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((b >> 32) & low) ^ c[1] ^ key[0], b & low, ((a >> 32) & low) ^ c[3] ^ key[1], a & low]
        key = [(key[0] + 0x9E3779B9) & low, (key[1] + 0xBB67AE85) & low]
    words = torch.stack(c, -1)
    numbers = torch.stack((words & 0xFFFF, words >> 16), -1).view(rows, groups * 8)[:, :cols]
    return numbers >= _threshold(s["case"]["p"])


def _plain_dropout(s):
    t = _threshold(s["case"]["p"])
    factor = 65536.0 / (65536 - t) if t < 65536 else 0.0
    y = torch.where(_plain_keep(s), s["X"].float() * factor, torch.zeros((), device=s["X"].device))
    return (y if s["base"] is None else s["base"].float() + y).to(s["X"].dtype)


def _plain(s):
    op = s["case"]["op"]
    if op == "quant":
        return _values(*_quantize(s["W"]), s["case"]["cols"]).to(s["W"].dtype)
    if op == "linear":
        return (s["X"].float() @ _weight(s).t()).to(s["X"].dtype)
    if op == "grad":
        return (s["dY"].float() @ _weight(s)).to(s["dY"].dtype)
    return _plain_dropout(s)


# ---------------------------------------------------------------- one pass


def run(s):
    if not own:
        return _plain(s)
    import unstructured_sparse_linear_gb300 as sp
    case = s["case"]
    if case["op"] == "quant":
        return sp.mx4_dequantize(sp.mx4_quantize(s["W"]))
    if case["op"] == "linear":
        return sp.mx4_linear(s["X"], s["W"], out=s["out"])
    if case["op"] == "grad":
        return sp.mx4_linear_grad(s["dY"], s["W"])
    return sp.dropout(s["X"], case["p"], s["state"], base=s["base"])


def work(case):
    b = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "dropout":
        count = case["rows"] * case["cols"]
        return {"bytes": (3 if case["base"] else 2) * count * b, "flops": 3 * count}
    if case["op"] == "quant":
        count, stored = case["rows"] * case["cols"], case["rows"] * -(-case["cols"] // BLOCK) * 17
        return {"bytes": 2 * count * b + 2 * stored, "flops": 4 * count}  # (what is stored is written and read)
    t, k, n = case["tokens"], case["k"], case["n"]
    return {"bytes": t * (k + n) * b + n * -(-k // BLOCK) * 17, "flops": 2 * t * k * n}


# ---------------------------------------------------------------- 64 bits


def _exact_values(w):
    """The 4-bit values of w's rows by the distances to the grid's points, ties to the even code."""
    x = torch.nn.functional.pad(w.double(), (0, -w.shape[1] % BLOCK)).view(w.shape[0], -1, BLOCK)
    most = x.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(most > 0, most, torch.ones_like(most))))
    e = torch.where(torch.exp2(e) > most, e - 1, e)  # (log2 next to a power of two)
    e = torch.where(torch.exp2(e + 1) <= most, e + 1, e)
    size = torch.exp2((e - 2).clamp(-127, 127))
    y = (x / size).abs()
    best, at = (y - GRID[0]).abs(), torch.zeros_like(y)
    for i in range(1, 8):
        d = (y - GRID[i]).abs()
        nearer = (d < best) | ((d == best) & (i % 2 == 0))
        best, at = torch.where(nearer, d, best), torch.where(nearer, torch.full_like(y, GRID[i]), at)
    return (torch.copysign(at, x) * size).flatten(1)[:, :w.shape[1]]


def _exact_weight(s):
    low, high = (s["codes"] & 15).double(), (s["codes"] >> 4).double()
    c = torch.stack((low, high), -1).flatten(1)
    sign, c = torch.where(c >= 8, -1.0, 1.0), c % 8
    two, half = torch.floor(c / 2), c % 2  # E2M1: exponent and mantissa
    v = torch.where(two > 0, torch.exp2(two - 1) * (1 + 0.5 * half), 0.5 * half)
    size = torch.exp2(s["scales"].double() - 127).repeat_interleave(BLOCK, 1)
    return (sign * v * size)[:, :s["case"]["k"]]


def _exact_dropout(s):
    case = s["case"]
    rows, cols = case["rows"], case["cols"]
    per_row, t = -(-cols // 8), _threshold(case["p"])
    u32, mask, sh = np.uint64, np.uint64(0xFFFFFFFF), np.uint64(32)
    keep = np.empty((rows, cols), dtype=bool)
    step = max(1, (1 << 20) // per_row)
    for r0 in range(0, rows, step):
        r1 = min(rows, r0 + step)
        g = np.arange(r0 * per_row, r1 * per_row, dtype=u32)
        x0, x1 = g & mask, g >> sh
        x2, x3 = np.full_like(g, s["call"] & 0xFFFFFFFF), np.full_like(g, s["call"] >> 32)
        for i in range(7):
            k0 = np.uint64((s["seed"] + i * 0x9E3779B9) & 0xFFFFFFFF)
            k1 = np.uint64(((s["seed"] >> 32) + i * 0xBB67AE85) & 0xFFFFFFFF)
            a, b = x0 * np.uint64(0xD2511F53), x2 * np.uint64(0xCD9E8D57)
            x0, x1, x2, x3 = (b >> sh) ^ x1 ^ k0, b & mask, (a >> sh) ^ x3 ^ k1, a & mask
        u = np.stack([v for x in (x0, x1, x2, x3) for v in (x & np.uint64(0xFFFF), x >> np.uint64(16))], -1)
        keep[r0:r1] = u.reshape(r1 - r0, per_row * 8)[:, :cols] >= t
    keep = torch.from_numpy(keep).to(s["X"].device)
    y = s["X"].double() * (65536.0 / (65536 - t) if t < 65536 else 0.0) * keep
    return y if s["base"] is None else y + s["base"].double()


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "quant":
        return _exact_values(s["W"])
    if case["op"] == "linear":
        return s["X"].double() @ _exact_weight(s).t()
    if case["op"] == "grad":
        return s["dY"].double() @ _exact_weight(s)
    return _exact_dropout(s)
