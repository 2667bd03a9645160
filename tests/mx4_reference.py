"""Microscaled 4-bit values and the dropout mask in numpy, from their definitions, for the tests."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
M32 = np.uint64(0xFFFFFFFF)


def blocks_of(cols):
    return -(-cols // 32)


def quantize(x):
    """(codes [rows, 16 blocks], scales [rows, blocks]) uint8 of a matrix in 64 bits."""
    rows, cols = x.shape
    nb = blocks_of(cols)
    b = np.zeros((rows, nb * 32))
    b[:, :cols] = x
    b = b.reshape(rows, nb, 32)
    most = np.max(np.abs(b), axis=-1)  # (NaN where there is one)
    ok = np.isfinite(most)
    e = np.frexp(np.where(ok, most, 0.0))[1] - 1  # floor(log2)
    byte = np.where(most > 0, np.maximum(e + 125, 0), 0)
    y = np.where(ok[..., None], b, 0.0) / np.ldexp(1.0, byte - 127)[..., None]
    d = np.abs(np.abs(y)[..., None] - GRID)
    best = d.min(-1, keepdims=True)
    tie = d == best
    code = np.where(tie.sum(-1) > 1, np.argmax(tie & (np.arange(8) % 2 == 0), -1), np.argmax(tie, -1))
    code = code + 8 * np.signbit(y)
    code[~ok] = 0
    byte = np.where(ok, byte, 255)
    pair = code.reshape(rows, nb * 16, 2).astype(np.uint8)
    return pair[..., 0] | pair[..., 1] << 4, byte.astype(np.uint8)


def values(codes, scales, cols):
    """The stored values in 64 bits."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)
    v = np.where(c >= 8, -1.0, 1.0) * GRID[c & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (v * np.repeat(s, 32, axis=1))[:, :cols]


def philox7(index, call, seed):
    """The four words (uint64 arrays below 2^32) of each index."""
    x = [index & M32, index >> np.uint64(32), np.full_like(index, call & 0xFFFFFFFF), np.full_like(index, call >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(7):
        a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [b >> np.uint64(32) ^ x[1] ^ np.uint64(k[0]), b & M32, a >> np.uint64(32) ^ x[3] ^ np.uint64(k[1]), a & M32]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return x


def numbers(rows, cols, seed, call):
    """The 16-bit number of every place."""
    per_row = -(-cols // 8)
    w = philox7(np.arange(rows * per_row, dtype=np.uint64), call, seed)
    u = np.stack([v for x in w for v in (x & np.uint64(0xFFFF), x >> np.uint64(16))], -1)
    return u.reshape(rows, per_row * 8)[:, :cols].astype(np.int64)


def threshold(p):
    return int(np.floor(p * 65536 + 0.5))


def dropout(x, p, seed, call, base=None):
    t = threshold(p)
    keep = numbers(*x.shape, seed, call) >= t
    y = np.where(keep, x, 0.0) * (65536.0 / (65536 - t) if t < 65536 else 0.0)
    return y if base is None else base + y
