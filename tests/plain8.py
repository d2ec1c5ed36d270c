"""The 8-bit operators from their definitions in numpy, in 64 bits (the tests' reference)."""
import numpy as np


def int8_rows(x):
    """q, scale (float32) and bad rows of x [n, k] float64."""
    with np.errstate(all="ignore"):
        a = np.abs(x).max(1)
        bad = ~np.isfinite(x).all(1)
        q = np.rint(x * 127.0 / a[:, None])  # 127 x is exact; a quotient that is no half rounds to no half
    q[bad | (a == 0)] = 0
    scale = np.where(bad, np.float32(np.nan), a.astype(np.float32) / np.float32(127))
    return q.astype(np.int8), scale.astype(np.float32), bad


def philox(seed, rows, n, row0=0):
    """Words of the Philox4x32-10 blocks 0 .. n-1 of rows row0 and on, third counter word 2: [rows, n, 4] uint64."""
    u, low = np.uint64, np.uint64(0xFFFFFFFF)
    c = [np.broadcast_to(np.arange(n, dtype=u), (rows, n)), np.broadcast_to(np.arange(row0, row0 + rows, dtype=u)[:, None], (rows, n)),
         np.full((rows, n), 2, u), np.zeros((rows, n), u)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF
    for _ in range(10):
        p, q = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(q >> u(32)) ^ c[1] ^ u(k0), q & low, (p >> u(32)) ^ c[3] ^ u(k1), p & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, -1)


def checkpoint(x, seed, row0=0):
    """q int8 [t, k] and scale bytes [t, blocks] of x [t, k] float64, rows row0 and on of a matrix."""
    t, k = x.shape
    blocks = (k + 31) // 32
    full = np.zeros((t, blocks * 32))
    full[:, :k] = x
    full = full.reshape(t, blocks, 32)
    size = np.abs(full)
    top = size.max(2)  # NaN where the block holds one
    mantissa, exponent = np.frexp(np.where(np.isfinite(top), top, 0))
    e = np.maximum(exponent - 7 + (mantissa > 127 / 128), -126)  # 127 = (127 / 128) 2^7
    e = np.where(top == 0, -126, e)
    bad = ~(top <= 127 * 2.0**121)
    b = np.where(bad, 255, e + 127).astype(np.uint8)
    z = np.where(bad[:, :, None], 0, size) / np.exp2(e)[:, :, None]
    w = philox(seed, t, blocks * 4, row0)
    u = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(z.shape).astype(np.float64)
    low = np.floor(z)
    q = np.where(full < 0, -1, 1) * (low + (u < np.rint((z - low) * 65536)))
    return q.reshape(t, -1)[:, :k].astype(np.int8), b


def values(q, b):
    """The values of a checkpoint in float64, NaN in marked blocks."""
    s = np.where(b == 255, np.nan, np.exp2(b.astype(np.float64) - 127)).repeat(32, 1)[:, : q.shape[1]]
    return q.astype(np.float64) * s
