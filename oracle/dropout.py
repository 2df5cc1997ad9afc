"""Float64 oracle of the counter-based dropout.  Philox4x32-10: Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as
1, 2, 3" (SC'11), table 2 and section 3.3."""
import numpy as np


def philox4x32(counter, key, rounds=10):
    """counter: four uint32 arrays, key: two ints; returns four uint32 arrays."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(key[0]), int(key[1])]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(rounds):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & low, (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return [v.astype(np.uint32) for v in c]


def keep(T, H, p, seed, offset, row0=0):
    """Truth values [T, H] of the rows row0 .."""
    quad = np.arange(-(-H // 4), dtype=np.uint32)[None, :]
    row = (row0 + np.arange(T, dtype=np.uint64)).astype(np.uint32)[:, None]
    shape = np.broadcast(quad, row).shape
    fill = lambda v: np.broadcast_to(v, shape)  # noqa: E731
    words = philox4x32([fill(quad), fill(row), fill(np.uint32(offset % 2 ** 32)), fill(np.uint32(offset // 2 ** 32 % 2 ** 32))],
                       [seed % 2 ** 32, seed // 2 ** 32])
    border = min(2 ** 32 - 1, int(np.floor(p * 2.0 ** 32 + 0.5)))
    return (np.stack(words, 2).reshape(T, -1)[:, :H] >= np.uint32(border)) if T else np.zeros((0, H), bool)


def forward(x, p, seed, offset, residual=None):
    y = np.where(keep(*x.shape, p, seed, offset), x / (1 - p), 0.0)
    return y if residual is None else y + residual
