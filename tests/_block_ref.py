"""64-bit plain forms of the operators around the layer, for their tests."""
import numpy as np

PHILOX_M = (0xD2511F53, 0xCD9E8D57)
PHILOX_W = (0x9E3779B9, 0xBB67AE85)


def philox(counter, key):
    """Philox-4x32-10 (Salmon et al., SC 2011) of uint64 arrays holding 32-bit words."""
    c, k, s, low = list(counter), list(key), np.uint64(32), np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(PHILOX_M[0]), c[2] * np.uint64(PHILOX_M[1])
        c = [(p1 >> s) ^ c[1] ^ np.uint64(k[0]), p1 & low, (p0 >> s) ^ c[3] ^ np.uint64(k[1]), p0 & low]
        k = [(k[0] + PHILOX_W[0]) & 0xFFFFFFFF, (k[1] + PHILOX_W[1]) & 0xFFFFFFFF]
    return c


def cut_of(p):
    return int(np.floor(float(np.float32(p)) * 65536 + 0.5))


def draws(first, n, seed, offset):
    """16-bit draws of elements first .. first + n."""
    b0, b1 = first // 8, (first + n + 7) // 8
    b = np.arange(b0, b1, dtype=np.uint64)
    o = np.uint64(offset)
    c = philox([b & np.uint64(0xFFFFFFFF), b >> np.uint64(32), np.full_like(b, o & np.uint64(0xFFFFFFFF)),
                np.full_like(b, o >> np.uint64(32))], [seed & 0xFFFFFFFF, seed >> 32])
    u = np.stack([(c[j // 2] >> np.uint64(16 * (j % 2))) & np.uint64(0xFFFF) for j in range(8)], 1).reshape(-1)
    return u[first - b0 * 8: first - b0 * 8 + n]


def dropout(y, p, seed, offset, first=0):
    cut = cut_of(p)
    keep = draws(first, y.size, seed, offset).reshape(y.shape) >= cut
    return np.where(keep, y * (65536.0 / (65536 - cut)), 0.0)


def norm_fwd(x, gamma, beta, eps):
    mean = x.mean(1)
    rstd = 1 / np.sqrt(x.var(1) + eps)
    return (x - mean[:, None]) * rstd[:, None] * gamma + beta, mean, rstd


def norm_bwd(x, dy, gamma, mean, rstd):
    n = (x - mean[:, None]) * rstd[:, None]
    v = dy * gamma
    dx = rstd[:, None] * (v - v.mean(1, keepdims=True) - n * (v * n).mean(1, keepdims=True))
    return dx, (dy * n).sum(0), dy.sum(0)
