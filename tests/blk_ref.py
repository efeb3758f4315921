"""Block-scaled 8-bit floating point and the RMS norm in 64 bits, from their definitions, for the tests (NumPy, no code
of the library)."""
import numpy as np

BLOCK = 128
GRID = np.array([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])


def scale_of(a):
    """The least 2^e, e >= -126, with a <= 448 2^e; NaN for a NaN or an infinity."""
    a = np.asarray(a, np.float64)
    bad = ~np.isfinite(a)
    m, e = np.frexp(np.where(bad, 0.0, a))                      # a = m 2^e, 0.5 <= m < 1
    e = np.where(a > 0, e - 9 + (m > 0.875), -126)              # 448 = 0.875 2^9
    return np.where(bad, np.nan, np.exp2(np.maximum(e, -126).astype(np.float64)))


def codes_of(v):
    """fp64 values (at most 448 in magnitude) -> E4M3 values; ties to the even code."""
    m = np.abs(v)
    up = np.clip(np.searchsorted(GRID, m, side="left"), 1, len(GRID) - 1)
    lo, hi = GRID[up - 1], GRID[up]
    mid = (lo + hi) / 2
    return np.where(m > mid, hi, np.where(m < mid, lo, np.where(up % 2 == 0, hi, lo))) * np.where(np.signbit(v), -1.0, 1.0)


def decode(q):
    """Code bytes -> values."""
    table = np.concatenate([GRID, [np.nan]])
    return table[q & 127] * np.where(q >> 7, -1.0, 1.0)


def encode(v):
    return np.searchsorted(GRID, np.abs(v)).astype(np.uint8) | (np.signbit(v).astype(np.uint8) << 7)


def spread(s, K):
    return np.repeat(s, BLOCK, -1)[..., :K]


def quantise(x):
    """fp64 [rows][K] -> E4M3 values [rows][K] and scales [rows][ceil(K/128)]."""
    x = np.asarray(x, np.float64)
    rows, K = x.shape
    pad = np.zeros((rows, -K % BLOCK))
    b = np.abs(np.concatenate([x, pad], 1)).reshape(rows, -1, BLOCK)
    s = scale_of(np.where(np.isnan(b).any(-1), np.nan, b.max(-1)))
    return codes_of(np.nan_to_num(x / spread(s, K), nan=0.0, posinf=0.0, neginf=0.0)), s


def rounded(x):
    v, s = quantise(x)
    return v * spread(s, x.shape[1])


def quantise_weights(w):
    """fp64 [E][N][K] -> E4M3 values and scales [E][ceil(N/128)][ceil(K/128)]."""
    E, N, K = w.shape
    s = np.empty((E, -(-N // BLOCK), -(-K // BLOCK)))
    for n in range(s.shape[1]):
        for k in range(s.shape[2]):
            b = np.abs(w[:, n * BLOCK:(n + 1) * BLOCK, k * BLOCK:(k + 1) * BLOCK])
            s[:, n, k] = scale_of(np.where(np.isnan(b).any((1, 2)), np.nan, b.max((1, 2))))
    full = np.repeat(np.repeat(s, BLOCK, 1)[:, :N], BLOCK, 2)[..., :K]
    return codes_of(np.nan_to_num(w / full, nan=0.0, posinf=0.0, neginf=0.0)), s


def draw_matrix(rng, E, N, K):
    """A checkpoint's matrix: code bytes and fp32 scales that are no powers of two."""
    w = rng.standard_normal((E, N, K)) / np.sqrt(K)
    s = np.empty((E, -(-N // BLOCK), -(-K // BLOCK)), np.float32)
    for n in range(s.shape[1]):
        for k in range(s.shape[2]):
            s[:, n, k] = np.abs(w[:, n * BLOCK:(n + 1) * BLOCK, k * BLOCK:(k + 1) * BLOCK]).max((1, 2)) / 448
    full = np.repeat(np.repeat(s, BLOCK, 1)[:, :N], BLOCK, 2)[..., :K]
    return encode(codes_of(np.clip(w / full, -448, 448))), s


def weights(mat):
    q, s = mat
    N, K = q.shape[1:]
    return decode(q) * np.repeat(np.repeat(s.astype(np.float64), BLOCK, 1)[:, :N], BLOCK, 2)[..., :K]


def layer(xq, routed, shared, ids, w):
    """Y [T][d] of the expert layer in 64 bits; xq: the activations' values."""
    def ffn(rows, mats, e):
        g, u, dn = (weights((m[0][e:e + 1], m[1][e:e + 1]))[0] for m in mats)
        gate = rows @ g.T
        h = gate / (1 + np.exp(-gate)) * (rows @ u.T)
        return rounded(h) @ dn.T

    y = np.zeros((xq.shape[0], routed[2][0].shape[1]))
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        y[t] += w[t, j][:, None] * ffn(xq[t], routed, e)
    if shared is not None:
        y += ffn(xq, shared, 0)
    return y


def norm(r, gamma, eps):
    return r / np.sqrt((r * r).mean(1, keepdims=True) + eps) * gamma
