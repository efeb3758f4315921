"""MXFP4 and scored routing in 64 bits, from their definitions, for the tests (NumPy, no code of the library)."""
import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
BLOCK = 32


def quantise(x):
    """fp64 [..., K] -> (E2M1 values [..., K], E8M0 bytes [..., K/32]); ties to the even code."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    a = np.abs(b).max(-1)
    exp = np.where(a > 0, np.frexp(a)[1] - 1, -1000)            # floor(log2 a)
    e = np.clip(exp - 2, -127, 127)
    m = np.minimum(np.abs(b) * np.exp2(-e.astype(np.float64))[..., None], 6.0)
    up = np.clip(np.searchsorted(GRID, m, side="left"), 1, 7)   # GRID[up-1] < m <= GRID[up]
    lo, hi = GRID[up - 1], GRID[up]
    mid = (lo + hi) / 2
    v = np.where(m > mid, hi, np.where(m < mid, lo, np.where(up % 2 == 0, hi, lo)))
    return (v * np.sign(b)).reshape(x.shape), np.where(bad, 255, e + 127).astype(np.uint8)


def scales(byte):
    return np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))


def values(v, byte):
    """E2M1 values and bytes -> what they stand for."""
    return (v.reshape(*v.shape[:-1], -1, BLOCK) * scales(byte)[..., None]).reshape(v.shape)


def rounded(x):
    return values(*quantise(x))


def decode(q):
    """Code bytes [..., K/2] -> E2M1 values [..., K]."""
    c = np.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], -1)
    return GRID[c & 7] * np.where(c >= 8, -1.0, 1.0)


def encode(v):
    """E2M1 values [..., K] -> code bytes [..., K/2]."""
    c = np.searchsorted(GRID, np.abs(v)).astype(np.uint8) | (np.where(v < 0, 8, 0).astype(np.uint8))
    c = c.reshape(*c.shape[:-1], -1, 2)
    return c[..., 0] | (c[..., 1] << 4)


def pack(byte):
    """Row-major scale bytes [E][N][G] -> [E][ceil(N/128)][ceil(G/4)][512], element by element."""
    E, N, G = byte.shape
    out = np.zeros((E, -(-N // 128), -(-G // 4), 512), np.uint8)
    n, g = np.meshgrid(np.arange(N), np.arange(G), indexing="ij")
    out[:, n // 128, g // 4, 16 * (n % 32) + 4 * (n % 128 // 32) + g % 4] = byte
    return out


def draw_matrix(rng, E, N, K):
    """A checkpoint's matrix: (codes [E][N][K/2], bytes [E][N][K/32])."""
    v, s = quantise(rng.standard_normal((E, N, K)) / np.sqrt(K))
    return encode(v), s


def weights(mat):
    return values(decode(mat[0]), mat[1])


def scores(l, kind):
    l = np.asarray(l, np.float64)
    if kind == "sigmoid":
        with np.errstate(over="ignore"):
            return 1 / (1 + np.exp(-l))
    top = l.max(-1, keepdims=True)
    e = np.where(np.isneginf(l), 0.0, np.exp(l - np.where(np.isneginf(top), 0.0, top)))
    s = e.sum(-1, keepdims=True)
    return e / np.where(s > 0, s, 1.0)


def route_row(l, kind, bias, k, n_group=1, topk_group=1, group_top=2, renormalize=True, scale=1.0):
    """One token: (experts, weights, gap): gap is the smallest distance that the selection hangs on."""
    l = np.asarray(l, np.float64)
    E = len(l)
    s = scores(l, kind)
    masked = np.isneginf(l)
    choice = np.where(masked, -np.inf, l if bias is None else s + np.asarray(bias, np.float64))
    by = np.where(masked, -np.inf, s if bias is None else choice)
    size = E // n_group
    gap = np.inf
    kept = list(range(n_group))
    if n_group > 1:
        value = []
        for g in range(n_group):
            best = sorted(by[g * size:(g + 1) * size], reverse=True)[:group_top]
            value.append(sum(b for b in best if b > -np.inf) if best[0] > -np.inf else -np.inf)
        order = sorted(range(n_group), key=lambda g: (-value[g], g))
        kept = order[:topk_group]
        if topk_group < n_group and np.isfinite(value[order[topk_group - 1]]):
            gap = min(gap, value[order[topk_group - 1]] - value[order[topk_group]])
    among = sorted((e for g in kept for e in range(g * size, (g + 1) * size)), key=lambda e: (-choice[e], e))
    c = choice[among[:k + 1]]
    c = c[np.isfinite(c)]
    if len(c) > 1:
        gap = min(gap, float(np.min(c[:-1] - c[1:])))
    ids = among[:k]
    w = s[ids]
    if renormalize:
        w = w / w.sum() if w.sum() > 0 else np.zeros(k)
    return np.array(ids), w * scale, gap


def tables(ids, E, block_rows):
    """counts, offsets, perm, inv_perm, block_map of a selection [T][k]."""
    flat = ids.reshape(-1)
    perm = np.argsort(flat, kind="stable")
    inv = np.empty_like(perm)
    inv[perm] = np.arange(len(flat))
    counts = np.bincount(flat, minlength=E)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    tiles = [(e, offsets[e] + r, min(block_rows, counts[e] - r)) for e in range(E) for r in range(0, counts[e], block_rows)]
    return counts, offsets, perm, inv, np.array(tiles, np.int64).reshape(-1, 3)


def layer(x, routed, shared, ids, w):
    """Y [T][d] of the expert layer in 64 bits."""
    xq = rounded(x)

    def ffn(rows, mats, e):
        g, u, dn = (weights((m[0][e], m[1][e])) for m in mats)
        gate = rows @ g.T
        h = gate / (1 + np.exp(-gate)) * (rows @ u.T)
        return rounded(h) @ dn.T

    y = np.zeros((x.shape[0], routed[2][0].shape[1]))
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        y[t] += w[t, j][:, None] * ffn(xq[t], routed, e)
    if shared is not None:
        y += ffn(xq, shared, 0)
    return y
