"""64-bit references of the microscaled 4-bit operators, written from their
definitions: the E2M1 grid, the scale rule, products of decoded matrices, and the
routing sums.  numpy only."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def nbytes(rows, cols):
    return (rows * cols * 17 // 32 + 15) // 16 * 16


def quantise(x):
    """[rows, cols] float64 -> (codes uint8 [rows, cols], scale bytes uint8 [rows, cols/32])."""
    rows, cols = x.shape
    g = x.reshape(rows, cols // 32, 32)
    fine = np.isfinite(g).all(-1)
    g = np.where(fine[..., None], g, 0.0)
    top = np.abs(g).max(-1)
    _, e = np.frexp(top)                       # top = m 2^e, 1/2 <= m < 1
    exp = np.where(top > 0, e - 1 - 2, -127)
    exp = np.maximum(exp, -127)
    a = np.ldexp(np.abs(g), -exp[..., None])
    # nearest grid value, ties to the even code
    code = np.zeros(g.shape, dtype=np.uint8)
    for i in range(7):
        mid = (GRID[i] + GRID[i + 1]) / 2
        up = (a > mid) if i % 2 == 0 else (a >= mid)
        code[up] = i + 1
    code |= np.where(np.signbit(g), 8, 0).astype(np.uint8)
    code = np.where(fine[..., None], code, 0).astype(np.uint8)
    k = np.where(fine, exp + 127, 255).astype(np.uint8)
    return code.reshape(rows, cols), k


def pack(code, k):
    """Codes and scale bytes -> the buffer (zero padding)."""
    rows, cols = code.shape
    out = np.zeros(nbytes(rows, cols), dtype=np.uint8)
    out[:rows * cols // 2] = (code[:, 0::2] | (code[:, 1::2] << 4)).reshape(-1)
    out[rows * cols // 2:rows * cols * 17 // 32] = k.reshape(-1)
    return out


def values(code, k):
    """Codes and scale bytes -> float64 values (NaN where k = 255)."""
    v = np.where(code & 8, -1.0, 1.0) * GRID[code & 7]
    s = np.where(k == 255, np.nan, np.ldexp(1.0, k.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=1)


def random_matrix(rng, rows, cols, lo=120, hi=131):
    """Uniform codes, scale bytes uniform in [lo, hi): (codes, scale bytes)."""
    return (rng.integers(0, 16, (rows, cols)).astype(np.uint8),
            rng.integers(lo, hi, (rows, cols // 32)).astype(np.uint8))


def sort_pairs(ids, top_k, n_experts):
    """(token_at, pos_of, offsets) of the stable counting sort."""
    ids = np.asarray(ids).reshape(-1)
    kept = [p for p in range(ids.size) if 0 <= ids[p] < n_experts]
    order = sorted(kept, key=lambda p: (ids[p], p))
    token_at = np.full(ids.size, -1, np.int32)
    pos_of = np.full(ids.size, -1, np.int32)
    for i, p in enumerate(order):
        token_at[i], pos_of[p] = p // top_k, i
    offsets = np.zeros(n_experts + 1, np.int32)
    for p in kept:
        offsets[ids[p] + 1:] += 1
    return token_at, pos_of, offsets
