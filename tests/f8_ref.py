"""64-bit references of the 8-bit block-scaled operators and the weight gradient, written from
their definitions: the E4M3 grid, the scale rule, products of decoded matrices.  numpy only."""
import numpy as np

B = 128


def blocks(n):
    return -(-n // B)


def _grid():
    """Values of the 256 codes: bias 7, 3 bits of fraction, codes 127 and 255 NaN."""
    v = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        m = f / 512 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if c & 127 == 127 else (-m if c & 128 else m)
    return v


VALUE = _grid()
_POS = VALUE[:127]
_MID = (_POS[:-1] + _POS[1:]) / 2


def encode(a):
    """Codes of the nearest values, ties to the even code; |a| <= 448."""
    mag = np.abs(a)
    code = np.searchsorted(_MID, mag, side="left")          # mag <= MID[i] -> i
    tie = (code < 126) & (mag == _MID[np.minimum(code, 125)])
    code = np.where(tie & (code % 2 == 1), code + 1, code)
    return (code + np.where(np.signbit(a), 128, 0)).astype(np.uint8)


def scale(top):
    """The least 2^k, k >= -126, with top <= 448 * 2^k; NaN where top is not finite."""
    if not np.isfinite(top):
        return np.nan
    k = -126
    if top > 0:
        k = max(-126, int(np.floor(np.log2(top))) - 10)
        while top > np.ldexp(448.0, k):
            k += 1
    return float(np.ldexp(1.0, k))


def _block_quant(x, height):
    """(codes, scales per block) of [rows, cols] float64, blocks of height x 128."""
    rows, cols = x.shape
    codes = np.zeros((rows, cols), np.uint8)
    s = np.empty((-(-rows // height), blocks(cols)))
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = np.s_[i * height:(i + 1) * height, j * B:(j + 1) * B]
            x_b = x[at]
            s[i, j] = scale(np.abs(x_b).max()) if np.isfinite(x_b).all() else np.nan
            if np.isfinite(s[i, j]):
                codes[at] = encode(x_b / s[i, j])
    return codes, s


def quantise_rows(x):
    """(codes [rows, cols], scales [blocks, rows])."""
    codes, s = _block_quant(x, 1)
    return codes, np.ascontiguousarray(s.T)


def quantise_matrix(w):
    """(codes [rows, cols], scales [row blocks, column blocks])."""
    return _block_quant(w, B)


def row_values(codes, s):
    return VALUE[codes] * np.repeat(s.T, B, axis=1)[:, :codes.shape[1]]


def matrix_values(codes, s):
    rows, cols = codes.shape
    return VALUE[codes] * np.repeat(np.repeat(s, B, 0)[:rows], B, 1)[:, :cols]


def random_codes(rng, shape):
    """Every finite code."""
    c = rng.integers(0, 254, shape)
    return np.where(c >= 127, c + 1, c).astype(np.uint8)


def random_scales(rng, shape):
    """No powers of two, a few binades wide."""
    return np.float32(np.exp2(rng.uniform(-9, -5, shape)))


def product(bank, bank_s, x, x_s, offsets=None, grad=False):
    """(Y, sum of magnitudes) of codes; bank [n, rows, cols].  Rows outside every expert: NaN."""
    n, rows, cols = bank.shape
    offsets = [0, x.shape[0]] if offsets is None else offsets
    xv = row_values(x, x_s.astype(np.float64))
    y = np.full((x.shape[0], cols if grad else rows), np.nan)
    l1 = np.zeros_like(y)
    for e in range(n):
        i, j = offsets[e], offsets[e + 1]
        if j > i:
            w = matrix_values(bank[e], bank_s[e].astype(np.float64))
            w = w if grad else w.T
            y[i:j], l1[i:j] = xv[i:j] @ w, np.abs(xv[i:j]) @ np.abs(w)
    return y, l1


def grad_w(dy, x, offsets):
    """(dW [n, rows, cols], sum of magnitudes)."""
    n = len(offsets) - 1
    dw = np.zeros((n, dy.shape[1], x.shape[1]))
    l1 = np.zeros_like(dw)
    for e in range(n):
        i, j = offsets[e], offsets[e + 1]
        dw[e], l1[e] = dy[i:j].T @ x[i:j], np.abs(dy[i:j]).T @ np.abs(x[i:j])
    return dw, l1


def sum_bound(k, step, blocks_added):
    """Relative to the sum of magnitudes: each addition loses less than 2^-23 of the running sum."""
    return (-(-k // step) + blocks_added + 8) * 2.0 ** -23
