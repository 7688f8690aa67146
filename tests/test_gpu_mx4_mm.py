"""Products of two MXFP4 matrices on the GPU (dense, and each expert's rows with its
matrix) against 64-bit products of the decoded matrices.

Bound: every product of two elements is exact and the sums are FP32, so |y - exact|
<= 1e-5 * sum |W X| (the library's FP32 bound).  A BF16 result is such a sum rounded
once: rounding is monotone, so it lies between the rounded ends of that interval."""
import numpy as np
import pytest

import mx4_ref as ref
from gpu_util import cuda, host, to_dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    return cuda()


def rounded(v, dtype):
    return torch.from_numpy(np.ascontiguousarray(v)).float().to(dtype).double().numpy()


def check(got, want, l1, dtype, what=""):
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN positions differ"
    ok = ~np.isnan(want)
    tol = (1e-5 * l1 + 1e-37)[ok]
    lo, hi = rounded(want[ok] - tol, dtype), rounded(want[ok] + tol, dtype)
    bad = (got[ok] < lo) | (got[ok] > hi)
    worst = np.max(np.abs(got[ok] - want[ok]) / tol) if tol.size else 0.0
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, furthest {worst} of the FP32 bound"


def product(mx, w, x, dtype=torch.float32, fill=float("nan")):
    (wc, wk), (xc, xk) = w, x
    rows, cols, nb = wc.shape[0], wc.shape[1], xc.shape[0]
    y = torch.full((nb, rows), fill, dtype=dtype, device="cuda:0")
    mx.mxfp4_mm_mx(to_dev(ref.pack(wc, wk)), rows, cols, to_dev(ref.pack(xc, xk)), nb, y)
    torch.cuda.synchronize()
    return y.double().cpu().numpy()


def both(w, x):
    wv, xv = ref.values(*w), ref.values(*x)
    return xv @ wv.T, np.abs(xv) @ np.abs(wv).T


SHAPES = [(1, 32, 1), (128, 256, 1), (16, 64, 3), (130, 96, 2), (257, 2880, 5), (128, 1024, 8), (1000, 512, 9),
          (40, 8192, 16), (129, 288, 17), (513, 4096, 31), (2303, 2880, 33), (300, 544, 64), (64, 2048, 65),
          (384, 768, 100), (255, 1056, 128), (640, 320, 129), (1024, 1024, 192), (33, 4160, 255), (511, 2880, 333),
          (2048, 512, 513), (128, 14336, 24), (4096, 4096, 1)]


@pytest.mark.parametrize("rows,cols,nb", SHAPES)
def test_against_64_bits(mx, rows, cols, nb):
    rng = np.random.default_rng(rows * 7 + cols * 3 + nb)
    w, x = ref.random_matrix(rng, rows, cols), ref.random_matrix(rng, nb, cols, 115, 140)
    want, l1 = both(w, x)
    check(product(mx, w, x), want, l1, torch.float32, "f32")
    check(product(mx, w, x, torch.bfloat16), want, l1, torch.bfloat16, "bf16")


@pytest.mark.parametrize("rows,cols,nb", [(200, 640, 3), (300, 2880, 70), (260, 1024, 300)])
def test_exact_sums_exactly(mx, rows, cols, nb):
    # all scales 1: sums of multiples of 1/4 below 2^17, exact in any order
    rng = np.random.default_rng(cols)
    w, x = ref.random_matrix(rng, rows, cols, 127, 128), ref.random_matrix(rng, nb, cols, 127, 128)
    assert np.array_equal(product(mx, w, x), both(w, x)[0])


@pytest.mark.parametrize("cols", [4096, 32768, 131072])
@pytest.mark.parametrize("nb", [2, 70])
def test_long_sums_of_one_sign(mx, cols, nb):
    # the running sum grows by 64 columns at a time, each addition losing less than 2^-23 of it:
    # cols/64 additions of a linearly growing sum lose less than cols/64 * 2^-24 of the whole,
    # and the sums within 64 columns and over slices of K a few units more
    rng = np.random.default_rng(cols + nb)
    w, x = ref.random_matrix(rng, 70, cols), ref.random_matrix(rng, nb, cols)
    w, x = (w[0] & 7, w[1]), (x[0] & 7, x[1])
    want, l1 = both(w, x)
    assert (np.abs(product(mx, w, x) - want) <= (cols / 64 + 8) * 2.0**-24 * l1).all()


@pytest.mark.parametrize("nb", [1, 20, 200])
def test_every_pair_of_codes(mx, nb):
    # row r holds code r % 16 in one place, token t code t % 16 there: the 256 products
    cols = 96
    wc, xc = np.zeros((64, cols), np.uint8), np.zeros((nb, cols), np.uint8)
    wc[:, 37], xc[:, 37] = np.arange(64) % 16, np.arange(nb) % 16
    k = lambda n: np.full((n, 3), 127, np.uint8)  # noqa: E731
    assert np.array_equal(product(mx, (wc, k(64)), (xc, k(nb))), both((wc, k(64)), (xc, k(nb)))[0])


@pytest.mark.parametrize("nb", [1, 12, 140])
def test_scale_bytes(mx, nb):
    # every pair of scale bytes whose product FP32 holds: w's byte a, x's byte b, one element each
    cols = 256 * 32
    for a in (0, 1, 2, 64, 126, 127, 200, 253, 254):
        wc, xc = np.zeros((130, cols), np.uint8), np.zeros((nb, cols), np.uint8)
        wk, xk = np.full((130, 256), a, np.uint8), np.tile(np.arange(256, dtype=np.uint8), (nb, 1))
        xk[:, 255] = 0
        # row r has its one element in group r + 60: y[t][r] is that group's product alone
        wc[np.arange(130), (np.arange(130) + 60) * 32 + np.arange(130) % 32] = 1 + np.arange(130) % 15
        xc[:] = 2
        want, l1 = both((wc, wk), (xc, xk))
        got = product(mx, (wc, wk), (xc, xk))
        ok = (np.abs(want) < 2.0**127) & ((np.abs(want) >= 2.0**-126) | (want == 0))
        assert ok.any()
        assert np.array_equal(got[ok], want[ok]), a
        # a result below FP32's normal range may be flushed or rounded, one above it is infinite
        small = np.abs(want) < 2.0**-126
        assert (np.abs(got[small] - want[small]) <= 2.0**-126).all()


@pytest.mark.parametrize("nb", [1, 12, 140])
def test_nan_scales(mx, nb):
    rng = np.random.default_rng(5)
    rows, cols = 140, 352
    w, x = ref.random_matrix(rng, rows, cols), ref.random_matrix(rng, nb, cols)
    w[1][3, 0], w[1][139, 10], w[1][64, 5] = 255, 255, 255
    w[0][64, 5 * 32:6 * 32] = 0                       # NaN even where every code is zero
    x[1][nb - 1, 7] = 255
    want, l1 = both(w, x)
    assert np.isnan(want[:, 3]).all() and np.isnan(want[nb - 1]).all() and np.isnan(want[:, 64]).all()
    check(product(mx, w, x), want, l1, torch.float32)


@pytest.mark.parametrize("cols", [32, 64, 96, 128, 160, 224, 256, 288, 480, 512, 544])
def test_nan_scales_next_to_short_rows(mx, cols):
    # a row's last tile reaches past its end: neither the next row's scale bytes nor the codes count
    rng = np.random.default_rng(cols)
    w, x = ref.random_matrix(rng, 70, cols), ref.random_matrix(rng, 20, cols)
    w[1][1::2] = 255
    x[1][1::2] = 255
    want, l1 = both(w, x)
    assert (~np.isnan(want)).sum() == 35 * 10
    check(product(mx, w, x), want, l1, torch.float32)


def test_writes_nothing_else(mx):
    rng = np.random.default_rng(6)
    w, x = ref.random_matrix(rng, 133, 320), ref.random_matrix(rng, 21, 320)
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.full((21 * 133 + 64,), 9.0, dtype=dtype, device="cuda:0")
        mx.mxfp4_mm_mx(to_dev(ref.pack(*w)), 133, 320, to_dev(ref.pack(*x)), 21, y)
        assert (host(y.float())[21 * 133:] == 9.0).all()


@pytest.mark.parametrize("rows,cols,nb", [(4096, 4096, 1), (512, 2880, 40), (1024, 2048, 700)])
def test_repeats_bit_for_bit(mx, rows, cols, nb):
    rng = np.random.default_rng(7)
    w, x = ref.random_matrix(rng, rows, cols), ref.random_matrix(rng, nb, cols)
    first = product(mx, w, x)
    for _ in range(3):
        assert np.array_equal(product(mx, w, x), first)


def test_another_stream_and_a_graph(mx):
    rng = np.random.default_rng(8)
    w, x = ref.random_matrix(rng, 300, 1024), ref.random_matrix(rng, 50, 1024)
    first = product(mx, w, x)
    wd, xd = to_dev(ref.pack(*w)), to_dev(ref.pack(*x))
    y = torch.zeros(50, 300, device="cuda:0")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mx.mxfp4_mm_mx(wd, 300, 1024, xd, 50, y, stream=s)
    torch.cuda.synchronize()
    assert np.array_equal(y.double().cpu().numpy(), first)
    y.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.mxfp4_mm_mx(wd, 300, 1024, xd, 50, y)
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(y.double().cpu().numpy(), first)


def test_output_offsets_past_32_bits(mx):
    # 2^16 + 100 tokens x 2^16 rows: y's element offsets pass 2^32
    rows, cols, nb = 1 << 16, 32, (1 << 16) + 100
    rng = np.random.default_rng(9)
    w, x = ref.random_matrix(rng, rows, cols, 127, 128), ref.random_matrix(rng, nb, cols, 127, 128)
    y = torch.empty(nb, rows, dtype=torch.bfloat16, device="cuda:0")
    mx.mxfp4_mm_mx(to_dev(ref.pack(*w)), rows, cols, to_dev(ref.pack(*x)), nb, y)
    wv, xv = ref.values(*w), ref.values(*x)
    for t in (0, 32767, 65535, 65536, nb - 1):
        want = torch.from_numpy(wv @ xv[t]).float().to(torch.bfloat16)
        assert torch.equal(y[t].cpu(), want)


# --- experts -----------------------------------------------------------------------


def experts(mx, banks, x, offsets, dtype=torch.float32, fill=123.0):
    n, rows, cols = len(banks), banks[0][0].shape[0], banks[0][0].shape[1]
    bank = np.concatenate([ref.pack(*b) for b in banks])
    n_rows = x[0].shape[0]
    y = torch.full((n_rows, rows), fill, dtype=dtype, device="cuda:0")
    mx.mxfp4_moe_mm_mx(to_dev(bank), n, rows, cols, to_dev(ref.pack(*x)), n_rows,
                       to_dev(np.asarray(offsets, np.int32)), y)
    torch.cuda.synchronize()
    return y.double().cpu().numpy()


def counts_case(kind, n, total, rng):
    if kind == "even":
        c = np.full(n, total // n)
        c[:total % n] += 1
    elif kind == "one":                     # one expert has every row, in the middle
        c = np.zeros(n, int)
        c[n // 2] = total
    elif kind == "gaps":                    # first, last and every other expert empty
        c = np.zeros(n, int)
        c[1:-1:2] = 1
        c[1] += total - c.sum()
    else:
        c = rng.multinomial(total, rng.dirichlet(np.full(n, 0.3)))
    return np.concatenate([[0], np.cumsum(c)])


@pytest.mark.parametrize("kind", ["even", "one", "gaps", "uneven"])
@pytest.mark.parametrize("n,rows,cols,total", [(5, 96, 160, 7), (8, 130, 288, 64), (16, 257, 544, 100), (4, 384, 1024, 700),
                                               (64, 64, 96, 90), (3, 2880, 2880, 50)])
def test_experts_against_64_bits(mx, kind, n, rows, cols, total):
    rng = np.random.default_rng(n * 1000 + total)
    banks = [ref.random_matrix(rng, rows, cols) for _ in range(n)]
    x = ref.random_matrix(rng, total, cols, 118, 136)
    off = counts_case(kind, n, total, rng)
    xv = ref.values(*x)
    want, l1 = np.empty((total, rows)), np.empty((total, rows))
    for e in range(n):
        wv, part = ref.values(*banks[e]), slice(off[e], off[e + 1])
        want[part], l1[part] = xv[part] @ wv.T, np.abs(xv[part]) @ np.abs(wv).T
    for dtype in (torch.float32, torch.bfloat16):
        check(experts(mx, banks, x, off, dtype), want, l1, dtype, kind)


def test_experts_leave_other_rows_alone(mx):
    rng = np.random.default_rng(11)
    banks = [ref.random_matrix(rng, 140, 96) for _ in range(4)]
    x = ref.random_matrix(rng, 40, 96)
    y = experts(mx, banks, x, [0, 3, 3, 10, 31])
    assert (y[31:] == 123.0).all() and not (y[:31] == 123.0).any(axis=1).any()
    # offsets past the rows are cut off at n_rows
    z = experts(mx, banks, x, [0, 3, 3, 10, 1000])
    assert np.array_equal(z[:31], y[:31]) and not (z == 123.0).any(axis=1).any()
    assert (experts(mx, banks, x, [0, 0, 0, 0, 0]) == 123.0).all()


def test_experts_nan_stays_with_its_expert(mx):
    rng = np.random.default_rng(12)
    banks = [ref.random_matrix(rng, 100, 160) for _ in range(3)]
    banks[1][1][:] = 255
    x = ref.random_matrix(rng, 30, 160)
    x[1][4] = 255                                     # a row of expert 0
    y = experts(mx, banks, x, [0, 9, 17, 30])
    nan = np.isnan(y)
    want = np.zeros_like(nan)
    want[9:17], want[4] = True, True
    assert np.array_equal(nan, want)


def test_one_expert_equals_the_product(mx):
    rng = np.random.default_rng(13)
    for nb in (1, 30, 300):
        w, x = ref.random_matrix(rng, 260, 1056), ref.random_matrix(rng, nb, 1056)
        want, l1 = both(w, x)
        check(experts(mx, [w], x, [0, nb]), want, l1, torch.float32)


def test_many_experts(mx):
    rng = np.random.default_rng(14)
    n = 1024
    banks = [ref.random_matrix(rng, 32, 32) for _ in range(n)]
    counts = rng.integers(0, 3, n)
    off = np.concatenate([[0], np.cumsum(counts)])
    x = ref.random_matrix(rng, int(off[-1]), 32)
    xv = ref.values(*x)
    got = experts(mx, banks, x, off)
    for e in range(n):
        part = slice(off[e], off[e + 1])
        wv = ref.values(*banks[e])
        check(got[part], xv[part] @ wv.T, np.abs(xv[part]) @ np.abs(wv).T, torch.float32)


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 7, 8, 9, 17, 32, 33])
@pytest.mark.parametrize("copies,nb", [(1, 3), (100, 5), (1, 40), (1, 130), (2, 200)])
def test_every_end_of_a_row_of_stages(mx, steps, copies, nb):
    # rows of K that end in the first or the second stage of a unit, short of a stage or at its
    # end, in slices of a split tile and (many rows, many tokens) in whole ones; sums exact in
    # any order.  The same 130 rows `copies` times.
    rng = np.random.default_rng(steps * 1000 + nb)
    for short in (0, 32, 224):
        cols, rows = 256 * steps - short, 130 * copies
        w = ref.random_matrix(rng, 130, cols, 127, 128)
        x = ref.random_matrix(rng, nb, cols, 127, 128)
        one, n = ref.pack(*w), 130 * cols
        many = np.zeros(ref.nbytes(rows, cols), np.uint8)
        many[:rows * cols // 2] = np.tile(one[:n // 2], copies)
        many[rows * cols // 2:rows * cols * 17 // 32] = np.tile(one[n // 2:n * 17 // 32], copies)
        y = torch.zeros(nb, rows, device="cuda:0")
        mx.mxfp4_mm_mx(to_dev(many), rows, cols, to_dev(ref.pack(*x)), nb, y)
        assert np.array_equal(host(y), np.tile(both(w, x)[0], (1, copies)))


@pytest.mark.parametrize("rows", [128, 132, 156, 160, 188, 252, 254, 255])
@pytest.mark.parametrize("nb", [65, 97, 209])
def test_stores_of_every_width(mx, rows, nb):
    # FP32 and BF16 results in units of four rows where the row count allows it, else one by one
    rng = np.random.default_rng(rows + nb)
    w, x = ref.random_matrix(rng, rows, 96, 127, 128), ref.random_matrix(rng, nb, 96, 127, 128)
    want, l1 = both(w, x)
    assert np.array_equal(product(mx, w, x), want)
    check(product(mx, w, x, torch.bfloat16), want, l1, torch.bfloat16, "bf16")


def stated_bound(cols):
    """The error bound of include/mx4.h, in units of sum |W X|."""
    import os
    import re
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mx4.h")) as f:
        add, power = re.search(r"\(cols / 64 \+ (\d+)\) \* 2\^-(\d+) \* sum_c", f.read()).groups()
    return (cols / 64 + int(add)) * 2.0**-int(power)


@pytest.mark.parametrize("cols", [4096, 32768])
@pytest.mark.parametrize("nb", [2, 70])
def test_sums_with_a_dominant_first_block(mx, cols, nb):
    # an element of 1, then 64 columns at a time that come to 63/64 of a last bit of the sum (2^-23):
    # every addition may lose all of it.  Row 0: one sign; 1: the rest negative; 2: signs in turn;
    # 3: an element of 1 at each eighth of the row, where slices of a split row begin; 4: as row 0
    # with 3/4 of a last bit.
    wc, wk = np.zeros((5, cols), np.uint8), np.full((5, cols // 32), 127 - 29, np.uint8)
    for r, (n, sign) in enumerate([(63, "+"), (63, "-"), (63, "+-"), (63, "+"), (48, "+")]):
        block = np.zeros(64, np.uint8)
        block[:n] = 2
        blocks = np.tile(block, (cols // 64, 1))
        blocks[(slice(None) if sign == "-" else slice(1, None, 2)) if "-" in sign else slice(0)] |= 8
        blocks = np.where(blocks == 8, 0, blocks)
        for b in range(0, cols // 64, cols // 512 if r == 3 else cols):
            blocks[b], wk[r, 2 * b:2 * b + 2] = 0, 127
            blocks[b, 0] = 2
        wc[r] = blocks.reshape(-1)
    w, x = (wc, wk), (np.full((nb, cols), 2, np.uint8), np.full((nb, cols // 32), 127, np.uint8))
    want, l1 = both(w, x)
    bound = stated_bound(cols)
    assert (np.abs(product(mx, w, x) - want) <= bound * l1).all()
    # the input is one that tells the bound from half of it: what an unsplit row can lose
    assert want[0, 0] - 1 > bound / 2
