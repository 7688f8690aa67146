"""The 4-bit and routing kernels at the sizes that choose their other variants: prompts' tiles of
more than 64 tokens with several stages, scale rows too long for the bulk copies, more tiles a CTA
than its table holds, many rows of the movers and the quantisers.

The references and bounds are those of the modules that test the same calls at small sizes."""
import numpy as np
import pytest

import mx4_ref as ref
import test_gpu_moe_route as route
import test_gpu_mx4_mm as mm
import test_gpu_mx4_quant as quant
from gpu_util import cuda

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def mx():
    return cuda()


def both(w, x):
    """mm.both in 64 bits on the GPU."""
    wv, xv = (torch.from_numpy(ref.values(*m)).cuda() for m in (w, x))
    return (xv @ wv.T).cpu().numpy(), (xv.abs() @ wv.abs().T).cpu().numpy()


# tiles of 112 and 128 tokens in single stages (scale rows by bulk copies) and in pairs (loaded);
# of 144 to 192 tokens, two blocks of scales, copied and loaded, aligned rows of scales and others;
# rows and tokens that fill no tile; a row's last stage short
DENSE = [(4864, 2880, 500), (1000, 2912, 2000), (2944, 4352, 1300), (4700, 4064, 490), (4864, 4096, 500), (4800, 4128, 499),
         (4096, 4096, 2048), (1216, 2880, 2000), (1200, 4128, 2001), (2880, 2880, 1000), (2501, 2336, 2430), (300, 5152, 3000),
         (16, 4096, 4000), (1, 288, 1500)]


@pytest.mark.parametrize("rows,cols,nb", DENSE)
def test_prompts_against_64_bits(mx, rows, cols, nb):
    rng = np.random.default_rng(rows * 7 + cols + nb)
    w, x = ref.random_matrix(rng, rows, cols), ref.random_matrix(rng, nb, cols)
    want, l1 = both(w, x)
    mm.check(mm.product(mx, w, x), want, l1, torch.float32, "f32")
    mm.check(mm.product(mx, w, x, torch.bfloat16), want, l1, torch.bfloat16, "bf16")


@pytest.mark.parametrize("rows,cols,nb", DENSE)
def test_prompts_exactly(mx, rows, cols, nb):
    # all scales 1: sums of multiples of 1/4 below 2^18, exact in any order
    rng = np.random.default_rng(rows + cols + nb)
    w, x = ref.random_matrix(rng, rows, cols, 127, 128), ref.random_matrix(rng, nb, cols, 127, 128)
    assert np.array_equal(mm.product(mx, w, x), both(w, x)[0])


@pytest.mark.parametrize("rows,cols,nb", [(4864, 2880, 500), (2944, 4352, 1300), (1200, 4128, 2001)])
def test_prompts_nan_scales(mx, rows, cols, nb):
    rng = np.random.default_rng(rows)
    w, x = ref.random_matrix(rng, rows, cols), ref.random_matrix(rng, nb, cols)
    w[1][[0, 127, 128, rows - 1], [0, 1, cols // 32 - 1, 7]] = 255
    x[1][[0, 111, 128, nb - 1], [3, cols // 32 - 1, 0, 5]] = 255
    want, l1 = both(w, x)
    assert np.isnan(want).sum() == 4 * nb + 4 * rows - 16
    mm.check(mm.product(mx, w, x), want, l1, torch.float32)


# (experts, rows, columns, rows of X): tiles of 16, 32, 96, 128 and 160 rows of X a tile, with scale
# rows loaded from each expert's own plane (long rows) and copied, aligned and not
@pytest.mark.parametrize("kind", ["even", "one", "gaps", "uneven"])
@pytest.mark.parametrize("n,rows,cols,total", [(4, 130, 14336, 20), (4, 130, 14368, 21), (3, 257, 7328, 60), (5, 130, 4640, 250),
                                               (3, 260, 4160, 360), (3, 130, 4128, 500), (3, 130, 2880, 370), (3, 200, 1056, 600)])
def test_experts_against_64_bits(mx, kind, n, rows, cols, total):
    rng = np.random.default_rng(n * 1000 + total + cols)
    banks = [ref.random_matrix(rng, rows, cols) for _ in range(n)]
    banks[0][1][rows - 1, cols // 32 - 1] = 255        # (next to the next expert's codes)
    x = ref.random_matrix(rng, total, cols, 118, 136)
    off = mm.counts_case(kind, n, total, rng)
    want, l1 = np.empty((total, rows)), np.empty((total, rows))
    for e in range(n):
        part = slice(off[e], off[e + 1])
        want[part], l1[part] = both(banks[e], (x[0][part], x[1][part]))
    for dtype in (torch.float32, torch.bfloat16):
        mm.check(mm.experts(mx, banks, x, off, dtype), want, l1, dtype, kind)


def test_more_tiles_than_a_ctas_table(mx):
    # 15 row tiles of some 680 experts over at most 152 CTAs: more than 64 each
    n, rows, cols = 1024, 1920, 32
    rng = np.random.default_rng(3)
    counts = rng.integers(0, 3, n)
    assert (counts > 0).sum() * 15 > 64 * 152
    off = np.concatenate([[0], np.cumsum(counts)])
    code, k = ref.random_matrix(rng, n * rows, cols, 127, 128)
    banks = [(code[e * rows:(e + 1) * rows], k[e * rows:(e + 1) * rows]) for e in range(n)]
    x = ref.random_matrix(rng, int(off[-1]), cols, 127, 128)
    got = mm.experts(mx, banks, x, off)
    xv = ref.values(*x)
    for e in range(n):
        part = slice(off[e], off[e + 1])
        assert np.array_equal(got[part], xv[part] @ ref.values(*banks[e]).T), e


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,k,width", [(608, 4, 2880), (700, 3, 1001), (1300, 2, 333), (900, 5, 66), (2000, 1, 1), (650, 4, 4100)])
def test_routing_of_many_tokens(mx, dtype, t, k, width):
    route.test_rows_and_gradients(mx, dtype, t, k, width)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad", [0, 8, 1])             # rows aligned to 32 bytes, to 16, to an element
def test_quantisation_of_many_rows(mx, dtype, pad):
    rows, cols = (1301, 4096) if dtype is torch.float32 else (2601, 4096)
    g = torch.Generator().manual_seed(pad)
    x = torch.randn(rows, cols + pad, generator=g) * torch.exp2(4 * torch.randn(rows, 1, generator=g))
    x[5, 64], x[rows - 1, cols - 1] = float("nan"), float("inf")
    quant.check(mx, x.to(dtype).cuda()[:, :cols], ld=cols + pad)
