"""8-bit block-scaled operators on the GPU against their definitions in 64 bits: bit for bit where
only a rounding is involved, within the stated bound for products."""
import numpy as np
import pytest

import f8_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BF16_HALF = 2.0 ** -8      # a rounding to bfloat16: half of its step, relative


@pytest.fixture(scope="module")
def mx():
    from gpu_util import cuda
    return cuda()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def spread(rng, rows, cols):
    """Normal values over many binades, a few zero blocks and signed zeros."""
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-30, 30, (rows, 1)))
    x[rng.random((rows, cols)) < 0.05] = -0.0
    if rows > 2:
        x[1, :128] = 0.0
    return x


def as_type(x, t):
    with np.errstate(over="ignore"):
        x = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float64))
    return x.clamp(-60000, 60000).to(DT[t]) if t == "f16" else x.to(DT[t])


def check_codes(codes, scales, values, want_codes, want_scales, t):
    got, s = codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy()
    assert np.array_equal(s, want_scales.astype(np.float32), equal_nan=True)
    assert np.array_equal(got, want_codes)
    if values is not None:
        v = ref.VALUE[got]
        if scales.dim() == 2 and s.shape[1] == got.shape[0]:
            v = ref.row_values(got, s.astype(np.float64))
        want = torch.from_numpy(v).to(DT[t]).double()
        have = values.double().cpu()
        assert torch.equal(torch.nan_to_num(have, nan=7.5), torch.nan_to_num(want, nan=7.5))


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 4096), (3, 128), (5, 144), (37, 2880), (130, 272)])
def test_rows(mx, rows, cols, t):
    rng = np.random.default_rng(rows * 10007 + cols)
    x = as_type(spread(rng, rows, cols), t)
    codes, s = ref.quantise_rows(x.double().numpy())
    xd = x.cuda()
    out = torch.full((rows, cols), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((ref.blocks(cols), rows), -1.0, device="cuda")
    values = torch.full((rows, cols), -1.0, dtype=DT[t], device="cuda")
    mx.mxfp4_f8_quant(xd, rows, cols, cols, None, rows, out, scales, values)
    check_codes(out, scales, values, codes, s, t)
    out2 = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
    mx.mxfp4_f8_quant(xd, rows, cols, cols, None, rows, out2, scales)
    assert torch.equal(out2.view(torch.uint8), out)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("ld,first", [(2880, 0), (2888, 0), (2881, 1), (3001, 3)])
def test_gathered_and_strided_rows(mx, t, ld, first):
    rng = np.random.default_rng(ld)
    src, rows, cols = 19, 45, 2880
    x = as_type(spread(rng, src, cols), t)
    buf = torch.zeros(first + src * ld, dtype=DT[t])
    view = torch.as_strided(buf, (src, cols), (ld, 1), first)
    view.copy_(x)
    pick = rng.integers(-2, src + 2, rows).astype(np.int32)
    want = np.where(((pick >= 0) & (pick < src))[:, None], x.double().numpy()[np.clip(pick, 0, src - 1)], 0.0)
    codes, s = ref.quantise_rows(want)
    out = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    scales = torch.empty(ref.blocks(cols), rows, device="cuda")
    values = torch.empty(rows, cols, dtype=DT[t], device="cuda")
    bd = buf.cuda()
    mx.mxfp4_f8_quant(torch.as_strided(bd, (src, cols), (ld, 1), first), src, cols, ld, dev(pick), rows, out, scales, values)
    check_codes(out, scales, values, codes, s, t)


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_every_binade_border_and_tie(mx, t):
    """Largest magnitudes next to 448 2^k, and values on and next to the middles of the grid."""
    pos = ref.VALUE[:127]
    mid = (pos[:-1] + pos[1:]) / 2
    rows = []
    for k in (-126, -100, -9, 0, 7, 100, 119):
        for top in (1.75, np.nextafter(np.float32(1.75), np.float32(2)), 1.0, np.nextafter(np.float32(1), np.float32(0))):
            rows.append(np.concatenate(([top * 256.0], mid[:127], np.zeros(1)))[:128] * 2.0 ** k)
    x = as_type(np.array(rows), t)
    xs = x.double().numpy()
    codes, s = ref.quantise_rows(xs)
    out = torch.empty(xs.shape, dtype=torch.uint8, device="cuda")
    scales = torch.empty(1, len(rows), device="cuda")
    mx.mxfp4_f8_quant(x.cuda(), len(rows), 128, 128, None, len(rows), out, scales)
    check_codes(out, scales, None, codes, s, t)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_infinities_and_nan_mark_their_block_alone(mx, t):
    rng = np.random.default_rng(5)
    x = spread(rng, 6, 300)
    x[0, 5], x[1, 130], x[2, 299] = np.inf, np.nan, -np.inf
    x = as_type(x, t)
    if t == "f16":
        x[0, 5], x[2, 299] = float("inf"), float("-inf")
    x = x[:, :288].contiguous()
    x[2, 287] = float("-inf")
    codes, s = ref.quantise_rows(x.double().numpy())
    out = torch.empty(6, 288, dtype=torch.uint8, device="cuda")
    scales = torch.empty(3, 6, device="cuda")
    values = torch.empty(6, 288, dtype=DT[t], device="cuda")
    mx.mxfp4_f8_quant(x.cuda(), 6, 288, 288, None, 6, out, scales, values)
    check_codes(out, scales, values, codes, s, t)
    assert np.isnan(s).sum() == 3


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,rows,cols", [(1, 1, 16), (1, 128, 128), (2, 129, 144), (3, 300, 272)])
def test_matrices(mx, n, rows, cols, t):
    rng = np.random.default_rng(rows + cols)
    w = as_type(rng.standard_normal((n, rows, cols)) * np.exp2(rng.integers(-8, 8, (n, rows, 1))), t)
    if rows > 128:
        w[1, 5, 3] = float("nan")
    out = torch.empty(n, rows, cols, dtype=torch.uint8, device="cuda")
    scales = torch.empty(n, ref.blocks(rows), ref.blocks(cols), device="cuda")
    values = torch.empty(n, rows, cols, dtype=DT[t], device="cuda")
    mx.mxfp4_f8_quant_weight(w.cuda(), n, rows, cols, out, scales, values)
    for i in range(n):
        codes, s = ref.quantise_matrix(w[i].double().numpy())
        check_codes(out[i], scales[i:i + 1].squeeze(0)[None].squeeze(0), None, codes, s, t)
        want = torch.from_numpy(ref.matrix_values(codes, s)).to(DT[t]).double()
        assert torch.equal(torch.nan_to_num(values[i].double().cpu(), nan=7.5), torch.nan_to_num(want, nan=7.5))


# --- products ----------------------------------------------------------------------------


def check_product(got, y, l1, k, out_type):
    got = got.double().cpu().numpy()
    tol = ref.sum_bound(k, 32, ref.blocks(k)) * l1
    if out_type == "bf16":
        tol = tol * (1 + BF16_HALF) + BF16_HALF * np.abs(y)
    bad = ~(np.abs(got - y) <= tol + 1e-37)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.nanmax(np.abs(got - y) / (tol + 1e-37)):.3g}"


def dense(mx, rows, cols, nb, out_type, grad):
    rng = np.random.default_rng(rows * 31 + cols * 7 + nb)
    k, n_out = (rows, cols) if grad else (cols, rows)
    w, x = ref.random_codes(rng, (1, rows, cols)), ref.random_codes(rng, (nb, k))
    ws = ref.random_scales(rng, (1, ref.blocks(rows), ref.blocks(cols)))
    xs = ref.random_scales(rng, (ref.blocks(k), nb))
    y, l1 = ref.product(w, ws, x, xs, grad=grad)
    out = torch.full((nb + 1, n_out), 7.0, dtype=DT[out_type], device="cuda")
    f = mx.mxfp4_f8_mm_grad if grad else mx.mxfp4_f8_mm
    f(dev(w), dev(ws), rows, cols, dev(x), dev(xs), nb, out[:nb])
    check_product(out[:nb], y, l1, k, out_type)
    assert (out[nb] == 7.0).all()


SHAPES = [(1, 16, 1), (16, 128, 1), (128, 128, 16), (130, 272, 3), (256, 1024, 17), (1000, 2048, 1), (2303, 2880, 5),
          (512, 4096, 33), (384, 640, 64), (77, 400, 65), (300, 1040, 128), (640, 512, 129), (2303, 2880, 333),
          (520, 784, 257), (1024, 768, 1000)]


@pytest.mark.parametrize("out_type", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,nb", SHAPES)
def test_product(mx, rows, cols, nb, out_type):
    dense(mx, rows, cols, nb, out_type, False)


@pytest.mark.parametrize("out_type", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,nb", [(max(16, r // 16 * 16), c, n) for r, c, n in SHAPES])
def test_grad(mx, rows, cols, nb, out_type):
    dense(mx, rows, cols, nb, out_type, True)


def ragged(rng, n_experts, n_rows, behind):
    """Offsets with empty experts, single rows, and `behind` rows past the last one."""
    cut = np.sort(rng.integers(0, n_rows - behind + 1, n_experts - 1))
    if n_experts > 3:
        cut[1] = cut[0]
    return np.concatenate(([0], cut, [n_rows - behind])).astype(np.int32)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("n,rows,cols,n_rows,behind,out_type",
                         [(1, 16, 16, 1, 0, "f32"), (4, 144, 272, 9, 2, "f32"), (8, 256, 400, 40, 0, "bf16"), (5, 400, 144, 200, 7, "f32"),
                          (3, 304, 528, 500, 3, "bf16"), (64, 144, 160, 130, 1, "f32"), (2, 528, 304, 900, 0, "f32"),
                          (1024, 32, 48, 3000, 5, "f32"), (3, 272, 256, 2000, 1, "bf16")])
def test_experts(mx, n, rows, cols, n_rows, behind, out_type, grad):
    rng = np.random.default_rng(n * 1000 + rows + n_rows)
    off = ragged(rng, n, n_rows, behind)
    k, n_out = (rows, cols) if grad else (cols, rows)
    bank, x = ref.random_codes(rng, (n, rows, cols)), ref.random_codes(rng, (n_rows, k))
    bs = ref.random_scales(rng, (n, ref.blocks(rows), ref.blocks(cols)))
    xs = ref.random_scales(rng, (ref.blocks(k), n_rows))
    x[n_rows - behind:] = 127                     # NaN rows that belong to no expert
    y, l1 = ref.product(bank, bs, x, xs, off, grad)
    out = torch.full((n_rows, n_out), 7.0, dtype=DT[out_type], device="cuda")
    f = mx.mxfp4_f8_moe_mm_grad if grad else mx.mxfp4_f8_moe_mm
    f(dev(bank), dev(bs), n, rows, cols, dev(x), dev(xs), n_rows, dev(off), out)
    m = n_rows - behind
    check_product(out[:m], y[:m], l1[:m], k, out_type)
    assert (out[m:] == 7.0).all()


# --- the gradient by the matrices ------------------------------------------------------------


def check_grad_w(got, dw, l1, m, out_type):
    got = got.double().cpu().numpy()
    tol = np.array([ref.sum_bound(int(i), 16, 0) for i in m])[:, None, None] * l1
    if out_type == "bf16":
        tol = tol * (1 + BF16_HALF) + BF16_HALF * np.abs(dw)
    bad = ~(np.abs(got - dw) <= tol + 1e-37)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.nanmax(np.abs(got - dw) / (tol + 1e-37)):.3g}"


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("out_type", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,n_rows", [(8, 8, 1), (16, 264, 15), (136, 520, 16), (256, 256, 64), (264, 72, 65), (128, 512, 300)])
def test_grad_w(mx, rows, cols, n_rows, t, out_type):
    rng = np.random.default_rng(rows + cols + n_rows)
    dy, x = as_type(rng.standard_normal((n_rows, rows)), t), as_type(rng.standard_normal((n_rows, cols)), t)
    dw, l1 = ref.grad_w(dy.double().numpy(), x.double().numpy(), [0, n_rows])
    out = torch.full((rows + 1, cols), 7.0, dtype=DT[out_type], device="cuda")
    mx.mxfp4_mm_grad_w(dy.cuda(), x.cuda(), rows, cols, n_rows, out[:rows])
    check_grad_w(out[None, :rows], dw, l1, [n_rows], out_type)
    assert (out[rows] == 7.0).all()


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("n,rows,cols,n_rows,behind,out_type",
                         [(4, 136, 264, 9, 2, "f32"), (9, 1048, 520, 154, 0, "bf16"), (5, 72, 512, 700, 33, "f32"),
                          (1024, 8, 16, 3000, 1, "f32"), (3, 256, 1024, 333, 5, "bf16")])
def test_experts_grad_w(mx, n, rows, cols, n_rows, behind, t, out_type):
    rng = np.random.default_rng(n * 1000 + rows + n_rows)
    off = ragged(rng, n, n_rows, behind)
    dy, x = as_type(rng.standard_normal((n_rows, rows)), t), as_type(rng.standard_normal((n_rows, cols)), t)
    dw, l1 = ref.grad_w(dy.double().numpy(), x.double().numpy(), off)
    dy[n_rows - behind:], x[n_rows - behind:] = float("nan"), float("inf")   # rows of no expert
    out = torch.full((n, rows, cols), 7.0, dtype=DT[out_type], device="cuda")
    mx.mxfp4_moe_mm_grad_w(dy.cuda(), x.cuda(), n, rows, cols, n_rows, dev(off), out)
    check_grad_w(out, dw, l1, np.diff(off), out_type)


def test_a_neighbours_nan_stays_with_it(mx):
    """Rows of the next expert share the last 16 of one: its NaN and infinities do not leak."""
    n_rows, rows, cols = 40, 64, 72
    off = np.array([0, 13, 40], np.int32)
    rng = np.random.default_rng(3)
    dy, x = as_type(rng.standard_normal((n_rows, rows)), "bf16"), as_type(rng.standard_normal((n_rows, cols)), "bf16")
    dw, l1 = ref.grad_w(dy.double().numpy(), x.double().numpy(), off)
    x[13:], dy[20] = float("nan"), float("inf")
    out = torch.empty(2, rows, cols, device="cuda")
    mx.mxfp4_moe_mm_grad_w(dy.cuda(), x.cuda(), 2, rows, cols, n_rows, dev(off), out)
    check_grad_w(out[:1], dw[:1], l1[:1], [13], "f32")
    assert torch.isnan(out[1]).all()
