"""Quantisation to MXFP4 on the GPU against the 64-bit reference: codes and scale
bytes bit for bit (the one rounding has an exact answer), the rounded values, every
input type, strides, gathered rows, special values, offsets past 32 bits."""
import numpy as np
import pytest

import mx4_ref as ref
from gpu_util import cuda, host, to_dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def mx():
    return cuda()


def run(mx, x, rows=None, row_of=None, ld=None, want_values=True):
    """x: [x_rows, cols] device tensor (rows ld apart) -> (codes, scale bytes, values)."""
    x_rows, cols = x.shape
    rows = x_rows if rows is None else rows
    out = torch.full((ref.nbytes(rows, cols),), 0xA5, dtype=torch.uint8, device="cuda:0")
    values = torch.full((rows, cols), 7.0, dtype=x.dtype, device="cuda:0") if want_values else None
    mx.mxfp4_quant(x, x_rows, cols, cols if ld is None else ld, row_of, rows, out, values)
    o = host(out)
    n = rows * cols
    byte = o[:n // 2].reshape(rows, cols // 2)
    code = np.empty((rows, cols), np.uint8)
    code[:, 0::2], code[:, 1::2] = byte & 15, byte >> 4
    assert (o[n * 17 // 32:] == 0xA5).all(), "the padding was written"
    return code, o[n // 2:n * 17 // 32].reshape(rows, cols // 32), \
        None if values is None else values.double().cpu().numpy()


def check(mx, x, want=None, **kw):
    want = x.double().cpu().numpy() if want is None else want
    code, k, v = run(mx, x, **kw)
    wc, wk = ref.quantise(want)
    assert np.array_equal(k, wk)
    bad = np.argwhere(code != wc)
    assert bad.size == 0, f"{len(bad)} codes differ, first at {bad[0]}: {code[tuple(bad[0])]} for {wc[tuple(bad[0])]}"
    if v is not None:
        wv = ref.values(wc, wk)
        assert np.array_equal(v, wv, equal_nan=True)
        assert np.array_equal(np.signbit(v[v == 0]), np.signbit(wv[wv == 0]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 4096), (3, 96), (65, 2880), (7, 160), (300, 1056)])
def test_random_values(mx, dtype, rows, cols):
    g = torch.Generator().manual_seed(rows * 31 + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(4 * torch.randn(rows, 1, generator=g))
    check(mx, x.to(dtype).cuda())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_every_16_bit_value(mx, dtype):
    # every finite bit pattern beside a largest element of each nearby binade: all ties,
    # all scales the type reaches, subnormals, both zeros
    bits = np.arange(65536, dtype=np.uint16)
    x = torch.from_numpy(bits.view(np.int16)).view(dtype)
    x = x[torch.isfinite(x.float())]
    for up in (1.0, 1.5, 4.0, 8.0):
        x2 = torch.stack([x.float(), x.float().abs() * up], 1).to(dtype)   # pairs (x, its amax)
        x2 = torch.where(torch.isfinite(x2.float()), x2, torch.zeros_like(x2))
        groups = torch.zeros(x2.shape[0], 32, dtype=dtype)
        groups[:, 5], groups[:, 30] = x2[:, 0], x2[:, 1]
        check(mx, groups.cuda())


def test_ties_and_neighbours_at_every_scale(mx):
    # each midpoint of the grid and its FP32 neighbours, at every exponent FP32 has
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    near = np.concatenate([mids, np.nextafter(mids, np.float32(9)), np.nextafter(mids, np.float32(0))])
    rows = []
    for e in range(-127, 126):
        row = np.zeros(32, np.float32)
        row[0] = np.ldexp(np.float32(4.0), e)
        row[1:22] = np.ldexp(near, e) * np.where(np.arange(21) % 2, -1, 1)
        rows.append(row)
    check(mx, torch.from_numpy(np.stack(rows)).cuda())


@pytest.mark.parametrize("dtype", TYPES)
def test_special_values(mx, dtype):
    fi = torch.finfo(dtype)
    x = torch.zeros(9, 64, dtype=dtype)
    x[0, 3], x[1, 40], x[2, 0], x[3, 63] = float("nan"), float("inf"), -float("inf"), -float("nan")
    x[2, 1], x[1, 1] = 3.0, -2.0                 # finite neighbours in the same and the other group
    x[4] = -0.0
    x[5, ::7], x[5, 1] = fi.max, fi.min
    x[6, 2] = fi.smallest_normal
    x[7, 2], x[7, 33] = fi.smallest_normal / 2, -fi.tiny / 4
    x[8, 0], x[8, 1] = fi.max, fi.tiny
    check(mx, x.cuda())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ld,shift", [(128, 0), (96, 0), (97, 0), (100, 4), (96, 1)])
def test_strides_and_alignment(mx, dtype, ld, shift):
    rows, cols = 11, 96
    flat = torch.randn(rows * ld + 8, generator=torch.Generator().manual_seed(ld)).to(dtype).cuda()
    x = flat[shift:shift + rows * ld].reshape(rows, ld)[:, :cols]
    check(mx, x, ld=ld)


def test_gathered_rows(mx):
    g = torch.Generator().manual_seed(4)
    x = torch.randn(50, 288, generator=g).to(torch.bfloat16)
    idx = torch.randint(0, 50, (133,), generator=g, dtype=torch.int32)
    idx[7], idx[20], idx[21], idx[132] = -1, 50, 2**31 - 1, -2**31
    want = torch.where(((idx >= 0) & (idx < 50))[:, None], x[idx.clamp(0, 49).long()].double(), 0.0).numpy()
    check(mx, x.cuda(), want=want, rows=133, row_of=idx.cuda())
    check(mx, x.cuda(), want=want, rows=133, row_of=idx.cuda(), want_values=False)


def test_dequant_reads_it_back(mx):
    x = torch.randn(40, 512, generator=torch.Generator().manual_seed(8)).cuda()
    out = torch.zeros(ref.nbytes(40, 512), dtype=torch.uint8, device="cuda:0")
    values, back = torch.empty_like(x), torch.empty_like(x)
    mx.mxfp4_quant(x, 40, 512, 512, None, 40, out, values)
    mx.mxfp4_dequant(out, 40, 512, back)
    assert torch.equal(values, back)


def test_another_stream(mx):
    x = torch.randn(64, 1024, generator=torch.Generator().manual_seed(9)).cuda()
    s = torch.cuda.Stream()
    out = [torch.zeros(ref.nbytes(64, 1024), dtype=torch.uint8, device="cuda:0") for _ in range(2)]
    mx.mxfp4_quant(x, 64, 1024, 1024, None, 64, out[0])
    s.wait_stream(torch.cuda.current_stream())
    mx.mxfp4_quant(x, 64, 1024, 1024, None, 64, out[1], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1])


def test_offsets_past_32_bits(mx):
    # 2.4e9 elements: element and byte offsets of x, of the codes and of the values pass 2^31 and 2^32
    rows, cols = 75000, 32768
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda:0")
    pick = torch.tensor([0, 1, 32767, 65535, 65536, rows - 1])
    part = torch.randn(len(pick), cols, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    x[pick.cuda()] = part.cuda()
    out = torch.empty(ref.nbytes(rows, cols), dtype=torch.uint8, device="cuda:0")
    values = torch.empty_like(x)
    mx.mxfp4_quant(x, rows, cols, cols, None, rows, out, values)
    code, k = ref.quantise(part.double().numpy())
    v = values[pick.cuda()].double().cpu().numpy()
    assert np.array_equal(v, ref.values(code, k))
    byte = (code[:, 0::2] | (code[:, 1::2] << 4))
    got = out[:rows * cols // 2].view(rows, cols // 2)[pick.cuda()].cpu().numpy()
    assert np.array_equal(got, byte)
    got = out[rows * cols // 2:rows * cols * 17 // 32].view(rows, cols // 32)[pick.cuda()].cpu().numpy()
    assert np.array_equal(got, k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("limit", [0.0, 1.5])
@pytest.mark.parametrize("rows,cols,ld", [(1, 32, 32), (33, 2880, 2880), (9, 96, 101)])
def test_swiglu(mx, dtype, limit, rows, cols, ld):
    """act in FP32 has a relative error of a few 2^-24 (expf 2 ulp, one add, one divide, one
    product): below 2^-20.  So the scale is that of amax (1 -+ 2^-20) and the code that of
    act (1 -+ 2^-20), both monotone."""
    g = torch.Generator().manual_seed(rows + cols)
    flat = [(3 * torch.randn(rows, ld, generator=g)).to(dtype) for _ in range(2)]
    gate, up = (f.cuda()[:, :cols] for f in flat)
    out = torch.zeros(ref.nbytes(rows, cols), dtype=torch.uint8, device="cuda:0")
    values = torch.zeros(rows, cols, dtype=dtype, device="cuda:0")
    mx.mxfp4_swiglu_quant(gate, up, rows, cols, ld, out, values, swiglu_limit=limit)
    gd, ud = (f[:, :cols].double().numpy() for f in flat)
    if limit > 0:
        ud, gd = np.clip(ud, -limit, limit), np.minimum(gd, limit)
    act = gd / (1 + np.exp(-gd)) * ud
    o = host(out)
    n = rows * cols
    byte = o[:n // 2].reshape(rows, cols // 2)
    code = np.empty((rows, cols), np.uint8)
    code[:, 0::2], code[:, 1::2] = byte & 15, byte >> 4
    k = o[n // 2:n * 17 // 32].reshape(rows, cols // 32)
    lo, hi = ref.quantise(act * (1 - 2.0**-20)), ref.quantise(act * (1 + 2.0**-20))
    assert ((k == lo[1]) | (k == hi[1])).all()
    sure = np.repeat(lo[1] == hi[1], 32, axis=1)          # the scale is settled
    ok = (code == lo[0]) | (code == hi[0])
    assert ok[sure].all() and sure.mean() > 0.9
    v = values.double().cpu().numpy()
    assert np.array_equal(v, ref.values(code, k))


def test_swiglu_nonfinite(mx):
    gate = torch.zeros(4, 32)
    up = torch.ones(4, 32)
    gate[0, 1], up[1, 2], gate[2, 3] = float("nan"), float("inf"), -float("inf")
    out = torch.zeros(ref.nbytes(4, 32), dtype=torch.uint8, device="cuda:0")
    mx.mxfp4_swiglu_quant(gate.cuda(), up.cuda(), 4, 32, 32, out)
    # row 1: silu(0) * inf = NaN; row 2: -inf / (1 + inf) = NaN
    assert host(out)[64:68].tolist() == [255, 255, 255, 0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("up_exp", [0, 60, 126])
def test_swiglu_far_gates(mx, dtype, up_exp):
    """Gates whose exponential is tiny, subnormal or nothing, under large ups: silu must fade out
    through exp's whole range, not end early.  Beside the relative 2^-20 an exponential below
    2^-126 is off by up to 2^-149."""
    far = [-60.0, -80.0, -86.0, -87.0, -88.0, -88.5, -89.0, -92.0, -96.0, -100.0, -104.0, -200.0]
    gate = torch.tensor(far).repeat_interleave(64).reshape(len(far), 64).to(dtype)
    up = (torch.linspace(-1.9, 1.9, 64).repeat(len(far), 1) * 2.0**up_exp).to(dtype)
    out = torch.zeros(ref.nbytes(len(far), 64), dtype=torch.uint8, device="cuda:0")
    mx.mxfp4_swiglu_quant(gate.cuda(), up.cuda(), len(far), 64, 64, out)
    g, u = gate.double().numpy(), up.double().numpy()
    act = g / (1 + np.exp(-g)) * u
    slack = np.abs(act) * 2.0**-20 + np.abs(g * u) * 2.0**-149 + 2.0**-149
    o = host(out)
    n = gate.numel()
    byte = o[:n // 2].reshape(len(far), 32)
    code = np.empty((len(far), 64), np.uint8)
    code[:, 0::2], code[:, 1::2] = byte & 15, byte >> 4
    k = o[n // 2:n * 17 // 32].reshape(len(far), 2)
    # as above, on magnitudes (a result that may be zero may have either sign)
    lo = ref.quantise(np.maximum(np.abs(act) - slack, 0.0))
    hi = ref.quantise(np.abs(act) + slack)
    assert ((k >= lo[1]) & (k <= hi[1])).all()
    sure = np.repeat(lo[1] == hi[1], 32, axis=1)
    mag = code & 7
    assert ((mag >= lo[0]) & (mag <= hi[0]))[sure].all()
    assert sure[:4].all()


def test_weights_quantised_ahead_of_an_overlapped_matvec(mx):
    """mxfp4_mv with launch overlap reads weights before it waits for the kernel ahead of it: a
    quantiser that writes them, directly ahead or with another launch between, has to be done."""
    rows, cols = 4096, 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    ws = [torch.randn(rows, cols, generator=g, device="cuda") for _ in range(4)]
    x = torch.randn(cols, generator=g, device="cuda")
    w = torch.zeros(ref.nbytes(rows, cols), dtype=torch.uint8, device="cuda:0")
    xq = torch.zeros(ref.nbytes(1, cols), dtype=torch.uint8, device="cuda:0")
    y4 = torch.zeros(1, rows, device="cuda")
    mx.mxfp4_quant(x, 1, cols, cols, None, 1, xq)
    want, got = [torch.zeros(rows, device="cuda") for _ in ws], []
    for v, y in zip(ws, want):
        mx.mxfp4_quant(v, rows, cols, cols, None, rows, w)
        torch.cuda.synchronize()
        mx.mxfp4_mv(w, rows, cols, x, y)
    torch.cuda.synchronize()
    mx.mxfp4_set_launch_overlap(True)
    try:
        for i in range(24):
            y = torch.zeros(rows, device="cuda")
            mx.mxfp4_quant(ws[i % 4], rows, cols, cols, None, rows, w)
            if i % 8 >= 4:
                mx.mxfp4_mm_mx(w, rows, cols, xq, 1, y4)
            mx.mxfp4_mv(w, rows, cols, x, y)
            got.append(y)
        torch.cuda.synchronize()
    finally:
        mx.mxfp4_set_launch_overlap(False)
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 4]), i


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ld", [64, 67])
def test_swiglu_nonfinite_under_a_limit(mx, dtype, ld):
    """A NaN gate or up is no larger than any limit: its group is NaN.  Infinities are clamped,
    but for a gate of -inf (-inf / (1 + inf) = NaN).  Aligned rows and others."""
    nan, inf, rows = float("nan"), float("inf"), 8
    gate, up = (torch.ones(rows, ld, dtype=dtype) for _ in range(2))
    gate[0, 1], gate[1, 40], up[2, 31], up[3, 32] = nan, -nan, nan, -nan
    gate[4, 0], up[5, 0], up[6, 0], gate[7, 63] = inf, inf, -inf, -inf
    out = torch.zeros(ref.nbytes(rows, 64), dtype=torch.uint8, device="cuda:0")
    values = torch.zeros(rows, 64, dtype=dtype, device="cuda:0")
    mx.mxfp4_swiglu_quant(gate.cuda(), up.cuda(), rows, 64, ld, out, values, swiglu_limit=2.0)
    k = host(out)[rows * 32:rows * 34].reshape(rows, 2)
    bad = np.zeros((rows, 2), bool)
    bad[[0, 1, 2, 3, 7], [0, 1, 0, 1, 1]] = True
    assert np.array_equal(k == 255, bad)
    v = values.double().cpu().numpy()
    assert np.array_equal(np.isnan(v), np.repeat(bad, 32, axis=1))
    assert not host(out)[:rows * 32].reshape(rows, 2, 16)[bad].any()   # codes of a NaN group: 0
    # silu(2) and silu(1) * 2 lie in [1, 2): scale 2^-2, so they are 1.7616 / 0.25 -> 6 and 1.4621 / 0.25 -> 6
    assert v[4, 0] == 1.5 and v[5, 0] == 1.5 and v[6, 0] == -1.5


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ld", [64, 69])
@pytest.mark.parametrize("gate,up", [(300.0, 300.0), (2000.0, -4000.0), (0.01, 2.0**-14), (2.0**-12, 2.0**-12), (300.0, 218.5)])
def test_swiglu_values_beyond_halves(mx, dtype, ld, gate, up):
    """The values are the codes' values rounded once to the type: exact in float and bfloat16,
    infinite, subnormal or zero in half where its range ends.  (The codes themselves: above.)"""
    g = torch.Generator().manual_seed(6)
    gt, u = (v * (1 - torch.rand(7, ld, generator=g) / 2) for v in (gate, up))
    out = torch.zeros(ref.nbytes(7, 64), dtype=torch.uint8, device="cuda:0")
    values = torch.zeros(7, 64, dtype=dtype, device="cuda:0")
    mx.mxfp4_swiglu_quant(gt.to(dtype).cuda(), u.to(dtype).cuda(), 7, 64, ld, out, values)
    o = host(out)
    byte = o[:7 * 32].reshape(7, 32)
    code = np.empty((7, 64), np.uint8)
    code[:, 0::2], code[:, 1::2] = byte & 15, byte >> 4
    exact = ref.values(code, o[7 * 32:7 * 34].reshape(7, 2))
    assert np.isfinite(exact).all() and exact.any()
    want = torch.from_numpy(exact).to(dtype)          # one rounding of an E2M1 value times a power of two
    assert torch.equal(values.cpu(), want)
    if dtype is not torch.float16:
        assert np.array_equal(want.double().numpy(), exact)
    elif gate == 300.0 and up == 300.0:
        assert torch.isinf(want).any()
