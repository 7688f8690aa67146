"""include/f8.h without a GPU: the refusals of every entry point and of the binding (nothing is
launched), the sources' loads, and the reference's own pins."""
import numpy as np
import pytest

import f8_ref as ref
from test_dependent_launch_cpu import NON_COHERENT, code

A = 1 << 20      # an aligned fake address; never dereferenced
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def mx():
    import __graft_entry__
    __graft_entry__.build()
    import mxfp4_dequant_matmul_gb300 as m
    m.lib()
    return m


def refused(f, ok, bad_args, bad_ptrs):
    """Each of bad_args, put into the arguments ok, gives status 1, each of bad_ptrs 2."""
    names = list(ok)
    for status, cases in ((1, bad_args), (2, bad_ptrs)):
        for kw in cases:
            assert set(kw) <= set(names), kw
            a = {**ok, **kw}
            assert f(*(a[n] for n in names), None) == status, kw


def test_quant(mx):
    refused(mx.lib().mxfp4_f8_quant,
            dict(x=A, type=BF16, x_rows=8, cols=48, ld=48, row_of=None, rows=8, codes=A, scales=A, values=None),
            [dict(type=3), dict(type=-1), dict(cols=40), dict(cols=0), dict(cols=8), dict(rows=0), dict(rows=9), dict(x_rows=0),
             dict(ld=47), dict(ld=1 << 41), dict(rows=1 << 24, x_rows=1 << 24, cols=1 << 21, ld=1 << 21)],
            [dict(x=None), dict(x=A + 1), dict(type=F32, x=A + 2), dict(codes=None), dict(codes=A + 8), dict(scales=None),
             dict(scales=A + 2), dict(row_of=A + 2), dict(values=A + 8)])


def test_quant_weight(mx):
    refused(mx.lib().mxfp4_f8_quant_weight,
            dict(w=A, type=F16, n=2, rows=5, cols=48, codes=A, scales=A, values=None),
            [dict(type=3), dict(n=0), dict(n=1025), dict(rows=0), dict(cols=24), dict(n=1024, rows=1 << 20, cols=1 << 16)],
            [dict(w=None), dict(w=A + 8), dict(codes=A + 4), dict(scales=None), dict(scales=A + 1), dict(values=A + 2)])


@pytest.mark.parametrize("grad", [False, True])
def test_product(mx, grad):
    f = mx.lib().mxfp4_f8_mm_grad if grad else mx.lib().mxfp4_f8_mm
    ok = dict(w=A, ws=A, rows=32, cols=48, x=A, xs=A, nb=3, y=A, type=F32)
    bad = [dict(rows=0), dict(cols=40), dict(cols=0), dict(nb=0), dict(nb=(1 << 24) + 1), dict(type=F16), dict(type=7),
           dict(rows=(1 << 24) + 16), dict(rows=1 << 24, cols=1 << 24), dict(rows=1 << 23, nb=1 << 22)]
    if grad:
        bad += [dict(rows=40), dict(rows=8)]     # a row of dY is a row of codes
    refused(f, ok, bad, [dict(w=None), dict(w=A + 8), dict(ws=None), dict(ws=A + 2), dict(x=A + 4), dict(xs=A + 1), dict(y=A + 8), dict(y=None)])


@pytest.mark.parametrize("grad", [False, True])
def test_experts(mx, grad):
    f = mx.lib().mxfp4_f8_moe_mm_grad if grad else mx.lib().mxfp4_f8_moe_mm
    refused(f, dict(w=A, ws=A, n=4, rows=32, cols=48, x=A, xs=A, n_rows=3, off=A, y=A, type=BF16),
            [dict(n=0), dict(n=1025), dict(rows=0), dict(cols=40), dict(n_rows=0), dict(type=F16), dict(n=1024, rows=1 << 20, cols=1 << 16)],
            [dict(w=A + 1), dict(ws=A + 1), dict(x=None), dict(xs=None), dict(off=None), dict(off=A + 2), dict(y=A + 4)])


def test_grad_w(mx):
    L = mx.lib()
    bad = [dict(type=F32), dict(type=5), dict(rows=12), dict(rows=0), dict(cols=4), dict(cols=20), dict(n_rows=0), dict(out=F16),
           dict(rows=(1 << 24) + 8), dict(n_rows=1 << 24, rows=1 << 21)]
    ptr = [dict(dy=None), dict(dy=A + 8), dict(x=A + 2), dict(dw=A + 8), dict(dw=None)]
    refused(L.mxfp4_mm_grad_w, dict(dy=A, x=A, type=BF16, rows=16, cols=24, n_rows=5, dw=A, out=F32), bad, ptr)
    refused(L.mxfp4_moe_mm_grad_w, dict(dy=A, x=A, type=F16, n=3, rows=16, cols=24, n_rows=5, off=A, dw=A, out=BF16),
            bad + [dict(n=0), dict(n=1025)], ptr + [dict(off=None), dict(off=A + 1)])


def test_the_binding_refuses_tensors_the_kernels_would_misread(mx):
    """Host tensors, and on any device other dtypes; addresses pass to the library's own checks."""
    torch = pytest.importorskip("torch")
    code8, s = torch.zeros(4, 48, dtype=torch.uint8), torch.zeros(1, 4)
    x, y, off = torch.zeros(4, 48), torch.zeros(4, 32), torch.zeros(3, dtype=torch.int32)
    h = torch.zeros(4, 48, dtype=torch.bfloat16)
    calls = [lambda: mx.mxfp4_f8_quant(x, 4, 48, 48, None, 4, code8, s), lambda: mx.mxfp4_f8_quant(A, 4, 48, 48, None, 4, code8, A, type=F32),
             lambda: mx.mxfp4_f8_quant(x, 4, 48, 48, None, 4, A, A),
             lambda: mx.mxfp4_f8_quant_weight(x, 1, 4, 48, code8, s), lambda: mx.mxfp4_f8_mm(code8, s, 4, 48, A, A, 4, A, y_type=F32),
             lambda: mx.mxfp4_f8_mm(A, A, 4, 48, A, A, 4, y), lambda: mx.mxfp4_f8_mm_grad(A, A, 32, 48, code8, s, 4, A, dx_type=F32),
             lambda: mx.mxfp4_f8_moe_mm(A, A, 2, 32, 48, A, A, 4, off, A, y_type=F32),
             lambda: mx.mxfp4_f8_moe_mm_grad(A, A, 2, 32, 48, A, A, 4, off, A, dx_type=F32),
             lambda: mx.mxfp4_mm_grad_w(h, h, 48, 48, 4, A, dw_type=F32), lambda: mx.mxfp4_moe_mm_grad_w(A, A, 2, 48, 48, 4, off, A, type=BF16, dw_type=F32)]
    for i, call in enumerate(calls):
        with pytest.raises(mx.Mxfp4Error) as e:
            call()
        assert e.value.status == 1, i


@pytest.mark.parametrize("name", ["f8_quant.cu", "f8_mm.cu", "grad_w.cu", "tc5.cuh"])
def test_no_non_coherent_loads(name):
    assert not NON_COHERENT.findall(code(name))


def test_reference_grid():
    """Pins of the 8-bit grid: largest value, smallest steps, ties to even, and what torch rounds to."""
    assert ref.VALUE[126] == 448 and ref.VALUE[1] == 2.0 ** -9 and ref.VALUE[8] == 2.0 ** -6 and np.isnan(ref.VALUE[127])
    assert list(ref.encode(np.array([0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0, -448.0]))) == [0, 128, 0, 2, 88, 90, 254]
    torch = pytest.importorskip("torch")
    x = np.random.default_rng(0).uniform(-448, 448, 4000).astype(np.float32)
    x = np.concatenate((x, x * 1e-4, ref._MID.astype(np.float32)))
    assert np.array_equal(ref.encode(x.astype(np.float64)), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_reference_scale():
    assert ref.scale(448.0) == 1.0 and ref.scale(448.5) == 2.0 and ref.scale(224.0) == 0.5 and ref.scale(224.1) == 1.0
    assert ref.scale(0.0) == 2.0 ** -126 and ref.scale(1e-45) == 2.0 ** -126 and np.isnan(ref.scale(np.inf))
