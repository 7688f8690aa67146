"""The product of a long prompt over a long sum (pairs of CTAs, 112 blocks): bit for bit the same each
time, its bfloat16 result the FP32 one rounded once, both within the stated bound of 64 bits."""
import pytest

import f8_ref as ref
from test_gpu_f8 import check_product
from test_gpu_f8_use import decoded, make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    from gpu_util import cuda
    return cuda()


@pytest.mark.parametrize("grad", [False, True])
def test_a_long_prompt_repeats(mx, grad):
    k, n_out, nb = 14336, 4096, 2048
    rows, cols = (k, n_out) if grad else (n_out, k)
    g = torch.Generator(device="cuda").manual_seed(14336 + grad)
    w, ws = make(g, rows, cols, (ref.blocks(rows), ref.blocks(cols)))
    x, xs = make(g, nb, k, (ref.blocks(k), nb))
    f = mx.mxfp4_f8_mm_grad if grad else mx.mxfp4_f8_mm
    first = [torch.empty(nb, n_out, dtype=t, device="cuda") for t in (torch.float32, torch.bfloat16)]
    for y in first:
        f(w, ws, rows, cols, x, xs, nb, y)
    assert torch.equal(first[1], first[0].bfloat16())
    for _ in range(20):
        for y in first:
            again = torch.full_like(y, 7.0)
            f(w, ws, rows, cols, x, xs, nb, again)
            assert torch.equal(again, y)
    some = torch.arange(0, nb, 37, device="cuda")
    wv, xv = decoded(w, ws, False), decoded(x[some], xs[:, some], True)
    wv = wv if grad else wv.T
    check_product(first[0][some], (xv @ wv).cpu().numpy(), (xv.abs() @ wv.abs()).cpu().numpy(), k, "f32")
