"""Matvecs with launch overlap whose outputs and inputs alternate between two buffers: a launch
may be resident while the one two ahead still reads the buffer that the one ahead will write."""
import numpy as np
import pytest

import synth
from gpu_util import assert_bits_equal, cuda, host, to_dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    return cuda()


@pytest.mark.parametrize("n,nb", [(256, 1), (1024, 1), (1024, 2), (4096, 1)])
def test_two_buffers(mx, n, nb):
    # scale bytes that keep the values' size about the same from step to step
    ws = [to_dev(synth.mxfp4_matrix(n, n, 940 + i, 118, 122)) for i in range(4)]
    x0 = to_dev(synth.normal_f32(950, nb * n))
    steps = 12

    def chain(wait):
        bufs = [x0.clone(), torch.zeros_like(x0)]
        torch.cuda.synchronize()
        for i in range(steps):
            x, y = bufs[i % 2], bufs[(i + 1) % 2]
            if nb == 1:
                mx.mxfp4_mv(ws[i % 4], n, n, x, y)
            else:
                mx.mxfp4_mm(ws[i % 4], n, n, x, nb, y)
            if wait:
                torch.cuda.synchronize()
        return [host(b) for b in bufs]

    want = chain(True)
    assert all(np.isfinite(b).all() and (np.abs(b) > 1e-6).mean() > 0.9 for b in want)
    mx.mxfp4_set_launch_overlap(True)
    try:
        got = [chain(False) for _ in range(4)]
    finally:
        mx.mxfp4_set_launch_overlap(False)
    for g in got:
        for a, b in zip(g, want):
            assert_bits_equal(a, b, f"{n}x{n}, {nb} tokens")
