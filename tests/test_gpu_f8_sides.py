"""8-bit quantisers on one row as long as an int holds: every code and scale of it, a pattern repeated
over the row (its last block holds 112 elements)."""
import numpy as np
import pytest

import f8_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
COLS, PERIOD = (1 << 31) - 16, 1 << 20


@pytest.fixture(scope="module")
def mx():
    from gpu_util import cuda
    return cuda()


@pytest.mark.parametrize("weight", [False, True])
def test_the_longest_row(mx, weight):
    rng = np.random.default_rng(31)
    base = (rng.standard_normal((PERIOD // 128, 128)) * np.exp2(rng.integers(-12, 6, (PERIOD // 128, 1)))).astype(np.float16)
    codes, s = ref.quantise_rows(base.astype(np.float64))     # a block a row
    x = torch.from_numpy(base).cuda().reshape(1, -1).expand(2048, -1).reshape(-1)[:COLS]
    out = torch.full((COLS + 16,), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((ref.blocks(COLS) + 1,), -1.0, device="cuda")
    if weight:
        mx.mxfp4_f8_quant_weight(x, 1, 1, COLS, out, scales)
    else:
        mx.mxfp4_f8_quant(x, 1, COLS, COLS, None, 1, out, scales)
    want = torch.from_numpy(codes.reshape(-1)).cuda()
    want_s = torch.from_numpy(np.float32(s.reshape(-1))).cuda()
    for i in range(0, COLS, PERIOD):
        n = min(PERIOD, COLS - i)
        assert torch.equal(out[i:i + n], want[:n]), i
    tail = np.float64(base.reshape(-1)[PERIOD - 128:PERIOD - 16])        # of the last block, cut off
    last = ref.scale(np.abs(tail).max())
    assert last == want_s[-1].item()      # (its largest is among what is left)
    assert torch.equal(scales[:-1], want_s.repeat(2048))
    assert (out[COLS:] == 0x55).all() and scales[-1] == -1.0
