"""The routed layer with a SwiGLU limit and NaN weights (scale byte 255): a NaN gate or up is no
larger than any limit, so the tokens whose experts have one are NaN, and only they."""
import numpy as np
import pytest

import oracle
import synth
from gpu_util import assert_within, cuda
from test_gpu_moe_v41 import run_ex

pytestmark = pytest.mark.gpu
V41, F32 = 1, 0


def case(hidden, inter, seed, matrix):
    cfg = synth.MoeConfig("nan", 6, hidden, inter, 10, 2, seed, scale_lo=113, scale_hi=121)
    banks = [b.copy() for b in cfg.banks()]
    # expert 2, one group of one row of its gate (0) or up (1) matrix
    scales = banks[matrix][2 * cfg.gu_stride + hidden * inter // 2:][:hidden * inter // 32]
    scales[5 * (hidden // 32) + 3] = 255
    ids, wts = cfg.routes()
    hit = (ids == 2).any(axis=1)
    assert hit.any() and not hit.all()
    return cfg, banks, cfg.activations(), ids, wts, hit


def expected(cfg, banks, x, ids, wts, mode):
    T, K = ids.shape
    return oracle.moe_forward_ex(*banks, cfg.gu_stride, cfg.down_stride, cfg.n_experts, cfg.hidden,
                                 cfg.inter, x, T, K, ids, wts, bf16_mode=mode == V41, limit=0.5)


@pytest.mark.parametrize("matrix", [0, 1])
@pytest.mark.parametrize("mode", [F32, V41])
@pytest.mark.parametrize("hidden,inter", [(256, 96), (4608, 64)])   # tensor cores; the FP32 passes
def test_layer(hidden, inter, mode, matrix):
    mx = cuda()
    cfg, banks, x, ids, wts, hit = case(hidden, inter, 7, matrix)
    ref = expected(cfg, banks, x, ids, wts, mode)
    y, _, _ = run_ex(mx, cfg, *banks, x, ids, wts, mode, 0.5)
    assert np.array_equal(np.isnan(y), np.repeat(hit[:, None], hidden, axis=1))
    assert_within(y, ref["out"], ref["bound"], 1.0, f"mode {mode} {hidden}x{inter}")
