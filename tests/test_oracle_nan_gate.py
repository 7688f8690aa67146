"""The oracle's routed layer with a SwiGLU limit: a NaN gate or up stays NaN."""
import numpy as np
import pytest

from test_gpu_moe_nan_gate import F32, V41, case, expected


@pytest.mark.parametrize("matrix", [0, 1])
@pytest.mark.parametrize("mode", [F32, V41])
def test_oracle(mode, matrix):
    cfg, banks, x, ids, wts, hit = case(256, 96, 7, matrix)
    out = expected(cfg, banks, x, ids, wts, mode)["out"]
    assert np.array_equal(np.isnan(out), np.repeat(hit[:, None], cfg.hidden, axis=1))
