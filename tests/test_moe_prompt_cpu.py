"""What the example's routed layer refuses, without a GPU: nothing below gets as far as a launch."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import moe_prompt
    return moe_prompt


def test_buffers_that_the_products_cannot_write(moe):
    for dtype in (torch.float16, torch.float64, torch.int8):
        with pytest.raises(ValueError):
            moe.MoePrompt(None, None, None, 4, 64, 32, 2, 8, dtype=dtype)


def test_arguments_of_other_shapes_and_strides(moe):
    layer = object.__new__(moe.MoePrompt)
    layer.max_tokens, layer.hidden, layer.inter, layer.top_k, layer.n_experts = 8, 64, 32, 2, 4
    layer.token_at = layer.pos_of = layer.offsets = None       # (the library would refuse these)
    ok = dict(x=torch.zeros(5, 64), expert_ids=torch.zeros(5, 2, dtype=torch.int32), route_w=torch.zeros(5, 2),
              y=torch.zeros(5, 64))
    for name, bad in (("x", torch.zeros(9, 64)), ("x", torch.zeros(5, 63)), ("x", torch.zeros(5, 128)[:, ::2]),
                      ("x", torch.zeros(64, 5).T), ("expert_ids", torch.zeros(5, 3, dtype=torch.int32)),
                      ("expert_ids", torch.zeros(4, 2, dtype=torch.int32)), ("route_w", torch.zeros(2, 5).T),
                      ("route_w", torch.zeros(10)), ("y", torch.zeros(4, 64)), ("y", torch.zeros(5, 65)[:, :64])):
        with pytest.raises(ValueError):
            layer(**{**ok, name: bad})
