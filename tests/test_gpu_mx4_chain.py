"""The 4-bit and routing calls back to back, without a synchronisation, on buffers that every
step writes again with other contents: several of the launches may be resident at once, and each
must see what the one ahead of it wrote.  Against the same calls one at a time on fresh buffers
(tested against 64 bits elsewhere), bit for bit."""
import numpy as np
import pytest

import mx4_ref as ref
from gpu_util import cuda, to_dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
STEPS = 6


@pytest.fixture(scope="module")
def mx():
    return cuda()


class Layer:
    """Sort, dispatch, quantise, experts' product, combine and both gradients."""

    def __init__(self, mx, tokens, top_k, n, width, rows, dtype):
        self.mx, self.shape, self.dtype = mx, (tokens, top_k, n, width, rows), dtype
        rng = np.random.default_rng(tokens + width)
        bank = np.concatenate([ref.pack(*ref.random_matrix(rng, rows, width)) for _ in range(n)])
        self.bank = to_dev(bank)
        g = torch.Generator(device="cuda").manual_seed(tokens + width)
        new = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        # every step's inputs, in memory of their own
        self.ids = [torch.rand(tokens, n, generator=g, device="cuda").topk(top_k).indices.int() for _ in range(STEPS)]
        for ids in self.ids:
            ids[torch.rand(tokens, top_k, generator=g, device="cuda") < 0.1] = -1
        self.x = [new(tokens, width).to(dtype) for _ in range(STEPS)]
        self.w = [torch.softmax(new(tokens, top_k), -1) for _ in range(STEPS)]

    def buffers(self):
        tokens, top_k, n, width, rows = self.shape
        p, i32 = tokens * top_k, dict(dtype=torch.int32, device="cuda")
        d = dict(dtype=self.dtype, device="cuda")
        return dict(token_at=torch.full((p,), -1, **i32), pos_of=torch.full((p,), -1, **i32),
                    offsets=torch.zeros(n + 1, **i32), xs=torch.zeros(p, width, **d),
                    xq=torch.zeros(ref.nbytes(p, width), dtype=torch.uint8, device="cuda"), d_o=torch.zeros(p, width, **d))

    def outputs(self):
        tokens, top_k, n, width, rows = self.shape
        d = dict(dtype=self.dtype, device="cuda")
        return dict(mm=torch.zeros(tokens * top_k, rows, device="cuda"), y=torch.zeros(tokens, width, **d),
                    dx=torch.zeros(tokens, width, **d), d_w=torch.zeros(tokens, top_k, device="cuda"))

    def step(self, i, b, o):
        mx, (tokens, top_k, n, width, rows) = self.mx, self.shape
        p = tokens * top_k
        mx.mxfp4_moe_sort(self.ids[i], tokens, top_k, n, b["token_at"], b["pos_of"], b["offsets"])
        mx.mxfp4_moe_dispatch(self.x[i], tokens, top_k, width, b["token_at"], b["xs"])
        mx.mxfp4_quant(self.x[i], tokens, width, width, b["token_at"], p, b["xq"])
        mx.mxfp4_moe_mm_mx(self.bank, n, rows, width, b["xq"], p, b["offsets"], o["mm"])
        mx.mxfp4_moe_combine(b["xs"], tokens, top_k, width, b["pos_of"], self.w[i], o["y"])
        mx.mxfp4_moe_combine_grad(self.x[i], b["xs"], tokens, top_k, width, b["pos_of"], self.w[i], b["d_o"], o["d_w"])
        mx.mxfp4_moe_dispatch_grad(b["d_o"], tokens, top_k, width, b["pos_of"], o["dx"])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,top_k,n,width,rows", [(1, 4, 8, 2880, 288), (32, 4, 64, 2880, 160), (700, 3, 23, 1056, 130)])
@pytest.mark.parametrize("form", ["stream", "graph"])
def test_steps_on_the_same_buffers(mx, form, tokens, top_k, n, width, rows, dtype):
    layer = Layer(mx, tokens, top_k, n, width, rows, dtype)
    want = []
    for i in range(STEPS):
        b, o = layer.buffers(), layer.outputs()
        layer.step(i, b, o)
        torch.cuda.synchronize()
        want.append(o)
    b, got = layer.buffers(), [layer.outputs() for _ in range(STEPS)]
    torch.cuda.synchronize()
    if form == "stream":
        for i in range(STEPS):
            layer.step(i, b, got[i])
    else:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for i in range(STEPS):
                layer.step(i, b, got[i])
        for o in got:
            for t in o.values():
                t.fill_(55.0)
        for i in range(STEPS):           # rows past the kept pairs stay untouched
            got[i]["mm"].zero_()
        for _ in range(3):
            graph.replay()
    torch.cuda.synchronize()
    for i in range(STEPS):
        for k in want[i]:
            assert torch.equal(got[i][k], want[i][k]), (i, k)
    assert not torch.equal(want[0]["y"], want[1]["y"])
