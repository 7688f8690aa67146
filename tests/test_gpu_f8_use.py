"""The 8-bit operators as they are used: a routed layer with all of its gradients, back to back on
buffers that change, captured and replayed, on several streams at once; the shapes that choose
the products' variants; sizes past 32 bits; gradients against differences; NaN where it belongs."""
import numpy as np
import pytest

import f8_ref as ref
from test_gpu_f8 import BF16_HALF, DT, check_grad_w, check_product, dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
STEPS = 5


@pytest.fixture(scope="module")
def mx():
    from gpu_util import cuda
    return cuda()


def bank_of(mx, g, n, rows, cols):
    w = 0.05 * torch.randn(n, rows, cols, generator=g, device="cuda")
    codes = torch.empty(n, rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(n, ref.blocks(rows), ref.blocks(cols), device="cuda")
    mx.mxfp4_f8_quant_weight(w, n, rows, cols, codes, scales)
    return codes, scales


class Layer:
    """Sort, quantise into expert order, the experts' product, combine; then all gradients."""

    def __init__(self, mx, tokens, top_k, n, cols, rows):
        self.mx, self.shape = mx, (tokens, top_k, n, cols, rows)
        g = torch.Generator(device="cuda").manual_seed(tokens + cols)
        self.bank, self.bs = bank_of(mx, g, n, rows, cols)
        self.ids = [torch.rand(tokens, n, generator=g, device="cuda").topk(top_k).indices.int() for _ in range(STEPS)]
        for ids in self.ids:
            ids[torch.rand(tokens, top_k, generator=g, device="cuda") < 0.1] = -1
        self.x = [torch.randn(tokens, cols, generator=g, device="cuda").bfloat16() for _ in range(STEPS)]
        self.dy = [torch.randn(tokens, rows, generator=g, device="cuda").bfloat16() for _ in range(STEPS)]
        self.w = [torch.softmax(torch.randn(tokens, top_k, generator=g, device="cuda"), -1) for _ in range(STEPS)]

    def buffers(self):
        tokens, top_k, n, cols, rows = self.shape
        p, i32, b16 = tokens * top_k, dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.bfloat16, device="cuda")
        f8 = dict(dtype=torch.float8_e4m3fn, device="cuda")
        return dict(token_at=torch.zeros(p, **i32), pos_of=torch.zeros(p, **i32), offsets=torch.zeros(n + 1, **i32),
                    xq=torch.zeros(p, cols, **f8), xs=torch.zeros(ref.blocks(cols), p, device="cuda"), xv=torch.zeros(p, cols, **b16),
                    o=torch.zeros(p, rows, **b16), d_o=torch.zeros(p, rows, **b16), dq=torch.zeros(p, rows, **f8),
                    ds=torch.zeros(ref.blocks(rows), p, device="cuda"), dxs=torch.zeros(p, cols, **b16))

    def outputs(self):
        tokens, top_k, n, cols, rows = self.shape
        return dict(y=torch.zeros(tokens, rows, dtype=torch.bfloat16, device="cuda"), d_w=torch.zeros(tokens, top_k, device="cuda"),
                    dx=torch.zeros(tokens, cols, dtype=torch.bfloat16, device="cuda"), dW=torch.zeros(n, rows, cols, device="cuda"))

    def step(self, i, b, o):
        mx, (tokens, top_k, n, cols, rows) = self.mx, self.shape
        p = tokens * top_k
        mx.mxfp4_moe_sort(self.ids[i], tokens, top_k, n, b["token_at"], b["pos_of"], b["offsets"])
        mx.mxfp4_f8_quant(self.x[i], tokens, cols, cols, b["token_at"], p, b["xq"], b["xs"], b["xv"])
        mx.mxfp4_f8_moe_mm(self.bank, self.bs, n, rows, cols, b["xq"], b["xs"], p, b["offsets"], b["o"])
        mx.mxfp4_moe_combine(b["o"], tokens, top_k, rows, b["pos_of"], self.w[i], o["y"])
        mx.mxfp4_moe_combine_grad(self.dy[i], b["o"], tokens, top_k, rows, b["pos_of"], self.w[i], b["d_o"], o["d_w"])
        mx.mxfp4_f8_quant(b["d_o"], p, rows, rows, None, p, b["dq"], b["ds"])
        mx.mxfp4_f8_moe_mm_grad(self.bank, self.bs, n, rows, cols, b["dq"], b["ds"], p, b["offsets"], b["dxs"])
        mx.mxfp4_moe_mm_grad_w(b["d_o"], b["xv"], n, rows, cols, p, b["offsets"], o["dW"])
        mx.mxfp4_moe_dispatch_grad(b["dxs"], tokens, top_k, cols, b["pos_of"], o["dx"])

    def fresh(self, i):
        b, o = self.buffers(), self.outputs()
        self.step(i, b, o)
        torch.cuda.synchronize()
        return b, o


LAYERS = [(1, 4, 8, 2880, 288), (32, 4, 16, 400, 160), (300, 3, 5, 1056, 144)]


@pytest.mark.parametrize("tokens,top_k,n,cols,rows", LAYERS)
def test_layer_and_its_gradients(mx, tokens, top_k, n, cols, rows):
    """One step against 64 bits, the roundings between the calls taken over from its buffers."""
    layer = Layer(mx, tokens, top_k, n, cols, rows)
    b, o = layer.fresh(0)
    ids, off = layer.ids[0].cpu().numpy().reshape(-1), b["offsets"].cpu().numpy()
    order = sorted((p for p in range(ids.size) if ids[p] >= 0), key=lambda p: (ids[p], p))
    m = off[-1]
    assert m == len(order)
    h = lambda t: t.double().cpu().numpy()                                    # noqa: E731
    u8 = lambda t: t.view(torch.uint8).cpu().numpy()                          # noqa: E731
    x, w, dy = h(layer.x[0]), h(layer.w[0]).reshape(-1), h(layer.dy[0])
    codes, s = ref.quantise_rows(x[np.array(order, int) // top_k].reshape(m, cols))
    assert np.array_equal(u8(b["xq"])[:m], codes) and np.array_equal(b["xs"].cpu().numpy()[:, :m], np.float32(s))
    y, l1 = ref.product(u8(layer.bank), h(layer.bs), u8(b["xq"]), b["xs"].cpu().numpy(), off)
    check_product(b["o"][:m], y[:m], l1[:m], cols, "bf16")
    dx, l1 = ref.product(u8(layer.bank), h(layer.bs), u8(b["dq"]), b["ds"].cpu().numpy(), off, grad=True)
    check_product(b["dxs"][:m], dx[:m], l1[:m], rows, "bf16")
    dw, l1 = ref.grad_w(h(b["d_o"]), h(b["xv"]), off)
    check_grad_w(o["dW"], dw, l1, np.diff(off), "f32")
    # the ends: combine and its gradient, and the rows' gradients gathered (sums of bf16 values)
    want_y, want_dx = np.zeros((tokens, rows)), np.zeros((tokens, cols))
    do = h(b["d_o"])
    for i, p in enumerate(order):
        want_y[p // top_k] += w[p] * h(b["o"])[i]
        want_dx[p // top_k] += h(b["dxs"])[i]
        assert np.abs(do[i] - w[p] * dy[p // top_k]).max() <= (BF16_HALF + 2.0 ** -23) * np.abs(w[p] * dy[p // top_k]).max()
    # FP32 sums of top_k terms, rounded to bfloat16: each term within 1, far above top_k * 2^-24 of it
    for got, want in ((o["y"], want_y), (o["dx"], want_dx)):
        assert np.abs(h(got) - want).max() <= BF16_HALF * np.abs(want).max() + 1e-5 * (1 + np.abs(want).max())


@pytest.mark.parametrize("form", ["stream", "graph", "streams"])
@pytest.mark.parametrize("tokens,top_k,n,cols,rows", LAYERS)
def test_steps_on_the_same_buffers(mx, form, tokens, top_k, n, cols, rows):
    """Launches that are resident together, replays of a graph, and steps on streams of their own at
    the same time: bit for bit what the same calls give one at a time."""
    layer = Layer(mx, tokens, top_k, n, cols, rows)
    want = [layer.fresh(i)[1] for i in range(STEPS)]
    b, got = layer.buffers(), [layer.outputs() for _ in range(STEPS)]
    torch.cuda.synchronize()
    if form == "stream":
        for i in range(STEPS):
            layer.step(i, b, got[i])
    elif form == "graph":
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for i in range(STEPS):
                layer.step(i, b, got[i])
        for o in got:
            for t in o.values():
                t.fill_(55.0)
        for _ in range(3):
            graph.replay()
    else:
        streams = [torch.cuda.Stream() for _ in range(STEPS)]
        own = [layer.buffers() for _ in range(STEPS)]
        torch.cuda.synchronize()
        for _ in range(3):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    layer.step(i, own[i], got[i])
    torch.cuda.synchronize()
    for i in range(STEPS):
        for k in want[i]:
            assert torch.equal(got[i][k], want[i][k]), (i, k)


# --- variants ----------------------------------------------------------------------------


def decoded(codes, s, rows):
    """Values in 64 bits on the GPU: rows of activations or a matrix."""
    v = codes.double()
    if rows:
        return v * s.double().T.repeat_interleave(128, 1)[:, :v.shape[1]]
    return v * s.double().repeat_interleave(128, 0)[:v.shape[0]].repeat_interleave(128, 1)[:, :v.shape[1]]


def make(g, rows, cols, scale_shape):
    c = torch.randint(0, 254, (rows, cols), generator=g, device="cuda", dtype=torch.int32)
    c = torch.where(c >= 127, c + 1, c).to(torch.uint8).view(torch.float8_e4m3fn)
    return c, torch.exp2(torch.rand(scale_shape, generator=g, device="cuda") * 4 - 9)


# tokens: not split, split over 2, 4 and 8 CTAs, tiles of 16, 32, 64 and 128 tokens, of 128 x 256;
# outputs that are 32-byte aligned and not, more tiles than SMs, a last tile of one row or column
VARIANTS = [(14336, 512, 1), (9728, 256, 9), (16385, 144, 30), (9729, 400, 50), (4096, 2048, 16), (2049, 4096, 17), (2000, 1536, 60),
            (1025, 2064, 100), (4100, 1040, 127), (12800, 272, 128), (12801, 272, 100), (640, 1024, 700), (643, 1040, 1025), (8200, 400, 900),
            (16, 14336, 130), (4097, 256, 2049)]


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("rows,cols,nb", VARIANTS)
def test_shapes_that_choose_the_variants(mx, rows, cols, nb, grad):
    g = torch.Generator(device="cuda").manual_seed(rows + cols + nb)
    if grad:
        rows, cols = cols, (rows + 15) // 16 * 16   # the same outputs and terms
    k, n_out = (rows, cols) if grad else (cols, rows)
    w, ws = make(g, rows, cols, (ref.blocks(rows), ref.blocks(cols)))
    x, xs = make(g, nb, k, (ref.blocks(k), nb))
    wv, xv = decoded(w, ws, False), decoded(x, xs, True)
    y = xv @ wv if grad else xv @ wv.T
    l1 = xv.abs() @ wv.abs() if grad else xv.abs() @ wv.abs().T
    f = mx.mxfp4_f8_mm_grad if grad else mx.mxfp4_f8_mm
    for t in ("f32", "bf16"):
        out = torch.full((nb + 1, n_out), 7.0, dtype=DT[t], device="cuda")
        f(w, ws, rows, cols, x, xs, nb, out[:nb])
        check_product(out[:nb], y.cpu().numpy(), l1.cpu().numpy(), k, t)
        assert (out[nb] == 7.0).all()
        again = torch.empty_like(out)
        f(w, ws, rows, cols, x, xs, nb, again[:nb])
        assert torch.equal(again[:nb], out[:nb])


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("n,rows,cols,mean", [(1024, 2048, 16, 1), (512, 1040, 144, 20), (300, 1296, 32, 40), (40, 2320, 272, 60),
                                              (200, 1552, 16, 70), (7, 272, 528, 300)])
def test_many_tiles_a_block(mx, n, rows, cols, mean, grad):
    """More tiles than a CTA lists at its start, in every width."""
    if grad:
        rows, cols = cols, rows
    k, n_out = (rows, cols) if grad else (cols, rows)
    g = torch.Generator(device="cuda").manual_seed(n + rows)
    rng = np.random.default_rng(n)
    counts = rng.integers(0, 2 * mean + 1, n)
    counts[-1] += n * mean - counts.sum() if counts.sum() < n * mean else 0
    off = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    n_rows = int(off[-1])
    w, ws = make(g, n * rows, cols, (n, ref.blocks(rows), ref.blocks(cols)))
    w = w.reshape(n, rows, cols)
    x, xs = make(g, n_rows, k, (ref.blocks(k), n_rows))
    xv = decoded(x, xs, True)
    y, l1 = (torch.empty(n_rows, n_out, dtype=torch.float64, device="cuda") for _ in range(2))
    for e in range(n):
        wv = decoded(w[e], ws[e], False)
        wv = wv if grad else wv.T
        i, j = off[e], off[e + 1]
        y[i:j], l1[i:j] = xv[i:j] @ wv, xv[i:j].abs() @ wv.abs()
    out = torch.empty(n_rows, n_out, device="cuda")
    f = mx.mxfp4_f8_moe_mm_grad if grad else mx.mxfp4_f8_moe_mm
    f(w, ws, n, rows, cols, x, xs, n_rows, dev(off), out)
    check_product(out, y.cpu().numpy(), l1.cpu().numpy(), k, "f32")


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("rows,cols,counts", [(520, 776, [1000, 0, 3, 257, 256, 64]), (2056, 264, [513, 5000]), (24, 2040, [17] * 40),
                                              (264, 136, [5001]), (256, 256, [2100, 3]), (248, 520, [0, 4099, 2, 4000]), (8, 8, [8192])])
def test_grad_w_of_long_sums_and_many_tiles(mx, rows, cols, counts, t):
    off = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    g = torch.Generator(device="cuda").manual_seed(rows)
    dy = torch.randn(int(off[-1]), rows, generator=g, device="cuda").to(DT[t])
    x = torch.randn(int(off[-1]), cols, generator=g, device="cuda").to(DT[t])
    n = len(counts)
    dw, l1 = (torch.zeros(n, rows, cols, dtype=torch.float64, device="cuda") for _ in range(2))
    for e in range(n):
        i, j = off[e], off[e + 1]
        dw[e], l1[e] = dy[i:j].double().T @ x[i:j].double(), dy[i:j].double().abs().T @ x[i:j].double().abs()
    for out_t in ("f32", "bf16"):
        out = torch.empty(n, rows, cols, dtype=DT[out_t], device="cuda")
        mx.mxfp4_moe_mm_grad_w(dy, x, n, rows, cols, int(off[-1]), dev(off), out)
        check_grad_w(out, dw.cpu().numpy(), l1.cpu().numpy(), counts, out_t)
        again = torch.empty_like(out)
        mx.mxfp4_moe_mm_grad_w(dy, x, n, rows, cols, int(off[-1]), dev(off), again)
        assert torch.equal(again, out)


# --- offsets, NaN, addresses -----------------------------------------------------------------


def test_offsets_past_the_rows_and_experts_without_any(mx):
    """Offsets beyond n_rows are cut off there; with no rows at all nothing is written (dW: zeros)."""
    rng = np.random.default_rng(1)
    n, rows, cols, n_rows = 4, 144, 272, 50
    bank, bs = ref.random_codes(rng, (n, rows, cols)), ref.random_scales(rng, (n, 2, 3))
    x, xs = ref.random_codes(rng, (n_rows, cols)), ref.random_scales(rng, (3, n_rows))
    cut = np.array([0, 0, 20, 50, 50], np.int32)
    y, l1 = ref.product(bank, bs, x, xs, cut)
    out = torch.empty(n_rows, rows, device="cuda")
    mx.mxfp4_f8_moe_mm(dev(bank), dev(bs), n, rows, cols, dev(x), dev(xs), n_rows, dev(np.array([0, 0, 20, 90, 4000], np.int32)), out)
    check_product(out, y, l1, cols, "f32")
    none = dev(np.zeros(n + 1, np.int32))
    out.fill_(7.0)
    mx.mxfp4_f8_moe_mm(dev(bank), dev(bs), n, rows, cols, dev(x), dev(xs), n_rows, none, out)
    assert (out == 7.0).all()
    big = torch.full((600, rows), 7.0, device="cuda")          # 150 rows an expert: the other kernel
    x, xs = ref.random_codes(rng, (600, cols)), ref.random_scales(rng, (3, 600))
    mx.mxfp4_f8_moe_mm(dev(bank), dev(bs), n, rows, cols, dev(x), dev(xs), 600, none, big)
    assert (big == 7.0).all()
    dw = torch.full((n, rows, cols), 7.0, device="cuda")
    h = torch.randn(n_rows, 272, device="cuda").bfloat16()
    mx.mxfp4_moe_mm_grad_w(h[:, :rows].contiguous(), h, n, rows, cols, n_rows, none, dw)
    assert (dw == 0.0).all()


@pytest.mark.parametrize("nb", [3, 40, 300])
def test_nan_stays_with_its_block(mx, nb):
    """A NaN scale or code of a token makes that token NaN; of the matrix, the outputs of its block or row."""
    rng = np.random.default_rng(nb)
    rows, cols = 300, 400
    w, ws = ref.random_codes(rng, (1, rows, cols)), ref.random_scales(rng, (1, 3, 4))
    x, xs = ref.random_codes(rng, (nb, cols)), ref.random_scales(rng, (4, nb))
    xs[3, 1], x[2, 7], ws[0, 1, 2], w[0, 290, 5] = np.nan, 255, np.nan, 127
    y, l1 = ref.product(w, ws, x, xs)
    out = torch.empty(nb, rows, device="cuda")
    mx.mxfp4_f8_mm(dev(w), dev(ws), rows, cols, dev(x), dev(xs), nb, out)
    bad = np.isnan(y)
    assert np.array_equal(torch.isnan(out).cpu().numpy(), bad)
    assert bad[1].all() and bad[2].all() and bad[0, 128:256].all() and bad[0, 290] and not bad[0, :128].any()
    out[torch.isnan(out)] = 0.0
    check_product(out, np.where(bad, 0.0, y), np.where(bad, 0.0, l1), cols, "f32")
    dq, dsc = ref.random_codes(rng, (nb, 304)), ref.random_scales(rng, (3, nb))
    w2, ws2 = ref.random_codes(rng, (1, 304, cols)), ref.random_scales(rng, (1, 3, 4))
    ws2[0, 1, 2] = np.nan
    dx, l1 = ref.product(w2, ws2, dq, dsc, grad=True)
    out = torch.empty(nb, cols, device="cuda")
    mx.mxfp4_f8_mm_grad(dev(w2), dev(ws2), 304, cols, dev(dq), dev(dsc), nb, out)
    assert np.array_equal(torch.isnan(out).cpu().numpy(), np.isnan(dx)) and np.isnan(dx[0, 256:384]).all()


def test_tensors_the_kernels_would_misread_are_refused(mx):
    rows, cols, nb = 144, 272, 5
    w, x = (torch.zeros(n, cols, dtype=torch.uint8, device="cuda") for n in (rows, nb))
    ws, xs, y = torch.zeros(2, 3, device="cuda"), torch.zeros(3, nb, device="cuda"), torch.zeros(nb, rows, device="cuda")
    mx.mxfp4_f8_mm(w, ws, rows, cols, x, xs, nb, y)
    for bad in (dict(w=w.bfloat16()), dict(ws=ws.double()), dict(xs=torch.zeros(nb, 3, device="cuda").T), dict(x=x.cpu()), dict(x=x[:4]),
                dict(w=w[:, ::2]), dict(xs=xs[:2]), dict(y=torch.zeros(nb, 2 * rows, device="cuda")[:, :rows]), dict(y=y.half())):
        a = {**dict(w=w, ws=ws, x=x, xs=xs, y=y), **bad}
        with pytest.raises(mx.Mxfp4Error):
            mx.mxfp4_f8_mm(a["w"], a["ws"], rows, cols, a["x"], a["xs"], nb, a["y"])
    h = torch.zeros(nb, cols, device="cuda", dtype=torch.bfloat16)
    for bad in (dict(codes=h), dict(scales=torch.zeros(nb, 3, device="cuda").T), dict(scales=xs.half()), dict(values=torch.zeros(nb, cols, device="cuda")),
                dict(row_of=torch.zeros(nb, dtype=torch.int64, device="cuda")), dict(codes=x[:, :256]), dict(x=h.cpu())):
        a = {**dict(x=h, codes=x, scales=xs, values=None, row_of=None), **bad}
        with pytest.raises(mx.Mxfp4Error):
            mx.mxfp4_f8_quant(a["x"], nb, cols, cols, a["row_of"], nb, a["codes"], a["scales"], a["values"])
    torch.cuda.synchronize()


def test_addresses_past_32_bits(mx):
    """Products, gradients and codes whose element offsets pass 2^31: the last rows are right."""
    g = torch.Generator(device="cuda").manual_seed(9)
    nb, rows, cols = 540000, 4096, 16
    w, ws = make(g, rows, cols, (32, 1))
    x, xs = make(g, nb, cols, (1, nb))
    y = torch.zeros(nb, rows, dtype=torch.bfloat16, device="cuda")
    mx.mxfp4_f8_mm(w, ws, rows, cols, x, xs, nb, y)
    at = torch.tensor([0, 1, 262143, 262144, 524287, 524288, nb - 1], device="cuda")
    xv, wv = decoded(x[at], xs[:, at], True), decoded(w, ws, False)
    check_product(y[at], (xv @ wv.T).cpu().numpy(), (xv.abs() @ wv.abs().T).cpu().numpy(), cols, "bf16")
    # the same rows quantised as they are: 2^31 elements and more in, their codes out
    codes = torch.zeros(nb, rows, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(32, nb, device="cuda")
    mx.mxfp4_f8_quant(y, nb, rows, rows, None, nb, codes, scales)
    c, s = ref.quantise_rows(y[at].double().cpu().numpy())
    assert np.array_equal(codes[at].cpu().numpy(), c) and np.array_equal(scales[:, at].cpu().numpy(), np.float32(s))
    # as the gradient's rows, their sum over 4096 terms
    dx = torch.zeros(nb, cols, device="cuda")
    mx.mxfp4_f8_mm_grad(w, ws, rows, cols, codes, scales, nb, dx)
    dv = decoded(codes[at].view(torch.float8_e4m3fn), scales[:, at], True)
    check_product(dx[at], (dv @ wv).cpu().numpy(), (dv.abs() @ wv.abs()).cpu().numpy(), rows, "f32")
    del codes, scales, dx
    # and in the weights' gradient: one expert's rows lie behind 2^31 elements
    off = torch.tensor([0, 3, nb - 5, nb], dtype=torch.int32, device="cuda")
    xb = torch.randn(nb, cols, generator=g, device="cuda").bfloat16()
    dw = torch.zeros(3, rows, cols, device="cuda")
    mx.mxfp4_moe_mm_grad_w(y, xb, 3, rows, cols, nb, off, dw)
    for e, (i, j) in ((0, (0, 3)), (2, (nb - 5, nb))):
        a, b = y[i:j].double(), xb[i:j].double()
        check_grad_w(dw[e][None], (a.T @ b)[None].cpu().numpy(), (a.abs().T @ b.abs())[None].cpu().numpy(), [j - i], "f32")


def test_a_bank_past_32_bits(mx):
    n, rows, cols = 70, 8192, 4096
    g = torch.Generator(device="cuda").manual_seed(4)
    bank = torch.randint(0, 120, (n, rows, cols), generator=g, device="cuda", dtype=torch.uint8)
    bs = torch.exp2(torch.rand(n, 64, 32, generator=g, device="cuda") - 9)
    n_rows = 140
    x, xs = make(g, n_rows, cols, (32, n_rows))
    off = torch.arange(0, n_rows + 1, 2, dtype=torch.int32, device="cuda")
    y = torch.zeros(n_rows, rows, device="cuda")
    mx.mxfp4_f8_moe_mm(bank, bs, n, rows, cols, x, xs, n_rows, off, y)
    dx = torch.zeros(n_rows, cols, device="cuda")
    dq, ds = make(g, n_rows, rows, (64, n_rows))
    mx.mxfp4_f8_moe_mm_grad(bank, bs, n, rows, cols, dq, ds, n_rows, off, dx)
    for e in (0, 63, 64, 69):
        wv = decoded(bank[e].view(torch.float8_e4m3fn), bs[e], False)
        xv, dv = decoded(x, xs, True)[2 * e: 2 * e + 2], decoded(dq, ds, True)[2 * e: 2 * e + 2]
        check_product(y[2 * e: 2 * e + 2], (xv @ wv.T).cpu().numpy(), (xv.abs() @ wv.abs().T).cpu().numpy(), cols, "f32")
        check_product(dx[2 * e: 2 * e + 2], (dv @ wv).cpu().numpy(), (dv.abs() @ wv.abs()).cpu().numpy(), rows, "f32")
    # dW of as many elements: the last expert's, and zeros where there are no rows
    h, k = torch.randn(6, rows, generator=g, device="cuda").bfloat16(), torch.randn(6, cols, generator=g, device="cuda").bfloat16()
    off = torch.full((n + 1,), 2, dtype=torch.int32, device="cuda")
    off[0], off[n] = 0, 6
    dw = torch.full((n, rows, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    mx.mxfp4_moe_mm_grad_w(h, k, n, rows, cols, 6, off, dw)
    a, b = h[2:].double(), k[2:].double()
    check_grad_w(dw[n - 1][None], (a.T @ b)[None].cpu().numpy(), (a.abs().T @ b.abs())[None].cpu().numpy(), [4], "bf16")
    assert (dw[1:n - 1] == 0).all()


# --- gradients against differences -------------------------------------------------------------


@pytest.mark.parametrize("nb", [4, 200])
def test_gradients_against_differences(mx, nb):
    """The product is linear in either factor: <dY, Y(x1) - Y(x0)> = <dX, x1 - x0> and the same for a
    change of the matrix, up to the stated bounds of the two sides."""
    rng = np.random.default_rng(nb)
    rows, cols = 272, 400
    w, ws = ref.random_codes(rng, (1, rows, cols)), ref.random_scales(rng, (1, 3, 4))
    s = ref.random_scales(rng, (4, nb))
    x0, x1 = (ref.random_codes(rng, (nb, cols)) for _ in range(2))
    dq, ds = ref.random_codes(rng, (nb, rows)), ref.random_scales(rng, (3, nb))
    y, bound = [], 0.0
    dyv = ref.row_values(dq, ds.astype(np.float64))
    for x in (x0, x1):
        out = torch.empty(nb, rows, device="cuda")
        mx.mxfp4_f8_mm(dev(w), dev(ws), rows, cols, dev(x), dev(s), nb, out)
        y.append(out.double().cpu().numpy())
        bound += (np.abs(dyv) * ref.sum_bound(cols, 32, 4) * ref.product(w, ws, x, s)[1]).sum()
    dx = torch.empty(nb, cols, device="cuda")
    mx.mxfp4_f8_mm_grad(dev(w), dev(ws), rows, cols, dev(dq), dev(ds), nb, dx)
    step = ref.row_values(x1, s.astype(np.float64)) - ref.row_values(x0, s.astype(np.float64))
    bound += (np.abs(step) * ref.sum_bound(rows, 32, 3) * ref.product(w, ws, dq, ds, grad=True)[1]).sum()
    got, want = (dx.double().cpu().numpy() * step).sum(), (dyv * (y[1] - y[0])).sum()
    assert abs(got - want) <= bound and abs(want) > 100 * bound
    # by the matrix: values that 16 bits hold, dW against the change of another matrix's product
    w1 = ref.random_codes(rng, (1, rows, cols))
    xv = ref.row_values(x0, np.ones_like(s, dtype=np.float64))
    dyv = ref.row_values(dq, np.ones_like(ds, dtype=np.float64))
    one_w, one_s = np.ones_like(ws), np.ones_like(s)
    z, bound = [], 0.0
    for m in (w, w1):
        out = torch.empty(nb, rows, device="cuda")
        mx.mxfp4_f8_mm(dev(m), dev(one_w), rows, cols, dev(x0), dev(one_s), nb, out)
        z.append(out.double().cpu().numpy())
        bound += (np.abs(dyv) * ref.sum_bound(cols, 32, 4) * ref.product(m, one_w, x0, one_s)[1]).sum()
    dw = torch.empty(rows, cols, device="cuda")
    mx.mxfp4_mm_grad_w(dev(dyv).bfloat16(), dev(xv).bfloat16(), rows, cols, nb, dw)
    step = ref.VALUE[w1[0]] - ref.VALUE[w[0]]
    bound += (np.abs(step) * ref.sum_bound(nb, 16, 0) * ref.grad_w(dyv, xv, [0, nb])[1][0]).sum()
    got, want = (dw.double().cpu().numpy() * step).sum(), (dyv * (z[1] - z[0])).sum()
    assert abs(got - want) <= bound


# --- streams and captures ----------------------------------------------------------------------


def test_a_stream_given_by_the_caller(mx):
    """Calls on a stream of the caller's, while torch's current one does something else."""
    layer = Layer(mx, 32, 4, 16, 400, 160)
    b, want = layer.fresh(1)
    s, xq, xs = torch.cuda.Stream(), torch.zeros_like(b["xq"]), torch.zeros_like(b["xs"])
    o, dW = torch.zeros_like(b["o"]), torch.zeros_like(want["dW"])
    torch.cuda.synchronize()
    mx.mxfp4_f8_quant(layer.x[1], 32, 400, 400, b["token_at"], 128, xq, xs, stream=s)
    mx.mxfp4_f8_moe_mm(layer.bank, layer.bs, 16, 160, 400, xq, xs, 128, b["offsets"], o, stream=s)
    mx.mxfp4_moe_mm_grad_w(b["d_o"], b["xv"], 16, 160, 400, 128, b["offsets"], dW, stream=s.cuda_stream)
    s.synchronize()
    m = int(b["offsets"][-1])
    assert torch.equal(o[:m], b["o"][:m]) and torch.equal(dW, want["dW"])


FIRST_CALL = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import mxfp4_dequant_matmul_gb300 as mx
torch.zeros(1, device="cuda")
g = torch.Generator(device="cuda").manual_seed(1)
code = lambda *s: torch.randint(0, 120, s, generator=g, device="cuda", dtype=torch.uint8)
num = lambda *s: torch.rand(s, generator=g, device="cuda")
new = lambda *s, **k: torch.zeros(s, device="cuda", **k)
off = torch.tensor([0, 3, 700], dtype=torch.int32, device="cuda")
w, ws, x, xs, d, ds = code(2, 1040, 528), num(2, 9, 5), code(700, 528), num(5, 700), code(700, 1040), num(9, 700)
h, k = num(4000, 1040).bfloat16(), num(4000, 528).bfloat16()
def calls():
    out = [new(700, 528, dtype=torch.uint8), new(5, 700), new(2, 1040, 528, dtype=torch.uint8), new(2, 9, 5)]
    mx.mxfp4_f8_quant(k, 700, 528, 528, None, 700, out[0], out[1])
    mx.mxfp4_f8_quant_weight(w.bfloat16(), 2, 1040, 528, out[2], out[3])
    for nb in (1, 100, 700):
        out += [new(nb, 1040), new(nb, 528)]
        mx.mxfp4_f8_mm(w, ws, 1040, 528, x, xs.flatten()[:5 * nb], nb, out[-2])
        mx.mxfp4_f8_mm_grad(w, ws, 1040, 528, d, ds.flatten()[:9 * nb], nb, out[-1])
    out += [new(700, 1040), new(700, 528), new(2, 1040, 528), new(1040, 528)]
    mx.mxfp4_f8_moe_mm(w, ws, 2, 1040, 528, x, xs, 700, off, out[-4])
    mx.mxfp4_f8_moe_mm_grad(w, ws, 2, 1040, 528, d, ds, 700, off, out[-3])
    mx.mxfp4_moe_mm_grad_w(h, k, 2, 1040, 528, 700, off, out[-2])
    mx.mxfp4_mm_grad_w(h, k, 1040, 528, 4000, out[-1])
    return out
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    first = calls()
graph.replay()
torch.cuda.synchronize()
again = calls()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(first, again)) and all(a.float().abs().sum() > 0 for a in first)
assert mx.mxfp4_device_faults() == 0
print("captured")
"""


def test_first_calls_under_capture(mx):
    """Nothing that a first call sets up (attributes, occupancies, modules) stops a capture."""
    import os
    import subprocess
    import sys
    tests = os.path.dirname(os.path.abspath(__file__))
    run = subprocess.run([sys.executable, "-c", FIRST_CALL.format(root=os.path.dirname(tests), tests=tests)],
                         capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "captured" in run.stdout, run.stdout + run.stderr
