"""The example's routed layer (4-bit weights and activations): every stage against the 64-bit
reference of that stage on the kernels' own inputs, the layer in a graph and with dropped
pairs, and its distance from the layer with FP32 activations."""
import os
import sys

import numpy as np
import pytest

import mx4_ref as ref
from gpu_util import cuda, host

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

E, HIDDEN, INTER, K = 6, 288, 160, 3


@pytest.fixture(scope="module")
def moe():
    cuda()
    import moe_prompt
    return moe_prompt


def matrix(buf, rows, cols):
    b = host(buf)[:ref.nbytes(rows, cols)]
    byte = b[:rows * cols // 2].reshape(rows, cols // 2)
    code = np.empty((rows, cols), np.uint8)
    code[:, 0::2], code[:, 1::2] = byte & 15, byte >> 4
    return code, b[rows * cols // 2:rows * cols * 17 // 32].reshape(rows, cols // 32)


def setup(moe, tokens, seed=0):
    torch.manual_seed(seed)
    gate, up = (moe.make_bank(E, INTER, HIDDEN, HIDDEN ** -0.5) for _ in range(2))
    down = moe.make_bank(E, HIDDEN, INTER, INTER ** -0.5)
    layer = moe.MoePrompt(gate, up, down, E, HIDDEN, INTER, K, tokens, dtype=torch.float32)
    x = torch.randn(tokens, HIDDEN, device="cuda")
    ids = torch.rand(tokens, E, device="cuda").topk(K).indices.int()
    w = torch.softmax(torch.randn(tokens, K, device="cuda"), -1)
    return layer, x, ids, w


@pytest.mark.parametrize("tokens", [1, 5, 200])
def test_stages_against_64_bits(moe, tokens):
    layer, x, ids, w = setup(moe, tokens)
    ids[0, 1] = -1                                     # a dropped pair
    y = torch.full((tokens, HIDDEN), float("nan"), device="cuda")
    layer(x, ids, w, y)
    token_at, pos_of, off = ref.sort_pairs(ids.cpu().numpy(), K, E)
    assert np.array_equal(host(layer.token_at), token_at) and np.array_equal(host(layer.pos_of), pos_of)
    assert np.array_equal(host(layer.offsets), off)
    pairs, rows = tokens * K, off[-1]
    xs = np.where(token_at[:, None] >= 0, x.double().cpu().numpy()[np.maximum(token_at, 0)], 0.0)
    code, k = matrix(layer.xq, pairs, HIDDEN)
    wc, wk = ref.quantise(xs)
    assert np.array_equal(code, wc) and np.array_equal(k, wk)

    def experts(bank, rows_, cols, xv):
        size, out, l1 = ref.nbytes(rows_, cols), np.zeros((rows, rows_)), np.zeros((rows, rows_))
        for e in range(E):
            wv = ref.values(*matrix(bank[e * size:(e + 1) * size], rows_, cols))
            part = slice(off[e], off[e + 1])
            out[part], l1[part] = xv[part] @ wv.T, np.abs(xv[part]) @ np.abs(wv).T
        return out, l1

    xv = ref.values(code, k)
    for bank, got in ((layer.gate, layer.g), (layer.up, layer.u)):
        want, l1 = experts(bank, INTER, HIDDEN, xv)
        assert (np.abs(got.double().cpu().numpy()[:rows] - want) <= 1e-5 * l1 + 1e-30).all()
    g, u = (t.double().cpu().numpy()[:rows] for t in (layer.g, layer.u))
    act = g / (1 + np.exp(-g)) * u
    ac, ak = matrix(layer.aq, pairs, INTER)
    lo, hi = ref.quantise(act * (1 - 2.0**-20)), ref.quantise(act * (1 + 2.0**-20))
    sure = np.repeat(lo[1] == hi[1], 32, axis=1)
    assert ((ac[:rows] == lo[0]) | (ac[:rows] == hi[0]))[sure].all()
    want, l1 = experts(layer.down, HIDDEN, INTER, ref.values(ac, ak))
    o = layer.o.double().cpu().numpy()[:rows]
    assert (np.abs(o - want) <= 1e-5 * l1 + 1e-30).all()
    kept = pos_of.reshape(tokens, K) >= 0
    terms = np.where(kept[..., None], o[np.maximum(pos_of, 0)].reshape(tokens, K, HIDDEN), 0.0) * \
        w.double().cpu().numpy()[..., None]
    got = y.double().cpu().numpy()
    assert (np.abs(got - terms.sum(1)) <= (K + 1) * 2.0**-24 * np.abs(terms).sum(1) + 1e-30).all()


def test_in_a_graph_and_again(moe):
    layer, x, ids, w = setup(moe, 70)
    y, z = torch.zeros(70, HIDDEN, device="cuda"), torch.zeros(70, HIDDEN, device="cuda")
    layer(x, ids, w, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, ids, w, z)
    for _ in range(3):
        z.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, z)
    with pytest.raises(ValueError):
        layer(torch.zeros(71, HIDDEN, device="cuda"), ids, w, y)


def test_near_the_layer_with_fp32_activations(moe):
    """The layers differ by the two roundings to E2M1.  Half a step is at most 1/4 of a value
    from 2 to 6 (2.5 -> 2 or 3), amax/scale lies in [4, 8) and saturates at most from 8 to 6
    (1/4 again), and values below a quarter of the scale vanish; on normal data the roundings
    come to about an eighth of the norm each.  A layer with one stage wrong (another expert's
    rows, gate and up exchanged) differs by about its norm: a half separates the two."""
    tokens = 48
    layer, x, ids, w = setup(moe, tokens, seed=4)
    y = torch.zeros(tokens, HIDDEN, device="cuda")
    layer(x, ids, w, y)
    mx = moe.mx
    act, want = torch.empty(tokens * K * INTER, device="cuda"), torch.empty(tokens, HIDDEN, device="cuda")
    ws = torch.empty(mx.mxfp4_moe_workspace_bytes(E, tokens, K, HIDDEN, INTER), dtype=torch.uint8, device="cuda")
    mx.mxfp4_moe_gate_up(layer.gate, layer.up, E, HIDDEN, INTER, x, tokens, K, ids, act, ws)
    mx.mxfp4_moe_down(layer.down, E, HIDDEN, INTER, act, tokens, K, ids, w, want, ws)
    assert ((y - want).norm() / want.norm()).item() < 0.5
