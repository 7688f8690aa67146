"""Routing of tokens to experts and back on the GPU: the plan against a stable sort,
the moved rows exactly, the weighted sums and gradients against 64-bit sums, and the
gradients against differences.

Bounds: a sum of K products in FP32 is within (K + 1) 2^-24 of sum |w o| (K + 1
roundings of partial sums no larger than that), a dot product of n elements within n
2^-24 of sum |dy o| in any order.  A 16-bit result is such a sum rounded once: rounding
is monotone, so it lies between the rounded ends of that interval."""
import numpy as np
import pytest

import mx4_ref as ref
from gpu_util import cuda, host, to_dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def mx():
    return cuda()


def plan(mx, ids, n_experts):
    t, k = ids.shape
    token_at, pos_of = (torch.full((t * k,), 99, dtype=torch.int32, device="cuda:0") for _ in range(2))
    offsets = torch.full((n_experts + 1,), 99, dtype=torch.int32, device="cuda:0")
    mx.mxfp4_moe_sort(to_dev(ids.astype(np.int32)), t, k, n_experts, token_at, pos_of, offsets)
    return token_at, pos_of, offsets


@pytest.mark.parametrize("t,k,n", [(1, 1, 1), (1, 4, 8), (7, 3, 5), (32, 4, 64), (1000, 1, 1), (341, 3, 128), (1025, 1, 7),
                                   (513, 8, 256), (3000, 6, 1024), (20000, 4, 33)])
@pytest.mark.parametrize("kind", ["uniform", "one", "drops", "none"])
def test_plan(mx, t, k, n, kind):
    rng = np.random.default_rng(t + k + n)
    ids = rng.integers(0, n, (t, k))
    if kind == "one":
        ids[:] = n - 1
    elif kind == "drops":                              # ids outside the range, far ones too
        out = rng.random((t, k)) < 0.3
        ids[out] = rng.choice([-1, n, -2**31, 2**31 - 1], out.sum())
    elif kind == "none":
        ids[:] = -1
    got = [host(x) for x in plan(mx, ids, n)]
    flat = ids.reshape(-1)
    kept = (flat >= 0) & (flat < n)
    order = np.flatnonzero(kept)[np.argsort(flat[kept], kind="stable")]
    token_at, pos_of = np.full(t * k, -1), np.full(t * k, -1)
    token_at[:order.size], pos_of[order] = order // k, np.arange(order.size)
    assert np.array_equal(got[0], token_at)
    assert np.array_equal(got[1], pos_of)
    assert np.array_equal(got[2], np.searchsorted(flat[order], np.arange(n + 1)))


def test_plan_of_the_largest_size(mx):
    rng = np.random.default_rng(1)
    ids = rng.integers(-1, 200, (1 << 19, 8))
    got = [host(x) for x in plan(mx, ids, 200)]
    flat = ids.reshape(-1)
    kept = flat >= 0
    order = np.flatnonzero(kept)[np.argsort(flat[kept], kind="stable")]
    assert np.array_equal(got[0][:order.size], order // 8) and (got[0][order.size:] == -1).all()
    assert np.array_equal(got[1][order], np.arange(order.size)) and (got[1][~kept] == -1).all()
    assert np.array_equal(got[2], np.searchsorted(flat[order], np.arange(201)))


def test_reference_plan():
    token_at, pos_of, offsets = ref.sort_pairs([[2, 0], [0, -1], [2, 2]], 2, 3)
    assert token_at.tolist() == [0, 1, 0, 2, 2, -1] and pos_of.tolist() == [2, 0, 1, -1, 3, 4]
    assert offsets.tolist() == [0, 2, 2, 5]


SHAPES = [(1, 1, 1), (1, 4, 2880), (5, 2, 33), (32, 4, 2880), (17, 3, 1001), (100, 8, 64), (9, 6, 4096), (3, 2, 9000)]


def case(t, k, width, dtype, seed=0, drop=0.2):
    rng = np.random.default_rng(seed + t * 10 + k + width)
    n = 2 * k + 1
    ids = np.argsort(rng.random((t, n)), axis=1)[:, :k]
    ids[rng.random((t, k)) < drop] = -1
    mk = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dtype)  # noqa: E731
    w = rng.random((t, k)).astype(np.float32)
    return ids, n, mk(t, width), mk(t * k, width), w, mk(t, width)


def close(got, want, bound, dtype, what):
    g = got.double().cpu().numpy()
    lo, hi = (torch.from_numpy(np.ascontiguousarray(want + s * (bound + 1e-37))).float().to(dtype).double().numpy()
              for s in (-1, 1))
    bad = (g < lo) | (g > hi)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,k,width", SHAPES)
def test_rows_and_gradients(mx, dtype, t, k, width):
    ids, n, x, o, w, dy = case(t, k, width, dtype)
    token_at, pos_of, offsets = plan(mx, ids, n)
    p = t * k
    dev = lambda a: a.cuda() if isinstance(a, torch.Tensor) else to_dev(a)  # noqa: E731
    new = lambda *s: torch.full(s, 55.0, dtype=dtype, device="cuda:0")  # noqa: E731
    tok, pos = host(token_at), host(pos_of)
    kept = pos >= 0

    xs = new(p, width)
    mx.mxfp4_moe_dispatch(dev(x), t, k, width, token_at, xs)
    want = torch.where(torch.from_numpy(tok >= 0)[:, None], x[torch.from_numpy(np.maximum(tok, 0)).long()], torch.zeros((), dtype=dtype))
    assert torch.equal(xs.cpu(), want)

    o64, w64 = o.double().numpy(), w.astype(np.float64)
    rows = np.where(kept[:, None], o64[np.maximum(pos, 0)], 0.0).reshape(t, k, width)
    y = new(t, width)
    mx.mxfp4_moe_combine(dev(o), t, k, width, pos_of, dev(w), y)
    l1 = np.abs(w64[..., None] * rows).sum(1)
    close(y, (w64[..., None] * rows).sum(1), (k + 1) * 2.0**-24 * l1, dtype, "combine")

    dx = new(t, width)
    mx.mxfp4_moe_dispatch_grad(dev(o), t, k, width, pos_of, dx)
    close(dx, rows.sum(1), (k + 1) * 2.0**-24 * np.abs(rows).sum(1), dtype, "dispatch_grad")

    d_o, d_w = new(p, width), torch.full((t, k), 55.0, device="cuda:0")
    mx.mxfp4_moe_combine_grad(dev(dy), dev(o), t, k, width, pos_of, dev(w), d_o, d_w)
    dy64 = dy.double().numpy()
    full = (w64[..., None] * dy64[:, None]).reshape(p, width)
    got = d_o.cpu()
    assert (got[kept.sum():].float() == 55.0).all(), "rows of no pair were written"
    close(got[pos[kept]], full[kept], 2.0**-24 * np.abs(full[kept]), dtype, "d_o")
    dots = (dy64[:, None] * rows)
    close(d_w, dots.sum(-1), width * 2.0**-24 * np.abs(dots).sum(-1), torch.float32, "d_route_w")
    assert (host(d_w).reshape(-1)[~kept] == 0).all()


def test_dropped_pairs_add_nothing(mx):
    # a token without any row, and infinite or NaN weights on dropped pairs
    ids = np.array([[0, 1], [-1, 5], [1, -1]])
    token_at, pos_of, _ = plan(mx, ids, 2)
    o = torch.arange(6 * 40, dtype=torch.float32).reshape(6, 40).cuda()
    w = torch.tensor([[1.0, 1.0], [float("nan"), float("inf")], [1.0, float("nan")]]).cuda()
    y = torch.full((3, 40), 5.0, device="cuda:0")
    mx.mxfp4_moe_combine(o, 3, 2, 40, pos_of, w, y)
    oc = o.cpu()
    assert torch.equal(y.cpu(), torch.stack([oc[0] + oc[1], torch.zeros(40), oc[2]]))
    d_o, d_w = torch.zeros(6, 40, device="cuda:0"), torch.full((3, 2), 5.0, device="cuda:0")
    mx.mxfp4_moe_combine_grad(y, o, 3, 2, 40, pos_of, w, d_o, d_w)
    assert torch.isfinite(d_o).all() and torch.isfinite(d_w).all()
    assert (d_w.cpu()[torch.from_numpy(host(pos_of).reshape(3, 2) < 0)] == 0).all()


def test_indexes_out_of_range_are_left_out(mx):
    x = torch.ones(4, 24, device="cuda:0")
    idx = torch.tensor([0, 4, -7, 3, 2**31 - 1, 1, -2**31, 2], dtype=torch.int32, device="cuda:0")
    xs = torch.full((8, 24), 9.0, device="cuda:0")
    mx.mxfp4_moe_dispatch(x, 4, 2, 24, idx, xs)
    assert xs[:, 0].tolist() == [1, 0, 0, 1, 0, 1, 0, 1]
    o, w, y = torch.ones(8, 24, device="cuda:0"), torch.ones(4, 2, device="cuda:0"), torch.zeros(4, 24, device="cuda:0")
    pos = torch.tensor([0, 8, -7, 3, 2**31 - 1, 1, -2**31, -1], dtype=torch.int32, device="cuda:0")
    mx.mxfp4_moe_combine(o, 4, 2, 24, pos, w, y)
    assert y[:, 0].tolist() == [1, 1, 1, 0]


def test_gradients_against_differences(mx):
    # y is linear in o and in the weights, so a difference over any step is the derivative:
    # <dy, y(o + s) - y(o)> = <d_o, s> and <dy, y(w + s) - y(w)> = <d_w, s>
    t, k, width = 12, 3, 200
    ids, n, x, o, w, dy = case(t, k, width, torch.float32, seed=3)
    token_at, pos_of, _ = plan(mx, ids, n)
    rng = np.random.default_rng(5)
    od, wd, dyd = o.cuda(), to_dev(w), dy.cuda()
    d_o, d_w = torch.zeros_like(od), torch.zeros_like(wd)
    mx.mxfp4_moe_combine_grad(dyd, od, t, k, width, pos_of, wd, d_o, d_w)

    def y_of(o_, w_):
        y = torch.zeros(t, width, device="cuda:0")
        mx.mxfp4_moe_combine(o_, t, k, width, pos_of, w_, y)
        return y.double()

    base = y_of(od, wd)
    for _ in range(4):
        so = torch.from_numpy(rng.standard_normal(o.shape).astype(np.float32)).cuda()
        sw = torch.from_numpy(rng.standard_normal(w.shape).astype(np.float32)).cuda()
        for diff, grad, step in ((y_of(od + so, wd) - base, d_o, so), (y_of(od, wd + sw) - base, d_w, sw)):
            left = (dyd.double() * diff).sum().item()
            right = (grad.double() * step.double()).sum().item()
            scale = (dyd.double().abs() * diff.abs()).sum().item() + (dyd.double().abs() * base.abs()).sum().item()
            # y has k + 1 roundings, the stepped input one, the gradient one (a dot product's for d_w)
            assert abs(left - right) <= (2 * (k + 2) + width) * 2.0**-24 * scale
    # dx is the adjoint of the dispatch: <dxs, dispatch(x)> = <dispatch_grad(dxs), x>
    xs, dx = torch.zeros_like(od), torch.zeros(t, width, device="cuda:0")
    mx.mxfp4_moe_dispatch(x.cuda(), t, k, width, token_at, xs)
    mx.mxfp4_moe_dispatch_grad(od, t, k, width, pos_of, dx)
    left, right = (od.double() * xs.double()).sum().item(), (dx.double() * x.cuda().double()).sum().item()
    assert abs(left - right) <= (k + 2) * 2.0**-24 * (od.double() * xs.double()).abs().sum().item()


def test_repeats_bit_for_bit_on_another_stream(mx):
    t, k, width = 300, 4, 1000
    ids, n, x, o, w, dy = case(t, k, width, torch.bfloat16, seed=8)
    args = [a.cuda() for a in (o, dy)] + [to_dev(w)]
    _, pos_of, _ = plan(mx, ids, n)
    out = []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (None, s, None):
        y, d_o = torch.zeros(t, width, dtype=o.dtype, device="cuda:0"), torch.zeros_like(args[0])
        d_w = torch.zeros(t, k, device="cuda:0")
        torch.cuda.synchronize()
        mx.mxfp4_moe_combine(args[0], t, k, width, pos_of, args[2], y, stream=stream)
        mx.mxfp4_moe_combine_grad(args[1], args[0], t, k, width, pos_of, args[2], d_o, d_w, stream=stream)
        torch.cuda.synchronize()
        out.append((y, d_o, d_w))
    for a in out[1:]:
        assert all(torch.equal(p, q) for p, q in zip(out[0], a))


def test_offsets_past_32_bits(mx):
    # 70000 rows of 32768 elements: element offsets pass 2^31, byte offsets 2^32
    t, k, width = 35000, 2, 32768
    x = torch.zeros(t, width, dtype=torch.bfloat16, device="cuda:0")
    x[-1], x[0] = 3.0, 1.0
    ids = np.zeros((t, k), np.int64)
    ids[:, 1] = 1
    token_at, pos_of, _ = plan(mx, ids, 2)
    xs = torch.empty(t * k, width, dtype=torch.bfloat16, device="cuda:0")
    mx.mxfp4_moe_dispatch(x, t, k, width, token_at, xs)
    assert [xs[i].float().mean().item() for i in (0, t - 1, t, 2 * t - 1, 2 * t - 2)] == [1.0, 3.0, 1.0, 3.0, 0.0]
    y = torch.empty_like(x)
    w = torch.ones(t, k, device="cuda:0")
    mx.mxfp4_moe_combine(xs, t, k, width, pos_of, w, y)
    assert [y[i].float().mean().item() for i in (0, t - 1, t - 2)] == [2.0, 6.0, 0.0]
    d_w = torch.empty(t, k, device="cuda:0")
    d_o = torch.empty_like(xs)
    mx.mxfp4_moe_combine_grad(x, xs, t, k, width, pos_of, w, d_o, d_w)
    assert d_w[0].tolist() == [width, width] and d_w[-1].tolist() == [9.0 * width] * 2
    assert d_o[2 * t - 1].float().mean().item() == 3.0 and d_o[t].float().mean().item() == 1.0
