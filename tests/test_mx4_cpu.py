"""include/mx4.h without a GPU: the refusals of every entry point (nothing is
launched), the binding's choice of element type, and the reference's own pins."""
import numpy as np
import pytest

import mx4_ref as ref

A = 1 << 20      # an aligned fake address; never dereferenced
BF16, F32 = 1, 0


@pytest.fixture(scope="module")
def mx():
    import __graft_entry__
    __graft_entry__.build()
    import mxfp4_dequant_matmul_gb300 as m
    m.lib()
    return m


def test_quant_refusals(mx):
    f = mx.lib().mxfp4_quant
    ok = dict(x=A, type=BF16, x_rows=8, cols=64, ld=64, row_of=None, rows=8, out=A, values=None)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["x"], a["type"], a["x_rows"], a["cols"], a["ld"], a["row_of"], a["rows"],
                 a["out"], a["values"], None)

    for kw in (dict(type=3), dict(type=-1), dict(cols=48), dict(cols=0), dict(rows=0), dict(x_rows=0),
               dict(ld=63), dict(rows=9), dict(ld=1 << 41), dict(rows=1 << 22, x_rows=1 << 22, cols=1 << 25, ld=1 << 25)):
        assert call(**kw) == 1, kw
    for kw in (dict(x=None), dict(x=A + 1), dict(out=None), dict(out=A + 8), dict(values=A + 4),
               dict(row_of=A + 2), dict(type=F32, x=A + 2)):
        assert call(**kw) == 2, kw


def test_swiglu_quant_refusals(mx):
    f = mx.lib().mxfp4_swiglu_quant
    assert f(A, A, BF16, 8, 64, 63, 0.0, A, None, None) == 1
    assert f(A, A, 7, 8, 64, 64, 0.0, A, None, None) == 1
    assert f(A, A, BF16, 8, 65, 65, 0.0, A, None, None) == 1
    assert f(A, A, BF16, 8, 64, 64, float("nan"), A, None, None) == 1
    assert f(A, A, BF16, 8, 64, 64, float("inf"), A, None, None) == 1
    for gate, up, out, values in ((None, A, A, None), (A, None, A, None), (A, A, None, None),
                                  (A, A + 1, A, None), (A, A, A + 4, None), (A, A, A, A + 2)):
        assert f(gate, up, BF16, 8, 64, 64, 0.0, out, values, None) == 2


def test_product_refusals(mx):
    f = mx.lib().mxfp4_mm_mx
    for rows, cols, nb, t in ((0, 64, 1, 0), (8, 48, 1, 0), (8, 64, 0, 0), (8, 64, 1, 2), (8, 64, 1, 5),
                              (8, 64, (1 << 24) + 1, 0), (1 << 22, 1 << 25, 1, 0)):
        assert f(A, rows, cols, A, nb, A, t, None) == 1, (rows, cols, nb, t)
    for w, x, y in ((None, A, A), (A, None, A), (A, A, None), (A + 8, A, A), (A, A + 8, A), (A, A, A + 8)):
        assert f(w, 8, 64, x, 2, y, 0, None) == 2


def test_experts_refusals(mx):
    f = mx.lib().mxfp4_moe_mm_mx
    for n, rows, cols, n_rows, t in ((0, 8, 64, 4, 0), (1025, 8, 64, 4, 0), (4, 8, 33, 4, 0), (4, 8, 64, 0, 0),
                                     (4, 8, 64, 4, 2), (1024, 1 << 20, 1 << 17, 4, 0)):
        assert f(A, n, rows, cols, A, n_rows, A, A, t, None) == 1, (n, rows, cols, n_rows, t)
    for bank, x, off, y in ((None, A, A, A), (A, None, A, A), (A, A, None, A), (A, A, A, None),
                            (A + 4, A, A, A), (A, A, A + 2, A), (A, A, A, A + 4)):
        assert f(bank, 4, 8, 64, x, 4, off, y, 0, None) == 2


def test_routing_refusals(mx):
    L = mx.lib()
    for t, k, n in ((0, 1, 4), (1, 0, 4), (1, 1, 0), (1, 1, 1025), ((1 << 22) + 1, 1, 4), (1 << 20, 5, 4)):
        assert L.mxfp4_moe_sort(A, t, k, n, A, A, A, None) == 1, (t, k, n)
    for p in range(4):
        a = [A, A, A, A]
        for bad in (None, A + 1):
            a[p] = bad
            assert L.mxfp4_moe_sort(a[0], 4, 2, 4, a[1], a[2], a[3], None) == 2
    for typ, t, k, width in ((3, 4, 2, 8), (0, 0, 2, 8), (0, 4, 0, 8), (0, 4, 2, 0), (0, 4, 2, (1 << 24) + 1)):
        assert L.mxfp4_moe_dispatch(A, typ, t, k, width, A, A, None) == 1
        assert L.mxfp4_moe_dispatch_grad(A, typ, t, k, width, A, A, None) == 1
        assert L.mxfp4_moe_combine(A, typ, t, k, width, A, A, A, None) == 1
        assert L.mxfp4_moe_combine_grad(A, A, typ, t, k, width, A, A, A, A, None) == 1
    for bad in (None, A + 8):
        assert L.mxfp4_moe_dispatch(bad, 0, 4, 2, 8, A, A, None) == 2
        assert L.mxfp4_moe_dispatch(A, 0, 4, 2, 8, A, bad, None) == 2
        assert L.mxfp4_moe_dispatch_grad(bad, 0, 4, 2, 8, A, A, None) == 2
        assert L.mxfp4_moe_combine(A, 0, 4, 2, 8, A, A, bad, None) == 2
        assert L.mxfp4_moe_combine_grad(A, bad, 0, 4, 2, 8, A, A, A, A, None) == 2
        assert L.mxfp4_moe_combine_grad(A, A, 0, 4, 2, 8, A, A, bad, A, None) == 2
    assert L.mxfp4_moe_dispatch(A, 0, 4, 2, 8, None, A, None) == 2
    assert L.mxfp4_moe_combine(A, 0, 4, 2, 8, A, None, A, None) == 2
    assert L.mxfp4_moe_combine_grad(A, A, 0, 4, 2, 8, A, A, A, None, None) == 2


def test_binding_takes_the_type_from_the_tensors(mx):
    torch = pytest.importorskip("torch")
    bf, f32 = torch.zeros(64, dtype=torch.bfloat16), torch.zeros(64)
    assert mx._type(None, bf) == mx.TYPE_BF16 and mx._type(None, f32, f32, None) == mx.TYPE_F32
    assert mx._type(None, torch.zeros(4, dtype=torch.float16)) == mx.TYPE_F16
    assert mx._type(None, bf, f32) == -1            # an output of another type than the input
    assert mx._type(None, torch.zeros(4, dtype=torch.float64)) == -1
    assert mx._type(None, A) == -1 and mx._type(mx.TYPE_BF16, A) == mx.TYPE_BF16
    with pytest.raises(mx.Mxfp4Error) as e:         # refused on the host: nothing is launched
        mx.mxfp4_quant(bf, 1, 64, 64, None, 1, A, values=f32, stream=0)
    assert e.value.status == 1


def test_reference_quantisation_by_hand():
    x = np.zeros((1, 64))
    x[0, :9] = [6.0, 5.0, 2.5, 0.25, -0.75, -0.0, 7.9, 1.75, 3.5]     # amax in [4, 8): scale 1
    x[0, 32] = 2.0 ** -140                                              # below the smallest scale
    code, k = ref.quantise(x)
    assert k.tolist() == [[127, 0]]
    assert code[0, :9].tolist() == [7, 6, 4, 0, 8 | 2, 8, 7, 4, 6]
    assert code[0, 32] == 0 and ref.values(code, k)[0, 6] == 6.0
    x[0, 40] = np.inf
    code, k = ref.quantise(x)
    assert k.tolist() == [[127, 255]] and not code[0, 32:].any()


def test_reference_agrees_with_the_oracle_decode(orc):
    rng = np.random.default_rng(1)
    code, k = ref.random_matrix(rng, 5, 96, 0, 255)
    got = orc.dequant(ref.pack(code, k), 5, 96)
    assert np.array_equal(got.astype(np.float64), ref.values(code, k))


def test_binding_refuses_other_index_and_weight_types(mx):
    """int64 ids (as topk gives them) would be read as pairs of halves, bfloat16 route weights past
    their end.  Every call below has a misaligned or null pointer as well, so that nothing could be
    launched: with the right dtypes that is what is refused (status 2)."""
    torch = pytest.importorskip("torch")
    i32, i64 = (lambda n, d=d: torch.zeros(n, dtype=d) for d in (torch.int32, torch.int64))
    f32, bf16 = (lambda n, d=d: torch.zeros(n, dtype=d) for d in (torch.float32, torch.bfloat16))
    odd = f32(65)[1:]                              # 4 bytes past a 16-byte boundary
    u8 = torch.zeros(256, dtype=torch.uint8)

    def sort(**kw):
        a = {**dict(ids=i32(8), token_at=i32(8), pos_of=i32(8), offsets=i32(5)), **kw}
        mx.mxfp4_moe_sort(a["ids"], 4, 2, 4, a["token_at"], a["pos_of"], a["offsets"], stream=0)

    def quant(**kw):
        mx.mxfp4_quant(f32(64), 2, 32, 32, kw.get("row_of", i32(2)), 2, u8[1:], stream=0)

    def experts(**kw):
        mx.mxfp4_moe_mm_mx(u8, 1, 2, 32, u8, 2, kw.get("offsets", i32(2)), odd, stream=0)

    def dispatch(**kw):
        mx.mxfp4_moe_dispatch(f32(64), 2, 1, 32, kw.get("token_at", i32(2)), odd, stream=0)

    def dispatch_grad(**kw):
        mx.mxfp4_moe_dispatch_grad(f32(64), 2, 1, 32, kw.get("pos_of", i32(2)), odd, stream=0)

    def combine(**kw):
        mx.mxfp4_moe_combine(f32(64), 2, 1, 32, kw.get("pos_of", i32(2)), kw.get("route_w", f32(2)), odd, stream=0)

    def combine_grad(**kw):
        mx.mxfp4_moe_combine_grad(f32(64), f32(64), 2, 1, 32, kw.get("pos_of", i32(2)), kw.get("route_w", f32(2)), odd,
                                  kw.get("d_route_w", f32(2)), stream=0)

    def status(call, **kw):
        with pytest.raises(mx.Mxfp4Error) as e:
            call(**kw)
        return e.value.status

    for call in (quant, experts, dispatch, dispatch_grad, combine, combine_grad):
        assert status(call) == 2, call
    assert status(sort, ids=None) == status(sort, offsets=None) == 2
    for call, name in ((quant, "row_of"), (experts, "offsets"), (dispatch, "token_at"), (dispatch_grad, "pos_of"),
                       (combine, "pos_of"), (combine_grad, "pos_of")):
        for bad in (i64(8), f32(8), torch.zeros(8, dtype=torch.int16)):
            assert status(call, **{name: bad}) == 1, (call, name)
    for call, name in ((combine, "route_w"), (combine_grad, "route_w"), (combine_grad, "d_route_w")):
        for bad in (bf16(8), torch.zeros(8, dtype=torch.float64), i32(8)):
            assert status(call, **{name: bad}) == 1, (call, name)
    for name in ("ids", "token_at", "pos_of", "offsets"):
        other = "ids" if name != "ids" else "offsets"
        assert status(sort, **{name: i64(8), other: None}) == 1, name
    # addresses pass, whatever they point to
    with pytest.raises(mx.Mxfp4Error) as e:
        mx.mxfp4_moe_combine(f32(64), 2, 1, 32, A, A, odd, stream=0)
    assert e.value.status == 2
