"""The binding of include/f8.h without a GPU, on host tensors that pass for the current device's and a
library that records its calls: what the kernels would read or write past a tensor's end, or as
something else, is refused (status 1) before the library is asked, or by it (type -1)."""
import pytest

torch = pytest.importorskip("torch")
F32, BF16, F16 = 0, 1, 2
TYPE = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
ROWS, COLS, NB, N = 32, 48, 4, 2


class Recorder:
    """Each entry point: notes its arguments; refuses a type that is none, as the library does."""

    def __init__(self, mx):
        self.mx, self.calls = mx, []

    def __getattr__(self, name):
        if name == "mxfp4_status_string":
            return lambda status: b"refused"
        types = [i for i, (got, arg) in enumerate(zip(self.mx._SIG[name][1], ARGS[name])) if arg in ("type", "y_type", "dw_type")]

        def call(*args):
            if any(args[i] not in (F32, BF16, F16) for i in types):
                return 1
            self.calls.append((name, args))
            return 0
        return call


ARGS = {"mxfp4_f8_quant": ("x", "type", "x_rows", "cols", "ld", "row_of", "rows", "codes", "scales", "values", "s"),
        "mxfp4_f8_quant_weight": ("w", "type", "n", "rows", "cols", "codes", "scales", "values", "s"),
        "mxfp4_mm_grad_w": ("dy", "x", "type", "rows", "cols", "n_rows", "dw", "dw_type", "s"),
        "mxfp4_moe_mm_grad_w": ("dy", "x", "type", "n", "rows", "cols", "n_rows", "off", "dw", "dw_type", "s")}
for _f in ("mxfp4_f8_mm", "mxfp4_f8_mm_grad"):
    ARGS[_f] = ("w", "ws", "rows", "cols", "x", "xs", "nb", "y", "y_type", "s")
for _f in ("mxfp4_f8_moe_mm", "mxfp4_f8_moe_mm_grad"):
    ARGS[_f] = ("w", "ws", "n", "rows", "cols", "x", "xs", "nb", "off", "y", "y_type", "s")


@pytest.fixture
def mx(monkeypatch):
    import mxfp4_dequant_matmul_gb300 as m
    m._f8_types()
    rec = Recorder(m)
    monkeypatch.setattr(m, "_lib", rec)
    monkeypatch.setattr(m, "_current_device", lambda: -1)   # a host tensor's get_device()
    monkeypatch.setattr(m, "_current_stream", lambda: 0)
    m.rec = rec
    return m


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def f32(*shape):
    return torch.zeros(shape)


OFF = torch.zeros(N + 1, dtype=torch.int32)
PRODUCTS = {"mxfp4_f8_mm": lambda mx, y, t: mx.mxfp4_f8_mm(u8(ROWS, COLS), f32(1, 1), ROWS, COLS, u8(NB, COLS), f32(1, NB), NB, y(NB, ROWS), y_type=t),
            "mxfp4_f8_mm_grad": lambda mx, y, t: mx.mxfp4_f8_mm_grad(u8(ROWS, COLS), f32(1, 1), ROWS, COLS, u8(NB, ROWS), f32(1, NB), NB,
                                                                     y(NB, COLS), dx_type=t),
            "mxfp4_f8_moe_mm": lambda mx, y, t: mx.mxfp4_f8_moe_mm(u8(N, ROWS, COLS), f32(N, 1, 1), N, ROWS, COLS, u8(NB, COLS), f32(1, NB), NB, OFF,
                                                                   y(NB, ROWS), y_type=t),
            "mxfp4_f8_moe_mm_grad": lambda mx, y, t: mx.mxfp4_f8_moe_mm_grad(u8(N, ROWS, COLS), f32(N, 1, 1), N, ROWS, COLS, u8(NB, ROWS), f32(1, NB),
                                                                             NB, OFF, y(NB, COLS), dx_type=t),
            "mxfp4_mm_grad_w": lambda mx, y, t: mx.mxfp4_mm_grad_w(f32(NB, ROWS).bfloat16(), f32(NB, COLS).bfloat16(), ROWS, COLS, NB, y(ROWS, COLS),
                                                                   dw_type=t),
            "mxfp4_moe_mm_grad_w": lambda mx, y, t: mx.mxfp4_moe_mm_grad_w(f32(NB, ROWS).bfloat16(), f32(NB, COLS).bfloat16(), N, ROWS, COLS, NB, OFF,
                                                                           y(N, ROWS, COLS), dw_type=t)}


def refused(mx, call, *args):
    with pytest.raises(mx.Mxfp4Error) as e:
        call(*args)
    assert e.value.status == 1 and not mx.rec.calls


@pytest.mark.parametrize("fn", list(PRODUCTS))
@pytest.mark.parametrize("dtype", list(TYPE))
@pytest.mark.parametrize("given", [None, F32, BF16, F16])
def test_the_results_type_is_the_tensors(mx, fn, dtype, given):
    """A type that is not the result's would be written past its end, or as other values."""
    def y(*shape):
        return torch.zeros(shape, dtype=dtype)
    if given is None or given == TYPE[dtype]:
        PRODUCTS[fn](mx, y, given)
        (name, args), = mx.rec.calls
        assert name == fn and args[len(ARGS[fn]) - 2] == TYPE[dtype]
    else:
        refused(mx, PRODUCTS[fn], mx, y, given)


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("dy,x,given", [(torch.bfloat16, torch.bfloat16, F16), (torch.float16, torch.float16, BF16), (torch.bfloat16, torch.float16, BF16),
                                        (torch.bfloat16, torch.float16, F16), (torch.float32, torch.float32, BF16)])
def test_the_operands_type_is_the_tensors(mx, grouped, dy, x, given):
    a, b = torch.zeros(NB, ROWS, dtype=dy), torch.zeros(NB, COLS, dtype=x)
    if grouped:
        refused(mx, lambda: mx.mxfp4_moe_mm_grad_w(a, b, N, ROWS, COLS, NB, OFF, f32(N, ROWS, COLS), type=given))
    else:
        refused(mx, lambda: mx.mxfp4_mm_grad_w(a, b, ROWS, COLS, NB, f32(ROWS, COLS), type=given))


@pytest.mark.parametrize("dtype", list(TYPE))
@pytest.mark.parametrize("given", [None, F32, BF16, F16])
@pytest.mark.parametrize("weight", [False, True])
def test_what_is_quantised_has_the_given_type(mx, weight, dtype, given):
    x, codes, values = torch.zeros(NB, COLS, dtype=dtype), u8(NB, COLS), torch.zeros(NB, COLS, dtype=dtype)

    def call(x, values):
        if weight:
            mx.mxfp4_f8_quant_weight(x, 1, NB, COLS, codes, f32(1, 1, 1), values, type=given)
        else:
            mx.mxfp4_f8_quant(x, NB, COLS, COLS, None, NB, codes, f32(1, NB), values, type=given)
    if given is None or given == TYPE[dtype]:
        call(x, values)
        call(x, None)
        assert [c[1][1] for c in mx.rec.calls] == [TYPE[dtype]] * 2
        mx.rec.calls.clear()
    else:
        refused(mx, call, x, values)
        refused(mx, call, x, None)
        refused(mx, call, 1 << 20, values)      # an address with values of another type
    other = torch.zeros(NB, COLS, dtype=torch.float16 if dtype is not torch.float16 else torch.bfloat16)
    refused(mx, call, x, other)


def test_addresses_take_the_given_type(mx):
    a = 1 << 20
    mx.mxfp4_f8_mm(a, a, ROWS, COLS, a, a, NB, a, y_type=BF16)
    mx.mxfp4_f8_quant(a, NB, COLS, COLS, None, NB, a, a, a, type=F16)
    mx.mxfp4_mm_grad_w(a, a, ROWS, COLS, NB, a, type=BF16, dw_type=F32)
    assert len(mx.rec.calls) == 3
    refused_before = len(mx.rec.calls)
    with pytest.raises(mx.Mxfp4Error):
        mx.mxfp4_f8_mm(a, a, ROWS, COLS, a, a, NB, a)          # no type at all
    assert len(mx.rec.calls) == refused_before


# --- the extent and the rows of what is quantised -------------------------------------------


def quantise(mx, x, x_rows, cols, ld, row_of=None, rows=None):
    rows = x_rows if rows is None else rows
    mx.mxfp4_f8_quant(x, x_rows, cols, ld, row_of, rows, u8(rows, cols), f32((cols + 127) // 128, rows))


FLAT = torch.zeros(1000, dtype=torch.bfloat16)
PICK = torch.zeros(9, dtype=torch.int32)


@pytest.mark.parametrize("x,x_rows,cols,ld", [
    (FLAT[:4 * 48].view(4, 48), 4, 48, 48), (FLAT[:4 * 48].view(4, 48), 3, 48, 48), (FLAT[:192], 4, 48, 48), (FLAT[:48], 1, 48, 1000),
    (FLAT[:960].view(10, 96)[:, 16:64], 10, 48, 96), (FLAT[:960].view(10, 96)[:, :48], 7, 48, 96), (FLAT[:960].view(10, 96)[3:, 48:], 7, 48, 96),
    (FLAT[:960].view(10, 96), 20, 48, 48), (FLAT[:960].view(10, 96), 5, 96, 192), (FLAT[:960].view(2, 5, 96)[:, :, 32:80], 10, 48, 96),
    (FLAT[3:3 + 9 * 97 + 48], 10, 48, 97), (torch.as_strided(FLAT, (10, 48), (97, 1), 3), 10, 48, 97), (FLAT[:960].view(20, 48)[::2], 10, 48, 96),
    (FLAT[:960].view(20, 48)[4:5, 16:32], 1, 16, 16), (FLAT[:960].view(20, 1, 48), 20, 48, 48), (FLAT[:960].view(10, 96)[:, None, :48], 10, 48, 96),
    (FLAT[:960].view(10, 96)[:, :48], 5, 48, 192), (FLAT[:960].view(10, 96)[1:2, :48], 1, 48, 48), (FLAT[:960].view(2, 5, 96)[:1, :, :48], 5, 32, 96),
    (FLAT[:960].view(2, 5, 3, 4, 8)[:, :, 1], 10, 32, 96), (FLAT[:960].view(10, 2, 3, 16)[:, 1], 10, 48, 96), (FLAT[:960].view(2, 5, 96)[:, :4], 4, 96, 96),
    (FLAT[:960].view(2, 10, 48)[:, :9], 2, 144, 480), (FLAT[:960].view(2, 10, 48)[:, :9], 3, 144, 144)])
def test_rows_within_the_tensor_pass(mx, x, x_rows, cols, ld):
    quantise(mx, x, x_rows, cols, ld)
    (_, args), = mx.rec.calls
    assert args[0] == x.data_ptr() and args[2:5] == (x_rows, cols, ld)
    quantise(mx, x, x_rows, cols, ld, PICK, 9)
    assert len(mx.rec.calls) == 2


@pytest.mark.parametrize("x,x_rows,cols,ld", [
    (FLAT[:192].view(4, 48), 5, 48, 48), (FLAT[:192].view(4, 48), 4, 48, 49), (FLAT[:192].view(4, 48), 4, 64, 64), (FLAT[:191], 4, 48, 48),
    (FLAT[:47], 1, 48, 48), (FLAT[:960].view(10, 96)[:, :48], 11, 48, 96), (FLAT[:960].view(10, 96)[:, :48], 10, 64, 96),
    (FLAT[:960].view(10, 96)[:4, :48], 5, 48, 96), (FLAT[:0], 1, 48, 48), (FLAT[:960].view(48, 20).T, 20, 48, 48), (FLAT[:96:2], 1, 48, 48),
    (FLAT[:48].expand(5, 48), 5, 48, 48), (FLAT[:960].view(2, 10, 48).transpose(0, 1), 20, 48, 48), (FLAT[:960].view(10, 96)[:, :48], 10, 48, 48),
    (FLAT[:960].view(2, 5, 96)[:, :4, 32:80], 8, 48, 96),
    (FLAT[:960].view(10, 96)[:, :48], 9, 64, 96), (FLAT[:960].view(10, 96)[:, :48], 6, 48, 192),
    (FLAT[:960].view(2, 5, 3, 4, 8)[:, :, 1], 10, 48, 96), (FLAT[:960].view(2, 5, 3, 4, 8)[:, :, 1], 11, 32, 96),
    (FLAT[:960].view(2, 5, 3, 4, 8)[..., 1, :], 10, 32, 96), (FLAT[:960].view(2, 5, 96)[:, :4], 5, 96, 96)])
def test_rows_past_the_tensor_or_elsewhere_are_refused(mx, x, x_rows, cols, ld):
    """Too few elements, another unit than 1 along a row, rows that are not ld apart."""
    refused(mx, quantise, mx, x, x_rows, cols, ld)
    refused(mx, lambda: quantise(mx, x, x_rows, cols, ld, PICK, 9))


def test_sizes_the_library_refuses_reach_it(mx):
    """Numbers that are wrong whatever the tensor is are the library's to refuse."""
    for x_rows, cols, ld in ((0, 48, 48), (4, 48, -48), (4, 0, 48), (4, -48, 48)):
        quantise_none = (x_rows, cols, ld)
        mx.rec.calls.clear()
        mx.mxfp4_f8_quant(FLAT[:192].view(4, 48), x_rows, cols, ld, None, 4, u8(4, 48), f32(1, 4))
        assert len(mx.rec.calls) == 1, quantise_none


def test_what_passes_is_read_within_the_tensor():
    """Random views and rows: those that pass read elements of the view alone, and of a view with rows
    at one distance every such choice passes."""
    import random
    import mxfp4_dequant_matmul_gb300 as m
    rng, flat, passed = random.Random(5), torch.arange(720), 0
    for _ in range(20000):
        x = flat.view(rng.choice([(720,), (45, 16), (9, 5, 16), (3, 15, 16), (5, 3, 3, 16), (15, 48), (5, 3, 48), (720, 1)]))
        for d in range(x.dim()):
            if rng.random() < 0.5:
                a = rng.randrange(x.shape[d])
                x = x.narrow(d, a, rng.randint(1, x.shape[d] - a))
        if rng.random() < 0.2 and x.dim() > 1:
            x = x.transpose(0, rng.randrange(x.dim()))
        if rng.random() < 0.1:
            x = x[::2]
        if rng.random() < 0.1:
            x = x.select(rng.randrange(x.dim()), 0) if x.dim() > 1 else x
        held = set(x.reshape(-1).tolist())
        cols = rng.choice([1, 8, 16, 32, 48])
        plain = x.dim() == 2 and x.shape[0] > 1 and x.stride(1) == 1 and x.stride(0) >= cols
        ld = x.stride(0) * rng.choice([1, 1, 2]) if plain and rng.random() < 0.7 else cols + rng.choice([0, 0, 0, 8, 16, 32, 96])
        x_rows = rng.randint(1, 12)
        inside = all(x.storage_offset() + i * ld + c in held for i in range(x_rows) for c in range(cols))
        out = m._outside(x, x_rows, cols, ld)
        assert inside or out, (x.shape, x.stride(), x_rows, cols, ld)
        if plain and inside and cols <= x.shape[1] and ld % x.stride(0) == 0:
            assert not out, (x.shape, x.stride(), x_rows, cols, ld)
        passed += not out
    assert passed > 2000
