"""Cases that time and check the microscaled 4-bit operators and the routing operators around them.

Four operators: quantisation to MXFP4, the product of two MXFP4 matrices, the product of each expert's rows with that
expert's MXFP4 matrix, and the routing of tokens to experts and back (with its gradient).  `own` chooses between the
plain form (elementary torch operations in 32 bits) and the library's entry points; both take what `prepare` makes.

MXFP4 buffer of a [rows, cols] matrix: rows*cols/2 code bytes (byte b of a group of 32 holds elements 2b and 2b+1, low
nibble first), rows*cols/32 scale bytes, padding to 16 bytes.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --- cases ---------------------------------------------------------------------------------------


def listed():
    return [
        # one token's activations, as each decoding step quantises them before a product: latency
        {"name": "quant one token", "op": "quant", "rows": 1, "cols": 4096, "type": "bf16", "source": 1, "gather": False},
        # a prompt's activations put in expert order while they are quantised (top-4 of 1999 tokens)
        {"name": "quant sorted prompt", "op": "quant", "rows": 7996, "cols": 2880, "type": "bf16", "source": 1999, "gather": True},
        # a weight matrix quantised from its f32 master copy, with the rounded values for the forward pass
        {"name": "quant weights", "op": "quant", "rows": 14336, "cols": 4096, "type": "f32", "source": 14336, "gather": False},
        # a decoding step's projection, one token
        {"name": "product one token", "op": "product", "rows": 14336, "cols": 4096, "tokens": 1, "out": "f32"},
        # a small batch of decoding requests, wide rows
        {"name": "product batch of 8", "op": "product", "rows": 4096, "cols": 14336, "tokens": 8, "out": "bf16"},
        # a ragged prompt on odd sizes: rows that fill no tile, a scale plane without alignment
        {"name": "product ragged prompt", "op": "product", "rows": 2303, "cols": 2880, "tokens": 333, "out": "bf16"},
        # a prompt's projection
        {"name": "product prompt", "op": "product", "rows": 4096, "cols": 4096, "tokens": 2048, "out": "f32"},
        # one decoding step of 32 requests through 64 experts: most experts see a row or two
        {"name": "experts decode", "op": "experts", "experts": 64, "rows": 2880, "cols": 2880, "tokens": 32, "top_k": 4, "out": "bf16"},
        # a prompt through the same experts
        {"name": "experts prompt", "op": "experts", "experts": 64, "rows": 2880, "cols": 2880, "tokens": 2048, "top_k": 4, "out": "bf16"},
        # routing of one decoding step, forward only
        {"name": "routing decode", "op": "routing", "tokens": 32, "top_k": 4, "experts": 64, "width": 2880, "type": "bf16", "train": False, "drop": 0.0},
        # routing of a training batch, forward and backward
        {"name": "routing training", "op": "routing", "tokens": 4096, "top_k": 4, "experts": 64, "width": 2880, "type": "bf16", "train": True, "drop": 0.0},
        # pairs dropped by a full expert, odd sizes, f32
        {"name": "routing ragged", "op": "routing", "tokens": 1111, "top_k": 3, "experts": 23, "width": 1001, "type": "f32", "train": True, "drop": 0.05},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quant", "product", "experts", "routing"))
    if op == "quant":
        cols = 32 * _log_int(rng, 1, 448)
        rows = _log_int(rng, 1, max(1, min(16384, 14336 * 4096 // cols)))
        gather = rng.random() < 0.5
        source = _log_int(rng, max(1, rows // 8), max(1, rows)) if gather else rows
        return {"op": op, "rows": rows, "cols": cols, "type": rng.choice(("f32", "bf16", "f16")), "source": source,
                "gather": gather}
    if op == "product":
        cols = 32 * _log_int(rng, 4, 448)
        rows = _log_int(rng, 16, min(16384, 14336 * 4096 // cols))
        tokens = _log_int(rng, 1, max(1, min(4096, 4096 * 4096 * 2048 // (rows * cols))))
        return {"op": op, "rows": rows, "cols": cols, "tokens": tokens, "out": rng.choice(("f32", "bf16"))}
    if op == "experts":
        cols = 32 * _log_int(rng, 4, 90)
        rows = _log_int(rng, 16, 2880)
        experts = _log_int(rng, 4, 64)
        top_k = rng.randint(1, min(8, experts))
        return {"op": op, "experts": experts, "rows": rows, "cols": cols, "tokens": _log_int(rng, 1, 8192 // top_k),
                "top_k": top_k, "out": rng.choice(("f32", "bf16"))}
    experts = _log_int(rng, 4, 256)
    top_k = rng.randint(1, min(8, experts))
    width = _log_int(rng, 32, 4096)
    return {"op": op, "tokens": _log_int(rng, 1, max(1, min(8192, 4096 * 4 * 2880 // (2 * top_k * width)))), "top_k": top_k,
            "experts": experts, "width": width, "type": rng.choice(("f32", "bf16", "f16")),
            "train": rng.random() < 0.5, "drop": rng.choice((0.0, 0.05))}


# --- the format, in 32-bit torch operations --------------------------------------------------------


def _nbytes(rows, cols):
    return (rows * cols * 17 // 32 + 15) // 16 * 16


def _encode(x):
    """[rows, cols] f32 -> (codes [rows, cols] uint8, scale bytes [rows, cols/32] uint8)."""
    g = x.reshape(x.shape[0], -1, 32)
    exponent = g.abs().amax(-1).contiguous().view(torch.int32) >> 23
    finite = torch.isfinite(g).all(-1)
    k = (exponent - 2).clamp(min=0)
    a = g * ((254 - k) << 23).view(torch.float32).unsqueeze(-1)
    s, a = torch.signbit(g), a.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = torch.where(finite.unsqueeze(-1), code + 8 * s, 0).to(torch.uint8)
    return code.reshape(x.shape), torch.where(finite, k, 255).to(torch.uint8)


def _pack(code, k):
    """Codes and scale bytes -> one MXFP4 buffer."""
    rows, cols = code.shape
    pair = code.reshape(rows, cols // 2, 2)
    out = torch.zeros(_nbytes(rows, cols), dtype=torch.uint8, device=code.device)
    out[: rows * cols // 2] = (pair[..., 0] | (pair[..., 1] << 4)).reshape(-1)
    out[rows * cols // 2: rows * cols * 17 // 32] = k.reshape(-1)
    return out


def _decode(buf, rows, cols, dtype=torch.float32):
    """[n, nbytes] (or one buffer) -> values [n, rows, cols]."""
    buf = buf.reshape(-1, _nbytes(rows, cols))
    grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=dtype, device=buf.device)
    byte = buf[:, : rows * cols // 2]
    k = buf[:, rows * cols // 2: rows * cols * 17 // 32].to(torch.int32)
    scale = torch.where(k == 0, 0x00400000, k << 23).to(torch.int32)
    scale = torch.where(k == 255, 0x7FC00000, scale).to(torch.int32).view(torch.float32).to(dtype)
    both = torch.stack((grid[(byte & 15).int()], grid[(byte >> 4).int()]), -1)
    return (both.reshape(-1, rows, cols // 32, 32) * scale.reshape(-1, rows, cols // 32, 1)).reshape(-1, rows, cols)


# --- states ----------------------------------------------------------------------------------------


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _activations(g, rows, cols):
    """Normal values, a few channels much larger than the rest, and rows of different size, as a residual stream has them."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    channel = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return x * channel * torch.exp2(torch.randn(rows, 1, generator=g, device="cuda"))


def _quantised(x):
    return _pack(*_encode(x))


def _weights(g, rows, cols):
    return 0.02 * torch.randn(rows, cols, generator=g, device="cuda") * torch.exp2(torch.randn(rows, 1, generator=g, device="cuda"))


def _ids(g, tokens, top_k, experts, drop):
    """Each token's distinct experts, some experts more popular than others; a dropped pair's id is -1."""
    liking = 0.5 * torch.randn(experts, generator=g, device="cuda")
    u = torch.rand(tokens, experts, generator=g, device="cuda")
    ids = (liking - torch.log(-torch.log(u.clamp(1e-6, 1 - 1e-6)))).topk(top_k, dim=1).indices.to(torch.int32)
    lost = torch.rand(tokens, top_k, generator=g, device="cuda") < drop
    return torch.where(lost, -1, ids).to(torch.int32).contiguous()


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    op = case["op"]
    if op == "quant":
        rows, cols, source = case["rows"], case["cols"], case["source"]
        dtype = TYPES[case["type"]]
        # a master weight copy is f32 and has no outlier channels; activations come in 16 bits as a rule
        s["x"] = (_weights(g, source, cols) if case["type"] == "f32" else _activations(g, source, cols)).to(dtype)
        s["row_of"] = None
        if case["gather"]:
            s["row_of"] = torch.randint(0, source, (rows,), generator=g, device="cuda", dtype=torch.int32)
        s["packed"] = torch.zeros(_nbytes(rows, cols), dtype=torch.uint8, device="cuda")
        s["values"] = torch.zeros(rows, cols, dtype=dtype, device="cuda")
    elif op == "product":
        s["w"] = _quantised(_weights(g, case["rows"], case["cols"]))
        s["x"] = _quantised(_activations(g, case["tokens"], case["cols"]))
        s["y"] = torch.zeros(case["tokens"], case["rows"], dtype=TYPES[case["out"]], device="cuda")
    elif op == "experts":
        n, rows, cols = case["experts"], case["rows"], case["cols"]
        s["bank"] = torch.stack([_quantised(_weights(g, rows, cols)) for _ in range(n)])
        ids = _ids(g, case["tokens"], case["top_k"], n, 0.0).reshape(-1).long()
        count = torch.bincount(ids, minlength=n)
        s["offsets"] = torch.cat((torch.zeros(1, device="cuda"), count.cumsum(0))).to(torch.int32)
        s["most"] = int(count.max())  # rows of the busiest expert, as the plan of a batch holds it
        pairs = case["tokens"] * case["top_k"]
        s["x"] = _quantised(_activations(g, pairs, cols))
        s["y"] = torch.zeros(pairs, rows, dtype=TYPES[case["out"]], device="cuda")
    else:
        tokens, top_k, width = case["tokens"], case["top_k"], case["width"]
        pairs, dtype = tokens * top_k, TYPES[case["type"]]
        s["ids"] = _ids(g, tokens, top_k, case["experts"], case["drop"])
        s["weights"] = torch.softmax(torch.randn(tokens, top_k, generator=g, device="cuda"), -1)
        s["x"] = _activations(g, tokens, width).to(dtype)
        s["o"] = torch.randn(pairs, width, generator=g, device="cuda").to(dtype)  # the experts' outputs, in expert order
        s["token_at"] = torch.zeros(pairs, dtype=torch.int32, device="cuda")
        s["pos_of"] = torch.zeros(pairs, dtype=torch.int32, device="cuda")
        s["offsets"] = torch.zeros(case["experts"] + 1, dtype=torch.int32, device="cuda")
        s["xs"] = torch.zeros(pairs, width, dtype=dtype, device="cuda")
        s["y"] = torch.zeros(tokens, width, dtype=dtype, device="cuda")
        if case["train"]:
            s["dy"] = torch.randn(tokens, width, generator=g, device="cuda").to(dtype)
            s["dxs"] = torch.randn(pairs, width, generator=g, device="cuda").to(dtype)
            s["do"] = torch.zeros(pairs, width, dtype=dtype, device="cuda")
            s["dweights"] = torch.zeros(tokens, top_k, device="cuda")
            s["dx"] = torch.zeros(tokens, width, dtype=dtype, device="cuda")
    return s


# --- one pass --------------------------------------------------------------------------------------


def run(state):
    return (_run_own if own else _run_plain)[state["op"]](state)


def _quant_plain(s):
    x = s["x"].float()
    if s["row_of"] is not None:
        x = x[s["row_of"]]
    buf = _pack(*_encode(x))
    return {"values": _decode(buf, s["rows"], s["cols"])[0].to(s["x"].dtype)}


def _product_plain(s):
    w = _decode(s["w"], s["rows"], s["cols"])[0]
    x = _decode(s["x"], s["tokens"], s["cols"])[0]
    return {"y": (x @ w.T).to(s["y"].dtype)}


def _experts_plain(s):
    n, cols, pairs, most = s["experts"], s["cols"], s["tokens"] * s["top_k"], s["most"]
    w = _decode(s["bank"], s["rows"], cols)
    x = _decode(s["x"], pairs, cols)[0]
    at = torch.arange(pairs, device=x.device, dtype=torch.int32)
    expert = torch.searchsorted(s["offsets"][1:], at, right=True)
    place = expert * most + (at - s["offsets"][expert])
    padded = torch.zeros(n * most, cols, device=x.device)
    padded[place] = x
    y = torch.bmm(padded.reshape(n, most, cols), w.transpose(1, 2))
    return {"y": y.reshape(n * most, -1)[place].to(s["y"].dtype)}


def _plan_plain(s):
    n, top_k = s["experts"], s["top_k"]
    ids = s["ids"].reshape(-1)
    key = torch.where((ids < 0) | (ids >= n), n, ids)
    sorted_key, order = torch.sort(key, stable=True)
    token_at = torch.where(sorted_key < n, order // top_k, -1).to(torch.int32)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    pos_of = torch.where(key < n, place, -1).to(torch.int32)
    offsets = torch.searchsorted(sorted_key, torch.arange(n + 1, device=key.device, dtype=torch.int32)).to(torch.int32)
    return token_at, pos_of, offsets


def _routing_plain(s):
    tokens, top_k, width, dtype = s["tokens"], s["top_k"], s["width"], s["x"].dtype
    token_at, pos_of, offsets = _plan_plain(s)
    kept_row = (token_at >= 0).unsqueeze(-1)
    kept = (pos_of >= 0).reshape(tokens, top_k, 1)
    row = pos_of.clamp(min=0)
    xs = torch.where(kept_row, s["x"][token_at.clamp(min=0)], 0)
    o = torch.where(kept, s["o"][row].float().reshape(tokens, top_k, width), 0.0)
    y = (s["weights"].unsqueeze(-1) * o).sum(1).to(dtype)
    out = {"token_at": token_at, "pos_of": pos_of, "offsets": offsets, "xs": xs, "y": y}
    if s["train"]:
        dy = s["dy"].float().unsqueeze(1)
        dpair = (s["weights"].unsqueeze(-1) * dy).reshape(-1, width).to(dtype)
        spread = torch.zeros(tokens * top_k + 1, width, dtype=dtype, device=dy.device)
        spread[torch.where(pos_of >= 0, pos_of, tokens * top_k)] = dpair
        out["do"] = spread[:-1]
        out["dweights"] = (dy * o).sum(-1)
        dxs = torch.where(kept, s["dxs"][row].float().reshape(tokens, top_k, width), 0.0)
        out["dx"] = dxs.sum(1).to(dtype)
    return out


def _mx():
    import mxfp4_dequant_matmul_gb300 as mx
    return mx


def _quant_own(s):
    mx = _mx()
    mx.mxfp4_quant(s["x"], s["source"], s["cols"], s["cols"], s["row_of"], s["rows"], s["packed"], s["values"])
    return {"values": s["values"]}


def _product_own(s):
    mx = _mx()
    mx.mxfp4_mm_mx(s["w"], s["rows"], s["cols"], s["x"], s["tokens"], s["y"])
    return {"y": s["y"]}


def _experts_own(s):
    mx = _mx()
    mx.mxfp4_moe_mm_mx(s["bank"], s["experts"], s["rows"], s["cols"], s["x"], s["tokens"] * s["top_k"], s["offsets"],
                       s["y"])
    return {"y": s["y"]}


def _routing_own(s):
    mx = _mx()
    tokens, top_k, width = s["tokens"], s["top_k"], s["width"]
    mx.mxfp4_moe_sort(s["ids"], tokens, top_k, s["experts"], s["token_at"], s["pos_of"], s["offsets"])
    mx.mxfp4_moe_dispatch(s["x"], tokens, top_k, width, s["token_at"], s["xs"])
    mx.mxfp4_moe_combine(s["o"], tokens, top_k, width, s["pos_of"], s["weights"], s["y"])
    out = {k: s[k] for k in ("token_at", "pos_of", "offsets", "xs", "y")}
    if s["train"]:
        mx.mxfp4_moe_combine_grad(s["dy"], s["o"], tokens, top_k, width, s["pos_of"], s["weights"], s["do"], s["dweights"])
        mx.mxfp4_moe_dispatch_grad(s["dxs"], tokens, top_k, width, s["pos_of"], s["dx"])
        out.update({k: s[k] for k in ("do", "dweights", "dx")})
    return out


_run_plain = {"quant": _quant_plain, "product": _product_plain, "experts": _experts_plain, "routing": _routing_plain}
_run_own = {"quant": _quant_own, "product": _product_own, "experts": _experts_own, "routing": _routing_own}


# --- what a pass cannot do without -------------------------------------------------------------------


def work(case):
    op = case["op"]
    if op == "quant":
        n, size = case["rows"] * case["cols"], SIZE[case["type"]]
        read = min(case["rows"], case["source"]) * case["cols"] * size + (4 * case["rows"] if case["gather"] else 0)
        return {"bytes": read + n * 17 // 32 + n * size, "flops": 2 * n}
    if op == "product":
        rows, cols, tokens = case["rows"], case["cols"], case["tokens"]
        return {"bytes": (rows + tokens) * cols * 17 // 32 + rows * tokens * SIZE[case["out"]],
                "flops": 2 * rows * cols * tokens}
    if op == "experts":
        rows, cols, n, k = case["rows"], case["cols"], case["experts"], case["top_k"]
        pairs = case["tokens"] * k
        touched = n * (1 - (1 - k / n) ** case["tokens"])
        return {"bytes": (touched * rows + pairs) * cols * 17 / 32 + pairs * rows * SIZE[case["out"]],
                "flops": 2 * pairs * rows * cols}
    size, width, tokens = SIZE[case["type"]], case["width"], case["tokens"]
    pairs = tokens * case["top_k"]
    moved = 2 * (tokens + pairs) * width * size + 4 * (4 * pairs + case["experts"])
    flops = 2 * pairs * width
    if case["train"]:
        moved += (2 * tokens + 3 * pairs) * width * size + 4 * pairs
        flops += 4 * pairs * width
    return {"bytes": moved, "flops": flops}


# --- the definition in 64 bits -------------------------------------------------------------------------


def _two_to(n):
    """2^n as a double, by its bits (pow() on the GPU may be an ulp off, which would break ties)."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _exact_values(buf, rows, cols):
    """The buffer's values from the format's definition: sign, exponent and mantissa of a code, a power of two a group."""
    byte = buf[: rows * cols // 2].reshape(rows, -1).long()
    code = torch.empty(rows, cols, dtype=torch.int64, device=buf.device)
    code[:, 0::2], code[:, 1::2] = byte % 16, byte // 16
    sign, exponent, mantissa = 1.0 - 2.0 * (code // 8), (code // 2) % 4, (code % 2).double()
    v = sign * torch.where(exponent == 0, 0.5 * mantissa, (1 + 0.5 * mantissa) * _two_to(exponent - 1))
    k = buf[rows * cols // 2: rows * cols * 17 // 32].reshape(rows, -1).long()
    return v * _two_to(k - 127).repeat_interleave(32, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        x = s["x"].double()
        x = x if s["row_of"] is None else x[s["row_of"].long()]
        g = x.reshape(x.shape[0], -1, 32)
        top = g.abs().amax(-1, keepdim=True)
        _, e = torch.frexp(top)  # top = m 2^e, 0.5 <= m < 1: floor(log2 top) = e - 1
        scale = _two_to(torch.where(top > 0, e - 3, -127).clamp(min=-127))
        a = (g / scale).abs().clamp(max=6.0)
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
        v = torch.round(a / step) * step  # torch.round is to even
        return {"values": (torch.where(g < 0, -v, v) * scale).reshape(x.shape)}
    if op == "product":
        w, x = _exact_values(s["w"], case["rows"], case["cols"]), _exact_values(s["x"], case["tokens"], case["cols"])
        return {"y": x @ w.T}
    if op == "experts":
        cols, pairs = case["cols"], case["tokens"] * case["top_k"]
        x, off = _exact_values(s["x"], pairs, cols), s["offsets"].tolist()
        y = torch.zeros(pairs, case["rows"], dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            if off[e + 1] > off[e]:
                y[off[e]: off[e + 1]] = x[off[e]: off[e + 1]] @ _exact_values(s["bank"][e], case["rows"], cols).T
        return {"y": y}
    tokens, top_k, width, n = case["tokens"], case["top_k"], case["width"], case["experts"]
    ids = s["ids"].reshape(-1).tolist()
    order = sorted((p for p in range(len(ids)) if 0 <= ids[p] < n), key=lambda p: (ids[p], p))
    token_at = torch.full((len(ids),), -1, dtype=torch.int32)
    pos_of = torch.full((len(ids),), -1, dtype=torch.int32)
    pair = torch.tensor(order, dtype=torch.long)
    token_at[: len(order)] = (pair // top_k).int()
    pos_of[pair] = torch.arange(len(order), dtype=torch.int32)
    count = [0] * (n + 1)
    for p in order:
        count[ids[p] + 1] += 1
    offsets = torch.tensor(count).cumsum(0).int()
    pair, t, m = pair.cuda(), (pair // top_k).cuda(), len(order)
    w = s["weights"].double().reshape(-1)[pair].unsqueeze(-1)
    o = s["o"][:m].double()
    xs = torch.zeros(len(ids), width, dtype=torch.float64, device="cuda")
    xs[:m] = s["x"].double()[t]
    y = torch.zeros(tokens, width, dtype=torch.float64, device="cuda").index_add_(0, t, w * o)
    out = {"token_at": token_at, "pos_of": pos_of, "offsets": offsets, "xs": xs, "y": y}
    if case["train"]:
        dy = s["dy"].double()[t]
        out["do"] = torch.zeros_like(xs)
        out["do"][:m] = w * dy
        out["dweights"] = torch.zeros(len(ids), dtype=torch.float64, device="cuda").index_add_(0, pair, (dy * o).sum(-1)).reshape(tokens, top_k)
        out["dx"] = torch.zeros_like(y).index_add_(0, t, s["dxs"][:m].double())
    return out
