"""The operators of the microscaled 4-bit path and of expert routing: what is
measured, on which sizes, and their plain forms.

Kinds of case:
  quantize  rows of activations or weights to 4-bit elements (sign, 2 exponent
            bits, 1 mantissa bit) with one power-of-two scale for every 32,
            optionally behind the sign flips and the 128-point Hadamard
            rotation, and back to values (what a calibration looks at);
  linear    a layer: its activations are rotated and quantised, then multiplied
            with 4-bit weights;
  product   the product of two operands that are 4-bit already;
  experts   tokens sorted by expert, quantised into that order, each expert's
            product, and the results brought back with the router's weights;
  route     tokens sorted by expert, copied into that order, and back with
            weights;
  grad      the gradients of `route`: of the tokens, of the experts' outputs
            and of the weights.

Layout of a 4-bit operand with r rows of k values (k along the sum): codes
uint8 [r, k/2], the element of even index in the low half of its byte; scales
uint8 [r, 16 ceil(k/512)], byte b the exponent (plus 127) of elements 32b ..
32b + 31, the bytes behind k/32 unused.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # a prompt's activations in front of a layer of the 70B shapes
        {"name": "quantize_prompt", "op": "quantize", "rows": 2048, "k": 8192, "dtype": "f16", "rotate": True},
        # a layer's weights (8B gate/up, one row per output channel) when a model is loaded
        {"name": "quantize_weights", "op": "quantize", "rows": 14336, "k": 4096, "dtype": "f32", "rotate": False},
        # one token through the 8B query layer
        {"name": "linear_token", "op": "linear", "m": 1, "k": 4096, "n": 4096, "dtype": "f16"},
        # a prompt through the 70B gate/up layer
        {"name": "linear_prompt", "op": "linear", "m": 2048, "k": 8192, "n": 28672, "dtype": "f16"},
        # 32 sequences, one token each, through the 70B gate/up layer, already quantised
        {"name": "product_batch", "op": "product", "m": 32, "k": 8192, "n": 28672, "dtype": "f16"},
        # sizes that fill no tile: a short prompt, a head of an odd width, k in the middle of a block of scales
        {"name": "product_ragged", "op": "product", "m": 333, "k": 4000, "n": 10001, "dtype": "bf16"},
        # a decoding step of 8 sequences, 2 of 8 experts of the 8B gate/up shape
        {"name": "experts_tokens", "op": "experts", "tokens": 8, "topk": 2, "experts": 8, "k": 4096, "n": 14336, "dtype": "f16", "pad": 0},
        # a prompt over many smaller experts, some of its tokens padding
        {"name": "experts_prompt", "op": "experts", "tokens": 4096, "topk": 4, "experts": 32, "k": 4096, "n": 2048, "dtype": "bf16", "pad": 100},
        # a decoding step: sorting and moving a handful of rows
        {"name": "route_tokens", "op": "route", "tokens": 8, "topk": 8, "experts": 128, "h": 4096, "dtype": "f16", "pad": 0},
        # a long prompt over many experts
        {"name": "route_prompt", "op": "route", "tokens": 8192, "topk": 8, "experts": 128, "h": 4096, "dtype": "bf16", "pad": 192},
        # a training step's gradients over a long batch
        {"name": "grad_prompt", "op": "grad", "tokens": 4096, "topk": 4, "experts": 32, "h": 4096, "dtype": "bf16", "pad": 96},
        # a small one, rows of an odd width
        {"name": "grad_ragged", "op": "grad", "tokens": 1001, "topk": 2, "experts": 8, "h": 1111, "dtype": "f32", "pad": 5},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["quantize", "linear", "product", "experts", "route", "grad"])
    half = rng.choice(["f16", "bf16"])
    any3 = rng.choice(["f16", "bf16", "f32"])
    if op == "quantize":
        rotate = rng.random() < 0.6
        k = 128 * log(1, 64) if rotate else 32 * log(1, 256)
        return {"op": op, "rows": log(1, 4096), "k": k, "dtype": any3, "rotate": rotate}
    if op == "linear":
        return {"op": op, "m": log(1, 2048), "k": 128 * log(1, 64), "n": log(16, 16384), "dtype": half}
    if op == "product":
        return {"op": op, "m": log(1, 2048), "k": 32 * log(1, 256), "n": log(1, 16384), "dtype": half}
    experts = log(2, 64)
    topk = rng.randint(1, min(8, experts))
    if op == "experts":
        tokens = log(1, 2048)
        return {"op": op, "tokens": tokens, "topk": topk, "experts": experts, "k": 128 * log(1, 32), "n": log(16, 2048),
                "dtype": half, "pad": rng.choice([0, tokens // 16])}
    tokens = log(1, 8192 if op == "route" else 4096)
    return {"op": op, "tokens": tokens, "topk": topk, "experts": experts, "h": log(1, 4096), "dtype": any3,
            "pad": rng.choice([0, tokens // 16])}


# ---------------------------------------------------------------- inputs ---

def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _activations(g, rows, k, dtype):
    """Normal values with one channel in a hundred larger, as activations have."""
    x = torch.randn((rows, k), generator=g, device="cuda", dtype=torch.float32)
    loud = torch.rand((k,), generator=g, device="cuda") < 0.01
    return torch.where(loud, 20.0 * x, x).to(dtype)


def _signs(g, k):
    return (torch.randint(0, 2, (k,), generator=g, device="cuda") * 2 - 1).to(torch.float16)


def _weights(g, rows, k):
    """A 4-bit operand from normal weights, made in parts of 64 Mi values."""
    codes = torch.empty((rows, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((rows, 16 * ((k + 511) // 512)), dtype=torch.uint8, device="cuda")
    part = max(1, (1 << 26) // k)
    for r in range(0, rows, part):
        w = _normal(g, (min(part, rows - r), k), torch.float32, 0.02)
        codes[r:r + part], scales[r:r + part] = _pack(*_plain_quantize(w, None, False))
    return codes, scales


def _routing(g, case):
    """Each token's distinct experts, some chosen more often than others, and
    the router's weights; `pad` tokens at the end are padding (expert -1)."""
    t, e, k = case["tokens"], case["experts"], case["topk"]
    liking = torch.randn((e,), generator=g, device="cuda")
    logits = torch.randn((t, e), generator=g, device="cuda") + liking
    top, ids = torch.topk(logits, k, dim=1)
    ids = ids.to(torch.int32)
    if case["pad"]:
        ids[t - case["pad"]:] = -1
    return ids.contiguous(), torch.softmax(top, dim=1).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, dtype = case["op"], DTYPES[case["dtype"]]
    s = {"case": dict(case)}
    if op == "quantize":
        s["x"] = _activations(g, case["rows"], case["k"], dtype) if dtype != torch.float32 else _normal(g, (case["rows"], case["k"]), dtype, 0.02)
        s["signs"] = _signs(g, case["k"]) if case["rotate"] else None
        return s
    # scratch memory that a program keeps for all of its calls
    s["workspace"] = torch.zeros(96 << 20, dtype=torch.uint8, device="cuda")
    if op in ("linear", "product"):
        m, k, n = case["m"], case["k"], case["n"]
        s["w"], s["ws"] = _weights(g, n, k)
        x = _activations(g, m, k, dtype)
        if op == "linear":
            s["x"], s["signs"] = x, _signs(g, k)
        else:
            s["xc"], s["xs"] = _pack(*_plain_quantize(x.float(), None, False))
        return s
    t, e, topk = case["tokens"], case["experts"], case["topk"]
    s["ids"], s["weights"] = _routing(g, case)
    if op == "experts":
        k, n = case["k"], case["n"]
        s["x"], s["signs"] = _activations(g, t, k, dtype), _signs(g, k)
        w, ws = _weights(g, e * n, k)
        s["w"], s["ws"] = w.view(e, n, -1), ws.view(e, n, -1)
        # rows of the fullest expert: the plain form pads every expert to it
        s["most"] = int(torch.bincount(s["ids"].flatten().clamp(min=0).long(), minlength=e).max())
        return s
    h = case["h"]
    if op == "route":
        s["x"] = _normal(g, (t, h), dtype)
        s["ys"] = _normal(g, (t * topk, h), dtype)
        s["out"] = torch.zeros((t * topk, h), dtype=dtype, device="cuda")
        return s
    s["positions"] = _plain_sort(s["ids"], e)[1]
    s["dy"] = _normal(g, (t, h), dtype)
    s["ys"] = _normal(g, (t * topk, h), dtype)
    s["dxs"] = _normal(g, (t * topk, h), dtype)
    s["out"] = torch.zeros((t * topk, h), dtype=dtype, device="cuda")
    return s


# ----------------------------------------------------------- plain forms ---

def _plain_rotate(x, signs):
    """H128(x .* signs)/sqrt(128) for every 128 values, in 64 bits: a value
    next to a border of the 4-bit rounding must not cross it."""
    rows, k = x.shape
    v = (x.double() * signs.double()).view(rows, k // 128, 128)
    v = v.view(-1, 128)
    h = 1
    while h < 128:
        v = v.view(-1, 128 // (2 * h), 2, h)
        v = torch.stack((v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]), dim=2)
        h *= 2
    return v.reshape(rows, k) * (1.0 / math.sqrt(128.0))


def _plain_quantize(x, signs, rotate):
    """Codes [r, k] (0..15) and exponent bytes [r, k/32]: the scale is 2 to the
    power floor(log2(largest magnitude)) - 2, elements round to nearest (ties
    to the even code) and saturate at 6."""
    v = _plain_rotate(x, signs) if rotate else x.float()
    b = v.view(v.shape[0], -1, 32)
    amax = b.abs().amax(dim=2)
    e = torch.frexp(amax)[1].long() - 1
    byte = torch.where(amax > 0, (e + 125).clamp(0, 254), torch.zeros_like(e))
    inv = ((1023 + 127 - byte) << 52).view(torch.float64)
    r = b.abs().double() * inv[:, :, None]
    code = (r > 0.25).to(torch.uint8)
    code += r >= 0.75
    code += r > 1.25
    code += r >= 1.75
    code += r > 2.5
    code += r >= 3.5
    code += r > 5.0
    code += 8 * torch.signbit(b).to(torch.uint8)
    return code.view(v.shape), byte.to(torch.uint8)


def _pack(code, byte):
    pairs = code.view(code.shape[0], -1, 2)
    scales = torch.zeros((code.shape[0], 16 * ((code.shape[1] + 511) // 512)), dtype=torch.uint8, device=code.device)
    scales[:, :byte.shape[1]] = byte
    return pairs[:, :, 0] | (pairs[:, :, 1] << 4), scales


def _table(device):
    return torch.tensor(MAGNITUDES + tuple(-v for v in MAGNITUDES), dtype=torch.float32, device=device)


def _plain_values(code, byte):
    """The fp32 values of codes and their exponent bytes."""
    scale = ((byte.long() + (1023 - 127)) << 52).view(torch.float64).float()
    v = _table(code.device)[code.int()].view(code.shape[0], -1, 32) * scale[:, :, None]
    return v.view(code.shape)


def _plain_unpack(codes, scales):
    k = codes.shape[-1] * 2
    codes, scales = codes.reshape(-1, k // 2), scales.reshape(-1, scales.shape[-1])
    code = torch.stack((codes & 15, codes >> 4), dim=2).view(-1, k)
    return _plain_values(code, scales[:, :k // 32])


def _plain_sort(ids, experts):
    """Where each expert's rows begin, and the row of each (token, choice)."""
    flat = ids.flatten().long()
    chosen = flat >= 0
    key = torch.where(chosen, flat, torch.full_like(flat, experts))
    order = torch.sort(key, stable=True)[1]
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    counts = torch.zeros(experts + 1, dtype=torch.long, device=ids.device).index_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.cumsum(counts[:experts], 0)
    positions = torch.where(chosen, place, torch.full_like(place, -1)).to(torch.int32)
    return offsets, positions.view(ids.shape)


def _plain_scatter(rows, positions, out):
    """out[positions[i]] = rows[i] where the position is not -1 (one more row
    takes those that are)."""
    p = positions.flatten().long()
    wide = torch.cat((out, out[:1]))
    wide[torch.where(p >= 0, p, torch.full_like(p, out.shape[0]))] = rows
    out.copy_(wide[:-1])
    return out


def _plain_combine(ys, positions, weights):
    """y[t] = sum over j of weights[t, j] ys[positions[t, j]], in 32 bits."""
    rows = ys[positions.clamp(min=0).long()].float()
    w = (positions >= 0).float() if weights is None else torch.where(positions >= 0, weights, torch.zeros_like(weights))
    rows = torch.where((positions >= 0)[:, :, None], rows, torch.zeros_like(rows))
    return (w[:, :, None] * rows).sum(dim=1).to(ys.dtype)


def _plain_experts(s, dtype):
    case = s["case"]
    e, n = case["experts"], case["n"]
    offsets, positions = _plain_sort(s["ids"], e)
    x = _plain_values(*_plain_quantize(s["x"], s["signs"], True))
    w = _plain_unpack(s["w"], s["ws"]).view(e, n, -1)
    # each (token, choice) in its expert's block of `most` rows
    ids = s["ids"].flatten().long()
    p = positions.flatten().long()
    spare = e * s["most"]
    slot = torch.where(ids >= 0, ids * s["most"] + p - offsets.long()[ids.clamp(min=0)], torch.full_like(ids, spare))
    padded = torch.zeros((spare + 1, case["k"]), dtype=torch.float32, device=x.device)
    padded[slot] = x.repeat_interleave(case["topk"], dim=0)
    y = torch.bmm(padded[:-1].view(e, s["most"], -1), w.transpose(1, 2)).view(spare, n)
    y = torch.where((ids >= 0)[:, None], y[slot.clamp(max=spare - 1)], torch.zeros_like(y[:1]))
    y = (y.view(case["tokens"], case["topk"], n) * s["weights"][:, :, None]).sum(dim=1)
    return {"offsets": offsets, "positions": positions, "y": y.to(dtype)}


def _run_plain(s):
    case = s["case"]
    op, dtype = case["op"], DTYPES[case["dtype"]]
    if op == "quantize":
        codes, scales = _pack(*_plain_quantize(s["x"], s["signs"], case["rotate"]))
        return _plain_unpack(codes, scales).to(dtype)
    if op == "linear":
        x = _plain_values(*_plain_quantize(s["x"], s["signs"], True))
        return (x @ _plain_unpack(s["w"], s["ws"]).t()).to(dtype)
    if op == "product":
        return (_plain_unpack(s["xc"], s["xs"]) @ _plain_unpack(s["w"], s["ws"]).t()).to(dtype)
    if op == "experts":
        return _plain_experts(s, dtype)
    if op == "route":
        offsets, positions = _plain_sort(s["ids"], case["experts"])
        xs = _plain_scatter(s["x"].repeat_interleave(case["topk"], dim=0), positions, s["out"])
        return {"offsets": offsets, "positions": positions, "xs": xs, "y": _plain_combine(s["ys"], positions, s["weights"])}
    p, w = s["positions"], s["weights"]
    dys = _plain_scatter((w[:, :, None] * s["dy"].float()[:, None, :]).flatten(0, 1).to(dtype), p, s["out"])
    rows = torch.where((p >= 0)[:, :, None], s["ys"][p.clamp(min=0).long()].float(), torch.zeros((), device="cuda"))
    dw = (rows * s["dy"].float()[:, None, :]).sum(dim=2)
    return {"dys": dys, "dw": dw, "dx": _plain_combine(s["dxs"], p, None)}


def _run_own(s):
    from trellis_coded_bit_b200 import exl3

    case = s["case"]
    op, dtype = case["op"], DTYPES[case["dtype"]]
    if op == "quantize":
        codes, scales = exl3.exl3_mx4_quantize(s["x"], signs=s["signs"], rotate=case["rotate"])
        return exl3.exl3_mx4_dequantize(codes, scales, dtype=dtype)
    if op == "linear":
        return exl3.exl3_mx4_linear(s["x"], s["w"], s["ws"], signs=s["signs"], rotate=True, workspace=s["workspace"])
    if op == "product":
        return exl3.exl3_mx4_matmul(s["xc"], s["xs"], s["w"], s["ws"], dtype=dtype, workspace=s["workspace"])
    if op == "experts":
        rows = case["tokens"] * case["topk"]
        offsets, positions = exl3.exl3_moe_sort(s["ids"], case["experts"], workspace=s["workspace"])
        xc, xs = exl3.exl3_mx4_quantize(s["x"], signs=s["signs"], rotate=True, positions=positions, out_rows=rows)
        # fp32 rows, so that the weighted sum is rounded once
        ys = exl3.exl3_mx4_matmul_experts(xc, xs, offsets, s["w"], s["ws"], dtype=torch.float32, workspace=s["workspace"])
        y = exl3.exl3_moe_combine(ys, positions, weights=s["weights"], dtype=dtype)
        return {"offsets": offsets, "positions": positions, "y": y}
    if op == "route":
        offsets, positions = exl3.exl3_moe_sort(s["ids"], case["experts"], workspace=s["workspace"])
        xs = exl3.exl3_moe_gather(s["x"], positions, out=s["out"])
        return {"offsets": offsets, "positions": positions, "xs": xs, "y": exl3.exl3_moe_combine(s["ys"], positions, weights=s["weights"])}
    dys, dw = exl3.exl3_moe_combine_grad(s["dy"], s["ys"], s["positions"], s["weights"], dys=s["out"])
    return {"dys": dys, "dw": dw, "dx": exl3.exl3_moe_combine(s["dxs"], s["positions"])}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------- 64 bits ---

def _exact_values(x, signs, rotate):
    """Quantised values from the definition: rotation as a product with the
    Hadamard matrix, elements rounded on the grid of their binade."""
    v = x.double()
    rows, k = v.shape
    if rotate:
        i = torch.arange(128, device=x.device)
        both = i[:, None] & i[None, :]
        ones = sum((both >> b) & 1 for b in range(7))
        hadamard = 1.0 - 2.0 * (ones % 2).double()
        v = ((v * signs.double()).view(-1, 128) @ hadamard / math.sqrt(128.0)).view(rows, k)
    b = v.view(rows, k // 32, 32)
    amax = b.abs().amax(dim=2, keepdim=True)
    scale = torch.exp2((torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax)))) - 2).round())
    # log2 of a value just below a power of two may round up to it
    scale = torch.where(scale * 4 > amax, scale / 2, scale)
    scale = torch.where(scale * 8 <= amax, scale * 2, scale).clamp(min=2.0 ** -127)
    r = b / scale
    grid = torch.where(r.abs() < 2, 0.5, torch.where(r.abs() < 4, 1.0, 2.0))
    return ((torch.round(r / grid) * grid).clamp(-6, 6) * scale).view(rows, k)


def _exact_operand(codes, scales):
    """Values of a stored operand: sign, exponent and mantissa bits by arithmetic."""
    k = codes.shape[1] * 2
    c = torch.stack((codes % 16, codes // 16), dim=2).view(-1, k).double()
    sign = torch.where(c >= 8, -1.0, 1.0)
    c = c % 8
    exponent, mantissa = torch.floor(c / 2), c % 2
    v = torch.where(exponent > 0, (1 + mantissa / 2) * torch.exp2(exponent - 1), mantissa / 2)
    scale = torch.exp2(scales[:, :k // 32].double() - 127).repeat_interleave(32, dim=1)
    return sign * v * scale


def _exact_route(ids, experts):
    """Offsets and positions by counting: how many earlier choices come first."""
    flat = ids.flatten().tolist()
    counts = [0] * experts
    for e in flat:
        if e >= 0:
            counts[e] += 1
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    following, positions = list(offsets), []
    for e in flat:
        positions.append(following[e] if e >= 0 else -1)
        if e >= 0:
            following[e] += 1
    return (torch.tensor(offsets, dtype=torch.int32, device="cuda"),
            torch.tensor(positions, dtype=torch.int32, device="cuda").view(ids.shape))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_values(s["x"], s["signs"], case["rotate"])
    if op in ("linear", "product"):
        x = _exact_values(s["x"], s["signs"], True) if op == "linear" else _exact_operand(s["xc"], s["xs"])
        y = torch.empty((case["m"], case["n"]), dtype=torch.float64, device="cuda")
        for i in range(0, case["n"], 4096):
            y[:, i:i + 4096] = x @ _exact_operand(s["w"][i:i + 4096], s["ws"][i:i + 4096]).t()
        return y
    topk = case["topk"]
    if op == "experts":
        offsets, positions = _exact_route(s["ids"], case["experts"])
        x = _exact_values(s["x"], s["signs"], True)
        y = torch.zeros((case["tokens"], case["n"]), dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            at = (s["ids"] == e).nonzero()
            if len(at):
                part = x[at[:, 0]] @ _exact_operand(s["w"][e], s["ws"][e]).t()
                y.index_add_(0, at[:, 0], part * s["weights"][at[:, 0], at[:, 1]].double()[:, None])
        return {"offsets": offsets, "positions": positions, "y": y}
    offsets, positions = (None, s["positions"]) if op == "grad" else _exact_route(s["ids"], case["experts"])
    t, h = case["tokens"], case["h"]
    first, second = torch.zeros((t * topk, h), dtype=torch.float64, device="cuda"), torch.zeros((t, h), dtype=torch.float64, device="cuda")
    dw = torch.zeros((t, topk), dtype=torch.float64, device="cuda")
    w = s["weights"].double()
    for j in range(topk):
        has = (positions[:, j] >= 0).nonzero()[:, 0]
        p = positions[has, j].long()
        if op == "route":
            first[p] = s["x"][has].double()
            second[has] += w[has, j, None] * s["ys"][p].double()
        else:
            first[p] = w[has, j, None] * s["dy"][has].double()
            second[has] += s["dxs"][p].double()
            dw[has, j] = (s["dy"][has].double() * s["ys"][p].double()).sum(dim=1)
    if op == "route":
        return {"offsets": offsets, "positions": positions, "xs": first, "y": second}
    return {"dys": first, "dw": dw, "dx": second}


def work(case):
    """Bytes: inputs read once, outputs written once (a 4-bit operand is k/2 +
    k/32 bytes a row). Operations: 2 per product term, 7 additions per rotated
    value, 2 per term of a weighted sum."""
    op, size = case["op"], {"f16": 2, "bf16": 2, "f32": 4}[case["dtype"]]

    def four(rows, k):
        return rows * (k // 2 + k // 32)

    if op == "quantize":
        r, k = case["rows"], case["k"]
        return {"bytes": 2 * r * k * size + 2 * four(r, k), "flops": r * k * (7 if case["rotate"] else 1)}
    if op in ("linear", "product"):
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": (m * k * size if op == "linear" else four(m, k)) + four(n, k) + m * n * size, "flops": 2 * m * k * n}
    t, topk, e = case["tokens"], case["topk"], case["experts"]
    used = (t - case["pad"]) * topk
    if op == "experts":
        k, n = case["k"], case["n"]
        return {"bytes": t * k * size + min(e, used) * four(n, k) + t * n * size + 8 * t * topk, "flops": 2 * used * k * n}
    h = case["h"]
    if op == "route":
        return {"bytes": (2 * t + 2 * used) * h * size + 12 * t * topk, "flops": 2 * used * h}
    return {"bytes": (2 * t + 3 * used) * h * size + 12 * t * topk, "flops": 4 * used * h}
