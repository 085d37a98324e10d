"""The 8-bit linear layer and the optimizer step: what is measured of them.

Three operators, as a training or a serving program calls them:
  quantize   a matrix to 8-bit integers with one scale for each row and / or each column
  product    the 8-bit product with scales for each token and channel: on held codes ("product"), with
             the tokens quantized on the way ("serve"), and a training step of the layer ("train")
  adamw      an AdamW step over all tensors of a model, states in 32 bits or in 8
"""

import math

import numpy as np
import torch

own = False

BLOCK = 128                # elements of a tensor that share one exponent of an 8-bit state
LR, BETA1, BETA2, EPS, DECAY = 3e-4, 0.9, 0.95, 1e-8, 0.1


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # activations of one layer before a forward product: a scale for each token
        dict(name="quantize tokens", op="quantize", rows=8192, cols=4096, dtype="bf16", sides="row"),
        # a master weight at the start of a training step: both products that read it
        dict(name="quantize weight", op="quantize", rows=4096, cols=14336, dtype="f32", sides="both"),
        # a gradient of a ragged batch and an odd width
        dict(name="quantize ragged", op="quantize", rows=1001, cols=1333, dtype="bf16", sides="both"),
        # one token of one request, the up-projection
        dict(name="serve one token", op="serve", l=1, m=4096, n=14336, out="bf16"),
        # a decoding step of some forty requests, an attention projection
        dict(name="serve forty tokens", op="serve", l=40, m=4096, n=4096, out="bf16"),
        # a long prompt, the up-projection: the largest product
        dict(name="serve prompt", op="serve", l=8192, m=4096, n=14336, out="bf16"),
        # codes already at hand, odd sizes, fp32 result
        dict(name="product ragged", op="product", l=515, m=1000, n=1333, out="f32"),
        # forward and both gradients of a layer at 8192 tokens
        dict(name="train step", op="train", l=8192, m=4096, n=4096),
        # the same of a small layer and a short batch, where launches count
        dict(name="train small", op="train", l=512, m=768, n=2304),
        # one block of the large model, states in 32 bits
        dict(name="adamw 32 bits", op="adamw", bits=32, blocks=1, hidden=4096, ffn=14336, dtype="f32", rounding="rn"),
        # a small model of twelve blocks (120 tensors), states in 8 bits, stochastic rounding
        dict(name="adamw 8 bits", op="adamw", bits=8, blocks=12, hidden=768, ffn=2304, dtype="f32", rounding="sr"),
        # a few odd bf16 tensors: the latency of a step
        dict(name="adamw 8 bits ragged", op="adamw", bits=8, blocks=2, hidden=257, ffn=701, dtype="bf16", rounding="rn"),
    ]


def _between(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["quantize", "quantize", "serve", "serve", "product", "train", "adamw", "adamw"])
    if op == "quantize":
        while True:
            rows, cols = _between(rng, 1, 16384), _between(rng, 1, 16384)
            if rows * cols <= 4096 * 14336:
                return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "f32"]),
                            sides=rng.choice(["row", "col", "both"]))
    if op == "adamw":
        while True:
            blocks, hidden, ffn = _between(rng, 1, 32), _between(rng, 16, 4096), _between(rng, 16, 14336)
            dtype, bits = rng.choice(["f32", "bf16"]), rng.choice([8, 32])
            if blocks * (4 * hidden + 2 * ffn) * hidden <= 5 * 10 ** 7:
                return dict(op=op, bits=bits, blocks=blocks, hidden=hidden, ffn=ffn, dtype=dtype,
                            rounding=rng.choice(["rn", "sr"]))
    while True:
        l, m, n = _between(rng, 1, 16384), _between(rng, 16, 14336), _between(rng, 16, 14336)
        if op == "train" and l * m * n <= 8192 * 4096 * 4096:
            return dict(op=op, l=l, m=m, n=n)
        if op != "train" and l * m * n <= 8192 * 4096 * 14336:
            return dict(op=op, l=l, m=m, n=n, out=rng.choice(["bf16", "f32"]))


def _shapes(case):
    h, f = case["hidden"], case["ffn"]
    return ([(h, h)] * 4 + [(h, f), (f, h)] + [(h,)] * 4) * case["blocks"]


def work(case):
    op = case["op"]
    if op == "quantize":
        n, sides = case["rows"] * case["cols"], 2 if case["sides"] == "both" else 1
        lines = (case["rows"] if case["sides"] != "col" else 0) + (case["cols"] if case["sides"] != "row" else 0)
        return {"bytes": n * ((2 if case["dtype"] == "bf16" else 4) + sides) + 4 * lines, "flops": 3 * n * sides}
    if op == "adamw":
        n = sum(math.prod(s) for s in _shapes(case))
        size = 2 if case["dtype"] == "bf16" else 4
        state = 16 if case["bits"] == 32 else 4 + 4 / BLOCK
        return {"bytes": n * (3 * size + state), "flops": 14 * n}
    l, m, n = case["l"], case["m"], case["n"]
    if op == "train":   # x, w, dy in; y, dx, dw out
        return {"bytes": 4 * l * m + 8 * m * n + 4 * l * n, "flops": 6 * l * m * n}
    read = l * m + 4 * l if op == "product" else 2 * l * m
    return {"bytes": read + m * n + 4 * n + l * n * (2 if case["out"] == "bf16" else 4), "flops": 2 * l * m * n}


# ---------------------------------------------------------------------------- inputs
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _activations(rows, cols, gen):
    """Normal entries, one column in fifty an outlier channel, some rows of zeros (padding)."""
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    x *= 1 + 20 * (torch.rand(cols, device="cuda", generator=gen) < 0.02)
    if rows > 8:
        x *= torch.rand(rows, 1, device="cuda", generator=gen) > 0.03
    return x


def _held(n, m, gen):
    """Codes and channel scales of a held weight, rows padded to 16 bytes as the operands' layout wants it."""
    ld = -(-m // 16) * 16
    buf = torch.randint(-127, 128, (n, ld), device="cuda", generator=gen, dtype=torch.int8)
    scales = (0.5 + torch.rand(n, device="cuda", generator=gen)) / (127 * math.sqrt(m))
    return buf[:, :m], scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, s = case["op"], dict(case)
    if op == "quantize":
        s["M"] = _activations(case["rows"], case["cols"], gen).to(_dtype(case["dtype"]))
        if own:
            s["ctx"] = _context()
            s["row"] = s["ctx"].new_int8(case["rows"], case["cols"]) if case["sides"] != "col" else None
            s["col"] = s["ctx"].new_int8(case["cols"], case["rows"]) if case["sides"] != "row" else None
    elif op in ("serve", "product"):
        l, m, n = case["l"], case["m"], case["n"]
        s["w"], s["sw"] = _held(n, m, gen)
        if op == "serve":
            s["x"] = _activations(l, m, gen).to(torch.bfloat16)
        else:
            s["a"], s["sa"] = _held(l, m, gen)
        if own:
            import spectral_quantized_gemm_b200 as sq
            s["ctx"] = _context()
            s["W"] = sq.Int8(n, m, codes=s["w"], scales=s["sw"])
            s["A"] = sq.Int8(l, m, codes=s["a"], scales=s["sa"]) if op == "product" else s["ctx"].new_int8(l, m)
            size = 8 if case["out"] == "bf16" else 4   # rows of the result start on 16 bytes
            s["y"] = torch.empty(l, -(-n // size) * size, dtype=_dtype(case["out"]), device="cuda")[:, :n]
    elif op == "train":
        l, m, n = case["l"], case["m"], case["n"]
        s["x"] = _activations(l, m, gen).to(torch.bfloat16)
        s["dy"] = (1e-4 * _activations(l, n, gen)).to(torch.bfloat16)
        s["w"] = (2 * torch.rand(m, n, device="cuda", generator=gen) - 1) / math.sqrt(m)
        if own:
            from spectral_quantized_gemm_b200.int8_linear import Int8Linear
            s["layer"] = Int8Linear(m, n, device="cuda")
            with torch.no_grad():
                s["layer"].weight.copy_(s["w"])
            s["x"].requires_grad_(True)
    else:
        _prepare_adamw(case, s, gen)
    return s


def _context():
    import spectral_quantized_gemm_b200 as sq
    return sq.Context()


def _prepare_adamw(case, s, gen):
    """All tensors as views of flat buffers, each at a multiple of BLOCK elements; the rest is zero and stays so.
    The states are those of a run in its hundredth step; some elements never had a gradient."""
    dtype = _dtype(case["dtype"])
    at, spans = 0, []
    for shape in _shapes(case):
        n = math.prod(shape)
        spans.append((at, n, shape))
        at += -(-n // BLOCK) * BLOCK
    live, scale = torch.zeros(at, device="cuda"), torch.zeros(at, device="cuda")
    for i, (a, n, _) in enumerate(spans):
        live[a:a + n] = 1
        scale[a:a + n] = 10.0 ** -(2 + i % 4)
    live *= torch.rand(at, device="cuda", generator=gen) > 0.02
    scale *= live

    def normal():
        return torch.randn(at, device="cuda", generator=gen)

    s["p"] = (0.02 * normal() * (live > 0)).to(dtype)
    s["g"] = (scale * normal()).to(dtype)
    m = 0.3 * scale * normal()
    v = (scale * (0.3 + normal().abs())) ** 2
    s["step"] = 100
    if case["bits"] == 8:
        s["m"], s["me"] = _encode_signed(m.double(), None)
        s["v"], s["ve"] = _encode_positive(v.double(), None)
    else:
        s["m"], s["v"] = m, v
    # where every group of four elements stands: its tensor and its place in it
    s["tensor"] = torch.zeros(at // 4, dtype=torch.int64, device="cuda")
    s["place"] = torch.zeros(at // 4, dtype=torch.int64, device="cuda")
    for i, (a, n, _) in enumerate(spans):
        e = a + -(-n // BLOCK) * BLOCK
        s["tensor"][a // 4:e // 4] = i
        s["place"][a // 4:e // 4] = torch.arange((e - a) // 4, device="cuda")
    if not own:
        return
    from spectral_quantized_gemm_b200.optim import AdamW
    # the calls step the same elements as the plain form: a tensor's whole span of the flat buffers, the rest of
    # its last BLOCK included, whose outputs are compared too
    spans = [(a, a + -(-n // BLOCK) * BLOCK) for a, n, _ in spans]
    params = [torch.nn.Parameter(s["p"][a:e]) for a, e in spans]
    opt = AdamW(params, lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY, state_bits=case["bits"],
                rounding=case["rounding"], seed=_seed(case))
    for p, (a, e) in zip(params, spans):
        p.grad = s["g"][a:e]
        st = {"step": s["step"], "exp_avg": s["m"][a:e], "exp_avg_sq": s["v"][a:e]}
        if case["bits"] == 8:
            st["exp_avg_exponent"], st["exp_avg_sq_exponent"] = s["me"][a // BLOCK:e // BLOCK], s["ve"][a // BLOCK:e // BLOCK]
        opt.state[p] = st
    s["opt"] = opt


def _seed(case):
    return 77 + case["hidden"]


# ---------------------------------------------------------------------------- one pass
def run(s):
    return {"quantize": _run_quantize, "serve": _run_product, "product": _run_product, "train": _run_train,
            "adamw": _run_adamw}[s["op"]](s)


def _run_quantize(s):
    if own:
        s["ctx"].quantize_int8(s["M"], rowwise=s["row"], colwise=s["col"])
        return [(q.codes, q.scales) for q in (s["row"], s["col"]) if q is not None]
    sides = {"row": (0,), "col": (1,), "both": (0, 1)}[s["sides"]]
    return [_quantize(s["M"] if side == 0 else s["M"].t()) for side in sides]


def _quantize(x):
    """Codes and scales for each row. The quotient is taken in 64 bits: a code is decided next to a border."""
    x = x.float()
    a = x.abs().amax(1).clamp_min(127 * 2.0 ** -126)
    codes = torch.round(127 * x.double() / a.double()[:, None]).to(torch.int8)
    return codes, a / 127


def _run_product(s):
    if own:
        if s["op"] == "serve":
            s["ctx"].linear_int8(s["x"], s["A"], s["W"], s["y"])
        else:
            s["ctx"].gemm_int8(s["A"], s["W"], s["y"])
        return s["y"]
    a, sa = _quantize(s["x"]) if s["op"] == "serve" else (s["a"], s["sa"])
    return _product(a, sa, s["w"], s["sw"]).to(_dtype(s["out"]))


def _product(a, sa, b, sb):
    return (a.float() @ b.float().t()) * sa[:, None] * sb[None, :]


def _run_train(s):
    if own:
        y = s["layer"](s["x"])
        dx, dw = torch.autograd.grad(y, (s["x"], s["layer"].weight), s["dy"])
        return {"y": y.detach(), "dx": dx, "dw": dw}
    x, w, dy = s["x"], s["w"], s["dy"]
    y = _product(*_quantize(x), *_quantize(w.t()))                 # over the inputs
    dx = _product(*_quantize(dy), *_quantize(w))                   # over the outputs
    dw = _product(*_quantize(x.t()), *_quantize(dy.t()))           # over the tokens
    return {"y": y.bfloat16(), "dx": dx.bfloat16(), "dw": dw}


def _run_adamw(s):
    # the 8-bit states are returned as their whole numbers, codes and shared exponents: equal or not
    names = ("p", "m", "v", "me", "ve") if s["bits"] == 8 else ("p", "m", "v")
    if own:
        s["opt"].step()
        return {k: s[k] for k in names}
    s["step"] += 1
    t = s["step"]
    if s["bits"] == 8:
        m, v, g = _decode_signed(s["m"], s["me"]), _decode_positive(s["v"], s["ve"]), s["g"].double()
    else:
        m, v, g = s["m"], s["v"], s["g"].float()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * (g * g)
    m32, v32 = m.float(), v.float()
    denom = v32.sqrt() / math.sqrt(1 - BETA2 ** t) + EPS
    p = s["p"].float() * (1 - LR * DECAY) - LR / (1 - BETA1 ** t) * (m32 / denom)
    stochastic = s["rounding"] == "sr"
    if s["bits"] == 8:
        words = _words(s, t, 0) if stochastic else None
        s["m"], s["me"] = _encode_signed(m, words)
        s["v"], s["ve"] = _encode_positive(v, words)
    else:
        s["m"], s["v"] = m32, v32
    if stochastic and s["dtype"] == "bf16":
        bits = (p.view(torch.int32) + (_words(s, t, 1) & 0xFFFF).int()) & -65536
        p = bits.view(torch.float32)
    s["p"] = p.to(_dtype(s["dtype"]))
    return {k: s[k] for k in names}


def _power(k):
    return ((k + 1023) << 52).view(torch.float64)


def _encode(x, words, octaves):
    """Magnitudes (64 bits, in blocks) to 3 bits of mantissa under the block's exponent, gradual underflow:
    the grid's step is 2^(top - octaves - 2) in the lowest two octaves and doubles with each octave above."""
    x = x.view(-1, BLOCK)
    top = (torch.frexp(x.amax(1)).exponent.long() - 1).clamp_(-111, 127)
    octave = (torch.frexp(x).exponent.long() - 1 - (top - octaves + 1)[:, None]).clamp_min_(0)
    t = x / _power((top - octaves - 2)[:, None] + octave)
    if words is None:
        t = torch.round(t)
    else:
        t = torch.floor(t + (words.view(-1, BLOCK).double() + 0.5) / 65536)
    return (t.long() + 8 * octave).clamp_max_(8 * octaves + 7), top


def _encode_signed(m, words):
    code, top = _encode(m.abs(), None if words is None else words & 0xFFFF, 15)
    code += 128 * ((m.view(-1, BLOCK) < 0) & (code > 0))
    return code.view(-1).to(torch.uint8), (top + 127).to(torch.uint8)


def _encode_positive(v, words):
    code, top = _encode(v, None if words is None else words >> 16, 31)
    code = torch.maximum(code, (v.view(-1, BLOCK) > 0).long())   # a positive second moment never becomes zero
    return code.view(-1).to(torch.uint8), (top + 127).to(torch.uint8)


def _decode(code, exponent, octaves):
    code = code.view(-1, BLOCK).long()
    octave = ((code >> 3) - 1).clamp_min_(0)
    unit = exponent.long() - 127 - octaves - 2
    return ((code - 8 * octave).double() * _power(unit[:, None] + octave)).view(-1)


def _decode_signed(code, exponent):
    x = _decode(code & 127, exponent, 15)
    return torch.where(code > 127, -x, x)


def _decode_positive(code, exponent):
    return _decode(code, exponent, 31)


def _words(s, step, sub):
    """The 32-bit Philox4x32-10 words of all elements, in 64-bit integers: the counter is (place, tensor and
    use, step), four elements a counter."""
    def product(a, b):
        low = a * (b & 0xFFFF)
        high = a * (b >> 16) + (low >> 16)
        return high >> 16, ((high & 0xFFFF) << 16) | (low & 0xFFFF)

    c0, c1 = s["place"] & 0xFFFFFFFF, s["place"] >> 32
    c2, c3 = (s["tensor"] << 8) | (4 << 4) | sub, torch.full_like(c0, step & 0xFFFFFFFF)
    k0, k1 = _seed(s) & 0xFFFFFFFF, _seed(s) >> 32
    for _ in range(10):
        h0, l0 = product(0xD2511F53, c0)
        h1, l1 = product(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return torch.stack((c0, c1, c2, c3), 1).view(-1)


# ---------------------------------------------------------------------------- from the definition, in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "quantize":
        M = s["M"].double()
        return [_exact_quantize(x) for x, at in ((M, "row"), (M.t(), "col")) if case["sides"] in (at, "both")]
    if op in ("serve", "product"):
        a, sa = _exact_quantize(s["x"].double()) if op == "serve" else (s["a"].double(), s["sa"].double())
        return _exact_product(a, sa, s["w"].double(), s["sw"].double())
    if op == "train":
        x, w, dy = s["x"].double(), s["w"].double(), s["dy"].double()
        y = _exact_product(*_exact_quantize(x), *_exact_quantize(w.t()))
        dx = _exact_product(*_exact_quantize(dy), *_exact_quantize(w))
        dw = _exact_product(*_exact_quantize(x.t()), *_exact_quantize(dy.t()))
        return {"y": y, "dx": dx, "dw": dw}
    return _exact_adamw(case, s)


def _inputs(case, seed):
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def _exact_quantize(x):
    top = x.abs().max(dim=1, keepdim=True).values
    top = torch.where(top < 127 * 2.0 ** -126, torch.full_like(top, 127 * 2.0 ** -126), top)
    twice = torch.floor(254 * x.abs() / top).clamp_max(253)       # half steps below |x|
    odd = twice % 2 == 1
    code = torch.floor(twice / 2)
    past = 254 * x.abs() - (2 * code + 1) * top                   # against the border above, both products exact
    up = torch.where(past == 0, code % 2 == 1, past > 0)
    code = torch.where(odd | up, code + up, code)
    return torch.sign(x) * code, (top / 127).squeeze(1)


def _exact_product(a, sa, b, sb):
    return torch.einsum("ik,jk->ij", a, b) * torch.outer(sa, sb)


def _exact_adamw(case, s):
    t = s["step"] + 1
    b1, b2 = BETA1, BETA2
    g = s["g"].double()
    if case["bits"] == 8:
        m, v = _table_values(s["m"], s["me"], True), _table_values(s["v"], s["ve"], False)
    else:
        m, v = s["m"].double(), s["v"].double()
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    step = LR / (1 - math.pow(b1, t)) * m / (torch.sqrt(v / (1 - math.pow(b2, t))) + EPS)
    p = s["p"].double() * (1 - LR * DECAY) - step
    if case["rounding"] == "sr" and case["dtype"] == "bf16":
        p = None                                                   # a random rounding of the value has no such value
    if case["bits"] == 32:
        return {"p": p, "m": m, "v": v}
    words = _exact_words(case, s, t) if case["rounding"] == "sr" else None
    out = {"p": p}
    out["m"], out["me"] = _table_codes(m, words, True)
    out["v"], out["ve"] = _table_codes(v, words, False)
    return out


def _table(signed):
    """All magnitudes of a state's code under the exponent 0."""
    octaves = 15 if signed else 31
    units = [c if c < 8 else (8 + c % 8) * 2 ** (c // 8 - 1) for c in range(8 * octaves + 8)]
    return torch.tensor([u * 2.0 ** -(octaves + 2) for u in units], dtype=torch.float64, device="cuda")


def _table_values(code, exponent, signed):
    code = code.long()
    table = _table(signed)
    scale = torch.pow(2.0, exponent.double() - 127).repeat_interleave(BLOCK)
    if signed:
        return table[code % 128] * scale * (1 - 2 * (code // 128)).double()
    return table[code] * scale


def _table_codes(x, words, signed):
    table, magnitude = _table(signed), x.abs().view(-1, BLOCK)
    top = torch.floor(torch.log2(magnitude.max(dim=1).values.clamp_min(1e-300)))
    most = magnitude.max(dim=1).values
    top = torch.where(torch.pow(2.0, top) > most, top - 1, top)    # log2 is itself rounded
    top = torch.where(torch.pow(2.0, top + 1) <= most, top + 1, top).clamp(-111, 127)
    y = magnitude * torch.pow(2.0, -top)[:, None]
    low = (torch.searchsorted(table, y, right=True) - 1).clamp(0, len(table) - 1)
    high = (low + 1).clamp_max(len(table) - 1)
    gap = torch.where(high > low, table[high] - table[low], torch.full_like(y, 2.0 ** -3))
    part = (y - table[low]) / gap
    if words is None:
        up = torch.where(part == 0.5, low % 2 == 1, part > 0.5)
    else:
        field = words % 65536 if signed else words // 65536
        up = part + (field.view(-1, BLOCK).double() + 0.5) / 65536 >= 1
    code = torch.where(up, high, low)
    if signed:
        code = code + 128 * ((x.view(-1, BLOCK) < 0) & (code > 0))
    else:
        code = torch.where((magnitude > 0) & (code == 0), torch.ones_like(code), code)
    return code.view(-1).to(torch.uint8), (top + 127).to(torch.uint8)


def _exact_words(case, s, step):
    """Philox4x32-10 in unsigned 64-bit numpy integers, for all elements."""
    place, tensor = s["place"].cpu().numpy().astype(np.uint64), s["tensor"].cpu().numpy().astype(np.uint64)
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    c = [place & low, place >> half, tensor * np.uint64(256) + np.uint64(64), np.full_like(place, step)]
    k = [_seed(case) & 0xFFFFFFFF, _seed(case) >> 32]
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> half) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> half) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return torch.from_numpy(np.stack(c, 1).reshape(-1).astype(np.int64)).cuda()
