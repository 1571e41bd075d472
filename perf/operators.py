"""Cases of the dense block in microscaled formats: the residual addition with the root-mean-square norm
and block-32 codes, the product with FP4 (E2M1) weights, SwiGLU with block-32 codes, and the dense FFN
that they form, each in its plain form (elementary torch operations) and as the library's calls.

Formats: E4M3 and E2M1 elements in blocks of 32 along the last axis with one E8M0 scale 2^(c - 127) each;
scale and element rounding as OCP Microscaling v1.0 (floor scale, nearest even, saturating)."""
import math

import torch

own = False

BLOCK = 32
EMAX = {"e4m3": 8, "e2m1": 2}                 # exponent of the format's largest value
EMIN = {"e4m3": -6, "e2m1": 0}                # exponent of its smallest normal value
MANT = {"e4m3": 3, "e2m1": 1}
MOST = {"e4m3": 448.0, "e2m1": 6.0}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the norm after a routed + shared layer of one row: y and y_shared join the residual stream
        dict(name="norm decode", op="norm", rows=1, cols=4096, x="f32", addends=2, res="bf16", fmt="e4m3"),
        # a verification batch at the pages' hidden width, codes in 4 bits
        dict(name="norm verify", op="norm", rows=48, cols=5120, x="bf16", addends=1, res="bf16", fmt="e2m1"),
        # a prefill chunk after attention
        dict(name="norm prefill", op="norm", rows=8192, cols=4096, x="bf16", addends=1, res="bf16", fmt="e4m3"),
        # an odd batch of an FFN of odd width, fp32 gate/up values
        dict(name="swiglu ragged", op="swiglu", rows=999, inner=1376, x="f32", fmt="e2m1"),
        # a prefill chunk, bf16 gate/up values
        dict(name="swiglu prefill", op="swiglu", rows=8192, inner=4096, x="bf16", fmt="e4m3"),
        # a projection of one decode row: 8-bit activations, 4-bit weights
        dict(name="product decode", op="product", rows=1, out=4096, inner=4096, a="e4m3", y="bf16"),
        # the verification batch in 4 x 4 bits, fp32 out
        dict(name="product verify", op="product", rows=48, out=4096, inner=4096, a="e2m1", y="f32"),
        # nothing a multiple of a tile: rows, columns and K
        dict(name="product ragged", op="product", rows=333, out=4100, inner=4128, a="e4m3", y="bf16"),
        # a prefill chunk, 8-bit and 4-bit activations
        dict(name="product prefill 8", op="product", rows=8192, out=4096, inner=4096, a="e4m3", y="bf16"),
        dict(name="product prefill 4", op="product", rows=8192, out=4096, inner=4096, a="e2m1", y="bf16"),
        # residual + norm + dense FFN of one decode row, and of a prefill chunk
        dict(name="ffn decode", op="ffn", rows=1, cols=4096, inner=2048, fmt="e4m3"),
        dict(name="ffn prefill", op="ffn", rows=2048, cols=4096, inner=8192, fmt="e2m1"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "swiglu", "product", "ffn"))
    rows, fmt = _log(rng, 1, 8192), rng.choice(("e4m3", "e2m1"))
    if op == "norm":
        cols = BLOCK * _log(rng, 1, 512)
        rows = min(rows, max(1, (8192 * 4096) // cols))
        res = rng.choice(("none", "bf16", "f32"))
        return dict(op=op, rows=rows, cols=cols, x=rng.choice(("f32", "bf16")), addends=rng.choice((1, 2)), res=res, fmt=fmt)
    if op == "swiglu":
        inner = BLOCK * _log(rng, 1, 256)
        return dict(op=op, rows=min(rows, max(1, (8192 * 4096) // inner)), inner=inner, x=rng.choice(("f32", "bf16")), fmt=fmt)
    if op == "product":
        out, inner = _log(rng, 16, 16384), BLOCK * _log(rng, 4, 512)
        rows = min(rows, max(1, (8192 * 4096 * 4096) // (out * inner)))
        # fp32 results of 8-bit activations are left to the tests: the matrix cores' own sum of E4M3 products is about
        # 4e-6 off, which a bf16 result does not show
        return dict(op=op, rows=rows, out=out, inner=inner, a=fmt, y=rng.choice(("bf16", "f32")) if fmt == "e2m1" else "bf16")
    cols, inner = BLOCK * _log(rng, 8, 256), BLOCK * _log(rng, 8, 256)
    return dict(op=op, rows=min(rows, max(1, (2048 * 4096 * 8192) // (cols * inner))), cols=cols, inner=inner, fmt=fmt)


def _code_bytes(n, fmt):
    return n if fmt == "e4m3" else n // 2


def work(case):
    op, T = case["op"], case["rows"]
    size = {"f32": 4, "bf16": 2, "none": 0}
    if op == "norm":
        n = T * case["cols"]
        moved = n * (size[case["x"]] * case["addends"] + 2 * size[case["res"]] + 2) + _code_bytes(n, case["fmt"]) + n // BLOCK
        if case["fmt"] == "e2m1":                 # the codes are read back as bf16 values
            moved += _code_bytes(n, "e2m1") + n // BLOCK + 2 * n
        return {"bytes": moved + 2 * case["cols"], "flops": 8.0 * n}
    if op == "swiglu":
        n = T * case["inner"]
        moved = 2 * n * size[case["x"]] + _code_bytes(n, case["fmt"]) + n // BLOCK
        if case["fmt"] == "e2m1":
            moved += _code_bytes(n, "e2m1") + n // BLOCK + 2 * n
        return {"bytes": moved, "flops": 10.0 * n}
    if op == "product":
        K, N = case["inner"], case["out"]
        moved = T * (_code_bytes(K, case["a"]) + K // BLOCK) + N * (K // 2 + K // BLOCK) + T * N * size[case["y"]]
        return {"bytes": moved, "flops": 2.0 * T * N * K}
    H, I = case["cols"], case["inner"]
    moved = 3 * H * (I // 2 + I // BLOCK) + T * H * 2 * 4 + 2 * H      # weights; x, residual in; h, y out; norm weight
    return {"bytes": moved, "flops": 6.0 * T * H * I}


# ----------------------------------------------------------------- inputs
def _power(e):
    """2^e in 64 bits of whole numbers, exactly (their exponent bits)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _codes(v, fmt):
    """fp32 [..., n] -> (element values fp64 under the scale, scale codes uint8 [..., n / 32])."""
    b = v.unflatten(-1, (-1, BLOCK))
    exponent = (b.abs().amax(-1).view(torch.int32) >> 23) & 0xFF
    code = (exponent - EMAX[fmt]).clamp(0, 254)
    t = b.double() * _power(127 - code).unsqueeze(-1)
    e = (torch.frexp(t.abs()).exponent - 1).clamp(EMIN[fmt], EMAX[fmt])
    step = _power(e - MANT[fmt])
    r = (torch.round(t / step) * step).clamp(-MOST[fmt], MOST[fmt])
    return r.flatten(-2), code.to(torch.uint8)


def _pack(values, fmt):
    """Element values -> code bytes: E4M3 one byte each, E2M1 two nibbles per byte (element 2j low)."""
    if fmt == "e4m3":
        return values.to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=values.dtype, device=values.device)
    c = torch.bucketize(values.abs(), mids).to(torch.uint8) | (torch.signbit(values).to(torch.uint8) << 3)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _weights(rows, cols, g):
    w = torch.randn((rows, cols), generator=g, device="cuda") * 0.02
    values, sc = _codes(w, "e2m1")
    return _pack(values, "e2m1"), sc


def _hidden(rows, cols, g, gain):
    return torch.randn((rows, cols), generator=g, device="cuda") * gain


def prepare(case, seed):
    """Inputs: activations with a few loud channels, weights N(0, 0.02^2) in E2M1; and the buffers of the outputs."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, op = case["rows"], case["op"]
    u8, bf = torch.uint8, torch.bfloat16

    def empty(*shape, dtype=u8):
        return torch.empty(shape, dtype=dtype, device="cuda")

    s = {"case": dict(case)}
    if op in ("norm", "ffn"):
        H, fmt = case["cols"], case["fmt"]
        gain = torch.exp(0.5 * torch.randn(H, generator=g, device="cuda"))
        xt = DTYPE[case.get("x", "bf16")]
        s["x"] = _hidden(T, H, g, gain).to(xt)
        s["x2"] = _hidden(T, H, g, gain).to(xt) if case.get("addends", 1) == 2 else None
        res = case.get("res", "bf16")
        s["residual"] = None if res == "none" else (_hidden(T, H, g, gain) * 4).to(DTYPE[res])
        s["weight"] = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(bf)
        s["h"] = None if res == "none" else torch.empty_like(s["residual"])
        s["n"] = empty(T, H, dtype=bf) if op == "norm" else None
        s["q"], s["sc"] = empty(T, _code_bytes(H, fmt)), empty(T, H // BLOCK)
        s["values"] = empty(T, H, dtype=bf)
    if op == "swiglu":
        I, fmt = case["inner"], case["fmt"]
        gain = torch.exp(0.5 * torch.randn(2 * I, generator=g, device="cuda"))
        s["gu"] = _hidden(T, 2 * I, g, gain).to(DTYPE[case["x"]])
        s["q"], s["sc"] = empty(T, _code_bytes(I, fmt)), empty(T, I // BLOCK)
        s["values"] = empty(T, I, dtype=bf)
    if op == "product":
        N, K = case["out"], case["inner"]
        gain = torch.exp(0.5 * torch.randn(K, generator=g, device="cuda"))
        values, s["a_sc"] = _codes(_hidden(T, K, g, gain), case["a"])
        s["a"] = _pack(values, case["a"])
        s["w"], s["w_sc"] = _weights(N, K, g)
        s["y"] = empty(T, N, dtype=DTYPE[case["y"]])
    if op == "ffn":
        H, I = case["cols"], case["inner"]
        s["w13"], s["w13_sc"] = _weights(2 * I, H, g)
        s["w2"], s["w2_sc"] = _weights(H, I, g)
        s["y"] = empty(T, H, dtype=bf)
        s["ws"] = empty(T * I * 10 + (1 << 16))
    return s


# ------------------------------------------------------------- plain form
def _scale(sc, dtype):
    """2^(c - 127) of E8M0 codes (code 0 is 2^-127)."""
    return _power(sc.to(torch.int64) - 127).to(dtype).repeat_interleave(BLOCK, -1)


def _values(codes, sc, fmt, dtype=torch.float32):
    """Codes and scales -> the values they stand for."""
    if fmt == "e4m3":
        v = codes.view(torch.float8_e4m3fn).to(dtype)
    else:
        lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=codes.device)
        v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).flatten(-2)
    return v * _scale(sc, dtype)


def _product(a, w):
    return a @ w.t()


def _norm(s):
    """(h, n in fp32): h = residual + x (+ x2) in fp32, rounded to the residual's type; n from the stored h, in 64 bits
    up to its own rounding because its codes lie next to rounding borders."""
    v = s["x"].float()
    if s["residual"] is not None:
        v = s["residual"].float() + v
    if s["x2"] is not None:
        v = v + s["x2"].float()
    h = v if s["residual"] is None else v.to(s["residual"].dtype)
    d = h.double()
    r = 1.0 / torch.sqrt(d.square().mean(-1, keepdim=True) + EPS)
    return h, (d * r * s["weight"].double()).float()


def _swiglu(gu):
    """silu(gate) * up in 64 bits, rounded once to fp32 (its codes lie next to rounding borders)."""
    g, u = gu.double().chunk(2, -1)
    return (g / (1.0 + torch.exp(-g)) * u).float()


def _told(values, code, fmt):
    """Codes as the values they stand for: E4M3 elements and E8M0 scales, or E2M1 elements times scales."""
    if fmt == "e4m3":
        return {"q": values.to(torch.float32).to(torch.float8_e4m3fn), "sc": code.view(torch.float8_e8m0fnu)}
    return {"values": (values * _scale(code, torch.float64)).to(torch.bfloat16)}


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        h, n = _norm(s)
        out = _told(*_codes(n, case["fmt"]), case["fmt"])
        out["n"] = n.to(torch.bfloat16)
        if s["residual"] is not None:
            out["h"] = h
        return out
    if op == "swiglu":
        return _told(*_codes(_swiglu(s["gu"]), case["fmt"]), case["fmt"])
    if op == "product":
        y = _product(_values(s["a"], s["a_sc"], case["a"]), _values(s["w"], s["w_sc"], "e2m1"))
        return {"y": y.to(s["y"].dtype)}
    h, n = _norm(s)
    values, code = _codes(n, case["fmt"])
    gu = _product((values * _scale(code, torch.float64)).float(), _values(s["w13"], s["w13_sc"], "e2m1"))
    values, code = _codes(_swiglu(gu), case["fmt"])
    y = _product((values * _scale(code, torch.float64)).float(), _values(s["w2"], s["w2_sc"], "e2m1"))
    return {"h": h, "y": y.to(torch.bfloat16)}


# ---------------------------------------------------------- library calls
def _calls(s):
    from block_scaled_fp8xfp4_amd import mxmoe
    case = s["case"]
    op = case["op"]
    formats = {"e4m3": mxmoe.MX_FMT_E4M3, "e2m1": mxmoe.MX_FMT_E2M1}

    def told(fmt):
        if fmt == "e4m3":
            return {"q": s["q"].view(torch.float8_e4m3fn), "sc": s["sc"].view(torch.float8_e8m0fnu)}
        mxmoe.mx_dequantize(s["q"], s["sc"], mxmoe.MX_FMT_E2M1, s["values"])
        return {"values": s["values"]}

    if op == "norm":
        mxmoe.mx_add_rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], x2=s["x2"], h=s["h"], n=s["n"],
                             q=s["q"], sc=s["sc"], fmt=formats[case["fmt"]])
        out = told(case["fmt"])
        out["n"] = s["n"]
        if s["h"] is not None:
            out["h"] = s["h"]
        return out
    if op == "swiglu":
        mxmoe.mx_swiglu_quantize(s["gu"], s["q"], s["sc"], formats[case["fmt"]])
        return told(case["fmt"])
    if op == "product":
        mxmoe.fp4_block_gemm(s["a"], s["a_sc"], formats[case["a"]], s["w"], s["w_sc"], s["y"])
        return {"y": s["y"]}
    fmt = formats[case["fmt"]]
    mxmoe.mx_add_rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], h=s["h"], q=s["q"], sc=s["sc"], fmt=fmt)
    mxmoe.fp4_dense_ffn(s["q"], s["sc"], fmt, s["w13"], s["w13_sc"], s["w2"], s["w2_sc"], fmt, s["y"], s["ws"])
    return {"h": s["h"], "y": s["y"]}


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------- the definition in 64 bits
def _twos(e):
    """2^e of whole numbers -127..127 from a table (pow and exp2 round on some devices)."""
    table = torch.tensor([2.0 ** k for k in range(-127, 129)], dtype=torch.float64, device=e.device)
    return table[e.long() + 127]


def _nearest(v, fmt):
    """64-bit values -> (elements, scales) by search among the format's values, ties to the even code."""
    if fmt == "e4m3":
        table = [m / 8.0 * 2.0 ** -6 for m in range(8)]
        table += [(1 + m / 8.0) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]
    else:
        table = list(E2M1)
    grid = torch.tensor(table, dtype=torch.float64, device=v.device)
    mids = (grid[1:] + grid[:-1]) / 2
    blocks = v.reshape(*v.shape[:-1], -1, BLOCK)
    most = blocks.abs().max(-1, keepdim=True).values
    exponent = torch.where(most > 0, torch.frexp(most).exponent - 1 - EMAX[fmt], -127).clamp(-127, 127)
    scale = _twos(exponent)
    t = blocks / scale
    low, high = torch.bucketize(t.abs(), mids, right=False), torch.bucketize(t.abs(), mids, right=True)
    at = torch.where(low % 2 == 0, low, high)
    return (torch.copysign(grid[at], t)).reshape(v.shape), scale


def _exact_told(v, fmt):
    elements, scale = _nearest(v, fmt)
    if fmt == "e4m3":
        return {"q": elements, "sc": scale.squeeze(-1)}
    return {"values": (elements.reshape(*scale.shape[:-1], BLOCK) * scale).reshape(v.shape)}


def _exact_values(codes, sc, fmt):
    i = codes.long()
    if fmt == "e2m1":
        i = torch.stack((i % 16, i // 16), -1).reshape(codes.shape[0], -1)
        mag, e, m = i % 8, i % 8 // 2, i % 2
        v = torch.where(e == 0, m * 0.5, (1 + 0.5 * m) * _twos(e - 1))
        sign = i // 8
    else:
        mag, e, m = i % 128, i % 128 // 8, i % 8
        v = torch.where(e == 0, m.double() / 512, (1 + m.double() / 8) * _twos(e - 7))
        sign = i // 128
    v = torch.where(sign == 1, -v, v).double().reshape(codes.shape[0], -1, BLOCK)
    return (v * _twos(sc.long() - 127).unsqueeze(-1)).reshape(codes.shape[0], -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "product":
        return {"y": torch.mm(_exact_values(s["a"], s["a_sc"], case["a"]), _exact_values(s["w"], s["w_sc"], "e2m1").t().contiguous())}
    if op == "swiglu":
        I = case["inner"]
        gate, up = s["gu"][:, :I].double(), s["gu"][:, I:].double()
        return _exact_told((gate * torch.sigmoid(gate) * up).float().double(), case["fmt"])
    # the residual stream is stored in its own type and the norm reads it so
    h = s["x"].double()
    for t in (s["residual"], s["x2"]):
        h = h if t is None else h + t.double()
    kept = h.float() if s["residual"] is None else h.to(s["residual"].dtype)
    k = kept.double()
    n = k * s["weight"].double() / (k.pow(2).sum(-1, keepdim=True) / case["cols"] + EPS).sqrt()
    if op == "norm":
        out = _exact_told(n.float().double(), case["fmt"])
        out["n"] = n
        if s["residual"] is not None:
            out["h"] = h
        return out
    I = case["inner"]
    told = lambda v: (lambda e, sc: (e.reshape(*sc.shape[:-1], BLOCK) * sc).reshape(v.shape))(*_nearest(v, case["fmt"]))  # noqa: E731
    gu = torch.mm(told(n.float().double()), _exact_values(s["w13"], s["w13_sc"], "e2m1").t().contiguous())
    a = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
    return {"h": h, "y": torch.mm(told(a.float().double()), _exact_values(s["w2"], s["w2_sc"], "e2m1").t().contiguous())}
