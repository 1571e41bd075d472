"""Cases of the experts' tokens and of FP8 products with a scale for each block of 128: rows sorted by expert and back
with the routing weights and their gradient, the casts to E4M3 codes with fp32 scales, the dense product, and the
experts' products with the gradient of their weights; each in its plain form (elementary torch operations) and as the
library's calls.

Format: E4M3 codes; a block's scale is max(amax, 2^-60) / 448 in fp32, a code the nearest E4M3 value to x / scale (ties to
even).  Blocks are 1 x 128 (rows), 128 x 128 (weights) or 128 x 1 (columns, for sums over tokens)."""
import math

import torch

own = False

BLOCK = 128
FLOOR = 2.0 ** -60
MOST = 448.0
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the rows of a verification batch, to their experts, at the pages' hidden width
        dict(name="sort verify", op="sort", rows=48, k=8, experts=384, cols=5120, x="bf16", live=0.8),
        # a prefill chunk, cast before it is sorted: codes and scales
        dict(name="sort prefill", op="sort", rows=8192, k=8, experts=256, cols=4096, x="e4m3", live=1.0),
        # the experts' outputs of a prefill chunk, back to their tokens
        dict(name="back prefill", op="back", way="forth", rows=8192, k=8, experts=256, cols=4096, o="bf16", y="bf16",
             weighted=True, live=1.0),
        # the gradient of a training batch of odd sizes: of the experts' outputs and of the routing weights
        dict(name="back gradient", op="back", way="gradient", rows=3999, k=6, experts=64, cols=2050, o="bf16", y="bf16",
             weighted=True, live=1.0),
        # rows of a prefill chunk before a projection
        dict(name="cast prefill", op="cast", how="rows", rows=8192, cols=4096, x="bf16"),
        # between an FFN's products, an odd batch of odd width
        dict(name="cast swiglu ragged", op="cast", how="swiglu", rows=999, cols=1376, x="f32"),
        # a training batch's rows by expert, along the tokens, for the weight gradient
        dict(name="cast columns", op="cast", how="columns", rows=32768, cols=2048, x="bf16", groups=64),
        # a projection of one decode row
        dict(name="product decode", op="product", rows=1, out=4096, inner=4096, w="tiles"),
        # of a prefill chunk
        dict(name="product prefill", op="product", rows=8192, out=4096, inner=4096, w="tiles"),
        # gate/up of one decode row's eight experts
        dict(name="experts decode", op="experts", way="forth", rows=1, k=8, experts=256, out=1152, inner=4096, live=1.0),
        # of a prefill chunk: 256 rows an expert on average, ragged
        dict(name="experts prefill", op="experts", way="forth", rows=8192, k=8, experts=256, out=1152, inner=4096, live=1.0),
        # the gradient of gate/up weights in training
        dict(name="experts weight gradient", op="experts", way="weights", rows=4096, k=8, experts=64, out=1152, inner=2048,
             live=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("sort", "back", "cast", "product", "experts"))
    rows = _log(rng, 1, 8192)
    experts = _log(rng, 8, 256)
    k = rng.choice((1, 2, 4, 6, 8))
    live = rng.choice((1.0, 1.0, 0.7))
    if op == "sort":
        x = rng.choice(("bf16", "f32", "e4m3"))
        cols = 16 * _log(rng, 4, 512) if x == "e4m3" else _log(rng, 64, 8192)
        rows = min(rows, max(1, (8192 * 8 * 4096) // (k * cols * SIZE[x])))
        return dict(op=op, rows=rows, k=k, experts=experts, cols=cols, x=x, live=live)
    if op == "back":
        way, cols = rng.choice(("forth", "gradient")), _log(rng, 64, 8192)
        rows = min(rows, max(1, (8192 * 8 * 2048) // (k * cols)))
        return dict(op=op, way=way, rows=rows, k=k, experts=experts, cols=cols, o=rng.choice(("bf16", "f32")),
                    y=rng.choice(("bf16", "f32")), weighted=way == "gradient" or rng.random() < 0.7, live=live)
    if op == "cast":
        how, x = rng.choice(("rows", "tiles", "swiglu", "columns")), rng.choice(("bf16", "f32"))
        cols = 16 * _log(rng, 4, 512)
        rows = min(rows, max(1, (8192 * 2048) // cols))
        case = dict(op=op, how=how, rows=rows, cols=cols, x=x)
        if how == "columns":
            case["groups"] = rng.choice((0, experts))
        return case
    if op == "product":
        out, inner, w = _log(rng, 16, 16384), 16 * _log(rng, 8, 512), rng.choice(("tiles", "tiles", "rows"))
        if w == "rows":                                  # a sum over tokens
            inner = -(-inner // BLOCK) * BLOCK
        # bf16 results only: the matrix cores' own sums of E4M3 products are a few 1e-6 off, which bf16 does not show
        rows = min(rows, max(1, (4096 * 4096 * 4096) // (out * inner)))
        return dict(op=op, rows=rows, out=out, inner=inner, w=w)
    way = rng.choice(("forth", "forth", "weights"))
    out, inner = _log(rng, 64, 2048), 16 * _log(rng, 8, 256)
    most = 2 ** 27 if way == "weights" else 2 ** 29
    experts = max(8, min(experts, most // (out * inner)))
    rows = min(rows, max(1, (4096 * 8 * 1152 * 2048) // (k * out * inner)))
    return dict(op=op, way=way, rows=rows, k=k, experts=experts, out=out, inner=inner, live=live)


def _active(case):
    """Experts with rows, on average."""
    return case["experts"] * (1.0 - (1.0 - case["k"] / case["experts"]) ** (case["rows"] * case["live"]))


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    op, T = case["op"], case["rows"]
    if op == "sort":
        row = case["cols"] * SIZE[case["x"]] + (4 * _blocks(case["cols"]) if case["x"] == "e4m3" else 0)
        return {"bytes": T * row * (1 + case["live"] * case["k"]) + 4 * T * case["k"], "flops": 0.0}
    if op == "back":
        H, P = case["cols"], T * case["k"] * case["live"]
        if case["way"] == "forth":
            return {"bytes": P * H * SIZE[case["o"]] + T * H * SIZE[case["y"]] + 8 * T * case["k"], "flops": 2.0 * P * H}
        return {"bytes": 2 * P * H * SIZE[case["o"]] + T * H * SIZE[case["y"]] + 12 * T * case["k"], "flops": 3.0 * P * H}
    if op == "cast":
        n = T * case["cols"]
        scales = n / BLOCK / (BLOCK if case["how"] == "tiles" else 1)
        return {"bytes": n * SIZE[case["x"]] * (2 if case["how"] == "swiglu" else 1) + n + 4 * scales,
                "flops": n * (12.0 if case["how"] == "swiglu" else 4.0)}
    N, K = case["out"], case["inner"]
    if op == "product":
        scales = 4 * _blocks(K) * (T + (N if case["w"] == "rows" else _blocks(N)))
        return {"bytes": T * K + N * K + scales + 2 * T * N, "flops": 2.0 * T * N * K}
    P = T * case["k"] * case["live"]
    if case["way"] == "forth":
        return {"bytes": _active(case) * N * K * (1 + 4 / BLOCK ** 2) + P * (K * (1 + 4 / BLOCK) + 2 * N), "flops": 2.0 * P * N * K}
    return {"bytes": P * (N + K) * (1 + 4 / BLOCK) + 2 * case["experts"] * N * K, "flops": 2.0 * P * N * K}


# ----------------------------------------------------------------- inputs
def _fit(values, scale):
    """64-bit values and their blocks' scales -> E4M3 values."""
    t = values / scale
    e = (torch.frexp(t.abs()).exponent - 1).clamp(-6, 8).to(torch.int64)
    step = ((e - 3 + 1023) << 52).view(torch.float64)
    return (torch.round(t / step) * step).clamp(-MOST, MOST)


def _scale(amax):
    return (amax.double().clamp(min=FLOOR) / MOST).float()


def _padded(v, rows, cols):
    """v [..., R, C] with zeros up to whole blocks of rows x cols."""
    return torch.nn.functional.pad(v, (0, -v.shape[-1] % cols, 0, -v.shape[-2] % rows))


def _cast(v, rows, cols):
    """fp32 [..., R, C] -> (E4M3 values as fp32 [..., R, C], scales [..., R / rows, C / cols])."""
    R, C = v.shape[-2:]
    b = _padded(v, rows, cols).unflatten(-1, (-1, cols)).unflatten(-3, (-1, rows))
    sc = _scale(b.abs().amax((-3, -1)))
    q = _fit(b.double(), sc.double()[..., :, None, :, None])
    return q.flatten(-4, -3).flatten(-2)[..., :R, :C].float(), sc


def _bytes(values):
    return values.to(torch.float8_e4m3fn).view(torch.uint8)


def _hidden(rows, cols, g):
    """Rows with a few loud channels."""
    gain = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    return torch.randn((rows, cols), generator=g, device="cuda") * gain


def _plan(case, g):
    """Where each (token, slot) goes: pairs sorted by expert, then token; rows that are not live go nowhere."""
    T, k, E = case["rows"], case["k"], case["experts"]
    score = torch.rand((T, E), generator=g, device="cuda")
    ids = torch.argsort(score, dim=1, descending=True)[:, :k]
    alive = torch.rand(T, generator=g, device="cuda") < case["live"]
    alive[0] = True
    key = torch.where(alive[:, None], ids, E).flatten()
    order = torch.argsort(key, stable=True)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(T * k, device="cuda")
    slot_pos = torch.where(alive[:, None], pos.view(T, k), -1).to(torch.int32)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = counts.cumsum(0)
    weights = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), 1)
    return {"slot_pos": slot_pos.contiguous(), "offsets": offsets.to(torch.int32), "w_route": weights,
            "bounds": offsets.tolist()}


def _places(bounds, rows):
    """Where rows in groups go as columns: (rows, their columns, each group's first column, columns in all)."""
    at = [0]
    for a, b in zip(bounds, bounds[1:]):
        at.append(at[-1] + _blocks(b - a) * BLOCK)
    src = torch.arange(bounds[-1], device="cuda")
    to = torch.cat([torch.arange(b - a) + s for a, b, s in zip(bounds, bounds[1:], at)]).cuda()
    return src, to, at, _width(rows, len(bounds) - 1)


def _columns(v, places):
    """fp32 [R, C], rows in groups -> (values [C, ld], scales [C, ld / 128]): each group's columns in blocks of 128 of its
    rows, from a multiple of 128 on."""
    src, to, at, ld = places
    wide = torch.zeros((v.shape[1], ld), device=v.device)
    wide[:, to] = v[src].t()
    values, sc = _cast(wide, 1, BLOCK)
    sc[:, at[-1] // BLOCK:] = 0                      # blocks behind the last group
    return values, sc


def _width(rows, groups):
    """Columns that hold any split of rows into groups, each from a multiple of 128 on."""
    return (rows + (BLOCK - 1) * min(groups, max(rows, 1))) // BLOCK * BLOCK


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, T = case["op"], case["rows"]

    def zeros(*shape, dtype=torch.uint8):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    s = {"case": dict(case)}
    if op in ("sort", "back", "experts"):
        s.update(_plan(case, g))
        P = T * case["k"]
    if op == "sort":
        H = case["cols"]
        if case["x"] == "e4m3":
            values, s["x_sc"] = _cast(_hidden(T, H, g), 1, BLOCK)
            s["x"], s["out_sc"] = _bytes(values), zeros(P, _blocks(H), dtype=torch.float32)
        else:
            s["x"], s["x_sc"], s["out_sc"] = _hidden(T, H, g).to(DTYPE[case["x"]]), None, None
        s["out"] = zeros(P, H, dtype=s["x"].dtype)
    if op == "back":
        H, o, y = case["cols"], DTYPE[case["o"]], DTYPE[case["y"]]
        s["o"] = _hidden(P, H, g).to(o)
        if case["way"] == "forth":
            s["y"] = zeros(T, H, dtype=y)
        else:
            s["dy"] = (_hidden(T, H, g) * 1e-3).to(y)
            s["d_o"], s["dw"] = zeros(P, H, dtype=o), zeros(T, case["k"], dtype=torch.float32)
    if op == "cast":
        C, how = case["cols"], case["how"]
        s["x"] = _hidden(T, 2 * C if how == "swiglu" else C, g).to(DTYPE[case["x"]])
        if how == "tiles":
            s["x"] = (s["x"] * 0.02).to(DTYPE[case["x"]])
        s["q"], s["sc"] = zeros(T, C), zeros(T, _blocks(C), dtype=torch.float32)
        if how == "tiles":
            s["sc"] = zeros(_blocks(T), _blocks(C), dtype=torch.float32)
        if how == "columns":
            E = case["groups"]
            cut = torch.sort(torch.randint(0, T + 1, (max(E, 1) - 1,), generator=g, device="cuda")).values.tolist()
            s["bounds"] = [0] + cut + [T]
            s["offsets"] = torch.tensor(s["bounds"], dtype=torch.int32, device="cuda") if E else None
            s["places"] = _places(s["bounds"], T)
            ld = s["places"][-1]
            s["q"], s["sc"] = zeros(C, ld), zeros(C, ld // BLOCK, dtype=torch.float32)
    if op == "product":
        N, K = case["out"], case["inner"]
        values, s["a_sc"] = _cast(_hidden(T, K, g), 1, BLOCK)
        s["a"] = _bytes(values)
        w = torch.randn((N, K), generator=g, device="cuda") * 0.02
        values, s["w_sc"] = _cast(w, 1 if case["w"] == "rows" else BLOCK, BLOCK)
        s["w"] = _bytes(values)
        s["y"] = zeros(T, N, dtype=torch.bfloat16)
    if op == "experts":
        N, K, E = case["out"], case["inner"], case["experts"]
        rows = s["bounds"][-1]
        if case["way"] == "forth":
            values, s["a_sc"] = _cast(_hidden(P, K, g), 1, BLOCK)
            s["a"] = _bytes(values)
            s["w"], s["w_sc"] = zeros(E, N, K), zeros(E, _blocks(N), _blocks(K), dtype=torch.float32)
            for e in range(E):
                values, s["w_sc"][e] = _cast(torch.randn((N, K), generator=g, device="cuda") * 0.02, BLOCK, BLOCK)
                s["w"][e] = _bytes(values)
            s["y"] = zeros(P, N, dtype=torch.bfloat16)
        else:
            places = _places(s["bounds"], rows)
            s["at"] = places[2]
            for name, n, size in (("a", N, 1e-3), ("b", K, 1.0)):
                values, s[name + "_sc"] = _columns(_hidden(rows, n, g) * size, places)
                s[name] = _bytes(values)
            s["y"] = zeros(E, N, K, dtype=torch.bfloat16)
    return s


# ------------------------------------------------------------- plain form
def _wide(codes, sc, rows=1):
    """Codes [R, C] and scales of blocks rows x 128 -> values in fp32."""
    R, C = codes.shape
    sc = sc.repeat_interleave(rows, 0)[:R] if rows > 1 else sc
    return codes.view(torch.float8_e4m3fn).float() * sc.repeat_interleave(BLOCK, 1)[:, :C]


def _silu(gu):
    """silu(gate) up in 64 bits, rounded once to fp32 (its codes lie next to rounding borders)."""
    g, u = gu.double().chunk(2, -1)
    return (g / (1.0 + torch.exp(-g)) * u).float()


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "sort":
        t, j = torch.where(s["slot_pos"] >= 0)
        p = s["slot_pos"][t, j].long()
        out = {"out": torch.zeros_like(s["out"]).index_copy_(0, p, s["x"][t])}
        if s["x_sc"] is not None:
            out["out_sc"] = torch.zeros_like(s["out_sc"]).index_copy_(0, p, s["x_sc"][t])
        return _told(out)
    if op == "back":
        pos, there = s["slot_pos"].clamp(min=0).long(), s["slot_pos"] >= 0
        w = s["w_route"] if case["weighted"] else torch.ones_like(s["w_route"])
        w = torch.where(there, w, 0.0)
        if case["way"] == "forth":
            y = torch.zeros(s["y"].shape, dtype=torch.float32, device="cuda")
            for j in range(case["k"]):
                y += w[:, j, None] * s["o"][pos[:, j]].float()
            return {"y": y.to(s["y"].dtype)}
        d_o, dw = torch.zeros_like(s["d_o"]), torch.zeros_like(s["dw"])
        dy = s["dy"].float()
        t, j = torch.where(there)
        p = pos[t, j]
        d_o[p] = (w[t, j, None] * dy[t]).to(d_o.dtype)
        dw[t, j] = (dy[t] * s["o"][p].float()).sum(-1)
        return {"d_o": d_o, "dw": dw}
    if op == "cast":
        how = case["how"]
        if how == "columns":
            values, sc = _columns(s["x"].float(), s["places"])
        else:
            values, sc = _cast(_silu(s["x"]) if how == "swiglu" else s["x"].float(), BLOCK if how == "tiles" else 1, BLOCK)
        return {"q": values.to(torch.float8_e4m3fn), "sc": sc}
    if op == "product":
        w = _wide(s["w"], s["w_sc"], 1 if case["w"] == "rows" else BLOCK)
        return {"y": (_wide(s["a"], s["a_sc"]) @ w.t()).to(torch.bfloat16)}
    y = torch.zeros_like(s["y"])
    if case["way"] == "forth":
        for e, (a, b) in enumerate(zip(s["bounds"], s["bounds"][1:])):
            if a < b:
                y[a:b] = _wide(s["a"][a:b], s["a_sc"][a:b]) @ _wide(s["w"][e], s["w_sc"][e], BLOCK).t()
        return {"y": y}
    a, b = _wide(s["a"], s["a_sc"]), _wide(s["b"], s["b_sc"])
    for e, (i, j) in enumerate(zip(s["at"], s["at"][1:])):
        y[e] = a[:, i:j] @ b[:, i:j].t()
    return {"y": y}


def _told(out):
    """Code rows as the values that they stand for, under their scales."""
    if "out_sc" in out:
        out["out"] = out["out"].view(torch.float8_e4m3fn)
    return out


# ---------------------------------------------------------- library calls
def _calls(s):
    from block_scaled_fp8xfp4_amd import mxmoe
    case = s["case"]
    op = case["op"]
    if op == "sort":
        mxmoe.moe_permute(s["x"], s["slot_pos"], s["out"], s["x_sc"], s["out_sc"])
        out = {"out": s["out"]}
        if s["x_sc"] is not None:
            out["out_sc"] = s["out_sc"]
        return _told(out)
    if op == "back":
        w = s["w_route"] if case["weighted"] else None
        if case["way"] == "forth":
            mxmoe.moe_unpermute(s["o"], w, s["slot_pos"], s["y"])
            return {"y": s["y"]}
        mxmoe.moe_unpermute_grad(s["dy"], s["o"], w, s["slot_pos"], s["d_o"], s["dw"])
        return {"d_o": s["d_o"], "dw": s["dw"]}
    if op == "cast":
        how = case["how"]
        if how == "columns":
            mxmoe.fp8_quantize128_t(s["x"], s["q"], s["sc"], s["offsets"])
        elif how == "swiglu":
            mxmoe.fp8_swiglu_quantize128(s["x"], s["q"], s["sc"])
        else:
            mxmoe.fp8_quantize128(s["x"], s["q"], s["sc"], BLOCK if how == "tiles" else 1)
        return {"q": s["q"].view(torch.float8_e4m3fn), "sc": s["sc"]}
    if op == "product":
        mxmoe.fp8_block128_gemm(s["a"], s["a_sc"], s["w"], s["w_sc"], s["y"])
    elif case["way"] == "forth":
        mxmoe.fp8_block128_grouped_gemm(s["a"], s["a_sc"], s["w"], s["w_sc"], s["offsets"], s["y"])
    else:
        mxmoe.fp8_block128_grouped_wgrad(s["a"], s["a_sc"], s["b"], s["b_sc"], s["offsets"], s["y"])
    return {"y": s["y"]}


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------- the definition in 64 bits
def _e4m3():
    table = [m / 8.0 * 2.0 ** -6 for m in range(8)]
    return table + [(1 + m / 8.0) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]


def _nearest(t):
    """64-bit values -> E4M3 values by search, ties to the even code."""
    grid = torch.tensor(_e4m3(), dtype=torch.float64, device=t.device)
    mids = (grid[1:] + grid[:-1]) / 2
    low, high = torch.bucketize(t.abs(), mids, right=False), torch.bucketize(t.abs(), mids, right=True)
    return torch.copysign(grid[torch.where(low % 2 == 0, low, high)], t)


def _exact_cast(v):
    """64-bit [R, C] in blocks of 128 along C -> (values, scales); a scale is kept in fp32."""
    R, C = v.shape
    values, scales = torch.zeros_like(v), torch.zeros((R, _blocks(C)), dtype=torch.float64, device=v.device)
    for i in range(_blocks(C)):
        b = v[:, i * BLOCK:(i + 1) * BLOCK]
        scales[:, i] = (b.abs().max(1).values.clamp(min=FLOOR) / 448.0).float().double()
        values[:, i * BLOCK:(i + 1) * BLOCK] = _nearest(b / scales[:, i:i + 1])
    return values, scales


def _exact_values(codes, sc, tile_rows):
    table = torch.tensor([x for x in _e4m3()] + [0.0], dtype=torch.float64, device=codes.device)
    i = codes.long()
    v = torch.where(i >= 128, -table[i % 128], table[i % 128])
    r = torch.arange(v.shape[0], device=v.device) // tile_rows
    c = torch.arange(v.shape[1], device=v.device) // BLOCK
    return v * sc.double()[r][:, c]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "sort":
        out, sc = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda"), None
        x = s["x"].view(torch.float8_e4m3fn).double() if case["x"] == "e4m3" else s["x"].double()
        if s["x_sc"] is not None:
            sc = torch.zeros(s["out_sc"].shape, dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            p = s["slot_pos"][:, j].long()
            out[p[p >= 0]] = x[p >= 0]
            if sc is not None:
                sc[p[p >= 0]] = s["x_sc"][p >= 0].double()
        return {"out": out} if sc is None else {"out": out, "out_sc": sc}
    if op == "back":
        w = s["w_route"].double() if case["weighted"] else torch.ones_like(s["w_route"]).double()
        if case["way"] == "forth":
            y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
            for j in range(case["k"]):
                p = s["slot_pos"][:, j].long()
                y[p >= 0] += w[p >= 0, j, None] * s["o"][p[p >= 0]].double()
            return {"y": y}
        d_o = torch.zeros(s["d_o"].shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(s["dw"].shape, dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            p = s["slot_pos"][:, j].long()
            on = p >= 0
            d_o[p[on]] = s["dy"][on].double() * w[on, j, None]
            dw[on, j] = torch.linalg.vecdot(s["dy"][on].double(), s["o"][p[on]].double())
        return {"d_o": d_o, "dw": dw}
    if op == "cast":
        how, x = case["how"], s["x"].double()
        if how == "swiglu":
            C = case["cols"]
            x = (x[:, :C] * torch.sigmoid(x[:, :C]) * x[:, C:]).float().double()
        if how == "tiles":
            q, sc = torch.zeros_like(x), torch.zeros(s["sc"].shape, dtype=torch.float64, device="cuda")
            for i in range(sc.shape[0]):
                b = x[i * BLOCK:(i + 1) * BLOCK]
                most = torch.nn.functional.pad(b.abs().max(0).values, (0, -b.shape[1] % BLOCK)).view(-1, BLOCK).max(1).values
                sc[i] = (most.clamp(min=FLOOR) / 448.0).float().double()
                q[i * BLOCK:(i + 1) * BLOCK] = _nearest(b / sc[i].repeat_interleave(BLOCK)[:b.shape[1]])
            return {"q": q, "sc": sc}
        if how == "columns":
            q = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
            sc, at = torch.zeros(s["sc"].shape, dtype=torch.float64, device="cuda"), 0
            for a, b in zip(s["bounds"], s["bounds"][1:]):
                n = _blocks(b - a)
                if n:
                    q[:, at * BLOCK:at * BLOCK + b - a], sc[:, at:at + n] = _exact_cast(x[a:b].t().contiguous())
                at += n
            return {"q": q, "sc": sc}
        q, sc = _exact_cast(x)
        return {"q": q, "sc": sc}
    if op == "product":
        w = _exact_values(s["w"], s["w_sc"], 1 if case["w"] == "rows" else BLOCK)
        return {"y": torch.mm(_exact_values(s["a"], s["a_sc"], 1), w.t().contiguous())}
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    if case["way"] == "forth":
        for e, (a, b) in enumerate(zip(s["bounds"], s["bounds"][1:])):
            if a < b:
                w = _exact_values(s["w"][e], s["w_sc"][e], BLOCK)
                y[a:b] = torch.mm(_exact_values(s["a"][a:b], s["a_sc"][a:b], 1), w.t().contiguous())
        return {"y": y}
    a, b = _exact_values(s["a"], s["a_sc"], 1), _exact_values(s["b"], s["b_sc"], 1)
    for e, (i, j) in enumerate(zip(s["at"], s["at"][1:])):
        y[e] = torch.mm(a[:, i:j].contiguous(), b[:, i:j].t().contiguous())
    return {"y": y}
