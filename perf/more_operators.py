"""Serving operators of the MoE layer with 4-bit operands, and the layer for a few tokens: what is
timed, and on which inputs.

Four operators:

* ``quant``: rows to microscaled 4-bit floating point (e2m1 with a scale a block of channels) and
  back to the values it stands for;
* ``swiglu``: SwiGLU of the experts' first products whose result is held in 4 bits, the operand of
  the second products;
* ``experts``: the experts' matrix products over ragged groups of rows, rows and weights both in
  4 bits;
* ``layer``: the whole layer (gate, routing, both products, the weighted sum) for a few tokens,
  with weights in 16 or in 4 bits.

4-bit tensors are of one of two formats. ``mx``: blocks of 32 channels, scale 2^(byte - 127), the
least power of two with every |value| / scale <= 6. ``nv``: blocks of 16 channels, scale an e4m3
number, amax / (6 g) rounded, with one 32-bit g for all rows or for each expert; a value is
code * scale * g. Codes are rounded to even, the low half of a byte first; a row of scales is
filled up to a multiple of 16 bytes.

``own = False`` computes them with elementary torch operations in 32 bits (64 where a value is
rounded to 4 bits, and in the gate), ``own = True`` with the framework's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = {"mx": 32, "nv": 16}
E4M3_MAX = 448.0
E2M1_MAX = 6.0

# The routing methods' codes, as the framework's moe_route takes them.
SOFTMAX_ALL, SOFTMAX_CHOSEN, GROUPED_BIASED, SIGMOID_SUM = 0, 1, 2, 6


def listed():
    return [
        # The rows of a prefill batch at the dsv3_layer width, before the first products.
        dict(name="quant_prefill", op="quant", R=8192, H=7168, fmt="nv", dtype="bf16"),
        # One decode step's rows, f16, with a last block that ends inside a vector: latency.
        dict(name="quant_decode_f16", op="quant", R=67, H=1504, fmt="mx", dtype="f16"),
        # Between the products of a prefill batch (mixtral_prefill's rows and I).
        dict(name="swiglu_prefill", op="swiglu", R=8192, I=14336, fmt="mx", dtype="bf16"),
        # Between the products of a decode step (qwen3_decode's 64 * 8 rows): latency.
        dict(name="swiglu_decode", op="swiglu", R=512, I=768, fmt="nv", dtype="bf16"),
        # The first products of a decode step: 512 rows over 128 experts, weights read once.
        dict(name="experts_decode", op="experts", R=512, E=128, K=2048, N=1536, fmt="nv",
             out="bf16", skew=0.0),
        # The first products of a prefill batch (mixtral_prefill): few experts, many rows.
        dict(name="experts_prefill", op="experts", R=8192, E=8, K=4096, N=28672, fmt="nv",
             out="bf16", skew=0.0),
        # The second products of the dsv3_layer workload: 16 rows an expert on average.
        dict(name="experts_many", op="experts", R=4096, E=256, K=2048, N=7168, fmt="mx",
             out="bf16", skew=0.3),
        # Uneven groups, and sizes that end inside every kind of tile.
        dict(name="experts_odd", op="experts", R=1941, E=54, K=1504, N=1000, fmt="mx",
             out="f16", skew=1.0),
        # One token through qwen3_decode's layer: latency.
        dict(name="layer_one", op="layer", T=1, H=2048, I=768, E=128, k=8, weights="bf16",
             dtype="bf16", method=SOFTMAX_CHOSEN, n_group=1, topk_group=1, rsf=1.0, shared=0),
        # Four sequences through mixtral_prefill's layer: most of the experts are read.
        dict(name="layer_four", op="layer", T=4, H=4096, I=14336, E=8, k=2, weights="bf16",
             dtype="bf16", method=SOFTMAX_CHOSEN, n_group=1, topk_group=1, rsf=1.0, shared=0),
        # Sixteen sequences through the dsv3_layer workload's layer with 4-bit weights, its shared
        # expert and its grouped routing.
        dict(name="layer_sixteen_nv", op="layer", T=16, H=7168, I=2048, E=256, k=8, weights="nv",
             dtype="bf16", method=GROUPED_BIASED, n_group=8, topk_group=4, rsf=2.5, shared=2048),
        # Odd numbers of tokens, experts and channels, f16 rows, 4-bit weights.
        dict(name="layer_odd_mx", op="layer", T=5, H=1504, I=736, E=60, k=4, weights="mx",
             dtype="f16", method=SIGMOID_SUM, n_group=1, topk_group=1, rsf=1.0, shared=352),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _by32(n):
    return max(32, n // 32 * 32)


def draw(rng):
    op = rng.choice(("quant", "swiglu", "experts", "experts", "layer", "layer"))
    fmt = rng.choice(("mx", "nv"))
    if op in ("quant", "swiglu"):
        case = dict(op=op, R=_log(rng, 1, 8192), fmt=fmt,
                    dtype=rng.choice(("bf16", "bf16", "f16", "f32")))
        case["H" if op == "quant" else "I"] = _by32(_log(rng, 64, 7168 if op == "quant" else 14336))
        return case
    if op == "experts":
        while True:
            E = _log(rng, 1, 256)
            R = _log(rng, 1, 32768)
            K = _by32(_log(rng, 64, 14336))
            N = _log(rng, 64, 28672) // 8 * 8
            if 2 * R * K * N <= 1.9e12 and E * K * N <= 256 * 2048 * 7168:
                break
        return dict(op=op, R=R, E=E, K=K, N=N, fmt=fmt, out=rng.choice(("bf16", "bf16", "f16")),
                    skew=round(rng.uniform(0, 1), 2))
    weights = rng.choice(("16", "mx", "nv"))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    grouped = rng.random() < 0.3
    while True:
        E = rng.choice((16, 32, 64, 128, 256)) if grouped else _log(rng, 4, 256)
        H = _by32(_log(rng, 128, 7168))
        I = _by32(_log(rng, 128, 14336))
        if E * H * I <= 256 * 2048 * 7168 / (4 if weights == "16" else 1):
            break
    return dict(op="layer", T=rng.randint(1, 16), H=H, I=I, E=E, k=rng.randint(1, min(8, E // 2)),
                weights=dtype if weights == "16" else weights, dtype=dtype,
                method=GROUPED_BIASED if grouped else rng.choice((SOFTMAX_ALL, SOFTMAX_CHOSEN,
                                                                  SIGMOID_SUM)),
                n_group=4 if grouped else 1, topk_group=2 if grouped else 1,
                rsf=2.5 if grouped else 1.0, shared=rng.choice((0, 0, I)))


# --------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(shape, g, dtype, std=1.0):
    """Normal values of the type, drawn a slice at a time so that no large f32 copy exists."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    step = 1 << 28
    for at in range(0, flat.numel(), step):
        part = flat[at:at + step]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(std))
    return out


def _scale_columns(K, fmt):
    return -(-(K // BLOCK[fmt]) // 16) * 16


def _four_bits(shape, g, fmt, std):
    """Normal values held in 4 bits, [rows, K] or [experts, rows, K]: (codes, scales, g or None)."""
    planes = shape[0] if len(shape) == 3 else 1
    rows, K = shape[-2:]
    codes = torch.empty((planes, rows, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((planes, rows, _scale_columns(K, fmt)), dtype=torch.uint8, device="cuda")
    # a calibrated range: five deviations are the largest value
    top = torch.full((planes,), 5.0 * std / (E2M1_MAX * E4M3_MAX), device="cuda") if fmt == "nv" else None
    step = max(1, (1 << 26) // K)
    for p in range(planes):
        for at in range(0, rows, step):
            n = min(step, rows - at)
            v = torch.randn((n, K), generator=g, device="cuda").mul_(std)
            codes[p, at:at + n], scales[p, at:at + n] = _to_codes(v, fmt, None if top is None else top[p], torch.float32)
    return codes.view(*shape[:-1], -1), scales.view(*shape[:-1], -1), top


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    op = case["op"]
    if op in ("quant", "swiglu"):
        R, dt = case["R"], DTYPES[case["dtype"]]
        cols = case["H"] if op == "quant" else 2 * case["I"]
        # the channels of unequal size, as activations have them
        size = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
        x = torch.empty((R, cols), dtype=dt, device="cuda")
        for at in range(0, R, 4096):
            part = x[at:at + 4096]
            part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(size))
        s["x"] = x
        s["g"] = torch.full((1,), 30.0 / (E2M1_MAX * E4M3_MAX), device="cuda") if case["fmt"] == "nv" else None
    elif op == "experts":
        R, E, K, N = case["R"], case["E"], case["K"], case["N"]
        p = torch.softmax(torch.randn(E, generator=g, device="cuda") * case["skew"], 0)
        e = torch.multinomial(p, R, replacement=True, generator=g)
        s["offsets"] = torch.cat([e.new_zeros(1), torch.bincount(e, minlength=E).cumsum(0)]).to(torch.int32)
        s["x"] = _four_bits((R, K), g, case["fmt"], 1.0)
        s["w"] = _four_bits((E, N, K), g, case["fmt"], K ** -0.5)
    else:
        T, H, I, E, dt = case["T"], case["H"], case["I"], case["E"], DTYPES[case["dtype"]]
        s["x"] = _randn((T, H), g, dt)
        s["wg"] = _randn((E, H), g, dt, H ** -0.5)
        s["bias"] = (torch.randn(E, generator=g, device="cuda") * 0.1
                     if case["method"] == GROUPED_BIASED else None)
        shapes = {"w13": (E, 2 * I, H), "w2": (E, H, I)}
        if case["shared"]:
            shapes.update(w13_s=(2 * case["shared"], H), w2_s=(H, case["shared"]))
        for name, shape in shapes.items():
            std = shape[-1] ** -0.5
            s[name] = (_four_bits(shape, g, case["weights"], std) if case["weights"] in BLOCK
                       else _randn(shape, g, dt, std))
    return s


# ------------------------------------------------------------------------------ plain form

def _to_codes(v, fmt, g, wide=torch.float64):
    """v [rows, K] to 4 bits: (codes [rows, K / 2], scales filled up to 16 columns)."""
    rows, K = v.shape
    b = v.to(wide).view(rows, -1, BLOCK[fmt])
    top = b.abs().amax(2)
    if fmt == "mx":
        m, e = torch.frexp(top)                            # top = m 2^e, m in [0.5, 1); 6 = 0.75 2^3
        e = (e - 3 + (m > 0.75).to(e.dtype)).clamp(-127, 127)
        e = torch.where(top == 0, torch.full_like(e, -127), e)
        byte = (e + 127).to(torch.uint8)
        unit = torch.ldexp(torch.ones_like(top), e)
    else:
        q = (top / (E2M1_MAX * g.to(wide))).clamp(max=E4M3_MAX).float().to(torch.float8_e4m3fn)
        byte = q.view(torch.uint8)
        unit = q.to(wide) * g.to(wide)
    a = b.abs() / torch.where(unit == 0, torch.full_like(unit, math.inf), unit)[:, :, None]
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(b).to(torch.uint8)).view(rows, K // 2, 2)
    scales = torch.zeros((rows, _scale_columns(K, fmt)), dtype=torch.uint8, device=v.device)
    scales[:, :byte.shape[1]] = byte
    return code[:, :, 0] + 16 * code[:, :, 1], scales


def _values(codes, scales, g, fmt, wide=torch.float32):
    """What the codes [..., K / 2] stand for, without g where that is one for each plane."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=wide, device=codes.device)
    table = torch.cat([table, -table])
    pair = torch.stack([codes & 15, codes >> 4], -1)
    v = table[pair.int()].flatten(-2)
    blocks = v.shape[-1] // BLOCK[fmt]
    sc = scales[..., :blocks]
    if fmt == "mx":
        sc = torch.ldexp(torch.ones((), dtype=wide, device=codes.device), sc.int() - 127)
    else:
        sc = sc.contiguous().view(torch.float8_e4m3fn).to(wide)
    v = (v.unflatten(-1, (blocks, BLOCK[fmt])) * sc[..., None]).flatten(-2)
    if g is not None:
        v = v * (g.to(wide) if g.numel() == 1 else g.to(wide)[:, None, None])
    return v


def _plain_quant(s):
    fmt = s["case"]["fmt"]
    codes, scales = _to_codes(s["x"], fmt, s["g"])
    return {"values": _values(codes, scales, s["g"], fmt).to(s["x"].dtype)}


def _plain_swiglu(s):
    fmt, x = s["case"]["fmt"], s["x"]
    I = s["case"]["I"]
    out = torch.empty((x.shape[0], I), dtype=x.dtype, device=x.device)
    for at in range(0, x.shape[0], 2048):
        part = x[at:at + 2048].double()
        h = part[:, :I] * torch.sigmoid(part[:, :I]) * part[:, I:]
        codes, scales = _to_codes(h, fmt, s["g"])
        out[at:at + 2048] = _values(codes, scales, s["g"], fmt).to(x.dtype)
    return {"values": out}


def _plain_experts(s):
    case = s["case"]
    fmt, E, R, N = case["fmt"], case["E"], case["R"], case["N"]
    off = s["offsets"]
    counts = off[1:] - off[:-1]
    most = max(1, int(counts.max()))
    at = torch.arange(most, device=off.device)
    place = (off[:-1, None] + at).clamp(max=R - 1).long()
    there = at < counts[:, None]
    x = _values(*s["x"], fmt)
    y = torch.empty((R, N), dtype=DTYPES[case["out"]], device=off.device)
    codes, scales, g = s["w"]
    step = max(1, (1 << 32) // (N * (codes.shape[-1] * 2 + most)))
    for e in range(0, E, step):
        w = _values(codes[e:e + step], scales[e:e + step], None if g is None else g[e:e + step], fmt)
        got = torch.bmm(x[place[e:e + step]], w.transpose(1, 2))
        y[place[e:e + step][there[e:e + step]]] = got[there[e:e + step]].to(y.dtype)
    return {"y": y}


def _route(logits, case, bias):
    """(ids, weights) of logits in 64 bits; ties to the lower index, slots by descending key."""
    k, method = case["k"], case["method"]

    def best(key):
        return key.sort(dim=1, descending=True, stable=True).indices[:, :k]

    if method in (SOFTMAX_ALL, SOFTMAX_CHOSEN):
        ids = best(logits)
        p = torch.softmax(logits, 1) if method == SOFTMAX_ALL else torch.softmax(logits.gather(1, ids), 1)
        return ids, p.gather(1, ids) if method == SOFTMAX_ALL else p
    score = torch.sigmoid(logits)
    if method == SIGMOID_SUM:
        ids = best(logits)
        p = score.gather(1, ids)
        return ids, p / p.sum(1, keepdim=True)
    key = score.float() + bias
    groups = key.view(key.shape[0], case["n_group"], -1)
    two = groups.topk(2, dim=2).values.sum(2)
    kept = two.sort(dim=1, descending=True, stable=True).indices[:, :case["topk_group"]]
    there = torch.zeros_like(two, dtype=torch.bool).scatter(1, kept, True)
    ids = best(torch.where(there[:, :, None], groups, torch.full_like(groups, -math.inf)).flatten(1))
    p = score.gather(1, ids)
    return ids, p / (p.sum(1, keepdim=True) + 1e-20) * case["rsf"]


def _weights(s, name, at, wide=torch.float32):
    """The weights of the experts `at` (or, None, of the shared one)."""
    w = s[name]
    if not isinstance(w, tuple):
        return (w if at is None else w[at]).to(wide)
    codes, scales, g = w
    if at is not None:
        codes, scales, g = codes[at], scales[at], None if g is None else g[at]
    return _values(codes, scales, g, s["case"]["weights"], wide)


def _plain_layer(s):
    case, x = s["case"], s["x"]
    I = case["I"]
    ids, p = _route(x.double() @ s["wg"].double().t(), case, s["bias"])
    xf, pf = x.float(), p.float()
    y = torch.zeros_like(xf)
    for t in range(case["T"]):
        a = (_weights(s, "w13", ids[t]) * xf[t]).sum(2)
        h = a[:, :I] * torch.sigmoid(a[:, :I]) * a[:, I:]
        y[t] = ((_weights(s, "w2", ids[t]) * h[:, None, :]).sum(2) * pf[t, :, None]).sum(0)
    if case["shared"]:
        a = xf @ _weights(s, "w13_s", None).t()
        h = a[:, :case["shared"]] * torch.sigmoid(a[:, :case["shared"]]) * a[:, case["shared"]:]
        y += h @ _weights(s, "w2_s", None).t()
    return {"y": y.to(x.dtype), "ids": ids.to(torch.int32), "scales": pf}


# ------------------------------------------------------------------- the framework's calls

def _own(s):
    import mixture_experts_layer_03_gb300 as moe
    case = s["case"]
    fmts = {"mx": moe.MOE_FP4_MX, "nv": moe.MOE_FP4_NV}
    if case["op"] == "quant":
        q = moe.moe_quantize_fp4(s["x"], fmts[case["fmt"]], s["g"])
        return {"values": moe.moe_dequantize_fp4(q, s["x"].dtype)}
    if case["op"] == "swiglu":
        q = moe.moe_swiglu_fp4(s["x"], fmts[case["fmt"]], s["g"])
        return {"values": moe.moe_dequantize_fp4(q, s["x"].dtype)}
    if case["op"] == "experts":
        fmt = fmts[case["fmt"]]
        return {"y": moe.moe_experts_matmul_fp4(moe.Fp4(s["x"][0], s["x"][1], fmt, s["x"][2]),
                                                moe.Fp4(s["w"][0], s["w"][1], fmt, s["w"][2]),
                                                s["offsets"], DTYPES[case["out"]])}

    def weights(name):
        w = s.get(name)
        return moe.Fp4(w[0], w[1], fmts[case["weights"]], w[2]) if isinstance(w, tuple) else w

    y, ids, scales = moe.moe_layer_few(
        s["x"], s["wg"], weights("w13"), weights("w2"), case["method"], case["k"], bias=s["bias"],
        n_group=case["n_group"], topk_group=case["topk_group"], routed_scaling_factor=case["rsf"],
        w13_s=weights("w13_s"), w2_s=weights("w2_s"))
    return {"y": y, "ids": ids, "scales": scales}


def run(state):
    if own:
        return _own(state)
    return {"quant": _plain_quant, "swiglu": _plain_swiglu, "experts": _plain_experts,
            "layer": _plain_layer}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------ work

def _held(rows, K, kind):
    """Bytes of rows of K channels as they are held."""
    if kind in BLOCK:
        return rows * (K // 2 + K // BLOCK[kind])
    return rows * K * BYTES[kind]


def work(case):
    op = case["op"]
    if op in ("quant", "swiglu"):
        R, b = case["R"], BYTES[case["dtype"]]
        out = case["H"] if op == "quant" else case["I"]
        read = out if op == "quant" else 2 * out
        # rows in, 4 bits out; 4 bits in, values out
        return {"bytes": R * read * b + 2 * _held(R, out, case["fmt"]) + R * out * b,
                "flops": R * out * (4 if op == "quant" else 12)}
    if op == "experts":
        R, E, K, N, fmt = case["R"], case["E"], case["K"], case["N"], case["fmt"]
        reached = E * (1 - (1 - 1 / E) ** R)        # experts that some row is expected to reach
        return {"bytes": _held(R, K, fmt) + reached * _held(N, K, fmt) + R * N * BYTES[case["out"]],
                "flops": 2 * R * N * K}
    T, H, I, E, k, kind = case["T"], case["H"], case["I"], case["E"], case["k"], case["weights"]
    reached = E * (1 - (1 - k / E) ** T)
    an_expert = _held(2 * I, H, kind) + _held(H, I, kind)
    shared = _held(2 * case["shared"], H, kind) + _held(H, case["shared"], kind) if case["shared"] else 0
    return {"bytes": int(reached * an_expert + shared + E * H * 2 + 4 * T * H + 8 * T * k),
            "flops": 6 * T * H * (k * I + case["shared"]) + 2 * T * E * H}


# --------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The definitions in 64 bits."""
    s = prepare(case, seed)
    return {"quant": _exact_rows, "swiglu": _exact_rows, "experts": _exact_experts,
            "layer": _exact_layer}[case["op"]](s, case)


def _exact_rows(s, case):
    x = s["x"]
    R, block = x.shape[0], BLOCK[case["fmt"]]
    out = torch.empty((R, case.get("H") or case["I"]), dtype=torch.float64, device="cuda")
    for a in range(0, R, 1024):
        v = x[a:a + 1024].double()
        if case["op"] == "swiglu":
            gate, up = v.chunk(2, 1)
            v = gate / (1 + torch.exp(-gate)) * up
        b = v.reshape(v.shape[0], -1, block)
        top = b.abs().max(2, keepdim=True).values
        if case["fmt"] == "mx":
            # the least power of two >= top / 6, no less than 2^-127
            want = (top / 6).clamp(min=2.0 ** -127)
            unit = torch.exp2(torch.ceil(torch.log2(want)))
            unit = torch.where(unit / 2 >= want, unit / 2, unit)
            unit = torch.where(unit < want, unit * 2, unit)
        else:
            # e4m3: m 2^(e - 3) with 8 <= m < 16, below 2^-6 multiples of 2^-9
            want = (top / (6 * s["g"].double())).clamp(max=448.0)
            step = torch.exp2(torch.floor(torch.log2(want.clamp(min=2.0 ** -6))) - 3)
            unit = torch.round(want / step) * step * s["g"].double()
        # e2m1: multiples of 1/2 up to 2, of 1 up to 4, of 2 up to 6, ties to the even multiple
        z = (b.abs() / torch.where(unit > 0, unit, torch.ones_like(unit))).clamp(max=6.0)
        z = torch.where(unit > 0, z, torch.zeros_like(z))
        step = torch.where(z < 2, 0.5, torch.where(z < 4, 1.0, 2.0)).to(torch.float64)
        z = (torch.round(z / step) * step).clamp(max=6.0)
        out[a:a + 1024] = (torch.sign(b) * z * unit).reshape(v.shape[0], -1)
    return {"values": out}


def _decoded(codes, scales, g, fmt):
    """What one plane of codes [rows, K / 2] stands for, in 64 bits."""
    both = torch.empty((codes.shape[0], codes.shape[1] * 2), dtype=torch.int64, device=codes.device)
    both[:, 0::2] = codes & 15
    both[:, 1::2] = codes >> 4
    e, m = (both >> 1) & 3, (both & 1).double()
    size = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2((e - 1).double()))
    v = torch.where(both >= 8, -size, size)
    block = BLOCK[fmt]
    byte = scales[:, :v.shape[1] // block].long()
    if fmt == "mx":
        sc = torch.exp2(byte.double() - 127)
    else:
        e, m = (byte >> 3) & 15, (byte & 7).double()
        sc = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).double())) * g.double()
    return v * sc.repeat_interleave(block, dim=1)


def _exact_experts(s, case):
    fmt = case["fmt"]
    x = _decoded(*s["x"], fmt)
    off = s["offsets"].tolist()
    y = torch.zeros((case["R"], case["N"]), dtype=torch.float64, device="cuda")
    codes, scales, g = s["w"]
    for e in range(case["E"]):
        a, b = off[e], off[e + 1]
        if b > a:
            y[a:b] = x[a:b] @ _decoded(codes[e], scales[e], None if g is None else g[e], fmt).t()
    return {"y": y}


def _exact_layer(s, case):
    x = s["x"].double()
    T, k, E, method = case["T"], case["k"], case["E"], case["method"]
    logits = (x @ s["wg"].double().t()).cpu().tolist()
    bias = [0.0] * E if s["bias"] is None else s["bias"].double().cpu().tolist()
    ids = torch.empty((T, k), dtype=torch.int64)
    weights = torch.empty((T, k), dtype=torch.float64)
    for t, l in enumerate(logits):
        sig = [1 / (1 + math.exp(-v)) for v in l]
        allowed = list(range(E))
        key = l
        if method == GROUPED_BIASED:
            key = (torch.tensor(sig).float() + torch.tensor(bias).float()).tolist()
            size = E // case["n_group"]
            rank = sorted(range(case["n_group"]), key=lambda gr: (
                -sum(sorted(key[gr * size:(gr + 1) * size])[-2:]), gr))
            allowed = [e for gr in rank[:case["topk_group"]] for e in range(gr * size, (gr + 1) * size)]
        chosen = sorted(allowed, key=lambda e: (-key[e], e))[:k]
        if method in (SOFTMAX_ALL, SOFTMAX_CHOSEN):
            top = max(l)
            ex = [math.exp(l[e] - top) for e in chosen]
            total = sum(math.exp(v - top) for v in l) if method == SOFTMAX_ALL else sum(ex)
        else:
            ex = [sig[e] for e in chosen]
            total = sum(ex)
        ids[t] = torch.tensor(chosen)
        weights[t] = torch.tensor([v / total * case["rsf"] for v in ex], dtype=torch.float64)

    def expert(xs, w13, w2):
        a = xs @ w13.t()
        gate, up = a.chunk(2, 1)
        return (gate / (1 + torch.exp(-gate)) * up) @ w2.t()

    def matrix(name, e):
        w = s[name]
        if not isinstance(w, tuple):
            return (w if e is None else w[e]).double()
        codes, scales, g = w
        if e is None:
            return _decoded(codes, scales, g, case["weights"])
        return _decoded(codes[e], scales[e], None if g is None else g[e], case["weights"])

    y = torch.zeros_like(x)
    for e in sorted(set(ids.flatten().tolist())):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        part = expert(x[t.cuda()], matrix("w13", e), matrix("w2", e))
        y.index_add_(0, t.cuda(), part * weights[t, j].cuda()[:, None])
    if case["shared"]:
        y += expert(x, matrix("w13_s", None), matrix("w2_s", None))
    return {"y": y, "ids": ids.to(torch.int32), "scales": weights}
