"""The operators of the MoE layer's training step: what is timed, and on which inputs.

Four operators, all over tokens routed to experts (T tokens, k slots a token, P = T * k rows,
E experts):

* ``sort``: rows of the tokens gathered by expert (dispatch) and summed back with the routing
  weights (combine), and both gradients;
* ``ckpt``: SwiGLU whose input is kept for the backward pass in 8 bits (e4m3 with one power of
  two per 32 channels), forward and backward;
* ``experts``: the experts' matrix products over ragged groups of rows, forward (``y = x w^T``)
  and backward (``dx = dy w``, ``dw = dy^T x``);
* ``route``: the gradient of the routing weights to the router's logits.

``own = False`` computes them with elementary torch operations in 32 bits, ``own = True`` with
the framework's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 32          # channels that share a scale in a checkpoint
E4M3_MAX = 448.0

# The routing methods' codes, as the framework's moe_route takes them.
SOFTMAX_ALL = (0,)                  # softmax over all experts, the chosen ones' probabilities
SOFTMAX_CHOSEN = (1, 4)             # softmax over the chosen
SIGMOID = (3,)                      # sigmoid of each chosen logit
SIGMOID_SUM = (2, 5, 6, 16)         # sigmoid over the chosen ones' sum (2 and 16 times a factor)


def listed():
    return [
        # One decode step of 64 sequences: latency. (T, H, E, k of the qwen3_decode workload)
        dict(name="sort_decode", op="sort", direction="forward", T=64, H=2048, E=128, k=8,
             dtype="bf16", skew=0.0, drop=0.0),
        # A prefill batch on few, unevenly loaded experts (the skewed workload's shape).
        dict(name="sort_prefill", op="sort", direction="forward", T=8192, H=4096, E=64, k=4,
             dtype="bf16", skew=1.0, drop=0.0),
        # The backward pass of a training micro-batch at the dsv3_layer width.
        dict(name="sort_train_grad", op="sort", direction="backward", T=8192, H=7168, E=256, k=8,
             dtype="bf16", skew=0.5, drop=0.0),
        # f32 rows of an odd width, and slots dropped by a capacity limit.
        dict(name="sort_odd_f32", op="sort", direction="both", T=1537, H=1001, E=60, k=6,
             dtype="f32", skew=0.5, drop=0.1),
        # SwiGLU of a training micro-batch, forward and backward (mixtral_prefill's rows and I).
        dict(name="ckpt_train", op="ckpt", R=8192, I=14336, dtype="bf16"),
        # Few rows, f16, and a width whose last block of 32 is short: latency.
        dict(name="ckpt_small_f16", op="ckpt", R=131, I=1000, dtype="f16"),
        # The first products of a decode step: 512 rows over 128 experts, weights read once.
        dict(name="experts_decode", op="experts", direction="forward", R=512, E=128, K=2048,
             N=1536, dtype="bf16", skew=0.0, drop=0.0),
        # The second products of a prefill batch (mixtral_prefill): few experts, many rows.
        dict(name="experts_prefill", op="experts", direction="forward", R=8192, E=8, K=14336,
             N=4096, dtype="bf16", skew=0.0, drop=0.0),
        # Backward of the skewed workload's second products: uneven groups of hundreds of rows.
        dict(name="experts_grad", op="experts", direction="backward", R=32768, E=64, K=1536,
             N=4096, dtype="bf16", skew=0.5, drop=0.0),
        # Backward over many experts with about 128 rows each (the dsv3_layer widths): the
        # weights and their gradients are most of the traffic.
        dict(name="experts_grad_many", op="experts", direction="backward", R=32768, E=256,
             K=2048, N=7168, dtype="bf16", skew=0.3, drop=0.0),
        # The router's gradient of a training micro-batch: sigmoid scores over 256 experts.
        dict(name="route_sigmoid", op="route", T=8192, E=256, k=8, method=2, rsf=2.5),
        # A small batch with the softmax over all experts, an odd number of them.
        dict(name="route_softmax", op="route", T=300, E=60, k=4, method=0, rsf=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("sort", "ckpt", "experts", "experts", "route"))
    if op == "sort":
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        E = _log(rng, 4, 256)
        k = rng.randint(1, min(8, E))
        T = _log(rng, 1, 8192)
        H = _log(rng, 64, 7168)
        if rng.random() < 0.7:
            H = H // 8 * 8
        return dict(op=op, direction=rng.choice(("forward", "backward", "both")), T=T, H=H, E=E,
                    k=k, dtype=dtype, skew=round(rng.uniform(0, 1), 2),
                    drop=rng.choice((0.0, 0.0, 0.05, 0.5)))
    if op == "ckpt":
        return dict(op=op, R=_log(rng, 1, 8192), I=_log(rng, 64, 14336),
                    dtype=rng.choice(("bf16", "bf16", "f16", "f32")))
    if op == "experts":
        while True:
            E = _log(rng, 1, 256)
            R = _log(rng, 1, 32768)
            K = _log(rng, 64, 14336) // 8 * 8
            N = _log(rng, 64, 14336) // 8 * 8
            if 4 * R * K * N <= 1.9e12 and E * K * N <= 256 * 2048 * 7168 and 3072 not in (K, N):
                break
        return dict(op=op, direction=rng.choice(("forward", "backward")), R=R, E=E, K=K, N=N,
                    dtype=rng.choice(("bf16", "bf16", "f16")), skew=round(rng.uniform(0, 0.5), 2),
                    drop=rng.choice((0.0, 0.0, 0.1)))
    E = _log(rng, 8, 256)
    method = rng.choice(SOFTMAX_ALL + SOFTMAX_CHOSEN + SIGMOID + SIGMOID_SUM)
    return dict(op=op, T=_log(rng, 1, 16384), E=E, k=rng.randint(1, min(8, E)), method=method,
                rsf=2.5 if method in (2, 16) else 1.0)


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


def _choices(T, E, k, skew, g):
    """Each token's k experts: the largest of its random scores plus a fixed bias an expert."""
    bias = torch.randn(E, generator=g, device="cuda") * skew
    score = torch.randn((T, E), generator=g, device="cuda") + bias
    return score.topk(k, dim=1).indices.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "sort":
        T, H, E, k, dt = case["T"], case["H"], case["E"], case["k"], DTYPES[case["dtype"]]
        ids = _choices(T, E, k, case["skew"], g)
        if case["drop"] > 0:
            gone = torch.rand((T, k), generator=g, device="cuda") < case["drop"]
            ids = torch.where(gone, torch.full_like(ids, -1), ids)
        s["ids"] = ids.contiguous()
        w = torch.rand((T, k), generator=g, device="cuda") + 0.1
        s["scales"] = (w / w.sum(1, keepdim=True)).contiguous()
        s["rows"] = _randn((T * k, H), g, dt)
        if case["direction"] != "backward":
            s["x"] = _randn((T, H), g, dt)
        if case["direction"] != "forward":
            s["dy"] = _randn((T, H), g, dt)
            s["dx_perm"] = _randn((T * k, H), g, dt)
            # the map that the forward pass kept
            s["inv"], _ = _sorted(s["ids"], E)
    elif case["op"] == "ckpt":
        R, I, dt = case["R"], case["I"], DTYPES[case["dtype"]]
        # pre-activations: unit normal, the channels of unequal size
        size = torch.exp(0.5 * torch.randn(2 * I, generator=g, device="cuda"))
        gu = torch.empty((R, 2 * I), dtype=dt, device="cuda")
        for at in range(0, R, 4096):
            part = gu[at:at + 4096]
            part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(size))
        s["gu"] = gu
        s["dh"] = _randn((R, I), g, dt)
    elif case["op"] == "experts":
        R, E, K, N, dt = case["R"], case["E"], case["K"], case["N"], DTYPES[case["dtype"]]
        p = torch.softmax(torch.randn(E, generator=g, device="cuda") * case["skew"], 0)
        kept = R - int(R * case["drop"])
        e = torch.multinomial(p, kept, replacement=True, generator=g) if kept else p.new_zeros(0, dtype=torch.int64)
        s["offsets"] = torch.cat([e.new_zeros(1), torch.bincount(e, minlength=E).cumsum(0)]).to(torch.int32)
        s["x"] = _randn((R, K), g, dt)
        s["w"] = _randn((E, N, K), g, dt, K ** -0.5)
        if case["direction"] == "backward":
            s["dy"] = _randn((R, N), g, dt)
    else:
        T, E, k = case["T"], case["E"], case["k"]
        logits = torch.randn((T, E), generator=g, device="cuda") * 1.5
        s["logits"] = logits
        # chosen by the logits (a selection bias, as the biased methods have, moves some)
        s["ids"] = (logits + 0.1 * torch.randn(E, generator=g, device="cuda")).topk(k, dim=1).indices.to(torch.int32).contiguous()
        s["dscales"] = torch.randn((T, k), generator=g, device="cuda")
    return s


# ------------------------------------------------------------------------------ plain form

def _sorted(ids, E):
    """(inv [T, k], offsets [E+1]): the place of each slot in the stable order by expert;
    dropped slots come last and their place r is held as -1 - r."""
    f = ids.reshape(-1).long()
    key = torch.where(f < 0, torch.full_like(f, E), f)
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=ids.device)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return (torch.where(f < 0, -1 - place, place).view(ids.shape).to(torch.int32),
            offsets.to(torch.int32))


def _gathered_sum(rows, inv, scales):
    T, k = inv.shape
    kept = inv >= 0
    picked = rows[inv.clamp(min=0).long()].float()
    picked = torch.where(kept[:, :, None], picked, torch.zeros_like(picked))
    if scales is not None:
        picked = picked * scales[:, :, None]
    return picked.sum(1).to(rows.dtype)


def _plain_sort_forward(s):
    ids, x = s["ids"], s["x"]
    T, k = ids.shape
    inv, offsets = _sorted(ids, s["case"]["E"])
    place = torch.where(inv < 0, -1 - inv, inv).long().reshape(-1)
    x_perm = torch.empty((T * k, x.shape[1]), dtype=x.dtype, device=x.device)
    spread = x[:, None, :].expand(T, k, x.shape[1])
    x_perm[place] = torch.where((inv >= 0)[:, :, None], spread, torch.zeros_like(spread)).reshape(T * k, -1)
    return {"x_perm": x_perm, "inv": inv, "offsets": offsets,
            "y": _gathered_sum(s["rows"], inv, s["scales"])}


def _plain_sort_backward(s):
    dy, rows, inv, scales = s["dy"], s["rows"], s["inv"], s["scales"]
    T, k = inv.shape
    kept = (inv >= 0)[:, :, None]
    place = torch.where(inv < 0, -1 - inv, inv).long()
    spread = dy.float()[:, None, :]
    drows = torch.empty_like(rows)
    drows[place.reshape(-1)] = torch.where(kept, spread * scales[:, :, None], torch.zeros_like(spread)).reshape(T * k, -1).to(rows.dtype)
    dscales = torch.where(kept[:, :, 0], (rows[place].float() * spread).sum(2), torch.zeros_like(scales))
    return {"drows": drows, "dscales": dscales, "dx": _gathered_sum(s["dx_perm"], inv, None)}


def _through_8_bits(v):
    """v [R, C] in 32 bits as its checkpoint holds it: per 32 channels one power of two, the
    least with every |value| / scale <= 448, and values of 8 bits (4 of them exponent)."""
    R, C = v.shape
    pad = -C % BLOCK
    b = torch.nn.functional.pad(v, (0, pad)).view(R, -1, BLOCK)
    m, e = torch.frexp(b.abs().amax(2, keepdim=True))         # amax = m 2^e, m in [0.5, 1)
    # 448 = 0.875 * 2^9
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-127)
    scale = torch.ldexp(torch.ones_like(m), e)
    q = (b / scale).to(torch.float8_e4m3fn).float() * scale
    return q.view(R, -1)[:, :C]


def _plain_ckpt(s):
    gu, dh = s["gu"].float(), s["dh"].float()
    I = dh.shape[1]
    g, u = gu[:, :I], gu[:, I:]
    h = g * torch.sigmoid(g) * u
    g, u = _through_8_bits(g), _through_8_bits(u)
    sig = torch.sigmoid(g)
    dgu = torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], 1)
    h2 = g * sig * u
    dt = s["gu"].dtype
    return {"h": h.to(dt), "dgu": dgu.to(dt), "h_again": h2.to(dt)}


def _padded(offsets, R):
    """Places [E, most] of each expert's rows, and which of them exist."""
    counts = offsets[1:] - offsets[:-1]
    most = max(1, int(counts.max()))
    at = torch.arange(most, device=offsets.device)
    return (offsets[:-1, None] + at).clamp(max=R - 1).long(), at < counts[:, None]


def _plain_experts(s):
    x, w = s["x"], s["w"]
    place, there = _padded(s["offsets"], x.shape[0])
    keep = there[:, :, None].float()
    if s["case"]["direction"] == "forward":
        got = torch.bmm(x[place].float() * keep, w.float().transpose(1, 2))
        y = torch.zeros((x.shape[0], w.shape[1]), dtype=x.dtype, device=x.device)
        y[place[there]] = got[there].to(x.dtype)
        return {"y": y}
    dy = s["dy"]
    dyp = dy[place].float() * keep
    got = torch.bmm(dyp, w.float())
    dx = torch.zeros_like(x)
    dx[place[there]] = got[there].to(x.dtype)
    del got
    dw = torch.bmm(dyp.transpose(1, 2), x[place].float() * keep).to(w.dtype)
    return {"dx": dx, "dw": dw}


def _plain_route(s):
    logits, ids, ds = s["logits"], s["ids"].long(), s["dscales"]
    method, c = s["case"]["method"], s["case"]["rsf"]
    dl = torch.zeros_like(logits)
    if method in SOFTMAX_ALL:
        p = torch.softmax(logits, 1)
        full = dl.scatter(1, ids, ds)
        return {"dlogits": p * (full - (full * p).sum(1, keepdim=True))}
    chosen = logits.gather(1, ids)
    if method in SOFTMAX_CHOSEN:
        p = torch.softmax(chosen, 1)
        d = p * (ds - (ds * p).sum(1, keepdim=True))
    else:
        sig = torch.sigmoid(chosen)
        if method in SIGMOID:
            d = ds
        else:
            total = sig.sum(1, keepdim=True) + (1e-20 if method == 2 else 0.0)
            d = c * (ds - (ds * sig).sum(1, keepdim=True) / total) / total
        d = d * sig * torch.sigmoid(-chosen)
    return {"dlogits": dl.scatter(1, ids, d)}


# ------------------------------------------------------------------- the framework's calls

def _own(s):
    import mixture_experts_layer_03_gb300 as moe
    case = s["case"]
    if case["op"] == "sort":
        out = {}
        if case["direction"] != "backward":
            x_perm, inv, offsets = moe.moe_dispatch(s["x"], s["ids"], case["E"])
            out = {"x_perm": x_perm, "inv": inv, "offsets": offsets,
                   "y": moe.moe_combine(s["rows"], inv, s["scales"])}
        if case["direction"] != "forward":
            drows, dscales = moe.moe_combine_backward(s["dy"], s["rows"], s["inv"], s["scales"])
            out.update(drows=drows, dscales=dscales,
                       dx=moe.moe_dispatch_backward(s["dx_perm"], s["inv"]))
        return out
    if case["op"] == "ckpt":
        h, ckpt = moe.moe_swiglu_ckpt(s["gu"])
        dgu, again = moe.moe_swiglu_ckpt_backward(s["dh"], ckpt, want_h=True)
        return {"h": h, "dgu": dgu, "h_again": again}
    if case["op"] == "experts":
        if case["direction"] == "forward":
            return {"y": moe.moe_experts_matmul(s["x"], s["w"], s["offsets"])}
        return {"dx": moe.moe_experts_matmul_dx(s["dy"], s["w"], s["offsets"]),
                "dw": moe.moe_experts_matmul_dw(s["dy"], s["x"], s["offsets"])}
    return {"dlogits": moe.moe_route_backward(s["logits"], s["ids"], s["dscales"], case["method"],
                                              routed_scaling_factor=case["rsf"])}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "sort":
        out = {}
        if state["case"]["direction"] != "backward":
            out.update(_plain_sort_forward(state))
        if state["case"]["direction"] != "forward":
            out.update(_plain_sort_backward(state))
        return out
    return {"ckpt": _plain_ckpt, "experts": _plain_experts, "route": _plain_route}[op](state)


# ------------------------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op == "sort":
        T, H, k, E, b = case["T"], case["H"], case["k"], case["E"], BYTES[case["dtype"]]
        P = T * k
        bytes_ = flops = 0
        if case["direction"] != "backward":
            # ids, x -> x_perm, inv, offsets; rows, scales -> y
            bytes_ += 4 * P + T * H * b + P * H * b + 4 * P + 4 * (E + 1) + P * H * b + 4 * P + T * H * b
            flops += 2 * P * H
        if case["direction"] != "forward":
            # dy, rows, inv, scales -> drows, dscales; dx_perm -> dx
            bytes_ += T * H * b + 2 * P * H * b + 12 * P + P * H * b + T * H * b
            flops += 4 * P * H
        return {"bytes": bytes_, "flops": flops}
    if op == "ckpt":
        R, I, b = case["R"], case["I"], BYTES[case["dtype"]]
        kept = R * (2 * I + 2 * (-(-I // BLOCK)))
        return {"bytes": R * I * (2 * b + b) + kept + kept + R * I * (b + 2 * b + b), "flops": 40 * R * I}
    if op == "experts":
        R, E, K, N, b = case["R"], case["E"], case["K"], case["N"], BYTES[case["dtype"]]
        kept = R - int(R * case["drop"])
        # experts that some row is expected to reach (equal chances)
        reached = E * (1 - (1 - 1 / E) ** kept)
        if case["direction"] == "forward":
            return {"bytes": kept * K * b + R * N * b + reached * N * K * b, "flops": 2 * kept * N * K}
        return {"bytes": kept * (N + K) * b + R * K * b + reached * N * K * b + E * N * K * b,
                "flops": 4 * kept * N * K}
    T, E, k = case["T"], case["E"], case["k"]
    read = 4 * T * E if case["method"] in SOFTMAX_ALL else 4 * T * k
    return {"bytes": read + 8 * T * k + 4 * T * E, "flops": 10 * T * (E if case["method"] in SOFTMAX_ALL else k)}


# --------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The definitions in 64 bits, one token block, expert or row block at a time."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "sort":
        return _exact_sort(s, case)
    if op == "ckpt":
        return _exact_ckpt(s)
    if op == "experts":
        return _exact_experts(s, case)
    return _exact_route(s, case)


def _exact_sort(s, case):
    ids = s["ids"].cpu().reshape(-1).tolist()
    T, k, E = case["T"], case["k"], case["E"]
    lists = [[] for _ in range(E + 1)]
    for f, e in enumerate(ids):
        lists[e if e >= 0 else E].append(f)
    starts, order = [0], []
    for e in range(E + 1):
        order += lists[e]
        starts.append(len(order))
    place = [0] * (T * k)
    for r, f in enumerate(order):
        place[f] = r
    dev = s["rows"].device
    at = torch.tensor(place, dtype=torch.int64, device=dev).view(T, k)
    kept = torch.tensor([e >= 0 for e in ids], device=dev).view(T, k)
    kd = kept.double()
    w = s["scales"].double() * kd
    out = {}
    H = case["H"]
    step = max(1, (1 << 26) // (k * H))

    def summed(rows, weight):
        y = torch.empty((T, H), dtype=torch.float64, device=dev)
        for a in range(0, T, step):
            b = min(T, a + step)
            y[a:b] = torch.einsum("tkh,tk->th", rows[at[a:b]].double(), weight[a:b])
        return y

    if case["direction"] != "backward":
        src = torch.tensor(order, dtype=torch.int64, device=dev)
        x_perm = s["x"].double()[src // k]
        x_perm[starts[E]:] = 0
        out = {"x_perm": x_perm,
               "inv": torch.tensor([r if e >= 0 else ~r for r, e in zip(place, ids)], dtype=torch.int32).view(T, k),
               "offsets": torch.tensor(starts[:E + 1], dtype=torch.int32),
               "y": summed(s["rows"], w)}
    if case["direction"] != "forward":
        drows = torch.zeros((T * k, H), dtype=torch.float64, device=dev)
        dscales = torch.zeros((T, k), dtype=torch.float64, device=dev)
        for a in range(0, T, step):
            b = min(T, a + step)
            dy = s["dy"][a:b].double()
            drows[at[a:b].reshape(-1)] = (dy[:, None, :] * w[a:b, :, None]).reshape(-1, H)
            dscales[a:b] = torch.einsum("tkh,th->tk", s["rows"][at[a:b]].double(), dy) * kd[a:b]
        out.update(drows=drows, dscales=dscales, dx=summed(s["dx_perm"], kd))
    return out


def _exact_ckpt(s):
    R, I = s["dh"].shape
    h = torch.empty((R, I), dtype=torch.float64, device="cuda")
    h2 = torch.empty_like(h)
    dgu = torch.empty((R, 2 * I), dtype=torch.float64, device="cuda")

    def kept(v):
        """What the checkpoint holds of v: m 2^(e - 3) with 8 <= |m| < 16 (fewer bits below the
        smallest normal exponent -6), rounded to even, times the block's power of two."""
        n = -(-I // BLOCK)
        b = torch.zeros((v.shape[0], n * BLOCK), dtype=torch.float64, device=v.device)
        b[:, :I] = v
        b = b.view(-1, n, BLOCK)
        top = b.abs().max(2, keepdim=True).values / E4M3_MAX
        sc = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** -127))))
        sc = torch.where(sc / 2 >= top, sc / 2, sc).clamp(min=2.0 ** -127)
        z = b / sc
        e = torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6)))
        e = torch.where(torch.exp2(e) > z.abs(), e - 1, e).clamp(min=-6)
        unit = torch.exp2(e - 3)
        return (torch.round(z / unit) * unit * sc).view(v.shape[0], -1)[:, :I]

    for a in range(0, R, 1024):
        gu, dh = s["gu"][a:a + 1024].double(), s["dh"][a:a + 1024].double()
        g, u = gu[:, :I], gu[:, I:]
        h[a:a + 1024] = g / (1 + torch.exp(-g)) * u
        g, u = kept(g), kept(u)
        sg = 1 / (1 + torch.exp(-g))
        h2[a:a + 1024] = g * sg * u
        dgu[a:a + 1024, :I] = dh * u * (sg + g * sg * (1 - sg))
        dgu[a:a + 1024, I:] = dh * g * sg
    return {"h": h, "dgu": dgu, "h_again": h2}


def _exact_experts(s, case):
    off = s["offsets"].tolist()
    x, w = s["x"], s["w"]
    R, K = x.shape
    E, N = w.shape[:2]
    if case["direction"] == "forward":
        y = torch.zeros((R, N), dtype=torch.float64, device="cuda")
        for e in range(E):
            a, b = off[e], off[e + 1]
            if b > a:
                y[a:b] = x[a:b].double() @ w[e].double().t()
        return {"y": y}
    dx = torch.zeros((R, K), dtype=torch.float64, device="cuda")
    dw = torch.zeros((E, N, K), dtype=torch.float64, device="cuda")
    for e in range(E):
        a, b = off[e], off[e + 1]
        if b > a:
            dy = s["dy"][a:b].double()
            dx[a:b] = dy @ w[e].double()
            dw[e] = dy.t() @ x[a:b].double()
    return {"dx": dx, "dw": dw}


def _exact_route(s, case):
    """From the weights' own derivative, d s_i / d l_j summed over the slots i."""
    l, ids, ds = s["logits"].double(), s["ids"].long(), s["dscales"].double()
    T, E = l.shape
    method, c = case["method"], case["rsf"]
    dl = torch.zeros((T, E), dtype=torch.float64, device="cuda")
    rows = torch.arange(T, device="cuda")[:, None]
    if method in SOFTMAX_ALL:
        ex = torch.exp(l - l.max(1, keepdim=True).values)
        p = ex / ex.sum(1, keepdim=True)
        pc = p[rows, ids]
        dl = -p * (ds * pc).sum(1, keepdim=True)
        dl[rows, ids] += ds * pc
        return {"dlogits": dl}
    lc = l[rows, ids]
    if method in SIGMOID:
        a = 1 / (1 + torch.exp(-lc))
        dl[rows, ids] = ds * a * (1 - a)
        return {"dlogits": dl}
    if method in SOFTMAX_CHOSEN:
        a = torch.exp(lc - lc.max(1, keepdim=True).values)
        slope, total = a, a.sum(1, keepdim=True)
        c = 1.0
    else:
        a = 1 / (1 + torch.exp(-lc))
        slope = a * (1 - a)
        total = a.sum(1, keepdim=True) + (1e-20 if method == 2 else 0.0)
    # s_i = c a_i / total: d s_i / d l_j = c slope_j ([i = j] / total - a_i / total^2)
    dl[rows, ids] = c * slope * (ds / total - (ds * a).sum(1, keepdim=True) / total ** 2)
    return {"dlogits": dl}
