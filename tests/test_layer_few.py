"""GPU: the layer for a few tokens against float64 (the oracle's gate, routing and experts on the same
weights).

The bound of y is worked out element by element from the arithmetic: logits summed in fp32 (2^-24 of the
terms' magnitudes an addition that a term goes through), whose error reaches the routing weights; the
first products' sums in the tensor cores (H * 2^-23) through SwiGLU, whose slopes are at most 1.1 |u| and |silu(g)|; h's one rounding
(bf16 2^-8; otherwise 2^-11, or 2^-39 of the token's largest where that is more); the second products' sums
(2^-23 of the magnitudes a term) and y's rounding. Chosen experts are float64's, or ones that its keys set
apart from these by no more than the logits' errors."""
import numpy as np
import pytest
import torch

import oracle
from oracle import serve_oracle as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_03_gb300 as m
    return m


def n64(t):
    return t.detach().cpu().double().numpy()


def held(moe, shape, weights, dtype, gen, g=True):
    """(what the call takes, its values in float64)."""
    w = torch.randn(shape, generator=gen) * shape[-1] ** -0.5
    if weights == "16":
        w = w.to(DT[dtype])
        return w.cuda(), w.double().numpy()
    fmt = {"mx": ref.MX, "nv": ref.NV}[weights]
    planes = shape[0] if len(shape) == 3 else 1
    gs = None
    if weights == "nv" and g:
        gs = (w.view(planes, -1).abs().amax(1) / (6 * 448)).float()
    flat = w.double().numpy().reshape(planes, -1, shape[-1])
    codes, scales, values = [], [], []
    for p in range(planes):
        gp = None if gs is None else float(gs[p].double())
        c, s = ref.quantize(flat[p], fmt, gp)
        values.append(ref.dequantize(c, s, fmt, gp))
        s[:, shape[-1] // ref.BLOCK[fmt]:] = 255        # what fills a row up is not looked at
        codes.append(c)
        scales.append(s)
    t = lambda a: torch.from_numpy(np.concatenate(a)).view(*shape[:-1], -1).cuda()   # noqa: E731
    return moe.Fp4(t(codes), t(scales), fmt, None if gs is None else gs.cuda()), np.concatenate(values).reshape(shape)


class Layer:
    def __init__(self, moe, T, H, I, E, k, method, weights, dtype, shared=0, gate=False, n_group=1, topk_group=1,
                 rsf=1.0, seed=0, g=True):
        gen = torch.Generator().manual_seed(seed)
        self.moe, self.k, self.method, self.dtype, self.weights = moe, k, method, dtype, weights
        size = torch.exp(torch.randn((T, 1), generator=gen))
        self.x = (torch.randn((T, H), generator=gen) * size).to(DT[dtype]).cuda()
        self.wg = (torch.randn((E + gate, H), generator=gen) * H ** -0.5).to(DT[dtype]).cuda()
        self.bias = (torch.randn(E, generator=gen) * 0.1).cuda() if method in (2, 5) else None
        self.kw = dict(bias=self.bias, n_group=n_group, topk_group=topk_group, routed_scaling_factor=rsf)
        self.w13, self.W13 = held(moe, (E, 2 * I, H), weights, dtype, gen, g)
        self.w2, self.W2 = held(moe, (E, H, I), weights, dtype, gen, g)
        self.E, self.I, self.shared, self.gate = E, I, shared, gate
        if shared:
            self.kw["w13_s"], self.W13s = held(moe, (2 * shared, H), weights, dtype, gen, g)
            self.kw["w2_s"], self.W2s = held(moe, (H, shared), weights, dtype, gen, g)

    def __call__(self, x=None, **kw):
        return self.moe.moe_layer_few(self.x if x is None else x, self.wg, self.w13, self.w2, self.method, self.k,
                                      **self.kw, **kw)

    def weights_of(self, l, ids):
        """The routing weights of the experts `ids` from the logits."""
        chosen = np.take_along_axis(l, ids, 1)
        if self.method in (0, 1, 4):
            e = np.exp(chosen - l.max(1, keepdims=True))
            total = np.exp(l - l.max(1, keepdims=True)) if self.method == 0 else e
            return e / total.sum(1, keepdims=True)
        s = oracle.sigmoid64(chosen)
        if self.method == 3:
            return s
        rsf = self.kw["routed_scaling_factor"] if self.method in (2, 16) else 1.0
        return s / s.sum(1, keepdims=True) * rsf

    def check(self, got, x=None):
        y, ids, scales = got
        assert self.moe.moe_read_timeouts() == (self.moe.MOE_OK, 0)
        x = n64(self.x if x is None else x)
        T, H = x.shape
        wg = n64(self.wg)
        logits = x @ wg.T
        # a thread adds 8 products of every 2048, then 5 and 8 partial sums meet: the additions of one term
        err = (8 * -(-H // 2048) + 13) * 2.0 ** -24 * (np.abs(x) @ np.abs(wg).T)
        b = None if self.bias is None else self.bias.cpu().numpy()
        kw = dict(n_group=self.kw["n_group"], topk_group=self.kw["topk_group"], routed_scaling_factor=self.kw["routed_scaling_factor"])
        want_ids = oracle.route(logits[:, :self.E].astype(np.float32), self.method, self.k, bias=b, **kw)[0]
        l, got_ids = logits[:, :self.E], ids.cpu().numpy()
        # Another expert may stand where float64 has one only if their keys are no further apart than the
        # logits' errors (the sigmoid's slope is under 1) and the roundings of fp32 keys below 2.
        key = l if self.method in (0, 1, 3, 4, 6) else oracle.sigmoid64(l) + (0 if b is None else b)
        at = lambda i: np.take_along_axis(key, i, 1)   # noqa: E731
        apart = np.abs(at(got_ids) - at(want_ids))
        assert (apart[got_ids != want_ids] <= (2 * err.max(1, keepdims=True) + 2.0 ** -22 + 0 * apart)[got_ids != want_ids]).all()
        assert all(len(set(r)) == self.k for r in got_ids.tolist())
        want_ids = got_ids
        want_sc = self.weights_of(l, want_ids)
        # a weight's slope to the logits is at most the weight itself, over all of them 2
        sc_err = want_sc * (2 * err.max(1, keepdims=True) + 2.0 ** -22)
        assert (np.abs(n64(scales) - want_sc) <= sc_err).all()

        def expert(t, w13, w2, wt, wt_err, terms, tmax):
            half = w13.shape[0] // 2
            a, mag = w13 @ x[t], np.abs(w13) @ np.abs(x[t])
            da = (H * 2.0 ** -23 + 2.0 ** -20) * mag
            gt, up = a[:half], a[half:]
            with np.errstate(over="ignore"):
                silu = gt / (1 + np.exp(-gt))
            h = silu * up * wt
            dh = wt * (1.1 * np.abs(up) * da[:half] + np.abs(silu) * da[half:] + 1.1 * da[:half] * da[half:]) + np.abs(h) * 2.0 ** -20 + np.abs(silu * up) * wt_err
            u = U["bf16" if self.dtype == "bf16" and self.weights == "16" else "f16"]
            dh = dh + u * (np.abs(h) + dh) + 2.0 ** -38 * tmax
            return w2 @ h, np.abs(w2) @ dh + terms * 2.0 ** -23 * (np.abs(w2) @ np.abs(h)), np.abs(h).max()

        Y, bound = np.zeros((T, H)), np.zeros((T, H))
        terms = self.k * self.I + self.shared
        for t in range(T):
            parts = [(self.W13[e], self.W2[e], want_sc[t, j], sc_err[t, j]) for j, e in enumerate(want_ids[t])]
            if self.shared:
                s = 1 / (1 + np.exp(-logits[t, self.E])) if self.gate else 1.0
                parts.append((self.W13s, self.W2s, s, s * (err[t, self.E] + 2.0 ** -22) if self.gate else 0.0))
            tmax = max(expert(t, *p, terms, 0.0)[2] for p in parts)
            for p in parts:
                v, d, _ = expert(t, *p, terms, tmax)
                Y[t] += v
                bound[t] += d
        bound = bound + U[self.dtype] * (np.abs(Y) + bound) + TINY[self.dtype]
        d = np.abs(n64(y) - Y) - bound
        assert d.max() <= 0, f"{d.max():.3e} over the bound"


CASES = [  # T, H, I, E, k, method, shared, gate, n_group, topk_group, rsf
    (1, 32, 32, 1, 1, 1, 0, False, 1, 1, 1.0),
    (1, 1056, 544, 8, 2, 4, 0, False, 1, 1, 1.0),
    (2, 64, 2080, 6, 6, 6, 32, False, 1, 1, 1.0),
    (3, 544, 96, 130, 8, 0, 0, False, 1, 1, 1.0),
    (5, 1504, 736, 20, 4, 6, 352, True, 1, 1, 1.0),
    (8, 512, 1024, 16, 1, 3, 1056, True, 1, 1, 1.0),
    (9, 2080, 64, 32, 8, 2, 64, False, 8, 4, 2.5),
    (13, 96, 160, 60, 3, 5, 0, False, 1, 1, 1.0),
    (16, 256, 512, 64, 8, 16, 0, False, 8, 4, 1.5),
    (16, 1568, 288, 256, 8, 2, 1600, True, 8, 4, 2.5),
    (15, 160, 4128, 3, 2, 1, 0, False, 1, 1, 1.0),
    (7, 4608, 96, 12, 2, 0, 0, False, 1, 1, 1.0),
]


@pytest.mark.parametrize("weights,dtype", [("16", "bf16"), ("16", "f16"), ("mx", "bf16"), ("nv", "bf16"), ("nv", "f16")])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c[:6]))
def test_layer(moe, case, weights, dtype):
    T, H, I, E, k, method, shared, gate, n_group, topk_group, rsf = case
    layer = Layer(moe, T, H, I, E, k, method, weights, dtype, shared, gate, n_group, topk_group, rsf, seed=T + H, g=T % 2 == 1)
    got = layer()
    layer.check(got)
    again = layer()
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_memory_of_the_callers(moe):
    """Results and workspace given, whatever they hold; nothing of the workspace has to be set."""
    layer = Layer(moe, 6, 288, 160, 12, 3, 1, "nv", "bf16", shared=96)
    want = layer()
    scratch = moe.alloc_few_scratch(moe.make_problem(6, 288, 160, 12, 3, 96))
    for fill in (0xFF, 0x00, 0x7F):
        scratch.buf.fill_(fill)
        y = torch.full((6, 288), float("nan"), dtype=torch.bfloat16, device="cuda")
        ids = torch.full((6, 3), -7, dtype=torch.int32, device="cuda")
        sc = torch.full((6, 3), float("nan"), device="cuda")
        got = layer(y=y, ids=ids, scales=sc, scratch=scratch)
        assert got[0] is y and got[1] is ids and got[2] is sc
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    small = moe.Scratch(scratch.buf[:scratch.nbytes - 1])
    with pytest.raises(moe.MoeError, match="workspace"):
        layer(scratch=small)


def test_no_tokens(moe):
    layer = Layer(moe, 1, 64, 32, 4, 2, 1, "mx", "bf16")
    y, ids, sc = layer(x=layer.x[:0])
    assert y.shape == (0, 64) and ids.shape == (0, 2) and sc.shape == (0, 2)


@pytest.mark.parametrize("weights", ["16", "mx", "nv"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_token_that_is_not_finite_stays_alone(moe, weights, bad):
    layer = Layer(moe, 11, 544, 96, 10, 2, 4, weights, "bf16", shared=64)
    want = layer()
    x = layer.x.clone()
    x[4, 100] = bad
    got = layer(x=x)
    rest = [t for t in range(11) if t != 4]
    for a, b in zip(got, want):
        assert torch.equal(a[rest], b[rest])
    assert not torch.isfinite(got[0][4].float()).all()
    assert moe.moe_read_timeouts() == (moe.MOE_OK, 0)


def test_tokens_of_very_unequal_size(moe):
    """Powers of two of a token move its h and y by the same where the routing does not see them."""
    for weights, dtype in (("nv", "bf16"), ("mx", "bf16")):
        layer = Layer(moe, 4, 256, 128, 4, 4, 3, weights, dtype)
        for size in (2.0 ** -30, 2.0 ** 20):
            layer.x = (layer.x.double() * size).to(DT[dtype])
            layer.check(layer())
            layer.x = (layer.x.double() / size).to(DT[dtype])


def test_a_scale_of_nan_reaches_its_expert_only(moe):
    layer = Layer(moe, 9, 256, 96, 6, 1, 3, "nv", "bf16")
    want, ids, _ = layer()
    e = int(ids[0, 0])
    layer.w2.scales[e, 17, 2] = 127
    y = layer()[0]
    hit = (ids[:, 0] == e).cpu()
    bad = torch.isnan(y).cpu()
    assert bad[hit, 17].all() and bad.sum() == hit.sum()
    ok = ~bad
    assert torch.equal(y.cpu()[ok], want.cpu()[ok])


def test_captured_and_replayed_beside_an_eager_one(moe):
    layer = Layer(moe, 5, 544, 288, 24, 4, 6, "mx", "f16", shared=96, gate=True)
    other = Layer(moe, 3, 544, 288, 24, 4, 6, "16", "f16", seed=3)
    eager = layer()
    x = layer.x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x=x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(x=x)
    x.neg_()
    graph.replay()
    kept = other()
    layer.check(got, x=x)
    x.neg_()
    graph.replay()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, eager))
    assert all(torch.equal(a, b) for a, b in zip(kept, other()))


def test_calls_on_two_streams_at_once(moe):
    """Blocks of both kernels share the SMs; none waits for one that is not there."""
    layers = [Layer(moe, 16, 512, 1024, 32, 8, 1, "16", "bf16", seed=1), Layer(moe, 16, 512, 1024, 32, 8, 1, "nv", "bf16", seed=2)]
    want = [l() for l in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = [[], []]
    for _ in range(20):
        for i, l in enumerate(layers):
            with torch.cuda.stream(streams[i]):
                got[i].append(l())
    # (stream= with memory of that stream)
    extra = layers[0](stream=streams[1])
    torch.cuda.synchronize()
    assert moe.moe_read_timeouts() == (moe.MOE_OK, 0)
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
    assert all(torch.equal(a, b) for a, b in zip(extra, want[0]))


def test_agrees_with_the_layer_of_many_tokens(moe):
    """The same experts as moe_gate_route, and y as moe_forward's within both one's roundings."""
    layer = Layer(moe, 16, 512, 256, 32, 4, 4, "16", "bf16")
    y, ids, sc = layer()
    ids2, sc2, _, _ = moe.moe_gate_route(layer.x, layer.wg, 4, 4, 32)
    assert torch.equal(ids, ids2)
    y2 = moe.moe_forward(layer.x, ids2, sc2, layer.w13, layer.w2)
    layer.check((y, ids, sc))
    assert (y - y2).abs().max() <= 2e-2 * y2.abs().max()
