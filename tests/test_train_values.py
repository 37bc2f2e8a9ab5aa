"""GPU: the training operators at values where a formula in 32 bits over- or underflows or cancels,
against the definitions in float64. Bounds are elementwise, from the arithmetic, as in
test_train_ops.py."""
import numpy as np
import pytest
import torch

from oracle import train_oracle as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_03_gb300 as m
    return m


def n64(t):
    return t.detach().cpu().double().numpy()


def within(got, want, bound, what):
    got = n64(got)
    assert np.isfinite(got).all(), f"{what}: not finite"
    worst = (np.abs(got - want) - bound).max()
    assert worst <= 0, f"{what}: {worst:.3e} over the bound"


# Chosen logits all far below zero: the sum of their sigmoids is tiny, the weights are ordinary.
# Steps of 1/1024, so that differences of logits are exact in 32 bits.
FAR = [[-90.0, -90.5, -91.25], [-95.0, -95.5, -100.0], [-100.0, -100.0, -100.0], [-110.0, -109.5, -103.25],
       [-300.0, -301.0, -300.5], [-60.0, -61.5, -90.0], [-30.0, -29.5, -31.0], [-20.5, -20.25, -33.0],
       [-19.5, -20.25, -40.0], [-20.0, -21.0, -20.0], [-15.0, -87.5, -88.5], [-104.0, float("-inf"), -103.0]]


@pytest.mark.parametrize("k", [1, 2, 3])
@pytest.mark.parametrize("method", [2, 5, 6, 16])
def test_route_backward_of_chosen_logits_far_below_zero(moe, method, k):
    rng = np.random.default_rng(method + k)
    T, E = len(FAR), 9
    logits = np.full((T, E), -500.0, np.float32)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    for t, row in enumerate(FAR):
        logits[t, ids[t]] = row[:k]
    ids[2, 0] = -1                           # of k = 1: no slot left
    ds = (rng.integers(-64, 65, (T, k)) / 32).astype(np.float32)
    rsf = 2.5 if method in (2, 16) else 1.0
    got = moe.moe_route_backward(torch.from_numpy(logits).cuda(), torch.from_numpy(ids).cuda(),
                                 torch.from_numpy(ds).cuda(), method, rsf)
    want, mag = ref.route_backward(logits, ids, ds.astype(np.float64), method, rsf)
    # expf within 2 ulp; k sums, two quotients and a few products
    within(got, want, 40 * 2.0 ** -24 * mag + 1e-37, "dlogits")


@pytest.mark.parametrize("method", [2, 5, 6, 16])
def test_route_backward_where_the_sigmoids_underflow_in_64_bits_squared(moe, method):
    """sigma(l) = e^l there: with nothing added to the sum the weights are a softmax, and with the 1e-20
    of it the gradient is nothing."""
    logits = np.array([[-700.0, -701.0, -699.5, 0.0]], np.float32)
    ids = np.array([[0, 1, 2]], np.int32)
    ds = np.array([[1.0, -0.5, 0.25]], np.float32)
    rsf = 2.5 if method in (2, 16) else 1.0
    got = moe.moe_route_backward(torch.from_numpy(logits).cuda(), torch.from_numpy(ids).cuda(),
                                 torch.from_numpy(ds).cuda(), method, rsf)
    want, mag = ref.route_backward(logits, ids, ds.astype(np.float64), 1)
    want, mag = (rsf * want, rsf * mag) if method != 2 else (0 * want, 0 * mag)
    within(got, want, 40 * 2.0 ** -24 * mag + 1e-37, "dlogits")


@pytest.mark.parametrize("I", [96, 33, 515])
def test_swiglu_in_f32_is_as_accurate_as_f32(moe, I):
    """At gates of up to 100 either way, in units of 2^-24: expf 4 (2 ulp), 1 + exp(-|g|) and its
    reciprocal 4 in all, sigma or 1 - sigma, their product, 9; two products more. Below the normal
    range a few of its steps, times the other factors."""
    R = 40
    g = torch.Generator().manual_seed(I)
    gu = torch.randn((R, 2 * I), generator=g)
    gu[:, :I] *= 10.0 ** torch.empty((R, 1)).uniform_(-2, 1.5, generator=g)
    gu[0, :I] = torch.linspace(-100, 100, I)
    gu[1, :I] = torch.linspace(-104, -80, I)
    gu[2, :I] = torch.linspace(10, 20, I)
    gu = gu.clamp(-104, 104).cuda()
    dh = torch.randn((R, I), generator=g).cuda()
    h, ckpt = moe.moe_swiglu_ckpt(gu)
    dgu, again = moe.moe_swiglu_ckpt_backward(dh, ckpt, want_h=True)
    unit = 2.0 ** -24

    def parts(v):
        gate, up = v[:, :I], v[:, I:]
        return gate, up, 2.0 ** -146 * (1 + np.abs(gate)) * (1 + np.abs(up))

    for got, v in ((h, n64(gu)), (again, ref.kept(*(t.cpu().numpy() for t in ckpt)))):
        want = ref.swiglu(v)
        within(got, want, 12 * unit * np.abs(want) + parts(v)[2], "h")
    gate, up, tiny = parts(v)
    d = n64(dh)
    want = ref.swiglu_backward(d, v)
    s, o = ref.sigmoid(gate), ref.sigmoid(-gate)
    # sigma + (g sigma) (1 - sigma): 9, and 13 and two products, the sum, two products more
    mag = np.concatenate([20 * np.abs(d * up) * (s + np.abs(gate) * s * o), 12 * np.abs(want[:, I:])], 1)
    tiny = tiny * (1 + np.abs(d))
    within(dgu, want, unit * mag + np.concatenate([tiny, tiny], 1), "dgu")
