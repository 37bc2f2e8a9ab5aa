"""Calls with stream=: what the binding allocates for a call belongs to the stream of its launch.

The caching allocator hands a freed block out again in the order of the stream it was allocated on.
A workspace of another stream's is free again as soon as the call returns, while its kernels still
run: the next call may get the same block, and the first one's tensor maps, sums or counts are
overwritten under it. And a block may still be in use, on the stream it was allocated on, by work
that the launch does not wait for. Both are checked on the CPU, with the library's calls and the
allocator stood in for, and once on a GPU with two streams' calls under way at once.
"""
import os
import shutil
from types import SimpleNamespace

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CALLER, SIDE = 64, 128          # stream handles


@pytest.fixture(scope="module")
def moe():
    if not os.path.exists(os.path.join(ROOT, "mixture_experts_layer_03_gb300", "libmoe_gb300.so")):
        if not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
            pytest.skip("library not built and nvcc unavailable")
        import __graft_entry__
        __graft_entry__.build()
    import mixture_experts_layer_03_gb300 as m
    return m


class OnGpu(torch.Tensor):
    """A CPU tensor that passes for a CUDA one and notes its streams."""
    is_cuda = True
    made_on = used_on = None

    def record_stream(self, stream):
        self.used_on = stream.cuda_stream


@pytest.fixture
def allocations(moe, monkeypatch):
    """Every tensor that torch.empty makes, with the stream it was made on; the library's calls only
    note the stream of their launch."""
    made, launched, current, real_empty = [], [], [CALLER], torch.empty

    def empty(shape, dtype=None, device=None):
        t = real_empty(shape, dtype=dtype).as_subclass(OnGpu)
        t.made_on = current[0]
        made.append(t)
        return t

    class Use:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream.cuda_stream)
            current[0] = self.stream.cuda_stream

        def __exit__(self, *_):
            current.pop()
            current[0] = current[-1] if len(current) > 1 else CALLER

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_bytes"):
                return lambda *a: 4096
            if name == "moe_workspace_layout":
                return lambda *a: 0
            def call(*a):
                launched.append(a[-1])
                return 0
            return call

    monkeypatch.setattr(moe, "_lib", Lib())
    monkeypatch.setattr(moe, "_raw_stream", lambda device: current[0])
    monkeypatch.setattr(moe, "_current_device", lambda: 0)
    monkeypatch.setattr(moe.torch, "empty", empty)
    monkeypatch.setattr(moe.torch, "empty_like", lambda t: empty(t.shape, t.dtype))
    cuda = moe.torch.cuda
    monkeypatch.setattr(cuda, "stream", Use)
    monkeypatch.setattr(cuda, "ExternalStream", lambda handle, device=None: SimpleNamespace(cuda_stream=int(handle)))
    monkeypatch.setattr(cuda, "current_stream", lambda device=None: SimpleNamespace(cuda_stream=current[0]))
    monkeypatch.setattr(cuda, "default_stream", lambda device=None: SimpleNamespace(cuda_stream=0))
    return SimpleNamespace(made=made, launched=launched)


def gpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


def i32(*shape):
    return gpu(*shape, dtype=torch.int32)


TRAINING = {
    "dispatch": lambda m, s: m.moe_dispatch(gpu(4, 64), i32(4, 2), 8, stream=s),
    "dispatch, three launches": lambda m, s: m.moe_dispatch(gpu(7000, 8), i32(7000, 2), 8, stream=s),
    "dispatch_rows": lambda m, s: m.moe_dispatch_rows(gpu(4, 64), i32(4, 2), stream=s),
    "dispatch_backward": lambda m, s: m.moe_dispatch_backward(gpu(8, 64), i32(4, 2), stream=s),
    "combine": lambda m, s: m.moe_combine(gpu(8, 64), i32(4, 2), stream=s),
    "combine_backward": lambda m, s: m.moe_combine_backward(gpu(4, 64), gpu(8, 64), i32(4, 2), stream=s),
    "swiglu_ckpt": lambda m, s: m.moe_swiglu_ckpt(gpu(4, 64), stream=s),
    "swiglu_ckpt_backward": lambda m, s: m.moe_swiglu_ckpt_backward(
        gpu(4, 32), (gpu(4, 64, dtype=torch.uint8), gpu(4, 2, dtype=torch.uint8)), want_h=True, stream=s),
    "experts_matmul": lambda m, s: m.moe_experts_matmul(gpu(4, 64), gpu(2, 32, 64), i32(3), stream=s),
    "experts_matmul_dx": lambda m, s: m.moe_experts_matmul_dx(gpu(4, 32), gpu(2, 32, 64), i32(3), stream=s),
    "experts_matmul_dw": lambda m, s: m.moe_experts_matmul_dw(gpu(4, 32), gpu(4, 64), i32(3), stream=s),
    "route_backward": lambda m, s: m.moe_route_backward(
        gpu(4, 8, dtype=torch.float32), i32(4, 2), gpu(4, 2, dtype=torch.float32), 0, stream=s),
}


def weights():
    return gpu(2, 128, 64), gpu(2, 64, 64)


FORWARD = {
    "route": lambda m, s: m.moe_route(gpu(4, 8, dtype=torch.float32), 0, 2, stream=s),
    "gate": lambda m, s: m.moe_gate(gpu(4, 64), gpu(9, 64), 8, stream=s),
    "gate_route": lambda m, s: m.moe_gate_route(gpu(4, 64), gpu(9, 64), 4, 2, 8, want_logits=True, stream=s),
    "forward": lambda m, s: m.moe_forward(gpu(4, 64), i32(4, 2), gpu(4, 2, dtype=torch.float32),
                                          *weights(), stream=s),
    "forward_partial": lambda m, s: m.moe_forward_partial(
        gpu(4, 64), i32(4, 2), gpu(4, 2, dtype=torch.float32), *weights(), 0, 2, 4, stream=s),
    "forward_static": lambda m, s: m.moe_forward_static(gpu(4, 64), i32(4, 2), gpu(4, 2, dtype=torch.float32),
                                                        *weights(), stream=s),
    "cast": lambda m, s: m.moe_cast_f32_to_bf16(gpu(4, dtype=torch.float32), stream=s),
}


def tensors(out):
    for t in out if isinstance(out, tuple) else (out,):
        if hasattr(t, "buf"):
            yield t.buf
        elif t is not None:
            yield t


def check(moe, allocations, call):
    for stream in (SIDE, SimpleNamespace(cuda_stream=SIDE)):
        allocations.made.clear()
        allocations.launched.clear()
        results = list(tensors(call(moe, stream)))
        assert allocations.launched == [SIDE]
        assert allocations.made and all(t.made_on == SIDE for t in allocations.made), \
            "allocated on another stream than the launch's"
        # The caller goes on with the results on its own stream.
        assert results and all(t.used_on == CALLER for t in results)
    for stream in (None, CALLER):
        allocations.made.clear()
        call(moe, stream)
        assert all(t.made_on == CALLER and t.used_on is None for t in allocations.made)


@pytest.mark.parametrize("name", TRAINING)
def test_a_training_calls_allocations_are_the_launchs_streams(moe, allocations, name):
    check(moe, allocations, TRAINING[name])


@pytest.mark.parametrize("name", FORWARD)
def test_a_forward_calls_allocations_are_the_launchs_streams(moe, allocations, name):
    check(moe, allocations, FORWARD[name])


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
def test_two_streams_forwards_under_way_at_once(moe):
    T, H, I, E, k = 300, 256, 192, 8, 2
    g = torch.Generator().manual_seed(2)
    draw = lambda *shape, std=1.0: (torch.randn(shape, generator=g) * std).bfloat16().cuda()   # noqa: E731
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32).cuda()
    scales = torch.rand((T, k), generator=g).cuda()
    xs, w13, w2 = [draw(T, H), draw(T, H)], draw(E, 2 * I, H, std=H ** -0.5), draw(E, H, I, std=I ** -0.5)
    want = [moe.moe_forward(x, ids, scales, w13, w2) for x in xs]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
    got = [moe.moe_forward(x, ids, scales, w13, w2, stream=s) for x, s in zip(xs, side)]
    scribble = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in (4096, 1 << 16, 1 << 20, 1 << 22)]
    torch.cuda.synchronize()
    del scribble
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
def test_two_streams_calls_under_way_at_once(moe, monkeypatch):
    """No workspace of one pending call overlaps another's, and the results are those of calls one
    after the other; so too when memory of the caller's stream is used again meanwhile."""
    T, k, H, E, N, R = 7000, 2, 64, 8, 136, 1500
    g = torch.Generator().manual_seed(1)
    ids = torch.randint(-1, E, (T, k), generator=g, dtype=torch.int32).cuda()
    off = torch.linspace(0, R, E + 1).int().cuda()
    few = torch.tensor([0, 100], dtype=torch.int32).cuda()
    draw = lambda *shape: torch.randn(shape, generator=g).bfloat16().cuda()   # noqa: E731
    long_w = draw(1, N, 6200)
    inputs = [(draw(T, H), draw(100, 6200), draw(R, N), draw(R, H)) for _ in range(2)]

    def calls(i, stream):
        x, long_x, dy, rows = inputs[i]
        return (*moe.moe_dispatch(x, ids, E, stream=stream),
                moe.moe_experts_matmul(long_x, long_w, few, stream=stream),
                moe.moe_experts_matmul_dw(dy, rows, off, stream=stream))

    want = [calls(i, None) for i in range(2)]
    torch.cuda.synchronize()
    spaces = []

    def spy(name, at):
        real = getattr(moe._lib, name)

        def call(*a):
            if a[at]:
                spaces.append((a[at], a[at] + a[at + 1], a[-1]))
            return real(*a)
        monkeypatch.setattr(moe._lib, name, call)

    for name, at in (("moe_dispatch", 10), ("moe_experts_matmul", 9), ("moe_experts_matmul_dw", 11)):
        spy(name, at)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)       # about 10 ms: every call below is pending at once
    got = [calls(i, s if i else s.cuda_stream) for i, s in enumerate(side)]
    scribble = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in (4096, 1 << 16, 1 << 20, 1 << 22)]
    torch.cuda.synchronize()
    assert len(spaces) >= 4 and {s for *_, s in spaces} == {s.cuda_stream for s in side}
    for a in spaces:
        for b in spaces:
            assert a[2] == b[2] or a[1] <= b[0] or b[1] <= a[0], "two pending calls share a workspace"
    del scribble
    for w, r in zip(want, got):
        for a, b in zip(w, r):
            assert torch.equal(a, b)
