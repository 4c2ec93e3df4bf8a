"""The allocating helpers on a stream that the caller names: memory that the current stream's queued work still uses is not
written by the named stream, and the named stream's results outlive what the current stream does next."""
import numpy as np
import pytest

import bit_mixed_precision_tri_amd as tri
from bit_mixed_precision_tri_amd import synth
from tests.gpu_helpers import say, cuda

pytestmark = pytest.mark.gpu
F2 = tri.TRI_FMT_2BIT


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tri.lib()
    yield
    torch.cuda.synchronize()


def calls():
    """name -> call(stream) that returns the tensors it made, and the sizes of what it makes besides."""
    import torch
    rng = np.random.default_rng(81)
    T, E, topk, K, N, group = 300, 8, 2, 256, 384, 64
    X = cuda(rng.standard_normal((T, K)).astype(np.float16))
    logits = cuda(rng.standard_normal((T, E)).astype(np.float32))
    Q, S = cuda(rng.integers(0, 16, (N, K), dtype=np.uint8)), cuda(rng.uniform(0.01, 0.02, (N, K // group)).astype(np.float16))
    Z = cuda(rng.integers(0, 16, (N, K // group), dtype=np.uint8))
    W = cuda((0.05 * rng.standard_normal((N, K))).astype(np.float32))
    Wp = tri.int4_pack(Q, S, group, Z)
    stack = lambda n, k: (tri.pack(cuda(synth.trits(rng, E * n, k)), F2).view(E, n, -1), torch.full((E,), 0.03, device="cuda"))
    gate, up, down = stack(N, K), stack(N, K), stack(K, N)
    r = tri.experts_route(logits, topk)
    H = tri.experts_pair(X, r.offsets, r.rows, *gate, *up, K, F2)
    Y = tri.experts_linear(H, r.offsets, None, *down, N, F2)
    ws = tri.tri_experts_route_workspace_bytes(T, E, topk)
    trits = cuda(synth.trits(rng, N, K))
    packed = tri.pack(trits, F2)
    return {
        "pack": (lambda s: [tri.pack(trits, F2, stream=s)], []),
        "unpack": (lambda s: [tri.unpack(packed, K, F2, stream=s)], []),
        "quantize": (lambda s: list(tri.quantize(W, F2, stream=s)), [tri.tri_quantize_workspace_bytes(N, K)]),
        "linear": (lambda s: [tri.linear(X, packed, 0.03, K, F2, stream=s)], []),
        "int4_pack": (lambda s: [tri.int4_pack(Q, S, group, Z, stream=s)], []),
        "int4_unpack": (lambda s: list(tri.int4_unpack(Wp, N, K, group, True, stream=s)), []),
        "int4_quantize": (lambda s: [tri.int4_quantize(W, group, True, stream=s)], []),
        "int4_linear": (lambda s: [tri.int4_linear(X, Wp, N, group, True, stream=s)], []),
        "experts_route": (lambda s: list(tri.experts_route(logits, topk, stream=s)), [ws]),
        "experts_linear": (lambda s: [tri.experts_linear(H, r.offsets, None, *down, N, F2, stream=s)], []),
        "experts_pair": (lambda s: [tri.experts_pair(X, r.offsets, r.rows, *gate, *up, K, F2, stream=s)], []),
        "experts_combine": (lambda s: [tri.experts_combine(Y, r.pos, r.weights, stream=s)], []),
        "experts_mlp": (lambda s: [tri.experts_mlp(X, logits, topk, gate, up, down, F2, stream=s)],
                        [ws, 4 * T * topk, 4 * (E + 1), H.numel() * 2, Y.numel() * 2]),
    }


NAMES = ["pack", "unpack", "quantize", "linear", "int4_pack", "int4_unpack", "int4_quantize", "int4_linear", "experts_route",
         "experts_linear", "experts_pair", "experts_combine", "experts_mlp"]


@pytest.mark.parametrize("kind", ["stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_writes(name, kind):
    """Tensors of the sizes that a helper needs are written on the current stream, behind some milliseconds of other work,
    and let go; the helper runs on another stream at once.  Its results hold nothing of those writes."""
    import torch
    call, more = calls()[name]
    want = [t.clone() for t in call(None)]
    sizes = [t.numel() * t.element_size() for t in want] + more
    big = torch.zeros(1 << 28, dtype=torch.float32, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    say("stream", name, kind)
    for _ in range(2):
        for _ in range(12):
            big.add_(1.0)                        # 2 GiB of traffic each
        old = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
        for t in old:
            t.fill_(0xFF)
        del old, t
        got = call(s if kind == "stream" else s.cuda_stream)
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), "output %d" % i
        del got, a


@pytest.mark.parametrize("name", NAMES)
def test_results_that_the_current_stream_still_reads(name):
    """A result that the current stream has yet to read, behind some milliseconds of other work, is let go: the helper's next
    call on the same named stream does not write into it."""
    import torch
    call, _ = calls()[name]
    want = [t.clone() for t in call(None)]
    big = torch.zeros(1 << 28, dtype=torch.float32, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    say("stream", name)
    got = call(s)
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(12):
        big.add_(1.0)
    copies = [t.clone() for t in got]
    sizes = [t.numel() * t.element_size() for t in got]
    del got
    with torch.cuda.stream(s):
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
    call(s)
    torch.cuda.synchronize()
    for a, b in zip(copies, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("handle", [False, True])
def test_the_default_stream_named_from_another(handle):
    """Stream 0, by its object and by its handle, while a side stream is the current one."""
    import torch
    zero = 0 if handle else torch.cuda.default_stream()
    for name, (call, _) in calls().items():
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.Stream()):
            got = call(zero)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), name


def test_a_named_stream_inside_a_capture():
    """A helper on a stream that was forked from the one being captured, its results and intermediate tensors made inside the
    capture, replayed on new inputs with eager calls between the replays."""
    import torch
    rng = np.random.default_rng(82)
    T, E, topk, K, N = 200, 8, 2, 256, 384
    mk = lambda *shape: torch.zeros(shape, dtype=torch.float16, device="cuda")
    X, logits = mk(T, K), mk(T, E)
    stack = lambda n, k: (tri.pack(cuda(synth.trits(rng, E * n, k)), F2).view(E, n, -1), torch.full((E,), 0.03, device="cuda"))
    mats = stack(N, K), stack(N, K), stack(K, N)

    def step(stream):
        return tri.experts_mlp(X, logits, topk, *mats, F2, residual=X, stream=stream)

    step(None)
    side, other, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            other.wait_stream(side)
            Y = step(other)
            side.wait_stream(other)
    torch.cuda.synchronize()
    for seed in (1, 2, 3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        X.copy_(torch.randn(X.shape, device="cuda", generator=g).half())
        logits.copy_(torch.randn(logits.shape, device="cuda", generator=g).half())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = Y.clone()
        assert torch.equal(got, step(None)) and torch.equal(got, step(other)), seed
        torch.cuda.synchronize()
    del graph
