"""Workspaces that the binding makes: each call has its own and holds it.

An entry point may launch several kernels that hand their results on through
the workspace.  ctypes releases the interpreter's lock during the call, so
another thread's call on the same stream may launch in between, and a captured
call's workspace is used whenever its graph is replayed.
"""
import sys
import threading
import types
import weakref

import pytest
import torch

import dora_adapter_factored_amd as D
from dora_adapter_factored_amd import binding as Bn
from dora_adapter_factored_amd import eightbit as E8


def bf16(*shape):
    return torch.ones(*shape, dtype=torch.bfloat16)


def f32(*shape):
    return torch.ones(*shape)


def codes(*shape):
    return torch.ones(*shape, dtype=torch.int8)


def norm(n):
    return D.factored_norm(bf16(n, 512), bf16(64, 512), bf16(n, 64), 1.0)


def product(T):
    return D.matmul_q8(codes(T, 5120), f32(T), codes(5120, 5120), f32(5120))


# entry point, a call of size n, n, a larger n
CALLS = [
    ("dora_matmul_q8", product, 24, 40),
    ("dora_rmsnorm_backward", lambda T: D.rmsnorm_backward(bf16(T, 4096), bf16(T, 4096), bf16(4096), f32(T)), 100, 300),
    ("dora_compose_backward", lambda T: D.compose_backward(bf16(T, 4096), bf16(T, 4096), bf16(T, 4096), f32(4096), f32(4096),
                                                           1.0), 100, 3000),
    ("dora_compose_backward_inner", lambda T: D.compose_backward_inner(bf16(T, 4096), bf16(T, 4096), f32(4096), f32(4096),
                                                                       1.0), 100, 3000),
    ("dora_factored_norm", norm, 256, 8192),
    ("dora_factored_norm_group", lambda n: D.factored_norm_group([(bf16(n, 512), bf16(64, 512), bf16(n, 64), 1.0, None)] * 2),
     256, 8192),
    ("dora_merge", lambda n: D.merge(bf16(64, n), bf16(64, n), bf16(64, 64), f32(64), 1.0), 4096, 1 << 15),
]


@pytest.mark.parametrize("name,call,small,large", CALLS, ids=[c[0] for c in CALLS])
def test_calls_in_flight_have_workspaces_of_their_own(monkeypatch, name, call, small, large):
    # the second and third calls are made from inside the first, as another
    # thread's would be between the first one's launches
    real = Bn.load()
    made, seen = [], []

    def workspace(nbytes, device, orig=Bn.workspace):
        ws = orig(nbytes, device)
        made.append(weakref.ref(ws))
        return ws

    class Stub:
        def __getattr__(self, attr):
            if attr != name:
                return getattr(real, attr)

            def launch(*args):
                ptr = getattr(args[-3], "value", args[-3])
                seen.append((ptr, ptr + args[-2]))
                if len(seen) == 1:
                    first = made[0]
                    call(small)
                    call(large)
                    assert first() is not None, "the first call's workspace is gone while it is in flight"
                return 0
            return launch

    for mod in (Bn, E8):
        monkeypatch.setattr(mod, "load", lambda: Stub())
        monkeypatch.setattr(mod, "workspace", workspace)
        monkeypatch.setattr(mod, "_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=0))
    call(small)
    assert len(seen) == 3 and len(made) == 3
    for lo, hi in seen[1:]:
        assert hi <= seen[0][0] or seen[0][1] <= lo, "two calls in flight share a workspace"


WITH_WS = [
    ("dora_matmul_q8", lambda ws: D.matmul_q8(codes(24, 5120), f32(24), codes(5120, 5120), f32(5120), ws=ws)),
    ("dora_matmul_q8", lambda ws: D.linear_q8(bf16(24, 5120), codes(5120, 5120), f32(5120), ws=ws)),
    ("dora_matmul_q8", lambda ws: D.linear_q8_backward(bf16(24, 5120), codes(5120, 5120), f32(5120), ws=ws)),
    ("dora_rmsnorm_backward", lambda ws: D.rmsnorm_backward(bf16(9, 64), bf16(9, 64), bf16(64), f32(9), ws=ws)),
    ("dora_compose_backward", lambda ws: D.compose_backward(bf16(9, 64), bf16(9, 64), bf16(9, 64), f32(64), f32(64), 1.0, ws=ws)),
    ("dora_compose_backward_inner", lambda ws: D.compose_backward_inner(bf16(9, 64), bf16(9, 64), f32(64), f32(64), 1.0, ws=ws)),
    ("dora_factored_norm", lambda ws: D.factored_norm(bf16(64, 512), bf16(64, 512), bf16(64, 64), 1.0, ws=ws)),
    ("dora_factored_norm_group", lambda ws: D.factored_norm_group([(bf16(64, 512), bf16(64, 512), bf16(64, 64), 1.0, None)], ws=ws)),
    ("dora_merge", lambda ws: D.merge(bf16(64, 512), bf16(64, 512), bf16(64, 64), f32(64), 1.0, ws=ws)),
]


@pytest.mark.parametrize("name,call", WITH_WS, ids=[str(i) + c[0] for i, c in enumerate(WITH_WS)])
def test_a_workspace_that_the_kernels_cannot_use_is_refused(monkeypatch, name, call):
    # on another device than the operands, scattered or repeated in memory, or
    # no tensor at all: before the call
    real, reached = Bn.load(), []

    class Stub:
        def __getattr__(self, attr):
            if attr.endswith("workspace_size"):
                return getattr(real, attr)
            return lambda *args: reached.append((attr, args[-2])) or 0

    for mod in (Bn, E8):
        monkeypatch.setattr(mod, "load", lambda: Stub())
        monkeypatch.setattr(mod, "_stream", lambda device: 0)
    n = 1 << 23
    for bad in (torch.empty(n, dtype=torch.uint8, device="meta"), torch.empty(1, dtype=torch.uint8).expand(n),
                torch.empty(2 * n, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="ws"):
            call(bad)
    with pytest.raises(TypeError, match="ws"):
        call(1 << 20)
    assert not [a for a, _ in reached if a == name]
    call(torch.empty(n // 4))   # any element type
    assert (name, n) in reached


# ------------------------------------------------------------------ on the GPU
DEV = torch.device("cuda:0")


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def operands(T, N, K, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    xq = torch.randint(-127, 128, (T, K), generator=g, device=DEV, dtype=torch.int8)
    wq = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    return xq, torch.rand(T, generator=g, device=DEV), wq, torch.rand(N, generator=g, device=DEV)


@pytest.mark.gpu
def test_threads_on_one_stream():
    """Calls of several launches from four threads on the default stream, each
    thread's results bitwise those of the same calls made alone."""
    say("[workspaces] threads")
    jobs = []
    for k, (T, N, K) in enumerate(((24, 5120, 5120), (48, 5120, 8192), (2000, 1299, 4099), (70, 3273, 5676))):
        a = operands(T, N, K, k)
        assert D.matmul_q8_workspace_size(T, N, K) > 0
        g = torch.Generator(device=DEV).manual_seed(100 + k)
        dy, h = (torch.randn(100 + 90 * k, 2048, generator=g, device=DEV) for _ in range(2))
        w, rstd = torch.rand(2048, generator=g, device=DEV), torch.rand(100 + 90 * k, generator=g, device=DEV)
        jobs.append(lambda a=a, b=(dy, h, w, rstd): (D.matmul_q8(*a), *D.rmsnorm_backward(*b)))
    want = [j() for j in jobs]
    torch.cuda.synchronize()
    got = [[] for _ in jobs]
    start = threading.Barrier(len(jobs))

    def work(k):
        start.wait(timeout=60)
        for _ in range(20):
            got[k].append(jobs[k]())

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for k, w in enumerate(want):
        assert len(got[k]) == 20
        for i, r in enumerate(got[k]):
            assert all(torch.equal(a, b) for a, b in zip(r, w)), (k, i)


@pytest.mark.gpu
def test_a_captured_call_keeps_its_workspace():
    """Replays after larger calls on the stream that was captured: the results
    hold, and so does whatever was allocated since."""
    say("[workspaces] capture, then larger calls")
    small, large = operands(24, 5120, 5120, 1), operands(333, 5120, 27648, 2)
    assert 0 < D.matmul_q8_workspace_size(24, 5120, 5120) < D.matmul_q8_workspace_size(333, 5120, 27648)
    want, want_large = D.matmul_q8(*small), D.matmul_q8(*large)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        D.matmul_q8(*small)
    side.synchronize()
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        D.matmul_q8(*small, out=out)
    with torch.cuda.stream(side):
        got = D.matmul_q8(*large)
        live = [torch.full((1 << 20,), 7, dtype=torch.int32, device=DEV) for _ in range(8)]
    side.synchronize()
    assert torch.equal(got, want_large)
    for k in range(3):
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), k
        assert all(bool((t == 7).all()) for t in live), k
        assert torch.equal(D.matmul_q8(*large), want_large), k


@pytest.mark.gpu
def test_two_captures_replayed_side_by_side():
    say("[workspaces] two captures on one stream, replayed on two")
    calls = [operands(24, 5120, 5120, 3), operands(48, 5120, 8192, 4)]
    want = [D.matmul_q8(*c) for c in calls]
    outs = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in calls]
    for graph, c, out in zip(graphs, calls, outs):
        with torch.cuda.graph(graph):
            D.matmul_q8(*c, out=out)
    streams = [torch.cuda.Stream() for _ in calls]
    for k in range(4):
        for out in outs:
            out.zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), k
