"""The convolution, the memory, the feed-forward block and AdamW together, as the example uses them; device waits that run
out; host threads that call at once."""
import importlib.util
import os
import threading
import time

import pytest
import torch

import test_neural_memory_gb300 as ttm

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ttm.build()
    yield
    assert ttm.device_status() == ttm.OK


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_gated_block.py")
    spec = importlib.util.spec_from_file_location("train_gated_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_the_example_runs_and_decodes(example):
    losses, off = example.main(12)
    assert all(v == v for v in losses)
    # bf16 on either way through the same block: the scan's parity bound
    assert off < 2e-2


def test_the_example_s_gradients(example):
    """Along each parameter's own gradient, where the loss changes most, against differences of the loss in fp32 weights.
    The pass rounds to bf16 (2^-8 of a value at most, evenly) a dozen times: 2^-4 of the change is the bound, and the step
    makes the change 2^-5 of the loss, whose own rounding noise, 1024 rows averaged, is far below that share of it."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    keys, values = (torch.randn((64, example.D), generator=gen, device="cuda") for _ in range(2))
    p = example.parameters(gen)
    x, target, ask, doc = example.batch(gen, keys, values)

    def loss_of(q):
        y, _ = example.block(q, x, doc)
        return torch.nn.functional.mse_loss(y[:, ask].float(), target[:, ask])
    used = example.leaves(p)
    loss = loss_of(used)
    grads = dict(zip(used, torch.autograd.grad(loss, list(used.values()))))
    for name in ("W_qkv", "W_o", "W_in", "W_down", "taps", "w1", "w2", "w3"):
        g = grads[name].float()
        step = float(loss.detach()) * 2.0 ** -5 / float(g.square().sum())
        ends = []
        for sign in (1, -1):
            q = dict(used)
            moved = used[name].detach().float() + sign * step * g
            q[name] = moved.to(used[name].dtype)
            with torch.no_grad():
                ends.append((float(loss_of(q)), float(((q[name].float() - used[name].float()) * g).sum())))
        (hi, up), (lo, down) = ends
        assert abs((hi - lo) / (up - down) - 1) < 2.0 ** -4, (name, (hi - lo) / (up - down))


def stalls(call, at):
    """The clean result of the call, then one with its wait `at` running out, then a clean one again."""
    want = [t.clone() for t in call()]
    assert ttm.device_status() == ttm.OK
    ttm.debug_set("wait_cycles", 20_000_000)          # ~10 ms at 2 GHz
    ttm.debug_set("stall_chunk", at)
    try:
        t0 = time.perf_counter()
        call()
        status = ttm.device_status()                  # synchronises
        assert status == ttm.ERR_TIMEOUT, ttm.status_str(status)
        assert time.perf_counter() - t0 < 10.0
        assert ttm.device_status() == ttm.OK          # the query cleared it
    finally:
        ttm.debug_set("stall_chunk", -1)
        ttm.debug_set("wait_cycles", 0)
    got = call()
    assert ttm.device_status() == ttm.OK
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("N,D,F,at", [(3, 256, 512, 0), (100, 512, 640, 1), (128, 64, 72, 0),      # few rows
                                      (200, 512, 1024, 0), (300, 2048, 256, 2),                     # a tile's K shared
                                      (3000, 512, 2048, 4), (9000, 256, 1024, 1)])                  # whole rounds
def test_a_wait_of_the_feed_forward_runs_out(N, D, F, at):
    r = torch.Generator(device="cuda").manual_seed(N)
    rand = lambda *s: torch.randn(s, generator=r, device="cuda").to(BF)  # noqa: E731
    x, dy, W_in, W_out = rand(N, D), rand(N, D), rand(D, 2 * F) / D ** 0.5, rand(F, D) / F ** 0.5
    gu = ttm.gated_ffn_fwd(x, W_in, W_out)[1]
    stalls(lambda: ttm.gated_ffn_fwd(x, W_in, W_out), at)
    stalls(lambda: tuple(ttm.gated_ffn_bwd(dy, x, gu, W_in, W_out).values()), at)


def at_once(*calls, times=1500):
    """Return codes other than OK of calls that run in a thread each (ctypes lets go of the interpreter)."""
    start, bad = threading.Barrier(len(calls)), []

    def loop(call):
        start.wait()
        bad.extend(r for r in (call() for _ in range(times)) if r != ttm.OK)
    threads = [threading.Thread(target=loop, args=(c,)) for c in calls]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    return bad


def test_feed_forward_blocks_of_two_threads():
    """Few rows and many, each thread on its own stream with its own workspace: no call fails, and the bits are those of
    calls one by one."""
    L = ttm.lib()

    def call(N, D=256, F=512):
        s = torch.cuda.Stream()
        x, W_in, W_out = (torch.randn(n, device="cuda").to(BF) for n in ((N, D), (D, 2 * F), (F, D)))
        want = ttm.gated_ffn_fwd(x, W_in, W_out)[0]
        y, n = torch.empty_like(x), L.ttm_gated_ffn_workspace_size(N, D, F, 0)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        keep = (s, x, W_in, W_out, y, ws, want)
        p = [t.data_ptr() for t in keep[1:6]]
        return keep, lambda: L.ttm_gated_ffn_fwd(N, D, F, 0, p[0], D, p[1], p[2], None, 0, p[3], None, p[4], n,
                                                 keep[0].cuda_stream)
    (a, run_a), (b, run_b) = call(20), call(700)
    assert not at_once(run_a, run_b)
    assert torch.equal(a[4], a[6]) and torch.equal(b[4], b[6])


def test_one_block_after_the_other_without_a_pause():
    """Each kernel may start while the one before ends: a chain of calls that read what the last one wrote, weights
    stepped in between, gives the bits of the same chain with the device waited for after every call, step by step (the
    block is quadratic in x, so that the rows of the second chain overflow near its end: bits are compared, NaN's too)."""
    def chain(wait):
        r = torch.Generator(device="cuda").manual_seed(7)
        rand = lambda *s: torch.randn(s, generator=r, device="cuda")  # noqa: E731
        D, F = 256, 512
        outs = []
        for N in (8, 300):
            x = rand(1, N, D).to(BF)
            master = [rand(D, 2 * F) / D ** 0.5, rand(F, D) / F ** 0.5]
            w = [m.to(BF) for m in master]
            taps, state = rand(D, 4) / 2, torch.zeros((1, 3, D), device="cuda", dtype=BF)
            opt = ttm.adamw_state(master, bits=8)
            go = torch.cuda.synchronize if wait else (lambda: None)
            for _ in range(6):
                x = ttm.causal_conv_step(x, taps, state)
                go()
                y, gu = ttm.gated_ffn_fwd(x, *w, residual=x)
                go()
                g = ttm.gated_ffn_bwd(y, x, gu, *w)
                go()
                ttm.adamw_step(master, [g["dW_in"], g["dW_out"]], opt, lr=1e-2, copies=w)
                go()
                c = ttm.causal_conv_bwd(y, x, taps)
                go()
                x = ttm.causal_conv_fwd(c["dx"], taps, want_state=False)[0]
                go()
                outs += [x, y, c["dw"], *g.values(), *(t.clone() for t in (*master, *w, state))]
            outs.append(ttm.adamw_moments(opt)[0])
        torch.cuda.synchronize()
        return [t.view(torch.uint8) for t in outs]
    assert all(torch.equal(a, b) for a, b in zip(chain(False), chain(True)))


def test_a_captured_step_of_many_rows():
    """A pass, its gradient and the optimiser's step in one graph, at a size whose tiles take a launch for the whole rounds and one
    beside it: replays give the bits of calls one by one, weights changing from replay to replay."""
    N, D, F = 9001, 264, 2008

    def made():
        r = torch.Generator(device="cuda").manual_seed(5)
        rand = lambda *s: torch.randn(s, generator=r, device="cuda")  # noqa: E731
        x, dy = rand(N, D).to(BF), rand(N, D).to(BF)
        master = [rand(D, 2 * F) / D ** 0.5, rand(F, D) / F ** 0.5]
        return x, dy, master, [m.to(BF) for m in master], ttm.adamw_state(master)

    def step(x, dy, master, w, state):
        y, gu = ttm.gated_ffn_fwd(x, *w, residual=dy)
        g = ttm.gated_ffn_bwd(dy, x, gu, *w)
        ttm.adamw_step(master, [g["dW_in"], g["dW_out"]], state, lr=1e-2, copies=w)
        return y, g["dx"]
    one = made()
    for _ in range(4):
        want = step(*one)
    two = made()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        got = step(*two)
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(torch.equal(a, b) for a, b in zip(one[2] + one[3], two[2] + two[3]))
