"""Host threads that call the C library at the same time, each on its own stream: no call makes
another one fail, whatever shared memory the two need of the same kernel."""
import threading

import pytest
import torch

import test_neural_memory_gb300 as ttm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ttm.build()
    yield
    assert ttm.device_status() == ttm.OK


def at_once(*calls, times=4000):
    """Return codes other than OK of calls that run in a thread each (ctypes lets go of the interpreter)."""
    start, bad = threading.Barrier(len(calls)), []

    def loop(call):
        start.wait()
        bad.extend(r for r in (call() for _ in range(times)) if r != ttm.OK)

    threads = [threading.Thread(target=loop, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return bad


def test_layer_norm_gradient_with_and_without_weights():
    L, N, D = ttm.lib(), 64, 1024
    x = torch.randn(N, D, device="cuda")

    def call(weights):
        s = torch.cuda.Stream()
        mean, rstd, dx = torch.zeros(N, device="cuda"), torch.ones(N, device="cuda"), torch.empty_like(x)
        dw, db = (torch.empty(D, device="cuda") for _ in range(2))
        n = L.ttm_layer_norm_bwd_workspace_size(N, D)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        keep = (s, mean, rstd, dx, dw, db, ws)
        p = [t.data_ptr() for t in keep[1:]]
        return lambda: L.ttm_layer_norm_bwd(N, 512, 0, x.data_ptr(), D, x.data_ptr(), D, None, p[0], p[1], p[2],
                                            p[3] if weights else None, p[4] if weights else None, p[5], n,
                                            keep[0].cuda_stream)

    assert not at_once(call(True), call(False))


def test_recurrence_of_few_and_many_channels():
    L = ttm.lib()

    def call(D):
        s, T = torch.cuda.Stream(), 64
        x, h = torch.randn(1, T, D, device="cuda"), torch.empty(1, T, D, device="cuda")
        g, last = torch.zeros(1, T, device="cuda"), torch.empty(1, D, device="cuda")
        torch.cuda.synchronize()
        keep = (s, x, h, g, last)
        return lambda: L.ttm_glr_fwd(1, T, D, 0, 1, keep[1].data_ptr(), T * D, D, keep[3].data_ptr(), T, 1, None,
                                     keep[2].data_ptr(), keep[4].data_ptr(), None, 0, keep[0].cuda_stream)

    assert not at_once(call(4), call(256))
