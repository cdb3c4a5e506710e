"""Calls of two host threads on a stream each, of sizes whose launches ask for different shared memory: each gives
what it gives alone."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def awq():
    from w4a16_weight_only_gb300 import build
    build.build()
    import w4a16_weight_only_gb300 as awq
    assert awq.runtime_available(), awq.last_error()
    return awq


def together(calls, times):
    """Every call `times` times, as fast as it can be made, from a thread and on a stream of its own; what went wrong."""
    want, failed = [[t.clone() for t in call()] for call in calls], []
    torch.cuda.synchronize()
    start = threading.Barrier(len(calls))

    def work(call, right):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for _ in range(times // 100):
                    for _ in range(100):
                        got = call()
                    if not all(torch.equal(a, b) for a, b in zip(got, right)):
                        failed.append("values")
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(calls, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return failed


def test_moe_layers_of_different_sizes(awq):
    g = torch.Generator(device="cuda").manual_seed(1)
    word = lambda *s: torch.randint(-2 ** 31, 2 ** 31, s, generator=g, device="cuda", dtype=torch.int64).int()  # noqa: E731
    linear = lambda K, N: (word(4, K, N // 8), word(4, K // 128, N // 8), 0.01 * torch.rand((4, K // 128, N), generator=g, device="cuda").half())  # noqa: E731
    up, down = linear(256, 256), linear(128, 256)

    def layer(T, k):
        x, ids = torch.randn((T, 256), generator=g, device="cuda").half(), word(T, k) & 3
        weights = torch.rand((T, k), generator=g, device="cuda")
        ws = torch.empty((awq.awq_moe_layer_workspace_size(T, k, 256, 128),), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(x)
        return lambda: (awq.awq_moe_layer(x, weights, ids, up, down, workspace=ws, out=out),)

    failed = together([layer(1, 1), layer(16, 32), layer(3, 1), layer(16, 16), layer(2, 1), layer(16, 31), layer(1, 2), layer(16, 30)], 3000)
    assert not failed, failed[:1]


def test_dispatches_of_different_numbers_of_experts(awq):
    g = torch.Generator(device="cuda").manual_seed(2)

    def dispatch(E):
        x = torch.randn((600, 64), generator=g, device="cuda").half()
        ids = torch.randint(0, E, (600, 4), generator=g, device="cuda", dtype=torch.int64).int()
        out = (torch.empty((2400, 64), dtype=torch.float16, device="cuda"), torch.empty((E + 1,), dtype=torch.int32, device="cuda"),
               torch.empty((600, 4), dtype=torch.int32, device="cuda"))
        ws = torch.empty((awq.awq_moe_dispatch_workspace_size(600, 4, E),), dtype=torch.uint8, device="cuda")
        return lambda: awq.awq_moe_dispatch(x, ids, E, out=out, workspace=ws)

    failed = together([dispatch(1500), dispatch(4096), dispatch(2000), dispatch(3500), dispatch(1300), dispatch(4000)], 3000)
    assert not failed, failed[:1]
