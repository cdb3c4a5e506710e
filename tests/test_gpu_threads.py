"""Host threads that share a stream.  A call of several launches must be enqueued as a whole: its kernels
hand results on through the stream's workspace."""
import threading
import time

import numpy as np
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


def in_threads(*functions):
    """Runs the functions at a time; re-raises the first exception."""
    failed = []

    def guarded(f):
        try:
            f()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=guarded, args=(f,)) for f in functions]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if failed:
        raise failed[0]


class Recorder:
    """Stands in for the library: launches nothing, notes which workspaces are being enqueued on."""

    def __init__(self):
        self.lock, self.busy, self.clashes, self.calls = threading.Lock(), [], 0, 0

    def size(self, *args):
        args[-1].value = 1 << 16
        return 0

    awq_moe_dispatch_workspace_size = awq_attention_shared_workspace_size = size

    def enqueue(self, workspace):
        with self.lock:
            self.clashes += workspace in self.busy
            self.busy.append(workspace)
            self.calls += 1
        time.sleep(0.01)
        with self.lock:
            self.busy.remove(workspace)
        return 0

    def awq_moe_dispatch(self, *args):
        return self.enqueue(args[10])

    def awq_attention_shared(self, *args):
        return self.enqueue(args[-3])


def test_launches_that_share_a_workspace_are_not_interleaved(awq, monkeypatch):
    from w4a16_weight_only_gb300 import _layer
    fake = Recorder()
    monkeypatch.setattr(_layer, "_library", lambda: fake)
    x, ids = torch.zeros((8, 64), dtype=torch.float16, device="cuda"), torch.zeros((8, 2), dtype=torch.int32, device="cuda")
    q = torch.zeros((2, 4, 64), dtype=torch.float16, device="cuda")
    cache = torch.zeros((4, 16, 4, 64), dtype=torch.float16, device="cuda")
    pages = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    dispatch = lambda: [awq.awq_moe_dispatch(x, ids, 4) for _ in range(10)]  # noqa: E731
    attend = lambda: [awq.awq_attention_shared(q, cache, cache, pages[0], 16, pages, pages[:, 0].contiguous())  # noqa: E731
                      for _ in range(10)]
    in_threads(dispatch, attend, dispatch, attend)
    assert fake.calls == 40 and fake.clashes == 0


def test_growing_a_workspace_in_two_threads(awq):
    from w4a16_weight_only_gb300 import _layer
    s = torch.cuda.Stream()
    for size in (1 << 20, 3 << 20, 9 << 20):
        got = {}
        in_threads(*[lambda n=n: got.__setitem__(n, _layer.scratch(0, s.cuda_stream, n)) for n in (size // 2, size, size // 4)])
        assert all(w[1] >= n for n, w in got.items())


def test_calls_of_several_launches_from_two_threads(awq):
    rng = np.random.default_rng(3)
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").half()  # noqa: E731
    jobs = []
    for T, k, E in ((3000, 4, 64), (1500, 2, 8)):
        x, ids = rand(T, 64), torch.from_numpy(rng.integers(-1, E, (T, k)).astype(np.int32)).cuda()
        jobs.append(lambda x=x, ids=ids, E=E: awq.awq_moe_dispatch(x, ids, E))
    for B, prefix, own in ((40, 700, 60), (6, 50, 900)):
        k, v = rand(300, 16, 2, 64), rand(300, 16, 2, 64)
        q, lens = rand(B, 8, 64), torch.randint(1, own + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        pages = torch.randint(0, 300, (B, -(-own // 16)), generator=g, device="cuda", dtype=torch.int32)
        pp = torch.randint(0, 300, (-(-prefix // 16),), generator=g, device="cuda", dtype=torch.int32)
        jobs.append(lambda q=q, k=k, v=v, pp=pp, prefix=prefix, pages=pages, lens=lens:
                    (awq.awq_attention_shared(q, k, v, pp, prefix, pages, lens),))
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    got = [[] for _ in jobs]
    in_threads(*[lambda i=i, job=job: got[i].extend(job() for _ in range(200)) for i, job in enumerate(jobs)])
    torch.cuda.synchronize()
    for w, results in zip(want, got):
        assert len(results) == 200
        assert all(torch.equal(a, b) for r in results for a, b in zip(r, w))
    awq.device_status()
