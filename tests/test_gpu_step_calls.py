"""Calls of the operators around a 4-bit cache that are made in the middle of other work: on another stream than
the current one, by threads that share a stream, under another current device, with bad arguments."""
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


def calls(awq):
    """name -> a call that takes stream= and returns a tuple of new tensors."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").half()  # noqa: E731
    T = 8192
    q, k, v = rand(T, 8, 128), rand(T, 2, 128), rand(T, 2, 128)
    table, pos = awq.awq_rope_table(64, 128), torch.arange(T, dtype=torch.int32, device="cuda") % 64
    cache = torch.zeros((T // 16, 2, awq.awq_kv4_page_bytes(16, 128)), dtype=torch.uint8, device="cuda")
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    awq.awq_rope_append_kv4(q, k, v, pos, table, cache, slots)
    pages, lens = slots[:T // 16].view(8, -1), torch.full((8,), T // 8, dtype=torch.int32, device="cuda")
    many = q.view(8, T // 8, 8, 128)[:, :130]
    x, r, w = rand(T, 1024), rand(T, 1024), rand(1024)
    word = lambda *s: torch.randint(-2 ** 31, 2 ** 31, s, generator=g, device="cuda", dtype=torch.int64).int()  # noqa: E731
    linear = lambda K, N: (word(4, K, N // 8), word(4, K // 128, N // 8), 0.01 * torch.rand((4, K // 128, N), generator=g, device="cuda").half())  # noqa: E731
    up, down = linear(1024, 512), linear(256, 1024)
    ids, weights = word(16, 2) & 3, torch.rand((16, 2), generator=g, device="cuda")
    return {
        "awq_rope_append_kv4": lambda **s: (awq.awq_rope_append_kv4(q, k, v, pos, table, cache, slots, **s),),
        "awq_kv4_read": lambda **s: awq.awq_kv4_read(cache, slots, 128, **s),
        "awq_attention_kv4": lambda **s: (awq.awq_attention_kv4(many, cache, pages, lens, **s),),
        "awq_residual_norm": lambda **s: awq.awq_residual_norm(x, r, weight=w, **s),
        "awq_moe_layer": lambda **s: (awq.awq_moe_layer(x[:16], weights, ids, up, down, **s),),
    }


NAMES = ["awq_rope_append_kv4", "awq_kv4_read", "awq_attention_kv4", "awq_residual_norm", "awq_moe_layer"]


@pytest.fixture(scope="module")
def table(awq):
    t = calls(awq)
    assert list(t) == NAMES
    return t


@pytest.mark.parametrize("form", ["object", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_outputs_on_another_stream_share_nothing_with_earlier_work(table, name, form):
    call, s = table[name], torch.cuda.Stream()
    arg = s if form == "object" else s.cuda_stream
    call(stream=arg)  # the stream's workspace exists
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.empty_like(t) for t in want]
    torch.cuda._sleep(20_000_000)
    for b in blocks:
        b.fill_(1.0)  # runs after the call's kernels have finished
    del blocks, b
    got = call(stream=arg)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_threads_that_share_a_stream(table, name):
    want, failed = [t.clone() for t in table[name]()], []

    def work():
        try:
            for _ in range(20):
                if not all(torch.equal(a, b) for a, b in zip(table[name](), want)):
                    failed.append("values")
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed[:1]


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_device(awq, table, monkeypatch, name):
    from w4a16_weight_only_gb300 import _layer, _step
    with monkeypatch.context() as m:  # one device is enough: another one is said to be current
        m.setattr(_layer, "_device", lambda: 1)
        m.setattr(_step, "_device", lambda: 1)
        with pytest.raises(ValueError, match="current device"):
            table[name]()
    table[name]()


def test_refusals(awq):
    half = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")  # noqa: E731
    ints = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = torch.zeros((2, 2, awq.awq_kv4_page_bytes(16, 64, 32)), dtype=torch.uint8, device="cuda")
    table = awq.awq_rope_table(16, 64)
    append = dict(q=half(3, 4, 64), k=half(3, 2, 64), v=half(3, 2, 64), positions=ints(3), table=table, cache=cache,
                  slots=torch.arange(3, dtype=torch.int32, device="cuda"), group_size=32)
    awq.awq_rope_append_kv4(**append)
    for change, error in ((dict(k=half(3, 64)), ValueError), (dict(v=half(3, 1, 64)), ValueError), (dict(group_size=64), ValueError),
                          (dict(group_size=48), ValueError), (dict(cache=cache[:, :, :-16]), ValueError),
                          (dict(cache=cache.view(2, 1, -1)), ValueError), (dict(cache=cache.int()), ValueError),
                          (dict(positions=None), ValueError), (dict(table=None), ValueError), (dict(q=half(2, 4, 64)), ValueError),
                          (dict(q=None, q_out=half(3, 4, 64)), ValueError), (dict(slots=ints(3).long()), TypeError),
                          (dict(k=append["k"].float()), TypeError), (dict(k=append["k"].cpu()), ValueError),
                          (dict(cache=cache.cpu()), ValueError)):
        with pytest.raises(error):
            awq.awq_rope_append_kv4(**{**append, **change})
    with pytest.raises(TypeError):
        awq.awq_kv4_read(cache, ints(3), 64, group_size=32, dtype=torch.float32)
    with pytest.raises(ValueError):
        awq.awq_kv4_read(cache, ints(3), 128, group_size=128)
    call = dict(q=half(2, 4, 64), cache=cache, pages=ints(2, 1), lens=ints(2), group_size=32)
    awq.awq_attention_kv4(**call)
    for change, error in ((dict(q=half(2, 64)), ValueError), (dict(q=half(2, 3, 64)), awq.AwqError), (dict(pages=ints(1, 1)), ValueError),
                          (dict(pages=ints(2, 1).long()), ValueError), (dict(lens=ints(3)), ValueError), (dict(window=-1), awq.AwqError),
                          (dict(sinks=-1), awq.AwqError), (dict(q=half(2, 4, 128)), ValueError), (dict(out=half(2, 4, 32)), ValueError),
                          (dict(q=half(2, 4, 65)[:, :, :64]), awq.AwqError),
                          (dict(workspace=torch.zeros((8,), dtype=torch.uint8, device="cuda")), awq.AwqError)):
        with pytest.raises(error):
            awq.awq_attention_kv4(**{**call, **change})


def test_the_step_in_one_graph(awq):
    # append, attention, norm and experts as a decode loop captures them: replayed for a second token
    g = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").half()  # noqa: E731
    cache = torch.zeros((16, 2, awq.awq_kv4_page_bytes(16, 64, 64)), dtype=torch.uint8, device="cuda")
    table = awq.awq_rope_table(64, 64)
    q, k, v, w = rand(3, 4, 64), rand(3, 2, 64), rand(3, 2, 64), rand(256)
    pages = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)
    pos, slots = torch.zeros((3,), dtype=torch.int32, device="cuda"), pages[:, 0] * 16
    lens, x = pos + 1, rand(3, 256)

    def step():
        turned = awq.awq_rope_append_kv4(q, k, v, pos, table, cache, slots, group_size=64)
        a = awq.awq_attention_kv4(turned, cache, pages, lens, group_size=64, window=2, sinks=1)
        return awq.awq_residual_norm(a.flatten(1), x, weight=w)

    step()  # the workspace exists
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    got = []
    for i in range(5):
        for t, value in ((pos, i), (lens, i + 1)):
            t.fill_(value)
        slots.copy_(pages[:, 0] * 16 + i)
        k.copy_(rand(3, 2, 64))
        graph.replay()
        got.append([t.clone() for t in out])
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[-1], want))
