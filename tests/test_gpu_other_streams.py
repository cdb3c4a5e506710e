"""What a call with stream= allocates itself: memory that neither shares a block with earlier work of the
current stream nor goes back to that stream while the call still writes it.

The caching allocator hands a block that was freed on a stream to the next allocation on that stream, at
once: right for work of that stream, which runs in order, wrong for a kernel on another one.  Each test
keeps one of the two streams busy, so that the wrong order shows in the values."""
import numpy as np
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu

T = 16384


@pytest.fixture(scope="module")
def awq():
    from w4a16_weight_only_gb300 import build
    build.build()
    import w4a16_weight_only_gb300 as awq
    assert awq.runtime_available(), awq.last_error()
    return awq


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def calls(awq):
    """name -> a call that takes stream= and returns a tuple of new tensors of 2 MB at least."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").half()  # noqa: E731
    q, k, v = rand(T, 4, 64), rand(T, 1, 64), rand(T, 1, 64)
    table, pos = awq.awq_rope_table(64, 64), torch.arange(T, dtype=torch.int32, device="cuda") % 64
    cache = [rand(T // 16, 16, 1, 64) for _ in range(2)]
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    logits, y = rand(2 * T, 64), rand(T, 128)
    rows = torch.randint(0, T, (T, 2), generator=g, device="cuda", dtype=torch.int32)
    weights = torch.rand((T, 2), generator=g, device="cuda")
    few, ids = rand(1000, 1024), torch.randint(0, 8, (1000, 2), generator=g, device="cuda", dtype=torch.int32)
    d = synth.awq_linear(20500, 512, 1024, 2048, group_size=128, bias=False)
    x, w = dev(d["x"]), [dev(d[n]) for n in ("qweight", "qzeros", "scales")]
    d8 = synth.awq8_linear(20600, 512, 1024, 2048, group_size=128, bias=False)
    x8, w8 = dev(d8["x"]), [dev(d8[n]) for n in ("qweight", "qzeros", "scales")]
    linear, packed = awq.AwqLinear(*w), awq.AwqLinear(*w, packed=True)
    stacked = [t[None].repeat(2, *[1] * t.dim()) for t in w]
    offsets = torch.tensor([0, 200, 512], dtype=torch.int32, device="cuda")
    dense = rand(4096, 2048)
    wide = [t.repeat(1, 4) for t in w]
    return {
        "awq_rope": lambda **s: awq.awq_rope(q, k, pos, table, **s),
        "awq_rope_append": lambda **s: (awq.awq_rope_append(q, k, v, pos, table, *cache, slots, **s),),
        "awq_rope_table": lambda **s: (awq.awq_rope_table(T, 64, **s),),
        "awq_attention_shared": lambda **s: (awq.awq_attention_shared(
            q, *cache, slots[:4], 60, slots[:T, None], torch.ones_like(slots), max_len=1, **s),),
        "awq_moe_route": lambda **s: awq.awq_moe_route(logits, 16, **s),
        "awq_moe_dispatch": lambda **s: awq.awq_moe_dispatch(few, ids, 8, **s)[:1],
        "awq_moe_combine": lambda **s: (awq.awq_moe_combine(y, weights, rows, **s),),
        "awq_gemm": lambda **s: (awq.awq_gemm(x, *w, **s),),
        "awq_gemm_w8": lambda **s: (awq.awq_gemm_w8(x8, *w8, **s),),
        "AwqLinear": lambda **s: (linear(x, **s),),
        "AwqLinear, packed": lambda **s: (packed(x, **s),),
        "awq_gemm_packed": lambda **s: (awq.awq_gemm_packed(x, packed.packed, None, 1024, 2048, **s),),
        "awq_gemm_packed_noalloc": lambda **s: (awq.awq_gemm_packed_noalloc(x, packed.packed, None, 1024, 2048, **s),),
        "awq_gemm_grouped": lambda **s: (awq.awq_gemm_grouped(x, *stacked, offsets, **s),),
        "awq_dequant": lambda **s: (awq.awq_dequant(*w, **s),),
        "awq_dequant_w8": lambda **s: (awq.awq_dequant_w8(*w8, **s),),
        "awq_quantize_rtn": lambda **s: awq.awq_quantize_rtn(dense, **s)[:1],
        "awq_repack": lambda **s: (awq.awq_repack(*wide, **s),),
    }


NAMES = ["awq_rope", "awq_rope_append", "awq_rope_table", "awq_attention_shared", "awq_moe_route", "awq_moe_dispatch",
         "awq_moe_combine", "awq_gemm", "awq_gemm_w8", "AwqLinear", "AwqLinear, packed", "awq_gemm_packed",
         "awq_gemm_packed_noalloc", "awq_gemm_grouped", "awq_dequant", "awq_dequant_w8", "awq_quantize_rtn", "awq_repack"]


@pytest.fixture(scope="module")
def table(awq):
    t = calls(awq)
    assert list(t) == NAMES
    return t


def block(t):
    return torch.empty((t.numel() * t.element_size(),), dtype=torch.uint8, device="cuda")


def keep_busy():
    torch.cuda._sleep(20_000_000)  # some 10 ms


@pytest.mark.parametrize("form", ["object", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_outputs_share_nothing_with_earlier_work(table, name, form):
    call, s = table[name], torch.cuda.Stream()
    arg = s if form == "object" else s.cuda_stream
    call(stream=arg)  # the stream's workspaces exist
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [block(t) for t in want]
    keep_busy()
    for b in blocks:
        b.fill_(0x7f)  # runs after the call's kernels have finished
    del blocks, b
    got = call(stream=arg)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_outputs_dropped_early_are_not_reused_early(table, name):
    call, s = table[name], torch.cuda.Stream()
    sizes = call(stream=s)
    torch.cuda.synchronize()
    blocks = [block(t) for t in sizes]
    del sizes, blocks
    torch.cuda.empty_cache()
    with torch.cuda.stream(s):
        keep_busy()
    got = call(stream=s)
    shapes = [(t.shape, t.dtype) for t in got]
    del got
    later = [torch.empty(shape, dtype=dtype, device="cuda").view(torch.uint8) for shape, dtype in shapes]
    for t in later:
        t.fill_(0x55)  # the call's kernels run after this
    torch.cuda.synchronize()
    assert all((t == 0x55).all() for t in later)


def test_outputs_may_be_used_and_dropped_on_the_current_stream(table):
    # the caller waits for the other stream, reads on its own one and drops: the block does not go back to
    # the other stream before that read
    call, s = table["awq_rope"], torch.cuda.Stream()
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    got = call(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    keep_busy()
    copies = [t.clone() for t in got]
    shapes = [t.shape for t in got]
    del got
    with torch.cuda.stream(s):
        for shape in shapes:
            torch.empty(shape, dtype=torch.float16, device="cuda").fill_(3.0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want))


@pytest.mark.parametrize("which", ["layer", "packed"])
def test_workspaces_come_from_the_stream_they_serve(awq, which):
    from w4a16_weight_only_gb300 import _binding, _layer
    s = torch.cuda.Stream()
    size = _binding.awq_gemm_packed_workspace_size() if which == "packed" else 24 << 20
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    freed = torch.empty((size,), dtype=torch.uint8, device="cuda")
    address = freed.data_ptr()
    del freed  # the current stream may still be using it
    if which == "layer":
        got = _layer.scratch(0, s.cuda_stream, size)[0]
    else:
        with torch.cuda.stream(s):
            keep_busy()
        ws = _binding.packed_workspace(0, s.cuda_stream)
        got = ws.data_ptr()
        s.synchronize()
        assert not ws.any()  # its zeros are written in the stream's order
    assert got != address


def test_the_default_stream_by_its_handle(awq, table):
    s = torch.cuda.Stream()
    want = [t.clone() for t in table["awq_rope"]()]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got = table["awq_rope"](stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
