"""The library launches on the current device: tensors of another one are refused, not handed to it."""
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


@pytest.mark.parametrize("name", ["awq_rope_table", "awq_rope", "awq_rope_append", "awq_attention_shared", "awq_moe_route",
                                  "awq_moe_dispatch", "awq_moe_combine"])
def test_tensors_of_another_device(awq, monkeypatch, name):
    from w4a16_weight_only_gb300 import _layer
    half = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")  # noqa: E731
    ints = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    table, cache = awq.awq_rope_table(16, 64), half(2, 16, 2, 64)
    call = {
        "awq_rope_table": lambda: awq.awq_rope_table(16, 64, out=table),
        "awq_rope": lambda: awq.awq_rope(half(3, 4, 64), half(3, 2, 64), ints(3), table),
        "awq_rope_append": lambda: awq.awq_rope_append(half(3, 4, 64), half(3, 2, 64), half(3, 2, 64), ints(3), table, cache,
                                                       cache.clone(), torch.arange(3, dtype=torch.int32, device="cuda")),
        "awq_attention_shared": lambda: awq.awq_attention_shared(half(2, 4, 64), cache, cache, ints(1), 5, ints(2, 1), ints(2)),
        "awq_moe_route": lambda: awq.awq_moe_route(half(3, 8), 2),
        "awq_moe_dispatch": lambda: awq.awq_moe_dispatch(half(3, 8), ints(3, 2), 4),
        "awq_moe_combine": lambda: awq.awq_moe_combine(half(6, 8), torch.zeros((3, 2), device="cuda"), ints(3, 2)),
    }[name]
    call()
    with monkeypatch.context() as m:  # one device is enough: another one is said to be current
        m.setattr(_layer, "_device", lambda: 1, raising=False)
        with pytest.raises(ValueError, match="current device"):
            call()
    call()
