"""The layout of rotary angles without a GPU."""

import pytest

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("method", ["linear", "base", "parts"])
def test_frequencies_under_another_default_device(method):
    """They are a CPU tensor wherever tensors are made by default."""
    import deepseek_sparse_attention_row_gb300 as dsa

    want = dsa.rotary_frequencies(32, stretch=4.0, method=method)
    with torch.device("meta"):
        got = dsa.rotary_frequencies(32, stretch=4.0, method=method)
    assert got.device.type == "cpu" and torch.equal(got, want)
    assert dsa.rotary_turns(got, device="cpu").device.type == "cpu"
