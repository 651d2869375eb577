"""Host-side checks of the cache in 4 bits and the rotary positions that need no GPU."""
import pytest
import torch

import verify_markov_head_gb300 as vm


def test_attention_over_four_bits_names_a_workspace_without_room_for_it():
    c, x = vm.Cache4(2, 1, 16, 64, device="cpu"), torch.zeros((1, 1, 64))
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    ws = type("W", (), {"buf": torch.zeros(1 << 20, dtype=torch.uint8), "buf4": None})()
    with pytest.raises(ValueError, match="four_bits"):
        vm.dspark_cache_attention4(x, *c.tensors, i(1, 2), i(1), i(2), i(2), x.clone(), ws, max_new=1, stream=0)


def test_a_factor_without_a_kind_is_refused():
    for bad in (dict(factor=8.0), dict(kind=None, factor=0.5)):
        with pytest.raises(ValueError, match="kind"):
            vm.rope_frequencies(64, 10000.0, bad)
        with pytest.raises(ValueError, match="kind"):
            vm.RopeTable(64, scaling=bad, device="cpu")
    assert vm.rope_frequencies(64, 10000.0, {}) == vm.rope_frequencies(64) == vm.rope_frequencies(64, scaling=dict(kind=None))


def test_an_order_of_pairs_that_is_no_truth_value_is_refused():
    with pytest.raises(RuntimeError, match="ambiguous"):
        vm.dspark_rope(torch.zeros((1, 1, 64)), None, torch.zeros(1, dtype=torch.int32), vm.RopeTable(64, device="cpu"), interleaved=torch.zeros(2),
                     stream=type("Stream", (), {"cuda_stream": 256})())   # (not used: the tensors are not on the device)
