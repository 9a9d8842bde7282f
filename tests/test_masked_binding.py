"""The binding of rf_attn_fwd_window without a GPU: numbers that the library's 32-bit ints
cannot hold are refused, not cut to their low bits."""
import pytest
import torch


@pytest.mark.parametrize("name", ["window", "sinks", "max_seqlen_q", "batch"])
@pytest.mark.parametrize("x", [2**31, 2**32, 2**32 + 5, -2**31 - 1, 2**64 + 5])
def test_numbers_beyond_32_bits_are_refused(name, x):
    import cascaded_reductions_loop_gb300 as rf
    q = torch.zeros(6, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match=name):
        rf.rf_attn_fwd_window(q, q, q, q, 0.1, **{"window": 4, name: x})
