"""Numbers of experts that do not fit the library's int are refused by the binding's quick checks
as well."""
import pytest
import torch

from decode_projection_gemms_gb300 import binding


@pytest.mark.parametrize("E", [2 ** 31, 2 ** 32 + 1])
def test_experts_past_32_bits_are_refused(E):
    x = torch.empty((5, 8), dtype=torch.bfloat16, device="meta")
    W = torch.empty((E, 1, 8), dtype=torch.bfloat16, device="meta")
    offsets = torch.empty(E + 1, dtype=torch.int32, device="meta")
    for operands in (lambda: binding._grouped_operands(x, W, "W", offsets, x.get_device()),
                     lambda: binding._grouped_gated_operands(x, W, W, offsets, x.get_device())):
        with pytest.raises(ValueError, match="2\\^31"):
            operands()
