"""The arithmetic that the fp8 tile kernel's queries rest on: a row scaled by a power
of two so that its largest element lies in (224, 448], split by rounding into two
(bf16) or three (f16) E4M3 parts."""
import pytest
import torch


@pytest.mark.parametrize("dtype,parts,exact", [(torch.bfloat16, 2, 2.0 ** -9), (torch.float16, 3, 2.0 ** -6)])
def test_parts_hold_what_the_header_says(dtype, parts, exact):
    """Every positive value of the type, for the largest elements in between as well."""
    x = torch.arange(0, 0x8000, dtype=torch.int32).to(torch.int16).view(dtype).float()
    x = x[torch.isfinite(x) & (x <= 448)]
    rest = x.clone()
    for _ in range(parts):
        rest = rest - rest.to(torch.float8_e4m3fn).float()
    worst = 0.0
    for largest in x[x > 224].tolist():
        row = x <= largest
        assert (rest[row & (x >= exact * largest)] == 0).all()
        worst = max(worst, float(rest[row].abs().max()) / largest)
    assert worst <= 2.0 ** -17
    assert (rest[x < 2.0 ** -10] != 0).any()
