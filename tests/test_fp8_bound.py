"""The bound that the SwiGLU codes are held to tells rounding to nearest from any other rounding."""
import pytest
import torch

from tests.fp8_bound import FORMATS, room


def codes_around(q, f8):
    """The format's finite values next to |q|, below (or equal) and above, and the nearest one."""
    v = torch.arange(0, 0x7F if f8 is torch.float8_e4m3fn else 0x7C, dtype=torch.uint8).view(f8).double()
    at = torch.searchsorted(v, q, right=True) - 1
    below, above = v[at], v[(at + 1).clamp(max=len(v) - 1)]
    return below, above, torch.where(q - below <= above - q, below, above)


@pytest.mark.parametrize("f8", FORMATS)
@pytest.mark.parametrize("rel", [0.0, 200 * 2.0**-24])
def test_nearest_passes_and_truncation_and_rounding_up_do_not(f8, rel):
    g = torch.Generator().manual_seed(1)
    top = FORMATS[f8][2]
    q = torch.cat([top * torch.rand(4000, generator=g, dtype=torch.float64),
                   2.0 ** (torch.rand(4000, generator=g, dtype=torch.float64) * 20 - 12).clamp(max=8.0)])
    below, above, nearest = codes_around(q, f8)
    limit = room(q, rel, f8)
    assert bool(((nearest - q).abs() <= limit).all())
    for wrong in (below, above):
        failed = (wrong - q).abs() > limit
        assert 0.4 < float(failed.double().mean()) < 0.6  # every second value rounds the other way


@pytest.mark.parametrize("f8", FORMATS)
def test_values_above_the_largest_saturate(f8):
    top = FORMATS[f8][2]
    q = torch.tensor([top * 1.01, top * 1.1, top * 1.14], dtype=torch.float64)
    assert bool(((top - q).abs() <= room(q, 0.0, f8)).all())
