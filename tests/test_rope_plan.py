"""How the rotary kernel shares out heads, asked through the C ABI on the host
(no device needed)."""
import pytest

import nvfp4_block_scaled_12_b200 as F

SMS = 148  # B200
LANES_AT_WORK = SMS * 2 * 256  # two blocks an SM


@pytest.mark.parametrize("heads0,heads1,tokens,head_dim,want", [
    (32, 8, 4, 64, (1, 1, 32, 8)),          # a token of four requests: a head a unit
    (24, 24, 4608, 128, (24, 24, 1, 1)),    # joint attention: every head of a token in one unit
    (12, 12, 30940, 128, (12, 12, 1, 1)),
    (25, 29, 1300, 128, (13, 15, 2, 2)),    # past 24 heads two units, the second with fewer
    (9, 25, 3200, 64, (9, 13, 1, 2)),
    (6, 5, 3000, 256, (6, 5, 1, 1)),
    (14, 1, 2100, 72, (7, 1, 2, 1)),        # at most 12: whole tensors would be too few units
    (9, 10, 5000, 64, (9, 10, 1, 1)),
    (24, 0, 9216, 128, (24, 0, 1, 0)),      # one tensor
])
def test_units(heads0, heads1, tokens, head_dim, want):
    assert F.nvfp4_rope_plan(heads0, heads1, tokens, head_dim, SMS) == want


def test_units_cover_every_head_and_fill_the_device_where_they_can():
    for heads0 in (1, 5, 24, 25, 100, 65535):
        for heads1 in (0, 1, 23, 48):
            for tokens in (1, 33, 1000, 4608, 30940):
                for head_dim in (8, 72, 128, 256):
                    h0, h1, n0, n1 = F.nvfp4_rope_plan(heads0, heads1, tokens, head_dim, SMS)
                    lanes = 1
                    while lanes * 8 < head_dim:
                        lanes *= 2
                    for heads, h, n in ((heads0, h0, n0), (heads1, h1, n1)):
                        assert h * n >= heads and h * (n - 1) < max(heads, 1) and h <= 24  # covered, none empty
                    assert (h0, h1) == (1, min(heads1, 1)) or tokens * (n0 + n1) * lanes >= LANES_AT_WORK


def test_bad_arguments():
    for args in ((0, 1, 1, 64, SMS), (1, -1, 1, 64, SMS), (65536, 0, 1, 64, SMS), (1, 65536, 1, 64, SMS),
                 (1, 1, 0, 64, SMS), (1, 1, 1 << 40, 64, SMS), (1, 1, 1, 4, SMS), (1, 1, 1, 60, SMS),
                 (1, 1, 1, 264, SMS), (1, 1, 1, 64, 0)):
        with pytest.raises(F.NVFP4Error) as e:
            F.nvfp4_rope_plan(*args)
        assert e.value.status == F.NVFP4_EINVAL
