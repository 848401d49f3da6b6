"""Buckets of distances whose logarithm's share comes closest to a whole number without
being one, and of those that are whole but come out farthest off (no GPU)."""
import pytest

import hadamard_rank_linear_amd as h
import oracle.attention_oracle as o

# (buckets a side, reach, distance) by a scan of all of them: off by 2^-36.4, 2^-31.3, .. 2^-23
CLOSE = [(21, 1006, 435), (73, 905, 347), (70, 1011, 568), (58, 282, 119), (50, 886, 666),
         (43, 328, 155), (72, 991, 273), (116, 564, 238), (91, 628, 560), (105, 680, 284),
         (44, 860, 728), (52, 659, 276), (19, 981, 23), (114, 681, 652)]
WHOLE = [(127, 700, 210)]      # 2^-47 off in 64 bits, the most of 252932


@pytest.mark.parametrize("side,reach,distance", CLOSE + WHOLE)
def test_borders(side, reach, distance):
    for d in (distance - 1, distance, distance + 1):
        assert h.hlq_relative_bucket(-d, side, reach, False) == o.bucket(-d, side, reach, False)
        if side <= 64:
            for s in (-d, d):
                assert h.hlq_relative_bucket(s, 2 * side, reach, True) == o.bucket(s, 2 * side, reach, True)


def test_numbers_beyond_32_bits():
    """A distance is as far as the farthest; a size is out of range."""
    far = h.hlq_relative_bucket(10 ** 6, 32), h.hlq_relative_bucket(-10 ** 6, 32)
    for n in (2 ** 31, 2 ** 32, 2 ** 32 + 3, 2 ** 40 - 1, 2 ** 64 + 1):
        assert (h.hlq_relative_bucket(n, 32), h.hlq_relative_bucket(-n, 32)) == far
        for args in ((2 ** 32 + 32, 128), (32, 2 ** 32 + 128), (-2 ** 32 + 32, 128)):
            with pytest.raises(ValueError):
                h.hlq_relative_bucket(n, *args)


@pytest.mark.parametrize("args", [(1.0,), (1, 32.0), (1, 32, 128.0), ("1",), (None,)])
def test_no_integers(args):
    with pytest.raises(TypeError):
        h.hlq_relative_bucket(*args, *(32,)[:2 - len(args)])
