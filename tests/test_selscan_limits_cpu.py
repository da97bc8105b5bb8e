"""Sizes inside the limits that the header states for the short convolution and the selective
scan are not refused as sizes (the calls end at their missing operands, before anything is enqueued)."""
import random

import pytest

from test_selscan_abi_cpu import NULL, SHAPE, cd, lib, sd  # noqa: F401


def spread(rng, lo, hi):
    return min(hi, int(lo * (hi / lo) ** rng.random()))


@pytest.mark.parametrize("seed", range(4))
def test_scan_limits(lib, seed):  # noqa: F811
    rng, served = random.Random(seed), 0
    while served < 500:
        n, T, N, per = spread(rng, 1, 1 << 20), spread(rng, 1, 1 << 30), rng.randint(1, 64), 8 * spread(rng, 1, 8192)
        G = spread(rng, 1, 65536 // per)
        if (n + T // 64 + 64) * (per * G // 8 + 1) >= 1 << 31 or T * G * N >= 1 << 37:
            continue
        served += 1
        for most in (0, 1, T):
            d = sd(nseqs=n, tokens=T, dim=per * G, dstate=N, ngroups=G, max_seqlen=most, dtype=rng.randint(0, 1))
            cu = 4096                                   # (never dereferenced)
            assert lib.ssd_selscan_fwd(d, *[None] * 8, cu, *[None] * 5, 0, None) == NULL
            assert lib.ssd_selscan_bwd(d, *[None] * 8, cu, *[None] * 13, 0, None) == NULL


@pytest.mark.parametrize("seed", range(4))
def test_conv_limits(lib, seed):  # noqa: F811
    rng, served = random.Random(seed), 0
    while served < 500:
        n, T, D = spread(rng, 1, 1 << 20), spread(rng, 1, 1 << 30), 8 * spread(rng, 1, 8192)
        d = cd(nseqs=n, tokens=T, dim=D, width=rng.randint(2, 8), dtype=rng.randint(0, 1))
        inside = (T // 8 + n + 1) * -(-D // 64) < (1 << 31) - 4
        served += inside
        assert lib.ssd_short_conv_fwd(d, None, None, None, 4096, None, None, None, None) == (NULL if inside else SHAPE)
        assert lib.ssd_short_conv_bwd(d, None, None, None, 4096, *[None] * 8, 0, None) == (NULL if inside else SHAPE)
