"""Where linear attention cuts sequences into ranges, as the workspace's size shows:
the host decides it, from the sizes alone (a host without a GPU counts 152 SMs)."""
import ctypes

import pytest
import torch

import state_space_sequence_chunk_gb300 as ssd
from state_space_sequence_chunk_gb300 import build as ssd_build

cpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="the cut follows the device's number of SMs")


@pytest.fixture(scope="module")
def lib():
    ssd_build.build()
    return ssd.load_library()


def need(lib, nseqs, tokens, H, G, K, V, dtype=ssd.SSD_BF16, max_seqlen=0, backward=0):
    d = ssd.LinattnDims(nseqs, tokens, H, G, K, V, 0, 0, 0, max_seqlen, dtype, 0)
    return lib.ssd_linattn_workspace_bytes(ctypes.byref(d), backward)


@pytest.mark.parametrize("dtype", [ssd.SSD_BF16, ssd.SSD_F32])
@pytest.mark.parametrize("tokens", [1000, 4096, 10000, 1 << 20])
def test_without_a_sequence_nothing_is_cut(lib, dtype, tokens):
    """Rows that belong to no sequence (offsets [0]) need no range states."""
    assert need(lib, 0, tokens, 4, 4, 64, 64, dtype) == 0
    assert need(lib, 0, tokens, 4, 4, 64, 64, dtype, backward=1) == 0
    # shared q and k: the per-head terms of dq and dk, and no more
    assert need(lib, 0, tokens, 4, 2, 64, 64, dtype, backward=1) == 2 * tokens * 4 * 64 * 4


def slots(tokens, R):
    """Range states: one for each multiple of R in the rows and one for each first range."""
    return 2 * (tokens // R + 1)


@cpu_only
def test_ranges_of_a_batch_that_may_hold_one_long_sequence(lib):
    """8 sequences of 4001 rows in all (which 8 does not divide: where it does, the query
    covers equal lengths too), 4 heads of 64 x 128: an SM's even share is 210 rows (two
    blocks of 64 columns a head), so that a sequence of more than 512 rows, and of more
    than 210 + 236 + 1152, is cut at multiples of 512."""
    state = 4 * 64 * 128 * 4
    assert need(lib, 8, 4001, 4, 2, 64, 128, max_seqlen=1598) == 0
    assert need(lib, 8, 4001, 4, 2, 64, 128, max_seqlen=1599) == slots(4001, 512) * state
    assert need(lib, 8, 4001, 4, 2, 64, 128) == slots(4001, 512) * state
    # fp32: of more than the least range of 128 rows, and of more than 210 + 84 + 176
    assert need(lib, 8, 4001, 4, 2, 64, 128, ssd.SSD_F32, max_seqlen=470) == 0
    assert need(lib, 8, 4001, 4, 2, 64, 128, ssd.SSD_F32, max_seqlen=471) == slots(4001, 128) * state
    # the gradient runs three of them, four blocks of columns a head (a share of 421: from
    # 421 + 473 + 1152), and keeps dq and dk of each head beside them
    part = 2 * 4001 * 4 * 64 * 4
    assert need(lib, 8, 4001, 4, 2, 64, 128, backward=1, max_seqlen=2046) == part
    assert need(lib, 8, 4001, 4, 2, 64, 128, backward=1, max_seqlen=2047) == 3 * slots(4001, 512) * state + part


@pytest.mark.parametrize("backward", [0, 1])
def test_more_work_than_a_grid_holds_is_refused_as_sizes(lib, backward):
    """2^20 sequences of 2 rows in bf16: up to 2^28 chains are served, more than a grid
    has CTAs for are refused before anything is enqueued; fp32 has a grid of its own."""
    ptrs = [ctypes.c_void_p(0x10000000000000 * (i + 1)) for i in range(13)]
    big, one = ctypes.c_size_t(1 << 62), ctypes.c_float(1.0)

    def call(H, dtype):
        d = ctypes.byref(ssd.LinattnDims(1 << 20, 1 << 21, H, H, 16, 128, 0, 0, 0, 2, dtype, 0))
        if backward:
            return lib.ssd_linattn_bwd(d, *ptrs[:5], one, *ptrs[5:13], big, None)
        return lib.ssd_linattn_fwd(d, *ptrs[:4], one, *ptrs[4:9], big, None)

    assert call(4096, ssd.SSD_BF16) == 2 and call(1024 if not backward else 512, ssd.SSD_BF16) == 2
    if not torch.cuda.is_available():      # past validation there is no device to launch on
        assert call(255, ssd.SSD_BF16) in (6, 7)
        assert call(4096, ssd.SSD_F32) in (6, 7)
