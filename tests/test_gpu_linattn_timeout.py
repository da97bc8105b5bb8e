"""Failure detection in bf16 linear attention, without a GPU fault: with its loads
withheld every wait runs out (about 1 s), the call ends early whatever its size, the
error is reported once, and the calls after that are right."""
import time

import pytest
import torch

import state_space_sequence_chunk_gb300 as ssd
from linattn_ref import off
from test_gpu_linattn import TOL, dev, make, num, ref

pytestmark = pytest.mark.gpu


# one chunk; more items than CTAs; a sequence that is cut (three launches); one so long,
# and not cut, that a wait for each of its chunks would take minutes
@pytest.mark.parametrize("lens,H,max_seqlen", [([40], 1, 0), ([200] * 60, 8, 200), ([9000], 2, 0),
                                               ([700000], 1, 100)])
def test_withheld_loads_time_out_and_are_reported(lens, H, max_seqlen):
    x = dev(make("bf16", lens, H, H, 64, 128, False, seed=18))
    kw = dict(cu_seqlens=x["cu"], max_seqlen=max_seqlen)
    assert ssd.ssd_take_device_errors() == 0
    t0 = time.time()
    try:
        ssd.ssd_debug_withhold_handoffs(True)
        ssd.linattn_fwd(x["q"], x["k"], x["v"], x["a"], **kw)      # enqueued
        torch.cuda.synchronize()
    finally:
        ssd.ssd_debug_withhold_handoffs(False)
    assert time.time() - t0 < 20
    with pytest.raises(ssd.SSDError, match="SSD_ERR_TIMEOUT") as e:
        ssd.linattn_fwd(x["q"], x["k"], x["v"], x["a"], **kw)
    assert e.value.code == 9
    assert ssd.ssd_take_device_errors() == 0                       # reported once, then cleared
    small = make("bf16", [300, 7], 2, 2, 64, 64, True, seed=19)
    d = dev(small)
    o, fin = ssd.linattn_fwd(d["q"], d["k"], d["v"], d["a"], cu_seqlens=d["cu"], init_state=d["S0"])
    torch.cuda.synchronize()
    assert ssd.ssd_take_device_errors() == 0
    want = ref(small, [300, 7], 64 ** -0.5)
    assert off(num(o), want[0]) < TOL["bf16"] and off(num(fin), want[1]) < TOL["f32"]


def test_gradient_times_out_and_sets_its_bit():
    x = dev(make("bf16", [600, 50], 4, 2, 128, 64, True, seed=20))
    try:
        ssd.ssd_debug_withhold_handoffs(True)
        ssd.linattn_bwd(x["q"], x["k"], x["v"], x["dout"], x["a"], cu_seqlens=x["cu"], init_state=x["S0"],
                        dfinal_state=x["dfin"])
        errs = ssd.ssd_take_device_errors()                        # synchronises
    finally:
        ssd.ssd_debug_withhold_handoffs(False)
    assert errs == 8
    torch.cuda.synchronize()
    assert ssd.ssd_take_device_errors() == 0
