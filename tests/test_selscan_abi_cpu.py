"""The short convolution and the selective scan refuse bad arguments on the host, before
anything is enqueued (the pointers here are never dereferenced)."""
import ctypes

import pytest
import torch

import state_space_sequence_chunk_gb300 as ssd
from state_space_sequence_chunk_gb300 import build as ssd_build
from test_operators_abi_cpu import ALIAS, ALIGN, BIG, DTYPE, NULL, SHAPE, WORKSPACE, accepted, inside, ptrs, put


@pytest.fixture(scope="module")
def lib():
    ssd_build.build()
    return ssd.load_library()


def cd(**kw):
    base = dict(nseqs=2, tokens=4000, dim=512, width=4, x_stride=0, activation=1, dtype=ssd.SSD_BF16, reserved=0)
    return ctypes.byref(ssd.ShortConvDims(*{**base, **kw}.values()))


def sd(**kw):
    base = dict(nseqs=2, tokens=4000, dim=512, dstate=16, ngroups=2, x_stride=0, dt_stride=0, z_stride=0, B_stride=0,
                C_stride=0, max_seqlen=0, dt_softplus=1, dtype=ssd.SSD_BF16, reserved=0)
    return ctypes.byref(ssd.SelscanDims(*{**base, **kw}.values()))


@pytest.mark.parametrize("kw,code", [
    (dict(dim=4), SHAPE), (dict(dim=12), SHAPE), (dict(dim=65544), SHAPE), (dict(width=1), SHAPE), (dict(width=9), SHAPE),
    (dict(tokens=-1), SHAPE), (dict(nseqs=-1), SHAPE), (dict(nseqs=(1 << 20) + 1), SHAPE), (dict(tokens=1 << 31), SHAPE),
    (dict(activation=2), SHAPE), (dict(dtype=2), DTYPE), (dict(reserved=1), SHAPE), (dict(x_stride=500), SHAPE),
    (dict(x_stride=516), SHAPE), (dict(tokens=1 << 30, dim=65536), SHAPE)])
def test_conv_sizes(lib, kw, code):
    d, p = cd(**kw), ptrs(13)
    assert lib.ssd_short_conv_fwd(d, *p[:7], None) == code
    assert lib.ssd_short_conv_bwd(d, *p[:12], BIG, None) == code
    assert lib.ssd_short_conv_step(d, *p[:5], 8, p[5], None) == code
    assert lib.ssd_short_conv_bwd_workspace_bytes(d) == 0


def test_conv_fwd_arguments(lib):
    # x, weight, bias, cu, init, out, final
    p = ptrs(7)
    call = lambda a, d=cd(): lib.ssd_short_conv_fwd(d, *a, None)
    for i in (0, 1, 5):
        assert call(put(p, i, None)) == NULL
    for i in range(7):
        assert call(put(p, i, inside(p[i], 8))) == ALIGN
    assert call(put(p, 5, p[0])) == ALIAS              # not in place
    assert call(put(p, 6, p[4])) == ALIAS              # nor the states
    assert call(put(p, 6, inside(p[5]))) == ALIAS
    assert call(put(p, 3, None), cd(nseqs=3)) == SHAPE  # equal lengths have to divide the tokens
    assert accepted(call, put(put(put(p, 2, None), 4, None), 6, None))
    assert call([None] * 7, cd(nseqs=0, tokens=0)) == 0


def test_conv_bwd_arguments(lib):
    # x, weight, bias, cu, init, dout, dfinal, dx, dweight, dbias, dinit, workspace
    p = ptrs(12)
    d = cd()
    call = lambda a, n=BIG, dd=d: lib.ssd_short_conv_bwd(dd, *a, n, None)
    for i in (0, 1, 5, 7, 8, 11):
        assert call(put(p, i, None)) == NULL
    for i in range(12):
        assert call(put(p, i, inside(p[i], 4))) == ALIGN
    need = lib.ssd_short_conv_bwd_workspace_bytes(d)
    assert need > 0 and call(p, ctypes.c_size_t(need - 1)) == WORKSPACE
    for i in (7, 8, 9, 10, 11):
        for j in (0, 1, 2, 4, 5, 6):
            assert call(put(p, i, inside(p[j]))) == ALIAS
    assert call(put(p, 8, inside(p[7]))) == ALIAS
    assert accepted(call, put(put(put(p, 6, None), 9, None), 10, None))


def test_conv_step_arguments(lib):
    # x, weight, bias, slots, cache, out
    p, d = ptrs(6), cd(nseqs=5, tokens=5)
    call = lambda a, n=8, dd=d: lib.ssd_short_conv_step(dd, *a[:5], n, a[5], None)
    for i in (0, 1, 4, 5):
        assert call(put(p, i, None)) == NULL
    for i in range(6):
        assert call(put(p, i, inside(p[i], 4))) == ALIGN
    assert call(put(p, 5, inside(p[4]))) == ALIAS
    assert call(put(p, 4, inside(p[0], 64))) == ALIAS
    assert call(p, n=-1) == SHAPE
    assert call(put(p, 3, None), n=4) == SHAPE         # without slots, row b needs slot b
    assert accepted(call, put(p, 3, None), n=5)
    assert call(p, dd=cd(nseqs=5, tokens=6)) == SHAPE
    assert call([None] * 6, n=0, dd=cd(nseqs=0, tokens=0)) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(dim=4), SHAPE), (dict(dim=65544, ngroups=1), SHAPE), (dict(dim=520), SHAPE), (dict(dstate=0), SHAPE),
    (dict(dstate=65), SHAPE), (dict(ngroups=0), SHAPE), (dict(ngroups=3), SHAPE), (dict(ngroups=128), SHAPE),
    (dict(tokens=-1), SHAPE), (dict(nseqs=-1), SHAPE), (dict(nseqs=(1 << 20) + 1), SHAPE), (dict(tokens=1 << 31), SHAPE),
    (dict(max_seqlen=-1), SHAPE), (dict(dt_softplus=2), SHAPE), (dict(dtype=3), DTYPE), (dict(reserved=1), SHAPE),
    (dict(x_stride=500), SHAPE), (dict(dt_stride=516), SHAPE), (dict(z_stride=508), SHAPE), (dict(B_stride=31), SHAPE),
    (dict(C_stride=1), SHAPE)])
def test_scan_sizes(lib, kw, code):
    d, p = sd(**kw), ptrs(22)
    assert lib.ssd_selscan_fwd(d, *p[:14], BIG, None) == code
    assert lib.ssd_selscan_bwd(d, *p[:22], BIG, None) == code
    assert lib.ssd_selscan_step(d, *p[:10], 8, p[10], None) == code
    assert lib.ssd_selscan_workspace_bytes(d, 0) == 0 and lib.ssd_selscan_workspace_bytes(d, 1) == 0


def test_scan_fwd_arguments(lib):
    # x, dt, A, B, C, D, z, bias, cu, init, y, final, states, workspace
    p, d = ptrs(14), sd()
    call = lambda a, n=BIG, dd=d: lib.ssd_selscan_fwd(dd, *a, n, None)
    for i in (0, 1, 2, 3, 4, 10, 13):
        assert call(put(p, i, None)) == NULL
    for i in range(14):
        if i not in (3, 4):
            assert call(put(p, i, inside(p[i], 8))) == ALIGN
    for i in (3, 4):                                   # B and C: their type's alignment only
        assert call(put(p, i, inside(p[i], 1))) == ALIGN
        assert accepted(call, put(p, i, inside(p[i], 2)))
    need = lib.ssd_selscan_workspace_bytes(d, 0)
    assert need > 0 and call(p, ctypes.c_size_t(need - 1)) == WORKSPACE
    assert lib.ssd_selscan_workspace_bytes(sd(nseqs=4000, max_seqlen=1), 0) == 0
    assert call(put(p, 10, p[0])) == ALIAS             # not in place
    assert call(put(p, 11, inside(p[9]))) == ALIAS     # final state across the initial one
    assert call(put(p, 13, inside(p[10]))) == ALIAS
    assert call(put(p, 12, inside(p[3]))) == ALIAS
    assert accepted(call, put(p, 11, p[9]))            # in place
    none = p
    for i in (5, 6, 7, 9, 11, 12):
        none = put(none, i, None)
    assert accepted(call, none)
    assert call(put(p, 8, None), dd=sd(nseqs=3)) == SHAPE
    assert call([None] * 14, 0, sd(nseqs=0, tokens=0)) == 0


def test_scan_bwd_arguments(lib):
    # x, dt, A, B, C, D, z, bias, cu, states, dout, dfinal | dx, ddt, dA, dB, dC, dD, dz, dbias, dinit, workspace
    p, d = ptrs(22), sd()
    call = lambda a, n=BIG, dd=d: lib.ssd_selscan_bwd(dd, *a, n, None)
    for i in (0, 1, 2, 3, 4, 9, 10, 12, 13, 14, 15, 16, 18, 21):
        assert call(put(p, i, None)) == NULL
    for i in range(22):
        if i not in (3, 4):
            assert call(put(p, i, inside(p[i], 4))) == ALIGN
    need = lib.ssd_selscan_workspace_bytes(d, 1)
    assert call(p, ctypes.c_size_t(need - 1)) == WORKSPACE
    for i in range(12, 22):
        for j in (0, 1, 2, 4, 6, 9, 10, 11):
            assert call(put(p, i, inside(p[j]))) == ALIAS
    assert call(put(p, 13, inside(p[12]))) == ALIAS
    none = p
    for i in (5, 6, 7, 11, 17, 18, 19, 20):
        none = put(none, i, None)
    assert accepted(call, none)


def test_scan_step_arguments(lib):
    # x, dt, A, B, C, D, z, bias, slots, cache, y
    p, d = ptrs(11), sd(nseqs=5, tokens=5)
    call = lambda a, n=8, dd=d: lib.ssd_selscan_step(dd, *a[:10], n, a[10], None)
    for i in (0, 1, 2, 3, 4, 9, 10):
        assert call(put(p, i, None)) == NULL
    for i in range(11):
        if i not in (3, 4):
            assert call(put(p, i, inside(p[i], 4))) == ALIGN
    assert call(put(p, 10, inside(p[9]))) == ALIAS
    assert call(put(p, 9, inside(p[0], 64))) == ALIAS
    assert call(p, n=-1) == SHAPE
    assert call(put(p, 8, None), n=4) == SHAPE         # without slots, row b needs slot b
    assert accepted(call, put(p, 8, None), n=5)
    assert call(p, dd=sd(nseqs=5, tokens=6)) == SHAPE
    assert call([None] * 11, n=0, dd=sd(nseqs=0, tokens=0)) == 0


class Stand:
    """A host tensor that passes for one on the GPU `index`: only its shape, strides and
    device are looked at here."""

    def __init__(self, t, index=0):
        self.t, self.index = t, index

    is_cuda = True

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


def operands(**kw):
    f = lambda *s: Stand(torch.zeros(*s))
    base = dict(x=f(6, 16), dt=f(6, 16), A=f(16, 4), B=f(6, 2, 4), C=f(6, 2, 4), D=f(16), z=f(6, 16), dt_bias=f(16))
    return {**base, **kw}


@pytest.mark.parametrize("kw,error", [
    (dict(x=Stand(torch.zeros(1, 16).expand(6, 16))), ValueError),        # rows that share memory
    (dict(B=Stand(torch.zeros(1, 2, 4).expand(6, 2, 4))), ValueError),
    (dict(dt=Stand(torch.zeros(6, 16, dtype=torch.bfloat16))), TypeError),
    (dict(A=Stand(torch.zeros(16, 4, dtype=torch.bfloat16))), TypeError),
    (dict(x=Stand(torch.zeros(6, 16, dtype=torch.float16)), dt=Stand(torch.zeros(6, 16, dtype=torch.float16))), TypeError),
    (dict(C=Stand(torch.zeros(6, 4, 2))), ValueError),
    (dict(D=Stand(torch.zeros(8))), ValueError),
    (dict(z=Stand(torch.zeros(5, 16))), ValueError)])
def test_scan_binding_refuses(kw, error):
    with pytest.raises(error):
        ssd._selscan_dims(**operands(**kw), dt_softplus=True, nseqs=1, max_seqlen=0, dev=0)


def test_scan_binding_takes_column_ranges():
    wide = torch.zeros(6, 100)
    d = ssd._selscan_dims(**operands(x=Stand(wide[:, 32:48]), B=Stand(wide[:, 3:11].view(6, 2, 4))), dt_softplus=False,
                          nseqs=1, max_seqlen=0, dev=0)[0]
    assert (d.x_stride, d.B_stride, d.C_stride, d.dt_softplus) == (100, 100, 8, 0)


def test_conv_binding_refuses():
    x, w, b = Stand(torch.zeros(6, 16)), Stand(torch.zeros(16, 4)), Stand(torch.zeros(16))
    with pytest.raises(ValueError):
        ssd._short_conv_dims(x, w, b, "relu", 1, 0)
    with pytest.raises(ValueError):
        ssd._short_conv_dims(Stand(torch.zeros(1, 16).expand(6, 16)), w, b, None, 1, 0)
    with pytest.raises(ValueError):
        ssd._short_conv_dims(x, Stand(torch.zeros(8, 4)), b, None, 1, 0)
    with pytest.raises(TypeError):
        ssd._short_conv_dims(x, w, Stand(torch.zeros(16, dtype=torch.bfloat16)), None, 1, 0)


@pytest.mark.parametrize("name", ["x", "dt", "A", "B", "C", "D", "z", "dt_bias"])
def test_operands_of_another_device_are_refused(name):
    for bad in (Stand(operands()[name].t, 1), operands()[name].t):      # another GPU's, the host's
        with pytest.raises(ValueError):
            ssd._selscan_dims(**operands(**{name: bad}), dt_softplus=True, nseqs=1, max_seqlen=0, dev=0)
    with pytest.raises(ValueError):
        ssd._selscan_dims(**operands(), dt_softplus=True, nseqs=1, max_seqlen=0, dev=1)   # the current one is another
