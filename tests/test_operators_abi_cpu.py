"""Linear attention and the block norms refuse bad arguments on the host, before
anything is enqueued (the pointers here are never dereferenced)."""
import ctypes

import pytest
import torch

import state_space_sequence_chunk_gb300 as ssd
from state_space_sequence_chunk_gb300 import build as ssd_build

NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, ALIAS = 1, 2, 3, 4, 5, 8
DEVICE = (6, 7)      # past validation: there is no device to launch on


@pytest.fixture(scope="module")
def lib():
    ssd_build.build()
    return ssd.load_library()


def accepted(call, *args, **kw):
    """Whether the arguments pass validation.  Where there is a device, a call that
    passes would launch with pointers that lead nowhere: it is not made."""
    return torch.cuda.is_available() or call(*args, **kw) in DEVICE


def la(**kw):
    base = dict(nseqs=2, tokens=4000, nheads=4, ngroups=2, kdim=64, vdim=128, q_stride=0, k_stride=0,
                v_stride=0, max_seqlen=0, dtype=ssd.SSD_BF16, reserved=0)
    return ssd.LinattnDims(*{**base, **kw}.values())


def nd(**kw):
    base = dict(tokens=100, width=512, ngroups=4, y_stride=0, z_stride=0, gate=1, eps=1e-5,
                dtype=ssd.SSD_BF16, rdtype=ssd.SSD_F32, reserved=0)
    return ssd.NormDims(*{**base, **kw}.values())


def ptrs(n):
    return [ctypes.c_void_p(0x10000000000 * (i + 1)) for i in range(n)]


def put(args, i, v):
    return args[:i] + [v] + args[i + 1:]


def inside(p, n=256):
    return ctypes.c_void_p(p.value + n)


BIG = ctypes.c_size_t(1 << 40)
BAD_LA = [(dict(kdim=40), SHAPE), (dict(kdim=144), SHAPE), (dict(vdim=8), SHAPE), (dict(ngroups=3), SHAPE),
          (dict(nheads=0), SHAPE), (dict(tokens=-1), SHAPE), (dict(nseqs=-1), SHAPE), (dict(dtype=4), DTYPE),
          (dict(reserved=1), SHAPE), (dict(q_stride=100), SHAPE), (dict(v_stride=516), SHAPE),
          (dict(max_seqlen=-1), SHAPE), (dict(tokens=1 << 31), SHAPE)]


@pytest.mark.parametrize("kw,code", BAD_LA)
def test_linattn_sizes(lib, kw, code):
    d = ctypes.byref(la(**kw))
    p = ptrs(14)
    f = ctypes.c_float(1.0)
    assert lib.ssd_linattn_fwd(d, *p[:4], f, *p[4:9], BIG, None) == code
    assert lib.ssd_linattn_bwd(d, *p[:5], f, *p[5:13], BIG, None) == code
    assert lib.ssd_linattn_step(d, *p[:4], f, p[4], p[5], 8, p[6], None) == code
    assert lib.ssd_linattn_workspace_bytes(d, 0) == 0


def test_linattn_fwd_arguments(lib):
    # q, k, v, log_decay | cu, init, o, final, workspace
    d, p, f = ctypes.byref(la()), ptrs(9), ctypes.c_float(1.0)
    call = lambda a, n=BIG, s=f, dd=d: lib.ssd_linattn_fwd(dd, *a[:4], s, *a[4:9], n, None)
    for i in (0, 1, 2, 3, 6, 8):
        assert call(put(p, i, None)) == NULL
    for i in range(9):
        assert call(put(p, i, inside(p[i], 8))) == ALIGN
    need = lib.ssd_linattn_workspace_bytes(d, 0)
    assert need > 0 and call(p, ctypes.c_size_t(need - 1)) == WORKSPACE
    assert call(p, s=ctypes.c_float(float("nan"))) == SHAPE
    assert call(put(p, 6, inside(p[0]))) == ALIAS      # o in q
    assert call(put(p, 7, inside(p[5]))) == ALIAS      # final state across the initial one
    assert call(put(p, 8, inside(p[6]))) == ALIAS      # workspace in o
    assert accepted(call, put(p, 7, p[5]))             # in place
    assert accepted(call, put(put(p, 5, None), 7, None))
    # equal lengths have to divide the tokens
    assert call(put(p, 4, None), dd=ctypes.byref(la(nseqs=3))) == SHAPE
    # nothing is cut when the caller says that no sequence is long
    short = ctypes.byref(la(max_seqlen=500))
    assert lib.ssd_linattn_workspace_bytes(ctypes.byref(la(nseqs=8, max_seqlen=500)), 0) == 0
    assert lib.ssd_linattn_workspace_bytes(short, 0) >= 0
    assert lib.ssd_linattn_fwd(ctypes.byref(la(nseqs=0, tokens=0)), *[None] * 4, f, *[None] * 5, 0, None) == 0


def test_linattn_bwd_arguments(lib):
    # q, k, v, dout, log_decay | cu, init, dfinal, dq, dk, dv, dinit, workspace
    d, p, f = ctypes.byref(la()), ptrs(13), ctypes.c_float(1.0)
    call = lambda a, n=BIG: lib.ssd_linattn_bwd(d, *a[:5], f, *a[5:13], n, None)
    for i in (0, 1, 2, 3, 4, 8, 9, 10, 12):
        assert call(put(p, i, None)) == NULL
    for i in range(13):
        assert call(put(p, i, inside(p[i], 4))) == ALIGN
    need = lib.ssd_linattn_workspace_bytes(d, 1)
    assert call(p, ctypes.c_size_t(need - 1)) == WORKSPACE
    for i in (8, 9, 10, 11):
        for j in (0, 1, 2, 3, 7):
            assert call(put(p, i, inside(p[j]))) == ALIAS
    assert call(put(p, 9, inside(p[8]))) == ALIAS
    assert accepted(call, put(put(put(p, 6, None), 7, None), 11, None))


def test_linattn_step_arguments(lib):
    d, p, f = ctypes.byref(la(nseqs=5, tokens=5)), ptrs(7), ctypes.c_float(1.0)
    call = lambda a, n=8, dd=d: lib.ssd_linattn_step(dd, *a[:4], f, a[4], a[5], n, a[6], None)
    for i in (0, 1, 2, 3, 5, 6):
        assert call(put(p, i, None)) == NULL
    for i in range(7):
        assert call(put(p, i, inside(p[i], 4))) == ALIGN
    assert call(put(p, 6, inside(p[5]))) == ALIAS
    assert call(put(p, 5, inside(p[0], 64))) == ALIAS
    assert call(p, n=-1) == SHAPE
    assert call(put(p, 4, None), n=4) == SHAPE         # without slots, row b needs slot b
    assert accepted(call, put(p, 4, None), n=5)
    assert call(p, dd=ctypes.byref(la(nseqs=5, tokens=6))) == SHAPE
    assert call([None] * 7, n=0, dd=ctypes.byref(la(nseqs=0, tokens=0))) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(width=4), SHAPE), (dict(width=16392), SHAPE), (dict(ngroups=3), SHAPE), (dict(ngroups=128), SHAPE),
    (dict(ngroups=0), SHAPE), (dict(tokens=-1), SHAPE), (dict(gate=3), SHAPE), (dict(eps=-1.0), SHAPE),
    (dict(eps=float("nan")), SHAPE), (dict(dtype=2), DTYPE), (dict(rdtype=7), DTYPE),
    (dict(dtype=ssd.SSD_F32, rdtype=ssd.SSD_BF16), DTYPE), (dict(y_stride=500), SHAPE),
    (dict(z_stride=514), SHAPE), (dict(reserved=2), SHAPE)])
def test_norm_sizes(lib, kw, code):
    d, p = ctypes.byref(nd(**kw)), ptrs(18)
    assert lib.ssd_block_norm_fwd(d, *p[:10], None) == code
    assert lib.ssd_block_norm_bwd(d, *p[:17], BIG, None) == code
    assert lib.ssd_block_norm_bwd_workspace_bytes(d) == 0


def test_norm_fwd_arguments(lib):
    # r, y, z, w_post, alpha, w_pre, r_out, n, rstd_post, rstd_pre
    d, p = ctypes.byref(nd()), ptrs(10)
    call = lambda a, dd=d: lib.ssd_block_norm_fwd(dd, *a, None)
    for i in (0, 1, 2, 5, 6, 7):
        assert call(put(p, i, None)) == NULL
    for i in range(10):
        assert call(put(p, i, inside(p[i], 4))) == ALIGN
    assert call(put(p, 7, inside(p[1]))) == ALIAS
    assert call(put(p, 6, inside(p[0]))) == ALIAS
    assert accepted(call, put(p, 6, p[0]))             # in place
    assert call(put(p, 8, inside(p[7]))) == ALIAS
    assert accepted(call, put(p, 2, None), ctypes.byref(nd(gate=0)))
    assert call([None] * 10, ctypes.byref(nd(tokens=0))) == 0


def test_norm_bwd_arguments(lib):
    # r, y, z, w_post, alpha, w_pre, dr_out, dn, rstd_post, rstd_pre, dr, dy, dz, dw_post, dalpha, dw_pre, ws
    d, p = ctypes.byref(nd()), ptrs(17)
    call = lambda a, n=BIG: lib.ssd_block_norm_bwd(d, *a, n, None)
    for i in (0, 1, 2, 5, 6, 7, 8, 9, 10, 11, 12, 15, 16):
        assert call(put(p, i, None)) == NULL
    for i in range(17):
        assert call(put(p, i, inside(p[i], 4))) == ALIGN
    need = lib.ssd_block_norm_bwd_workspace_bytes(d)
    assert call(p, ctypes.c_size_t(need - 1)) == WORKSPACE
    assert call(put(p, 10, p[6])) == ALIAS
    assert call(put(p, 16, inside(p[11]))) == ALIAS
    assert accepted(call, put(put(p, 13, None), 14, None))
