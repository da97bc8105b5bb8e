"""Rows that share memory are refused by the binding, before any pointer reaches
the library: a tensor expanded over its rows has a row stride of 0, which the
library reads as contiguous rows."""
import pytest
import torch

import state_space_sequence_chunk_gb300 as ssd


class Stand:
    """A host tensor that passes for one on the GPU: only its shape and strides are
    looked at here."""

    def __init__(self, t):
        self.t = t

    is_cuda = True

    def __getattr__(self, name):
        return getattr(self.t, name)


T, G, H, K, V, D = 6, 2, 4, 32, 16, 64
ONE = Stand(torch.zeros(H))


def dims(q=None, k=None, v=None):
    rows = lambda *s: Stand(torch.zeros(*s))
    return ssd._linattn_dims(q or rows(T, G, K), k or rows(T, G, K), v or rows(T, H, V), ONE, 1, 0)


def norms(y=None, z=None):
    rows = lambda: Stand(torch.zeros(T, D))
    w = Stand(torch.zeros(D))
    return ssd._norm_dims(rows(), y or rows(), z or rows(), w, w, w, "silu", 4, 1e-5)


def expanded(*s):
    return Stand(torch.zeros(1, *s).expand(T, *s))


def overlapping(*s):
    inner = torch.Size(s).numel()
    return Stand(torch.zeros(T * inner).as_strided((T, *s), (inner - 8, *torch.zeros(*s).stride())))


@pytest.mark.parametrize("made", [expanded, overlapping])
def test_rows_that_share_memory_are_refused(made):
    for kw in (dict(q=made(G, K)), dict(k=made(G, K)), dict(v=made(H, V))):
        with pytest.raises(ValueError):
            dims(**kw)
    for kw in (dict(y=made(D)), dict(z=made(D))):
        with pytest.raises(ValueError):
            norms(**kw)


def test_rows_that_do_not_share_memory_pass():
    d = dims()[0]
    assert (d.q_stride, d.k_stride, d.v_stride) == (G * K, G * K, H * V)
    d = dims(q=Stand(torch.zeros(T, 3 * G * K)[:, G * K:2 * G * K].view(T, G, K)))[0]
    assert d.q_stride == 3 * G * K
    d = norms(z=Stand(torch.zeros(T, 2 * D)[:, D:]))[0]
    assert d.z_stride == 2 * D
    # one row has no next one: its stride does not count
    one = Stand(torch.zeros(1, 1, K).expand(1, G, K).contiguous().as_strided((1, G, K), (0, K, 1)))
    assert ssd._rows(one, G * K)[1] == G * K
