"""Strided rows as the binding takes them (CPU only): heads have to lie side by side in a
row, and a view has to hold the rows that the call will use."""
import pytest
import torch

import gguf_block_quant_qmm_amd as q

CPU = -1  # get_device() of a host tensor: the checks themselves need no GPU


def rows(t, n, width, stride):
    return q._rows(CPU, t, n, width, stride, "X", torch.float32)


def test_heads_side_by_side_are_taken():
    N, H, D = 5, 4, 16
    qkv = torch.zeros(N, 3 * H * D)
    wide = 3 * H * D
    for part in (qkv, qkv[:, H * D:], qkv[:, 2 * H * D:], qkv.view(N, 3, H, D)[:, 1], qkv.view(N, 3 * H, D)[:, H:2 * H],
                 qkv.view(N, 3, H * D)[:, 2], qkv.view(-1)[H * D:], qkv.view(1, -1), qkv.view(N, 3, 1, H, D)[:, 1]):
        assert rows(part, N, H * D, wide) == part.data_ptr()
    assert rows(qkv[2:3, H * D:], 1, H * D, wide) == qkv.data_ptr() + 4 * (2 * wide + H * D)
    assert rows(qkv[1:], N - 1, H * D, wide) == qkv.data_ptr() + 4 * wide


@pytest.mark.parametrize("view", [
    lambda t: t.view(5, 4, 3, 16)[:, :, 0],             # q, k and v of a head side by side: heads 3 D apart
    lambda t: t.view(5, 4, 48)[:, :, :16],              # the same
    lambda t: t.view(5, 12, 16)[:, ::3],
    lambda t: t.view(5, 12, 16)[:, :4].transpose(1, 2),
    lambda t: t.view(5, 3, 4, 16)[:, 0].transpose(1, 2),
    lambda t: t[:, ::2],
])
def test_heads_apart_are_refused(view):
    t = view(torch.zeros(5, 3 * 4 * 16))
    with pytest.raises(ValueError):
        rows(t, 5, 4 * 16, 3 * 4 * 16)


@pytest.mark.parametrize("view,n", [
    (lambda t: t[:3], 5),               # fewer rows than the call uses, the storage has more
    (lambda t: t[:, :60], 5),           # narrower than the heads
    (lambda t: t.view(5, 3, 64)[:2, 1], 4),
    (lambda t: t[:1, :60], 1),
    (lambda t: t[1:], 5), (lambda t: t.view(-1)[64:], 6),
])
def test_views_that_do_not_hold_the_rows_are_refused(view, n):
    with pytest.raises(ValueError):
        rows(view(torch.zeros(5, 192)), n, 64, 192)


def test_other_strides_types_and_devices_are_refused():
    t = torch.zeros(5, 192)
    for bad, stride in ((t, 128), (t.double(), 192), (t.t(), 192)):
        with pytest.raises(ValueError):
            rows(bad, 5, 64, stride)
    with pytest.raises(ValueError, match="device"):
        q._rows(0, t, 5, 64, 192, "X", torch.float32)
