"""The update's workspace holds its planes from the first 32-byte boundary on
(their rows move 32 bytes at a time), wherever the 16-byte aligned scratch
begins: its size, asked on the host."""

import ctypes

import pytest


@pytest.mark.parametrize("n,rows,cols", [(1, 200, 300), (2, 64, 192), (22, 2048, 2048), (3, 771, 1003), (1, 1, 700)])
@pytest.mark.parametrize("yt", [0, 1])
def test_room_for_the_way_to_a_32_byte_boundary(n, rows, cols, yt):
    from reduction_groups_gb300 import _native as N
    from reduction_groups_gb300 import build as BD

    BD.build()
    v = ctypes.c_uint64(0)
    assert N.lib().psk_orthogonalize_workspace(n, rows, cols, yt, ctypes.byref(v)) == 0
    assert v.value % 32 == 16       # whole 256-byte pieces, and the 16 bytes to the boundary
