"""Where linear attention cuts the sequence axis: the rule's choice, read from the workspace sizes, against times that were
measured (B200, us, calls replayed one behind the other) with every cut forced."""
import ctypes

import pytest

from selective_state_space_43_b200 import build as build_mod
from selective_state_space_43_b200 import ops

BF16, F32 = ops.SSD_BF16, ops.SSD_F32
# dtype, backward, sequences, rows of all, packed, heads, kv heads, key width, value width, {rows of a segment (0: whole): us}
MEASURED = [
    (F32, False, 15, 4636, True, 16, 4, 64, 96, {0: 308, 32: 307, 64: 264, 128: 253, 256: 268, 512: 321, 1024: 454}),
    (F32, True, 4, 4000, False, 16, 16, 128, 64, {0: 736, 32: 733, 64: 618, 128: 598, 256: 575, 512: 705}),
    (F32, True, 1, 11511, True, 16, 16, 128, 64,
     {0: 8281, 32: 2080, 64: 1720, 128: 1540, 256: 1509, 512: 1810, 1024: 2138, 2048: 2714, 4096: 4707}),
    (F32, True, 2, 7780, False, 16, 4, 128, 64,
     {0: 2839, 32: 1414, 64: 1174, 128: 1085, 256: 1124, 512: 1110, 1024: 1378, 2048: 2366}),
    (F32, False, 8, 2328, True, 32, 32, 32, 96, {0: 150, 32: 210, 64: 186, 128: 186, 256: 203, 512: 292}),
    (F32, False, 1, 22511, False, 8, 2, 32, 64,
     {0: 2977, 32: 321, 64: 254, 128: 221, 256: 227, 512: 287, 1024: 337, 2048: 530, 4096: 1009}),
    (F32, True, 1, 100, False, 4, 4, 32, 32, {0: 48, 32: 31, 64: 48}),
    (F32, False, 1, 256, False, 4, 4, 32, 64, {0: 33, 32: 17, 64: 23, 128: 36}),
    (F32, False, 2, 4096, False, 8, 8, 128, 128, {0: 543, 32: 267, 64: 216, 128: 194, 256: 177, 512: 218, 1024: 410}),
    (F32, False, 4, 4000, False, 32, 32, 128, 128, {0: 446, 32: 1103, 64: 849, 128: 719, 256: 705, 512: 726}),
    (F32, False, 8, 19976, False, 16, 16, 32, 96,
     {0: 541, 32: 888, 64: 777, 128: 739, 256: 724, 512: 805, 1024: 808, 2048: 1087}),
    (F32, False, 16, 4800, False, 8, 8, 96, 64, {0: 74, 32: 136, 64: 117, 128: 121, 256: 158}),
    (BF16, False, 12, 9000, True, 10, 10, 64, 64, {0: 37, 256: 54, 512: 51, 1024: 54}),
    (BF16, False, 1, 8192, False, 40, 40, 64, 64, {0: 111, 256: 109, 512: 94, 1024: 91, 2048: 105, 4096: 107}),
    (BF16, True, 15, 7163, True, 1, 1, 128, 128, {0: 31, 256: 42, 512: 38, 1024: 44}),
    (BF16, False, 1, 8191, False, 16, 16, 128, 128, {0: 120, 256: 111, 512: 90, 1024: 78, 2048: 72, 4096: 113}),
    (BF16, False, 4, 32768, False, 64, 64, 128, 64, {0: 289, 256: 884, 512: 625, 1024: 500, 2048: 459, 4096: 474}),
    (BF16, False, 24, 16384, True, 40, 8, 64, 64, {0: 104, 256: 285, 512: 226, 1024: 207, 2048: 195}),
    (BF16, True, 7, 3001, True, 16, 4, 64, 128, {0: 68, 256: 119, 512: 111, 1024: 109}),
]


def chosen(dtype, backward, n, rows, packed, H, Hk, dk, dv):
    """Rows of a segment as the workspace's size tells them (0: whole sequences)."""
    L = build_mod.build() and ops.lib()
    dims = ops.SsdLinearAttnDims(n, rows if packed else rows // n, H, Hk, dk, dv)
    if backward:
        size = L.ssd_linear_attn_backward_workspace_bytes(ctypes.byref(dims), dtype, packed)
        if H != Hk:
            size -= rows * H * (dk + dv) * 4  # the shared heads' gradients
        size //= 2  # two scans' states
    else:
        size = L.ssd_linear_attn_prefill_workspace_bytes(ctypes.byref(dims), dtype, packed)
    slots = size // (H * dk * dv * 4)
    if slots == 0:
        return 0
    for m in (32 << i for i in range(16)):
        if slots == (rows // m + n if packed else n * -(-(rows // n) // m)):
            return m
    raise AssertionError(f"{slots} segments")


@pytest.mark.parametrize("case", MEASURED, ids=lambda c: "-".join(str(int(x)) for x in c[:9]))
def test_the_cut_is_within_a_tenth_of_the_fastest(case):
    times = case[9]
    assert times[chosen(*case[:9])] <= 1.1 * min(times.values())
