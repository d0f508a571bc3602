"""How many blocks of rows the layer norm's gradient runs (CPU: 256 compute units are assumed without a GPU).  One block to a run is
for the sums of the columns, whose second launch it saves; without sums there is none to save, and the card is filled."""
import ctypes

import pytest

from bit_diffusion_model_amd import svdq


class Plan(ctypes.Structure):
    _fields_ = [("runs", ctypes.c_int64), ("len", ctypes.c_int64), ("per", ctypes.c_int64), ("parts", ctypes.c_uint32),
                ("cols", ctypes.c_uint32), ("w", ctypes.c_int), ("waves", ctypes.c_int), ("cw", ctypes.c_int),
                ("bytes", ctypes.c_size_t)]


def plan(B, S, C, each, sums, apart):
    f = svdq.lib()._ZN4svdq20plan_layer_norm_gradEllibbb  # svdq::plan_layer_norm_grad
    f.restype = Plan
    f.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_bool, ctypes.c_bool, ctypes.c_bool]
    return f(B, S, C, each, sums, apart)


def rows_at_a_time(C):
    """Rows that a block of 16 waves has at a time: 8, 16, 32 lanes a row, or waves of 512 values (1024 past 8192)."""
    if C <= 256:
        return 16 * 64 // (8 if C <= 64 else 16 if C <= 128 else 32)
    per = 512 if C <= 8192 else 1024
    return 16 // -(-C // per)


@pytest.mark.parametrize("B,S,C,each", [(1, 512, 64, False), (1, 300, 33, False), (1, 256, 128, False), (1, 64, 400, False),
                                        (2, 500, 64, True), (3, 100, 100, False), (1, 4, 5000, False), (1, 2000, 320, False)])
def test_rows_without_sums_fill_the_card(B, S, C, each):
    p, rows = plan(B, S, C, each, False, True), rows_at_a_time(C)
    run = S if each else B * S
    runs = B if each else 1
    most = -(-256 // runs)
    turns = -(-run // (rows * most))
    assert (p.runs, p.len, p.bytes, p.cw, p.cols) == (runs, run, 0, 0, 0)
    assert p.parts == -(-run // (turns * rows))


@pytest.mark.parametrize("S,C", [(512, 64), (256, 128), (64, 400), (4, 5000)])
def test_sums_in_one_launch_as_before(S, C):
    """In place (no blocks of columns) up to four turns of rows are one block's, and the next row is another's."""
    rows = rows_at_a_time(C)
    assert S <= 4 * rows and plan(1, S, C, False, True, False).parts == 1
    assert plan(1, 4 * rows, C, False, True, False).parts == 1 and plan(1, 4 * rows + 1, C, False, True, False).parts > 1
