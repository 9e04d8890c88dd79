"""Overlaps that the 8-bit products and the token scoring refuse on the host: what
a kernel writes is counted to its last byte.  No call here is launched."""
import pytest

import attention_free_long_b200 as av

A = 0x100000  # 256-byte aligned addresses, never dereferenced


@pytest.mark.parametrize("dt,at", [(av.AVEY_F32, 44), (av.AVEY_BF16, 42), (av.AVEY_BF16, 46), (av.AVEY_BF16X2, 46)])
@pytest.mark.parametrize("rows", [1, 4])
def test_x_in_the_padding_of_the_last_rounded_row(rows, dt, at):
    # 42 columns and 6 zeros a row: x begins among the zeros of the last one
    x = A + (rows - 1) * 64 + at
    code = av.lib().avey_quantize_rows(x, dt, rows, 42, 64, 0, A, 64, A - 4096, None)
    assert code == 1 and "overlaps" in av.lib().avey_last_error_detail().decode()


O = 0x900000


@pytest.mark.parametrize("x,out,res,word", [
    # rows every 416 bytes: x takes 160 of them, out and residual 96 each
    (0, 160, None, "workspace"), (0, 320, None, "workspace"), (96, 0, None, "workspace"),
    (240, 0, 96, "workspace"), (0, 160, 256, "workspace"), (0, 160, 160, "workspace"),
    (416 * 3, 160, None, "workspace"), (160 - 416 * 30, 0, None, "workspace"),
    (0, 144, None, "out overlaps x"), (0, 336, None, "out overlaps x"), (80, 0, None, "out overlaps x"),
    (416 * 3 + 80, 0, None, "out overlaps x"), (0, 416 * 39 + 144, None, "out overlaps x"),
    (416 * 39 - 16, 416 * 78, None, "out overlaps x"), (0, 160, 240, "out overlaps the residual"),
    (416 * 80, 0, 4, "out overlaps the residual"), (416 * 80, 0, 416, "out overlaps the residual"),
])
def test_columns_of_one_buffer_are_taken(x, out, res, word):
    # without a workspace: refused for that where the overlap check lets the call pass
    p = av.LinearI8Params(40, 24, A, 48, A, None, 0)
    code = av.lib().avey_linear_i8(p, O + x, av.AVEY_F32, 104, None, 0, 40, None if res is None else O + res, 104,
                                   O + out, av.AVEY_F32, 104, None, 0, None)
    assert code == 1 and word in av.lib().avey_last_error_detail().decode()


def test_planes_of_a_pair_are_rows_too():
    # a bf16 pair's 40 + 40 rows of 80 of 160 bytes, an output in the other columns or across
    for out, word in ((O + 80, "workspace"), (O + 80 + 160 * 41, "workspace"), (O + 64 + 160 * 41, "out overlaps x"),
                      (O + 80 + 160 * 80, "workspace"), (O + 64 + 160 * 79, "out overlaps x"),
                      (O + 64 + 160 * 80, "workspace")):
        p = av.LinearI8Params(40, 20, A, 48, A, None, 0)
        code = av.lib().avey_linear_i8(p, O, av.AVEY_BF16X2, 80, None, 0, 40, None, 0, out, av.AVEY_F32, 40, None, 0,
                                       None)
        assert code == 1 and word in av.lib().avey_last_error_detail().decode(), hex(out - O)
