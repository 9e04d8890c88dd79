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
