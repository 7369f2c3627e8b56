"""Refusals of the calls around a decoding step that test_step_host.py leaves out.  No test here launches a kernel."""
import pytest

import mixed_bitrate_quantized_amd as exq
from tests.test_step_host import B, U, at, expect, sample_args


@pytest.mark.parametrize("rows", [1 << 22, (1 << 31) - 1])
@pytest.mark.parametrize("bits", [16, 32])
def test_sample_rejects_rows_beyond_a_launch(rows, bits):
    """A workgroup of 1024 threads to a row, and 2^32 threads are more than a launch has."""
    apart = B * B.bit_length() * 16
    expect(U, exq.exq_sample, *sample_args(rows=rows, bits=bits, vocab=8, stride=8, logits=at(0), u=apart, tokens=2 * apart, logs=3 * apart))
