"""Refusals of the serving operators at the limits of their arguments, on the host."""
import pytest

from test_serving_host import INVALID, P, append, attn, cache, lib, prompt  # noqa: F401 (lib: a fixture)
from attention_jvp_attn_b200 import _abi


def test_scales_beyond_32_bits_in_powers_of_two_are_refused(lib):
    """The softmax works in powers of two: scale log2 e has to be finite, or 0 times it is NaN."""
    for scale in (2.4e38, 3.4e38):
        assert attn(lib, scale=scale, B=0) == INVALID and prompt(lib, scale=scale, B=0) == INVALID
    for scale in (2.3e38, 1e-40):
        assert attn(lib, scale=scale, B=0) == _abi.OK and prompt(lib, scale=scale, B=0) == _abi.OK
