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


@pytest.mark.parametrize("c", [
    cache(scale=(1, 1)),                                  # scales of (page 1, head 0) and (page 0, head 1)
    cache(scale=(4, 8)), cache(strides=(4096, 4096, 64), scale=(2, 1)),
    cache(strides=(64, 64 * 64 * 9, 64), scale=(2, 1)),   # pages where tokens are
    cache(strides=(8192, 64, 64), scale=(2, 1)),          # heads where tokens are
    cache(strides=(8192, 64, 112), scale=(2, 1)),
    cache(v=P[2], scale=(2, 1)), cache(vs=P[4], scale=(2, 1))])
def test_append_to_a_cache_that_overlaps_itself_is_refused(lib, c):
    assert append(lib, c=c) == INVALID


@pytest.mark.parametrize("kw", [
    dict(scale=(2, 1)), dict(scale=(1, 9)), dict(strides=(8192, 64, 128), scale=(2, 1)),   # heads inside tokens
    dict(strides=(4096, 9 * 4096, 64), scale=(2, 1)),                                    # pages inside heads
    dict(strides=(128, 64, 9 * 128), scale=(4, 2)),                                      # pages inside tokens
    dict(pages=1, strides=(16, 4096, 64), scale=(0, 1))])                                # a stride that no page uses
def test_append_takes_any_order_of_pages_heads_and_tokens(lib, kw):
    """Accepted by every check: what is left is that there is no GPU, or nothing to write to."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the call would be launched")
    assert append(lib, c=cache(**kw)) in (_abi.ERR_NO_DEVICE, _abi.ERR_CUDA)
