"""Compaction whose outputs overlap its lengths without being them: refused on the host. The pointers here are numbers; the
module is left out where a GPU could be reached with them."""

import ctypes

import pytest
import torch

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers used here are no device memory")

ARG, CUDA = -1, -3
P, B = 0x7F0000000000, 4  # stands for a device pointer; sequences
LEN, ACC, OUT, STATUS = P + (1 << 32), P + (2 << 32), P + (3 << 32), P + (4 << 32)


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_29_gb300 import _lib, build

    build.build()
    return _lib.load()


def latent(lib, new_len=OUT, status=STATUS):
    from speculative_decoding_verification_29_gb300 import _lib

    c = _lib.LatentCache(P, P + (5 << 32), LEN, B, 100, 20, 32, 512, 64, 1, 32 * 1152, 1152)
    return lib.spec_latent_compact(ctypes.byref(c), 32, 1 << 24, P, 8, ACC, new_len, status, None)


def kv8(lib, new_len=OUT, status=STATUS):
    from speculative_decoding_verification_29_gb300 import _lib

    c = _lib.Kv8Cache(P, P, P, P, P + (5 << 32), LEN, B, 100, 20, 32, 8, 128, 8 * 32 * 128, 32 * 128, 128)
    return lib.spec_kv8_compact(ctypes.byref(c), 32, 1 << 24, 1 << 16, P, 8, ACC, new_len, status, None)


def kv(lib, new_len=OUT, status=STATUS):
    return lib.spec_kv_compact(P, 2, 64, B, 100, 1024, B * 102400, 102400, 1024, LEN, P, 8, ACC, new_len, status, None)


CALLS = [latent, kv8, kv]


@pytest.mark.parametrize("call", CALLS)
def test_overlaps(lib, call):
    assert call(lib) == CUDA  # without a GPU sound arguments get as far as the launch, which fails
    for at in (LEN, ACC):
        assert call(lib, new_len=at) == CUDA and call(lib, status=at) == CUDA  # in place
        for off in (4, -4, 4 * B - 4, 4 - 4 * B):
            assert call(lib, new_len=at + off) == ARG and call(lib, status=at + off) == ARG
        assert call(lib, new_len=at + 4 * B) == CUDA and call(lib, status=at - 4 * B) == CUDA
