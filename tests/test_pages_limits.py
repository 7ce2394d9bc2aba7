"""The limits of the pages' call in C. The pointers here are numbers; the module is left out where a GPU could be reached with
them."""

import pytest
import torch

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers used here are no device memory")

ARG, CUDA, LIMIT = -1, -3, -5
P = 0x7F0000000000  # stands for a device pointer


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_29_gb300 import _lib, build

    build.build()
    return _lib.load()


def pages(lib, new=P, source=None, B=4, M=20, nb=100):
    return lib.spec_pages_update(P, new, P + (1 << 32), None, source, None, P + (2 << 32), B, M, nb, 32, None, 0, P + (3 << 32),
                                 P + (4 << 32), P + (5 << 32), 1 << 40, None)


def test_pools_of_very_many_blocks(lib):
    """The search for free blocks counts them in 32 bits, 4096 at a time."""
    assert pages(lib, nb=1 << 30) == CUDA  # without a GPU sound arguments get as far as the launch, which fails
    assert lib.spec_pages_workspace_bytes(4, 20, 1 << 30) > 3 << 32
    for nb in ((1 << 30) + 1, (1 << 31) - 4096, (1 << 31) - 1):
        assert pages(lib, nb=nb) == LIMIT and lib.spec_pages_workspace_bytes(4, 20, nb) == 0


def test_new_rows_over_old_ones(lib):
    """The rows after the call lie where the old ones do, or in memory of their own: rows of other sequences are read."""
    B, M = 4, 20
    assert pages(lib) == CUDA and pages(lib, source=P + (6 << 32)) == ARG
    for source in (None, P + (6 << 32)):
        for off in (4, -4, 4 * M, -4 * M, 4 * (B * M - 1), 4 - 4 * B * M):
            assert pages(lib, new=P + off, source=source) == ARG
        for off in (4 * B * M, -4 * B * M):
            assert pages(lib, new=P + off, source=source) == CUDA
