"""What the 8-bit paged cache's Python calls refuse to write to: outputs and workspaces that a caller passes in. The checks run
here on tensors of the host, whose device stands for the cache's."""

import pytest
import torch

HOST, META = torch.device("cpu"), torch.device("meta")


def api():
    from speculative_decoding_verification_29_gb300 import api as m

    return m


def test_statuses_and_lengths():
    i32 = torch.int32
    api()._int32(torch.zeros(4, dtype=i32), "row_status", HOST, 4)
    api()._int32(torch.zeros(9, dtype=i32), "row_status", HOST, 4)
    for bad in (torch.zeros(3, dtype=i32), torch.zeros(0, dtype=i32), torch.zeros(4), torch.zeros(4, dtype=torch.int64),
                torch.zeros(8, dtype=i32)[::2], torch.zeros(1, dtype=i32).expand(4), torch.zeros(4, dtype=i32, device=META)):
        with pytest.raises(ValueError):
            api()._int32(bad, "row_status", HOST, 4)


def test_rows():
    x = torch.zeros(3, 4, 64, dtype=torch.float16)
    assert api()._kv8_rows(x, "out", 64, HOST, True) == (256, 64)
    assert api()._kv8_rows(x.transpose(0, 1), "out", 64, HOST, True) == (64, 256)
    assert api()._kv8_rows(x[:1].expand(1, 4, 64), "out", 64, HOST, True) == (256, 64)
    one = torch.zeros(1, 1, 64, dtype=torch.float16)
    for shared in (one.expand(3, 1, 64), one.expand(1, 4, 64), x[:1].expand(3, 4, 64),
                   torch.zeros(400, dtype=torch.float16).as_strided((3, 2, 64), (128, 32, 1))):
        api()._kv8_rows(shared, "q", 64, HOST)  # may be read
        with pytest.raises(ValueError):
            api()._kv8_rows(shared, "out", 64, HOST, True)


def test_workspace():
    api()._kv8_workspace(torch.zeros(64, dtype=torch.uint8), HOST)
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(64), torch.zeros(128, dtype=torch.uint8)[::2],
                torch.zeros(64, dtype=torch.uint8, device=META)):
        with pytest.raises(ValueError):
            api()._kv8_workspace(bad, HOST)
