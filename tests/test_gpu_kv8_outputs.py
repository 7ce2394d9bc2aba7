"""Outputs and workspaces that a caller passes to the 8-bit paged cache's calls: what is refused, and that larger and strided
ones serve."""

import pytest
import torch

import kv8_plain as plain
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def sv():
    import speculative_decoding_verification_29_gb300 as m

    return m


def i32(n, device="cuda"):
    return torch.zeros(n, dtype=torch.int32, device=device)


def setup():
    c = plain.Cache([40, 7], [3, 2], 2, 64, 16, seed=1).fill()
    x = torch.randn(5, 2, 64, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    return c, c.to("cuda"), c.cu.cuda(), x


BAD = [lambda: i32(1), lambda: i32(2, "cpu"), lambda: i32(2).long(), lambda: i32(4)[::2], lambda: i32(1).expand(2)]


@pytest.mark.parametrize("bad", range(len(BAD)))
def test_statuses_and_lengths_are_refused(bad):
    c, args, cu, x = setup()
    before = [a.clone() for a in args]
    with pytest.raises(ValueError):
        sv().spec_kv8_append(x, x, *args, cu, out=dict(row_status=BAD[bad]()))
    with pytest.raises(ValueError):
        sv().spec_kv8_attention(x, *args, cu, max_tokens=3, out=dict(out=torch.empty_like(x), row_status=BAD[bad]()))
    for out in (dict(new_len=BAD[bad](), row_status=i32(2)), dict(new_len=i32(2), row_status=BAD[bad]())):
        with pytest.raises(ValueError):
            sv().spec_kv8_compact(*args, i32(2), out=out)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(args, before))


def test_rows_and_workspaces_are_refused():
    c, args, cu, x = setup()
    shared = torch.empty(1, 2, 64, dtype=BF, device="cuda").expand(5, 2, 64)
    with pytest.raises(ValueError):
        sv().spec_kv8_append(x, x, *args, cu, q=x, q_out=shared)
    for out in (shared, x):
        with pytest.raises(ValueError):
            sv().spec_kv8_attention(x, *args, cu, max_tokens=3, out=dict(out=out, row_status=i32(2)))
    n = sv().kv8_workspace_bytes(args[0], args[4], 2, 3, BF)
    for ws in (torch.empty(n, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(n),
               torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            sv().spec_kv8_attention(x, *args, cu, max_tokens=3, workspace=ws)


def test_larger_and_strided_outputs_serve():
    c, args, cu, x = setup()
    want = sv().spec_kv8_attention(x, *args, cu, max_tokens=3)["out"]
    status, out = i32(9) + 5, torch.zeros(2, 5, 100, dtype=BF, device="cuda").transpose(0, 1)[..., :64]
    n = sv().kv8_workspace_bytes(args[0], args[4], 2, 3, BF)
    r = sv().spec_kv8_attention(x, *args, cu, max_tokens=3, out=dict(out=out, row_status=status),
                                workspace=sv().alloc_workspace(n + 77, "cuda"))
    assert r["out"] is out and torch.equal(out, want) and status.tolist() == [0, 0] + [5] * 7
    lens, status = i32(3) + 5, i32(3) + 5
    sv().spec_kv8_compact(*args, i32(2) + 1, out=dict(new_len=lens, row_status=status))
    assert lens.tolist() == [42, 9, 5] and status.tolist() == [0, 0, 5]
    status = i32(3) + 5
    r = sv().spec_kv8_append(x, x, *args, cu, q=x, q_out=x, out=dict(row_status=status))
    assert status.tolist() == [0, 0, 5] and r["q_out"] is x
