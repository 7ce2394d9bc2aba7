"""Calls on a stream that is not the current one: what they allocate is theirs alone, whatever is still queued on the current
stream, and stays the caller's for as long as the current stream reads it."""

import pytest
import torch

import kv8_plain as plain
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
WAIT = 200_000_000  # clocks that the current stream is kept busy for, some 0.1 s


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def sv():
    import speculative_decoding_verification_29_gb300 as m

    return m


def kv8_calls():
    c = plain.Cache([600, 40, 7], [9, 3, 2], 2, 128, 32, seed=1).fill()
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(14, 2, 128, generator=g).to(BF).cuda() for _ in range(2))
    q = torch.randn(14, 8, 128, generator=g).to(BF).cuda()
    args, cu, acc = c.to("cuda"), c.cu.cuda(), torch.tensor([1, 0, -1], dtype=torch.int32, device="cuda")
    return [lambda **kw: sv().spec_kv8_append(k, v, *args, cu, inv_freq=[0.5] * 8, q=q, **kw),
            lambda **kw: sv().spec_kv8_attention(q, *args, cu, max_tokens=9, **kw),
            lambda **kw: sv().spec_kv8_compact(*args, acc, **kw)]


def check_call(call):
    want = {k: v.clone() for k, v in call().items() if isinstance(v, torch.Tensor)}
    sizes = [v.numel() * v.element_size() for v in want.values()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in (streams[0], streams[1].cuda_stream):  # a stream, and its handle
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        # blocks of the outputs' sizes, freed while the current stream has still to write them
        junk = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
        torch.cuda._sleep(WAIT)
        for j in junk:
            j.fill_(0x55)
        del j, junk
        got = call(stream=s)
        torch.cuda.synchronize()
        for k, v in want.items():
            assert torch.equal(got[k], v), k
        # outputs dropped while the current stream has still to read them
        torch.cuda._sleep(WAIT)
        kept = {k: got[k].clone() for k in want}
        del got
        with torch.cuda.stream(streams[0] if s is streams[0] else torch.cuda.ExternalStream(s)):
            junk = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
        torch.cuda.synchronize()
        for k, v in want.items():
            assert torch.equal(kept[k], v), k


@pytest.mark.parametrize("which", range(3))
def test_kv8_calls(which):
    check_call(kv8_calls()[which])
