"""Calls on a stream that is not the current one: what they allocate is theirs alone, whatever is still queued on the current
stream, and stays the caller's for as long as the current stream reads it."""

import pytest
import torch

import gen
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


def bits(t):
    return t.contiguous().view(torch.uint8)


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
            assert torch.equal(bits(got[k]), bits(v)), k
        # outputs dropped while the current stream has still to read them
        torch.cuda._sleep(WAIT)
        kept = {k: got[k].clone() for k in want}
        del got
        with torch.cuda.stream(streams[0] if s is streams[0] else torch.cuda.ExternalStream(s)):
            junk = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
        torch.cuda.synchronize()
        for k, v in want.items():
            assert torch.equal(bits(kept[k]), bits(v)), k


@pytest.mark.parametrize("which", range(3))
def test_kv8_calls(which):
    check_call(kv8_calls()[which])


def verification_calls():
    def dev(*t):
        return [x.cuda() for x in t]

    c, c0 = gen.chain_tiny(0), gen.chain_tiny(1, T=0.0)
    chain = dev(c.Lp, c.Lq, c.x.long(), c.ua.double(), c.ur)  # some inputs are converted on the way
    tb = gen.tree_batch(4, n_per_tree=6, V=500, dtype=torch.float32, seed=0, max_depth=4)
    tree = dev(tb.Lt, tb.tok.long(), tb.R)
    conf, draft = tb.conf.cuda(), gen.tree_draft_logits(tb, 0).cuda()
    Ld, logc = dev(*gen.expand_frontier(2, 3, 5000, torch.bfloat16, seed=1))
    kv = torch.randn(2, 3, 20, 64, generator=torch.Generator().manual_seed(3)).cuda()
    base, acc = dev(torch.tensor([0, 5, 9]), torch.tensor([3, -1, 0]))
    R, mask, pos = gen.tree_from_parents([-1, 0, 0, 1])
    one = [torch.tensor([[7, 8, 9, 10]], dtype=torch.int32), torch.as_tensor(mask)[None], torch.as_tensor(R)[None],
           torch.as_tensor(pos)[None]]
    two = [torch.tensor([[7, 8, 11, 12]], dtype=torch.int32), *one[1:]]
    merge = dev(*one, *two)
    return dict(
        chain=lambda **kw: sv().spec_verify_chain(*chain, c.T, **kw),
        greedy=lambda **kw: sv().spec_verify_chain_greedy(c0.Lp.cuda(), c0.x.long().cuda(), **kw),
        warped=lambda **kw: sv().spec_verify_chain_warped(*chain, c.T, top_k=8, top_p=0.9, **kw),
        tree=lambda **kw: sv().spec_verify_tree_greedy(*tree, tb.n1, **kw),
        confidence=lambda **kw: sv().spec_tree_confidence(conf, tb.n1, **kw),
        entropy=lambda **kw: sv().spec_tree_entropy(draft, tb.n1, 1.0, **kw),
        expand=lambda **kw: sv().spec_tree_expand(Ld, logc, 5, **kw),
        merge=lambda **kw: sv().spec_merge_trees(*merge, **kw),
        compact=lambda **kw: sv().spec_kv_compact(kv, base, acc, **kw),
    )


NAMES = ["chain", "greedy", "warped", "tree", "confidence", "entropy", "expand", "merge", "compact"]


@pytest.mark.parametrize("name", NAMES)
def test_verification_calls(name):
    check_call(verification_calls()[name])


@pytest.mark.parametrize("name", NAMES)
def test_another_device_is_refused(name, monkeypatch):
    """Tensors on a device that is not the current one (one GPU: the current device is faked)."""
    call = verification_calls()[name]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError):
        call()
