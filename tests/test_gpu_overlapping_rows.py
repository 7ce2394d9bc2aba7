"""Results and queries in one buffer: side by side they are as with memory of their own, overlapping they are refused."""

import pytest
import torch

import kv8_plain
import latent_plain
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def sv():
    import speculative_decoding_verification_29_gb300 as m

    return m


def latent(heads):
    c = latent_plain.Cache([40, 300], [9, 9], 512, 64, 32, BF, seed=1).fill()
    args, cu = c.to("cuda"), c.cu.cuda()
    q = torch.randn(18, heads, 576, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    call = lambda x, **kw: sv().spec_latent_attention(x, *args, cu, max_tokens=9, value_dim=512, sm_scale=0.05, **kw)  # noqa: E731
    return q, 512, call


def kv8(heads):
    c = kv8_plain.Cache([40, 300], [9, 9], 2, 64, 16, seed=1).fill()
    args, cu = c.to("cuda"), c.cu.cuda()
    q = torch.randn(18, heads, 64, generator=torch.Generator().manual_seed(3)).to(BF).cuda()
    return q, 64, lambda x, **kw: sv().spec_kv8_attention(x, *args, cu, max_tokens=9, **kw)


@pytest.mark.parametrize("make,heads", [(latent, 4), (latent, 24), (kv8, 8)])
def test_side_by_side(make, heads):
    q, V, call = make(heads)
    T, H, W = q.shape
    want = call(q)["out"]
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    both = torch.zeros(T, H, W + V, dtype=BF, device="cuda")  # in every head
    tokens = torch.zeros(T, H * (W + V), dtype=BF, device="cuda")  # in every token
    for x, o in ((both[..., :W], both[..., W:]), (both[..., V:], both[..., :V]),
                 (tokens[:, : H * W].view(T, H, W), tokens[:, H * W:].view(T, H, V))):
        x.copy_(q)
        assert torch.equal(call(x, out=dict(out=o, row_status=status))["out"], want)


@pytest.mark.parametrize("make,heads", [(latent, 4), (latent, 24), (kv8, 8)])
def test_overlaps(make, heads):
    q, V, call = make(heads)
    T, H, W = q.shape
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    keep = q.clone()
    far = torch.zeros(2 * T * H * W, dtype=BF, device="cuda")
    x = far[: T * H * W].view(T, H, W)
    cases = [(q, q[..., W - V:]), (q, q[..., :V]), (q[1:], q[:-1, :, :V]), (x, far[T * H * W - 1:][: T * H * V].view(T, H, V))]
    if make is latent:  # any number of heads
        cases.append((q[:, 1:], q[:, :-1, :V]))
    for rows, o in cases:
        with pytest.raises(ValueError, match="overlap"):
            call(rows, out=dict(out=o, row_status=status))
    assert torch.equal(q, keep)


@pytest.mark.parametrize("kv", [False, True])
def test_rotated_queries(kv):
    """In place and side by side with the queries, but not over other rows of them."""
    freq = [0.5 ** i for i in range(16)]
    if kv:
        c = kv8_plain.Cache([40, 7], [3, 2], 2, 64, 16, seed=4).fill()
        args, cu, D = c.to("cuda"), c.cu.cuda(), 64
        x = torch.randn(5, 2, 64, generator=torch.Generator().manual_seed(5)).to(BF).cuda()
        call = lambda q, o: sv().spec_kv8_append(x, x, *args, cu, inv_freq=freq, q=q, q_out=o)["q_out"]  # noqa: E731
    else:
        c = latent_plain.Cache([40, 7], [3, 2], 128, 32, 16, BF, seed=4).fill()
        args, cu, D = c.to("cuda"), c.cu.cuda(), 32
        x = torch.randn(5, 160, generator=torch.Generator().manual_seed(5)).to(BF).cuda()
        call = lambda q, o: sv().spec_latent_append(x[:, :128], x[:, 128:], *args, cu, inv_freq=freq, q_rope=q, q_out=o)["q_out"]  # noqa: E731
    wide = torch.randn(6, 4, 2 * D, generator=torch.Generator().manual_seed(6)).to(BF).cuda()
    q = wide[:5, :, :D]
    want, keep = call(q, None).clone(), wide.clone()
    with pytest.raises(ValueError, match="overlap"):
        call(q, wide[1:, :, :D])
    with pytest.raises(ValueError, match="overlap"):
        call(q, wide[:5, :, D // 2: D // 2 + D])
    assert torch.equal(wide, keep)
    assert torch.equal(call(q, wide[:5, :, D:]), want)
    assert torch.equal(wide[:5, :, :D], keep[:5, :, :D])
    assert torch.equal(call(q, q), want)
