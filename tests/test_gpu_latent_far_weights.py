"""fp16 attention over the paged latent cache where one entry leads and very many lie far below it: alone they weigh next to
nothing, together they count."""

import pytest
import torch

import latent_plain as plain
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
HF = torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("heads", [3, 81])  # 16 rows an item, 128
def test_many_far_below_one(heads):
    """304 sequences over the same blocks, so that every thread block has whole ones and no share has a reference of its own.

    Tolerance: that of latent_plain.attention, but for two terms. Weights in fp16's subnormals are off by 2^-25 where the row's
    largest is at least 2^7: (1 + sum |v - o|) 2^-32. And the second product's sums: a step of the tensor cores adds 16 products
    to the running sum, all cut towards zero to multiples of 2^-25 of the largest one's power of two (131,072 products of 2^-25
    of the sum arrive whole, of 2^-26 not at all), and keeps 24 bits. The running sum is at most S = sum p |v| of the weights'
    sum, so a step is off by at most 16 2^-25 S + 2^-23 S, and N / 16 steps by N (2^-25 + 2^-27) S: 0.0049 S here. Where the
    weights were lost, heads of the first kind were off by their whole mass, 0.0034, times what the leader's vector differs by,
    2: more than all terms together."""
    import speculative_decoding_verification_29_gb300 as sv

    N, C, R, bs, B = 131072, 128, 16, 128, 304
    g = torch.Generator().manual_seed(1)
    pool = torch.zeros(N, C + R)
    pool[:, :C] = 1 + 0.1 * torch.randn(N, C, generator=g)
    pool[100] = -pool[100]  # the leader's
    pool[:, C] = -1.0
    pool[100, C] = 0.0
    pool = pool.to(HF)
    below = torch.tensor([25.2, 20.3, 16.4]).repeat(heads // 3) * 0.6931471805599453  # of the three kinds of heads
    q = torch.zeros(B, heads, C + R)
    q[:, :, C] = below
    q = q.to(HF)
    table = torch.arange(N // bs, dtype=torch.int32).repeat(B, 1)
    r = sv.spec_latent_attention(q.cuda(), pool.view(-1, bs, C + R).cuda(), table.cuda(),
                                 torch.full((B,), N - 1, dtype=torch.int32, device="cuda"),
                                 torch.arange(B + 1, dtype=torch.int32, device="cuda"), max_tokens=1, value_dim=C, sm_scale=1.0)
    assert not bool(r["row_status"].any())
    u = plain.half_step(HF)
    e, v = pool.double(), pool[:, :C].double()
    for h in range(3):
        x = q[0, h].double()
        p = torch.softmax(e @ x, 0)
        o = p @ v
        apart, big = p @ (v - o).abs(), p @ v.abs()
        s = (e.abs() @ x.abs()).max() * (C + R + 4) * 2.0 ** -23 + 2.0 ** -22
        t = (u / (1 - u) + 2 * s) * apart + N * (2.0 ** -25 + 2.0 ** -27) * big + 2.0 ** -32 * (1 + (v - o).abs().sum(0))
        t = t + u * (o.abs() + t)
        got = r["out"][:, h::3].double().cpu()
        d = (got - o).abs()
        assert bool((d <= t).all()), (h, float(d.max()), float((d / t).max()))
