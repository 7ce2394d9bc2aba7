"""What the Python calls of the paged latent cache and of the pages refuse before anything is launched."""

import pytest
import torch

from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32
BAD = (ValueError, RuntimeError)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def sv():
    import speculative_decoding_verification_29_gb300 as m

    return m


def z(*shape, dtype=BF, device="cuda"):
    return torch.zeros(*shape, dtype=dtype, device=device)


def cache(**kw):
    a = dict(cache=z(6, 32, 576), block_table=z(2, 3, dtype=I32), cache_len=z(2, dtype=I32))
    a.update(kw)
    return tuple(a.values())


def cu():
    return torch.tensor([0, 1, 3], dtype=I32, device="cuda")


FREQ = [1.0] * 32


def everywhere(c, error=ValueError):
    x = z(3, 576)
    with pytest.raises(error):
        sv().spec_latent_append(x[:, :512], x[:, 512:], *c, cu(), inv_freq=FREQ)
    with pytest.raises(error):
        sv().spec_latent_attention(z(3, 4, 576), *c, cu(), max_tokens=2, value_dim=512, sm_scale=0.1)
    with pytest.raises(error):
        sv().spec_latent_compact(*c, z(2, dtype=I32))


def test_caches(monkeypatch):
    everywhere(cache(cache=z(6, 576)))
    everywhere(cache(cache=z(6, 32, 576, dtype=torch.float32)), TypeError)
    everywhere(cache(cache=z(6, 32, 576, device="cpu")))
    everywhere(cache(cache=z(6, 32, 1152)[..., ::2]))
    everywhere(cache(cache=z(6, 32, 580)[..., :576]), BAD)  # slots of 1160 bytes
    everywhere(cache(cache=z(6, 24, 576)), BAD)
    everywhere(cache(block_table=z(3, 3, dtype=I32)))
    everywhere(cache(block_table=z(2, 3, dtype=torch.int64)))
    everywhere(cache(block_table=z(2, 6, dtype=I32)[:, ::2]))
    everywhere(cache(cache_len=z(2, dtype=I32, device="cpu")))
    everywhere(cache(cache_len=z(2, 1, dtype=I32)))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)  # one GPU: another current device is faked
    everywhere(cache())


def test_append_arguments():
    x, q = z(3, 576), z(3, 4, 64)

    def refuses(error, l=x[:, :512], r=x[:, 512:], c=None, cu_tokens=None, **kw):  # noqa: E741
        kw.setdefault("inv_freq", FREQ)
        with pytest.raises(error):
            sv().spec_latent_append(l, r, *(c or cache()), cu() if cu_tokens is None else cu_tokens, **kw)

    refuses(ValueError, l=z(3, 576))
    refuses(ValueError, l=z(3, 1, 512))
    refuses(ValueError, r=z(3, 32))
    refuses(ValueError, r=z(2, 64))
    refuses(TypeError, r=z(3, 64, dtype=torch.float16))
    refuses(TypeError, l=x[:, :512].half(), r=x[:, 512:].half())
    refuses(ValueError, l=z(3, 1024)[:, ::2])
    refuses(ValueError, r=z(3, 64, device="cpu"))
    refuses(ValueError, inv_freq=[1.0] * 16)
    refuses(BAD, inv_freq=[float("nan")] * 32)
    refuses(ValueError, cu_tokens=cu()[:2])
    refuses(ValueError, cu_tokens=cu().long())
    refuses(ValueError, positions=cu()[:2])
    refuses(ValueError, norm_weight=z(64))
    refuses(TypeError, norm_weight=z(512, dtype=torch.float16))
    refuses(BAD, norm_weight=z(512), eps=-1.0)
    refuses(ValueError, q_rope=z(2, 4, 64))
    refuses(ValueError, q_rope=z(3, 4, 32))
    refuses(ValueError, q_rope=q.half())
    refuses(ValueError, q_rope=q, q_out=q[:, :2])
    refuses(ValueError, q_rope=q, q_out=q[:1].expand(3, 4, 64))
    refuses(ValueError, out=dict(row_status=z(1, dtype=I32)))


def test_attention_arguments():
    q, status = z(3, 4, 576), z(2, dtype=I32)

    def refuses(error, q=q, c=None, cu_tokens=None, **kw):
        args = dict(max_tokens=2, value_dim=512, sm_scale=0.1)
        args.update(kw)
        with pytest.raises(error):
            sv().spec_latent_attention(q, *(c or cache()), cu() if cu_tokens is None else cu_tokens, **args)

    refuses(TypeError, q=q.half())
    refuses(ValueError, q=q[..., :512])
    refuses(ValueError, value_dim=576)
    refuses(BAD, value_dim=500)
    refuses(ValueError, value_dim=0)
    refuses(ValueError, cu_tokens=cu()[:2])
    refuses(ValueError, tree_mask=z(2, 3, 3, dtype=torch.uint8))
    refuses(ValueError, tree_mask=z(2, 2, 2))
    refuses(ValueError, out=dict(out=z(3, 4, 576), row_status=status))
    refuses(ValueError, out=dict(out=z(3, 4, 512, dtype=torch.float16), row_status=status))
    refuses(ValueError, out=dict(out=z(1, 1, 512).expand(3, 4, 512), row_status=status))
    refuses(ValueError, out=dict(out=z(3, 4, 512), row_status=status[:1]))
    refuses(ValueError, out=dict(out=q.view(-1)[: 3 * 4 * 512].view(3, 4, 512), row_status=status))
    refuses(BAD, max_tokens=0)
    refuses(BAD, sm_scale=float("nan"))
    refuses(BAD, workspace=z(256, dtype=torch.uint8))
    refuses(BAD, q=z(3, 1025, 576))


def test_compact_arguments():
    i = z(2, dtype=I32)
    for kw in (dict(accept_len=i[:1]), dict(accept_len=i.long()), dict(path=i), dict(path=z(3, 4, dtype=I32)),
               dict(path=z(2, 257, dtype=I32)), dict(out=dict(new_len=i[:1], row_status=i))):
        args = dict(accept_len=i)
        args.update(kw)
        with pytest.raises(BAD):
            sv().spec_latent_compact(*cache(), **args)


def test_pages_arguments(monkeypatch):
    t, n, r = z(2, 3, dtype=I32), z(2, dtype=I32), z(6, dtype=I32)

    def refuses(error, t=t, n=n, r=r, pools=(), **kw):
        kw.setdefault("block", 16)
        with pytest.raises(error):
            sv().spec_pages_update(t, n, r, pools, **kw)

    refuses(ValueError, t=t.long())
    refuses(ValueError, t=t.cpu())
    refuses(ValueError, n=n[:1])
    refuses(ValueError, r=r.long())
    refuses(ValueError, r=r[None])
    refuses(ValueError, keep_len=n[:1])
    refuses(ValueError, need=n.long())
    refuses(ValueError, block=None)
    refuses(BAD, block=0)
    refuses(ValueError, pools=[z(5, 16, 64)])
    refuses(ValueError, pools=[z(6, 16, 64, device="cpu")])
    refuses(ValueError, pools=[z(6, 64, 16).transpose(1, 2)])
    refuses(ValueError, pools=[z(2, 6, 16, 64)])
    refuses(BAD, pools=[z(6, 16, 64)] * 9)
    out = dict(cache_len=z(2, dtype=I32), row_status=z(2, dtype=I32))
    refuses(ValueError, source=n, out=dict(out, block_table=t))
    refuses(ValueError, out=dict(out, block_table=z(2, 4, dtype=I32)))
    refuses(ValueError, out=dict(out, cache_len=n))
    refuses(ValueError, out=dict(out, row_status=z(1, dtype=I32)))
    refuses(BAD, workspace=z(64, dtype=torch.uint8))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    refuses(ValueError)
