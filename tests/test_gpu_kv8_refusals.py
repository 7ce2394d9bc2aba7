"""What the Python calls of the 8-bit paged cache refuse before anything is launched: types, shapes, strides, devices."""

import pytest
import torch

from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def sv():
    import speculative_decoding_verification_29_gb300 as m

    return m


def z(*shape, dtype=torch.uint8, device="cuda"):
    return torch.zeros(*shape, dtype=dtype, device=device)


def cache(**kw):
    i32 = torch.int32
    a = dict(k_cache=z(6, 2, 32, 128), v_cache=z(6, 2, 32, 128), k_scale=z(6, 2), v_scale=z(6, 2),
             block_table=z(2, 3, dtype=i32), cache_len=z(2, dtype=i32))
    a.update(kw)
    return tuple(a.values())


CU = [0, 1, 3]
BAD_CACHE = [
    dict(v_cache=(6, 2, 32, 64)), dict(k_cache=(6, 2, 32)), dict(k_scale=(6, 3)), dict(v_scale=(5, 2)),
    dict(block_table=(3, 3)), dict(block_table=(6,)), dict(cache_len=(2, 1)),
]


@pytest.mark.parametrize("bad", BAD_CACHE)
def test_cache_shapes(bad):
    (name, shape), = bad.items()
    t = z(*shape, dtype=torch.int32 if name in ("block_table", "cache_len") else torch.uint8)
    everywhere(cache(**{name: t}))


def test_cache_types_strides_devices():
    everywhere(cache(k_cache=z(6, 2, 32, 128, dtype=torch.int16)))
    everywhere(cache(v_cache=z(6, 32, 2, 128).transpose(1, 2)))
    both = z(6, 2, 32, 256)[..., ::2]
    everywhere(cache(k_cache=both, v_cache=both))
    odd = z(6, 2, 32, 136)[..., :128]  # slots of 136 bytes
    everywhere(cache(k_cache=odd, v_cache=odd), (ValueError, RuntimeError))
    everywhere(cache(k_scale=z(2, 6).T))
    everywhere(cache(k_scale=z(6, 2, dtype=torch.float32)))
    everywhere(cache(block_table=z(2, 3, dtype=torch.int64)))
    everywhere(cache(cache_len=z(2, dtype=torch.int32, device="cpu")))
    everywhere(cache(v_cache=z(6, 2, 32, 128, device="cpu")))


def everywhere(c, error=ValueError):
    cu = torch.tensor(CU, dtype=torch.int32, device="cuda")
    x = z(3, 2, 128, dtype=BF)
    with pytest.raises(error):
        sv().spec_kv8_append(x, x, *c, cu)
    with pytest.raises(error):
        sv().spec_kv8_attention(x, *c, cu, max_tokens=2)
    with pytest.raises(error):
        sv().spec_kv8_compact(*c, z(2, dtype=torch.int32))


def test_append_arguments():
    cu = torch.tensor(CU, dtype=torch.int32, device="cuda")
    x, q = z(3, 2, 128, dtype=BF), z(3, 4, 128, dtype=BF)

    def refuses(error, k=x, v=x, c=None, cu=cu, **kw):
        with pytest.raises(error):
            sv().spec_kv8_append(k, v, *(c or cache()), cu, **kw)

    refuses(ValueError, v=z(3, 2, 64, dtype=BF))
    refuses(ValueError, v=z(3, 1, 128, dtype=BF))
    refuses(ValueError, v=z(3, 2, 128, dtype=torch.float16))
    refuses(ValueError, k=z(3, 256, dtype=BF))
    refuses(ValueError, k=z(3, 2, 256, dtype=BF)[..., ::2])
    refuses(ValueError, k=z(3, 2, 128, dtype=BF, device="cpu"))
    refuses(TypeError, k=z(3, 2, 128, dtype=torch.float64), v=z(3, 2, 128, dtype=torch.float64))
    refuses(ValueError, cu=cu[:2])
    refuses(ValueError, cu=cu.long())
    refuses(ValueError, positions=cu[:2])
    refuses(ValueError, positions=cu.long())
    refuses(ValueError, q=q[:2])
    refuses(ValueError, q=q.half())
    refuses(ValueError, q=q, q_out=q[:, :2])
    for freq in ([1.0] * 4, [1.0] * 72, [float("nan")] * 8, torch.full((8,), 1e10)):
        refuses((ValueError, RuntimeError), inv_freq=freq)


def test_attention_arguments():
    cu = torch.tensor(CU, dtype=torch.int32, device="cuda")
    x = z(3, 4, 128, dtype=BF)

    def refuses(error, q=x, c=None, cu=cu, max_tokens=2, **kw):
        with pytest.raises(error):
            sv().spec_kv8_attention(q, *(c or cache()), cu, max_tokens=max_tokens, **kw)

    refuses(TypeError, q=x.float())
    refuses(ValueError, q=x[..., :64])
    refuses(ValueError, cu=cu[:2])
    refuses(ValueError, tree_mask=z(2, 3, 3))
    refuses(ValueError, tree_mask=z(2, 2, 2, dtype=torch.int32))
    refuses(ValueError, tree_mask=z(2, 2, 4)[..., ::2])
    status = z(2, dtype=torch.int32)
    refuses(ValueError, out=dict(out=x[:2], row_status=status))
    refuses(ValueError, out=dict(out=x.half(), row_status=status))
    bad = (ValueError, RuntimeError)
    refuses(bad, q=z(3, 3, 128, dtype=BF))
    refuses(bad, max_tokens=0)
    refuses(bad, sm_scale=float("nan"))
    refuses(bad, workspace=z(256))
    refuses(bad, q=z(3, 130, 128, dtype=BF))


def test_compact_arguments():
    i = z(2, dtype=torch.int32)
    for kw in (dict(accept_len=i[:1]), dict(accept_len=i.long()), dict(path=i), dict(path=z(3, 4, dtype=torch.int32)),
               dict(path=z(2, 4)), dict(path=z(2, 65, dtype=torch.int32))):
        args = dict(accept_len=i)
        args.update(kw)
        with pytest.raises((ValueError, RuntimeError)):
            sv().spec_kv8_compact(*cache(), **args)
    planes = [z(3, 6, 2, 32, 128), z(3, 6, 2, 32, 128), z(3, 6, 2), z(4, 6, 3)[:3, :, :2]]
    with pytest.raises(ValueError):
        sv().spec_kv8_compact(*planes, *cache()[4:], i)


def test_another_device_is_refused(monkeypatch):
    """Kernels are launched on the current device; a cache on another one is refused (one GPU: the current device is faked)."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    everywhere(cache())
