"""What the 8-bit paged cache's C entry points refuse. Validation runs on the host before anything is enqueued, so the
pointers here are numbers; the module is left out where a GPU could be reached with them."""

import ctypes
import math

import pytest
import torch

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers used here are no device memory")

OK, ARG, WORKSPACE, CUDA, LIMIT = 0, -1, -2, -3, -5
F32, BF16, F16 = 0, 1, 2
P = 0x7F0000000000  # stands for a device pointer


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_29_gb300 import _lib, build

    build.build()
    return _lib.load()


def cache(**kw):
    from speculative_decoding_verification_29_gb300 import _lib

    f = dict(k=P, v=P + (1 << 32), k_scale=P + (2 << 32), v_scale=P + (3 << 32), block_table=P + (4 << 32),
             cache_len=P + (5 << 32), B=4, num_blocks=100, max_blocks=20, block=32, kv_heads=8, head_dim=128)
    f.update(kw)
    D, bs, H = (max(1, f[x]) for x in ("head_dim", "block", "kv_heads"))
    strides = dict(stride_block=H * bs * D, stride_head=bs * D, stride_slot=D)
    strides.update({x: f.pop(x) for x in list(f) if x in strides})
    c = _lib.Kv8Cache(*[f[x] for x in ("k", "v", "k_scale", "v_scale", "block_table", "cache_len", "B", "num_blocks",
                                       "max_blocks", "block", "kv_heads", "head_dim")],
                      strides["stride_block"], strides["stride_head"], strides["stride_slot"])
    return c


def append(lib, c=None, keys=P, kst=1024, ksh=128, values=P, vst=1024, vsh=128, dtype=BF16, T=36, cu=P, pos=None,
           freq=None, rot=0, inter=0, q=None, qst=0, qsh=0, qo=None, ost=0, osh=0, hq=0, status=P):
    freq = None if freq is None else (ctypes.c_double * len(freq))(*freq)
    p = None if freq is None else ctypes.addressof(freq)
    return lib.spec_kv8_append(ctypes.byref(c if c is not None else cache()), keys, kst, ksh, values, vst, vsh, dtype, T, cu,
                               pos, p, rot, inter, q, qst, qsh, qo, ost, osh, hq, status, None)


def attention(lib, c=None, q=P, qst=4096, qsh=128, dtype=BF16, T=36, hq=32, cu=P, most=9, mask=None, scale=0.1, out=P,
              ost=4096, osh=128, status=P, ws=P, nbytes=1 << 40):
    return lib.spec_kv8_attention(ctypes.byref(c if c is not None else cache()), q, qst, qsh, dtype, T, hq, cu, most, mask,
                                  scale, out, ost, osh, status, ws, nbytes, None)


def compact(lib, c=None, planes=1, sp=0, ssp=0, path=P, D=8, acc=P, new_len=P, status=P):
    return lib.spec_kv8_compact(ctypes.byref(c if c is not None else cache()), planes, sp, ssp, path, D, acc, new_len,
                                status, None)


def test_sound_arguments_reach_the_launch(lib):
    """The base of the refusals below: without a GPU these calls get as far as the launch, which fails."""
    assert append(lib) == CUDA
    assert append(lib, freq=[1.0] * 8, rot=16, q=P, qst=4096, qsh=128, qo=P, ost=4096, osh=128, hq=32) == CUDA
    assert attention(lib) == CUDA
    assert compact(lib) == CUDA


BAD_CACHE = [
    ({x: None}, ARG) for x in ("k", "v", "k_scale", "v_scale", "block_table", "cache_len")
] + [
    ({x: n}, ARG) for x in ("B", "num_blocks", "max_blocks", "block", "kv_heads", "head_dim") for n in (0, -1)
] + [
    (dict(k=P + 8), ARG), (dict(v=P + 4), ARG),
    (dict(stride_slot=112), ARG), (dict(stride_slot=136), ARG), (dict(stride_slot=-128), ARG),
    (dict(stride_head=-4096), ARG), (dict(stride_head=4104), ARG), (dict(stride_block=8), ARG), (dict(stride_block=-16), ARG),
    (dict(block=8), LIMIT), (dict(block=48), LIMIT), (dict(block=256), LIMIT),
    (dict(head_dim=32), LIMIT), (dict(head_dim=96), LIMIT), (dict(head_dim=256), LIMIT),
    (dict(B=65536), LIMIT), (dict(kv_heads=1025), LIMIT),
    (dict(num_blocks=1 << 30, kv_heads=2), LIMIT), (dict(max_blocks=1 << 26), LIMIT),
    (dict(stride_block=1 << 40), LIMIT), (dict(stride_head=1 << 40), LIMIT), (dict(stride_slot=1 << 40), LIMIT),
]


@pytest.mark.parametrize("kw,rc", BAD_CACHE)
def test_cache_is_refused_by_every_call(lib, kw, rc):
    c = cache(**kw)
    assert append(lib, c) == rc
    assert attention(lib, c, hq=c.kv_heads) == rc
    assert compact(lib, c) == rc
    assert lib.spec_kv8_workspace_bytes(ctypes.byref(c), max(1, c.kv_heads), 9, BF16) == 0


def test_null_cache(lib):
    assert lib.spec_kv8_append(None, P, 1024, 128, P, 1024, 128, BF16, 36, P, None, None, 0, 0, None, 0, 0, None, 0, 0, 0, P,
                               None) == ARG
    assert lib.spec_kv8_attention(None, P, 4096, 128, BF16, 36, 32, P, 9, None, 0.1, P, 4096, 128, P, P, 1 << 40, None) == ARG
    assert lib.spec_kv8_compact(None, 1, 0, 0, P, 8, P, P, P, None) == ARG
    assert lib.spec_kv8_workspace_bytes(None, 32, 9, BF16) == 0


@pytest.mark.parametrize("kw,rc", [
    (dict(keys=None), ARG), (dict(values=None), ARG), (dict(cu=None), ARG), (dict(status=None), ARG), (dict(T=-1), ARG),
    (dict(dtype=3), ARG), (dict(dtype=-1), ARG),
    (dict(kst=-1), ARG), (dict(ksh=-1), ARG), (dict(vst=-1), ARG), (dict(vsh=1 << 40), ARG),
    (dict(q=P, hq=32), ARG), (dict(qo=P, hq=32), ARG), (dict(q=P, qo=P, hq=0), ARG), (dict(q=P, qo=P, hq=4, qst=-1), ARG),
    (dict(q=P, qo=P, hq=4, osh=-1), ARG),
    (dict(rot=16), ARG), (dict(freq=[1.0] * 8), ARG), (dict(freq=[1.0] * 4, rot=8), ARG), (dict(freq=[1.0] * 8, rot=-16), ARG),
    (dict(freq=[1.0] * 72, rot=144), ARG),
    (dict(freq=[1.0] * 7 + [math.nan], rot=16), ARG), (dict(freq=[1.0] * 7 + [math.inf], rot=16), ARG),
    (dict(freq=[1.0] * 7 + [2e9], rot=16), ARG),
    (dict(T=1 << 23), LIMIT), (dict(T=(1 << 23) - 1, q=P, qo=P, hq=257), LIMIT),
])
def test_append_refuses(lib, kw, rc):
    assert append(lib, **kw) == rc


def test_append_rotation_fits_the_head(lib):
    c = cache(head_dim=64)
    assert append(lib, c, freq=[1.0] * 32, rot=64) == CUDA
    assert append(lib, c, freq=[1.0] * 40, rot=80) == ARG


@pytest.mark.parametrize("kw,rc", [
    (dict(q=None), ARG), (dict(out=None), ARG), (dict(cu=None), ARG), (dict(status=None), ARG), (dict(T=-1), ARG),
    (dict(hq=0), ARG), (dict(hq=12), ARG), (dict(hq=-8), ARG), (dict(most=0), ARG), (dict(dtype=F32), ARG), (dict(dtype=7), ARG),
    (dict(scale=math.nan), ARG), (dict(scale=math.inf), ARG), (dict(qst=-1), ARG), (dict(osh=1 << 40), ARG),
    (dict(hq=8 * 65), LIMIT), (dict(T=1 << 26), LIMIT), (dict(mask=P, most=1025), LIMIT),
    (dict(ws=None), WORKSPACE), (dict(ws=P + 128), WORKSPACE), (dict(nbytes=0), WORKSPACE),
])
def test_attention_refuses(lib, kw, rc):
    assert attention(lib, **kw) == rc


@pytest.mark.parametrize("most", [1, 4, 5, 9, 12, 13, 16, 17, 64, 65, 4096, 2 ** 31 - 1])
@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, BF16), (128, F16)])
def test_attention_workspace(lib, most, D, dtype):
    c = cache(head_dim=D)
    n = lib.spec_kv8_workspace_bytes(ctypes.byref(c), 32, most, dtype)
    assert n > 0 and n % 256 == 0 and n < 1 << 27
    assert attention(lib, c, most=most, dtype=dtype, nbytes=n) == CUDA
    assert attention(lib, c, most=most, dtype=dtype, nbytes=n - 1) == WORKSPACE


def test_workspace_query_refuses(lib):
    c = ctypes.byref(cache())
    assert lib.spec_kv8_workspace_bytes(c, 12, 9, BF16) == 0
    assert lib.spec_kv8_workspace_bytes(c, 0, 9, BF16) == 0
    assert lib.spec_kv8_workspace_bytes(c, 32, 0, BF16) == 0
    assert lib.spec_kv8_workspace_bytes(c, 32, 9, F32) == 0


def test_attention_grid_limit(lib):
    """Sequences times row tiles stays below 2^31."""
    c = cache(B=65535, kv_heads=1)
    assert attention(lib, c, T=(1 << 25) - 1, hq=32, most=1 << 24) == LIMIT


@pytest.mark.parametrize("kw,rc", [
    (dict(acc=None), ARG), (dict(new_len=None), ARG), (dict(status=None), ARG), (dict(planes=0), ARG), (dict(D=0), ARG),
    (dict(planes=2, sp=-16), ARG), (dict(planes=2, sp=8), ARG), (dict(planes=2, ssp=-1), ARG),
    (dict(D=65), LIMIT), (dict(planes=1 << 25), LIMIT), (dict(sp=1 << 46), LIMIT), (dict(ssp=1 << 46), LIMIT),
])
def test_compact_refuses(lib, kw, rc):
    assert compact(lib, **kw) == rc


def test_python_refuses_host_tensors():
    import speculative_decoding_verification_29_gb300 as sv

    k = torch.zeros(4, 2, 32, 128, dtype=torch.uint8)
    s = torch.zeros(4, 2, dtype=torch.uint8)
    i = torch.zeros(1, dtype=torch.int32)
    x = torch.zeros(1, 2, 128, dtype=torch.bfloat16)
    args = (k, k, s, s, i.view(1, 1), i)
    with pytest.raises(ValueError):
        sv.spec_kv8_append(x, x, *args, torch.tensor([0, 1], dtype=torch.int32))
    with pytest.raises(ValueError):
        sv.spec_kv8_attention(x, *args, torch.tensor([0, 1], dtype=torch.int32), max_tokens=1)
    with pytest.raises(ValueError):
        sv.spec_kv8_compact(*args, i)


@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_longest_sequence(lib, block):
    """A position rounded up to a whole tile of 128 slots stays below 2^31, whatever cache_len says."""
    most = (2 ** 31 - 128) // block
    for call in (append, attention, compact):
        assert call(lib, cache(block=block, max_blocks=most)) == CUDA
        assert call(lib, cache(block=block, max_blocks=most + 1)) == LIMIT
