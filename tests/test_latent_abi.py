"""What the C entry points of the paged latent cache and of the pages refuse. Validation runs on the host before anything is
enqueued, so the pointers here are numbers; the module is left out where a GPU could be reached with them."""

import ctypes
import math

import pytest
import torch

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers used here are no device memory")

ARG, WORKSPACE, CUDA, LIMIT = -1, -2, -3, -5
F32, BF16, F16 = 0, 1, 2
P = 0x7F0000000000  # stands for a device pointer


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_29_gb300 import _lib, build

    build.build()
    return _lib.load()


def cache(**kw):
    from speculative_decoding_verification_29_gb300 import _lib

    f = dict(data=P, block_table=P + (1 << 32), cache_len=P + (2 << 32), B=4, num_blocks=100, max_blocks=20, block=32,
             latent_dim=512, rot_dim=64, dtype=BF16)
    f.update(kw)
    entry = 2 * (max(1, f["latent_dim"]) + max(1, f["rot_dim"]))
    sb, ss = f.pop("stride_block", max(1, f["block"]) * entry), f.pop("stride_slot", entry)
    return _lib.LatentCache(*f.values(), sb, ss)


FREQ = (ctypes.c_double * 32)(*[0.5] * 32)


def append(lib, c=None, x=P, xst=576, r=P, rst=576, dtype=BF16, T=36, cu=P, pos=None, freq=FREQ, inter=0, w=None, wt=0, eps=1e-6,
           q=None, qst=0, qsh=0, qo=None, ost=0, osh=0, hq=0, status=P):
    return lib.spec_latent_append(ctypes.byref(c or cache()), x, xst, r, rst, dtype, T, cu, pos,
                                  None if freq is None else ctypes.addressof(freq), inter, w, wt, eps, q, qst, qsh, qo, ost, osh, hq,
                                  status, None)


def attention(lib, c=None, q=P, qst=18432, qsh=576, T=36, hq=32, cu=P, most=9, mask=None, scale=0.1, out=P, ost=16384, osh=512,
              status=P, ws=P, nbytes=1 << 40):
    return lib.spec_latent_attention(ctypes.byref(c or cache()), q, qst, qsh, T, hq, cu, most, mask, scale, out, ost, osh, status,
                                     ws, nbytes, None)


def compact(lib, c=None, planes=1, sp=0, path=P, D=8, acc=P, new_len=P, status=P):
    return lib.spec_latent_compact(ctypes.byref(c or cache()), planes, sp, path, D, acc, new_len, status, None)


def pages(lib, table=P, new=P, length=P, keep=None, source=None, need=None, refs=P, B=4, M=20, nb=100, block=32, pools=(), n=None,
          new_len=P + 4096, status=P, ws=P, nbytes=1 << 40):
    from speculative_decoding_verification_29_gb300 import _lib

    recs = (_lib.PagesPool * max(1, len(pools)))(*[_lib.PagesPool(*p) for p in pools])
    return lib.spec_pages_update(table, new, length, keep, source, need, refs, B, M, nb, block, recs,
                                 len(pools) if n is None else n, new_len, status, ws, nbytes, None)


def test_sound_arguments_reach_the_launch(lib):
    """The base of the refusals below: without a GPU these calls get as far as the launch, which fails."""
    assert append(lib) == CUDA
    assert append(lib, dtype=F32, w=P, wt=F32, q=P, qst=4096, qsh=64, qo=P, ost=4096, osh=64, hq=32) == CUDA
    assert attention(lib) == CUDA
    assert compact(lib) == CUDA
    assert pages(lib, pools=[(P, 2, 4096, 64, 64)]) == CUDA


BAD_CACHE = [({x: None}, ARG) for x in ("data", "block_table", "cache_len")] + [
    ({x: n}, ARG) for x in ("B", "num_blocks", "max_blocks", "block", "latent_dim", "rot_dim") for n in (0, -1)
] + [
    (dict(dtype=F32), ARG), (dict(dtype=7), ARG), (dict(data=P + 8), ARG), (dict(stride_slot=1136), ARG),
    (dict(stride_slot=1160), ARG), (dict(stride_block=-16), ARG), (dict(stride_block=8), ARG),
    (dict(block=8), LIMIT), (dict(block=48), LIMIT), (dict(block=256), LIMIT),
    (dict(latent_dim=64), LIMIT), (dict(latent_dim=640), LIMIT), (dict(latent_dim=200), LIMIT),
    (dict(rot_dim=8), LIMIT), (dict(rot_dim=72), LIMIT), (dict(rot_dim=80), LIMIT),
    (dict(B=65536), LIMIT), (dict(max_blocks=1 << 26), LIMIT), (dict(stride_block=1 << 40), LIMIT), (dict(stride_slot=1 << 40), LIMIT),
]


@pytest.mark.parametrize("bad,code", BAD_CACHE)
def test_bad_caches(lib, bad, code):
    c = cache(**bad)
    assert append(lib, c) == code and attention(lib, c) == code and compact(lib, c) == code
    assert lib.spec_latent_workspace_bytes(ctypes.byref(c), 32, 9) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), ARG), (dict(r=None), ARG), (dict(cu=None), ARG), (dict(status=None), ARG), (dict(freq=None), ARG),
    (dict(T=-1), ARG), (dict(dtype=F16), ARG), (dict(xst=-1), ARG), (dict(rst=1 << 40), ARG),
    (dict(w=P, wt=F16), ARG), (dict(w=P, wt=F32, eps=-1.0), ARG), (dict(w=P, wt=F32, eps=math.nan), ARG),
    (dict(w=P, wt=F32, eps=math.inf), ARG), (dict(q=P), ARG), (dict(qo=P), ARG), (dict(q=P, qo=P), ARG),
    (dict(q=P, qo=P, hq=4, qst=-1), ARG), (dict(q=P, qo=P, hq=4, osh=-1), ARG),
    (dict(freq=(ctypes.c_double * 32)(*[math.nan] * 32)), ARG), (dict(freq=(ctypes.c_double * 32)(*[2e9] * 32)), ARG),
    (dict(T=1 << 26), LIMIT), (dict(T=1 << 20, q=P, qo=P, hq=1 << 12), LIMIT), (dict(q=P, qo=P, hq=65537), LIMIT),
])
def test_append_arguments(lib, kw, code):
    assert append(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), ARG), (dict(out=None), ARG), (dict(cu=None), ARG), (dict(status=None), ARG), (dict(T=-1), ARG),
    (dict(hq=0), ARG), (dict(most=0), ARG), (dict(scale=math.nan), ARG), (dict(scale=math.inf), ARG), (dict(qst=-1), ARG),
    (dict(osh=1 << 40), ARG), (dict(hq=1025), LIMIT), (dict(T=1 << 27, hq=32), LIMIT), (dict(mask=P, most=1025), LIMIT),
    (dict(ws=None), WORKSPACE), (dict(ws=P + 128), WORKSPACE), (dict(nbytes=1 << 20), WORKSPACE),
])
def test_attention_arguments(lib, kw, code):
    assert attention(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(acc=None), ARG), (dict(new_len=None), ARG), (dict(status=None), ARG), (dict(planes=0), ARG), (dict(D=0), ARG),
    (dict(sp=-16), ARG), (dict(sp=8), ARG), (dict(D=257), LIMIT), (dict(planes=1 << 24), LIMIT), (dict(sp=1 << 46), LIMIT),
])
def test_compact_arguments(lib, kw, code):
    assert compact(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(table=None), ARG), (dict(new=None), ARG), (dict(length=None), ARG), (dict(refs=None), ARG), (dict(new_len=None), ARG),
    (dict(status=None), ARG), (dict(B=0), ARG), (dict(M=0), ARG), (dict(nb=0), ARG), (dict(block=0), ARG), (dict(n=-1), ARG),
    (dict(source=P), ARG), (dict(new_len=P), ARG),
    (dict(pools=[(None, 1, 0, 64, 64)]), ARG), (dict(pools=[(P, 0, 0, 64, 64)]), ARG), (dict(pools=[(P, 1, 0, 64, 0)]), ARG),
    (dict(pools=[(P, 1, -1, 64, 64)]), ARG), (dict(pools=[(P, 1, 0, 63, 64)]), ARG),
    (dict(B=65536), LIMIT), (dict(M=1 << 28), LIMIT), (dict(M=1 << 27, block=16), LIMIT),
    (dict(pools=[(P, 1, 0, 64, 64)] * 9), LIMIT), (dict(pools=[(P, 1, 0, 1 << 40, 64)]), LIMIT),
    (dict(ws=None), WORKSPACE), (dict(ws=P + 8), WORKSPACE), (dict(nbytes=1000), WORKSPACE),
])
def test_pages_arguments(lib, kw, code):
    assert pages(lib, **kw) == code


def test_workspace_sizes(lib):
    assert lib.spec_pages_workspace_bytes(0, 1, 1) == lib.spec_pages_workspace_bytes(1, 0, 1) == 0
    need = lib.spec_pages_workspace_bytes(4, 20, 100)
    assert pages(lib, nbytes=need) == CUDA and pages(lib, nbytes=need - 1) == WORKSPACE
    for hq, most in ((1, 1), (16, 1), (32, 9), (128, 64)):
        need = lib.spec_latent_workspace_bytes(ctypes.byref(cache()), hq, most)
        T = most * 4
        assert attention(lib, hq=hq, most=most, T=T, nbytes=need) == CUDA
        assert attention(lib, hq=hq, most=most, T=T, nbytes=need - 1) == WORKSPACE
