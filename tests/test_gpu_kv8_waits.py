"""Attention over the 8-bit paged cache whose waits run out: the same sources, built with limits of up to two microseconds,
so that waits end early at every place of the kernels. Such a call returns, says so in row_status, stores nothing outside its
outputs, and leaves the context usable."""

import ctypes
import os
import random
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import kv8_plain as plain
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
LIMITS = (0, 300, 2000)  # ns; at 0 a wait ends at its first look


@pytest.fixture(scope="module")
def short():
    """The library with each limit."""
    need_gpu()
    from speculative_decoding_verification_29_gb300 import _lib, build

    work = os.path.join(build.BUILD_DIR, "waits")
    os.makedirs(work, exist_ok=True)
    names = [n for n in build.SOURCES if n.startswith("kv8_attn") or n.startswith("kv8_wide")]
    rest = [os.path.join(build.BUILD_DIR, os.path.splitext(n)[0] + ".o") for n in build.SOURCES if n not in names]
    if not all(map(os.path.exists, rest)):
        build.build(force=True)

    def compile_one(job):
        ns, name = job
        obj = os.path.join(work, f"{os.path.splitext(name)[0]}_{ns}.o")
        subprocess.run([build._nvcc(), *build.NVCC_FLAGS, f"-DSPECV_WAIT_NS={ns}", "-c", os.path.join(build.CSRC, name), "-o", obj],
                       check=True)
        return obj

    with ThreadPoolExecutor(4) as ex:
        objs = list(ex.map(compile_one, [(ns, n) for ns in LIMITS for n in names]))
    libs = {}
    for i, ns in enumerate(LIMITS):
        path = os.path.join(work, f"libspecverify_{ns}.so")
        subprocess.run([build._nvcc(), *build.ARCH, "-shared", "-o", path, *rest, *objs[i * len(names): (i + 1) * len(names)]],
                       check=True)
        lib = ctypes.CDLL(path)
        for name, (res, args) in _lib.SIGNATURES.items():
            getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
        libs[ns] = lib
    return libs


CASES = [
    # ctx, new, Hq, H, D, dtype, tree
    ([517], [1], 32, 8, 128, BF, False),
    ([900, 1500, 40, 2100] * 4, [1] * 16, 16, 8, 64, HF, False),
    ([700, 20, 3000, 300], [9, 5, 9, 1], 16, 4, 128, BF, False),
    ([700, 20, 1100, 300], [16, 5, 9, 1], 16, 4, 128, HF, False),
    ([900, 20], [25, 32], 8, 2, 128, BF, False),
    ([300, 1000, 64], [61, 61, 61], 8, 2, 128, BF, True),
    ([10, 800], [400, 129], 8, 4, 128, HF, False),
    ([90, 0], [140, 70], 4, 2, 64, BF, False),
]


@pytest.mark.parametrize("ns", LIMITS)
@pytest.mark.parametrize("ctx,new,Hq,H,D,dt,tree", CASES)
def test_waits_that_run_out(short, monkeypatch, ns, ctx, new, Hq, H, D, dt, tree):
    import speculative_decoding_verification_29_gb300 as sv
    from speculative_decoding_verification_29_gb300 import _lib

    c = plain.Cache(ctx, new, H, D, 64, seed=3).fill()
    T, B, most = sum(new), len(ctx), max(new)
    q = torch.randn(T, Hq, D, generator=torch.Generator().manual_seed(4)).to(dt).cuda()
    mask = plain.tree_mask(random.Random(1), B, most)[0].cuda() if tree else None
    args, cu = c.to("cuda"), c.cu.cuda()
    kw = dict(max_tokens=most, tree_mask=mask)
    want = sv.spec_kv8_attention(q, *args, cu, **kw)
    assert want["row_status"].tolist() == [0] * B
    before = [a.clone() for a in args]
    nbytes = sv.kv8_workspace_bytes(args[0], args[4], Hq, most, dt)
    out = torch.full((T + 2, Hq, D), 7.0, dtype=dt, device="cuda")
    ws = torch.full((nbytes + 512,), 77, dtype=torch.uint8, device="cuda")
    at = 256 + -ws.data_ptr() % 256
    status = torch.full((B + 2,), 5, dtype=torch.int32, device="cuda")
    ran_out = 0  # calls in which a wait did
    with monkeypatch.context() as m:
        m.setattr(_lib, "_lib", short[ns])
        for _ in range(10):
            sv.spec_kv8_attention(q, *args, cu, out=dict(out=out[1: T + 1], row_status=status[1: B + 1]),
                                  workspace=ws[at: at + nbytes], **kw)
            torch.cuda.synchronize()
            s = status.tolist()
            assert s[0] == 5 and s[-1] == 5 and s[1:-1] in ([0] * B, [_lib.SPEC_ROW_TIMEOUT] * B)
            ran_out += s[1] != 0
            if s[1] == 0:
                assert torch.equal(out[1: T + 1], want["out"])
    assert (out[0] == 7).all() and (out[-1] == 7).all()
    assert (ws[:at] == 77).all() and (ws[at + nbytes:] == 77).all()
    assert all(torch.equal(a, b) for a, b in zip(args, before))
    if ns == LIMITS[0]:
        assert ran_out == 10
    again = sv.spec_kv8_attention(q, *args, cu, **kw)
    assert torch.equal(again["out"], want["out"]) and again["row_status"].tolist() == [0] * B
