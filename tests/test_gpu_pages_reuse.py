"""The pages' calls made again: one dict of outputs for several tables, and what of the pools a call may not guess."""

import pytest
import torch

import latent_plain as plain
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def sv():
    import speculative_decoding_verification_29_gb300 as m

    return m


def i32(*x):
    return torch.tensor(x, dtype=I32)


def test_one_out_for_several_tables():
    """Each call's rows go into the table that it was given, or with source into a new one, whatever the last call did."""
    bs = 16
    tables = [i32([0, 1, -1], [2, -1, -1]), i32([5, -1, -1], [3, 4, -1])]
    lens = [i32(20, 16), i32(9, 30)]
    out = dict(cache_len=torch.zeros(2, dtype=I32, device="cuda"), row_status=torch.zeros(2, dtype=I32, device="cuda"))
    keys = set(out)
    need = i32(20, 3)
    for source in (None, i32(1, 1)):
        for table, length in zip(tables, lens):
            refs = torch.zeros(12, dtype=I32)
            for i in table[table >= 0].tolist():
                refs[i] += 1
            rows, kept, counts, status, _ = plain.pages(table, length, refs, bs, source=source, need=need)
            t, r = table.cuda(), refs.cuda()
            got = sv().spec_pages_update(t, length.cuda(), r, block=bs, need=need.cuda(), out=out,
                                         source=None if source is None else source.cuda())
            assert got["block_table"].tolist() == rows and r.tolist() == counts and got["refs"] is r
            assert got["cache_len"] is out["cache_len"] and out["cache_len"].tolist() == kept
            assert out["row_status"].tolist() == status
            assert (got["block_table"] is t) == (source is None)
            if source is not None:
                assert torch.equal(t.cpu(), table)
            assert set(out) == keys


def test_a_block_that_no_pool_tells():
    """The scales of an 8-bit cache, [blocks, heads], have no dimension of tokens: block is asked for."""
    table, length, refs, need = i32([0, 1, -1], [2, -1, -1]).cuda(), i32(20, 16).cuda(), i32(1, 1, 1, 0, 0, 0).cuda(), i32(1, 1).cuda()
    scales = torch.zeros(6, 4, dtype=torch.uint8, device="cuda")
    codes = torch.zeros(6, 4, 16, 64, dtype=torch.uint8, device="cuda")
    for pools, planes in (((scales, codes), False), ((scales[None], codes[None]), True), ((torch.zeros(6, 16, device="cuda"),), False)):
        with pytest.raises(ValueError, match="block is needed"):
            sv().spec_pages_update(table, length, refs, pools, planes=planes, need=need)
    assert table.tolist() == [[0, 1, -1], [2, -1, -1]] and refs.tolist() == [1, 1, 1, 0, 0, 0]
    r = sv().spec_pages_update(table, length, refs, (codes, scales), need=need)
    assert r["block_table"].tolist() == [[0, 1, -1], [2, 3, -1]]
    r = sv().spec_pages_update(table, length, refs, (scales, codes), block=16, keep_len=i32(20, 17 - 1).cuda())
    assert r["block_table"].tolist() == [[0, 1, -1], [2, -1, -1]]


def test_room_after_a_request_that_failed():
    """Later sequences that ask are refused with it, those too that have their room, and all keep their tokens; asked again without
    it, they are served. One that asks nothing is not marked."""
    r = sv().spec_pages_update(i32([0, -1, -1], [3, -1, -1], [4, -1, -1], [5, -1, -1]).cuda(), i32(15, 10, 16, 9).cuda(),
                               i32(1, 0, 1, 1, 1, 1).cuda(), block=16, need=i32(33, 6, 1, 0).cuda())
    assert r["row_status"].tolist() == [64, 64, 64, 0] and r["cache_len"].tolist() == [15, 10, 16, 9]
    assert r["block_table"].tolist() == [[0, -1, -1], [3, -1, -1], [4, -1, -1], [5, -1, -1]] and r["refs"].tolist() == [1, 0, 1, 1, 1, 1]
    r = sv().spec_pages_update(r["block_table"], r["cache_len"], r["refs"], block=16, need=i32(0, 6, 1, 0).cuda())
    assert r["row_status"].tolist() == [0, 0, 0, 0] and r["block_table"].tolist() == [[0, -1, -1], [3, -1, -1], [4, 1, -1], [5, -1, -1]]
