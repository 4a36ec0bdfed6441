"""Fork and compact of a pool with more pages than the planning warps keep in their lanes (above 2^19):
the words behind a warp's first 32 go through memory."""

import pytest
import torch

from paged_latent_attention_mla_gb300 import NO_PAGE, cache_compact, cache_fork, cache_workspace
from paged_latent_attention_mla_gb300 import _native as n
from paged_latent_attention_mla_gb300 import build as nbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    nbuild.build()
    n.load()


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pools(pages, P=8, dtype=torch.bfloat16):
    return tuple(torch.zeros((pages, P, d), dtype=dtype, device="cuda") for d in (512, 64))


PAGES = 1_200_007  # 73 32-page words to a planning warp: more than its lanes hold


def test_fork_of_a_pool_past_the_warps_lanes():
    """Free pages are the lowest ids, in order, also behind a planning warp's first 32 words."""
    P, W, rows = 8, 40, 1000
    ckv, kpe = pools(PAGES, P, torch.float8_e4m3fn)
    g = torch.Generator(device="cuda").manual_seed(1)
    ref = (torch.rand(PAGES, generator=g, device="cuda") < 0.97).int()  # somebody else's pages
    free = (ref == 0).nonzero()[:, 0].int()
    new = torch.randint(0, W * P + 1, (rows,), generator=g, device="cuda", dtype=torch.int32)
    need = (new + P - 1) // P
    ws = cache_workspace(num_pages=PAGES, page_table_stride=W, rows=rows, page_size=P)
    ws.random_(0, 256)
    table, lens = torch.full((1, W), NO_PAGE, dtype=torch.int32, device="cuda"), dev([0])
    word = dev([0])
    t, l, r = cache_fork(table, lens, torch.full((rows,), -1, dtype=torch.int32, device="cuda"), ref, ckv, kpe, ws,
                         new_tokens=new, status=word)
    assert n.mla_cache_status(word) == n.MLA_OK and int(need.sum()) < free.numel()
    held = torch.arange(W, device="cuda") < need[:, None]
    assert torch.equal(t[held], free[: int(need.sum())]) and (t[~held] == NO_PAGE).all() and torch.equal(l, new)
    want = ref.clone()
    want[t[held].long()] = 1
    assert torch.equal(r, want)


def test_compact_of_a_pool_past_the_warps_lanes():
    P, W, rows = 8, 50, 100
    ckv, kpe = pools(PAGES, P, torch.float8_e4m3fn)
    g = torch.Generator(device="cuda").manual_seed(2)
    marks = torch.randint(0, 256, (PAGES,), generator=g, device="cuda").to(torch.uint8)
    ckv.view(torch.uint8)[:, 0, 0] = marks
    kpe.view(torch.uint8)[:, P - 1, 63] = marks
    ref = (torch.rand(PAGES, generator=g, device="cuda") < 0.4).int() * 3
    used = ref > 0
    count = int(used.sum())
    ids = torch.arange(PAGES, device="cuda")
    to = torch.where(used, ids, -1)
    src, dst = ids[used & (ids >= count)], ids[~used & (ids < count)]
    to[src] = dst
    table = torch.randint(0, PAGES, (rows, W), generator=g, device="cuda", dtype=torch.int32)
    want_marks, want_ref = marks.clone(), ref.clone()
    want_marks[dst], want_ref[dst], want_ref[src] = marks[src], ref[src], 0
    ws = cache_workspace(num_pages=PAGES, page_table_stride=W, rows=rows, page_size=P)
    ws.random_(0, 256)
    t, r, page_map, num = cache_compact(table, ref, ckv, kpe, ws)
    assert num.item() == count and torch.equal(page_map, to.int()) and torch.equal(r, want_ref)
    assert torch.equal(t, to.int()[table.long()])
    assert torch.equal(ckv.view(torch.uint8)[:, 0, 0], want_marks) and torch.equal(kpe.view(torch.uint8)[:, P - 1, 63], want_marks)
