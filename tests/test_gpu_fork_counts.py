"""Fork of pools whose counts are below zero: a count of 0 or less is a free page."""

import pytest
import torch

from paged_latent_attention_mla_gb300 import NO_PAGE, cache_fork, cache_workspace
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


@pytest.mark.parametrize("low", [-1, -2, -7, -16384, 2 ** 14 - 2 ** 31])
@pytest.mark.parametrize("in_place", [False, True])
def test_counts_below_zero_are_free_pages(low, in_place):
    """As compact takes them: a page whose count is 0 or less is given out, and one that is not stays as it was."""
    ckv, kpe = pools(6)
    ws = cache_workspace(num_pages=6, page_table_stride=3, rows=2, page_size=8)
    word, ref = dev([0]), dev([low, 1, low, 0, low, 1])
    table, lens = dev([[1, NO_PAGE, NO_PAGE], [5, NO_PAGE, NO_PAGE]]), dev([8, 3])
    out = dict(page_table_out=table, seq_lens_out=lens, ref_count_out=ref) if in_place else {}
    t, l, r = cache_fork(table, lens, dev([0, 1]), ref, ckv, kpe, ws, new_tokens=dev([9, 6]), status=word, **out)
    assert n.mla_cache_status(word) == n.MLA_OK
    assert t.tolist() == [[1, 0, 2], [5, 3, NO_PAGE]] and l.tolist() == [17, 9]
    assert r.tolist() == [1, 1, 1, 1, low, 1]


@pytest.mark.parametrize("low", [0, -1, -2, -3])
def test_claims_beside_counts_below_zero(low):
    """Three branches of one row write on in its shared page while free pages' counts look like claims."""
    ckv, kpe = pools(6)
    ckv[4] = torch.arange(8, device="cuda").view(8, 1)
    ws = cache_workspace(num_pages=6, page_table_stride=2, rows=3, page_size=8)
    word, ref = dev([0]), dev([low, 2, low, low, 2, 1])
    table, lens = dev([[1, 4], [1, 4]]), dev([13, 12])
    t, l, r = cache_fork(table, lens, dev([0, 1, 0]), ref, ckv, kpe, ws, new_tokens=dev([1, 1, 1]), status=word)
    assert n.mla_cache_status(word) == n.MLA_OK
    assert t.tolist() == [[1, 4], [1, 0], [1, 2]] and l.tolist() == [14, 13, 14]
    assert r.tolist() == [1, 3, 1, low, 1, 1]
    assert torch.equal(ckv[0, :4], ckv[4, :4]) and not ckv[0, 4:].any() and torch.equal(ckv[2, :5], ckv[4, :5])
