"""The split-KV kernel on small batches, which by default another kernel takes: num_clusters pins it.

Bad pages and lengths are reported by its loaders (one page box to a 64-key group, and several), with
and without a window; results do not depend on where pages lie; packed rows, bounds and windows without
sinks against the definition.  Tolerances as in test_gpu_features.py (oracle) and test_gpu_sinks.py."""

import numpy as np
import pytest
import torch
from test_gpu_features import PACKED, compare, host
from test_gpu_sinks import check, give_up_pages, reference

import oracle
from paged_latent_attention_mla_gb300 import NO_PAGE, decoder_for
from paged_latent_attention_mla_gb300 import _native as n
from paged_latent_attention_mla_gb300 import build as nbuild
from paged_latent_attention_mla_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    nbuild.build()
    n.load()


def decoder(prob, clusters=76, **options):
    dec = decoder_for(prob, num_clusters=clusters, **options)
    assert dec.launches_per_call() == 2  # the split-KV kernel and the reduction
    return dec


def call(dec, d, **over):
    d = {**d, **over}
    out, lse = dec(d["q_latent"], d["q_rope"], d["ckv"], d["kpe"], d["page_table"], d["seq_lens"], d["scale"],
                   local_visible_lens=d.get("local_visible_lens"))
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("dtype,P", [("bf16", 64), ("bf16", 8), ("bf16", 256), ("e4m3", 64), ("e4m3", 32)])
@pytest.mark.parametrize("window,sinks", [(-1, 0), (300, 0), (300, 70)])
@pytest.mark.parametrize("clusters", [76, 3])
def test_bad_pages_are_flagged_and_the_others_right(dtype, P, window, sinks, clusters):
    """A visible page id outside the pool, at the ends and inside of a request's keys, is read as zeros and
    reported; other requests are not touched, and a clean call on the same workspace clears the word."""
    prob = wl.make_problem("uniform", seed=4, H=128, Sq=2, causal=True, window_left=window, dtype=dtype, page_size=P,
                           seq_lens=[700, 300, 513])
    d = prob.device_inputs("cuda")
    dec = decoder(prob, clusters, sink_tokens=sinks)
    good = call(dec, d)
    assert dec.status() == n.MLA_OK
    last = (700 - 1) // P
    places = [last, (700 - 250) // P] + ([0] if window < 0 or sinks else [])
    for at, bad in [(j, e) for j in places for e in (prob.pool_pages, 2 ** 31 - 1, NO_PAGE, -(2 ** 31))]:
        table = d["page_table"].clone()
        table[0, at] = bad
        out, lse = call(dec, d, page_table=table)
        assert dec.status() == n.MLA_ERR_INVALID_ARG
        assert torch.equal(out[1:], good[0][1:]) and torch.equal(lse[1:], good[1][1:])
        assert torch.isfinite(out).all()
    again = call(dec, d)
    assert dec.status() == n.MLA_OK and torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])


@pytest.mark.parametrize("dtype,P", [("bf16", 64), ("e4m3", 16)])
def test_pages_before_the_window_are_not_looked_up(dtype, P):
    prob = wl.make_problem("uniform", seed=4, H=128, Sq=2, causal=True, window_left=100, dtype=dtype, page_size=P,
                           seq_lens=[900, 700])
    d = prob.device_inputs("cuda")
    dec = decoder(prob)
    good = call(dec, d)
    d["page_table"][:, : (700 - 2 - 100) // P] = prob.pool_pages + 1
    out, lse = call(dec, d)
    assert dec.status() == n.MLA_OK and torch.equal(out, good[0]) and torch.equal(lse, good[1])


def test_lengths_outside_the_table_are_flagged():
    prob = wl.make_problem("uniform", seed=6, H=128, Sq=1, seq_lens=[700, 300])
    d = prob.device_inputs("cuda")
    dec = decoder(prob)
    for K in (1 << 20, -1):
        lens = d["seq_lens"].clone()
        lens[1] = K
        table = d["page_table"].clone()
        table[1] = table[0]  # a request clamped to the table's width finds pages there
        call(dec, d, seq_lens=lens, page_table=table)
        assert dec.status() == n.MLA_ERR_INVALID_ARG
    call(dec, d)
    assert dec.status() == n.MLA_OK


def test_the_decode_without_allocation_reports_bad_pages():
    prob = wl.make_problem("uniform", seed=34, H=128, seq_lens=[700, 300])
    d = prob.device_inputs("cuda")
    cfg = decoder(prob).cfg
    out = torch.empty((2, 1, 128, 512), dtype=torch.bfloat16, device="cuda")
    for bad, status in ((prob.pool_pages + 11, n.MLA_ERR_INVALID_ARG), (int(d["page_table"][0, 3]), n.MLA_OK)):
        d["page_table"][0, 3] = bad
        n.mla_decode_noalloc(d["q_latent"], d["q_rope"], d["ckv"], d["kpe"], d["page_table"], d["seq_lens"], d["scale"], -1,
                             out, None, cfg)
        assert n.mla_noalloc_status() == status


@pytest.mark.parametrize("dtype,P,window,sinks", [("bf16", 64, -1, 0), ("e4m3", 64, -1, 0), ("bf16", 16, 300, 0),
                                                  ("e4m3", 128, 300, 9)])
def test_page_permutation_and_repetition_are_bit_identical(dtype, P, window, sinks):
    prob = wl.make_problem("uniform", seed=5, H=128, Sq=2, causal=True, window_left=window, dtype=dtype, page_size=P,
                           seq_lens=[900, 1300, 50])
    perm = torch.randperm(prob.phys_ids.numel(), generator=torch.Generator().manual_seed(1))
    moved = wl.Problem(**{**prob.__dict__, "phys_ids": prob.phys_ids[perm]})
    first, again, other = (call(decoder(p, sink_tokens=sinks), p.device_inputs("cuda")) for p in (prob, prob, moved))
    for a, b in ((first, again), (first, other)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("name", list(PACKED))
@pytest.mark.parametrize("clusters", [76, 5])
def test_packed_rows_all_rows(name, clusters):
    prob = wl.make_problem("uniform", seed=101, **PACKED[name])
    O, L = host(*call(decoder(prob, clusters), prob.device_inputs("cuda")))
    compare(prob.w.dtype, O, L, *oracle.decode(prob.host_inputs()))


@pytest.mark.parametrize("H,window,dtype", [(128, -1, "bf16"), (16, -1, "bf16"), (128, 300, "e4m3"), (16, 300, "bf16")])
def test_local_bounds_all_rows(H, window, dtype):
    lens, Sq = [1500, 90, 700, 2], 3
    prob = wl.make_problem("uniform", seed=303, H=H, Sq=Sq, causal=False, window_left=window, dtype=dtype, seq_lens=lens)
    g = torch.Generator().manual_seed(5)
    lvl = torch.stack([torch.randint(0, K + 40, (Sq,), generator=g) for K in lens]).to(torch.int32)
    lvl[1, 0] = 0  # an empty row
    d = {**prob.device_inputs("cuda"), "local_visible_lens": lvl.cuda()}
    O, L = host(*call(decoder(prob), d))
    compare(dtype, O, L, *oracle.decode_ex(prob.host_inputs(), local_visible_lens=lvl))


@pytest.mark.parametrize("clusters", [76, 3])
@pytest.mark.parametrize("dtype,P", [("bf16", 64), ("bf16", 8), ("e4m3", 16), ("e4m3", 1024)])
@pytest.mark.parametrize("Sq,causal,window", [(1, False, 300), (2, True, 300), (3, True, 0), (2, False, 5000)])
def test_windows_without_sinks_all_rows(clusters, dtype, P, Sq, causal, window):
    prob = wl.make_problem("uniform", seed=9, H=128, Sq=Sq, causal=causal, window_left=window, dtype=dtype, page_size=P,
                           seq_lens=[2000, 77, 611, 0, 1])
    d = prob.device_inputs("cuda")
    given = give_up_pages(prob, d, 0)
    assert given or P == 1024 or window == 5000
    dec = decoder(prob, clusters)
    out, lse = call(dec, d)
    assert dec.status() == n.MLA_OK
    check(out, lse, reference(prob, 0))


def test_sinks_without_a_window_change_no_bit():
    prob = wl.make_problem("uniform", seed=8, H=128, Sq=2, causal=True, seq_lens=[2000, 77, 600])
    d = prob.device_inputs("cuda")
    a, b = (call(decoder(prob, sink_tokens=s), d) for s in (0, 9))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    compare("bf16", *host(*a), *oracle.decode(prob.host_inputs()))
    assert np.isfinite(host(*a)[0]).all()
