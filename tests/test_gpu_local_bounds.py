"""Decode with per-token local bounds on the GPU: the pages that no token sees are not read, whatever
their entries and bytes are.  Every row against the definition in 64 bits, with the tolerances that
test_gpu_sinks.py derives."""

import pytest
import torch
from test_gpu_sinks import check, give_up_pages, reference

from paged_latent_attention_mla_gb300 import NO_PAGE, decoder_for, merge_ranks
from paged_latent_attention_mla_gb300 import _native as n
from paged_latent_attention_mla_gb300 import build as nbuild
from paged_latent_attention_mla_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

# (heads, clusters, kernels of the call): the short-span kernel, the split-KV kernel with a row in one
# and in several pieces
KERNELS = [(16, 0, 1), (128, 76, 2), (128, 3, 2)]


@pytest.fixture(scope="module", autouse=True)
def built():
    nbuild.build()
    n.load()


def run(prob, d, lvl, sinks, kernels, **options):
    dec = decoder_for(prob, sink_tokens=sinks, **options)
    assert dec.launches_per_call() == kernels
    out, lse = dec(d["q_latent"], d["q_rope"], d["ckv"], d["kpe"], d["page_table"], d["seq_lens"], d["scale"],
                   local_visible_lens=lvl.cuda())
    torch.cuda.synchronize()
    assert dec.status() == n.MLA_OK
    return out, lse


def nan_page(prob, d, page):
    raw, nan = (torch.uint8, 0x7F) if prob.w.dtype == "e4m3" else (torch.int16, 0x7FC0)
    d["ckv"].view(raw)[page] = nan
    d["kpe"].view(raw)[page] = nan


BOUNDS = {
    1: [[2], [4], [64], [448], [500], [1898], [1899], [1900], [1950], [2100], [0]],
    3: [[2, 500, 2], [500, 500, 500], [0, 0, 0], [64, 1950, 3], [1897, 1898, 1899], [448, 448, 4], [1990, 7, 2000]],
}


@pytest.mark.parametrize("H,clusters,kernels", KERNELS)
@pytest.mark.parametrize("dtype,P", [("bf16", 16), ("bf16", 64), ("e4m3", 64), ("bf16", 128)])
@pytest.mark.parametrize("Sq", [1, 3])
@pytest.mark.parametrize("sinks", [4, 0, 300])
def test_bounds_below_the_window_read_no_page_given_up(H, clusters, kernels, dtype, P, Sq, sinks):
    """Tokens whose bound lies at or below the window's floor see sinks or nothing; what lies between the
    sinks and the floor has been given up (no page, or a page outside the pool)."""
    lvl = torch.tensor(BOUNDS[Sq], dtype=torch.int32)
    prob = wl.make_problem("uniform", seed=P + Sq, H=H, Sq=Sq, causal=False, window_left=100, dtype=dtype, page_size=P,
                           seq_lens=[2000] * len(lvl))
    d = prob.device_inputs("cuda")
    assert give_up_pages(prob, d, sinks) > 0
    check(*run(prob, d, lvl, sinks, kernels, num_clusters=clusters), reference(prob, sinks, lvl))


@pytest.mark.parametrize("H,clusters,kernels", KERNELS)
@pytest.mark.parametrize("dtype,P", [("bf16", 8), ("e4m3", 16), ("bf16", 64), ("e4m3", 128)])
@pytest.mark.parametrize("window,sinks", [(-1, 0), (900, 0), (300, 5)])
def test_pages_past_every_bound_hold_any_bits(H, clusters, kernels, dtype, P, window, sinks):
    """Pages below the request's length whose keys no token sees, because they lie past every bound."""
    lvl = torch.tensor([[10, 3], [64, 64], [500, 1], [0, 1], [999, 700], [600, 990]], dtype=torch.int32)
    prob = wl.make_problem("uniform", seed=P + window, H=H, Sq=2, causal=False, window_left=window, dtype=dtype, page_size=P,
                           seq_lens=[1000] * len(lvl))
    d = prob.device_inputs("cuda")
    poisoned = 0
    for b, bounds in enumerate(lvl.tolist()):
        for j in range(-(-max(bounds) // P), -(-1000 // P)):
            nan_page(prob, d, int(d["page_table"][b, j]))
            poisoned += 1
    assert poisoned > 0
    check(*run(prob, d, lvl, sinks, kernels, num_clusters=clusters), reference(prob, sinks, lvl))


@pytest.mark.parametrize("clusters", [0, 76])
@pytest.mark.parametrize("P", [16, 64])
def test_ranks_without_window_keys_read_no_page_given_up(clusters, P):
    """Context parallelism: a short window lies on some ranks only; the others see their sinks."""
    world, inter, window, sinks, lens = 4, 16, 10, 60, [1000, 777]
    prob = wl.make_problem("uniform", seed=404, H=64, Sq=2, causal=True, window_left=window, page_size=P, seq_lens=lens)
    outs, lses, given = [], [], 0
    for r in range(world):
        sh = wl.dcp_shard(prob, world, r, inter, seed=1)
        d = sh.device_inputs("cuda")
        for b, K in enumerate(sh.seq_lens.tolist()):
            at = [(j // inter * world + r) * inter + j % inter for j in range(K)]  # the local keys' positions
            for j in range(-(-K // P)):
                if all(sinks <= g < lens[b] - 2 - window for g in at[j * P : (j + 1) * P]):
                    nan_page(sh, d, int(d["page_table"][b, j]))
                    d["page_table"][b, j] = NO_PAGE
                    given += 1
        dec = decoder_for(sh, sink_tokens=sinks, out_dtype=torch.float32, num_clusters=clusters)
        out, lse = dec(d["q_latent"], d["q_rope"], d["ckv"], d["kpe"], d["page_table"], d["seq_lens"], d["scale"],
                       global_seq_lens=sh.extra["global_seq_lens"].cuda())
        assert dec.status() == n.MLA_OK
        outs.append(out)
        lses.append(lse)
    assert given > 0
    check(*merge_ranks(torch.stack(outs), torch.stack(lses)), reference(prob, sinks))


@pytest.mark.parametrize("window,sinks", [(-1, 0), (60, 3)])
def test_segment_lists_past_shared_memory(window, sinks):
    """600 requests on 2 clusters: more pieces to a cluster than shared memory keeps, each ended by its bound."""
    lens = [40 + (97 * i) % 260 for i in range(600)]
    prob = wl.make_problem("uniform", seed=7, H=128, Sq=1, causal=False, window_left=window, page_size=16, seq_lens=lens)
    lvl = torch.tensor([[1 + (61 * i) % K] for i, K in enumerate(lens)], dtype=torch.int32)
    d = prob.device_inputs("cuda")
    table = d["page_table"].tolist()
    pages = [table[b][j] for b, K in enumerate(lens) for j in range(-(-int(lvl[b, 0]) // 16), -(-K // 16))]
    nan_page(prob, d, torch.tensor(pages, device="cuda"))
    check(*run(prob, d, lvl, sinks, 2, num_clusters=2), reference(prob, sinks, lvl))


@pytest.mark.parametrize("H,clusters,kernels", [(8, 0, 1), (8, 76, 2), (128, 3, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_bounds_of_tokens_that_see_sinks_only_load_nothing(H, clusters, kernels, dtype):
    """A bound past the last key that the other tokens' windows hold, and below its own token's floor."""
    lvl = torch.tensor([[703] + [1] * 14 + [714], [0] * 15 + [715], [707] + [90] * 15], dtype=torch.int32)
    prob = wl.make_problem("uniform", seed=8, H=H, Sq=16, causal=False, window_left=5, dtype=dtype, page_size=8,
                           seq_lens=[721] * 3)  # the floor of token t is 700 + t
    d = prob.device_inputs("cuda")
    for b, first in ((0, 704), (1, 64), (2, 712)):  # request 1 sees its 63 sinks only
        for j in range(first // 8, 91):
            nan_page(prob, d, int(d["page_table"][b, j]))
    check(*run(prob, d, lvl, 63, kernels, num_clusters=clusters), reference(prob, 63, lvl))
